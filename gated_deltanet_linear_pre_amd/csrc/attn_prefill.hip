// attn_prefill.hip -- causal attention of prompts, or of chunks of them, over the
// paged cache.
//
//   o = sum_j w_j V_j / sum_j w_j,  w_j = exp(scale q.K_j - max)   over the keys a token sees
//
// One pass over the keys with the running maximum and sum of the softmax.  The g
// query heads of a key-value head share its keys: a block's 128 rows are g heads of
// 128 / g consecutive tokens, whatever g is, so a short prompt fills its rows too.
// Bound by the matrix pipes and, beside them, by the vector unit's exponentials.
//
// gfx950 mapping.  Wave w of 4 takes rows 32w..32w+31 as the columns of 32 x 32
// matrix products.  S^T = K Q^T puts a key a row and a query a column: maximum and
// sum of a query stay in its two lanes, and the weights of lane (h, c) are keys
// 4 h + 0..3 of every 8, which is at once the operand of O^T = V^T w if V^T is read
// in the same order of keys.  So neither the weights nor O move between lanes.
// Tiles of KT keys go from memory through registers to LDS, one tile ahead and in two
// buffers, one barrier a tile; V^T is read by the transposing LDS reads.
//
// The maximum that the weights are taken against follows the scores only when they
// pass it by 2^8: O and the sum are scaled then, at most a few times a row, and
// weights up to 2^8 lose nothing.
//
// Few rows over many keys (a chunk that goes on from a long cache) would leave most
// CUs idle: the keys are then cut in pieces, a block each, whose sums, maxima and O a
// second kernel joins.
//
// Precision.  Scores, maxima, sums and O are fp32; 16-bit weights are rounded to the
// io type for the product with V (half a step of each weight, of random sign: as much as
// the rounding of the output; a second part would be half of the products again).
//
// In a tile that a row does not see whole hidden scores are -inf, their weights 0.  A
// V that is not finite would turn 0 into NaN there, so it goes to LDS as 0 in such
// a tile, and the rows that see it are made NaN in its channel.
#include "attn_device.h"
#include "mfma_device.h"

namespace gdn {

namespace {

constexpr int BLOCK = 256;
typedef float f16v __attribute__((ext_vector_type(16)));

// Products of W x W values over 8 G deep operands, G = 64 / W lane groups: lane (h, c)
// holds 8 values of row (column) c, and of the result the rows 4 G j + 4 h + 0..3 of
// column c, j < W / (4 G)
template <typename T, int W> struct Mma;
template <typename T> struct Mma<T, 16> {
    typedef f4 acc;
    static __device__ __forceinline__ f4 mma(typename Mat<T>::frag a, typename Mat<T>::frag b, f4 c) { return Mat<T>::mma(a, b, c); }
    // and the sum that its (last) instruction takes
    static __device__ __forceinline__ f4 mma(typename Mat<T>::frag a, typename Mat<T>::frag b, f4 c, f4 &taken)
    {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 7; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
            taken = c;
            return __builtin_amdgcn_mfma_f32_16x16x4f32(a[7], b[7], c, 0, 0, 0);
        } else {
            taken = c;
            return mma(a, b, c);
        }
    }
};
template <> struct Mma<bf16, 32> {
    typedef f16v acc;
    static __device__ __forceinline__ f16v mma(Mat<bf16>::frag a, Mat<bf16>::frag b, f16v c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
};
template <> struct Mma<_Float16, 32> {
    typedef f16v acc;
    static __device__ __forceinline__ f16v mma(Mat<_Float16>::frag a, Mat<_Float16>::frag b, f16v c)
    {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
};
// fp32: eight 2-deep products; product i contracts value i of both lane halves
template <> struct Mma<float, 32> {
    typedef f16v acc;
    static __device__ __forceinline__ f16v mma(Mat<float>::frag a, Mat<float>::frag b, f16v c)
    {
#pragma unroll
        for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], b[i], c, 0, 0, 0);
        return c;
    }
};

#ifndef W_WIDE
#define W_WIDE 16
#endif
#ifndef KT_NARROW
#define KT_NARROW 64
#endif
#ifndef KT_WIDE
#define KT_WIDE 32
#endif
template <typename T, int D> struct Tile {
    static constexpr int W = sizeof(T) == 4 ? 16 : D <= 128 ? 32 : W_WIDE;  // rows of a wave
    static constexpr int G = 64 / W, NA = W * W / 64, ROWS = 4 * W;
    static constexpr int KT = sizeof(T) == 4 ? 32 : D <= 128 ? KT_NARROW : KT_WIDE;  // keys
    static constexpr int NT = KT / W, NC = D / (8 * G), ND = D / W, NK = KT / (8 * G);
    // operands read from LDS ahead of their product.  Their registers are those of a product whose
    // result the product just issued took as its sum: no load is given registers of an operand in use.
    static constexpr int AHEAD = 4;
    static constexpr int V = Vec16<T>::n;
    static constexpr int NV = KT * D / V / BLOCK;  // vectors of K (and of V) a thread moves
    static constexpr int E16 = 16 / sizeof(T);
    static constexpr int KP = D + (W == 32 ? 1 : 2) * E16;  // pitch of K's rows in LDS
    // of V's rows.  16 bits: a transposing read takes 2 W bytes of 4 rows a lane group: an odd multiple of 2 W.
    // fp32: 32 bytes more
    static constexpr int VP = sizeof(T) == 4 ? D + 8 : D / W % 2 ? D : D + W;
    static constexpr int BLOCKS = D <= 128 || (W == 16 && sizeof(T) == 2) ? 2 : 1;  // on a CU
    static_assert(NV * BLOCK * V == KT * D, "whole vectors");
};

struct PrefillArgs {
    AttnArgs a;
    int heads, parts;  // of a key-value head's group that a block takes; parts of the group
    int tokens;   // of a block: rows / heads
    int slots;    // blocks along the tokens
    int pieces;   // of a row's keys, at most
    int piece;    // keys of a piece
    float2 *ml;   // [slot][KV parts][pieces][rows]
    float *o;     // [slot][KV parts][pieces][rows][D]
};

// out = o r, gated, 4 channels
template <typename T>
__device__ __forceinline__ void finish(const AttnDims &d, const AttnArgs &a, int64_t row, int head, int col, f4 o, float r)
{
    typedef T t4 __attribute__((ext_vector_type(4)));
    t4 y;
    if (a.gate) {
        const t4 gate = *reinterpret_cast<const t4 *>(static_cast<const T *>(a.gate) + row * d.gate_stride + head * d.D + col);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = (T)(o[i] * r / (1.0f + expf(-(float)gate[i])));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = (T)(o[i] * r);
    }
    *reinterpret_cast<t4 *>(static_cast<T *>(a.out) + (row * d.H + head) * d.D + col) = y;
}
// 1 / sum of weights; no key: o and the sum are 0 (a NaN stays one)
__device__ __forceinline__ float inverse_sum(float l) { return l > 0.f ? 1.0f / l : l; }

// over the G lanes of a column
template <int G>
__device__ __forceinline__ float column_max(float x)
{
    if (G == 4) return max_of_groups(x);
    const unsigned u = __float_as_uint(x);
    const auto h = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return fmaxf(__uint_as_float(h[0]), __uint_as_float(h[1]));
}
template <int G>
__device__ __forceinline__ float column_sum(float x)
{
    if (G == 4) x += __shfl_xor(x, 16, 64);
    return x + __shfl_xor(x, 32, 64);
}

// A block's tokens and keys
struct Work {
    int n, tokens;        // sequence; tokens of the block that are there
    int64_t row;          // first token's row
    int p0;               // its position
    int begin, end;       // keys that the rows see (begin: on a tile)
};
template <int KT>
__device__ __forceinline__ bool locate(const AttnDims &d, const PrefillArgs &s, int slot, Work &b)
{
    SeqTile st;
    if (!find_tile(s.a.cu, d.n_seq, d.T, s.tokens, slot, st)) return false;
    const int len = st.end - st.begin, first = st.c * s.tokens;
    if (first >= len) return false;
    b.n = st.n;
    b.tokens = len - first < s.tokens ? len - first : s.tokens;
    b.row = st.begin + first;
    const int kv = kv_bound(d, s.a.kv_len, st.n);
    b.p0 = kv - len + first;
    b.end = b.p0 + b.tokens > 0 ? b.p0 + b.tokens : 0;
    b.begin = first_key(d, b.p0) / KT * KT;
    return true;
}

// V^T: channel W t + c, keys 8 G k + 4 h + 0..3 and 4 G more
template <typename T, int W, int VP>
__device__ __forceinline__ typename Mat<T>::frag column(const T *v, int k, int t, int lane)
{
    constexpr int G = 64 / W;
    if constexpr (sizeof(T) == 4) {
        const T *p = v + (8 * G * k + 4 * (lane / W)) * VP + W * t + (lane & (W - 1));
        typename Mat<T>::frag f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = p[i * VP];
            f[i + 4] = p[(i + 4 * G) * VP];
        }
        return f;
    } else {
        typedef short s4 __attribute__((ext_vector_type(4)));
        typedef short s8 __attribute__((ext_vector_type(8)));
        typedef __attribute__((address_space(3))) s4 lds_s4;
        const T *p = v + (8 * G * k + 4 * (lane / W) + ((lane & 15) >> 2)) * VP + W * t + 16 * ((lane >> 4) & (W / 16 - 1)) + 4 * (lane & 3);
        const s4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)(p));
        const s4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)(p + 4 * G * VP));
        return __builtin_bit_cast(typename Mat<T>::frag, (s8)__builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
}

// Keeps an operand's registers from being given away before this point
template <typename F>
__device__ __forceinline__ void in_use(const F &f)
{
#ifdef __HIP_DEVICE_COMPILE__  // (the host's pass does not know the constraint)
    __asm__ volatile("" ::"v"(f));
#endif
}
// (the last of an fp32 product's eight instructions takes value 7)
template <typename T>
__device__ __forceinline__ void operand_in_use(const typename Mat<T>::frag &f)
{
    if constexpr (sizeof(T) == 4) in_use((float)f[7]);
    else in_use(f);
}

template <typename T>
__device__ __forceinline__ bool not_finite(T x) { return !(fabsf((float)x) <= 3.402823466e38f); }

template <typename T, int D>
__global__ __launch_bounds__(BLOCK, (Tile<T, D>::BLOCKS)) void prefill_kernel(AttnDims d, PrefillArgs s)
{
    typedef Tile<T, D> TL;
    typedef typename Mat<T>::frag frag;
    typedef typename Vec16<T>::type vec;
    typedef Mma<T, TL::W> MM;
    typedef typename MM::acc acc;
    constexpr int W = TL::W, G = TL::G, NA = TL::NA, UNITS = NA / 4;
    constexpr int KT = TL::KT, NT = TL::NT, NC = TL::NC, ND = TL::ND, NK = TL::NK, NV = TL::NV, V = TL::V;
    __shared__ __attribute__((aligned(16))) T sk[2][KT * TL::KP];
    __shared__ __attribute__((aligned(16))) T sv[2][KT * TL::VP];
    // of a tile that some row does not see whole: values of V that are not finite (0 in sv), a bit each,
    // and whether a wave met one
    __shared__ unsigned char s_bits[2][KT * D / V];
    __shared__ int s_bad[2][BLOCK / 64];
    const int tid = threadIdx.x, lane = tid & 63, h = lane / W, c = lane & (W - 1);
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int slot = s.slots - 1 - blockIdx.x;  // (the rows with the most keys first)
    const int kh = blockIdx.y / s.parts, head0 = kh * d.g + (blockIdx.y - kh * s.parts) * s.heads;
    const int g = (kh + 1) * d.g - head0 < s.heads ? (kh + 1) * d.g - head0 : s.heads;

    Work b;
    if (!locate<KT>(d, s, slot, b)) return;
    const int begin = b.begin + blockIdx.z * s.piece;
    if (blockIdx.z > 0 && begin >= b.end) return;
    const int end = b.end - begin > s.piece ? begin + s.piece : b.end;
    const bool whole = blockIdx.z == 0 && end == b.end;

    // ---- this lane's query: column c of the products ----
    const int r = W * w + c;
    const int used = b.tokens * g;
    const int rr = r < used ? r : used - 1;  // (rows that are not there follow the last one, and are not written)
    const int tok = rr / g, head = head0 + rr - tok * g;
    const int p = b.p0 + tok, low = first_key(d, p);
    // of the wave: the rows' first and last positions
    const int wr = W * w < used ? W * w : used - 1, wl = W * w + W - 1 < used ? W * w + W - 1 : used - 1;
    const int pw0 = b.p0 + wr / g, pw1 = b.p0 + wl / g;
    const bool busy = W * w < used;
    const int low_last = first_key(d, b.p0 + b.tokens - 1);
    frag qf[NC];
    {
        const T *q = static_cast<const T *>(s.a.q) + (b.row + tok) * d.q_stride + (int64_t)head * D + 8 * h;
#pragma unroll
        for (int i = 0; i < NC; ++i) qf[i] = *reinterpret_cast<const typename Frag16<T>::type *>(q + 8 * G * i);
    }
    acc o[ND];
#pragma unroll
    for (int t = 0; t < ND; ++t) o[t] = acc(0.f);
    float m = -INFINITY, l = 0.f;
    unsigned dead[(ND * NA + 31) / 32] = {};  // values of o that a V that is not finite has reached
    const float cs = d.scale * 1.44269504f;

    auto cut = [&](int k0) { return k0 + KT - 1 > b.p0 || k0 < low_last; };  // a row may not see all of a tile

    // ---- tiles from memory ----
    const int32_t *table = s.a.table + (int64_t)b.n * d.table_pages;
    // Vector i of a wave's 64 lanes lies in 16 consecutive rows (whole lines of D / V vectors
    // never straddle 16 rows there), so in one page: its number and base are scalars.
    const int64_t head_at = (int64_t)kh * d.page * D;
    const T *K = static_cast<const T *>(s.a.k_cache) + head_at, *Vc = static_cast<const T *>(s.a.v_cache) + head_at;
    vec rk[NV], rv[NV];
    int page[NV];
    constexpr int LINE = D / V;
    static_assert(16 * LINE % 64 == 0, "16 rows are whole vectors of a wave");
    constexpr bool even = BLOCK % LINE == 0;  // the same channel for every i
    const int row0 = tid / LINE, col0 = (tid - row0 * LINE) * V;
    auto row_of = [&](int i) { return even ? row0 + i * (BLOCK / LINE) : (i * BLOCK + tid) / LINE; };
    auto col_of = [&](int i) { return even ? col0 : (i * BLOCK + tid - row_of(i) * LINE) * V; };
    const int last = end - 1;
    auto ask = [&](int k0) {  // the pages of a tile (behind the end: of the last key)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int key = k0 + (i * BLOCK + w * 64) / LINE;
            page[i] = table[(unsigned)(key < end ? key : last) >> d.log_page];
        }
    };
    auto load = [&](int k0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t at = page_bound(d, __builtin_amdgcn_readfirstlane(page[i])) * d.page_stride;
            int key = k0 + row_of(i);
            key = key < end ? key : last;
            const unsigned in = (unsigned)(key & (d.page - 1)) * D + col_of(i);
            rk[i] = ld16_at(K + at, in * (unsigned)sizeof(T));
            rv[i] = ld16_at(Vc + at, in * (unsigned)sizeof(T));
        }
    };
    auto store = [&](int k0, int buf) {
        if (cut(k0)) {
            const bool tail = k0 + KT > end;
            bool bad = false;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (tail && k0 + row_of(i) >= end) rv[i] = vec(0);  // whatever the cache holds there
                unsigned bits = 0;
#pragma unroll
                for (int j = 0; j < V; ++j) bits |= (unsigned)not_finite(rv[i][j]) << j;
                if (bits) {
#pragma unroll
                    for (int j = 0; j < V; ++j) rv[i][j] = bits >> j & 1 ? T(0.f) : rv[i][j];
                }
                bad |= bits != 0;
                s_bits[buf][i * BLOCK + tid] = (unsigned char)bits;
            }
            const bool any = __any(bad);
            if (lane == 0) s_bad[buf][w] = any;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            st16(&sk[buf][row_of(i) * TL::KP + col_of(i)], rk[i]);
            st16(&sv[buf][row_of(i) * TL::VP + col_of(i)], rv[i]);
        }
    };
    if (begin < end) {
        // (behind the end the last row again and again: a branch would keep the old values beside the new)
        ask(begin);
        load(begin);
        ask(begin + KT);
        store(begin, 0);
        load(begin + KT);
        ask(begin + 2 * KT);
    }
    lds_sync();

    int buf = 0;
    for (int k0 = begin; k0 < end; k0 += KT, buf ^= 1) {
        const bool mine = busy && k0 <= pw1 && k0 + KT > first_key(d, pw0);
        acc sc[NT];
        bool masked = false;
        if (mine) {
#pragma unroll
            for (int t = 0; t < NT; ++t) sc[t] = acc(0.f);
            // product u: chunk u / NT of the channels, keys W (u % NT)..
            auto key_rows = [&](int u) {
                return *reinterpret_cast<const typename Frag16<T>::type *>(&sk[buf][(W * (u % NT) + c) * TL::KP + 8 * G * (u / NT) + 8 * h]);
            };
            constexpr int R = NT + TL::AHEAD;
            frag kf[R];
            acc taken[NT];  // (16 x 16: the sum is not updated in place)
#pragma unroll
            for (int u = 0; u < TL::AHEAD; ++u) kf[u] = key_rows(u);
#pragma unroll
            for (int u = 0; u < NC * NT; ++u) {
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (W == 16) sc[u % NT] = MM::mma(kf[u % R], qf[u / NT], sc[u % NT], taken[u % NT]);
                else sc[u % NT] = MM::mma(kf[u % R], qf[u / NT], sc[u % NT]);
                __builtin_amdgcn_sched_barrier(0);
                constexpr int LAST = NC * NT - TL::AHEAD - 1;  // of the steps that load
                if (u <= LAST) kf[(u + TL::AHEAD) % R] = key_rows(u + TL::AHEAD);
#pragma unroll
                for (int v = 0; v <= u; ++v)  // operands of sums that no product has taken yet
                    if (v == u - NT + 1 || (u == LAST && v > u - NT)) operand_in_use<T>(kf[v % R]);
                if (W == 16) {
#pragma unroll
                    for (int t = 0; t < NT && t <= u; ++t) in_use(taken[t]);
                }
            }
            masked = k0 + KT - 1 > pw0 || k0 < first_key(d, pw1);
            if (masked) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int i = 0; i < NA; ++i) {
                        const int key = k0 + W * t + 4 * G * (i >> 2) + 4 * h + (i & 3);
                        sc[t][i] = key <= p && key >= low ? sc[t][i] : -INFINITY;
                    }
            }
            float most = -INFINITY;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < NA; ++i) most = fmaxf(most, sc[t][i]);
            most = column_max<G>(most) * cs;
            if (__any(most > m + 8.f)) {
                const float m1 = fmaxf(m, most), keep = __builtin_amdgcn_exp2f(m - (m1 == -INFINITY ? 0.f : m1));
                m = m1;
                l *= keep;
#pragma unroll
                for (int t = 0; t < ND; ++t) o[t] *= keep;
            }
            if (cut(k0) && (s_bad[buf][0] | s_bad[buf][1] | s_bad[buf][2] | s_bad[buf][3])) {  // (rare: no care for its time)
                for (int j = 0; j < KT; ++j) {
                    const bool sees = k0 + j <= p && k0 + j >= low && k0 + j < end;
#pragma unroll
                    for (int t = 0; t < ND; ++t)
#pragma unroll
                        for (int i = 0; i < UNITS; ++i) {
                            const int ch = W * t + 4 * G * i + 4 * h;
                            const unsigned bits = sees ? s_bits[buf][(j * D + ch) / V] >> (ch % V) & 15 : 0;
                            dead[(t * NA + 4 * i) / 32] |= bits << (t * NA + 4 * i) % 32;
                            __builtin_amdgcn_sched_barrier(0);
                        }
                }
            }
        }
        // the next tile goes to the other buffer, the one after it is asked for
        __builtin_amdgcn_sched_barrier(0);
        store(k0 + KT, buf ^ 1);
        load(k0 + 2 * KT);
        ask(k0 + 3 * KT);
        if (mine) {
            // product u: channels W (u % ND).., keys 8 G (u / ND)..
            auto channels = [&](int u) { return column<T, W, TL::VP>(sv[buf], u / ND, u % ND, lane); };
            constexpr int R = ND + TL::AHEAD;
            frag vf[R];
            acc held[ND];
#pragma unroll
            for (int u = 0; u < TL::AHEAD; ++u) vf[u] = channels(u);
            const float m0 = m == -INFINITY ? 0.f : m;
            frag pf[NK];
#pragma unroll
            for (int k = 0; k < NK; ++k) {
                float wt[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int at = 2 * k + (i >> 2);  // in units of 4 G keys
                    wt[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[at / UNITS][at % UNITS * 4 + (i & 3)], cs, -m0));
                    l += wt[i];
                }
                frag one[1];
                split8<T, 1>(wt, one);
                pf[k] = one[0];
                __builtin_amdgcn_sched_barrier(0);  // (or all the weights live at once)
            }
#pragma unroll
            for (int u = 0; u < NK * ND; ++u) {
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (sizeof(T) == 4) o[u % ND] = MM::mma(vf[u % R], pf[u / ND], o[u % ND], held[u % ND]);
                else o[u % ND] = MM::mma(vf[u % R], pf[u / ND], o[u % ND]);
                __builtin_amdgcn_sched_barrier(0);
                constexpr int LAST = NK * ND - TL::AHEAD - 1;
                if (u <= LAST) vf[(u + TL::AHEAD) % R] = channels(u + TL::AHEAD);
#pragma unroll
                for (int v = 0; v <= u; ++v)
                    if (v == u - ND + 1 || (u == LAST && v > u - ND)) operand_in_use<T>(vf[v % R]);
                if (sizeof(T) == 4 && u <= LAST) {
#pragma unroll
                    for (int t = 0; t < ND && t <= u; ++t) in_use(held[t]);
                }
            }
#pragma unroll
            for (int k = 0; k < NK; ++k) operand_in_use<T>(pf[k]);
        }
        lds_sync();
    }

    l = column_sum<G>(l);
    if (r >= used) return;
#pragma unroll
    for (int t = 0; t < ND; ++t)
#pragma unroll
        for (int i = 0; i < NA; ++i) o[t][i] = dead[(t * NA + i) / 32] >> (t * NA + i) % 32 & 1 ? NAN : o[t][i];
    if (whole) {
        const float inv = inverse_sum(l);
#pragma unroll
        for (int t = 0; t < ND; ++t)
#pragma unroll
            for (int i = 0; i < UNITS; ++i) {
                const f4 x = {o[t][4 * i], o[t][4 * i + 1], o[t][4 * i + 2], o[t][4 * i + 3]};
                finish<T>(d, s.a, b.row + tok, head, W * t + 4 * G * i + 4 * h, x, inv);
            }
    } else {
        const int64_t at = (((int64_t)slot * gridDim.y + blockIdx.y) * s.pieces + blockIdx.z) * TL::ROWS + r;
        if (h == 0) s.ml[at] = make_float2(m, l);
#pragma unroll
        for (int t = 0; t < ND; ++t)
#pragma unroll
            for (int i = 0; i < UNITS; ++i) {
                const f4 x = {o[t][4 * i], o[t][4 * i + 1], o[t][4 * i + 2], o[t][4 * i + 3]};
                *reinterpret_cast<f4 *>(s.o + at * D + W * t + 4 * G * i + 4 * h) = x;
            }
    }
}

// The rows whose keys were cut: a thread 4 channels of a row
template <typename T, int D>
__global__ __launch_bounds__(BLOCK) void join_kernel(AttnDims d, PrefillArgs s)
{
    constexpr int LANES = D / 4, KT = Tile<T, D>::KT, ROWS = Tile<T, D>::ROWS;
    const int slot = blockIdx.x;
    const int kh = blockIdx.y / s.parts, head0 = kh * d.g + (blockIdx.y - kh * s.parts) * s.heads;
    const int g = (kh + 1) * d.g - head0 < s.heads ? (kh + 1) * d.g - head0 : s.heads;
    Work b;
    if (!locate<KT>(d, s, slot, b)) return;
    const int n = (b.end - b.begin + s.piece - 1) / s.piece;
    if (n <= 1) return;
    const int i = blockIdx.z * BLOCK + threadIdx.x, r = i / LANES, col = (i - r * LANES) * 4;
    if (r >= b.tokens * g) return;
    const int64_t at = ((int64_t)slot * gridDim.y + blockIdx.y) * s.pieces * ROWS + r;
    float big = -INFINITY;
    for (int u = 0; u < n; ++u) big = fmaxf(big, s.ml[at + (int64_t)u * ROWS].x);
    const float big0 = big == -INFINITY ? 0.f : big;
    float l = 0.f;
    f4 sum = f4(0.f);
#pragma unroll 4
    for (int u = 0; u < n; ++u) {
        const float2 x = s.ml[at + (int64_t)u * ROWS];
        const float f = __builtin_amdgcn_exp2f(x.x - big0);
        l += f * x.y;
        sum += f * *reinterpret_cast<const f4 *>(s.o + (at + (int64_t)u * ROWS) * D + col);
    }
    const int tok = r / g;
    finish<T>(d, s.a, b.row + tok, head0 + r - tok * g, col, sum, inverse_sum(l));
}

// Keys are cut where a launch would have less than 512 blocks (two a CU), into
// pieces of 512 at least.
struct Plan {
    int heads, parts, tokens, slots, pieces, piece;
    size_t ml, o;
};
Plan plan_of(const AttnDims &d, int rows)
{
    Plan p;
    p.heads = d.g < rows ? d.g : rows;
    p.parts = (d.g + p.heads - 1) / p.heads;
    p.tokens = rows / p.heads;
    p.slots = (int)(d.T / p.tokens) + d.n_seq;
    const int64_t blocks = (int64_t)p.slots * d.KV * p.parts;
    int64_t span = d.max_kv;
    if (d.window < span) span = (int64_t)d.window + p.tokens + 64 < span ? (int64_t)d.window + p.tokens + 64 : span;
    int64_t piece = span * blocks / 512;
    piece = (piece < 512 ? 512 : piece) / 64 * 64 + 64;
    p.pieces = blocks >= 512 || span <= piece ? 1 : (int)((span + 64 + piece - 1) / piece);
    p.piece = p.pieces == 1 ? INT32_MAX / 2 : (int)piece;
    const size_t cut = p.pieces == 1 ? 0 : (size_t)blocks * p.pieces * rows;
    p.ml = (cut * sizeof(float2) + 255) / 256 * 256;
    p.o = cut * d.D * sizeof(float);
    return p;
}

template <typename T, int D>
void launch_prefill_t(const AttnDims &d, const AttnArgs &a, hipStream_t st)
{
    constexpr int ROWS = Tile<T, D>::ROWS;
    const Plan p = plan_of(d, ROWS);
    const PrefillArgs s{a, p.heads, p.parts, p.tokens, p.slots, p.pieces, p.piece, static_cast<float2 *>(a.ws),
                        reinterpret_cast<float *>(static_cast<char *>(a.ws) + p.ml)};
    hipLaunchKernelGGL((prefill_kernel<T, D>), dim3(s.slots, d.KV * s.parts, s.pieces), dim3(BLOCK), 0, st, d, s);
    if (s.pieces > 1)
        hipLaunchKernelGGL((join_kernel<T, D>), dim3(s.slots, d.KV * s.parts, ROWS * (D / 4) / BLOCK), dim3(BLOCK), 0, st, d, s);
}

#define GDN_ATTN_D(...)                                    \
    switch (s.head_dim) {                                  \
    case 64: { constexpr int D = 64; __VA_ARGS__ } break;  \
    case 96: { constexpr int D = 96; __VA_ARGS__ } break;  \
    case 128: { constexpr int D = 128; __VA_ARGS__ } break; \
    case 192: { constexpr int D = 192; __VA_ARGS__ } break; \
    default: { constexpr int D = 256; __VA_ARGS__ } break; \
    }

} // namespace

size_t attn_prefill_workspace_bytes(const gdn_attn_shape &s)
{
    int rows = 0;
    GDN_SSM_IO(s.io_dtype, GDN_ATTN_D(rows = Tile<TI, D>::ROWS;))
    const Plan p = plan_of(attn_dims(s), rows);
    return p.ml + p.o;
}

hipError_t launch_attn_prefill(const gdn_attn_shape &s, const AttnArgs &a, hipStream_t st)
{
    const AttnDims d = attn_dims(s);
    GDN_SSM_IO(s.io_dtype, GDN_ATTN_D(launch_prefill_t<TI, D>(d, a, st);))
    return hipGetLastError();
}

} // namespace gdn
