// attn_prefill.hip -- causal attention of prompts, or of chunks of them, over the
// paged cache.
//
//   o = sum_j w_j V_j / sum_j w_j,  w_j = exp(scale q.K_j - max)   over the keys a token sees
//
// One pass over the keys with the running maximum and sum of the softmax.  The g
// query heads of a key-value head share its keys: a block's rows (128; 64 for fp32) are g heads
// of as many consecutive tokens as fit, whatever g is, so a short prompt fills its rows
// too.  Bound by what a wave can issue between its products: matrix instructions, their
// LDS reads and the softmax.
//
// gfx950 mapping.  A wave takes W rows (32; 16 where a head is wide) as the columns of
// W x W matrix products.  S^T = K Q^T puts a key a row and a query a column: maximum and sum of a
// query stay in its lanes, and the weights of lane (h, c) are 4 consecutive keys of
// every 4 G, which is at once the operand of O^T = V^T w if V^T is read in the same order
// of keys.  So neither the weights nor O move between lanes.  Tiles of KT keys go from memory to LDS
// directly, one tile ahead, in two buffers, one barrier a tile, their copies spread over the
// products; V^T is read by the transposing LDS reads.  8 waves share a tile at D = 256, where
// 4 would spend 40% of the time on the copies (through registers: 8192 tokens of 16 heads 0.77 ms,
// copied by 4 waves 0.69, by 8 0.67, spread 0.64).
//
// The maximum that the weights are taken against follows the scores only when they
// pass it by 2^8: O and the sum are scaled then, at most a few times a row, and
// weights up to 2^8 lose nothing.
//
// Few rows over many keys (a chunk that goes on from a long cache) would leave most CUs idle.
// The keys of all rows then form one line that is cut into equal parts, one a block, as in the
// step: rows within one part are finished there, of rows that are cut each part leaves O, maximum
// and sum in the workspace, and a second kernel joins them.  Whether that pays is said by line_us(), first
// by the bounds that the host knows, then by the lengths on the device.
//
// Precision.  Scores, maxima, sums and O are fp32; 16-bit weights are rounded to the
// io type for the product with V (half a step of each weight, of random sign: as much as
// the rounding of the output; a second part would be half of the products again).
//
// In a tile that a row does not see whole hidden scores are -inf, their weights 0.  A
// V that is not finite would turn 0 into NaN there, so it is made 0 in LDS in such
// a tile, and the rows that see it become NaN in its channel at the end.
//
// Measured: 2048 tokens of 32 heads of 128, fp16, 56 us (619 TFLOP/s of what the mask leaves), 8192
// tokens 0.59 ms (930); 8192 tokens of 16 heads of 256, bf16, 0.63 ms (875); chunks of
// 391 tokens over caches of up to 32768 keys 219 us (726).  fp32, 4096 tokens: 32 heads of 128 1.14 ms (120), 16
// of 256 1.33 (103).
#include "attn_device.h"
#include "mfma_device.h"

namespace gdn {

namespace {

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

template <typename T, int D> struct Tile {
    static constexpr int W = sizeof(T) == 4 || D > 128 ? 16 : 32;  // rows of a wave
    // Waves that share a tile, and blocks on a CU: 8 waves of 256 registers; fp32 of wide heads, whose queries alone
    // take up to 64, 4 of 512
    static constexpr bool big = sizeof(T) == 4 && D > 128;
    static constexpr int WAVES = D > 128 && !big ? 8 : 4, BLOCK = 64 * WAVES, BLOCKS = D > 128 ? 1 : 2;
    static constexpr int G = 64 / W, NA = W * W / 64, ROWS = WAVES * W;
    static constexpr int KT = sizeof(T) == 4 || D == 256 ? 32 : 64;  // keys
    static constexpr int NT = KT / W, NC = D / (8 * G), ND = D / W, NK = KT / (8 * G);
    // operands read from LDS ahead of their product.  Their registers are those of a product whose
    // result the product just issued took as its sum: no load is given registers of an operand in use.
    static constexpr int AHEAD = sizeof(T) == 4 ? 2 : D == 96 ? 3 : 4;
    static constexpr int V = Vec16<T>::n, LINE = D / V;  // values of a vector of 16 bytes, vectors of a row
    static constexpr int NV = KT * LINE / BLOCK;         // vectors of K (and of V) a thread moves
    static_assert(NV * BLOCK == KT * LINE, "whole vectors");
    static_assert(16 * LINE % 64 == 0, "16 rows are whole vectors of a wave");

    // Rows lie in LDS without gaps; vector x of a row stands at place x ^ swap of its row, which lets a read
    // meet every bank once.  FOLD: rows (of 4 banks a vector, 64 in all) until the banks repeat.
    static constexpr int FOLD = LINE % 16 == 0 ? 1 : LINE % 8 == 0 ? 2 : 4;
    // K: 16 rows of one vector
    static __device__ __forceinline__ int swap_k(int row) { return (row / FOLD) & (16 / FOLD - 1); }
    // V: 16 bits, 2 W bytes (UNIT vectors) of 16 / UNIT rows; fp32, 4 vectors of rows that are 4 apart
    static constexpr int UNIT = sizeof(T) == 4 ? 4 : W / 8, APART = sizeof(T) == 4 ? 4 : 1;
    static constexpr int SHIFT = FOLD > APART ? FOLD : APART, KINDS = 16 / UNIT / FOLD > 0 ? 16 / UNIT / FOLD : 1;
    static __device__ __forceinline__ int swap_v(int row) { return (row / SHIFT) % KINDS * UNIT; }
    static_assert(LINE % (16 / FOLD) == 0 && LINE % (KINDS * UNIT) == 0, "vectors change places within a row");
};

struct PrefillArgs {
    AttnArgs a;
    int heads, parts;  // of a key-value head's group that a block takes; parts of the group
    int tokens;        // of a block: rows / heads
    int slots;         // blocks along the tokens
    bool paired;       // the blocks that have rows are all resident at once
    int line;          // blocks among which all keys are dealt in equal parts; 0: a block takes its rows' keys
    unsigned worth;    // so many keys fewer in the longest part are worth what it costs
    // of the line's parts
    struct Cut *cut;      // [slots][key-value heads and parts of their groups]
    float2 *ml;           // [2 line][rows] maximum (of scores times scale log2 e) and sum of weights
    f4 *o;                // [2 line][wave][4 channels of a row, as a lane holds them][lane]
};

// Keys that rows are cut at, and the longest line of slots
constexpr int CHUNK = 128, MOST_SLOTS = 512;

// Rows of a slot and the heads hy of it, whose keys are cut: where their tokens begin and how many they are, the
// part that the keys begin in, and how many parts have a piece (0: they are not cut)
struct Cut {
    int row, tokens, first, pieces;
};

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
// from the sequence, the tokens' first row and number, and the first one's position
template <int KT>
__device__ __forceinline__ Work work_of(const AttnDims &d, int n, int row, int tokens, int p0)
{
    Work b;
    b.n = n;
    b.tokens = tokens;
    b.row = row;
    b.p0 = p0;
    b.end = p0 + tokens > 0 ? p0 + tokens : 0;
    b.begin = first_key(d, p0) / KT * KT;
    return b;
}
template <int KT>
__device__ __forceinline__ bool locate(const AttnDims &d, const PrefillArgs &s, int slot, Work &b)
{
    SeqTile st;
    if (!find_tile(s.a.cu, d.n_seq, d.T, s.tokens, slot, st)) return false;
    const int len = st.end - st.begin, first = st.c * s.tokens;
    if (first >= len) return false;
    b = work_of<KT>(d, st.n, st.begin + first, len - first < s.tokens ? len - first : s.tokens, kv_bound(d, s.a.kv_len, st.n) - len + first);
    return true;
}

// V^T: channel W t + c, keys 8 G k + 4 h + 0..3 and 4 G more
template <typename T, int D>
__device__ __forceinline__ typename Mat<T>::frag column(const T *v, int k, int t, int lane)
{
    typedef Tile<T, D> TL;
    constexpr int G = TL::G, W = TL::W, V = TL::V;
    if constexpr (sizeof(T) == 4) {
        // (the rows 8 G k.. are whole periods of the places, and the four rows of a lane share theirs)
        static_assert(TL::SHIFT >= 4 && 4 * G % (TL::SHIFT * TL::KINDS) == 0, "one address for all rows");
        typename Mat<T>::frag f;
        const int row = 4 * (lane / W), ch = W * t + (lane & (W - 1));
        const T *p = v + (8 * G * k + row) * D + ((ch / V) ^ TL::swap_v(row)) * V + ch % V;
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = p[((i & 3) + (i >> 2) * 4 * G) * D];
        return f;
    } else {
        typedef short s4 __attribute__((ext_vector_type(4)));
        typedef short s8 __attribute__((ext_vector_type(8)));
        typedef __attribute__((address_space(3))) s4 lds_s4;
        // (the second read's row is 4 G further, which changes no vector's place)
        static_assert(4 * G % (TL::SHIFT * TL::KINDS) == 0, "one address for both reads");
        const int row = 4 * (lane / W) + ((lane & 15) >> 2), ch = W * t + 16 * ((lane >> 4) & (W / 16 - 1)) + 4 * (lane & 3);
        const T *p = v + (8 * G * k + row) * D + ((ch / V) ^ TL::swap_v(row)) * V + ch % V;
        const s4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)(p));
        const s4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)(p + 4 * G * D));
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

template <typename T, int D, bool LINED>
__global__ __launch_bounds__((Tile<T, D>::BLOCK), (Tile<T, D>::BLOCKS)) void prefill_kernel(AttnDims d, PrefillArgs s)
{
    typedef Tile<T, D> TL;
    typedef typename Mat<T>::frag frag;
    typedef typename Vec16<T>::type vec;
    typedef Mma<T, TL::W> MM;
    typedef typename MM::acc acc;
    constexpr int W = TL::W, G = TL::G, NA = TL::NA, UNITS = NA / 4;
    constexpr int BLOCK = TL::BLOCK, LINE = TL::LINE;
    constexpr int KT = TL::KT, NT = TL::NT, NC = TL::NC, ND = TL::ND, NK = TL::NK, NV = TL::NV, V = TL::V;
    __shared__ __attribute__((aligned(1024))) T sk[2][KT * D];
    __shared__ __attribute__((aligned(1024))) T sv[2][KT * D];
    // of a tile that some row does not see whole: values of V that are not finite (0 in sv), a bit each,
    // and whether a wave met one
    __shared__ unsigned char s_bits[2][KT * LINE];
    __shared__ int s_bad[2][TL::WAVES];
    const int w = scalar(threadIdx.x >> 6);
    const int heads = d.KV * s.parts;

    // ---- this block's rows, or its part of the line ----
    __shared__ unsigned s_pre[LINED ? MOST_SLOTS + 1 : 1], s_sum[TL::WAVES], s_most[TL::WAVES];
    __shared__ int4 s_work[LINED ? MOST_SLOTS : 1];  // a slot's sequence, row, tokens, position
    int slot = 0, hy = 0;
    unsigned pos = 0, stop = 1, quantum = 0;
    __shared__ unsigned s_next[2];  // other rows' keys, which a block takes after these: lower in the line (or none)
    if constexpr (LINED) {
        const int tid = threadIdx.x, lane = tid & 63;
        const int per = (s.slots + BLOCK - 1) / BLOCK;
        unsigned mine = 0, most = 0;
        for (int i = tid * per; i < s.slots && i < (tid + 1) * per; ++i) {
            Work b;
            const bool in = locate<KT>(d, s, i, b);
            s_pre[i] = !in ? 0 : b.end - b.begin <= CHUNK ? 1 : (b.end - b.begin + CHUNK - 1) / CHUNK;
            if (in) s_work[i] = make_int4(b.n, (int)b.row, b.tokens, b.p0);
            if (!in && blockIdx.x == 0)
                for (int k = 0; k < heads; ++k) s.cut[i * heads + k].pieces = 0;
            mine += s_pre[i];
            most = most > s_pre[i] ? most : s_pre[i];
        }
        unsigned upto = mine;
#pragma unroll
        for (int u = 1; u < 64; u <<= 1) {
            const unsigned x = __shfl_up(upto, u, 64);
            if (lane >= u) upto += x;
            const unsigned y = __shfl_xor(most, u, 64);
            most = most > y ? most : y;
        }
        if (lane == 63) {
            s_sum[w] = upto;
            s_most[w] = most;
        }
        __syncthreads();
        unsigned total = 0;
#pragma unroll
        for (int i = 0; i < TL::WAVES; ++i) {
            most = most > s_most[i] ? most : s_most[i];
            if (i < w) upto += s_sum[i];
            total += s_sum[i];
        }
        unsigned at = upto - mine;
        for (int i = tid * per; i < s.slots && i < (tid + 1) * per; ++i) {
            const unsigned n = s_pre[i];
            s_pre[i] = at;
            at += n;
        }
        if (tid == 0) s_pre[s.slots] = total;
        __syncthreads();
        total = __builtin_amdgcn_readfirstlane(total * heads);
        quantum = scalar(total / gridDim.x + (total % gridDim.x != 0));
        // Not dealt, a block takes its rows' keys; where there are more rows than blocks, the last ones first, and the
        // blocks that have the fewest keys then take second rows.
        const int blocks = gridDim.x, all = s.slots * heads, extra = all > blocks ? all - blocks : 0;
        auto first_of = [&](int i) { return extra ? all - 1 - i : i; };
        auto second_of = [&](int i) { return i - (blocks - extra); };  // (below 0: none)
        if (extra) {  // the longest of two rows
            most = 0;
            for (int i = tid; i < blocks; i += BLOCK) {
                const int one = first_of(i) / heads, two = second_of(i) / heads;
                const unsigned n = s_pre[one + 1] - s_pre[one] + (second_of(i) < 0 ? 0 : s_pre[two + 1] - s_pre[two]);
                most = most > n ? most : n;
            }
#pragma unroll
            for (int u = 1; u < 64; u <<= 1) {
                const unsigned y = __shfl_xor(most, u, 64);
                most = most > y ? most : y;
            }
            if (lane == 0) s_most[w] = most;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < TL::WAVES; ++i) most = most > s_most[i] ? most : s_most[i];
        }
        most = scalar(most);
        unsigned next = 0, next_stop = 0xffffffff;
        if (most > quantum && (uint64_t)(most - quantum) * CHUNK > s.worth) {
            const uint64_t from = (uint64_t)blockIdx.x * quantum;
            pos = from < total ? (unsigned)from : total;
            stop = total - pos < quantum ? total : pos + quantum;
        } else {  // not worth its cost
            auto take = [&](int row, unsigned &pos, unsigned &stop) {
                const int i = row / heads, k = row - i * heads;
                const unsigned here = i < s.slots ? s_pre[i] : 0, nc = i < s.slots ? s_pre[i + 1] - here : 0;
                pos = scalar(here * heads + k * nc);
                stop = pos + scalar(nc);
            };
            take(first_of(blockIdx.x), pos, stop);
            if (extra && second_of(blockIdx.x) >= 0) take(second_of(blockIdx.x), next, next_stop);
            if (pos == stop && next_stop != 0xffffffff) {
                pos = next;
                stop = next_stop;
            }
        }
        if (tid == 0) {
            s_next[0] = next;
            s_next[1] = next_stop;
        }
    } else {
        // the rows with the most keys first; where all blocks are resident at once, those of the second round the
        // other way about, so that a CU gets a long and a short one (2048 tokens of 32 heads of 128 60.5 -> 58.8 us, two
        // prompts of 1000 42.6 -> 37.0; with more blocks it costs: 2079 tokens after 2000 153 -> 173, 2480 73 -> 79)
        int q = blockIdx.z * gridDim.y + blockIdx.y;
        if (q >= s.slots) return;
        hy = blockIdx.x;
        constexpr int FIRST = 256;
        if (TL::BLOCKS == 2 && s.paired) {
            const int all = s.slots * heads, at = q * heads + hy;
            if (at >= FIRST) {
                q = scalar((all - 1 - (at - FIRST)) / heads);
                hy = all - 1 - (at - FIRST) - q * heads;
            }
        }
        slot = s.slots - 1 - q;
    }

    while (pos < stop) {
        int tid = threadIdx.x;
#ifdef __HIP_DEVICE_COMPILE__
        if (LINED) __asm__("" : "+v"(tid));  // (what is derived from it would be kept through the tiles for the next rows)
#endif
        const int lane = tid & 63, h = lane / W, c = lane & (W - 1);
        bool whole = true;
        int ch = 0, count = 0;
        unsigned left_over = 0;  // chunks of these rows that later parts take
        Work b;
        if constexpr (LINED) {
            int lo = 0, hi = s.slots;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if ((unsigned)scalar(s_pre[mid]) * heads <= pos) lo = mid;
                else hi = mid;
            }
            slot = lo;
            const unsigned here = scalar(s_pre[lo]), nc = scalar(s_pre[lo + 1]) - here;
            const unsigned local = pos - here * heads, left = stop - pos;
            hy = scalar(local / nc);
            ch = local - hy * nc;
            count = left < nc - ch ? left : nc - ch;
            whole = count == (int)nc;
            left_over = nc - ch - count;
        }
        const int kh = scalar(hy / s.parts), head0 = kh * d.g + (hy - kh * s.parts) * s.heads;
        const int g = (kh + 1) * d.g - head0 < s.heads ? (kh + 1) * d.g - head0 : s.heads;
        if constexpr (LINED) {
            const int4 x = s_work[slot];
            b = work_of<KT>(d, scalar(x.x), scalar(x.y), scalar(x.z), scalar(x.w));
        } else if (!locate<KT>(d, s, slot, b)) {
            return;
        }
        // (the same for all lanes, which a compiler that divides in vector registers does not see)
        b.n = scalar(b.n);
        b.tokens = scalar(b.tokens);
        b.row = scalar((int)b.row);
        b.p0 = scalar(b.p0);
        if (LINED && ch == 0 && tid == 0)
            s.cut[slot * heads + hy] = Cut{(int)b.row, b.tokens, (int)blockIdx.x, left_over == 0 ? 0 : 1 + (int)((left_over + quantum - 1) / quantum)};
        const int begin = scalar(b.begin) + ch * CHUNK, rows_end = scalar(b.end);
        const int end = LINED && rows_end - begin > count * CHUNK ? begin + count * CHUNK : rows_end;

        // ---- this lane's query: column c of the products ----
        const int r = W * w + c;
        const int used = b.tokens * g;
        const int rr = r < used ? r : used - 1;  // (rows that are not there follow the last one, and are not written)
        const int tok = rr / g, head = head0 + rr - tok * g;
        const int p = b.p0 + tok, low = first_key(d, p);
        // of the wave: the rows' first and last positions
        const int wr = W * w < used ? W * w : used - 1, wl = W * w + W - 1 < used ? W * w + W - 1 : used - 1;
        const int pw0 = b.p0 + scalar(wr / g), pw1 = b.p0 + scalar(wl / g);
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
        // Vector i of a wave's 64 lanes lies in 16 consecutive rows, so in one page: its number and first row are
        // scalars.
        const int64_t head_at = (int64_t)kh * d.page * D;
        const T *K = static_cast<const T *>(s.a.k_cache) + head_at, *Vc = static_cast<const T *>(s.a.v_cache) + head_at;
        auto top_of = [&](int i) { return (i * BLOCK + w * 64) / LINE; };  // the vector's first row
        auto row_of = [&](int i) { return (i * BLOCK + tid) / LINE; };
        auto from_of = [&](int i, int swap) {  // the lane's bytes from there, for its place in LDS
            return (unsigned)(((row_of(i) - top_of(i)) * D + ((i * BLOCK + tid) % LINE ^ swap) * V) * sizeof(T));
        };
        const unsigned lds_k = (unsigned)(uintptr_t)(__attribute__((address_space(3))) void *)sk;
        const unsigned lds_v = (unsigned)(uintptr_t)(__attribute__((address_space(3))) void *)sv;
        const int last = end - 1;
        // Lane i < NV (and NV + i) keeps the address of the wave's vector i of K (of V): a wave has a handful of them
        static_assert(2 * NV <= 64, "a lane an address");
        const int mine_top = (lane % NV * BLOCK + w * 64) / LINE;
        const T *mine_base = lane < NV ? K : Vc;
        int page = 0;
        auto ask = [&](int k0) {  // the pages of a tile (behind the end: of the last key)
            const int key = k0 + mine_top;
            page = table[(unsigned)(key < end ? key : last) >> d.log_page];
        };
        uint64_t at = 0;
        auto place = [&](int k0) {
            at = (uint64_t)(mine_base + page_bound(d, page) * d.page_stride + ((k0 + mine_top) & (d.page - 1)) * D);
        };
        auto copy = [&](int buf, int i) {
            const uint64_t base = (uint64_t)(unsigned)__builtin_amdgcn_readlane((int)(at >> 32), i) << 32 |
                                  (unsigned)__builtin_amdgcn_readlane((int)at, i);
            const int j = i % NV;
            const unsigned to = (buf * KT * LINE + j * BLOCK + w * 64) * 16;
            if (i < NV) copy_to_lds((const void *)base, from_of(j, TL::swap_k(row_of(j))), lds_k + to);
            else copy_to_lds((const void *)base, from_of(j, TL::swap_v(row_of(j))), lds_v + to);
        };
        auto load = [&](int k0, int buf) {
            place(k0);
#pragma unroll
            for (int i = 0; i < 2 * NV; ++i) copy(buf, i);
        };
        // V of a cut tile: rows behind the end and values that are not finite are made 0
        auto clean = [&](int k0, int buf) {
            bool bad = false;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int x = i * BLOCK + tid, row = row_of(i);
                vec v = ld16(&sv[buf][x * V]);
                unsigned bits = 0;
#pragma unroll
                for (int j = 0; j < V; ++j) bits |= (unsigned)not_finite(v[j]) << j;
                if (k0 + row >= end) bits = 0;  // (whatever the cache holds there)
#pragma unroll
                for (int j = 0; j < V; ++j) v[j] = k0 + row >= end || (bits >> j & 1) ? T(0.f) : v[j];
                st16(&sv[buf][x * V], v);
                s_bits[buf][row * LINE + (x - row * LINE ^ TL::swap_v(row))] = (unsigned char)bits;
                bad |= bits != 0;
            }
            const bool any = __any(bad);
            if (lane == 0) s_bad[buf][w] = any;
        };
        if (begin < end) {
            ask(begin);
            load(begin, 0);
            ask(begin + KT);
        }

        auto met = [&](int buf) {
            int x = 0;
#pragma unroll
            for (int i = 0; i < TL::WAVES; ++i) x |= s_bad[buf][i];
            return x != 0;
        };
        int buf = 0;
        for (int k0 = begin; k0 < end; k0 += KT, buf ^= 1) {
            wait_vmem_all();  // this wave's part of the tile has come
            lds_sync();       // and every wave's; the other buffer has been read
            place(k0 + KT);
            ask(k0 + 2 * KT);
            if (cut(k0)) {
                clean(k0, buf);
                lds_sync();
            }
            // copies of the next tile beside the scores' products from the second on, the rest after them
            constexpr int START = 1, EVERY = (NC * NT - START) / (2 * NV) > 0 ? (NC * NT - START) / (2 * NV) : 1;
            constexpr int BESIDE = (NC * NT - START + EVERY - 1) / EVERY < 2 * NV ? (NC * NT - START + EVERY - 1) / EVERY : 2 * NV;
            const bool mine = busy && k0 <= pw1 && k0 + KT > first_key(d, pw0);
            acc sc[NT];
            bool masked = false;
            if (mine) {
#pragma unroll
                for (int t = 0; t < NT; ++t) sc[t] = acc(0.f);
                // product u: channels 8 G (u / NT).., keys W (u % NT)..
                auto key_rows = [&](int u) {
                    const T *row = &sk[buf][(W * (u % NT) + c) * D];
                    const int x = (8 * G * (u / NT) + 8 * h) / V, swap = TL::swap_k(c);
                    if constexpr (sizeof(T) == 4) {
                        const f4 a = *reinterpret_cast<const f4 *>(row + (x ^ swap) * V), b = *reinterpret_cast<const f4 *>(row + ((x + 1) ^ swap) * V);
                        return (frag)__builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
                    } else {
                        return *reinterpret_cast<const frag *>(row + (x ^ swap) * V);
                    }
                };
                __builtin_amdgcn_s_setprio(1);
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
                    if (u >= START && (u - START) % EVERY == 0 && (u - START) / EVERY < 2 * NV) copy(buf ^ 1, (u - START) / EVERY);
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
                __builtin_amdgcn_s_setprio(0);
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
                if (cut(k0) && met(buf)) {  // (rare: no care for its time)
#pragma unroll 1
                    for (int j = 0; j < KT; ++j) {
                        const bool sees = k0 + j <= p && k0 + j >= low && k0 + j < end;
#pragma unroll
                        for (int t = 0; t < ND; ++t)
#pragma unroll
                            for (int i = 0; i < UNITS; ++i) {
                                const int ch = W * t + 4 * G * i + 4 * h;
                                const unsigned bits = sees ? s_bits[buf][j * LINE + ch / V] >> (ch % V) & 15 : 0;
                                dead[(t * NA + 4 * i) / 32] |= bits << (t * NA + 4 * i) % 32;
                                __builtin_amdgcn_sched_barrier(0);
                            }
                    }
                }
            }
#pragma unroll
            for (int i = BESIDE; i < 2 * NV; ++i) copy(buf ^ 1, i);
            if (!mine) {
#pragma unroll
                for (int i = 0; i < BESIDE; ++i) copy(buf ^ 1, i);
            }
            if (mine) {
                // product u: channels W (u % ND).., keys 8 G (u / ND)..
                auto channels = [&](int u) { return column<T, D>(sv[buf], u / ND, u % ND, lane); };
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
                __builtin_amdgcn_s_setprio(1);
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
                __builtin_amdgcn_s_setprio(0);
            }
        }

        l = column_sum<G>(l);
        wait_vmem_all();  // (the copy of the tile behind the last one)
#pragma unroll
        for (int t = 0; t < ND; ++t)
#pragma unroll
            for (int i = 0; i < NA; ++i) o[t][i] = dead[(t * NA + i) / 32] >> (t * NA + i) % 32 & 1 ? NAN : o[t][i];
        // ---- the rows' ends, from the lane anew ----
        int own = tid;
#ifdef __HIP_DEVICE_COMPILE__
        if (LINED) __asm__("" : "+v"(own));  // (as above)
#endif
        const int my = own & 63, col0 = 4 * (my / W), mc = my & (W - 1), mr = W * w + mc;
        if (!LINED || whole) {
            // Rows leave through LDS, and their gates come so: whole lines of memory, not 8 bytes of each (1024 tokens of
            // 16 heads of 256 46 -> 44 us)
            lds_sync();  // every wave has read its last tile
            constexpr int HELD = 2 * KT / W, NO = W * LINE / 64;  // waves whose rows fit in a buffer; vectors a lane moves
            T *rows = w < HELD ? sk[0] + w * W * D : sv[0] + (w - HELD) * W * D;
            const int mrr = mr < used ? mr : used - 1, mt = mrr / g, head = head0 + mrr - mt * g;
            const int64_t row = b.row + mt, out_at = (row * d.H + head) * D, gate_at = row * d.gate_stride + (int64_t)head * D;
            auto vector_of = [&](int x) { return rows + (x / LINE * LINE + (x % LINE ^ TL::swap_k(x / LINE))) * V; };
            auto quad_of = [&](int col) {
                return reinterpret_cast<typename Quad<T>::t4 *>(rows + (mc * LINE + (col / V ^ TL::swap_k(mc))) * V + col % V);
            };
            const float inv = inverse_sum(l);
            if (s.a.gate) {
                vec gate[NO];
#pragma unroll
                for (int i = 0; i < NO; ++i) {
                    const int x = i * 64 + my;
                    gate[i] = ld16(static_cast<const T *>(s.a.gate) + __shfl((long long)gate_at, x / LINE, 64) + x % LINE * V);
                }
#pragma unroll
                for (int i = 0; i < NO; ++i) st16(vector_of(i * 64 + my), gate[i]);
                wave_sync();
            }
#pragma unroll
            for (int t = 0; t < ND; ++t)
#pragma unroll
                for (int i = 0; i < UNITS; ++i) {
                    const f4 x = {o[t][4 * i], o[t][4 * i + 1], o[t][4 * i + 2], o[t][4 * i + 3]};
                    typename Quad<T>::t4 *at = quad_of(W * t + 4 * G * i + col0);
                    typename Quad<T>::t4 gate = {};
                    if (s.a.gate) gate = *at;
                    *at = finished<T>(s.a, x, inv, gate);
                }
            wave_sync();
#pragma unroll
            for (int i = 0; i < NO; ++i) {
                const int x = i * 64 + my;
                const int64_t to = __shfl((long long)out_at, x / LINE, 64) + x % LINE * V;
                if (W * w + x / LINE < used) st16(static_cast<T *>(s.a.out) + to, ld16(vector_of(x)));
            }
        } else if (mr < used) {
            const int64_t piece = 2 * (int64_t)blockIdx.x + (ch == 0);
            if (col0 == 0) s.ml[piece * TL::ROWS + mr] = make_float2(m, l);
#pragma unroll
            for (int t = 0; t < ND; ++t)
#pragma unroll
                for (int i = 0; i < UNITS; ++i) {
                    const f4 x = {o[t][4 * i], o[t][4 * i + 1], o[t][4 * i + 2], o[t][4 * i + 3]};
                    s.o[((piece * TL::WAVES + w) * ND * UNITS + t * UNITS + i) * 64 + my] = x;  // whole lines
                }
        }
        if constexpr (!LINED) return;
        pos += count;
        lds_sync();  // LDS is free for the next rows
        if (pos == stop && (unsigned)scalar(s_next[1]) < stop) {
            pos = scalar(s_next[0]);
            stop = scalar(s_next[1]);
        }
    }
}

// The rows whose keys the line is cut in: a block such rows and 1024 values, every piece read once, BATCH at a time
constexpr int BATCH = 8;
template <typename T, int D>
__global__ __launch_bounds__(256) void join_kernel(AttnDims d, PrefillArgs s)
{
    typedef Tile<T, D> TL;
    constexpr int ROWS = TL::ROWS, W = TL::W, G = TL::G, UNITS = TL::NA / 4;
    const Cut cut = s.cut[blockIdx.x];
    if (cut.pieces == 0) return;
    const int hy = blockIdx.x % (d.KV * s.parts);
    const int kh = hy / s.parts, head0 = kh * d.g + (hy - kh * s.parts) * s.heads;
    const int g = (kh + 1) * d.g - head0 < s.heads ? (kh + 1) * d.g - head0 : s.heads;
    const int at = blockIdx.y * 256 + threadIdx.x, lane = at % 64, unit = at / 64 % (D * W / 256), w = at / 64 / (D * W / 256);
    const int r = W * w + lane % W, col = W * (unit / UNITS) + 4 * G * (unit % UNITS) + 4 * (lane / W);
    if (r >= cut.tokens * g) return;
    const int tok = r / g, head = head0 + r - tok * g;
    const int64_t row = (int64_t)cut.row + tok;
    typename Quad<T>::t4 gate = {};
    if (s.a.gate) gate = gate_of<T>(d, s.a, row, head, col);
    float m = -INFINITY, l = 0.f;
    f4 o = f4(0.f);
#pragma unroll 1
    for (int p0 = 0; p0 < cut.pieces; p0 += BATCH) {
        float2 ml[BATCH];
        f4 x[BATCH];
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            const int p = p0 + u;
            ml[u] = make_float2(-INFINITY, 0.f);
            x[u] = f4(0.f);
            if (p >= cut.pieces) continue;
            // the first piece is the end of its part, the others begin in theirs
            const int64_t piece = p == 0 ? 2 * (int64_t)cut.first + 1 : 2 * ((int64_t)cut.first + p);
            ml[u] = s.ml[piece * ROWS + r];
            x[u] = s.o[piece * (ROWS * D / 4) + at];
        }
        join<BATCH>(ml, x, m, l, o);
    }
    finish<T>(d, s.a, row, head, col, o, inverse_sum(l), gate);
}

// What the line costs beside its keys, in us: ends of the parts and the join, more the more parts there are, and
// the more of them hold ends of two rows.  Measured without and with it: 16 heads of 256, 64 tokens after
// 1000 46 and 20 us, 300 after 300 31 and 23, 600 from their start 31 and 28, 900 41 and 43, 1500 61 and 84; 32 heads
// of 128, 512 tokens 20 and 25, after 1500 50 and 42, 1024 31 and 49.  Of batches, 115 tokens after 3780 with five short
// prompts, 20 heads of 192, 94 and 59; more blocks than are resident, 1475 tokens after 5788, 24 heads of 256, 422 and 318.
double line_us(double full, double parts) { return 6.6 * (1 + parts + full) + 66 * full * full; }
// and a key of a block alone on its CU
double key_us(bool f32, int D) { return f32 ? 0.0006 * D : 0.006 + 0.000105 * D; }

struct Plan {
    int heads, parts, tokens, slots, line;
    bool paired;
    unsigned worth;
    size_t cut, ml, o;
};
Plan plan_of(const AttnDims &d, bool f32, int rows, int on_cu)
{
    Plan p;
    p.heads = d.g < rows ? d.g : rows;
    p.parts = (d.g + p.heads - 1) / p.heads;
    p.tokens = rows / p.heads;
    p.slots = (int)(d.T / p.tokens) + d.n_seq;
    const int64_t blocks = (int64_t)p.slots * d.KV * p.parts;
    int64_t span = d.max_kv;
    if (d.window < span && (int64_t)d.window + p.tokens + 64 < span) span = (int64_t)d.window + p.tokens + 64;
    const int64_t most = blocks * ((span + CHUNK - 1) / CHUNK + 1);
    // Without the line the longest rows' keys are the launch's time, or two rows' of a block that comes second; with it
    // the average, dealt to all blocks that are resident at once.  The lengths are not known here but for their
    // bounds: where the line may pay the kernel decides, by the same rule (4 us if it does not deal; prompts from their
    // start with max_kv 32768, 16 heads of 256: 2100 tokens 137 -> 87 us, 3500 298 -> 141).
    const int64_t resident = 256 * on_cu, line = most < resident ? most : resident;
    p.paired = ((d.T > d.n_seq ? (d.T - d.n_seq) / p.tokens : 0) + d.n_seq) * d.KV * p.parts <= resident;
    const double full = (double)blocks / resident, newest = (double)(d.max_T < span ? d.max_T : span), held = span - newest / 2;
    const double key = key_us(f32, d.D), cost = line_us(full, (double)line / resident) / key;
    const bool second = blocks > resident;
    const double alone = second && 2 * (span - newest / full) > span ? 2 * (span - newest / full) : span;
    const double dealt = held * full / (second ? 1 : d.n_seq);
    p.line = p.slots <= MOST_SLOTS && blocks <= 2 * resident && most < (int64_t)1 << 31 && alone - dealt > cost + (d.n_seq > 1 ? 4 / key : 0) ? (int)line : 0;
    p.worth = 1 + (unsigned)cost;
    p.cut = p.line ? ((size_t)blocks * sizeof(Cut) + 255) / 256 * 256 : 0;
    p.ml = (size_t)p.line * 2 * rows * sizeof(float2);
    p.o = (size_t)p.line * 2 * rows * d.D * sizeof(float);
    return p;
}

template <typename T, int D>
void launch_prefill_t(const AttnDims &d, const AttnArgs &a, hipStream_t st)
{
    typedef Tile<T, D> TL;
    const Plan p = plan_of(d, sizeof(T) == 4, TL::ROWS, TL::BLOCKS);
    char *ws = static_cast<char *>(a.ws);
    const PrefillArgs s{a, p.heads, p.parts, p.tokens, p.slots, p.paired, p.line, p.worth, reinterpret_cast<Cut *>(ws),
                        reinterpret_cast<float2 *>(ws + p.cut), reinterpret_cast<f4 *>(ws + p.cut + p.ml)};
    const int gy = p.slots < 32768 ? p.slots : 32768;
    const dim3 grid = p.line ? dim3(p.line) : dim3(d.KV * p.parts, gy, (p.slots + gy - 1) / gy);
    hipLaunchKernelGGL((p.line ? prefill_kernel<T, D, true> : prefill_kernel<T, D, false>), grid, dim3(TL::BLOCK), 0, st, d, s);
    if (p.line > 1) hipLaunchKernelGGL((join_kernel<T, D>), dim3(p.slots * d.KV * p.parts, TL::ROWS * (D / 4) / 256), dim3(256), 0, st, d, s);
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
    int rows = 0, blocks = 0;
    GDN_SSM_IO(s.io_dtype, GDN_ATTN_D(rows = Tile<TI, D>::ROWS; blocks = Tile<TI, D>::BLOCKS;))
    const Plan p = plan_of(attn_dims(s), s.io_dtype == GDN_F32, rows, blocks);
    return p.cut + p.ml + p.o;
}

hipError_t launch_attn_prefill(const gdn_attn_shape &s, const AttnArgs &a, hipStream_t st)
{
    const AttnDims d = attn_dims(s);
    GDN_SSM_IO(s.io_dtype, GDN_ATTN_D(launch_prefill_t<TI, D>(d, a, st);))
    return hipGetLastError();
}

} // namespace gdn
