// attn_step.hip -- attention of one new token a sequence over the paged cache.
//
//   o = sum_j w_j V_j / sum_j w_j,  w_j = exp(scale q.K_j - max)   over the keys the token sees
//
// The g query heads of a key-value head share its keys, so they are the 16 columns of
// a matrix product (a unit: sequence, key-value head, 16 query heads), and K and V
// are read once: bound by HBM bandwidth.
//
// Work.  The keys of all units, in chunks of 128, form one line that is cut into equal
// parts, one a block: every block finds its place by a prefix sum over kv_len, so the
// parts are equal whatever the lengths are, also in a captured call whose lengths
// have grown.  A block walks the segments (units, or pieces of them) of its part.  A
// unit within one part is finished there; of one that is cut, each part leaves its sums,
// maximum and weights' sum in the workspace (a part cuts two units at most, at its
// ends), and a second kernel joins them.
//
// gfx950 mapping.  Within a segment the block's 4 waves take tiles of KT keys in turn,
// each on its own, with no barrier.  S^T = K Q^T puts a key a row and a query a
// column: the columns' maxima and sums stay in their lanes, and the weights of lane
// (gq, c) are keys 4 gq + 0..3 of a tile, which is at once the operand of O^T = V^T w
// if V^T is read in the same order of keys.  K goes from memory to the operands
// directly; V through LDS, whose transposing reads give 4 keys of a channel a lane.
// While a tile is computed the next one's K and V are loaded to registers.
//
// Precision.  Scores, maxima, sums and O are fp32.  16-bit weights enter the product
// with V in two parts of the matrix type (2^-16 of a weight at bf16, 2^-22 at fp16, or
// 2^-25 of the largest): the matrix pipes have the time.
#include "attn_device.h"
#include "mfma_device.h"

namespace gdn {

namespace {

constexpr int BLOCK = 256, WAVES = 4;
constexpr int CHUNK = 128;   // keys that a unit is cut at
constexpr int PARTS_MAX = 512;  // blocks of a launch

// What a part leaves of its place for the kernel that joins: the chunk its first
// sequence begins at, that sequence (-1: the part is empty), chunks of a part
struct Place {
    int64_t base, quantum;
    int n, pad;
};

struct StepArgs {
    AttnArgs a;
    int tiles;      // of 16 query heads in a key-value head
    Place *place;   // [parts]
    float2 *ml;     // [2 parts][16] maximum (of scores times scale log2 e) and sum of weights
    float *o;       // [2 parts][16][D]
};

__device__ __forceinline__ int chunks_of(const AttnDims &d, int len)
{
    const int span = len - first_key(d, len - 1);
    return span <= CHUNK ? 1 : (span + CHUNK - 1) / CHUNK;
}

template <typename T, int D> struct Tile {
    static constexpr int KT = sizeof(T) == 2 ? 32 : 16;  // keys
    static constexpr int NT = KT / 16, NC = D / 32, ND = D / 16;
    static constexpr int V = Vec16<T>::n;
    static constexpr int NV = KT * D / V / 64;      // vectors of V a lane
    static constexpr int PITCH = D + 32 / sizeof(T);  // of V in LDS: 16 rows of 32 bytes then lie in 8 different groups of banks
    static constexpr int OP = D + 4;                // of O in LDS
    static constexpr int BYTES = KT * PITCH * sizeof(T) > 16 * OP * 4 ? KT * PITCH * sizeof(T) : 16 * OP * 4;
};

// 16 keys x 16 queries, or 16 channels x 16 queries
template <typename T, int D>
__device__ __forceinline__ void weigh(const T *v, const float *w, int lane, f4 (&o)[D / 16])
{
    typedef Mat<T> MT;
    constexpr int PITCH = Tile<T, D>::PITCH;
    typename MT::frag p[2];
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = w[i];
    split8<T, 2>(x, p);
    const int gq = lane >> 4, c = lane & 15;
    typedef short s4 __attribute__((ext_vector_type(4)));
    typedef short s8 __attribute__((ext_vector_type(8)));
    typedef __attribute__((address_space(3))) s4 lds_s4;
    const T *at = v + (4 * gq + (c >> 2)) * PITCH + 4 * (c & 3);
    typename MT::frag f[D / 16];
#pragma unroll
    for (int t = 0; t < D / 16; ++t) {
        const s4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)(at + 16 * t));
        const s4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)(at + 16 * PITCH + 16 * t));
        f[t] = __builtin_bit_cast(typename MT::frag, (s8)__builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
    __builtin_amdgcn_sched_barrier(0);  // no load is given registers of an operand in use
#pragma unroll
    for (int t = 0; t < D / 16; ++t) o[t] = MT::mma(f[t], p[0], o[t]);
#pragma unroll
    for (int t = 0; t < D / 16; ++t) o[t] = MT::mma(f[t], p[1], o[t]);
}
template <int D>
__device__ __forceinline__ void weigh(const float *v, const float *w, int lane, f4 (&o)[D / 16])
{
    constexpr int PITCH = Tile<float, D>::PITCH;
    const float *at = v + 4 * (lane >> 4) * PITCH + (lane & 15);
    float f[D / 16][4];
#pragma unroll
    for (int t = 0; t < D / 16; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) f[t][i] = at[i * PITCH + 16 * t];
    __builtin_amdgcn_sched_barrier(0);  // no load is given registers of an operand in use
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int t = 0; t < D / 16; ++t) o[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(f[t][i], w[i], o[t], 0, 0, 0);
}

__device__ __forceinline__ float sum_of_groups(float x)
{
    x += __shfl_xor(x, 16, 64);
    return x + __shfl_xor(x, 32, 64);
}

// out = o / l, gated, 4 channels
template <typename T>
__device__ __forceinline__ void finish(const AttnDims &d, const AttnArgs &a, int64_t row, int head, int col, f4 o, float l)
{
    typedef T t4 __attribute__((ext_vector_type(4)));
    const float r = l > 0.f ? 1.0f / l : l;  // no key: o and l are 0 (a NaN stays one)
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

template <typename T, int D>
__global__ __launch_bounds__(BLOCK, D <= 128 ? 2 : 1) void step_kernel(AttnDims d, StepArgs s)
{
    typedef Mat<T> MT;
    typedef typename MT::frag frag;
    typedef Tile<T, D> TL;
    typedef typename Vec16<T>::type vec;
    constexpr int KT = TL::KT, NT = TL::NT, NC = TL::NC, ND = TL::ND, NV = TL::NV, V = TL::V;
    __shared__ __attribute__((aligned(16))) char lds[WAVES * TL::BYTES];
    __shared__ float sm[WAVES][16], sl[WAVES][16];
    __shared__ int64_t s_wave[WAVES], s_base;
    __shared__ int s_n;
    const int tid = threadIdx.x, lane = tid & 63, gq = lane >> 4, c = lane & 15;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int units = d.KV * s.tiles;  // of a sequence

    // ---- this block's part of the chunks ----
    const int per = (d.n_seq + BLOCK - 1) / BLOCK;
    int64_t mine = 0;
    for (int i = tid * per; i < d.n_seq && i < (tid + 1) * per; ++i) mine += chunks_of(d, kv_bound(d, s.a.kv_len, i));
    mine *= units;
    int64_t upto = mine;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
        const int64_t x = __shfl_up((long long)upto, m, 64);
        if (lane >= m) upto += x;
    }
    if (lane == 63) s_wave[w] = upto;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) {
        if (i < w) upto += s_wave[i];
        total += s_wave[i];
    }
    const int64_t quantum = (total + gridDim.x - 1) / gridDim.x;
    int64_t pos = blockIdx.x * quantum;
    const int64_t stop = pos + quantum < total ? pos + quantum : total;
    if (pos >= total) {
        if (tid == 0) s.place[blockIdx.x].n = -1;
        return;
    }
    if (pos >= upto - mine && pos < upto) {
        int64_t base = upto - mine;
        int n = tid * per;
        for (;; ++n) {
            const int64_t size = (int64_t)chunks_of(d, kv_bound(d, s.a.kv_len, n)) * units;
            if (pos < base + size) break;
            base += size;
        }
        s_base = base;
        s_n = n;
        s.place[blockIdx.x] = Place{base, quantum, n, 0};
    }
    __syncthreads();
    int64_t base = s_base;
    int n = __builtin_amdgcn_readfirstlane(s_n);

    T *sv = reinterpret_cast<T *>(lds + w * TL::BYTES);
    float *so = reinterpret_cast<float *>(lds + w * TL::BYTES);
    const float cs = d.scale * 1.44269504f;

    while (pos < stop) {
        const int len = kv_bound(d, s.a.kv_len, n), first = first_key(d, len - 1), nc = chunks_of(d, len);
        const int64_t local = pos - base;
        if (local >= (int64_t)nc * units) {
            base += (int64_t)nc * units;
            ++n;
            continue;
        }
        const int unit = (int)(local / nc), ch = (int)(local - (int64_t)unit * nc);
        const int count = stop - pos < nc - ch ? (int)(stop - pos) : nc - ch;
        const int kh = unit / s.tiles, head0 = kh * d.g + (unit - kh * s.tiles) * 16;
        const int rows = (kh + 1) * d.g - head0 < 16 ? (kh + 1) * d.g - head0 : 16;
        const int begin = first + ch * CHUNK;
        const int end = ch + count < nc ? begin + count * CHUNK : len;

        // ---- queries: column c of the products ----
        frag qf[NC];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            qf[i] = frag(0);
            if (c < rows) {
                const T *p = static_cast<const T *>(s.a.q) + (int64_t)n * d.q_stride + (int64_t)(head0 + c) * D + 32 * i + 8 * gq;
                qf[i] = *reinterpret_cast<const typename Frag16<T>::type *>(p);
            }
        }
        f4 o[ND];
#pragma unroll
        for (int t = 0; t < ND; ++t) o[t] = f4(0.f);
        float m = -INFINITY, l = 0.f;

        const int32_t *table = s.a.table + (int64_t)n * d.table_pages;
        const T *K = static_cast<const T *>(s.a.k_cache), *Vc = static_cast<const T *>(s.a.v_cache);
        frag kf[NT][NC];
        vec vv[NV];
        // a lane's key of a tile (behind the end: the last one), and its row in the cache
        auto page_of = [&](int k0) {
            const int key = k0 + (lane & (KT - 1));
            return table[(key < end ? key : end - 1) >> d.log_page];
        };
        auto load = [&](int k0, int page) {
            int key = k0 + (lane & (KT - 1));
            key = key < end ? key : end - 1;
            const int64_t at = cache_row(d, page_bound(d, page), kh, key & (d.page - 1));
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const T *p = K + __shfl((long long)at, 16 * t + c, 64) + 8 * gq;
#pragma unroll
                for (int i = 0; i < NC; ++i) kf[t][i] = *reinterpret_cast<const typename Frag16<T>::type *>(p + 32 * i);
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int x = i * 64 + lane, r = x / (D / V);
                vv[i] = ld16(Vc + __shfl((long long)at, r, 64) + (x - r * (D / V)) * V);
            }
        };
        int k0 = begin + w * KT;
        constexpr int STEP = WAVES * KT;
        int page = 0;
        if (k0 < end) {
            load(k0, page_of(k0));
            if (k0 + STEP < end) page = page_of(k0 + STEP);
        }
        for (; k0 < end; k0 += STEP) {
            const bool tail = k0 + KT > end;
            // V to LDS: rows behind the end as zeros, whatever the cache holds
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int x = i * 64 + lane, r = x / (D / V);
                if (tail && k0 + r >= end) vv[i] = vec(0);
                st16(sv + r * TL::PITCH + (x - r * (D / V)) * V, vv[i]);
            }
            f4 sc[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                sc[t] = f4(0.f);
#pragma unroll
                for (int i = 0; i < NC; ++i) sc[t] = MT::mma(kf[t][i], qf[i], sc[t]);
            }
            if (tail) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) sc[t][i] = k0 + 16 * t + 4 * gq + i < end ? sc[t][i] : -INFINITY;
            }
            float most = -INFINITY;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) most = fmaxf(most, sc[t][i]);
            const float m1 = fmaxf(m, max_of_groups(most) * cs);
            // the next tile, once the products that read these registers are through
            __builtin_amdgcn_sched_barrier(0);
            if (k0 + STEP < end) {
                load(k0 + STEP, page);
                if (k0 + 2 * STEP < end) page = page_of(k0 + 2 * STEP);
            }
            if (__any(m1 != m)) {
                const float keep = __builtin_amdgcn_exp2f(m - (m1 == -INFINITY ? 0.f : m1));
                m = m1;
                l *= keep;
#pragma unroll
                for (int t = 0; t < ND; ++t) o[t] *= keep;
            }
            const float m0 = m == -INFINITY ? 0.f : m;
            float wt[4 * NT];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    wt[4 * t + i] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[t][i], cs, -m0));
                    l += wt[4 * t + i];
                }
            if constexpr (sizeof(T) == 2) weigh<T, D>(sv, wt, lane, o);
            else weigh<D>(sv, wt, lane, o);
        }

        // ---- the four waves' sums joined ----
        l = sum_of_groups(l);
        __syncthreads();  // V has been read
        if (gq == 0) {
            sm[w][c] = m;
            sl[w][c] = l;
        }
#pragma unroll
        for (int t = 0; t < ND; ++t) *reinterpret_cast<f4 *>(so + c * TL::OP + 16 * t + 4 * gq) = o[t];
        __syncthreads();
        const bool whole = count == nc;
        const int64_t slot = 2 * (int64_t)blockIdx.x + (ch == 0);
        for (int i = tid; i < rows * (D / 4); i += BLOCK) {
            const int r = i / (D / 4), col = (i - r * (D / 4)) * 4;
            const float big = fmaxf(fmaxf(sm[0][r], sm[1][r]), fmaxf(sm[2][r], sm[3][r]));
            const float big0 = big == -INFINITY ? 0.f : big;
            f4 sum = f4(0.f);
            float lsum = 0.f;
#pragma unroll
            for (int u = 0; u < WAVES; ++u) {
                const float f = __builtin_amdgcn_exp2f(sm[u][r] - big0);
                lsum += f * sl[u][r];
                sum += f * *reinterpret_cast<const f4 *>(reinterpret_cast<const float *>(lds + u * TL::BYTES) + r * TL::OP + col);
            }
            if (whole) {
                finish<T>(d, s.a, n, head0 + r, col, sum, lsum);
            } else {
                *reinterpret_cast<f4 *>(s.o + (slot * 16 + r) * D + col) = sum;
                if (col == 0) s.ml[slot * 16 + r] = make_float2(big, lsum);
            }
        }
        __syncthreads();  // LDS is free for the next segment
        pos += count;
    }
}

// The units that are cut: a block a cut and row.  The first cut of a unit stands for
// it; the others leave.
constexpr int JOIN = 512;
template <typename T, int D>
__global__ __launch_bounds__(JOIN) void join_kernel(AttnDims d, StepArgs s)
{
    constexpr int LANES = D / 4, TEAMS = JOIN / LANES;
    __shared__ float fac[PARTS_MAX];
    __shared__ float red[JOIN / 64], sl[JOIN / 64];
    __shared__ f4 so[TEAMS][LANES];
    const int64_t b = blockIdx.x + 1;
    const Place pl = s.place[b];
    if (pl.n < 0) return;
    const int64_t pos = b * pl.quantum, local = pos - pl.base;
    const int nc = chunks_of(d, kv_bound(d, s.a.kv_len, pl.n));
    const int unit = (int)(local / nc), ch = (int)(local - (int64_t)unit * nc);
    if (ch == 0 || ch > pl.quantum) return;  // no cut, or not the first one
    const int kh = unit / s.tiles, head0 = kh * d.g + (unit - kh * s.tiles) * 16, r = blockIdx.y;
    if (head0 + r >= (kh + 1) * d.g) return;
    const int parts = 1 + (int)((nc - ch + pl.quantum - 1) / pl.quantum);
    const int tid = threadIdx.x, team = tid / LANES, lane = tid - team * LANES;
    // part 0 is the end of block b - 1, the others begin in their block
    auto slot = [&](int i) { return i == 0 ? 2 * (b - 1) + 1 : 2 * (b - 1 + i); };
    float m = -INFINITY, l = 0.f;
    if (tid < parts) {
        const float2 x = s.ml[slot(tid) * 16 + r];
        m = x.x;
        l = x.y;
    }
    float big = m;
#pragma unroll
    for (int u = 32; u > 0; u >>= 1) big = fmaxf(big, __shfl_xor(big, u, 64));
    if ((tid & 63) == 0) red[tid >> 6] = big;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < JOIN / 64; ++u) big = fmaxf(big, red[u]);
    const float f = __builtin_amdgcn_exp2f(m - (big == -INFINITY ? 0.f : big));
    if (tid < parts) fac[tid] = f;
    l *= f;
#pragma unroll
    for (int u = 32; u > 0; u >>= 1) l += __shfl_xor(l, u, 64);
    if ((tid & 63) == 0) sl[tid >> 6] = l;
    __syncthreads();
    f4 sum = f4(0.f);
    if (team < TEAMS) {
#pragma unroll 4
        for (int i = team; i < parts; i += TEAMS)
            sum += fac[i] * *reinterpret_cast<const f4 *>(s.o + (slot(i) * 16 + r) * D + lane * 4);
        so[team][lane] = sum;
    }
    __syncthreads();
    if (team == 0) {
        l = 0.f;
#pragma unroll
        for (int u = 0; u < JOIN / 64; ++u) l += sl[u];
        sum = f4(0.f);
#pragma unroll
        for (int u = 0; u < TEAMS; ++u) sum += so[u][lane];
        finish<T>(d, s.a, pl.n, head0 + r, lane * 4, sum, l);
    }
}

struct Plan {
    int tiles, parts;
    bool cut;  // a unit may be cut
    size_t place, ml, o;  // bytes
    size_t bytes() const { return place + ml + o; }
};

Plan plan_of(const gdn_attn_shape &s)
{
    const AttnDims d = attn_dims(s);
    Plan p;
    p.tiles = (d.g + 15) / 16;
    const int64_t span = d.window < d.max_kv ? d.window : d.max_kv;
    const int64_t units = (int64_t)d.n_seq * d.KV * p.tiles, most = units * (span <= CHUNK ? 1 : (span + CHUNK - 1) / CHUNK);
    p.parts = (int)(most < PARTS_MAX ? most : PARTS_MAX);
    p.cut = span > CHUNK;
    p.place = ((size_t)p.parts * sizeof(Place) + 255) / 256 * 256;
    p.ml = p.cut ? (size_t)p.parts * 32 * sizeof(float2) : 0;
    p.o = p.cut ? (size_t)p.parts * 32 * d.D * sizeof(float) : 0;
    return p;
}

template <typename T, int D>
void launch_step_t(const AttnDims &d, const AttnArgs &a, const Plan &p, hipStream_t st)
{
    char *ws = static_cast<char *>(a.ws);
    const StepArgs s{a, p.tiles, reinterpret_cast<Place *>(ws), reinterpret_cast<float2 *>(ws + p.place),
                     reinterpret_cast<float *>(ws + p.place + p.ml)};
    hipLaunchKernelGGL((step_kernel<T, D>), dim3(p.parts), dim3(BLOCK), 0, st, d, s);
    if (p.cut && p.parts > 1)
        hipLaunchKernelGGL((join_kernel<T, D>), dim3(p.parts - 1, d.g < 16 ? d.g : 16), dim3(JOIN), 0, st, d, s);
}

} // namespace

size_t attn_step_workspace_bytes(const gdn_attn_shape &s) { return plan_of(s).bytes(); }

hipError_t launch_attn_step(const gdn_attn_shape &s, const AttnArgs &a, hipStream_t st)
{
    const AttnDims d = attn_dims(s);
    const Plan p = plan_of(s);
    GDN_SSM_IO(s.io_dtype,
        switch (s.head_dim) {
        case 64: launch_step_t<TI, 64>(d, a, p, st); break;
        case 96: launch_step_t<TI, 96>(d, a, p, st); break;
        case 128: launch_step_t<TI, 128>(d, a, p, st); break;
        case 192: launch_step_t<TI, 192>(d, a, p, st); break;
        default: launch_step_t<TI, 256>(d, a, p, st); break;
        })
    return hipGetLastError();
}

} // namespace gdn
