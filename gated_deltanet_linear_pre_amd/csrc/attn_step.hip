// attn_step.hip -- attention of one new token a sequence over the paged cache.
//
//   o = sum_j w_j V_j / sum_j w_j,  w_j = exp(scale q.K_j - max)   over the keys the token sees
//
// The g query heads of a key-value head share its keys: 16 are the columns of a matrix
// product, and up to 8 waves of a block take as many such tiles over the same keys (a unit:
// sequence, key-value head, those tiles), so that K and V come from memory once: bound by HBM
// bandwidth.  (Tile after tile, 32 sequences of 8000 keys of 64 heads of 128 over one take 90 us, side by
// side 56; 16 of 64 heads of 256 over two 90 and 69.)
//
// Work.  The keys of all units, in chunks of 64, form one line that is cut into equal
// parts, one a block: every block finds its place by a prefix sum over kv_len, so the
// parts are equal whatever the lengths are, also in a captured call whose lengths
// have grown.  A block walks the segments (units, or pieces of them) of its part.  A
// unit within one part is finished there; of one that is cut, each part leaves its sums,
// maximum and weights' sum in the workspace (a part cuts two units at most, at its
// ends), and a second kernel joins them.
//
// gfx950 mapping.  256 parts, one a CU (512: 3 to 10 us more, for their joins and ends), of 8 waves (4 of
// twice the registers for fp32 of wide heads) that take tiles of KT keys in turn, each on its own,
// with no barrier.  S^T = K Q^T puts a key a row and a query a
// column: the columns' maxima and sums stay in their lanes, and the weights of lane
// (gq, c) are keys 4 gq + 0..3 of a tile, which is at once the operand of O^T = V^T w
// if V^T is read in the same order of keys.  While a tile is computed the next one's K is loaded to the
// operands and its V copied to LDS without registers, whose transposing reads give 4 keys of a channel a
// lane (V through registers, and so 4 waves a CU at D = 256: 88 us for what takes 79).
// Both are read once, so past the caches' order (83 us without for 76); not where several waves want the same
// keys (56 us above, 73 so).
//
// Precision.  Scores, maxima, sums and O are fp32.  16-bit weights enter the product
// with V in two parts of the matrix type (2^-16 of a weight at bf16, 2^-22 at fp16, or
// 2^-25 of the largest): the matrix pipes have the time.
//
// Measured: one sequence of 99991 keys, 32 heads of 128 over 8, fp16, 71 us (5.8 TB/s); 64 sequences of up to
// 20011 keys, 16 heads of 256 over 2, bf16, 80 us (5.2 TB/s); one of 701 keys 11 us; fp32, 32 of 4001 keys, 32 heads
// of 128 over 8, 162 us (6.5 TB/s).  Units of at most 64 keys, of which 2 waves at most have a tile, are slow:
// 4096 sequences of 61 keys 545 us (2.1 TB/s).
#include "attn_device.h"
#include "mfma_device.h"

namespace gdn {

namespace {

// Keys that a unit is cut at (128: 701 keys 11.7 us for 10.9, 64 ragged sequences 77.7 for 79.3; 32: 85.2) and
// blocks of a launch
constexpr int CHUNK = 64, PARTS_MAX = 256;
constexpr int waves_of(bool f32, int D) { return f32 && D > 128 ? 4 : 8; }

// A unit that is cut, for the kernel that joins: its sequence and place in it, the part it begins in, and
// how many parts have a piece (0: it is not cut)
struct Cut {
    int n, unit, first, pieces;
};

struct StepArgs {
    AttnArgs a;
    int wide, log_wide;  // tiles of 16 query heads of a unit: 1, 2, 4 or 8, no more than waves
    int groups;          // units of a key-value head
    bool by_unit;  // there are no more units than parts: cuts are listed by unit, else by the part they begin in
    Cut *cut;      // [parts]
    float2 *ml;    // [2 parts][16 wide] maximum (of scores times scale log2 e) and sum of weights
    float *o;      // [2 parts][16 wide][D]
};

// Chunks, tiles and the 16 keys of a product begin at multiples of 16, so that each of the latter
// lies in one page
__device__ __forceinline__ int first_chunk(const AttnDims &d, int len) { return first_key(d, len - 1) & ~15; }
__device__ __forceinline__ int chunks_of(const AttnDims &d, int len)
{
    const int span = len - first_chunk(d, len);
    return span <= CHUNK ? 1 : (span + CHUNK - 1) / CHUNK;
}

template <typename T, int D> struct Tile {
    static constexpr int KT = sizeof(T) == 2 && D <= 128 ? 32 : 16;  // keys
    static constexpr int NT = KT / 16, NC = D / 32, ND = D / 16;
    static constexpr int WAVES = waves_of(sizeof(T) == 4, D);
    static constexpr int PER_SIMD = WAVES == 8 ? 2 : 1;  // waves
    static constexpr int V = Vec16<T>::n, LINE = D / V;  // values of a vector of 16 bytes, vectors of a row
    static constexpr int NV = KT * LINE / 64;            // vectors of V a lane moves
    static constexpr int GV = 16 * LINE / 64;            // of 16 rows
    static_assert(GV * 64 == 16 * LINE, "16 rows are whole vectors of a wave");
    // Rows of V lie in LDS without gaps; vector x of a row stands at place x ^ swap of its row, which lets a
    // read meet every bank once: 16 bits, 2 vectors of 8 rows; fp32, 4 vectors of rows that are 4 apart.
    // FOLD: rows until the banks repeat.
    static constexpr int FOLD = LINE % 16 == 0 ? 1 : LINE % 8 == 0 ? 2 : 4;
    static constexpr int UNIT = sizeof(T) == 4 ? 4 : 2, APART = sizeof(T) == 4 ? 4 : 1;
    static constexpr int SHIFT = FOLD > APART ? FOLD : APART, KINDS = 16 / UNIT / FOLD > 0 ? 16 / UNIT / FOLD : 1;
    static __device__ __forceinline__ int swap(int row) { return (row / SHIFT) % KINDS * UNIT; }
    static_assert(LINE % (KINDS * UNIT) == 0 && 16 % (SHIFT * KINDS) == 0, "within a row, and the same 16 rows further");
    static constexpr int OP = D + 4;  // of O in LDS
    static constexpr int BYTES = 2 * KT * D * sizeof(T) > 16 * OP * 4 ? 2 * KT * D * sizeof(T) : 16 * OP * 4;
};

// o += V^T w of a tile, its weights in two parts.  KT = 16 takes products of half the depth.
typedef short s4 __attribute__((ext_vector_type(4)));
typedef short s8 __attribute__((ext_vector_type(8)));
__device__ __forceinline__ f4 mma16(_Float16 __attribute__((ext_vector_type(4))) a, _Float16 __attribute__((ext_vector_type(4))) b, f4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x16f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f4 mma16(bf16 __attribute__((ext_vector_type(4))) a, bf16 __attribute__((ext_vector_type(4))) b, f4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(s4, a), __builtin_bit_cast(s4, b), c, 0, 0, 0);
}
template <typename T, int D>
__device__ __forceinline__ void weigh(const T *v, const float *w, int lane, f4 (&o)[D / 16])
{
    typedef Mat<T> MT;
    typedef T t4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) s4 lds_s4;
    const int row = 4 * (lane >> 4) + ((lane & 15) >> 2), ch = 4 * (lane & 3);
    const T *rows = v + row * D + ch % 8;
    auto at = [&](int t) { return rows + (((16 * t + ch) / 8) ^ Tile<T, D>::swap(row)) * 8; };
    if constexpr (Tile<T, D>::NT == 2) {
        typename MT::frag p[2], f[D / 16];
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = w[i];
        split8<T, 2>(x, p);
#pragma unroll
        for (int t = 0; t < D / 16; ++t) {
            const s4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)at(t));
            const s4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)(at(t) + 16 * D));
            f[t] = __builtin_bit_cast(typename MT::frag, (s8)__builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
        }
        __builtin_amdgcn_sched_barrier(0);  // no load is given registers of an operand in use
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int t = 0; t < D / 16; ++t) o[t] = MT::mma(f[t], p[i], o[t]);
    } else {
        T part[2][4];
        t4 p[2], f[D / 16];
        split<T, 2, 4>(w, part);
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i / 4][i % 4] = part[i / 4][i % 4];
#pragma unroll
        for (int t = 0; t < D / 16; ++t)
            f[t] = __builtin_bit_cast(t4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)at(t)));
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int t = 0; t < D / 16; ++t) o[t] = mma16(f[t], p[i], o[t]);
    }
}
template <int D>
__device__ __forceinline__ void weigh(const float *v, const float *w, int lane, f4 (&o)[D / 16])
{
    const int row = 4 * (lane >> 4), ch = lane & 15;  // (four rows share their places)
    const float *rows = v + row * D + ch % 4;
    float f[D / 16][4];
#pragma unroll
    for (int t = 0; t < D / 16; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) f[t][i] = rows[i * D + (((16 * t + ch) / 4) ^ Tile<float, D>::swap(row)) * 4];
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

// a / b of numbers that nearly always fit in 32 bits
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b)
{
    return ((uint64_t)(a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

template <typename T, int D, bool WIDE>
__global__ __launch_bounds__((Tile<T, D>::WAVES * 64), (Tile<T, D>::PER_SIMD)) void step_kernel(AttnDims d, StepArgs s)
{
    constexpr int WAVES = Tile<T, D>::WAVES, BLOCK = 64 * WAVES;
    typedef Mat<T> MT;
    typedef typename MT::frag frag;
    typedef Tile<T, D> TL;
    typedef typename Vec16<T>::type vec;
    constexpr int KT = TL::KT, NT = TL::NT, NC = TL::NC, ND = TL::ND, NV = TL::NV, V = TL::V;
    __shared__ __attribute__((aligned(1024))) char lds[WAVES * TL::BYTES];
    __shared__ float sm[WAVES][16], sl[WAVES][16];
    __shared__ int64_t s_wave[WAVES], s_base;
    __shared__ int s_n;
    const int tid = threadIdx.x, lane = tid & 63, gq = lane >> 4, c = lane & 15;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int units = d.KV * s.groups;  // of a sequence
    // the wave's tile of query heads, and its place among the waves that have it
    const int wide = WIDE ? s.wide : 1, log_wide = WIDE ? s.log_wide : 0;
    const int qt = w & (wide - 1), team = w >> log_wide, teams = WAVES >> log_wide;

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
    const int64_t quantum = quotient(total + gridDim.x - 1, gridDim.x);
    int64_t pos = blockIdx.x * quantum;
    const int64_t stop = pos + quantum < total ? pos + quantum : total;
    if (pos >= total) {
        if (tid == 0 && !s.by_unit) s.cut[blockIdx.x].pieces = 0;
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
    }
    __syncthreads();
    int64_t base = s_base;
    int n = scalar(s_n);

    T *sv = reinterpret_cast<T *>(lds + w * TL::BYTES);
    float *so = reinterpret_cast<float *>(lds + w * TL::BYTES);
    const unsigned lds_v = (unsigned)(uintptr_t)(__attribute__((address_space(3))) void *)sv;
    const float cs = d.scale * 1.44269504f;

    while (pos < stop) {
        const int len = kv_bound(d, s.a.kv_len, n), low = first_key(d, len - 1), nc = chunks_of(d, len);
        const int64_t local = pos - base;
        if (local >= (int64_t)nc * units) {
            base += (int64_t)nc * units;
            ++n;
            continue;
        }
        const int unit = (int)quotient(local, nc), ch = (int)(local - (int64_t)unit * nc);
        const int count = stop - pos < nc - ch ? (int)(stop - pos) : nc - ch;
        const int kh = unit / s.groups, head0 = kh * d.g + (unit - kh * s.groups) * 16 * wide;
        const int rows = (kh + 1) * d.g - head0 < 16 * wide ? (kh + 1) * d.g - head0 : 16 * wide;
        const int begin = first_chunk(d, len) + ch * CHUNK;
        const int end = ch + count < nc ? begin + count * CHUNK : len;

        // ---- queries: column c of the products ----
        frag qf[NC];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            qf[i] = frag(0);
            if (16 * qt + c < rows) {
                const T *p = static_cast<const T *>(s.a.q) + (int64_t)n * d.q_stride + (int64_t)(head0 + 16 * qt + c) * D + 32 * i + 8 * gq;
                qf[i] = *reinterpret_cast<const typename Frag16<T>::type *>(p);
            }
        }
        const bool whole = count == nc;
        constexpr int NR = (16 * (D / 4) + BLOCK - 1) / BLOCK;
        typename Quad<T>::t4 gate[NR] = {};
        auto ask_gates = [&](int first, int tid) {  // of 16 rows
            if (!whole || !s.a.gate) return;
#pragma unroll
            for (int u = 0; u < NR; ++u) {
                const int i = u * BLOCK + tid, r = i / (D / 4);
                if (r < 16 && first + r < rows) gate[u] = gate_of<T>(d, s.a, n, head0 + first + r, (i - r * (D / 4)) * 4);
            }
        };
        ask_gates(0, tid);
        f4 o[ND];
#pragma unroll
        for (int t = 0; t < ND; ++t) o[t] = f4(0.f);
        float m = -INFINITY, l = 0.f;

        const int32_t *table = s.a.table + (int64_t)n * d.table_pages;
        const int64_t head_at = (int64_t)kh * d.page * D;
        const T *K = static_cast<const T *>(s.a.k_cache) + head_at, *Vc = static_cast<const T *>(s.a.v_cache) + head_at;
        frag kf[NT][NC];
        // lane t < NT: the page of keys k0 + 16 t.. (behind the end: of the last one), and where they lie
        const int mine = 16 * (lane & (NT - 1));
        int page = 0;
        auto ask = [&](int k0) {
            const int key = k0 + mine;
            page = table[(unsigned)(key < end ? key : end - 1) >> d.log_page];
        };
        auto once = [&](const typename Frag16<T>::type *p) -> frag {
            if constexpr (WIDE) return *p;
            else return __builtin_nontemporal_load(p);
        };
        auto load = [&](int k0, int buf) {
            const int64_t at = page_bound(d, page) * d.page_stride + ((k0 + mine) & (d.page - 1)) * D;
            int64_t from[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t)
                from[t] = (uint64_t)(unsigned)__builtin_amdgcn_readlane((int)(at >> 32), t) << 32 | (unsigned)__builtin_amdgcn_readlane((int)at, t);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int t = i / TL::GV, x = i * 64 + lane, r = x / TL::LINE;
                copy_to_lds<!WIDE>(Vc + from[t], (unsigned)(((r - 16 * t) * D + ((x - r * TL::LINE) ^ TL::swap(r)) * V) * sizeof(T)),
                            lds_v + buf * (int)(KT * D * sizeof(T)) + i * 1024);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const T *p = K + from[t];
#pragma unroll
                for (int i = 0; i < NC; ++i)
                    kf[t][i] = once(reinterpret_cast<const typename Frag16<T>::type *>(p + (unsigned)(c * D + 8 * gq) + 32 * i));
            }
        };
        int k0 = 16 * qt < rows ? begin + team * KT : end, buf = 0;
        const int STEP = teams * KT;
        if (k0 < end) {
            ask(k0);
            load(k0, 0);
            ask(k0 + STEP);
        }
        for (; k0 < end; k0 += STEP, buf ^= 1) {
            wait_vmem_all();  // this tile's V has come
            __asm__ volatile("" ::: "memory");
            T *v = sv + buf * (KT * D);
            const bool cut = k0 + KT > end || k0 < low;
            if (cut) {  // V of keys that are not seen as zeros, whatever the cache holds
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int x = i * 64 + lane, key = k0 + x / TL::LINE;
                    if (key < low || key >= end) st16(v + x * V, vec(0));
                }
            }
            f4 sc[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                sc[t] = f4(0.f);
#pragma unroll
                for (int i = 0; i < NC; ++i) sc[t] = MT::mma(kf[t][i], qf[i], sc[t]);
            }
            if (cut) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = k0 + 16 * t + 4 * gq + i;
                        sc[t][i] = key >= low && key < end ? sc[t][i] : -INFINITY;
                    }
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
                load(k0 + STEP, buf ^ 1);
                ask(k0 + 2 * STEP);
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
            if constexpr (sizeof(T) == 2) weigh<T, D>(v, wt, lane, o);
            else weigh<D>(v, wt, lane, o);
        }

        // ---- the waves' sums joined ----
        l = sum_of_groups(l);
        __syncthreads();  // V has been read
        if (gq == 0) {
            sm[w][c] = m;
            sl[w][c] = l;
        }
#pragma unroll
        for (int t = 0; t < ND; ++t) *reinterpret_cast<f4 *>(so + c * TL::OP + 16 * t + 4 * gq) = o[t];
        __syncthreads();
        const int64_t slot = 2 * (int64_t)blockIdx.x + (ch == 0);
        if (tid == 0 && (s.by_unit ? ch == 0 : pos + count == stop)) {
            const int64_t later = ch == 0 ? nc - count : 0;
            s.cut[s.by_unit ? n * units + unit : (int)blockIdx.x] =
                Cut{n, unit, (int)blockIdx.x, later == 0 ? 0 : 1 + (int)quotient(later + quantum - 1, quantum)};
        }
        int own = tid;
#ifdef __HIP_DEVICE_COMPILE__
        if (WIDE) __asm__("" : "+v"(own));  // (what is derived from it would be kept through the tiles)
#endif
#pragma unroll 1
        for (int first = 0; first < (WIDE ? rows : 1); first += 16) {  // the rows of a tile, from the waves that had it
            if (first > 0) ask_gates(first, own);
#pragma unroll
            for (int u = 0; u < NR; ++u) {
                const int i = u * BLOCK + own, r = i / (D / 4), col = (i - r * (D / 4)) * 4;
                if (r >= 16 || first + r >= rows) break;
                float big = -INFINITY, lsum = 0.f;
                f4 sum = f4(0.f);
                auto most = [&](int v) { big = fmaxf(big, sm[v][r]); };
                auto add = [&](int v) {
                    const float f = __builtin_amdgcn_exp2f(sm[v][r] - (big == -INFINITY ? 0.f : big));
                    lsum += f * sl[v][r];
                    sum += f * *reinterpret_cast<const f4 *>(reinterpret_cast<const float *>(lds + v * TL::BYTES) + r * TL::OP + col);
                };
                if constexpr (WIDE) {
                    for (int v = first / 16; v < WAVES; v += wide) most(v);
                    for (int v = first / 16; v < WAVES; v += wide) add(v);
                } else {
#pragma unroll
                    for (int v = 0; v < WAVES; ++v) most(v);
#pragma unroll
                    for (int v = 0; v < WAVES; ++v) add(v);
                }
                if (whole) {
                    finish<T>(d, s.a, n, head0 + first + r, col, sum, inverse_sum(lsum), gate[u]);
                } else {
                    const int64_t row = slot * 16 * wide + first + r;
                    *reinterpret_cast<f4 *>(s.o + row * D + col) = sum;
                    if (col == 0) s.ml[row] = make_float2(big, lsum);
                }
            }
        }
        __syncthreads();  // LDS is free for the next segment
        pos += count;
    }
}

// The units that are cut: a block a unit and 64 quadruples of its rows' channels; each of its waves joins
// every fourth piece, BATCH at a time.
constexpr int JOIN = 4, BATCH = 8;
template <typename T, int D>
__global__ __launch_bounds__(64 * JOIN) void join_kernel(AttnDims d, StepArgs s)
{
    __shared__ f4 so[JOIN][64];
    __shared__ float2 sml[JOIN][64];
    const Cut cut = s.cut[blockIdx.x];
    if (cut.pieces == 0) return;
    const int kh = cut.unit / s.groups, head0 = kh * d.g + (cut.unit - kh * s.groups) * 16 * s.wide;
    const int w = scalar(threadIdx.x >> 6), lane = threadIdx.x & 63, i = blockIdx.y * 64 + lane;
    const int r = i / (D / 4), col = (i - r * (D / 4)) * 4;
    const bool in = r < 16 * s.wide && head0 + r < (kh + 1) * d.g;
    typename Quad<T>::t4 gate = {};
    if (in && s.a.gate && w == 0) gate = gate_of<T>(d, s.a, cut.n, head0 + r, col);
    float m = -INFINITY, l = 0.f;
    f4 o = f4(0.f);
    for (int p0 = w; in && p0 < cut.pieces; p0 += JOIN * BATCH) {
        float2 ml[BATCH];
        f4 x[BATCH];
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            const int p = p0 + u * JOIN;
            ml[u] = make_float2(-INFINITY, 0.f);
            x[u] = f4(0.f);
            if (p >= cut.pieces) continue;
            // the first piece is the end of its part, the others begin in theirs
            const int64_t row = (int64_t)(p == 0 ? 2 * cut.first + 1 : 2 * (cut.first + p)) * 16 * s.wide + r;
            ml[u] = s.ml[row];
            x[u] = *reinterpret_cast<const f4 *>(s.o + row * D + col);
        }
        join<BATCH>(ml, x, m, l, o);
    }
    so[w][lane] = o;
    sml[w][lane] = make_float2(m, l);
    __syncthreads();
    if (w != 0 || !in) return;
    float big = m;
#pragma unroll
    for (int u = 1; u < JOIN; ++u) big = fmaxf(big, sml[u][lane].x);
    const float big0 = big == -INFINITY ? 0.f : big;
    l = 0.f;
    o = f4(0.f);
#pragma unroll
    for (int u = 0; u < JOIN; ++u) {
        const float f = __builtin_amdgcn_exp2f(sml[u][lane].x - big0);
        l += f * sml[u][lane].y;
        o += f * so[u][lane];
    }
    finish<T>(d, s.a, cut.n, head0 + r, col, o, inverse_sum(l), gate);
}

struct Plan {
    int wide, log_wide, groups, parts;
    int64_t units;
    bool may_cut;
    size_t cut, ml, o;  // bytes
    size_t bytes() const { return cut + ml + o; }
};

Plan plan_of(const gdn_attn_shape &s)
{
    const AttnDims d = attn_dims(s);
    Plan p;
    const int tiles = (d.g + 15) / 16, waves = waves_of(s.io_dtype == GDN_F32, d.D);
    for (p.wide = 1, p.log_wide = 0; p.wide < tiles && p.wide < waves; p.wide <<= 1) ++p.log_wide;
    p.groups = (tiles + p.wide - 1) / p.wide;
    const int64_t span = (int64_t)d.window + 15 < d.max_kv ? d.window + 15 : d.max_kv;
    p.units = (int64_t)d.n_seq * d.KV * p.groups;
    const int64_t most = p.units * (span <= CHUNK ? 1 : (span + CHUNK - 1) / CHUNK);
    p.parts = (int)(most < PARTS_MAX ? most : PARTS_MAX);
    p.may_cut = span > CHUNK;
    p.cut = ((size_t)p.parts * sizeof(Cut) + 255) / 256 * 256;
    p.ml = p.may_cut ? (size_t)p.parts * 32 * p.wide * sizeof(float2) : 0;
    p.o = p.may_cut ? (size_t)p.parts * 32 * p.wide * d.D * sizeof(float) : 0;
    return p;
}

template <typename T, int D>
void launch_step_t(const AttnDims &d, const AttnArgs &a, const Plan &p, hipStream_t st)
{
    char *ws = static_cast<char *>(a.ws);
    const bool by_unit = p.units <= p.parts;
    const StepArgs s{a, p.wide, p.log_wide, p.groups, by_unit, reinterpret_cast<Cut *>(ws), reinterpret_cast<float2 *>(ws + p.cut),
                     reinterpret_cast<float *>(ws + p.cut + p.ml)};
    hipLaunchKernelGGL((p.wide > 1 ? step_kernel<T, D, true> : step_kernel<T, D, false>), dim3(p.parts), dim3(64 * Tile<T, D>::WAVES), 0, st, d, s);
    if (p.may_cut && p.parts > 1)
        hipLaunchKernelGGL((join_kernel<T, D>), dim3(by_unit ? (int)p.units : p.parts - 1, ((d.g < 16 * p.wide ? d.g : 16 * p.wide) * (D / 4) + 63) / 64),
                           dim3(64 * JOIN), 0, st, d, s);
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
