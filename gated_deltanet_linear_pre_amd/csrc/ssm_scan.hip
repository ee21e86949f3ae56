// ssm_scan.hip -- the selective state space recurrence over whole prompts.
//
//   dt = clamp(softplus(dt_raw + dt_bias)), lam = -exp(A_log) dt
//   S <- exp(lam) S + dt x B^T,  y = S C + D x      per token, S the P x N state of a head
//
// Chunks.  With L_t the sum of lam up to token t of a chunk of Q tokens and S
// the state at its start, the recurrence is
//   y_t = exp(L_t) S C_t + sum_{s<=t} M_ts x_s,   M_ts = (C_t . B_s) exp(L_t - L_s) dt_s  (+ D on the diagonal)
//   S'  = exp(L_Q) S + sum_s exp(L_Q - L_s) dt_s x_s B_s^T
// three matrix products a chunk, every exponent <= 0.  The sums L are formed in
// 64 bits and kept as two floats, so that differences of them are exact to
// fp32 however far the decays have run.
//
// Segments.  A sequence's chunks follow one another, so a launch with few
// (sequence, head) pairs cuts sequences into segments: a first kernel forms
// every segment's own end state from zero and its decay, and a last one walks
// all segments at once for the outputs.  Between them a small kernel runs over
// the segments of a sequence and leaves the state each starts from; where a
// sequence has few, the last kernel's blocks do that as they start.
//
// gfx950 mapping.  A block of 4 waves takes one (segment, head, 64 state rows
// p); wave w owns rows 16w..16w+15 of them, S in its accumulators as [n][p]
// tiles of 16 x 16 (N/4 registers a lane).  The tile rows are numbered so that
// lane (g, p) holds n = 32j + 8g + 0..7, which is at once the operand layout
// of S in S C^T: the state never moves.  B, C and x of a chunk lie in LDS (their
// pitches: ScanShared); x^T and B^T are read by the transposing LDS reads.  The
// waves share M: each forms some of its 16 x 16 tiles (form_m's callers) and
// writes them to LDS as operands.  The next chunk's rows are loaded to registers
// while this one is computed.
//
// Precision.  bf16 (and fp16, fp32) inputs enter the products as they are.  The
// fp32 operands (S, M and the weighted x) are split into parts of the matrix
// type whose products are summed in fp32, whatever y's type:
//   bf16: 3 parts, 24 bits.  (2 parts are off by up to 2^-17 of a term, and 0.1% of
//         the outputs of bf16 came out one step from those of an fp32 evaluation:
//         1.0e-4 of y.  The third part costs 332 -> 411 us on the packed batch);
//   fp16: 2 parts, off by at most 2^-23 of a value (an fp32 rounding: 2^-24) or
//         2^-38 of the largest value of the row or column that shares a
//         contraction, to which all are scaled by a power of two, as fp16's range
//         asks.  That is below what the sums of an fp32 evaluation lose;
//   fp32: one part, on the fp32 matrix instructions.
//
// Bound.  At 16 bits by what a wave can issue between the barriers of a chunk: with
// three parts, N = 128, 57 matrix instructions of 16 cycles and 450 vector ones of 4
// a wave and chunk of 32 tokens, 2700 cycles, of which three waves share a SIMD:
// the 7800 cycles that a chunk of the packed batch takes.  The matrix pipe is busy
// 23% of the time, HBM moves 1.4 TB/s.  fp32 is bound by the rate of its matrix
// instructions, an eighth of the 16-bit one.  Measured, 64 heads of 64, N = 128:
// 2048 tokens bf16 51 us (end states 15, segments 8, outputs 33), fp16 49 (14, 8,
// 30), fp32 98 (31, 8, 67); 27135 tokens in 4 sequences bf16 417 us (end states 89).
#include <type_traits>

#include "ssm_device.h"
#include "ssm_internal.h"

namespace gdn {

namespace {

typedef float f4 __attribute__((ext_vector_type(4)));

// ---- matrix operands: 8 values of a 32-deep contraction a lane -------------
template <typename T> struct Mat;
template <> struct Mat<bf16> {
    typedef bf16 frag __attribute__((ext_vector_type(8)));
    static constexpr int PARTS = 3;
    static constexpr bool scaled = false;
    static __device__ __forceinline__ f4 mma(frag a, frag b, f4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
template <> struct Mat<_Float16> {
    typedef _Float16 frag __attribute__((ext_vector_type(8)));
    static constexpr int PARTS = 2;
    static constexpr bool scaled = true;
    static __device__ __forceinline__ f4 mma(frag a, frag b, f4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};
// fp32: eight 4-deep products; product i contracts value i of every lane group
template <> struct Mat<float> {
    typedef float frag __attribute__((ext_vector_type(8)));
    static constexpr int PARTS = 1;
    static constexpr bool scaled = false;
    static __device__ __forceinline__ f4 mma(frag a, frag b, f4 c)
    {
#pragma unroll
        for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
        return c;
    }
};

// Tokens of a chunk; PARTS: those of M in LDS.  64 halve the times that S is split
// into operands; 32 leave LDS for two blocks on a CU with N = 256 or fp32, and for
// three with three parts of S and M.  Measured: N = 256, bf16 to fp32, 2005 tokens of
// 32 heads of 128: 80 us by 32, 104 by 64; N = 128, 64 heads of 64, bf16, 2048 tokens
// 51 and 60, 27135 packed tokens 417 and 487 (but 512 tokens 24.4 and 24.0); fp16,
// 8192 tokens: 107 and 93.
template <typename T, int N, int PARTS> constexpr int chunk_tokens()
{
    return sizeof(T) == 4 || N == 256 || (N == 128 && PARTS == 3) ? 32 : 64;
}

// v = sum of PARTS values of the matrix type, each the nearest to what the
// ones before it leave.  Two values at a time: their conversion and packing
// are one instruction.
template <typename T> struct Pair {
    typedef T t2 __attribute__((ext_vector_type(2)));
    typedef float f2 __attribute__((ext_vector_type(2)));
    static __device__ __forceinline__ t2 narrow(f2 v) { return __builtin_convertvector(v, t2); }
    static __device__ __forceinline__ f2 widen(t2 v) { return f2{(float)v[0], (float)v[1]}; }
};
template <typename T, int PARTS, int NV>
__device__ __forceinline__ void split(const float *v, T (*out)[NV])
{
#pragma unroll
    for (int i = 0; i < NV; i += 2) {
        typename Pair<T>::f2 r = {v[i], v[i + 1]};
#pragma unroll
        for (int p = 0; p < PARTS; ++p) {
            const typename Pair<T>::t2 h = Pair<T>::narrow(r);
            out[p][i] = h[0];
            out[p][i + 1] = h[1];
            if (p + 1 < PARTS) {
                const typename Pair<T>::f2 w = Pair<T>::widen(h);
                r[0] -= w[0];
                r[1] -= w[1];
            }
        }
    }
}
template <typename T, int PARTS>
__device__ __forceinline__ void split8(const float (&v)[8], typename Mat<T>::frag (&out)[PARTS])
{
    T o[PARTS][8];
    split<T, PARTS, 8>(v, o);
#pragma unroll
    for (int p = 0; p < PARTS; ++p)
#pragma unroll
        for (int i = 0; i < 8; ++i) out[p][i] = o[p][i];
}

// 8 consecutive values of an LDS row
template <typename T>
__device__ __forceinline__ typename Mat<T>::frag row8(const T *p)
{
    return *reinterpret_cast<const typename Mat<T>::frag *>(p);
}
template <>
__device__ __forceinline__ Mat<float>::frag row8<float>(const float *p)
{
    const f4 a = *reinterpret_cast<const f4 *>(p), b = *reinterpret_cast<const f4 *>(p + 4);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// 4 values of a row of B, whose rows start on 8 bytes (see ScanShared)
template <typename T> struct BQuad {
    typedef T t4 __attribute__((ext_vector_type(4)));
    typedef t4 type __attribute__((aligned(8)));
};
// A 16-byte vector of a row of B (columns col..) to its places
__device__ __forceinline__ void store_b(float *row, int col, Vec16<float>::type v)
{
    *reinterpret_cast<BQuad<float>::type *>(row + (col & ~31) + (col & 4) * 4 + (col & 24) / 2) = v;
}
template <typename T>
__device__ __forceinline__ void store_b(T *row, int col, typename Vec16<T>::type v)
{
    typedef typename BQuad<T>::type quad;
    T *p = row + (col & ~31) + (col & 24) / 2;
    *reinterpret_cast<quad *>(p) = __builtin_shufflevector(v, v, 0, 1, 2, 3);
    *reinterpret_cast<quad *>(p + 16) = __builtin_shufflevector(v, v, 4, 5, 6, 7);
}
// n = 32j + 8g + 0..7 of a permuted row of B
template <typename T>
__device__ __forceinline__ typename Mat<T>::frag rowb(const T *row, int j, int g)
{
    typedef typename BQuad<T>::type quad;
    const typename BQuad<T>::t4 a = *reinterpret_cast<const quad *>(row + 32 * j + 4 * g);
    const typename BQuad<T>::t4 b = *reinterpret_cast<const quad *>(row + 32 * j + 16 + 4 * g);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Transposed operand: lane (g, r) gets rows row0 + 8g + 0..7 of column
// col0 + r.  16-bit: two transposing reads, in which lane i of 16
// addresses row i/4 and columns 4(i%4).. and receives column i of the 4 rows.
template <typename T>
__device__ __forceinline__ typename Mat<T>::frag col8(const T *base, int pitch, int row0, int col0, int lane)
{
    const int g = lane >> 4, c = lane & 15;
    typedef short s4 __attribute__((ext_vector_type(4)));
    typedef short s8 __attribute__((ext_vector_type(8)));
    typedef __attribute__((address_space(3))) s4 lds_s4;
    const T *p = base + (row0 + 8 * g + (c >> 2)) * pitch + col0 + 4 * (c & 3);
    const s4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)(p));
    const s4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)(p + 4 * pitch));
    return __builtin_bit_cast(typename Mat<T>::frag, (s8)__builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}
template <>
__device__ __forceinline__ Mat<float>::frag col8<float>(const float *base, int pitch, int row0, int col0, int lane)
{
    const int g = lane >> 4, c = lane & 15;
    const float *p = base + (row0 + 8 * g) * pitch + col0 + c;
    Mat<float>::frag v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = p[i * pitch];
    return v;
}

// ---- values that are not finite: all bits of the exponent set ----------------
template <typename T> struct Bits {
    typedef unsigned short u;
    static constexpr unsigned short INF = std::is_same<T, _Float16>::value ? 0x7C00 : 0x7F80, VALUE = 0x7FFF;
};
template <> struct Bits<float> {
    typedef unsigned u;
    static constexpr unsigned INF = 0x7F800000, VALUE = 0x7FFFFFFF;
};
template <typename T, int KK>
__device__ __forceinline__ bool any_not_finite(const typename Mat<T>::frag (&x)[KK])
{
    typedef typename Bits<T>::u u;
    typedef u u2 __attribute__((ext_vector_type(2)));
    typedef u u8 __attribute__((ext_vector_type(8)));
    u2 most = u2(0);
#pragma unroll
    for (int k = 0; k < KK; ++k) {
        const u8 b = __builtin_bit_cast(u8, x[k]) & Bits<T>::VALUE;
#pragma unroll
        for (int i = 0; i < 8; i += 2) most = __builtin_elementwise_max(most, u2{b[i], b[i + 1]});
    }
    return most[0] >= Bits<T>::INF || most[1] >= Bits<T>::INF;
}
template <typename T>
__device__ __forceinline__ bool not_finite(T v)
{
    return (__builtin_bit_cast(typename Bits<T>::u, v) & Bits<T>::VALUE) >= Bits<T>::INF;
}

// the inverse of a power of two
__device__ __forceinline__ float inverse(float x) { return __int_as_float((254 << 23) - __float_as_int(x)); }
// Power of two that brings `most` (>= 0) to 2^13..2^14, at most 2^40 (smaller
// values than 2^-26 keep an error of 2^-65), and its inverse: products with
// it are exact.  Non-finite values stay so.
__device__ __forceinline__ void scale_of(float most, float &up, float &down)
{
    int k = 14 - __builtin_amdgcn_frexp_expf(most);  // (-114 at least)
    k = k > 40 ? 40 : k;
    up = __int_as_float((127 + k) << 23);
    down = inverse(up);
}
// The same for the x that S gathers, whose scale S takes: at most 2^86 / size, with
// S below 2^14 size, so that a scaled S stays below 2^100.  (size is a power of two;
// up to 2^46, S up to 2^60, nothing is held back.)
__device__ __forceinline__ void scale_beside(float most, float size, float &up, float &down)
{
    scale_of(most, up, down);
    const float cap = __uint_as_float((340u << 23) - __float_as_uint(fmaxf(size, 0x1p46f)));
    up = fminf(up, cap);
    down = inverse(up);
}
// the largest of the four lanes that share lane & 15 (x >= 0): a lane-half
// swap of x with itself leaves the two halves' values side by side, and a
// swap of 16-lane rows likewise
__device__ __forceinline__ float max_of_groups(float x)
{
    const unsigned u = __float_as_uint(x);
    const auto h = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const unsigned v = __float_as_uint(fmaxf(__uint_as_float(h[0]), __uint_as_float(h[1])));
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// ---- 64-bit values across lanes ---------------------------------------------
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp64(double x)  // 0 where the source lane or the row is left out
{
    const unsigned long long u = __builtin_bit_cast(unsigned long long, x);
    const unsigned lo = __builtin_amdgcn_update_dpp(0, (int)(unsigned)u, CTRL, ROWS, 0xF, false);
    const unsigned hi = __builtin_amdgcn_update_dpp(0, (int)(unsigned)(u >> 32), CTRL, ROWS, 0xF, false);
    return __builtin_bit_cast(double, (unsigned long long)hi << 32 | lo);
}
// Sum of the lanes up to this one, over runs of W (32 or 64) lanes: shifts by
// 1, 2, 4, 8 inside the rows of 16, then the last lane of the row before, then
// that of the half before
template <int W>
__device__ __forceinline__ double scan64(double x)
{
    x += dpp64<0x111, 0xF>(x);
    x += dpp64<0x112, 0xF>(x);
    x += dpp64<0x114, 0xF>(x);
    x += dpp64<0x118, 0xF>(x);
    x += dpp64<0x142, 0xA>(x);
    if (W == 64) x += dpp64<0x143, 0xC>(x);
    return x;
}
// lane `at` of this lane's run of W lanes
template <int W>
__device__ __forceinline__ double lane64(double x, int at, int lane)
{
    const unsigned long long u = __builtin_bit_cast(unsigned long long, x);
    auto pick = [&](int l) {
        const unsigned lo = __builtin_amdgcn_readlane((int)(unsigned)u, l);
        const unsigned hi = __builtin_amdgcn_readlane((int)(unsigned)(u >> 32), l);
        return __builtin_bit_cast(double, (unsigned long long)hi << 32 | lo);
    };
    return W == 64 || lane < 32 ? pick(at) : pick(at + 32);
}

// Barrier that orders LDS only: global loads and stores in flight stay so.
__device__ __forceinline__ void lds_sync()
{
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __asm__ volatile("" ::: "memory");
}

constexpr int BATCH = 256;  // tokens whose decays are formed at a time, one a thread

// Rows of B are permuted: the 32 values n = 32j + 8q + 4a + i stand at
// 32j + 16a + 4q + i, so that the 16 columns of a state tile (j, a) are
// consecutive for the transposing reads, and 40 bytes longer than N (a row
// read takes two 8-byte halves: 16 rows then start in 16 different bank pairs).
// Rows of C and X are 32 bytes longer, those of M (also written in 8-byte
// columns) 16.  Measured in cycles of an instruction, 4 waves reading: 16-byte
// row reads 4.1 at 32 bytes, 8.1 at 16; transposing reads 4.1; 8-byte ones 4.8.
template <typename TI, int N, int PARTS> struct __attribute__((aligned(16))) ScanShared {
    static constexpr int Q = chunk_tokens<TI, N, PARTS>(), E16 = 16 / sizeof(TI), REFS = Q / 16 - 1;
    static constexpr int BP = N + 40 / sizeof(TI), CP = N + 2 * E16, XP = 64 + 2 * E16, MP = Q + E16;
    static_assert(BP * sizeof(TI) % alignof(typename BQuad<TI>::type) == 0, "rows of B start where its vectors may");
    static_assert(CP * sizeof(TI) % 16 == 0 && XP * sizeof(TI) % 16 == 0 && MP * sizeof(TI) % 16 == 0, "16-byte vectors");
    TI C[Q][CP];
    TI X[Q][XP];
    TI M[PARTS][Q][MP];
    TI B[Q][BP];
    float2 lam[BATCH];           // L_t in two floats
    float dt[BATCH], E[BATCH];   // dt_t, exp(L_t)
    float W[BATCH];              // exp(L_Q - L_t) dt_t
    float F[BATCH];              // exp(L_t - L_r), r the first token of t's tile of 16
    float G[REFS][BATCH];        // exp(L_r - L_t) dt_t, r the first token of a later tile
    float alpha[BATCH / Q];      // exp(L_Q)
    float mscale[Q];             // fp16: 1 / scale of M's row t
};

struct ScanArgsT {
    const int32_t *cu;
    const void *xbc, *dt;
    const float *A_log, *dt_bias, *D, *state;
    float *state_out;
    void *y;
    float *seg_state;  // [slot][H][P][N]
    float *seg_decay;  // [slot][H]
    int tile;          // tokens of a segment
    bool joined;       // seg_state holds start states (else the segments' own end states)
    bool copied;       // the last segment's place holds a copy of the sequence's state
};

// A block's part of the work: segment b.slot of a sequence, rows 64 b.pt.. of
// the state of head b.h
struct Part {
    int64_t slot, row;       // row: the segment's first token row
    int n, h, pt, n_tok;     // sequence, ..., tokens of the segment
    int c, after;            // segments of the sequence before it and after it
    int cols;                // rows of the state that are there, at most 64
    int xc, bc, cc;          // first channels of x, B and C
    bool single, last;       // the sequence is one segment; this is its last one
};
__device__ __forceinline__ bool locate(const SsmDims &d, const ScanArgsT &a, Part &b)
{
    SeqTile st;
    b.slot = (int64_t)blockIdx.z * gridDim.y + blockIdx.y;
    if (b.slot >= d.T / a.tile + d.n_seq) return false;
    if (!find_tile(a.cu, d.n_seq, d.T, a.tile, (int)b.slot, st)) return false;
    const int len = st.end - st.begin, first = st.c * a.tile, pt_n = (d.P + 63) / 64;
    b.n = st.n;
    b.c = st.c;
    b.after = len > first ? (len - first - 1) / a.tile : 0;
    b.single = len <= a.tile;
    b.last = len - first <= a.tile;
    b.n_tok = b.last ? len - first : a.tile;
    b.row = st.begin + first;
    // blocks go to the 8 XCDs in turn: neighbouring heads, which share B and C,
    // go to one XCD and its L2; in another order for each segment, or a CU would
    // get two blocks of one head, which a slow decay makes long in the end states
    // (packed batch 425 -> 417 us)
    const unsigned each = gridDim.x / 8;
    const int bx = gridDim.x % 8 ? blockIdx.x : blockIdx.x % 8 * each + (blockIdx.x / 8 + (unsigned)b.slot) % each;
    b.h = bx / pt_n;
    b.pt = bx - b.h * pt_n;
    b.cols = d.P - b.pt * 64 < 64 ? d.P - b.pt * 64 : 64;
    const int grp = b.h / d.hg;
    b.xc = b.h * d.P + b.pt * 64;
    b.bc = d.H * d.P + grp * d.N;
    b.cc = b.bc + d.G * d.N;
    return true;
}

// The outputs of every segment, and the end state of the last one of a sequence.
template <typename TI, typename TO, int N>
__global__ __launch_bounds__(256, N == 128 && Mat<TI>::PARTS == 3 ? 3 : 2) void ssm_chunk_kernel(SsmDims d, ScanArgsT a)
{
    typedef Mat<TI> MT;
    typedef typename MT::frag frag;
    constexpr int PARTS = MT::PARTS;
    typedef ScanShared<TI, N, PARTS> Shared;
    constexpr int Q = chunk_tokens<TI, N, PARTS>(), J = N / 32, TT = Q / 16, KK = Q / 32;
    constexpr int V = Vec16<TI>::n;
    typedef typename Vec16<TI>::type vec;
    constexpr int NB = Q * N / V / 256;  // vectors of B (and C) a thread moves
    constexpr int NX = Q * 64 / V / 256;
    __shared__ Shared sh;

    Part b;
    if (!locate(d, a, b)) return;
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, c = lane & 15;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int p0 = b.pt * 64 + w * 16;  // of this wave
    const bool mine = p0 < d.P;         // (a wave past P only helps with loads and M)
    const bool keep = b.last && a.state_out;  // the end state is asked for
    const int n_tok = b.n_tok, h = b.h;
    const TI *xrow = static_cast<const TI *>(a.xbc) + b.row * d.C;
    const TI *dtp = static_cast<const TI *>(a.dt) + b.row * d.dt_stride + h;

    // ---- state: lane (g, p = c), n = 32j + 8g + 4a + i.  fp16: S stands
    // for S * sdown, a power of two of row p that the last chunk's products needed.
    f4 S[J][2];
    float sdown = 1.f;
    const int64_t head_at = ((int64_t)h * d.P + p0 + c) * N + 8 * g;
    const int64_t seq_size = (int64_t)d.H * d.P * N;
    const float neg_a = -expf(a.A_log[h]), dt_bias = a.dt_bias[h], Dh = a.D ? a.D[h] : 0.f;

    // ---- rows of a chunk in registers: vector i of a thread is row
    // i*RB + tid / (N/V) of B and C, i*RX + tid / (64/V) of X
    constexpr int RB = 256 * V / N, RX = 256 * V / 64;
    vec rB[NB], rC[NB], rX[NX];
    const int brow = tid / (N / V), bcol = tid % (N / V) * V, xr = tid / (64 / V), xcol = tid % (64 / V) * V;
    // (byte offsets of 32 bits beside a uniform base: one register for all rows)
    const uint32_t ob = ((uint32_t)brow * d.C + bcol) * sizeof(TI);
    const uint32_t ox = ((uint32_t)xr * d.C + (xcol < b.cols ? xcol : 0)) * sizeof(TI);
    const uint32_t oy = ((uint32_t)c * d.H * d.P + 4 * g) * sizeof(TO);
    auto fetch = [&](int t0) {
        const TI *base = xrow + (int64_t)t0 * d.C;
        if (t0 + Q <= n_tok) {
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                rB[i] = ld16_at(base + b.bc + (int64_t)i * RB * d.C, ob);
                rC[i] = ld16_at(base + b.cc + (int64_t)i * RB * d.C, ob);
            }
#pragma unroll
            for (int i = 0; i < NX; ++i) rX[i] = ld16_at(base + b.xc + (int64_t)i * RX * d.C, ox);
        } else {  // rows past the end are zero
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const bool in = t0 + i * RB + brow < n_tok;
                rB[i] = in ? ld16_at(base + b.bc + (int64_t)i * RB * d.C, ob) : vec(TI(0));
                rC[i] = in ? ld16_at(base + b.cc + (int64_t)i * RB * d.C, ob) : vec(TI(0));
            }
#pragma unroll
            for (int i = 0; i < NX; ++i)
                rX[i] = t0 + i * RX + xr < n_tok ? ld16_at(base + b.xc + (int64_t)i * RX * d.C, ox) : vec(TI(0));
        }
    };
    TI raw = tid < n_tok ? dtp[tid * d.dt_stride] : TI(0);
    fetch(0);
    const float *S0 = nullptr;
    if (mine) {
        if (!b.single && a.joined) S0 = a.seg_state + b.slot * seq_size + head_at;
        else if (!b.single && a.copied) S0 = a.seg_state + (b.slot + b.after) * seq_size + head_at;
        else if (a.state) S0 = a.state + b.n * seq_size + head_at;
    }
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int q = 0; q < 2; ++q)
            S[j][q] = S0 ? *reinterpret_cast<const f4 *>(S0 + 32 * j + 4 * q) : f4(0.f);
    if (mine && !a.joined && b.c) {  // over the segments before this one
        constexpr int JG = J < 4 ? J : 4, AHEAD = 3;  // loads in flight
        const float *own0 = a.seg_state + (b.slot - b.c) * seq_size + head_at, *dec = a.seg_decay + (b.slot - b.c) * d.H + h;
#pragma unroll
        for (int j0 = 0; j0 < J; j0 += JG)
            for (int s0 = 0; s0 < b.c; s0 += AHEAD) {
                f4 own[AHEAD][JG][2];
                float decay[AHEAD];
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    const int s = s0 + i < b.c ? s0 + i : b.c - 1;
                    decay[i] = dec[(int64_t)s * d.H];
#pragma unroll
                    for (int j = 0; j < JG; ++j)
#pragma unroll
                        for (int q = 0; q < 2; ++q)
                            own[i][j][q] = *reinterpret_cast<const f4 *>(own0 + s * seq_size + 32 * (j0 + j) + 4 * q);
                }
#pragma unroll
                for (int i = 0; i < AHEAD; ++i)
                    if (s0 + i < b.c) {
#pragma unroll
                        for (int j = 0; j < JG; ++j)
#pragma unroll
                            for (int q = 0; q < 2; ++q) S[j0 + j][q] = S[j0 + j][q] * decay[i] + own[i][j][q];
                    }
            }
    }

    // M's t tile of a wave: the two blocks that usually share a CU take them
    // in opposite order (tile t costs t + 1 products)
    const int mt = TT == 4 && ((b.slot * gridDim.x + blockIdx.x) >> 8 & 1) ? 3 - w : w;

    // ---- M's rows t of tile T, columns s of tiles FROM to TO - 1: D = B C^T has
    // rows s, lane (g, t = c)
    auto form_m = [&](auto tile, auto from, auto to, int bt) {
        constexpr int T = decltype(tile)::value, FROM = decltype(from)::value, TO_ = decltype(to)::value, SN = TO_ - FROM;
        constexpr int OFF = TO_ > T ? SN - 1 : SN;  // tiles below the diagonal
        frag cf[J], bf[SN][J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            cf[j] = row8(&sh.C[16 * T + c][32 * j + 8 * g]);
#pragma unroll
            for (int s = 0; s < SN; ++s) bf[s][j] = rowb(&sh.B[16 * (FROM + s) + c][0], j, g);
        }
        const float2 lt = sh.lam[bt + 16 * T + c];
        const float Ft = sh.F[bt + 16 * T + c];
        float2 ls[4];
        float ds[4];
        f4 Gs[OFF > 0 ? OFF : 1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ls[i] = sh.lam[bt + 16 * T + 4 * g + i];
            ds[i] = sh.dt[bt + 16 * T + 4 * g + i];
        }
#pragma unroll
        for (int s = 0; s < OFF; ++s) Gs[s] = *reinterpret_cast<const f4 *>(&sh.G[T > 0 ? T - 1 : 0][bt + 16 * (FROM + s) + 4 * g]);
        __builtin_amdgcn_sched_barrier(0);
        f4 dd[SN];
#pragma unroll
        for (int s = 0; s < SN; ++s) dd[s] = f4(0.f);
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int s = 0; s < SN; ++s) dd[s] = MT::mma(bf[s][j], cf[j], dd[s]);
        float most = 0.f;
#pragma unroll
        for (int s = 0; s < OFF; ++s) dd[s] = dd[s] * Gs[s] * Ft;
#pragma unroll
        for (int i = 0; i < 4 && OFF < SN; ++i) {
            const int si = 4 * g + i;
            const float v = dd[SN - 1][i] * (exp_fast((lt.x - ls[i].x) + (lt.y - ls[i].y)) * ds[i]);
            dd[SN - 1][i] = si < c ? v : si == c ? v + Dh : 0.f;
        }
        if (MT::scaled) {
#pragma unroll
            for (int s = 0; s < SN; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) most = fmaxf(most, fabsf(dd[s][i]));
            float up, down;
            scale_of(max_of_groups(most), up, down);
            if (g == 0) sh.mscale[16 * T + c] = down;
#pragma unroll
            for (int s = 0; s < SN; ++s) dd[s] *= up;
        }
#pragma unroll
        for (int s = 0; s < SN; ++s) {
            typedef TI t4 __attribute__((ext_vector_type(4)));
            const float v[4] = {dd[s][0], dd[s][1], dd[s][2], dd[s][3]};
            TI o[PARTS][4];
            split<TI, PARTS, 4>(v, o);
#pragma unroll
            for (int p = 0; p < PARTS; ++p) {
                const t4 q = {o[p][0], o[p][1], o[p][2], o[p][3]};
                *reinterpret_cast<t4 *>(&sh.M[p][16 * T + c][16 * (FROM + s) + 4 * g]) = q;
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    {  // the tiles of M above the diagonal that a 32-deep product touches
        typedef TI t4 __attribute__((ext_vector_type(4)));
        if (w < KK)
#pragma unroll
            for (int p = 0; p < PARTS; ++p)
                *reinterpret_cast<t4 *>(&sh.M[p][32 * w + c][32 * w + 16 + 4 * g]) = t4(TI(0));
    }

    for (int t0 = 0; t0 < n_tok; t0 += Q) {
        if (t0) lds_sync();  // every wave is done with the last chunk
        const int bt = t0 & (BATCH - 1);
        if (bt == 0) {
            // decays of the next BATCH tokens: thread i takes token t0 + i, the
            // sums run over the Q lanes of its chunk
            const bool in = t0 + tid < n_tok;
            float dt = 0.f, lam = 0.f;
            if (in) step_size((float)raw, dt_bias, neg_a, d.dt_min, d.dt_max, dt, lam);
            const double L = scan64<Q>(lam), LQ = lane64<Q>(L, Q - 1, lane);
            const float hi = (float)L;
            sh.lam[tid] = make_float2(hi, (float)(L - (double)hi));
            sh.dt[tid] = dt;
            sh.E[tid] = exp_fast(hi);
            const int place = lane & (Q - 1);
            double first_of_tile = lane64<Q>(L, 0, lane);
#pragma unroll
            for (int r = 1; r < TT; ++r) {
                const double Lr = lane64<Q>(L, 16 * r, lane);
                if (place >= 16 * r) first_of_tile = Lr;
                sh.G[r - 1][tid] = place < 16 * r ? exp_fast((float)(Lr - L)) * dt : 0.f;
            }
            sh.F[tid] = exp_fast((float)(L - first_of_tile));
            if (place == 0) sh.alpha[tid / Q] = exp_fast((float)LQ);
            sh.W[tid] = exp_fast((float)(LQ - L)) * dt;
            const int nt = t0 + BATCH + tid;
            raw = nt < n_tok ? dtp[nt * d.dt_stride] : TI(0);
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            store_b(&sh.B[i * RB + brow][0], bcol, rB[i]);
            st16(&sh.C[i * RB + brow][bcol], rC[i]);
        }
#pragma unroll
        for (int i = 0; i < NX; ++i) st16(&sh.X[i * RX + xr][xcol], rX[i]);
        lds_sync();

        const int rows = n_tok - t0 < Q ? n_tok - t0 : Q;  // (the others are zero)
        // Each product below loads all its operands from LDS, then issues its
        // matrix instructions, and its results are taken before the next
        // product's loads: no load is given registers of an operand in use.
        f4 acc[TT];
        float down = 1.f;  // fp16: the largest value of S's row p = c is below 2^14 down
        {
            constexpr std::integral_constant<int, 0> i0;
            constexpr std::integral_constant<int, 1> i1;
            constexpr std::integral_constant<int, 2> i2;
            constexpr std::integral_constant<int, 3> i3;
            constexpr std::integral_constant<int, 4> i4;
            if constexpr (TT == 4) {
                if (mt == 0) form_m(i0, i0, i1, bt);
                else if (mt == 1) form_m(i1, i0, i2, bt);
                else if (mt == 2) form_m(i2, i0, i3, bt);
                else form_m(i3, i0, i4, bt);
            } else if constexpr (MT::scaled) {  // a row's scale is that of all its columns
                if (mt == 0) form_m(i0, i0, i1, bt);
                else if (mt == 1) form_m(i1, i0, i2, bt);
            } else {  // a tile a wave (packed batch 423 -> 417 us)
                if (w == 0) form_m(i0, i0, i1, bt);
                else if (w == 1) form_m(i1, i0, i1, bt);
                else if (w == 2) form_m(i1, i1, i2, bt);
            }
            __builtin_amdgcn_s_setprio(2);
            if (mine) {
                // ---- y^T = S C^T: rows p, lane (g, t = c); then exp(L_t)
                frag cf[J][TT];
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int t = 0; t < TT; ++t) cf[j][t] = row8(&sh.C[16 * t + c][32 * j + 8 * g]);
                float e[TT];
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    acc[t] = f4(0.f);
                    e[t] = sh.E[bt + 16 * t + c];
                }
                float up = 1.f, rdown[4] = {1.f, 1.f, 1.f, 1.f};
                down = 1.f;
                if (MT::scaled) {
                    float most = 0.f;
#pragma unroll
                    for (int j = 0; j < J; ++j)
#pragma unroll
                        for (int i = 0; i < 8; ++i) most = fmaxf(most, fabsf(S[j][i >> 2][i & 3]));
                    scale_of(max_of_groups(most), up, down);  // of row p = c
                    down *= sdown;
#pragma unroll
                    for (int i = 0; i < 4; ++i) rdown[i] = __shfl(down, 4 * g + i, 64);
                }
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    float v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = MT::scaled ? S[j][i >> 2][i & 3] * up : S[j][i >> 2][i & 3];
                    frag sp[PARTS];
                    split8<TI, PARTS>(v, sp);
#pragma unroll
                    for (int p = 0; p < PARTS; ++p)
#pragma unroll
                        for (int t = 0; t < TT; ++t) acc[t] = MT::mma(sp[p], cf[j][t], acc[t]);
                }
#pragma unroll
                for (int t = 0; t < TT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[t][i] *= MT::scaled ? e[t] * rdown[i] : e[t];
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        fetch(t0 + Q);  // (past the end: zeros; without a branch, as the old values would live on beside it)
        frag xf[KK];
        if (mine) {
#pragma unroll
            for (int k = 0; k < KK; ++k) xf[k] = col8(&sh.X[0][0], Shared::XP, 32 * k, 16 * w, lane);
            // ---- S <- alpha S + B^T (W x)
            if (t0 + Q < n_tok || keep) {
                float wt[KK][8];
                float alpha = sh.alpha[bt / Q];
#pragma unroll
                for (int k = 0; k < KK; ++k)
#pragma unroll
                    for (int i = 0; i < 8; ++i) wt[k][i] = sh.W[bt + 32 * k + 8 * g + i];
                float u[KK][8];
#pragma unroll
                for (int k = 0; k < KK; ++k)
#pragma unroll
                    for (int i = 0; i < 8; ++i) u[k][i] = (float)xf[k][i] * wt[k][i];
                if (MT::scaled) {
                    float most = 0.f, up;
#pragma unroll
                    for (int k = 0; k < KK; ++k)
#pragma unroll
                        for (int i = 0; i < 8; ++i) most = fmaxf(most, fabsf(u[k][i]));
                    alpha *= sdown;
                    scale_beside(max_of_groups(most), down, up, sdown);
                    alpha *= up;
#pragma unroll
                    for (int k = 0; k < KK; ++k)
#pragma unroll
                        for (int i = 0; i < 8; ++i) u[k][i] *= up;
                }
                frag uf[KK][PARTS];
#pragma unroll
                for (int k = 0; k < KK; ++k) split8<TI, PARTS>(u[k], uf[k]);
                __builtin_amdgcn_sched_barrier(0);
                // (in two parts of n, which bounds the registers: at N = 128 all
                // of B^T at once takes 417 us on the packed batch of 27135 tokens
                // to 481, and 79 of the ragged one at N = 256 to 125)
                constexpr int JS = J < 2 ? J : J / 2;
#pragma unroll
                for (int j0 = 0; j0 < J; j0 += JS) {
                    frag bf[JS][2][KK];
#pragma unroll
                    for (int j = 0; j < JS; ++j)
#pragma unroll
                        for (int q = 0; q < 2; ++q)
#pragma unroll
                            for (int k = 0; k < KK; ++k)
                                bf[j][q][k] = col8(&sh.B[0][0], Shared::BP, 32 * k, 32 * (j0 + j) + 16 * q, lane);
                    __builtin_amdgcn_sched_barrier(0);
                    f4 z[JS][2];
#pragma unroll
                    for (int k = 0; k < KK; ++k)
#pragma unroll
                        for (int p = 0; p < PARTS; ++p)
#pragma unroll
                            for (int j = 0; j < JS; ++j)
#pragma unroll
                                for (int q = 0; q < 2; ++q) z[j][q] = MT::mma(bf[j][q][k], uf[k][p], k + p ? z[j][q] : f4(0.f));
#pragma unroll
                    for (int j = 0; j < JS; ++j)
#pragma unroll
                        for (int q = 0; q < 2; ++q) S[j0 + j][q] = S[j0 + j][q] * alpha + z[j][q];
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
        {
            __builtin_amdgcn_s_setprio(0);
            lds_sync();  // M is complete
            if (mine) {
                // ---- y^T += x^T M^T, and out
                frag mf[PARTS][TT][KK];
                float md[TT];
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    md[t] = MT::scaled ? sh.mscale[16 * t + c] : 1.f;
#pragma unroll
                    for (int k = 0; k < KK; ++k)
                        if (2 * k <= t) {
#pragma unroll
                            for (int p = 0; p < PARTS; ++p) mf[p][t][k] = row8(&sh.M[p][16 * t + c][32 * k + 8 * g]);
                        }
                }
                // A value of x that is not finite would meet M's zeros above the
                // diagonal, and be NaN in the tokens before its own.  It is left
                // out of the product, and its channel's outputs from it on are NaN.
                const bool odd = __builtin_amdgcn_ballot_w64(any_not_finite<TI, KK>(xf)) != 0;
                unsigned from = 0;  // the place of the first such value in channels p = 4g..4g+3, a byte each
                if (odd) {
                    int first = Q;  // of channel p = c
#pragma unroll
                    for (int k = KK - 1; k >= 0; --k)
#pragma unroll
                        for (int i = 7; i >= 0; --i)
                            if (not_finite<TI>(xf[k][i])) {
                                first = 32 * k + 8 * g + i;
                                xf[k][i] = TI(0);
                            }
                    first = min(first, __shfl_xor(first, 16, 64));
                    first = min(first, __shfl_xor(first, 32, 64));
#pragma unroll
                    for (int i = 0; i < 4; ++i) from |= (unsigned)__shfl(first, 4 * g + i, 64) << 8 * i;
                }
                __builtin_amdgcn_sched_barrier(0);
                f4 z[TT];
#pragma unroll
                for (int t = 0; t < TT; ++t) z[t] = MT::scaled ? f4(0.f) : acc[t];
#pragma unroll
                for (int k = 0; k < KK; ++k)
#pragma unroll
                    for (int p = 0; p < PARTS; ++p)
#pragma unroll
                        for (int t = 2 * k; t < TT; ++t) z[t] = MT::mma(xf[k], mf[p][t][k], z[t]);
                if (odd) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int t = 0; t < TT; ++t) z[t][i] = 16 * t + c >= (int)(from >> 8 * i & 0xFF) ? __builtin_nanf("") : z[t][i];
                }
                char *yp = reinterpret_cast<char *>(static_cast<TO *>(a.y) + ((b.row + t0) * d.H + h) * d.P + p0);
                typedef TO o4 __attribute__((ext_vector_type(4)));
                o4 o[TT];
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    const f4 v = MT::scaled ? z[t] * md[t] + acc[t] : z[t];
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[t][i] = (TO)v[i];
                    __asm__ volatile("" : "+v"(o[t]));  // (taken here, not where it is stored)
                }
#pragma unroll
                for (int t = 0; t < TT; ++t)
                    if (16 * t + c < rows) *reinterpret_cast<o4 *>(yp + (int64_t)t * 16 * d.H * d.P * sizeof(TO) + oy) = o[t];
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    }

    if (!mine) return;
    int lane_end = threadIdx.x & 63;
    __asm__ volatile("" : "+v"(lane_end));  // (the state's address is formed again, not kept)
    const int64_t end_at = ((int64_t)h * d.P + p0 + (lane_end & 15)) * N + 8 * (lane_end >> 4);
    if (keep) {
        float *to = a.state_out + b.n * seq_size + end_at;
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int q = 0; q < 2; ++q) *reinterpret_cast<f4 *>(to + 32 * j + 4 * q) = MT::scaled ? S[j][q] * sdown : S[j][q];
    }
}

// ---- the end states of all segments of a sequence but its last -------------
// S_end = sum_t exp(L_end - L_t) dt_t x_t B_t^T over a segment, from a zero state:
// one long product with no step that waits for another, so its chunks may come
// in any order.  They come from the last to the first, and a block stops where
// the decay to the segment's end has fallen below e^-110: every weight before
// that is 0 in fp32, and so is the segment's own decay.  (At the decays models
// start from, half the heads' segments of 3584 tokens end within a few hundred.)
template <typename TI, int N> struct __attribute__((aligned(16))) EndShared {
    typedef ScanShared<TI, N, 1> S;
    TI X[S::Q][S::XP];
    TI B[S::Q][S::BP];
    float W[BATCH];   // exp(L_end - L_t) dt_t
    double total[4];  // log decay of 64 tokens
};

template <typename TI, int N>
__global__ __launch_bounds__(256, 2) void ssm_end_kernel(SsmDims d, ScanArgsT a)
{
    typedef Mat<TI> MT;
    typedef typename MT::frag frag;
    typedef EndShared<TI, N> Shared;
    constexpr int PARTS = MT::PARTS;
    constexpr int Q = chunk_tokens<TI, N, 1>(), J = N / 32, KK = Q / 32;
    constexpr int V = Vec16<TI>::n, NB = Q * N / V / 256, NX = Q * 64 / V / 256;
    constexpr int RB = 256 * V / N, RX = 256 * V / 64;
    // products accumulate onto S itself, all of B^T's operands at once (fp16
    // changes S's scale between chunks; N = 256 has no registers for it)
    constexpr bool DIRECT = !MT::scaled && N <= 128;
    constexpr int JS = DIRECT || J < 2 ? J : J / 2;
    typedef typename Vec16<TI>::type vec;
    __shared__ Shared sh;

    Part b;
    if (!locate(d, a, b) || b.single) return;
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, c = lane & 15;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int p0 = b.pt * 64 + w * 16;
    const bool mine = p0 < d.P;
    if (b.last) {
        // the chunk kernel's block of this segment writes the sequence's state,
        // perhaps before those of the other segments have read it: they read this copy
        if (!a.copied || !mine) return;
        const int64_t seq_size = (int64_t)d.H * d.P * N, at = ((int64_t)b.h * d.P + p0 + c) * N + 8 * g;
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int q = 0; q < 2; ++q)
                *reinterpret_cast<f4 *>(a.seg_state + b.slot * seq_size + at + 32 * j + 4 * q) =
                    *reinterpret_cast<const f4 *>(a.state + b.n * seq_size + at + 32 * j + 4 * q);
        return;
    }
    const int n_tok = b.n_tok;
    const TI *xrow = static_cast<const TI *>(a.xbc) + b.row * d.C;
    const TI *dtp = static_cast<const TI *>(a.dt) + b.row * d.dt_stride + b.h;

    int t0 = (n_tok - 1) / Q * Q;
    const int first_raw = (t0 & ~(BATCH - 1)) + tid;
    TI raw = first_raw < n_tok ? dtp[first_raw * d.dt_stride] : TI(0);
    vec rB[NB], rX[NX];
    const int brow = tid / (N / V), bcol = tid % (N / V) * V, xr = tid / (64 / V), xcol = tid % (64 / V) * V;
    const uint32_t ob = ((uint32_t)brow * d.C + bcol) * sizeof(TI);
    const uint32_t ox = ((uint32_t)xr * d.C + (xcol < b.cols ? xcol : 0)) * sizeof(TI);
    auto fetch = [&](int t) {
        const TI *base = xrow + (int64_t)t * d.C;
        if (t + Q <= n_tok) {
#pragma unroll
            for (int i = 0; i < NB; ++i) rB[i] = ld16_at(base + b.bc + (int64_t)i * RB * d.C, ob);
#pragma unroll
            for (int i = 0; i < NX; ++i) rX[i] = ld16_at(base + b.xc + (int64_t)i * RX * d.C, ox);
        } else {  // rows past the end are zero
#pragma unroll
            for (int i = 0; i < NB; ++i)
                rB[i] = t + i * RB + brow < n_tok ? ld16_at(base + b.bc + (int64_t)i * RB * d.C, ob) : vec(TI(0));
#pragma unroll
            for (int i = 0; i < NX; ++i)
                rX[i] = t + i * RX + xr < n_tok ? ld16_at(base + b.xc + (int64_t)i * RX * d.C, ox) : vec(TI(0));
        }
    };
    fetch(t0);

    f4 S[J][2];
#pragma unroll
    for (int j = 0; j < J; ++j) S[j][0] = S[j][1] = f4(0.f);
    float sdown = 1.f, largest = 0.f;  // largest: of u in row p = c so far
    const float neg_a = -expf(a.A_log[b.h]), dt_bias = a.dt_bias[b.h];
    double after = 0.0, all = 0.0;  // log decay after this batch, and of it
    float rest[4];                  // log decay after each 64 tokens of it
    bool fresh = true, faded = false;

    for (; t0 >= 0; t0 -= Q) {
        if (!fresh) lds_sync();  // every wave is done with the last chunk
        const int bt = t0 & (BATCH - 1);
        if (fresh || bt == BATCH - Q) {
            after += all;
            float dt = 0.f, lam = 0.f;
            const int t = t0 - bt + tid;
            if (t < n_tok) step_size((float)raw, dt_bias, neg_a, d.dt_min, d.dt_max, dt, lam);
            const double L = scan64<64>(lam);
            if (lane == 63) sh.total[w] = L;
            lds_sync();
            all = 0.0;
            double to_end = after;  // after this wave's tokens
#pragma unroll
            for (int i = 3; i >= 0; --i) {
                rest[i] = (float)(after + all);
                if (i == w) to_end = after + all;
                all += sh.total[i];
            }
            sh.W[tid] = exp_fast((float)(lane64<64>(L, 63, lane) - L + to_end)) * dt;
            const int nt = t - BATCH;
            raw = nt >= 0 ? dtp[nt * d.dt_stride] : TI(0);
        }
        fresh = false;
        const int quarter = bt / 64;
        const float left = quarter == 0 ? rest[0] : quarter == 1 ? rest[1] : quarter == 2 ? rest[2] : rest[3];
        faded = left < -110.f;
        if (faded) break;
#pragma unroll
        for (int i = 0; i < NB; ++i) store_b(&sh.B[i * RB + brow][0], bcol, rB[i]);
#pragma unroll
        for (int i = 0; i < NX; ++i) st16(&sh.X[i * RX + xr][xcol], rX[i]);
        lds_sync();
        fetch(t0 >= Q ? t0 - Q : 0);  // (without a branch, see the chunk kernel)

        __builtin_amdgcn_s_setprio(2);
        if (mine) {
            frag xf[KK], bf[JS][2][KK];
            float u[KK][8];
            auto load_b = [&](int j0) {
#pragma unroll
                for (int j = 0; j < JS; ++j)
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int k = 0; k < KK; ++k)
                            bf[j][q][k] = col8(&sh.B[0][0], Shared::S::BP, 32 * k, 32 * (j0 + j) + 16 * q, lane);
            };
#pragma unroll
            for (int k = 0; k < KK; ++k) {
                xf[k] = col8(&sh.X[0][0], Shared::S::XP, 32 * k, 16 * w, lane);
#pragma unroll
                for (int i = 0; i < 8; ++i) u[k][i] = sh.W[bt + 32 * k + 8 * g + i];
            }
            load_b(0);
#pragma unroll
            for (int k = 0; k < KK; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) u[k][i] *= (float)xf[k][i];
            float scale = 1.f;  // of S before this chunk
            if (MT::scaled) {
                float most = 0.f, up;
#pragma unroll
                for (int k = 0; k < KK; ++k)
#pragma unroll
                    for (int i = 0; i < 8; ++i) most = fmaxf(most, fabsf(u[k][i]));
                scale = sdown;
                // |S| <= tokens max|u| max|B|, below 2^27 2^(e + 1) 2^16 with 2^e <= max|u|
                most = max_of_groups(most);
                largest = fmaxf(largest, most);
                const float power = __uint_as_float(__float_as_uint(largest) & 0x7F800000u);
                scale_beside(most, fminf(power, 0x1p84f) * 0x1p30f, up, sdown);
                scale *= up;
#pragma unroll
                for (int k = 0; k < KK; ++k)
#pragma unroll
                    for (int i = 0; i < 8; ++i) u[k][i] *= up;
            }
            frag uf[KK][PARTS];
#pragma unroll
            for (int k = 0; k < KK; ++k) split8<TI, PARTS>(u[k], uf[k]);
#pragma unroll
            for (int j0 = 0; j0 < J; j0 += JS) {
                if (j0) load_b(j0);
                __builtin_amdgcn_sched_barrier(0);
                f4 z[JS][2];
#pragma unroll
                for (int j = 0; j < JS; ++j)
#pragma unroll
                    for (int q = 0; q < 2; ++q) z[j][q] = DIRECT ? S[j0 + j][q] : f4(0.f);
#pragma unroll
                for (int k = 0; k < KK; ++k)
#pragma unroll
                    for (int p = 0; p < PARTS; ++p)
#pragma unroll
                        for (int j = 0; j < JS; ++j)
#pragma unroll
                            for (int q = 0; q < 2; ++q) z[j][q] = MT::mma(bf[j][q][k], uf[k][p], z[j][q]);
#pragma unroll
                for (int j = 0; j < JS; ++j)
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        S[j0 + j][q] = DIRECT ? z[j][q] : MT::scaled ? S[j0 + j][q] * scale + z[j][q] : S[j0 + j][q] + z[j][q];
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        __builtin_amdgcn_s_setprio(0);
    }

    if (tid == 0 && b.pt == 0) a.seg_decay[b.slot * d.H + b.h] = faded ? 0.f : expf((float)(after + all));
    if (!mine) return;
    float *to = a.seg_state + b.slot * ((int64_t)d.H * d.P * N) + ((int64_t)b.h * d.P + p0 + c) * N + 8 * g;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int q = 0; q < 2; ++q) *reinterpret_cast<f4 *>(to + 32 * j + 4 * q) = MT::scaled ? S[j][q] * sdown : S[j][q];
}

// Over the segments of a sequence: the state each starts from takes the place of
// its own end state.  One float4 a thread.
__global__ __launch_bounds__(256) void ssm_segment_kernel(SsmDims d, ScanArgsT a)
{
    const int64_t n = (int64_t)blockIdx.z * gridDim.y + blockIdx.y;
    if (n >= d.n_seq) return;
    const int begin = seq_bound(a.cu, n, d.T), end = seq_bound(a.cu, n + 1, d.T);
    if (end - begin <= a.tile) return;
    const int segs = (int)(((int64_t)end - begin + a.tile - 1) / a.tile);
    const int64_t seq_size = (int64_t)d.H * d.P * d.N;
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (at >= seq_size) return;
    const int h = (int)(at / ((int64_t)d.P * d.N));
    const int64_t slot0 = begin / a.tile + n;
    f4 S = a.state ? *reinterpret_cast<const f4 *>(a.state + n * seq_size + at) : f4(0.f);
    float *p = a.seg_state + slot0 * seq_size + at;
    const float *dec = a.seg_decay + slot0 * d.H + h;
    constexpr int AHEAD = 8;  // loads in flight: the stores would otherwise hold each one back
    for (int s0 = 0; s0 < segs; s0 += AHEAD) {
        f4 own[AHEAD];
        float decay[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int64_t s = s0 + i < segs - 1 ? s0 + i : segs - 2;  // (the last has no end state here)
            own[i] = *reinterpret_cast<const f4 *>(p + s * seq_size);
            decay[i] = dec[s * d.H];
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (s0 + i < segs) {
                *reinterpret_cast<f4 *>(p + (s0 + i) * seq_size) = S;
                S = S * decay[i] + own[i];
            }
    }
}

constexpr int NO_SEGMENTS = 1 << 30;  // tokens: more than a call may have

// Tokens of a segment, in whole chunks: as many as give the chip's 256 CUs two
// blocks each, which hide one another's latency; where that would leave a block
// 128 tokens or less, one block each, of at least 128.  A batch of sequences of
// up to 256 tokens is not cut: two segments cost two more kernels' latency.
// Measured, 64 heads of 64, N = 128, bf16, by blocks: 2048 tokens 256 58.8 us, 512
// 50.8, 1024 60.8; 27135 packed tokens 567, 417, 411; 1024 tokens 256 36, 512 38;
// 512 tokens 128 34, 256 24.4, 512 34; 4 sequences of 256 uncut 24.8, 512 30.8; one
// of 256 uncut 21.3, 128 22.5 (256 blocks of 64 tokens 18.9).
int segment_tokens(const SsmDims &d, int64_t max_T)
{
    const int64_t all = d.T * d.H * ((d.P + 63) / 64);  // tokens of all blocks
    auto share = [&](int64_t blocks) { return (all + blocks * 64 - 1) / (blocks * 64) * 64; };
    int64_t tile = share(512);
    if (tile <= 128) tile = share(256) < 128 ? 128 : share(256);
    if (max_T <= 256 && tile < 256) tile = 256;
    // (at the ends of the sizes a share passes 32 bits; no sequence is that long)
    return tile < NO_SEGMENTS ? (int)tile : NO_SEGMENTS;
}

// Up to this many segments of a sequence the chunk kernel's blocks run over the
// ones before theirs themselves, which costs them reads that grow with the
// segments and saves a launch.  Measured against ssm_segment_kernel, as above:
// 4 segments 24.4 and 31.2 us (512 tokens), 35.9 and 40.6 (1024), 7 39.9 and 41.3
// (1280), 48.1 and 48.4 (1792), 8 50.6 and 51.0 (2048), 16 143 and 133 (16384 of 32
// heads).
constexpr int JOIN_SEGMENTS = 7;

size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

} // namespace

size_t ssm_scan_workspace_bytes(const gdn_ssm_shape &s)
{
    const SsmDims d = ssm_dims(s);
    const int tile = segment_tokens(d, s.max_T);
    if (s.max_T <= tile) return 0;
    const size_t slots = (size_t)(d.T / tile + d.n_seq);
    return round256(slots * d.H * d.P * d.N * sizeof(float)) + round256(slots * d.H * sizeof(float));
}

template <typename TI, typename TO, int N>
static void launch_scan_t(const SsmDims &d, const SsmScanArgs &a, bool segments, int64_t max_T, hipStream_t st)
{
    ScanArgsT t{a.cu, a.xbc, a.dt, a.A_log, a.dt_bias, a.D, a.state, a.state_out, a.y, nullptr, nullptr, segment_tokens(d, max_T), false, false};
    if (!segments) t.tile = NO_SEGMENTS;  // every sequence is one segment, whatever cu_seqlens holds
    const int64_t slots = d.T / t.tile + d.n_seq;
    const int pt_n = (d.P + 63) / 64;
    auto grid = [](int64_t x, int64_t yz) {
        const int64_t y = yz < 32768 ? yz : 32768;
        return dim3((unsigned)x, (unsigned)y, (unsigned)((yz + y - 1) / y));
    };
    if (segments) {
        t.seg_state = static_cast<float *>(a.ws);
        t.seg_decay = reinterpret_cast<float *>(static_cast<char *>(a.ws) + round256((size_t)slots * d.H * d.P * N * sizeof(float)));
        t.joined = max_T > (int64_t)JOIN_SEGMENTS * t.tile;
        t.copied = !t.joined && a.state && a.state == a.state_out;
        hipLaunchKernelGGL((ssm_end_kernel<TI, N>), grid((int64_t)d.H * pt_n, slots), dim3(256), 0, st, d, t);
        if (t.joined)
            hipLaunchKernelGGL(ssm_segment_kernel, grid(((int64_t)d.H * d.P * N / 4 + 255) / 256, d.n_seq), dim3(256), 0, st, d, t);
    }
    hipLaunchKernelGGL((ssm_chunk_kernel<TI, TO, N>), grid((int64_t)d.H * pt_n, slots), dim3(256), 0, st, d, t);
}

template <typename TI, typename TO>
static void launch_scan_n(const SsmDims &d, const SsmScanArgs &a, bool segments, int64_t max_T, hipStream_t st)
{
    if (d.N == 32) launch_scan_t<TI, TO, 32>(d, a, segments, max_T, st);
    else if (d.N == 64) launch_scan_t<TI, TO, 64>(d, a, segments, max_T, st);
    else if (d.N == 128) launch_scan_t<TI, TO, 128>(d, a, segments, max_T, st);
    else launch_scan_t<TI, TO, 256>(d, a, segments, max_T, st);
}

hipError_t launch_ssm_scan(const gdn_ssm_shape &s, const SsmScanArgs &a, hipStream_t st)
{
    const SsmDims d = ssm_dims(s);
    const bool segments = ssm_scan_workspace_bytes(s) > 0;
    GDN_SSM_IO(s.io_dtype,
        if (s.out_dtype == GDN_F32) launch_scan_n<TI, float>(d, a, segments, s.max_T, st);
        else launch_scan_n<TI, TI>(d, a, segments, s.max_T, st);)
    return hipGetLastError();
}

} // namespace gdn
