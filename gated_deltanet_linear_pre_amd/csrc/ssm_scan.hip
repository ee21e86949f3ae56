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
// every segment's own end state from zero and its decay, a small one runs over
// the segments of a sequence and leaves the state each starts from, and the
// third walks all segments at once for the outputs.
//
// gfx950 mapping.  A block of 4 waves takes one (segment, head, 64 state rows
// p); wave w owns rows 16w..16w+15 of them, S in its accumulators as [n][p]
// tiles of 16 x 16 (N/4 registers a lane).  The tile rows are numbered so that
// lane (g, p) holds n = 32j + 8g + 0..7, which is at once the operand layout
// of S in S C^T: the state never moves.  B, C and x of a chunk lie in LDS,
// padded by 16 bytes a row (16-byte column reads of 16 rows then touch every
// bank once); x^T and B^T are read by the transposing LDS reads.  The waves
// share M: wave w forms its t tile w and writes it to LDS as an operand.  The
// next chunk's rows are loaded to registers while this one is computed.
//
// Precision.  bf16 (and fp16, fp32) inputs enter the products as they are.  The
// fp32 operands (S, M and the weighted x) are split into parts of the matrix
// type whose products are summed in fp32:
//   bf16: 3 parts (24 bits) for the state, and for S and M where y is fp32; 2
//         parts (16 bits, an error of 2^-18 of each term) where y is bf16,
//         whose own rounding is 2^-9;
//   fp16: 2 parts (22 bits), scaled by a power of two to the largest value of
//         the row or column that shares a contraction, as fp16's range asks;
//   fp32: one part, on the fp32 matrix instructions.
#include "ssm_device.h"
#include "ssm_internal.h"

namespace gdn {

namespace {

typedef float f4 __attribute__((ext_vector_type(4)));

// ---- matrix operands: 8 values of a 32-deep contraction a lane -------------
template <typename T> struct Mat;
template <> struct Mat<bf16> {
    typedef bf16 frag __attribute__((ext_vector_type(8)));
    static constexpr int Q = 64, STATE_PARTS = 3;
    static constexpr bool scaled = false;
    static __device__ __forceinline__ f4 mma(frag a, frag b, f4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
template <> struct Mat<_Float16> {
    typedef _Float16 frag __attribute__((ext_vector_type(8)));
    static constexpr int Q = 64, STATE_PARTS = 2;
    static constexpr bool scaled = true;
    static __device__ __forceinline__ f4 mma(frag a, frag b, f4 c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};
// fp32: eight 4-deep products; product i contracts value i of every lane group
template <> struct Mat<float> {
    typedef float frag __attribute__((ext_vector_type(8)));
    static constexpr int Q = 32, STATE_PARTS = 1;
    static constexpr bool scaled = false;
    static __device__ __forceinline__ f4 mma(frag a, frag b, f4 c)
    {
#pragma unroll
        for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
        return c;
    }
};

// v as a sum of PARTS operands
template <typename TI, int PARTS>
__device__ __forceinline__ void split(const float (&v)[8], typename Mat<TI>::frag (&out)[PARTS])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float r = v[i];
#pragma unroll
        for (int p = 0; p < PARTS; ++p) {
            const TI h = (TI)r;
            out[p][i] = h;
            r -= (float)h;
        }
    }
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

// Transposed operand: lane (g, r) gets rows row0 + 8g + 0..7 of one column,
// column r of the 16 that the four column quads col(q) = 4 columns each make
// up.  16-bit: two transposing reads, in which lane i of 16 addresses row i/4
// and quad i%4 and receives column i of the 4 rows.
template <typename T, typename Col>
__device__ __forceinline__ typename Mat<T>::frag col8(const T *base, int pitch, int row0, int lane, Col col)
{
    const int g = lane >> 4, c = lane & 15;
    typedef short s4 __attribute__((ext_vector_type(4)));
    typedef short s8 __attribute__((ext_vector_type(8)));
    typedef __attribute__((address_space(3))) s4 lds_s4;
    const T *p = base + (row0 + 8 * g + (c >> 2)) * pitch + col(c & 3);
    const s4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)(p));
    const s4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4 *)(p + 4 * pitch));
    return __builtin_bit_cast(typename Mat<T>::frag, (s8)__builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}
template <typename Col>
__device__ __forceinline__ Mat<float>::frag col8(const float *base, int pitch, int row0, int lane, Col col)
{
    const int g = lane >> 4, c = lane & 15;
    const float *p = base + (row0 + 8 * g) * pitch + col(c >> 2) + (c & 3);
    Mat<float>::frag v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = p[i * pitch];
    return v;
}

// Power of two that brings `most` (>= 0) to 2^13..2^14, and its inverse:
// products with it are exact.  Non-finite values stay so.
__device__ __forceinline__ void scale_of(float most, float &up, float &down)
{
    int k = 14 - __builtin_amdgcn_frexp_expf(most);
    k = k < -100 ? -100 : k > 100 ? 100 : k;
    up = __int_as_float((127 + k) << 23);
    down = __int_as_float((127 - k) << 23);
}
// the largest of the four lanes that share lane & 15
__device__ __forceinline__ float max_of_groups(float x)
{
    x = fmaxf(x, __shfl_xor(x, 16, 64));
    return fmaxf(x, __shfl_xor(x, 32, 64));
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

template <typename TI, int N, int PARTS, bool OUT> struct __attribute__((aligned(16))) ScanShared {
    static constexpr int Q = Mat<TI>::Q, PAD = 16 / sizeof(TI);
    static constexpr int NP = N + PAD, XP = 64 + PAD, MP = Q + PAD;
    TI B[Q][NP];
    TI X[Q][XP];
    TI C[OUT ? Q : 1][NP];
    TI M[OUT ? PARTS : 1][OUT ? Q : 1][MP];
    float2 lam[BATCH];           // L_t in two floats
    float dt[BATCH], E[BATCH];   // dt_t, exp(L_t)
    float W[BATCH];              // exp(L_Q - L_t) dt_t
    float alpha[BATCH / Q];      // exp(L_Q)
    double total[BATCH / Q];     // L_Q
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
};

// OUT: the outputs (and the end state of sequences of one segment); else the
// segments' own end states and decays.  PARTS: parts of S and M.
template <typename TI, typename TO, int N, int PARTS, bool OUT>
__global__ __launch_bounds__(256, N == 256 ? 1 : 2) void ssm_chunk_kernel(SsmDims d, ScanArgsT a)
{
    typedef Mat<TI> MT;
    typedef typename MT::frag frag;
    typedef ScanShared<TI, N, PARTS, OUT> Shared;
    constexpr int Q = MT::Q, SP = MT::STATE_PARTS, J = N / 32, TT = Q / 16, KK = Q / 32;
    constexpr int V = Vec16<TI>::n;
    typedef typename Vec16<TI>::type vec;
    constexpr int NB = Q * N / V / 256 > 0 ? Q * N / V / 256 : 1;  // vectors of B (and C) a thread moves
    constexpr int NX = Q * 64 / V / 256;
    __shared__ Shared sh;

    SeqTile st;
    const int64_t slot = (int64_t)blockIdx.z * gridDim.y + blockIdx.y;
    if (slot >= d.T / a.tile + d.n_seq) return;
    if (!find_tile(a.cu, d.n_seq, d.T, a.tile, (int)slot, st)) return;
    const int len = st.end - st.begin;
    const bool single = len <= a.tile;
    if (!OUT && single) return;
    const int pt_n = (d.P + 63) / 64;
    const int h = blockIdx.x / pt_n, pt = blockIdx.x - h * pt_n;
    const int grp = h / d.hg;
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, g = lane >> 4, c = lane & 15;
    const int p0 = pt * 64 + w * 16;      // of this wave
    const bool mine = p0 < d.P;           // (a wave past P only helps with loads and M)
    const int cols = d.P - pt * 64 < 64 ? d.P - pt * 64 : 64;
    const int first = st.c * a.tile;      // in the sequence
    const int n_tok = len - first < a.tile ? len - first : a.tile;
    const TI *xrow = static_cast<const TI *>(a.xbc) + (int64_t)(st.begin + first) * d.C;
    const TI *dtp = static_cast<const TI *>(a.dt) + (int64_t)(st.begin + first) * d.dt_stride + h;
    const int xc = h * d.P + pt * 64, bc = d.H * d.P + grp * N, cc = bc + d.G * N;

    // ---- state: lane (g, p = c), n = 32j + 8g + 4a + i
    f4 S[J][2];
    const int64_t head_at = ((int64_t)h * d.P + p0 + c) * N + 8 * g;
    const int64_t seq_size = (int64_t)d.H * d.P * N;
    const float *S0 = nullptr;
    if (OUT && mine) {
        if (!single) S0 = a.seg_state + slot * seq_size + head_at;
        else if (a.state) S0 = a.state + st.n * seq_size + head_at;
    }
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int q = 0; q < 2; ++q)
            S[j][q] = S0 ? *reinterpret_cast<const f4 *>(S0 + 32 * j + 4 * q) : f4(0.f);

    const float neg_a = -expf(a.A_log[h]), dt_bias = a.dt_bias[h], Dh = OUT && a.D ? a.D[h] : 0.f;
    double total = 0.0;  // log decay of the segment

    // ---- rows of the next chunk, in registers (zero past the end)
    vec rB[NB], rC[OUT ? NB : 1], rX[NX];
    auto fetch = [&](int t0) {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int at = i * 256 + tid, row = at / (N / V), col = at % (N / V) * V;
            const bool in = row < Q && t0 + row < n_tok;
            const TI *p = xrow + (int64_t)(t0 + row) * d.C + col;
            rB[i] = in ? ld16(p + bc) : vec(TI(0));
            if (OUT) rC[i] = in ? ld16(p + cc) : vec(TI(0));
        }
#pragma unroll
        for (int i = 0; i < NX; ++i) {
            const int at = i * 256 + tid, row = at / (64 / V), col = at % (64 / V) * V;
            const bool in = t0 + row < n_tok && col < cols;
            rX[i] = in ? ld16(xrow + (int64_t)(t0 + row) * d.C + xc + col) : vec(TI(0));
        }
    };
    fetch(0);
    TI raw = tid < n_tok ? dtp[tid * d.dt_stride] : TI(0);

    for (int t0 = 0; t0 < n_tok; t0 += Q) {
        if (t0) lds_sync();  // every wave is done with the last chunk
        const int bt = t0 & (BATCH - 1);
        if (bt == 0) {
            // decays of the next BATCH tokens: thread i takes token t0 + i, the
            // sums run over the Q lanes of its chunk
            const bool in = t0 + tid < n_tok;
            float dt = 0.f, lam = 0.f;
            if (in) step_size((float)raw, dt_bias, neg_a, d.dt_min, d.dt_max, dt, lam);
            double L = lam;
#pragma unroll
            for (int m = 1; m < Q; m <<= 1) {
                const double o = __shfl_up(L, m, Q);
                if ((lane & (Q - 1)) >= m) L += o;
            }
            const double LQ = __shfl(L, Q - 1, Q);
            const float hi = (float)L;
            sh.lam[tid] = make_float2(hi, (float)(L - (double)hi));
            sh.dt[tid] = dt;
            sh.E[tid] = expf(hi);
            sh.W[tid] = expf((float)(LQ - L)) * dt;
            if ((lane & (Q - 1)) == 0) {
                sh.alpha[tid / Q] = expf((float)LQ);
                sh.total[tid / Q] = LQ;
            }
            const int nt = t0 + BATCH + tid;
            raw = nt < n_tok ? dtp[nt * d.dt_stride] : TI(0);
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int at = i * 256 + tid, row = at / (N / V), col = at % (N / V) * V;
            if (row < Q) {
                st16(&sh.B[row][col], rB[i]);
                if (OUT) st16(&sh.C[row][col], rC[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < NX; ++i) {
            const int at = i * 256 + tid, row = at / (64 / V), col = at % (64 / V) * V;
            st16(&sh.X[row][col], rX[i]);
        }
        if (t0 + Q < n_tok) fetch(t0 + Q);
        lds_sync();

        const int rows = n_tok - t0 < Q ? n_tok - t0 : Q;  // (the others are zero)
        // Each product below loads all its operands from LDS, then issues its
        // matrix instructions, and its results are taken before the next
        // product's loads: no load is given registers of an operand in use.
        if (OUT && w < TT) {
            // ---- M's rows t of tile w: D = B C^T has rows s, lane (g, t = c)
            frag cf[J], bf[TT][J];
#pragma unroll
            for (int j = 0; j < J; ++j) cf[j] = row8(&sh.C[16 * w + c][32 * j + 8 * g]);
#pragma unroll
            for (int s = 0; s < TT; ++s)
#pragma unroll
                for (int j = 0; j < J; ++j) bf[s][j] = row8(&sh.B[16 * s + c][32 * j + 8 * g]);
            const float2 lt = sh.lam[bt + 16 * w + c];
            float2 ls[TT][4];
            float ds[TT][4];
#pragma unroll
            for (int s = 0; s < TT; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    ls[s][i] = sh.lam[bt + 16 * s + 4 * g + i];
                    ds[s][i] = sh.dt[bt + 16 * s + 4 * g + i];
                }
            __builtin_amdgcn_sched_barrier(0);
            f4 dd[TT];
#pragma unroll
            for (int s = 0; s < TT; ++s) dd[s] = f4(0.f);
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int s = 0; s < TT; ++s) dd[s] = MT::mma(bf[s][j], cf[j], dd[s]);
            float m[TT][4], most = 0.f;
#pragma unroll
            for (int s = 0; s < TT; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int si = 16 * s + 4 * g + i, ti = 16 * w + c;
                    const float e = exp_fast((lt.x - ls[s][i].x) + (lt.y - ls[s][i].y)) * ds[s][i];
                    float v = si <= ti ? dd[s][i] * e : 0.f;
                    if (si == ti) v += Dh;
                    m[s][i] = v;
                    most = fmaxf(most, fabsf(v));
                }
            float up = 1.f, down = 1.f;
            if (MT::scaled) {
                scale_of(max_of_groups(most), up, down);
                if (g == 0) sh.mscale[16 * w + c] = down;
            }
#pragma unroll
            for (int s = 0; s < TT; ++s) {
                TI o[PARTS][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float r = MT::scaled ? m[s][i] * up : m[s][i];
#pragma unroll
                    for (int p = 0; p < PARTS; ++p) {
                        o[p][i] = (TI)r;
                        r -= (float)o[p][i];
                    }
                }
#pragma unroll
                for (int p = 0; p < PARTS; ++p) {
                    typedef TI t4 __attribute__((ext_vector_type(4)));
                    const t4 v = {o[p][0], o[p][1], o[p][2], o[p][3]};
                    *reinterpret_cast<t4 *>(&sh.M[p][16 * w + c][16 * s + 4 * g]) = v;
                }
            }
        }

        // ---- y^T = S C^T: rows p, lane (g, t = c); then exp(L_t)
        f4 acc[TT];
        if (OUT && mine) {
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
            float sup = 1.f, sdown = 1.f, rdown[4] = {1.f, 1.f, 1.f, 1.f};
            if (MT::scaled) {
                float most = 0.f;
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int i = 0; i < 8; ++i) most = fmaxf(most, fabsf(S[j][i >> 2][i & 3]));
                scale_of(max_of_groups(most), sup, sdown);  // of row p = c
#pragma unroll
                for (int i = 0; i < 4; ++i) rdown[i] = __shfl(sdown, 4 * g + i, 64);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < J; ++j) {
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = MT::scaled ? S[j][i >> 2][i & 3] * sup : S[j][i >> 2][i & 3];
                frag sp[PARTS];
                split<TI, PARTS>(v, sp);
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

        if (OUT) lds_sync();  // M is complete
        if (mine) {
            frag xf[KK];
#pragma unroll
            for (int k = 0; k < KK; ++k) xf[k] = col8(&sh.X[0][0], Shared::XP, 32 * k, lane, [&](int q) { return 16 * w + 4 * q; });
            if (OUT) {
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
                __builtin_amdgcn_sched_barrier(0);
                if (MT::scaled) {
#pragma unroll
                    for (int t = 0; t < TT; ++t) acc[t] *= 1.0f / md[t];  // (a power of two: exact)
                }
#pragma unroll
                for (int k = 0; k < KK; ++k)
#pragma unroll
                    for (int p = 0; p < PARTS; ++p)
#pragma unroll
                        for (int t = 2 * k; t < TT; ++t) acc[t] = MT::mma(xf[k], mf[p][t][k], acc[t]);
                TO *yp = static_cast<TO *>(a.y) + ((int64_t)(st.begin + first + t0) * d.H + h) * d.P + p0 + 4 * g;
                typedef TO o4 __attribute__((ext_vector_type(4)));
                o4 o[TT];
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    const f4 v = MT::scaled ? acc[t] * md[t] : acc[t];
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[t][i] = (TO)v[i];
                    __asm__ volatile("" : "+v"(o[t]));  // (taken here, not where it is stored)
                }
#pragma unroll
                for (int t = 0; t < TT; ++t)
                    if (16 * t + c < rows) *reinterpret_cast<o4 *>(yp + (int64_t)(16 * t + c) * d.H * d.P) = o[t];
                __builtin_amdgcn_sched_barrier(0);
            }
            // ---- S <- alpha S + B^T (W x)
            if (!OUT || t0 + Q < n_tok || (single && a.state_out)) {
                frag bf[J][2][KK];
                float wt[KK][8];
                const float alpha = sh.alpha[bt / Q];
#pragma unroll
                for (int k = 0; k < KK; ++k)
#pragma unroll
                    for (int i = 0; i < 8; ++i) wt[k][i] = sh.W[bt + 32 * k + 8 * g + i];
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int k = 0; k < KK; ++k)
                            bf[j][q][k] = col8(&sh.B[0][0], Shared::NP, 32 * k, lane, [&](int r) { return 32 * j + 8 * r + 4 * q; });
                float u[KK][8], most = 0.f;
#pragma unroll
                for (int k = 0; k < KK; ++k)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        u[k][i] = (float)xf[k][i] * wt[k][i];
                        most = fmaxf(most, fabsf(u[k][i]));
                    }
                float up = 1.f, down = 1.f;
                if (MT::scaled) {
                    scale_of(max_of_groups(most), up, down);
#pragma unroll
                    for (int k = 0; k < KK; ++k)
#pragma unroll
                        for (int i = 0; i < 8; ++i) u[k][i] *= up;
                }
                frag uf[KK][SP];
#pragma unroll
                for (int k = 0; k < KK; ++k) split<TI, SP>(u[k], uf[k]);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        f4 z = MT::scaled ? f4(0.f) : S[j][q] * alpha;
#pragma unroll
                        for (int k = 0; k < KK; ++k)
#pragma unroll
                            for (int p = 0; p < SP; ++p) z = MT::mma(bf[j][q][k], uf[k][p], z);
                        if (MT::scaled) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) S[j][q][i] = fmaf(z[i], down, alpha * S[j][q][i]);
                        } else {
                            S[j][q] = z;
                        }
                    }
            }
        }
        if (!OUT) total += sh.total[bt / Q];
    }

    if (!mine) return;
    float *to = nullptr;
    if (!OUT) to = a.seg_state + slot * seq_size + head_at;
    else if (single && a.state_out) to = a.state_out + st.n * seq_size + head_at;
    if (to) {
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int q = 0; q < 2; ++q) *reinterpret_cast<f4 *>(to + 32 * j + 4 * q) = S[j][q];
    }
    if (!OUT && tid == 0 && pt == 0) a.seg_decay[slot * d.H + h] = expf((float)total);
}

// Over the segments of a sequence: the state each starts from replaces its own
// end state, and the last one's end is the sequence's.  One float4 a thread.
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
    for (int s = 0; s < segs; ++s) {
        const f4 own = *reinterpret_cast<const f4 *>(p + s * seq_size);
        *reinterpret_cast<f4 *>(p + s * seq_size) = S;
        S = S * dec[(int64_t)s * d.H] + own;
    }
    if (a.state_out) *reinterpret_cast<f4 *>(a.state_out + n * seq_size + at) = S;
}

// Tokens of a segment: as many as give the launch about SEG_BLOCKS blocks (two
// on each of the 256 CUs), in whole batches of decays.
constexpr int SEG_BLOCKS = 512;
int segment_tokens(const SsmDims &d)
{
    const int64_t blocks = (int64_t)d.H * ((d.P + 63) / 64);
    int64_t tile = (d.T * blocks + SEG_BLOCKS - 1) / SEG_BLOCKS;
    tile = (tile + BATCH - 1) / BATCH * BATCH;
    return (int)(tile < BATCH ? BATCH : tile > (1 << 27) ? 1 << 27 : tile);
}

size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

} // namespace

size_t ssm_scan_workspace_bytes(const gdn_ssm_shape &s)
{
    const SsmDims d = ssm_dims(s);
    const int tile = segment_tokens(d);
    if (s.max_T <= tile) return 0;
    const size_t slots = (size_t)(d.T / tile + d.n_seq);
    return round256(slots * d.H * d.P * d.N * sizeof(float)) + round256(slots * d.H * sizeof(float));
}

template <typename TI, typename TO, int N>
static void launch_scan_t(const SsmDims &d, const SsmScanArgs &a, bool segments, hipStream_t st)
{
    constexpr int PARTS = sizeof(TI) == 4 ? 1 : Mat<TI>::scaled ? 2 : sizeof(TO) == 4 ? 3 : 2;
    ScanArgsT t{a.cu, a.xbc, a.dt, a.A_log, a.dt_bias, a.D, a.state, a.state_out, a.y, nullptr, nullptr, segment_tokens(d)};
    const int64_t slots = d.T / t.tile + d.n_seq;
    const int pt_n = (d.P + 63) / 64;
    auto grid = [](int64_t x, int64_t yz) {
        const int64_t y = yz < 32768 ? yz : 32768;
        return dim3((unsigned)x, (unsigned)y, (unsigned)((yz + y - 1) / y));
    };
    if (segments) {
        t.seg_state = static_cast<float *>(a.ws);
        t.seg_decay = reinterpret_cast<float *>(static_cast<char *>(a.ws) + round256((size_t)slots * d.H * d.P * N * sizeof(float)));
        hipLaunchKernelGGL((ssm_chunk_kernel<TI, TI, N, 1, false>), grid((int64_t)d.H * pt_n, slots), dim3(256), 0, st, d, t);
        hipLaunchKernelGGL(ssm_segment_kernel, grid(((int64_t)d.H * d.P * N / 4 + 255) / 256, d.n_seq), dim3(256), 0, st, d, t);
    }
    hipLaunchKernelGGL((ssm_chunk_kernel<TI, TO, N, PARTS, true>), grid((int64_t)d.H * pt_n, slots), dim3(256), 0, st, d, t);
}

template <typename TI, typename TO>
static void launch_scan_n(const SsmDims &d, const SsmScanArgs &a, bool segments, hipStream_t st)
{
    if (d.N == 32) launch_scan_t<TI, TO, 32>(d, a, segments, st);
    else if (d.N == 64) launch_scan_t<TI, TO, 64>(d, a, segments, st);
    else if (d.N == 128) launch_scan_t<TI, TO, 128>(d, a, segments, st);
    else launch_scan_t<TI, TO, 256>(d, a, segments, st);
}

hipError_t launch_ssm_scan(const gdn_ssm_shape &s, const SsmScanArgs &a, hipStream_t st)
{
    const SsmDims d = ssm_dims(s);
    const bool segments = ssm_scan_workspace_bytes(s) > 0;
    GDN_SSM_IO(s.io_dtype,
        if (s.out_dtype == GDN_F32) launch_scan_n<TI, float>(d, a, segments, st);
        else launch_scan_n<TI, TI>(d, a, segments, st);)
    return hipGetLastError();
}

} // namespace gdn
