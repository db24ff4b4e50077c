// la_gated_simt.cu -- the gated recurrence and its gradient on the CUDA cores,
// in fp32, for fp32 inputs and for the head sizes that the tensor-core kernels
// do not take.  The formulas stand in la_gated.h; chunks of 32 tokens.
//
// Bound by fp32 FMAs: at d_k = d_v = 128 the chunk phase of the gradient does
// about 5 x 128 x 128 x 2 + 5 x 32 x 128 x 2 flops a token for 7 x 128 x 4
// bytes.  Each product keeps a 4 x 4 tile per thread: one warp owns four rows
// (their operand is a broadcast), its lanes own columns lane + 32 m, so an
// operand read along either of its dimensions is free of bank conflicts when
// rows are an odd number of floats apart.  Prefix sums of the gates are held in
// float64: their differences, the exponents of the decays, stay exact to
// fp32 however strong the gates are.
#include <cuda_bf16.h>

#include <algorithm>

#include "la_gated.h"
#include "la_internal.h"

namespace la {
namespace {

constexpr int C = kGatedSimtChunk;
// Tiles are [.][32 NM] with NM = ceil(max(d_k, d_v) / 32), rows 32 NM + 1 apart.
constexpr int kLdC = 33;   // row stride of [C][C] tiles
constexpr int kThreads = 256;

__device__ __forceinline__ float ld1(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float ld1(const __nv_bfloat16* p, int64_t i) { return __bfloat162float(p[i]); }
__device__ __forceinline__ void st1(float* p, int64_t i, float x) { p[i] = x; }
__device__ __forceinline__ void st1(__nv_bfloat16* p, int64_t i, float x) { p[i] = __float2bfloat16_rn(x); }

__device__ __forceinline__ float decay(double x) { return exp2f(static_cast<float>(x * 1.4426950408889634)); }

// Inclusive prefix sum of the chunk's log gates at token `lane` (every warp for itself; tokens >= nv add 0).
template <typename T>
__device__ __forceinline__ float load_gate(const GatedProblem& p, int64_t row0, int nv) {
    const int lane = threadIdx.x & 31;
    float x = 0.f;
    if (p.g != nullptr && lane < nv) {
        x = ld1(static_cast<const T*>(p.g), row0 + lane);
        x = x < kGateFloor ? kGateFloor : x;
    }
    return x;
}
__device__ __forceinline__ double gate_scan(float x) {
    const int lane = threadIdx.x & 31;
    double s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    return s;
}

// Rows row0 .. row0 + nv - 1 of x [.][d] into dst [C][32 NM + 1], the rest zero.  All loads of a thread are in flight
// before the first is stored.
template <typename T, int NM>
__device__ __forceinline__ void load_tile(float* dst, const void* x, int64_t row0, int nv, int d) {
    const T* X = static_cast<const T*>(x) + row0 * d;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float v[4][NM];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            const int r = w + 8 * i, c = lane + 32 * m;
            v[i][m] = (r < nv && c < d) ? ld1(X, static_cast<int64_t>(r) * d + c) : 0.f;
        }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int m = 0; m < NM; ++m) dst[(w + 8 * i) * (32 * NM + 1) + lane + 32 * m] = v[i][m];
}

// A state [dk][dv] into dst [32 NM][32 NM + 1]; rows behind d_k and columns behind d_v zero (all enter products).
template <int NM>
__device__ __forceinline__ void load_state(float* dst, const float* src, int dk, int dv) {
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int b = 0; b < NM; ++b) {
        float v[4][NM];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                const int r = 32 * b + w + 8 * i, c = lane + 32 * m;
                v[i][m] = (r < dk && c < dv) ? src[r * dv + c] : 0.f;
            }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int m = 0; m < NM; ++m) dst[(32 * b + w + 8 * i) * (32 * NM + 1) + lane + 32 * m] = v[i][m];
    }
}

// acc[i][m] += sum_{k < K} a(4 w + i, k) b(k, lane + 32 m): 32 x 32 NM outputs over 8 warps.
template <int NM>
struct Acc {
    float x[4][NM];
};
template <int NM>
__device__ __forceinline__ void mm(Acc<NM>& acc, const float* a, int ai, int ak, const float* b, int bk, int bn, int K) {
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float* A = a + 4 * w * ai;
    const float* B = b + lane * bn;
#pragma unroll 4
    for (int k = 0; k < K; ++k) {
        float av[4], bv[NM];
#pragma unroll
        for (int i = 0; i < 4; ++i) av[i] = A[i * ai + k * ak];
#pragma unroll
        for (int m = 0; m < NM; ++m) bv[m] = B[k * bk + 32 * m * bn];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int m = 0; m < NM; ++m) acc.x[i][m] = fmaf(av[i], bv[m], acc.x[i][m]);
    }
}

// a_i . b_j over K columns, 32 x 32 outputs over 8 warps (four rows each, j = lane).
template <int NM>
__device__ __forceinline__ void scores(float (&acc)[4], const float* a, const float* b, int K) {
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = 0.f;
#pragma unroll 4
    for (int k = 0; k < K; ++k) {
        const float y = b[lane * (32 * NM + 1) + k];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = fmaf(a[(4 * w + i) * (32 * NM + 1) + k], y, acc[i]);
    }
}

template <typename T, int NM>
__device__ __forceinline__ void store_rows(void* y, int64_t row0, int nv, int d, const Acc<NM>& acc) {
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    T* Y = static_cast<T*>(y) + row0 * d;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            const int r = 4 * w + i, c = lane + 32 * m;
            if (r < nv && c < d) st1(Y, static_cast<int64_t>(r) * d + c, acc.x[i][m]);
        }
}

// ---------------------------------------------------------------------------
// State phase.  One CTA owns 32 of the d_v columns of a unit's state (a state
// column depends on no other), in registers, 4 x 4 per thread, and walks the
// chunks; the next chunk's rows are loaded while one is computed.  Forward:
// X = K, Y = V, weights e^{G_C - G_j}; for the gradient also, in the second
// half of the grid, in reverse: X = Q, Y = dO, weights e^{G_i}.  The weights go
// to Y, the smaller tile.
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(kThreads) gated_states_simt_kernel(const GatedProblem p, int col_blocks) {
    __shared__ float X[C][132];
    __shared__ float Y[C][36];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x;
    const int64_t item = blockIdx.x / col_blocks;  // [direction][unit][segment]
    const int seg = static_cast<int>(item % p.segs);
    const bool rev = item / p.segs >= p.n_units;
    const int64_t u = item / p.segs - (rev ? p.n_units : 0);
    const int c0 = static_cast<int>(blockIdx.x % col_blocks) * 32;
    const GatedUnit un = gated_unit(p, u);
    if (un.len == 0) return;
    const int r0 = 4 * (tid >> 3), n0 = c0 + 4 * (tid & 7);
    const int dk = p.dk, dv = p.dv;
    const int64_t usz = static_cast<int64_t>(dk) * dv;
    const float* in = rev ? p.dstate + u * usz : (p.state ? p.state + u * usz : (p.s0 ? p.s0 + u * usz : nullptr));
    float* out = rev ? p.dstate + u * usz : (p.state ? p.state + u * usz : nullptr);
    float* slots = static_cast<float*>(rev ? p.e_states : p.s_states);
    const int nch = gated_chunks(un.len, C);
    const int cc0 = seg * p.seg_chunks, cc1 = min(nch, cc0 + p.seg_chunks);
    if (cc0 >= cc1 || (p.sums && cc1 == nch)) return;  // (nothing starts from the last one's sum)
    if (p.segs > 1) {
        float* start = p.seg_states + item * usz;
        in = p.sums ? nullptr : start;
        out = p.sums ? start : (cc1 == nch ? out : nullptr);
    }
    float S[4][4];
    double whole = 0.0;  // log gates of the segment
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int m = 0; m < 4; ++m)
            S[i][m] = (in && r0 + i < dk && n0 + m < dv) ? in[(r0 + i) * dv + n0 + m] : 0.f;
    const T* xs = static_cast<const T*>(rev ? p.q : p.k);
    const T* ys = static_cast<const T*>(rev ? p.d_o : p.v);
    auto chunk = [&](int cc) { return rev ? nch - 1 - cc : cc; };
    const int xc = tid & 127, xr = tid >> 7, yc = tid & 31, yr = tid >> 5;
    float xv[C / 2], yv[C / 8], gv;
    auto fetch = [&](int cc) {  // chunk cc of the walk into registers
        const int nv = min(C, un.len - chunk(cc) * C);
        const int64_t row0 = un.row0 + static_cast<int64_t>(chunk(cc)) * C;
#pragma unroll
        for (int i = 0; i < C / 2; ++i) {
            const int r = xr + 2 * i;
            xv[i] = (r < nv && xc < dk) ? ld1(xs, (row0 + r) * dk + xc) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < C / 8; ++i) {
            const int r = yr + 8 * i;
            yv[i] = (r < nv && c0 + yc < dv) ? ld1(ys, (row0 + r) * dv + c0 + yc) : 0.f;
        }
        gv = load_gate<T>(p, row0, nv);
    };
    fetch(cc0);
    for (int cc = cc0; cc < cc1; ++cc) {
        const int c = chunk(cc), nv = min(C, un.len - c * C);
        const double G = gate_scan(gv), all = __shfl_sync(0xffffffffu, G, 31);
        const float wt = decay(rev ? G : all - G), gamma = decay(all);  // of token `lane`
        __syncthreads();  // X and Y of the chunk before are read
#pragma unroll
        for (int i = 0; i < C / 2; ++i) X[xr + 2 * i][xc] = xv[i];
#pragma unroll
        for (int i = 0; i < C / 8; ++i) Y[yr + 8 * i][yc] = yv[i] * __shfl_sync(0xffffffffu, wt, yr + 8 * i);
        __syncthreads();
        if (cc + 1 < cc1) fetch(cc + 1);
        whole += all;
        float* slot = slots + (un.slot0 + c) * usz;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                if (!p.sums && r0 + i < dk && n0 + m < dv) slot[(r0 + i) * dv + n0 + m] = S[i][m];
                S[i][m] *= gamma;
            }
#pragma unroll 8
        for (int j = 0; j < nv; ++j) {
            const float4 x = *reinterpret_cast<const float4*>(&X[j][r0]);
            const float4 y = *reinterpret_cast<const float4*>(&Y[j][n0 - c0]);
            const float xa[4] = {x.x, x.y, x.z, x.w}, ya[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int m = 0; m < 4; ++m) S[i][m] = fmaf(xa[i], ya[m], S[i][m]);
        }
    }
    if (p.sums && blockIdx.x % col_blocks == 0 && tid == 0) p.seg_decays[item] = static_cast<float>(whole * 1.4426950408889634);
    if (out) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int m = 0; m < 4; ++m)
                if (r0 + i < dk && n0 + m < dv) out[(r0 + i) * dv + n0 + m] = S[i][m];
    }
}

// ---------------------------------------------------------------------------
// Chunk phase of the prefill: one CTA per chunk.
// ---------------------------------------------------------------------------
constexpr int out_smem(int nm) {
    return static_cast<int>(sizeof(float)) * ((3 * C + 32 * nm) * (32 * nm + 1) + C * kLdC) +
           static_cast<int>(sizeof(double)) * C;
}

template <typename T, int NM>
__global__ void __launch_bounds__(kThreads) gated_out_simt_kernel(const GatedProblem p) {
    constexpr int LD = 32 * NM + 1;
    extern __shared__ double sm_d[];
    double* G = sm_d;
    float* Q = reinterpret_cast<float*>(G + C);
    float* K = Q + C * LD;
    float* V = K + C * LD;
    float* S = V + C * LD;
    float* P = S + 32 * NM * LD;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const GatedChunk ch = gated_chunk(p, blockIdx.x, C);
    if (ch.nv <= 0) return;
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    const float gv = load_gate<T>(p, ch.row0, ch.nv);
    load_state<NM>(S, static_cast<const float*>(p.s_states) + static_cast<int64_t>(blockIdx.x) * p.dk * p.dv, p.dk, p.dv);
    load_tile<T, NM>(Q, p.q, ch.row0, ch.nv, p.dk);
    load_tile<T, NM>(K, p.k, ch.row0, ch.nv, p.dk);
    load_tile<T, NM>(V, p.v, ch.row0, ch.nv, p.dv);
    if (w == 0) G[lane] = gate_scan(gv);
    __syncthreads();
    float a[4];
    scores<NM>(a, Q, K, p.dk);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * w + i;
        P[r * kLdC + lane] = lane <= r ? a[i] * decay(G[r] - G[lane]) : 0.f;
    }
    Acc<NM> acc = {};
    mm(acc, Q, LD, 1, S, LD, 1, p.dk);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float f = decay(G[4 * w + i]);
#pragma unroll
        for (int m = 0; m < NM; ++m) acc.x[i][m] *= f;
    }
    __syncwarp();  // a warp reads the rows of P that it wrote
    mm(acc, P, kLdC, 1, V, LD, 1, min(4 * w + 4, ch.nv));  // rows 4w..4w+3 read keys up to 4w+3
    store_rows<T>(p.o, ch.row0, ch.nv, p.dv, acc);
}

// ---------------------------------------------------------------------------
// Chunk phase of the gradient: one CTA per chunk.
// ---------------------------------------------------------------------------
constexpr int grad_smem(int nm) {
    return static_cast<int>(sizeof(float)) * ((4 * C + 2 * 32 * nm) * (32 * nm + 1) + 2 * C * kLdC + 2 * C + 8) +
           static_cast<int>(sizeof(double)) * C;
}

template <int NM>
__device__ __forceinline__ float row_dot(const float (&x)[NM], const float* y) {
    const int lane = threadIdx.x & 31;
    float s = 0.f;
#pragma unroll
    for (int m = 0; m < NM; ++m) s = fmaf(x[m], y[lane + 32 * m], s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

template <typename T, int NM>
__global__ void __launch_bounds__(kThreads) gated_grad_simt_kernel(const GatedProblem p) {
    constexpr int LD = 32 * NM + 1;
    extern __shared__ double sm_d[];
    double* G = sm_d;
    float* Q = reinterpret_cast<float*>(G + C);
    float* K = Q + C * LD;
    float* V = K + C * LD;
    float* DO = V + C * LD;
    float* S = DO + C * LD;
    float* E = S + 32 * NM * LD;
    float* W = E + 32 * NM * LD;  // w_ij (do_i . v_j), later M
    float* P = W + C * kLdC;      // w_ij (q_i . k_j)
    float* ri = P + C * kLdC;     // e^{G_i} q_i . (S do_i)
    float* cj = ri + C;           // e^{G_C - G_j} k_j . (E v_j)
    float* es = cj + C;           // per-warp sums of e^{G_C} <E, S>
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const GatedChunk ch = gated_chunk(p, blockIdx.x, C);
    if (ch.nv <= 0) return;
    const int nv = ch.nv, dk = p.dk, dv = p.dv;
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
    const int64_t usz = static_cast<int64_t>(dk) * dv;
    const float gv = load_gate<T>(p, ch.row0, nv);
    load_state<NM>(S, static_cast<const float*>(p.s_states) + blockIdx.x * usz, dk, dv);
    load_state<NM>(E, static_cast<const float*>(p.e_states) + blockIdx.x * usz, dk, dv);
    load_tile<T, NM>(Q, p.q, ch.row0, nv, dk);
    load_tile<T, NM>(K, p.k, ch.row0, nv, dk);
    load_tile<T, NM>(V, p.v, ch.row0, nv, dv);
    load_tile<T, NM>(DO, p.d_o, ch.row0, nv, dv);
    if (w == 0) G[lane] = gate_scan(gv);
    __syncthreads();
    float a[4], b[4];
    scores<NM>(a, Q, K, dk);
    scores<NM>(b, DO, V, dv);
    float mij[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * w + i;
        const float wij = lane <= r ? decay(G[r] - G[lane]) : 0.f;
        P[r * kLdC + lane] = lane <= r ? wij * a[i] : 0.f;
        W[r * kLdC + lane] = lane <= r ? wij * b[i] : 0.f;
        mij[i] = lane < r ? wij * a[i] * b[i] : 0.f;
    }
    // e^{G_C} <E, S>, half of the decay on either side: behind a memory that grew, ahead of one that will, E S alone may
    // leave float32
    float part = 0.f;
    const float half = decay(G[C - 1]) == 0.f ? 0.f : decay(0.5 * G[C - 1]);
    for (int r = w; r < dk; r += 8)
#pragma unroll
        for (int m = 0; m < NM; ++m)
            part = fmaf(half * S[r * LD + lane + 32 * m], half * E[r * LD + lane + 32 * m], part);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
    if (lane == 0) es[w] = part;
    __syncthreads();
    {  // dq
        Acc<NM> acc = {};
        mm(acc, DO, LD, 1, S, 1, LD, dv);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * w + i;
            const float f = decay(G[r]);
#pragma unroll
            for (int m = 0; m < NM; ++m) acc.x[i][m] *= f;
            const float s = row_dot<NM>(acc.x[i], Q + r * LD);
            if (lane == 0) ri[r] = s;
        }
        mm(acc, W, kLdC, 1, K, LD, 1, min(4 * w + 4, nv));
        store_rows<T>(p.dq, ch.row0, nv, dk, acc);
    }
    {  // dk
        Acc<NM> acc = {};
        mm(acc, V, LD, 1, E, 1, LD, dv);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = 4 * w + i;
            const float f = decay(G[C - 1] - G[r]);
#pragma unroll
            for (int m = 0; m < NM; ++m) acc.x[i][m] *= f;
            const float s = row_dot<NM>(acc.x[i], K + r * LD);
            if (lane == 0) cj[r] = s;
        }
        mm(acc, W, 1, kLdC, Q, LD, 1, nv);
        store_rows<T>(p.dk_, ch.row0, nv, dk, acc);
    }
    {  // dv
        Acc<NM> acc = {};
        mm(acc, K, LD, 1, E, LD, 1, dk);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float f = decay(G[C - 1] - G[4 * w + i]);
#pragma unroll
            for (int m = 0; m < NM; ++m) acc.x[i][m] *= f;
        }
        mm(acc, P, 1, kLdC, DO, LD, 1, nv);
        store_rows<T>(p.dv_, ch.row0, nv, dv, acc);
    }
    if (p.dg == nullptr) return;
    __syncthreads();  // every warp is done with W
#pragma unroll
    for (int i = 0; i < 4; ++i) W[(4 * w + i) * kLdC + lane] = mij[i];
    __syncthreads();
    // dg_t: warp w takes t = w, w + 8, ..; lane j sums column j over i >= t
    for (int t = w; t < nv; t += 8) {
        float s = 0.f;
        if (lane < t) {
            s = cj[lane];
            for (int i = t; i < nv; ++i) s += W[i * kLdC + lane];
        } else if (lane < nv) {
            s = ri[lane];
        }
        if (lane < 8) s += es[lane];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        // nothing passes a gate at the floor, whatever positive gates follow it
        if (__shfl_sync(0xffffffffu, gv, t) <= kGateFloor) s = 0.f;
        if (lane == 0) st1(static_cast<T*>(p.dg), ch.row0 + t, s);
    }
}

__global__ void __launch_bounds__(1024) chunk_offsets_kernel(const int32_t* __restrict__ cu, int num_seqs, int64_t rows,
                                                             int chunk, int32_t* __restrict__ choff, int32_t* __restrict__ order, int64_t nc,
                                                             unsigned int* __restrict__ used) {
    __shared__ int64_t warp_sum[32];
    __shared__ int32_t chunks[kMaxGatedOrder];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    int64_t before = 0;
    for (int n0 = 0; n0 < num_seqs; n0 += 1024) {
        const int n = n0 + tid;
        int32_t x = 0;
        if (n < num_seqs) {
            const int a = cu[n], b = cu[n + 1];
            if (!(a < 0 || b < a || static_cast<int64_t>(b) > rows)) x = gated_chunks(b - a, chunk);
            if (order != nullptr) chunks[n] = x;
        }
        int64_t s = x;
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        if (lane == 31) warp_sum[w] = s;
        __syncthreads();
        int64_t base = before, all = 0;
        for (int i = 0; i < 32; ++i) {
            if (i < w) base += warp_sum[i];
            all += warp_sum[i];
        }
        if (n < num_seqs) choff[n] = static_cast<int32_t>(min(base + s - x, static_cast<int64_t>(0x7fffffff)));
        // the last sequence that ends within the slots
        if (used != nullptr && n < num_seqs && base + s <= nc) atomicMax(used, static_cast<unsigned int>(base + s));
        before += all;
        __syncthreads();
    }
    if (tid == 0) choff[num_seqs] = static_cast<int32_t>(min(before, static_cast<int64_t>(0x7fffffff)));
    if (order != nullptr && tid < num_seqs) {  // the rank: how many sort before this one
        const int32_t x = chunks[tid];
        int rank = 0;
        for (int n = 0; n < num_seqs; ++n) rank += chunks[n] > x || (chunks[n] == x && n < tid) ? 1 : 0;
        order[rank] = tid;
    }
}

// One thread per element of a unit's state: walks the unit's segments.
__global__ void __launch_bounds__(256) segment_starts_kernel(const GatedProblem p, int chunk, int usz) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int per = (usz + 255) / 256;
    const int64_t du = blockIdx.x / per;  // [direction][unit]
    const int e = static_cast<int>(blockIdx.x % per) * 256 + threadIdx.x;
    if (e >= usz) return;
    const bool rev = du >= p.n_units;
    const int64_t u = du - (rev ? p.n_units : 0);
    const int nch = gated_chunks(gated_unit(p, u).len, chunk);
    const float* in = rev ? p.dstate : (p.state ? p.state : p.s0);
    float cur = in ? in[u * usz + e] : 0.f;
    const int segs = (nch + p.seg_chunks - 1) / p.seg_chunks;
    float* at = p.seg_states + du * p.segs * usz + e;
    const float* decay = p.seg_decays + du * p.segs;
    constexpr int kAhead = 8;  // sums in flight: one after the other, 37 segments took 25 us
    for (int s0 = 0; s0 < segs; s0 += kAhead) {
        float add[kAhead], f[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const bool more = s0 + i + 1 < segs;  // (the last has no sum)
            add[i] = more ? at[static_cast<int64_t>(s0 + i) * usz] : 0.f;
            f[i] = more ? decay[s0 + i] : 0.f;
        }
        // half of the decay, applied twice: a segment's may leave float32 (beyond 2^+-250 nothing of a state would be left)
#pragma unroll
        for (int i = 0; i < kAhead; ++i) f[i] = exp2f(0.5f * fminf(fmaxf(f[i], -250.f), 250.f));
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (s0 + i < segs) {
                at[static_cast<int64_t>(s0 + i) * usz] = cur;
                cur = fmaf(f[i] * cur, f[i], add[i]);
            }
    }
}

template <typename F>
cudaError_t launch_chunks(PerDeviceOnce& once, F kern, int smem, const GatedProblem& p, cudaStream_t s) {
    const cudaError_t e =
        once.run([&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(static_cast<unsigned>(p.groups * p.nc)), dim3(kThreads), smem, s, p);
}
template <typename T, int NM>
cudaError_t out_n(const GatedProblem& p, cudaStream_t s) {
    static PerDeviceOnce once;
    return launch_chunks(once, gated_out_simt_kernel<T, NM>, out_smem(NM), p, s);
}
template <typename T, int NM>
cudaError_t grad_n(const GatedProblem& p, cudaStream_t s) {
    static PerDeviceOnce once;
    return launch_chunks(once, gated_grad_simt_kernel<T, NM>, grad_smem(NM), p, s);
}
template <typename T>
cudaError_t chunks_t(const GatedProblem& p, bool grad, cudaStream_t s) {
    switch ((std::max(p.dk, p.dv) + 31) / 32) {
        case 1: return grad ? grad_n<T, 1>(p, s) : out_n<T, 1>(p, s);
        case 2: return grad ? grad_n<T, 2>(p, s) : out_n<T, 2>(p, s);
        case 3: return grad ? grad_n<T, 3>(p, s) : out_n<T, 3>(p, s);
        default: return grad ? grad_n<T, 4>(p, s) : out_n<T, 4>(p, s);
    }
}

}  // namespace

cudaError_t launch_chunk_offsets(const int32_t* cu, int num_seqs, int64_t rows, int chunk, int32_t* choff,
                                 int32_t* order, int64_t nc, unsigned int* used, cudaStream_t s) {
    if (num_seqs > kMaxGatedOrder) order = nullptr;
    return launch_pdl(chunk_offsets_kernel, dim3(1), dim3(1024), 0, s, cu, num_seqs, rows, chunk, choff, order, nc, used);
}

cudaError_t launch_segment_starts(const GatedProblem& p, int chunk, bool grad, cudaStream_t s) {
    const int usz = p.dk * p.dv;
    const int64_t grid = p.n_units * (grad ? 2 : 1) * ((usz + 255) / 256);
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_pdl(segment_starts_kernel, dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, p, chunk, usz);
}

cudaError_t launch_gated_states_simt(const GatedProblem& p, bool grad, cudaStream_t s) {
    const int cb = (p.dv + 31) / 32;
    const int64_t grid = p.n_units * p.segs * cb * (grad ? 2 : 1);
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    const auto kern = p.dtype ? gated_states_simt_kernel<__nv_bfloat16> : gated_states_simt_kernel<float>;
    return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, s, p, cb);
}
cudaError_t launch_gated_out_simt(const GatedProblem& p, cudaStream_t s) {
    return p.dtype ? chunks_t<__nv_bfloat16>(p, false, s) : chunks_t<float>(p, false, s);
}
cudaError_t launch_gated_grad_simt(const GatedProblem& p, cudaStream_t s) {
    return p.dtype ? chunks_t<__nv_bfloat16>(p, true, s) : chunks_t<float>(p, true, s);
}

}  // namespace la
