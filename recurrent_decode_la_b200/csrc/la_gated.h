// la_gated.h -- host-side launch interfaces of the gated recurrence (prefill
// and its gradient) and of the rotary positions, shared by the library's .cu
// files; and the chunk walk its kernels share.
//
// The recurrence: S_t = a_t S_{t-1} + k_t v_t^T, o_t = q_t^T S_t with the
// log-gate g_t = log a_t.  Within a chunk of C tokens, with the inclusive
// prefix sums G_i = g_1 + .. + g_i of the chunk,
//     O_i = e^{G_i} q_i^T S_in + sum_{j <= i} e^{G_i - G_j} (q_i . k_j) v_j
//     S_out = e^{G_C} S_in + sum_j e^{G_C - G_j} k_j v_j^T.
// Its gradient, with E the gradient of the state at the chunk's end and
// w_ij = e^{G_i - G_j}:
//     dq_i = e^{G_i} S_in do_i + sum_{j <= i} w_ij (do_i . v_j) k_j
//     dk_j = e^{G_C - G_j} E v_j + sum_{i >= j} w_ij (do_i . v_j) q_i
//     dv_j = e^{G_C - G_j} E^T k_j + sum_{i >= j} w_ij (q_i . k_j) do_i
//     E_in = e^{G_C} E + sum_i e^{G_i} q_i do_i^T        (the gradient of S_in)
//     dg_t = e^{G_C} <E, S_in> + sum_{i >= t} e^{G_i} q_i . (S_in do_i)
//          + sum_{j < t} e^{G_C - G_j} k_j . (E v_j) + sum_{i >= t > j} M_ij,
//            M_ij = w_ij (q_i . k_j)(do_i . v_j),
// a sum over exactly the (source, reader) pairs whose path crosses gate t: no
// two large terms are subtracted over a long range.
//
// The state phase walks the chunks of a unit in order (in reverse for E) and
// writes the state at every chunk's edge to the workspace; the chunk phase
// computes all chunks independently (in the tensor-core prefill the same launch,
// each chunk as soon as its state is there; else the next one).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace la {

// Dense input: groups = B*H, N = 0, unit u = group u.  Packed input: groups =
// H, unit n*H + h.  Workspace slot of chunk c of a unit: group * nc + ci with
// ci = c (dense) or choff[n] + c (packed); nc bounds ci.
struct GatedProblem {
    const void* q;
    const void* k;
    const void* v;
    const void* g;  // log gates [groups][rows]; nullptr: no decay
    void* o;
    float* state;  // prefill: S_0 in, S_T out
    // gradient only
    const float* s0;  // S_0 (nullptr: zero)
    const void* d_o;
    float* dstate;  // dS_T in, dS_0 out
    void* dq;
    void* dk_;
    void* dv_;
    void* dg;
    int dtype;  // 0 = f32, 1 = bf16
    int H;
    int64_t rows;  // rows per group
    int64_t groups;
    int num_seqs;  // 0: dense
    int64_t n_units;
    int dk;
    int dv;
    const int32_t* cu;     // nullptr: dense
    const int32_t* choff;  // packed: chunks before sequence n, num_seqs + 1 entries
    const int32_t* order;  // packed: the sequences, longest first (nullptr: in their order)
    int64_t nc;            // chunk slots per group
    // Tensor-core prefill: [0] chunks published, [1] chunks taken, [2] chunks per group (packed), [3] units claimed, then
    // from kQueueHead on the published slots, plus one.  All zero at the start but [2].
    unsigned int* queue;
    // Segments of a unit's walk (few long units): segs runs of seg_chunks chunks, each walked by itself.  A first pass
    // (sums) makes what each adds to a state of zero, with its decay; their prefix gives each one's start; the second
    // pass goes on from there.  seg_states [directions][units][segs][d_k][d_v], seg_decays [directions][units][segs], as
    // powers of two (positive gates may let a segment grow by more than fp32 holds).
    int segs;
    int seg_chunks;
    bool sums;
    float* seg_states;
    float* seg_decays;
    void* s_states;        // state at each chunk's start
    void* e_states;        // gradient of the state at each chunk's end
    uint64_t timeout_ns;
};

// A log gate below this decays by exactly zero in fp32 (e^-110 < 2^-149); the
// prefix sums take it in place of smaller ones, -inf included, so that no
// difference of two of them is inf - inf.  A NaN passes through.
constexpr float kGateFloor = -110.f;

struct GatedUnit {
    int64_t row0;   // first row in the [groups][rows] token layout
    int64_t slot0;  // workspace slot of its first chunk
    int len;
};

__device__ __forceinline__ GatedUnit gated_unit(const GatedProblem& p, int64_t u) {
    if (p.cu == nullptr) return {u * p.rows, u * p.nc, static_cast<int>(p.rows)};
    const int n = static_cast<int>(u / p.H);
    const int64_t h = u % p.H;
    const int a = p.cu[n], b = p.cu[n + 1];
    // offsets that do not rise (the chunk slots would run out): an empty sequence
    if (a < 0 || b < a || static_cast<int64_t>(b) > p.rows || p.choff[n + 1] > p.nc) return {0, 0, 0};
    return {h * p.rows + a, h * p.nc + p.choff[n], b - a};
}

// Chunks of C tokens in len (len + C - 1 need not fit an int).
__host__ __device__ constexpr int gated_chunks(int len, int C) { return len / C + (len % C != 0 ? 1 : 0); }

struct GatedChunk {
    int64_t row0;  // first row of the chunk in the [groups][rows] token layout
    int group;
    int row;  // row0 = group * rows + row
    int nv;   // its tokens; 0: the slot holds no chunk
    bool alone;  // its unit's only one
};

constexpr int kQueueHead = 4;

// The chunk of a workspace slot.
__device__ __forceinline__ GatedChunk gated_chunk(const GatedProblem& p, int64_t slot, int C) {
    const int64_t group = slot / p.nc;
    const int ci = static_cast<int>(slot % p.nc);
    if (p.cu == nullptr) {
        const int64_t r = static_cast<int64_t>(ci) * C;
        const int64_t left = p.rows - r;
        return {group * p.rows + r, static_cast<int>(group), static_cast<int>(r), static_cast<int>(left < C ? left : C), p.rows <= C};
    }
    if (ci >= p.choff[p.num_seqs]) return {0, 0, 0, 0, false};
    int lo = 0, hi = p.num_seqs - 1;  // the last sequence with choff[n] <= ci
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.choff[mid] <= ci) lo = mid; else hi = mid - 1;
    }
    if (p.choff[lo + 1] > p.nc) return {0, 0, 0, 0, false};
    const int c = ci - p.choff[lo];
    const int64_t a = p.cu[lo] + static_cast<int64_t>(c) * C;
    const int64_t left = p.cu[lo + 1] - a;
    return {group * p.rows + a, static_cast<int>(group), static_cast<int>(a), static_cast<int>(left < C ? left : C),
            p.choff[lo + 1] - p.choff[lo] == 1};
}

// choff[n] = chunks of C tokens in the sequences before n (offsets out of
// range or decreasing: an empty sequence), n = 0 .. num_seqs.  order (may be
// nullptr): the sequences by decreasing chunks, ties by index, for at most
// kMaxGatedOrder of them.  used (may be nullptr): the chunks of the sequences
// that fit into nc slots.
constexpr int kMaxGatedOrder = 1024;
cudaError_t launch_chunk_offsets(const int32_t* cu, int num_seqs, int64_t rows, int C, int32_t* choff, int32_t* order,
                                 int64_t nc, unsigned int* used, cudaStream_t s);

// seg_states[..][s] = the start of segment s, from S_0 (dS_T) and the sums of
// the segments before it.
cudaError_t launch_segment_starts(const GatedProblem& p, int chunk, bool grad, cudaStream_t s);

// CUDA-core kernels: fp32 throughout, fp32 chunk states, any d_k, d_v <= 128.
constexpr int kGatedSimtChunk = 32;
cudaError_t launch_gated_states_simt(const GatedProblem& p, bool grad, cudaStream_t s);
cudaError_t launch_gated_out_simt(const GatedProblem& p, cudaStream_t s);
cudaError_t launch_gated_grad_simt(const GatedProblem& p, cudaStream_t s);

// Tensor-core kernels: bf16, d_k == d_v in {64, 128}, 16-byte aligned tensors;
// chunks of 128 tokens, chunk states in bf16 as the swizzled shared-memory
// image of the tile (two panels of 64 columns at d = 128).
constexpr int kGatedTcChunk = 128;
struct GatedMaps {
    CUtensorMap q, k, v, d_o;       // loads: 64 columns x 128 rows
    CUtensorMap o;                  // stores: 64 columns x 32 rows
    CUtensorMap dq, dk, dv;         // stores: 64 columns x 128 rows
};
// States at the chunk starts and, for the gradient, gradients at the chunk ends; or the segments' sums.
cudaError_t launch_gated_states_tc(const GatedProblem& p, const GatedMaps& m, bool grad, int num_sms, cudaStream_t s);
// The whole prefill.
cudaError_t launch_gated_prefill_tc(const GatedProblem& p, const GatedMaps& m, int num_sms, cudaStream_t s);
cudaError_t launch_gated_grad_tc(const GatedProblem& p, const GatedMaps& m, int num_sms, cudaStream_t s);

struct RotaryProblem {
    const void* x[2];  // q and k (k may be nullptr)
    void* y[2];
    int dtype;
    int64_t B;
    int64_t H;
    int64_t T;  // rows per head
    int d;
    int rot;
    const float* freq;     // [rot / 2]
    const int32_t* start;  // [B] or [num_seqs]; nullptr: 0
    const int32_t* cu;     // nullptr: dense
    int num_seqs;
    float scale;
    bool interleaved;
    bool inverse;
};
cudaError_t launch_rotary(const RotaryProblem& p, int num_sms, cudaStream_t s);
cudaError_t launch_rotary_init(float* freq, int rot, double base, int scaling, double factor, double original,
                               double beta_fast, double beta_slow, cudaStream_t s);

}  // namespace la
