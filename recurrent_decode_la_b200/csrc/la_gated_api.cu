// la_gated_api.cu -- the C ABI of the gated recurrence and of the rotary
// positions (declared in include/linattn.h): argument checks, kernel choice,
// workspace layout and launches.  Host code only.
#include <stdio.h>

#include <algorithm>

#include "../../include/linattn.h"
#include "la_gated.h"
#include "la_internal.h"

namespace la {
namespace {

la_status fail(cudaError_t e) { return static_cast<la_status>(cuda_fail_status(e)); }
la_status refuse(la_status s, const char* why) {
    set_last_error(why);
    return s;
}
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
size_t up256(size_t x) { return (x + 255) / 256 * 256; }

enum Kernel { kNone, kShort, kTc, kSimt };

// The kernels for these sizes.  max_tokens: T (dense) or max_seqlen (packed, 0: unknown).
Kernel choose(la_dtype dtype, int64_t max_tokens, int dk, int dv, bool grad) {
    if (dk < 1 || dv < 1 || dk > 128 || dv > 128) return kNone;
    if (!grad && tuning().short_kernel && prefill_short_supported(max_tokens, dk, dv, nullptr)) return kShort;
    if (dtype == LA_BF16 && dk == dv && (dk == 64 || dk == 128)) return kTc;
    return kSimt;
}

// The gradient of few short units (T: all rows of packed ones) runs on the CUDA cores where the tensor cores could take it:
// one chunk of 32 tokens each, in fp32 throughout.  A gate's gradient is a sum of large terms that may cancel, and the bf16 operands that it is made of
// on the tensor cores show in it where few others stand beside it: dg of a single unit of 5 tokens at d 128 was over 0.005
// of itself off in 4 of 100 calls and up to 0.016 (here 0.0036 at most); of 32 units never.  20 tokens: 6 units at d 64 21
// us, on the tensor cores 25, 64 units 25 and 26; at d 128 38 and 33, 51 and 37 (512 units: 309 and 136).
constexpr int64_t kFewUnits = 32, kFewTokens = kGatedSimtChunk;
Kernel choose_grad(la_dtype dtype, int64_t units, int64_t T, int dk, int dv) {
    const Kernel kind = choose(dtype, 0, dk, dv, true);
    return kind == kTc && units <= kFewUnits && T <= kFewTokens ? kSimt : kind;
}

// CTAs that the split of few units aims at: one a SM of the part this is written for.  Not the current device's count: the
// workspace that a caller asked for has to fit on any.
constexpr int64_t kPlanSms = 148;

// Chunk states in the workspace: packed, first the chunk offsets (num_seqs + 1
// int32) and the sequences by length (num_seqs int32); for the tensor-core prefill
// the queue of published chunks; room for the sums of segments and their decays;
// then one state per chunk slot, and for the gradient one gradient of a state per
// slot.
struct Layout {
    int chunk = 0;
    int64_t nc = 0;
    int segs = 1, seg_chunks = 0;
    int64_t seg_slots = 0;
    size_t queue = 0, seg = 0, s = 0, e = 0, bytes = 0;
};
Layout plan(Kernel kind, int64_t groups, int64_t T, int dk, int dv, int num_seqs, bool grad) {
    Layout w;
    if (kind == kShort || kind == kNone) return w;
    w.chunk = kind == kTc ? kGatedTcChunk : kGatedSimtChunk;
    // a packed sequence begins a chunk of its own
    w.nc = num_seqs > 0 ? T / w.chunk + num_seqs : (T + w.chunk - 1) / w.chunk;
    const size_t states = up256(static_cast<size_t>(groups) * w.nc * dk * dv * (kind == kTc ? 2 : 4));
    // Few long units: the walk is cut into segments, walked twice (their sums, then their chunks), so that more of the
    // device works on it, where that leaves at most half of it one behind the other (with three segments 32 heads of
    // 4096 tokens took 118 us, unsplit 107).  From four tensor-core chunks a segment, or two of the CUDA cores: below,
    // the second walk costs what it saves (two tensor-core chunks, 2 heads of 1000 tokens: 43 us, unsplit 35).  Unsplit
    // and split: 8 heads of 16384 tokens 270 and 101 us, their gradient 310 and 173; 8 heads of 4000 83 and 54; fp32, 4
    // heads of 8000 180 and 70, their gradient 751 and 237 (with four CTAs of the CUDA cores an SM instead of two 78 and
    // 244).
    const int64_t units = groups * std::max(1, num_seqs), nch = (T + w.chunk - 1) / w.chunk, dirs = grad ? 2 : 1;
    const int64_t room = (kind == kSimt ? 2 * kPlanSms / ((dv + 31) / 32) : grad ? kPlanSms : kPlanSms * 3 / 4) / dirs;
    const int64_t most = std::min<int64_t>(nch / (kind == kTc ? 4 : 2), 64);
    const int64_t segs = std::min(room / units, most) < 4 ? 1 : std::min(room / units, most);
    w.seg_chunks = static_cast<int>((nch + segs - 1) / segs);
    w.segs = static_cast<int>((nch + w.seg_chunks - 1) / w.seg_chunks);
    // Room for the segments of any call with fewer units or tokens, so that a workspace fits those too.
    w.seg_slots = most < 4 ? 0 : dirs * std::min(room, units * most);
    w.queue = num_seqs > 0 ? up256((2 * static_cast<size_t>(num_seqs) + 1) * 4) : 0;
    w.seg = w.queue + (kind == kTc && !grad ? up256((static_cast<size_t>(groups) * w.nc + kQueueHead) * 4) : 0);
    w.s = w.seg + up256(static_cast<size_t>(w.seg_slots) * (static_cast<size_t>(dk) * dv + 1) * 4);
    w.e = w.s + states;
    w.bytes = w.e + (grad ? states : 0);
    return w;
}

size_t workspace_bytes_for(la_dtype dtype, int B, int H, int64_t T, int dk, int dv, int num_seqs, bool grad) {
    if ((dtype != LA_F32 && dtype != LA_BF16) || B <= 0 || H <= 0 || T <= 0 || num_seqs < 0) return 0;
    const int64_t groups = static_cast<int64_t>(num_seqs > 0 ? 1 : B) * H;
    if (grad) {
        auto need = [&](int64_t groups, int64_t T, int n) {
            return plan(choose_grad(dtype, groups * std::max(1, n), T, dk, dv), groups, T, dk, dv, n, true).bytes;
        };
        size_t bytes = need(groups, T, num_seqs);
        // room for any call with fewer units or tokens too
        for (int64_t few = 1; few <= std::min(groups, kFewUnits); ++few)
            bytes = std::max(bytes, need(few, std::min(T, kFewTokens),
                                         static_cast<int>(std::min<int64_t>(num_seqs, kFewUnits / few))));
        return bytes;
    }
    // packed input, whose longest sequence is not known here, may need the chunked kernels
    const Kernel kind = choose(dtype, num_seqs > 0 ? 0 : T, dk, dv, false);
    return plan(kind, groups, T, dk, dv, num_seqs, false).bytes;
}

// Sizes and layout that every sequence entry point shares.  LA_OK with
// p.n_units == 0: nothing to do.
la_status sizes(GatedProblem& p, la_dtype dtype, int B, int H, int64_t T, int dk, int dv, const int32_t* cu,
                int num_seqs) {
    if (dtype != LA_F32 && dtype != LA_BF16) return refuse(LA_ERR_INVALID_ARG, "dtype must be LA_F32 or LA_BF16");
    if (B < 0 || H < 0 || T < 0 || dk <= 0 || dv <= 0) return refuse(LA_ERR_INVALID_ARG, "a size is out of range");
    if (cu && (B != 1 || num_seqs < 0)) return refuse(LA_ERR_INVALID_ARG, "packed input needs B == 1");
    if (T > 0x7fffffffLL || dk > 128 || dv > 128)
        return refuse(LA_ERR_UNSUPPORTED, "d_k and d_v are at most 128, T below 2^31");
    p = GatedProblem{};
    p.dtype = dtype == LA_BF16 ? 1 : 0;
    p.H = H;
    p.rows = T;
    p.groups = static_cast<int64_t>(cu ? 1 : B) * H;
    p.num_seqs = cu ? num_seqs : 0;
    p.n_units = cu ? static_cast<int64_t>(num_seqs) * H : p.groups;
    p.dk = dk;
    p.dv = dv;
    p.cu = cu;
    p.timeout_ns = tuning().wait_timeout_ns;
    if (T == 0) p.n_units = 0;
    return LA_OK;
}

la_status place(GatedProblem& p, const Layout& w, void* workspace, size_t bytes) {
    if (p.groups * w.nc > 0x7fffffffLL || p.n_units > (1 << 28)) return refuse(LA_ERR_UNSUPPORTED, "too many chunks for one call");
    if (!workspace || bytes < w.bytes || !aligned16(workspace)) {
        char why[128];
        snprintf(why, sizeof(why), "needs a 16-byte aligned workspace of %zu bytes, got %zu", w.bytes,
                 workspace ? bytes : static_cast<size_t>(0));
        return refuse(LA_ERR_INVALID_ARG, why);
    }
    char* base = static_cast<char*>(workspace);
    p.nc = w.nc;
    p.segs = w.segs;
    p.seg_chunks = w.seg_chunks;
    p.choff = p.cu ? reinterpret_cast<const int32_t*>(base) : nullptr;
    p.order = p.cu && p.num_seqs <= kMaxGatedOrder ? p.choff + p.num_seqs + 1 : nullptr;
    if (w.segs > 1) {
        p.seg_states = reinterpret_cast<float*>(base + w.seg);
        p.seg_decays = p.seg_states + w.seg_slots * p.dk * p.dv;
    }
    p.s_states = base + w.s;
    p.e_states = base + w.e;
    return LA_OK;
}

cudaError_t chunk_offsets(const GatedProblem& p, const Layout& w, cudaStream_t s) {
    if (!p.cu) return cudaSuccess;
    return launch_chunk_offsets(p.cu, p.num_seqs, p.rows, w.chunk, const_cast<int32_t*>(p.choff), const_cast<int32_t*>(p.order), w.nc,
                                p.queue ? p.queue + 2 : nullptr, s);
}

// Where the walk is cut: every segment's sum, then its start.
template <typename F>
cudaError_t segment_starts(const GatedProblem& p, const Layout& w, bool grad, F&& states, cudaStream_t s) {
    if (p.segs == 1) return cudaSuccess;
    GatedProblem q = p;
    q.sums = true;
    q.queue = nullptr;
    const cudaError_t e = states(q);
    return e != cudaSuccess ? e : launch_segment_starts(p, w.chunk, grad, s);
}

// The tensor maps of the tensor-core kernels (every tensor 16-byte aligned).
la_status maps(GatedMaps& m, const GatedProblem& p, bool grad) {
    const void* all[] = {p.q, p.k, p.v, grad ? p.d_o : p.o, grad ? p.dq : p.q, grad ? p.dk_ : p.q, grad ? p.dv_ : p.q,
                         grad ? p.dstate : p.state, p.s0};
    for (const void* x : all)
        if (!aligned16(x)) return refuse(LA_ERR_UNSUPPORTED, "bf16 with d 64 or 128 needs 16-byte aligned tensors");
    const auto enc = [&](CUtensorMap& map, const void* x, int box_rows) {
        return encode_bf16_map(&map, x, p.dk, p.rows, p.groups, box_rows);
    };
    bool ok = enc(m.q, p.q, kGatedTcChunk) && enc(m.k, p.k, kGatedTcChunk) && enc(m.v, p.v, kGatedTcChunk);
    if (grad)
        ok = ok && enc(m.d_o, p.d_o, kGatedTcChunk) && enc(m.dq, p.dq, kGatedTcChunk) && enc(m.dk, p.dk_, kGatedTcChunk) &&
             enc(m.dv, p.dv_, kGatedTcChunk);
    else
        ok = ok && enc(m.o, p.o, 32);
    return ok ? LA_OK : refuse(LA_ERR_CUDA, "cuTensorMapEncodeTiled failed");
}

}  // namespace
}  // namespace la

using namespace la;

extern "C" {

const char* la_gated_prefill_kernel(la_dtype dtype, int64_t max_tokens, int d_k, int d_v) {
    switch (choose(dtype, max_tokens, d_k, d_v, false)) {
        case kShort: return "short";
        case kTc: return "tc";
        case kSimt: return "simt";
        default: return "unsupported";
    }
}

size_t la_gated_prefill_workspace_size(la_dtype dtype, int B, int H, int64_t T, int d_k, int d_v, int num_seqs) {
    return workspace_bytes_for(dtype, B, H, T, d_k, d_v, num_seqs, false);
}

size_t la_gated_prefill_backward_workspace_size(la_dtype dtype, int B, int H, int64_t T, int d_k, int d_v,
                                                int num_seqs) {
    return workspace_bytes_for(dtype, B, H, T, d_k, d_v, num_seqs, true);
}

la_status la_gated_prefill(const void* q, const void* k, const void* v, const void* g, void* o, float* state,
                           la_dtype dtype, int B, int H, int64_t T, int d_k, int d_v, const int32_t* cu_seqlens,
                           int num_seqs, int64_t max_seqlen, void* workspace, size_t workspace_bytes, void* stream) {
    GatedProblem p;
    la_status st = sizes(p, dtype, B, H, T, d_k, d_v, cu_seqlens, num_seqs);
    if (st != LA_OK || p.n_units == 0) return st;
    if (!q || !k || !v || !o || !state) return refuse(LA_ERR_INVALID_ARG, "a tensor is NULL");
    const int64_t max_tokens = cu_seqlens ? max_seqlen : T;
    const Kernel kind = choose(dtype, max_tokens, d_k, d_v, false);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (kind == kShort) {
        if (!aligned16(state)) return refuse(LA_ERR_UNSUPPORTED, "state must be 16-byte aligned");
        PrefillProblem f = {};
        f.q = q; f.k = k; f.v = v; f.g = g; f.o = o; f.state = state;
        f.dtype = p.dtype;
        f.H = H;
        f.rows_per_group = T;
        f.n_units = p.n_units;
        f.dk = d_k; f.dv = d_v;
        f.cu = cu_seqlens;
        e = launch_prefill_short(f, max_tokens, current_sm_count(), s);
        return e == cudaSuccess ? LA_OK : fail(e);
    }
    const Layout w = plan(kind, p.groups, T, d_k, d_v, p.num_seqs, false);
    if ((st = place(p, w, workspace, workspace_bytes)) != LA_OK) return st;
    p.q = q; p.k = k; p.v = v; p.g = g; p.o = o; p.state = state;
    if (kind == kTc) {
        GatedMaps m = {};
        if ((st = maps(m, p, false)) != LA_OK) return st;
        p.queue = reinterpret_cast<unsigned int*>(static_cast<char*>(workspace) + w.queue);
        const int sms = current_sm_count();
        e = cudaMemsetAsync(p.queue, 0, w.seg - w.queue, s);
        if (e == cudaSuccess) e = chunk_offsets(p, w, s);
        if (e == cudaSuccess)
            e = segment_starts(p, w, false, [&](const GatedProblem& q) { return launch_gated_states_tc(q, m, false, sms, s); }, s);
        if (e == cudaSuccess) e = launch_gated_prefill_tc(p, m, sms, s);
        return e == cudaSuccess ? LA_OK : fail(e);
    }
    e = chunk_offsets(p, w, s);
    if (e == cudaSuccess)
        e = segment_starts(p, w, false, [&](const GatedProblem& q) { return launch_gated_states_simt(q, false, s); }, s);
    if (e == cudaSuccess) e = launch_gated_states_simt(p, false, s);
    if (e == cudaSuccess) e = launch_gated_out_simt(p, s);
    return e == cudaSuccess ? LA_OK : fail(e);
}

la_status la_gated_prefill_backward(const void* q, const void* k, const void* v, const void* g, const float* state0,
                                    const void* d_o, float* dstate, void* dq, void* dk, void* dv, void* dg,
                                    la_dtype dtype, int B, int H, int64_t T, int d_k, int d_v,
                                    const int32_t* cu_seqlens, int num_seqs, void* workspace, size_t workspace_bytes,
                                    void* stream) {
    GatedProblem p;
    la_status st = sizes(p, dtype, B, H, T, d_k, d_v, cu_seqlens, num_seqs);
    if (st != LA_OK || p.n_units == 0) return st;
    if (!q || !k || !v || !d_o || !dstate || !dq || !dk || !dv)
        return refuse(LA_ERR_INVALID_ARG, "a tensor is NULL");
    const Kernel kind = choose_grad(dtype, p.n_units, T, d_k, d_v);
    const Layout w = plan(kind, p.groups, T, d_k, d_v, p.num_seqs, true);
    if ((st = place(p, w, workspace, workspace_bytes)) != LA_OK) return st;
    p.q = q; p.k = k; p.v = v; p.g = g;
    p.s0 = state0;
    p.d_o = d_o;
    p.dstate = dstate;
    p.dq = dq; p.dk_ = dk; p.dv_ = dv; p.dg = dg;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (kind == kTc) {
        GatedMaps m = {};
        if ((st = maps(m, p, true)) != LA_OK) return st;
        const int sms = current_sm_count();
        e = chunk_offsets(p, w, s);
        if (e == cudaSuccess)
            e = segment_starts(p, w, true, [&](const GatedProblem& q) { return launch_gated_states_tc(q, m, true, sms, s); }, s);
        if (e == cudaSuccess) e = launch_gated_states_tc(p, m, true, sms, s);
        if (e == cudaSuccess) e = launch_gated_grad_tc(p, m, sms, s);
        return e == cudaSuccess ? LA_OK : fail(e);
    }
    e = chunk_offsets(p, w, s);
    if (e == cudaSuccess)
        e = segment_starts(p, w, true, [&](const GatedProblem& q) { return launch_gated_states_simt(q, true, s); }, s);
    if (e == cudaSuccess) e = launch_gated_states_simt(p, true, s);
    if (e == cudaSuccess) e = launch_gated_grad_simt(p, s);
    return e == cudaSuccess ? LA_OK : fail(e);
}

la_status la_gated_decode_step(const void* q, const void* k, const void* v, const void* g, void* o, float* state,
                               la_dtype dtype, int B, int H, int d_k, int d_v, void* stream) {
    if (dtype != LA_F32 && dtype != LA_BF16) return refuse(LA_ERR_INVALID_ARG, "dtype must be LA_F32 or LA_BF16");
    if (B < 0 || H < 0 || d_k <= 0 || d_v <= 0) return refuse(LA_ERR_INVALID_ARG, "a size is out of range");
    if (d_k > 128 || d_v > 128) return refuse(LA_ERR_UNSUPPORTED, "d_k and d_v are at most 128");
    const int64_t n_units = static_cast<int64_t>(B) * H;
    if (n_units == 0) return LA_OK;
    if (!q || !k || !v || !o || !state) return refuse(LA_ERR_INVALID_ARG, "a tensor is NULL");
    const cudaError_t e = launch_decode(q, k, v, g, o, state, dtype == LA_BF16 ? 1 : 0, n_units, d_k, d_v,
                                        current_sm_count(), static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? LA_OK : fail(e);
}

la_status la_rotary_init(float* freq, int rot, double base, la_rotary_scaling scaling, double factor,
                         double original, double beta_fast, double beta_slow, void* stream) {
    if (rot < 0 || rot % 2 != 0) return refuse(LA_ERR_INVALID_ARG, "rot must be even");
    if (scaling < LA_ROTARY_PLAIN || scaling > LA_ROTARY_PARTS) return refuse(LA_ERR_INVALID_ARG, "unknown scaling");
    if (!(base > 0.0) || (scaling != LA_ROTARY_PLAIN && !(factor > 0.0)))
        return refuse(LA_ERR_INVALID_ARG, "base and factor must be positive");
    if (scaling == LA_ROTARY_PARTS && (!(original > 0.0) || !(beta_fast > beta_slow)))
        return refuse(LA_ERR_INVALID_ARG, "scaling by parts needs original > 0 and beta_fast > beta_slow");
    if (rot == 0) return LA_OK;
    if (!freq) return refuse(LA_ERR_INVALID_ARG, "a tensor is NULL");
    const cudaError_t e = launch_rotary_init(freq, rot, base, static_cast<int>(scaling), factor, original, beta_fast,
                                             beta_slow, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? LA_OK : fail(e);
}

la_status la_rotary(const void* q, const void* k, void* q_out, void* k_out, la_dtype dtype, int B, int H, int64_t T,
                    int d, int rot, const float* freq, const int32_t* start, float scale, int interleaved,
                    int inverse, const int32_t* cu_seqlens, int num_seqs, void* stream) {
    if (dtype != LA_F32 && dtype != LA_BF16) return refuse(LA_ERR_INVALID_ARG, "dtype must be LA_F32 or LA_BF16");
    if (B < 0 || H < 0 || T < 0 || d <= 0) return refuse(LA_ERR_INVALID_ARG, "a size is out of range");
    if (rot < 0 || rot % 2 != 0 || rot > d) return refuse(LA_ERR_INVALID_ARG, "rot must be even and at most d");
    if (cu_seqlens && (B != 1 || num_seqs < 0)) return refuse(LA_ERR_INVALID_ARG, "packed input needs B == 1");
    if (T > 0x7fffffffLL || d > 128) return refuse(LA_ERR_UNSUPPORTED, "d is at most 128, T below 2^31");
    if (B == 0 || H == 0 || T == 0 || (cu_seqlens && num_seqs == 0)) return LA_OK;
    if (!q || !q_out || (k == nullptr) != (k_out == nullptr) || (rot > 0 && !freq))
        return refuse(LA_ERR_INVALID_ARG, "a tensor is NULL");
    RotaryProblem p = {};
    p.x[0] = q; p.x[1] = k;
    p.y[0] = q_out; p.y[1] = k_out;
    p.dtype = dtype == LA_BF16 ? 1 : 0;
    p.B = B; p.H = H; p.T = T;
    p.d = d; p.rot = rot;
    p.freq = freq;
    p.start = start;
    p.cu = cu_seqlens;
    p.num_seqs = num_seqs;
    p.scale = scale;
    p.interleaved = interleaved != 0;
    p.inverse = inverse != 0;
    const cudaError_t e = launch_rotary(p, current_sm_count(), static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? LA_OK : fail(e);
}

}  // extern "C"
