// la_rotary.cu -- rotary positions of q and k, and the table of their
// frequencies.
//
// Pair i of a head (elements i and i + rot/2, or 2i and 2i + 1) at position
// pos turns by the angle pos * freq[i]:
//     y_a = (x_a cos - x_b sin) * scale,   y_b = (x_b cos + x_a sin) * scale,
// the inverse (also the gradient: the map is linear and orthogonal up to
// `scale`) by the negated angle.  Elements rot .. d-1 pass unchanged.
//
// Bound by memory: each element is read once and written once.  The angle is
// taken in float64, as a fraction of a turn whose whole turns are dropped, so
// far positions lose nothing (a float32 product is off by a twentieth of a
// radian at position 2^20); that costs about fifty instructions a pair, so a
// thread takes V pairs (two 16-byte vectors) of one token and walks the heads
// with them, q and k together.
#include <cuda_bf16.h>

#include "la_gated.h"
#include "la_internal.h"

namespace la {
namespace {

constexpr int kThreads = 256;
// Heads in flight per thread and tensor.  16-byte vectors: two (4 and 8 with fewer CTAs: up to 8 % slower); narrower ones, of
// which a thread moves less at a time, four (eight spilled registers).
constexpr int batch_of(int bytes) { return bytes >= 16 ? 2 : 4; }
// Above this (bytes read and written) nothing of the tensors is left in L2 for the next kernel anyway: loads and stores
// then go past it (evict first).  B8 H16 T8192 d128: 169 us, as a plain copy, against 212 us with the default policy.
constexpr int64_t kStreamBytes = 126 << 20;

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    T x[V];
};
template <int BYTES>
struct Word;
template <>
struct Word<16> { using type = int4; };
template <>
struct Word<8> { using type = int2; };
template <>
struct Word<4> { using type = int; };
template <>
struct Word<2> { using type = short; };
template <bool STREAM, typename W>
__device__ __forceinline__ W load_vec(const W* p) {
    using I = typename Word<sizeof(W)>::type;
    if constexpr (STREAM) {
        const I r = __ldcs(reinterpret_cast<const I*>(p));
        return *reinterpret_cast<const W*>(&r);
    } else {
        return *p;
    }
}
template <bool STREAM, typename W>
__device__ __forceinline__ void store_vec(W* p, const W& x) {
    using I = typename Word<sizeof(W)>::type;
    if constexpr (STREAM)
        __stcs(reinterpret_cast<I*>(p), *reinterpret_cast<const I*>(&x));
    else
        *p = x;
}
__device__ __forceinline__ float get(float x) { return x; }
__device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float& y, float x) { y = x; }
__device__ __forceinline__ void put(__nv_bfloat16& y, float x) { y = __float2bfloat16_rn(x); }

// Row t of the packed layout: its place in its sequence n (-1: in none).
__device__ __forceinline__ int packed_place(const int32_t* cu, int num_seqs, int64_t t, int* seq) {
    if (t < cu[0] || t >= cu[num_seqs]) return -1;
    int lo = 0, hi = num_seqs - 1;  // the last sequence that begins at or before t
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= t) lo = mid; else hi = mid - 1;
    }
    *seq = lo;
    return static_cast<int>(t - cu[lo]);
}

// One thread: V pairs (or V passed elements) of one token, heads h0 .. h0 + heads - 1 of both tensors.
template <typename T, int V, bool INTERLEAVED, bool STREAM>
__global__ void __launch_bounds__(kThreads, 3) rotary_kernel(const RotaryProblem p, int items, int heads) {
    constexpr int kBatch = batch_of(sizeof(T) * V);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t i = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x;
    if (i >= p.B * p.T * items) return;
    const int item = static_cast<int>(i % items);
    const int64_t bt = i / items, b = bt / p.T, t = bt % p.T;
    const int pair_items = p.rot / 2 / V;
    const int64_t h0 = static_cast<int64_t>(blockIdx.y) * heads;
    const int64_t h1 = h0 + heads < p.H ? h0 + heads : p.H;
    int seq = static_cast<int>(b);
    int64_t place = t;
    if (p.cu != nullptr) {
        place = packed_place(p.cu, p.num_seqs, t, &seq);
        if (place < 0) return;
    }
    const int64_t step = p.T * p.d;  // between heads
    const int64_t base = ((b * p.H + h0) * p.T + t) * p.d;
    if (item >= pair_items) {  // passed through (nothing to do in place)
        const int64_t at = base + p.rot + static_cast<int64_t>(item - pair_items) * V;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            const T* x = static_cast<const T*>(p.x[which]);
            T* y = static_cast<T*>(p.y[which]);
            if (x == nullptr || x == y) continue;
            for (int64_t hb = 0; hb < h1 - h0; hb += kBatch) {
                Vec<T, V> u[kBatch];
#pragma unroll
                for (int n = 0; n < kBatch; ++n)
                    if (hb + n < h1 - h0) u[n] = load_vec<STREAM>(reinterpret_cast<const Vec<T, V>*>(x + at + (hb + n) * step));
#pragma unroll
                for (int n = 0; n < kBatch; ++n)
                    if (hb + n < h1 - h0) store_vec<STREAM>(reinterpret_cast<Vec<T, V>*>(y + at + (hb + n) * step), u[n]);
            }
        }
        return;
    }
    const int64_t pos = place + (p.start ? p.start[seq] : 0);
    float c[V], s[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const double turns = static_cast<double>(pos) * (static_cast<double>(p.freq[item * V + e]) * 0.15915494309189535);
        sincospif(static_cast<float>(2.0 * (turns - rint(turns))), &s[e], &c[e]);
        c[e] *= p.scale;
        s[e] *= p.inverse ? -p.scale : p.scale;
    }
    const int64_t a0 = base + (INTERLEAVED ? 2 * item * V : item * V);
    const int64_t a1 = a0 + (INTERLEAVED ? V : p.rot / 2);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const T* x = static_cast<const T*>(p.x[which]);
        T* y = static_cast<T*>(p.y[which]);
        if (x == nullptr) continue;
        // kBatch heads are loaded before the first is stored (the output may be the input)
        for (int64_t hb = 0; hb < h1 - h0; hb += kBatch) {
            Vec<T, V> u[kBatch], w[kBatch];
#pragma unroll
            for (int n = 0; n < kBatch; ++n)
                if (hb + n < h1 - h0) {
                    u[n] = load_vec<STREAM>(reinterpret_cast<const Vec<T, V>*>(x + a0 + (hb + n) * step));
                    w[n] = load_vec<STREAM>(reinterpret_cast<const Vec<T, V>*>(x + a1 + (hb + n) * step));
                }
#pragma unroll
            for (int n = 0; n < kBatch; ++n) {
                if (hb + n >= h1 - h0) break;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    // the pair's elements: (u[e], w[e]), or, interleaved, entries 2e and 2e + 1 of u followed by w
                    T& ra = INTERLEAVED ? (2 * e < V ? u[n].x[(2 * e) % V] : w[n].x[(2 * e) % V]) : u[n].x[e];
                    T& rb = INTERLEAVED ? (2 * e + 1 < V ? u[n].x[(2 * e + 1) % V] : w[n].x[(2 * e + 1) % V]) : w[n].x[e];
                    const float fa = get(ra), fb = get(rb);
                    put(ra, fa * c[e] - fb * s[e]);
                    put(rb, fb * c[e] + fa * s[e]);
                }
                store_vec<STREAM>(reinterpret_cast<Vec<T, V>*>(y + a0 + (hb + n) * step), u[n]);
                store_vec<STREAM>(reinterpret_cast<Vec<T, V>*>(y + a1 + (hb + n) * step), w[n]);
            }
        }
    }
}

template <typename T, int V>
cudaError_t rotary_v(const RotaryProblem& p, int num_sms, cudaStream_t s) {
    const int items = (p.rot / 2 + p.d - p.rot) / V;
    const int64_t threads = p.B * p.T * items;
    const int64_t blocks = (threads + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    // few tokens: the heads are shared out over the grid until it covers the SMs
    int64_t groups = (static_cast<int64_t>(num_sms) * 8 + blocks - 1) / blocks;
    if (groups > p.H) groups = p.H;
    if (groups > 65535) groups = 65535;
    const int heads = static_cast<int>((p.H + groups - 1) / groups);
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((p.H + heads - 1) / heads));
    const int64_t bytes = 2 * p.B * p.H * p.T * p.d * static_cast<int64_t>(sizeof(T)) * (p.x[1] ? 2 : 1);
    const bool stream = bytes > kStreamBytes;
    const auto kern = p.interleaved ? (stream ? rotary_kernel<T, V, true, true> : rotary_kernel<T, V, true, false>)
                                    : (stream ? rotary_kernel<T, V, false, true> : rotary_kernel<T, V, false, false>);
    return launch_pdl(kern, grid, dim3(kThreads), 0, s, p, items, heads);
}

__global__ void rotary_init_kernel(float* freq, int rot, double base, int scaling, double factor, double original,
                                   double beta_fast, double beta_slow) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= rot / 2) return;
    if (scaling == 2 && rot > 2) base *= pow(factor, static_cast<double>(rot) / (rot - 2));
    double f = pow(base, -2.0 * i / rot);
    if (scaling == 1) f /= factor;
    if (scaling == 3) {
        // turns within the original length: many keep their frequency, few are stretched
        const double turns = original * f / 6.283185307179586;
        double keep = (turns - beta_slow) / (beta_fast - beta_slow);
        keep = keep < 0.0 ? 0.0 : (keep > 1.0 ? 1.0 : keep);
        f = f * keep + f / factor * (1.0 - keep);
    }
    freq[i] = static_cast<float>(f);
}

}  // namespace

cudaError_t launch_rotary(const RotaryProblem& p, int num_sms, cudaStream_t s) {
    uintptr_t bits = 0;
    for (int w = 0; w < 2; ++w) bits |= reinterpret_cast<uintptr_t>(p.x[w]) | reinterpret_cast<uintptr_t>(p.y[w]);
    // the widest accesses at which every vector of a row is aligned and whole (8 x 16 heads of 4096, bf16, interleaved, 36 of
    // 128 turned: 221 us with two elements, 672 with one)
    auto fits = [&](int v) { return bits % (v * (p.dtype ? 2 : 4)) == 0 && p.d % v == 0 && (p.rot / 2) % v == 0; };
    if (p.dtype) {
        using T = __nv_bfloat16;
        return fits(8) ? rotary_v<T, 8>(p, num_sms, s) : fits(4) ? rotary_v<T, 4>(p, num_sms, s)
             : fits(2) ? rotary_v<T, 2>(p, num_sms, s) : rotary_v<T, 1>(p, num_sms, s);
    }
    return fits(4) ? rotary_v<float, 4>(p, num_sms, s) : fits(2) ? rotary_v<float, 2>(p, num_sms, s)
                                                                 : rotary_v<float, 1>(p, num_sms, s);
}

cudaError_t launch_rotary_init(float* freq, int rot, double base, int scaling, double factor, double original,
                               double beta_fast, double beta_slow, cudaStream_t s) {
    rotary_init_kernel<<<(rot / 2 + 127) / 128, 128, 0, s>>>(freq, rot, base, scaling, factor, original, beta_fast,
                                                             beta_slow);
    return cudaGetLastError();
}

}  // namespace la
