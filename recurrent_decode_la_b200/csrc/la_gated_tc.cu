// la_gated_tc.cu -- the gated recurrence and its gradient on the tensor cores
// (bf16, d_k == d_v == D in {64, 128}, chunks of 128 tokens).  The formulas
// stand in la_gated.h.
//
// Three kernels.  gated_prefill_tc does the prefill in one launch: some of its
// CTAs walk the chunks of the units and write the state at every chunk's start,
// the only serial part; the others turn chunks whose state is there into
// outputs.  For the gradient gated_states_tc walks the units in both directions
// and gated_grad_tc then takes the chunks in any order.  A chunk's addition to
// the state needs no earlier state, so the chain is one multiply-add per element
// and chunk.
//
// What binds them is first the time of an SM, then memory.  A chunk's state costs
// a CTA 2.3 us (three products of 128^3 on decayed keys, whose splitting takes as
// long as the products), its output 3.7 us.  Per 128 tokens at D = 128 the prefill
// has to move 128 KB.  It moves 1.08 times that while the second reading of K and
// V and that of the states hit L2 (B2 H16 T4096), twice that when the states run
// further ahead than L2 reaches (B8 H16 T4096: 1032 MB in 196 us, 80 % of the copy
// rate; evict-first policies on the second readings changed nothing).  B8 H16
// T8192: 420 to 450 us in a long run; the floor of its bytes is 167, and the
// ungated prefill, which walks a unit and makes its outputs in one CTA and reads
// every byte once, takes 215.  (Times that compare two forms below were taken in
// turn in short runs, where this case takes 370.)  The gradient moves 955 MB at
// B4 H16 T4096 where 483 are the least: both states at 72 % of the copy rate
// (145 us of B4 H16 T8192), then the chunks at 58 %, each a chain of seven products and the steps between them that takes a CTA
// 16k clocks (272 us); in all 455 to 485 us, floor 145.
//
// Rounding.  Sums, states and decays are fp32.  An operand of a product is
// rounded to bf16 once where its result is bf16 too (decayed scores, chunk
// states).  Where the result is an fp32 state, the decayed keys (queries) are
// kept as the sum of three bf16 numbers, 2^-24 of them, at the price of two
// more products (two parts would leave the state 2.4e-6 of itself off, three
// 1e-7).  A row's decay is applied to the fp32 accumulator, not to a bf16 operand.
// dg's term e^{G_C} <E, S>, the same for all tokens of a chunk, is an fp32 sum: over
// the fp32 states of a unit's only chunk (summed where the states are made; the
// rounded ones put dg of 32 units of 1 token 0.0029 off, so 0.0017), but over the
// rounded ones of a longer unit's chunks, since their fp32 ones are in two CTAs and
// nowhere at once.  Where that outweighs the other terms and its products nearly
// cancel, dg is further off than dq, dk and dv (one unit of 150 to 500 tokens: 0.0024
// on average and up to 0.0042, the others 0.0025).  With the next eight bits of
// either state beside it the gradient of B4 H16 T8192 took 639 us, not 460.
// The tensor core drops bits when it adds to an accumulator: a state summed there
// over 8192 tokens is off by 9e-6 of itself, so the states live in registers and an
// accumulator spans one chunk only.
//
// Waits are bounded: on expiry the kernel records the device error word, every
// role winds down, copies and products in flight are drained (bounded), tensor
// memory is freed and the kernel returns.
#include <algorithm>

#include "la_device.cuh"
#include "la_gated.h"
#include "la_internal.h"

namespace la {
namespace {

constexpr int C = kGatedTcChunk;
constexpr int kPanel = C * 128;  // 64 bf16 columns of a [128][D] tile
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Poll until f() holds; gives up like mbar_wait.
template <typename F>
__device__ __forceinline__ bool wait_until(uint64_t timeout_ns, volatile int* abort, unsigned int where, F&& f) {
    if (f()) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
        if (f()) return true;
        if ((it & 15u) == 0) {
            if (*abort) return false;
            if (globaltimer_ns() - t0 > timeout_ns) {
                record_timeout(where);
                *abort = 1;
                return false;
            }
        }
    }
}

// Four log gates (times log2 e) of this lane, tokens 4 lane .. 4 lane + 3 of
// the chunk at row0; tokens at nv and behind decay by nothing.
__device__ __forceinline__ void load_gates(const GatedProblem& p, int64_t row0, int nv, float (&x)[4]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float v = 0.f;
        if (p.g != nullptr && 4 * lane + e < nv)
            v = __bfloat162float(static_cast<const __nv_bfloat16*>(p.g)[row0 + 4 * lane + e]);
        v = v < kGateFloor ? kGateFloor : v;
        x[e] = v * kLog2e;
    }
}

// Inclusive prefix sums over the 128 tokens.
__device__ __forceinline__ void scan_up(const float (&x)[4], float (&G)[4]) {
    const int lane = threadIdx.x & 31;
    G[0] = x[0];
#pragma unroll
    for (int e = 1; e < 4; ++e) G[e] = G[e - 1] + x[e];
    float s = G[3];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    float before = __shfl_up_sync(0xffffffffu, s, 1);
    if (lane == 0) before = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) G[e] += before;
}

// Sums over the tokens behind each one (exclusive suffix sums); all = total.
__device__ __forceinline__ void scan_down(const float (&x)[4], float (&B)[4], float& all) {
    const int lane = threadIdx.x & 31;
    B[3] = 0.f;
#pragma unroll
    for (int e = 2; e >= 0; --e) B[e] = B[e + 1] + x[e + 1];
    float s = B[0] + x[0];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float y = __shfl_down_sync(0xffffffffu, s, o);
        if (lane + o < 32) s += y;
    }
    float behind = __shfl_down_sync(0xffffffffu, s, 1);
    if (lane == 31) behind = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) B[e] += behind;
    all = __shfl_sync(0xffffffffu, s, 0);
}

// Where the states' kernel of the gradient leaves e^{G_C} <E, S_0> of a unit's only chunk for the chunks' kernel, a number
// a state warp: the row of dq that the chunk's first token will take.
template <int D>
__device__ __forceinline__ float* alone_sums(const GatedProblem& p, int64_t row0) {
    return reinterpret_cast<float*>(static_cast<uint16_t*>(p.dq) + row0 * D);
}

// Zero rows nv .. 127 of a [128][D] tile (one warp).
template <int D>
__device__ __forceinline__ void zero_rows(uint32_t tile, int nv) {
    const int n = (C - nv) * (D / 8);
    for (int i = threadIdx.x & 31; i < n; i += 32) {
        const int row = nv + i / (D / 8), ch = i % (D / 8);
        st_shared_v4(tile + (ch >> 3) * kPanel + row * 128 + (ch & 7) * 16, 0u, 0u, 0u, 0u);
    }
}

// The kernels below work on accumulator rows 16 columns at a time in loops that are kept rolled: no slower than whole rows
// unrolled (the gradient up to 3 % faster), and twenty warps in different roles share the instruction cache.

// 16 fp32 values of a row -> bf16, two 16-byte pieces of a 128-byte swizzled panel row.
__device__ __forceinline__ void put_row16(uint32_t panel, int row, int chunk0, const float (&x)[16]) {
#pragma unroll
    for (int ch = 0; ch < 2; ++ch)
        st_shared_v4(panel + sw128_off(row, chunk0 + ch), pack_bf16x2(x[8 * ch], x[8 * ch + 1]),
                     pack_bf16x2(x[8 * ch + 2], x[8 * ch + 3]), pack_bf16x2(x[8 * ch + 4], x[8 * ch + 5]),
                     pack_bf16x2(x[8 * ch + 6], x[8 * ch + 7]));
}
// The same straight to global memory.
__device__ __forceinline__ void put_row16(uint16_t* out, const float (&x)[16]) {
#pragma unroll
    for (int ch = 0; ch < 2; ++ch)
        reinterpret_cast<uint4*>(out)[ch] =
            make_uint4(pack_bf16x2(x[8 * ch], x[8 * ch + 1]), pack_bf16x2(x[8 * ch + 2], x[8 * ch + 3]),
                       pack_bf16x2(x[8 * ch + 4], x[8 * ch + 5]), pack_bf16x2(x[8 * ch + 6], x[8 * ch + 7]));
}

__device__ __forceinline__ void ld16f(uint32_t taddr, float (&x)[16]) {
    uint32_t r[16];
    tmem_ld16(taddr, r);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        asm volatile("" : "+r"(r[i]));
        x[i] = __uint_as_float(r[i]);
    }
}

// Two loads in flight, one wait.
__device__ __forceinline__ void ld16f2(uint32_t ta, uint32_t tb, float (&x)[16], float (&y)[16]) {
    uint32_t r[16], q[16];
    tmem_ld16(ta, r);
    tmem_ld16(tb, q);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        asm volatile("" : "+r"(r[i]), "+r"(q[i]));
        x[i] = __uint_as_float(r[i]);
        y[i] = __uint_as_float(q[i]);
    }
}

__device__ __forceinline__ uint32_t tile_k(uint32_t tile, int ks, uint32_t panel) {  // K-major step ks
    return tile + (ks >> 2) * panel + (ks & 3) * 32;
}

// ---------------------------------------------------------------------------
// States.  A work item is a segment of a unit (mostly all of it), forward: X = K,
// Y = V; for the gradient also in reverse: X = Q, Y = dO.  The units of packed input come longest first
// (p.order): for the gradient dealt to the CTAs in turn and back, so that no CTA
// gets the longer item of every round; in the prefill claimed from a counter.
// Per chunk
//     U = X'^T Y (X' = the decayed rows, as the sum of three bf16 numbers),
//     S = gamma S + U.
//   warp 0       TMA producer        warp 1  MMA issuer
//   warp 2       decays of the chunk's tokens
//   warps 4-11   X -> its three decayed parts.  At D = 128 transposed into
//                tensor memory, whence the product takes them: with the parts
//                in shared memory its bandwidth (parts written and read, 3.6k
//                clocks a chunk) binds.  At D = 64 in shared memory, the high
//                part in place.
//   warps 12-19  (12-15 at D = 64) the state, 64 columns of a row per thread
// ---------------------------------------------------------------------------
template <int D>
struct StCfg {
    static constexpr int kThreads = 640;
    static constexpr int NPAN = D / 64;
    static constexpr int TILE = C * D * 2;
    static constexpr bool TS = D == 128;    // decayed parts in tensor memory
    static constexpr int STAGE = 2 * TILE;  // X, Y
    static constexpr int NS = D == 128 ? 3 : 4;
    static constexpr int NL = 2;            // buffers of the decayed parts
    static constexpr int NU = TS ? 1 : 2;   // accumulators
    static constexpr int SB = D * D * 2, SB_PANEL = D * 128;
    static constexpr int kGam = 8;  // live gammas: those of at most six chunks
    static constexpr int OFF_LO = NS * STAGE;
    static constexpr int OFF_SB = OFF_LO + (TS ? 0 : NL * 2 * TILE);
    static constexpr int OFF_W = OFF_SB + SB;
    static constexpr int NW = 2;            // sets of decays, each [3][128] bf16: w = w0 + w1 + w2
    static constexpr int OFF_GAM = OFF_W + NW * 3 * C * 2;
    static constexpr int kItems = 4;  // claimed items that the roles may be apart
    static constexpr int OFF_ITEMS = OFF_GAM + kGam * 4;
    static constexpr int OFF_BAR = OFF_ITEMS + kItems * 4;
    static constexpr int B_FULL = 0, B_EMPTY = NS, B_GFULL = 2 * NS, B_SCALED = 3 * NS, B_UFULL = 4 * NS,
                         B_UEMPTY = 4 * NS + NU, B_DONE = 4 * NS + 2 * NU, B_LOEMPTY = B_DONE + 1, B_IFULL = B_LOEMPTY + NL,
                         B_IEMPTY = B_IFULL + kItems, NBAR = B_IEMPTY + kItems;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
    static constexpr int OFF_STORED = OFF_MISC + 8;  // chunks stored, a word for each state warp
    static constexpr int SMEM = OFF_STORED + 4 * NPAN * 4 + 8 + 1024;
    // columns of part k of buffer l (TS)
    static constexpr int tm_part(int l, int k) { return NU * D + (l * 3 + k) * 64; }
    static_assert(SMEM <= 232448, "shared memory");
};

// `worker` of `workers` CTAs; smem 1 KB aligned, tmem all 512 columns.  With p.queue (prefill) the slots are published as
// their states are stored.  ALONE: units of one chunk may be among them (their sums for dg are made here; that takes
// registers, which others need not pay for).
template <int D, bool ALONE>
__device__ __forceinline__ void gated_states_body(const GatedMaps& m, const GatedProblem& p, int64_t n_items, bool grad,
                                                  uint8_t* smem, uint32_t tmem, int64_t worker, int64_t workers) {
    using Cfg = StCfg<D>;
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + Cfg::OFF_BAR);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::OFF_MISC);
    const uint32_t stored = smem_u32(smem + Cfg::OFF_STORED);
    float* gam = reinterpret_cast<float*>(smem + Cfg::OFF_GAM);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint64_t tmo = p.timeout_ns;
    const uint32_t sbase = smem_u32(smem);

    if (threadIdx.x == 0) {
        for (int s = 0; s < Cfg::NS; ++s) {
            mbar_init(&bar[Cfg::B_FULL + s], 1);
            mbar_init(&bar[Cfg::B_EMPTY + s], 1);
            mbar_init(&bar[Cfg::B_GFULL + s], 1);
            mbar_init(&bar[Cfg::B_SCALED + s], 8);
        }
        for (int b = 0; b < Cfg::NU; ++b) {
            mbar_init(&bar[Cfg::B_UFULL + b], 1);
            mbar_init(&bar[Cfg::B_UEMPTY + b], 4 * Cfg::NPAN);
        }
        mbar_init(&bar[Cfg::B_DONE], 1);
        for (int l = 0; l < Cfg::NL; ++l) mbar_init(&bar[Cfg::B_LOEMPTY + l], 1);
        for (int r = 0; r < Cfg::kItems; ++r) {
            mbar_init(&bar[Cfg::B_IFULL + r], 1);
            mbar_init(&bar[Cfg::B_IEMPTY + r], 3 + 8 + 4 * Cfg::NPAN);
        }
        *abort_flag = 0;
        for (int w = 0; w < 4 * Cfg::NPAN; ++w)
            reinterpret_cast<volatile unsigned int*>(smem + Cfg::OFF_STORED)[w] = 0;
        fence_barrier_init();
    }
    __syncthreads();

    // Claimed items (prefill): the producer takes them from the counter and publishes them to the other roles, whose
    // threads are a whole warp or its lane 0 alone.
    enum Role { kProducer, kLane, kWarp };
    volatile int* claimed = reinterpret_cast<volatile int*>(smem + Cfg::OFF_ITEMS);
    auto claim = [&](Role role, int64_t k, int64_t& i) -> bool {
        const int r = static_cast<int>(k % Cfg::kItems);
        const uint32_t ph = static_cast<uint32_t>(k / Cfg::kItems) & 1;
        if (role == kProducer) {
            const unsigned int at = atomicAdd(&p.queue[3], 1u);
            i = at < n_items ? static_cast<int64_t>(at) : -1;
            if (k >= Cfg::kItems && !mbar_wait(&bar[Cfg::B_IEMPTY + r], ph ^ 1u, abort_flag, tmo, 0x660)) return false;
            claimed[r] = static_cast<int>(i);
            mbar_arrive(&bar[Cfg::B_IFULL + r]);
            return true;
        }
        if (!(role == kWarp ? mbar_wait_warp(&bar[Cfg::B_IFULL + r], ph, abort_flag, tmo, 0x661)
                            : mbar_wait(&bar[Cfg::B_IFULL + r], ph, abort_flag, tmo, 0x662)))
            return false;
        i = claimed[r];
        if (role == kWarp) __syncwarp();
        if (lane == 0) mbar_arrive(&bar[Cfg::B_IEMPTY + r]);
        return true;
    };
    // Calls f(unit, its state, reverse, segment, chunks of the unit, first and last of the walk) for every item of this CTA
    // until f gives up.
    auto items = [&](Role role, auto&& f) {
        for (int64_t k = 0;; ++k) {
            int64_t i;
            if (p.queue != nullptr) {
                if (!claim(role, k, i)) return false;
                if (i < 0) return true;
            } else {
                i = k * workers + (k & 1 ? workers - 1 - worker : worker);
                if (k * workers >= n_items) return true;
                if (i >= n_items) continue;
            }
            int seg = 0;
            if (p.segs > 1) {
                seg = static_cast<int>(i % p.segs);
                i /= p.segs;
            }
            const bool rev = grad && (i & 1);
            int64_t u = grad ? i >> 1 : i;
            if (p.order != nullptr) u = static_cast<int64_t>(p.order[u / p.H]) * p.H + u % p.H;
            const GatedUnit un = gated_unit(p, u);
            const int nch = gated_chunks(un.len, C), cc0 = seg * p.seg_chunks, cc1 = min(nch, cc0 + p.seg_chunks);
            if (cc0 >= cc1 || (p.sums && cc1 == nch)) continue;  // (nothing starts from the last one's sum)
            if (!f(un, u, rev, seg, nch, cc0, cc1)) return false;
        }
    };
    // Calls f(unit, reverse, chunk, rows of it, chunks before it, item, whether it begins the item) for every chunk of them.
    auto walk = [&](Role role, auto&& f) -> bool {
        int64_t g = 0;
        return items(role, [&](const GatedUnit& un, int64_t u, bool rev, int seg, int nch, int cc0, int cc1) {
            const int64_t item = ((rev ? p.n_units : 0) + u) * p.segs + seg;
            for (int cc = cc0; cc < cc1; ++cc, ++g) {
                const int c = rev ? nch - 1 - cc : cc;
                if (!f(un, rev, c, min(C, un.len - c * C), g, item, cc == cc0)) return false;
            }
            return true;
        });
    };

    if (warp == 0) {
        if (lane == 0) {
            int64_t started = 0;
            auto coords = [&](const GatedUnit& un, int c, int& row, int& group) {
                const int64_t r = un.row0 + static_cast<int64_t>(c) * C;
                group = static_cast<int>(un.row0 / p.rows);
                row = static_cast<int>(r - group * p.rows);
            };
            const bool ok = walk(kProducer, [&](const GatedUnit& un, bool rev, int c, int, int64_t g, int64_t, bool) {
                const int s = static_cast<int>(g % Cfg::NS);
                if (g >= Cfg::NS &&
                    !mbar_wait(&bar[Cfg::B_EMPTY + s], ((g / Cfg::NS) + 1) & 1, abort_flag, tmo, 0x600 + s))
                    return false;
                const CUtensorMap* mx = rev ? &m.q : &m.k;
                const CUtensorMap* my = rev ? &m.d_o : &m.v;
                int row, group;
                coords(un, c, row, group);
                mbar_arrive_expect_tx(&bar[Cfg::B_FULL + s], 2 * Cfg::TILE);
                uint8_t* st = smem + s * Cfg::STAGE;
#pragma unroll
                for (int pn = 0; pn < Cfg::NPAN; ++pn) {
                    tma_load_3d(st + pn * kPanel, mx, &bar[Cfg::B_FULL + s], pn * 64, row, group);
                    tma_load_3d(st + Cfg::TILE + pn * kPanel, my, &bar[Cfg::B_FULL + s], pn * 64, row, group);
                }
                started = g + 1;
                const int c2 = rev ? c - 1 : c + 1;
                if (c2 >= 0 && c2 < gated_chunks(un.len, C)) {
                    coords(un, c2, row, group);
#pragma unroll
                    for (int pn = 0; pn < Cfg::NPAN; ++pn) {
                        tma_prefetch_l2_3d(mx, pn * 64, row, group);
                        tma_prefetch_l2_3d(my, pn * 64, row, group);
                    }
                }
                return true;
            });
            if (!ok || *abort_flag)
                for (int64_t g = started > Cfg::NS ? started - Cfg::NS : 0; g < started; ++g)
                    mbar_wait_drain(&bar[Cfg::B_FULL + g % Cfg::NS], (g / Cfg::NS) & 1, tmo);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t kId = idesc_bf16_f32(D, D, !Cfg::TS, true);
            bool issued = false;
            walk(kLane, [&](const GatedUnit&, bool, int, int, int64_t g, int64_t, bool) {
                const int s = static_cast<int>(g % Cfg::NS), b = static_cast<int>(g % Cfg::NU), l = static_cast<int>(g % Cfg::NL);
                if (!mbar_wait(&bar[Cfg::B_SCALED + s], (g / Cfg::NS) & 1, abort_flag, tmo, 0x610 + s)) return false;
                if (g >= Cfg::NU &&
                    !mbar_wait(&bar[Cfg::B_UEMPTY + b], ((g / Cfg::NU) + 1) & 1, abort_flag, tmo, 0x618 + b))
                    return false;
                tc_fence_after();
                const uint32_t x = sbase + s * Cfg::STAGE, y = x + Cfg::TILE,
                               lo = sbase + Cfg::OFF_LO + l * 2 * Cfg::TILE;
                // the smallest part first
#pragma unroll
                for (int part = 2; part >= 0; --part) {
#pragma unroll
                    for (int ks = 0; ks < C / 16; ++ks) {
                        const uint64_t yd = sdesc_sw128(y + ks * 2048, kPanel, 1024);
                        const uint32_t acc = part < 2 || ks > 0;
                        if constexpr (Cfg::TS)
                            mma_bf16_ts(tmem + b * D, tmem + Cfg::tm_part(l, part) + ks * 8, yd, kId, acc);
                        else
                            mma_bf16_ss(tmem + b * D,
                                        sdesc_sw128((part == 0 ? x : lo + (part - 1) * Cfg::TILE) + ks * 2048, kPanel, 1024),
                                        yd, kId, acc);
                    }
                    if (part == (Cfg::TS ? 0 : 1)) mma_commit(&bar[Cfg::B_LOEMPTY + l]);
                }
                mma_commit(&bar[Cfg::B_EMPTY + s]);
                mma_commit(&bar[Cfg::B_UFULL + b]);
                issued = true;
                return true;
            });
            if (issued) {
                mma_commit(&bar[Cfg::B_DONE]);
                mbar_wait_drain(&bar[Cfg::B_DONE], 0, tmo);
            }
        }
        __syncwarp();
    } else if (warp == 2) {
        float decay = 0.f;  // log2 of the segment's
        walk(kWarp, [&](const GatedUnit& un, bool rev, int c, int nv, int64_t g, int64_t item, bool first) {
            const int s = static_cast<int>(g % Cfg::NS);
            float x[4], w[4], all;
            load_gates(p, un.row0 + static_cast<int64_t>(c) * C, nv, x);
            if (rev) {
                scan_up(x, w);
                all = __shfl_sync(0xffffffffu, w[3], 31);
            } else {
                scan_down(x, w, all);
            }
            if (g >= 2 && !mbar_wait_warp(&bar[Cfg::B_SCALED + (g - 2) % Cfg::NS], ((g - 2) / Cfg::NS) & 1, abort_flag,
                                          tmo, 0x620 + s))
                return false;
            uint2* o = reinterpret_cast<uint2*>(smem + Cfg::OFF_W + (g % Cfg::NW) * 3 * C * 2);
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = ex2(w[e]);
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                const uint2 h = make_uint2(pack_bf16x2(w[0], w[1]), pack_bf16x2(w[2], w[3]));
                o[32 * k + lane] = h;
                w[0] -= bf16_lo(h.x);
                w[1] -= bf16_hi(h.x);
                w[2] -= bf16_lo(h.y);
                w[3] -= bf16_hi(h.y);
            }
            if (lane == 0) gam[g % Cfg::kGam] = ex2(all);
            if (p.sums) {
                decay = first ? all : decay + all;
                if (lane == 0) p.seg_decays[item] = decay;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[Cfg::B_GFULL + s]);
            return true;
        });
    } else if (warp == 3) {
        // Publish a chunk's slot once every state warp's part of it is in global memory: each warp counts for itself.  (A
        // sum over the warps would not do: one that has counted the next chunk already makes up for one whose store of this
        // chunk is still on its way, since a warp lets the next product start before it waits for its store.)
        if (lane == 0 && p.queue != nullptr) {
            walk(kLane, [&](const GatedUnit& un, bool, int c, int, int64_t g, int64_t, bool) {
                const unsigned int want = static_cast<unsigned int>(g + 1);
                for (int w = 0; w < 4 * Cfg::NPAN; ++w)
                    if (!wait_until(tmo, abort_flag, 0x650, [&] {
                            unsigned int have;
                            asm volatile("ld.acquire.cta.shared.u32 %0, [%1];" : "=r"(have) : "r"(stored + 4 * w) : "memory");
                            return static_cast<int>(have - want) >= 0;
                        }))
                        return false;
                __threadfence();
                const unsigned int at = atomicAdd(&p.queue[0], 1u);
                asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p.queue + kQueueHead + at),
                             "r"(static_cast<unsigned int>(un.slot0 + c) + 1u)
                             : "memory");
                return true;
            });
        }
        __syncwarp();
    } else if (warp >= 4 && warp < 12) {
        walk(kWarp, [&](const GatedUnit&, bool, int, int nv, int64_t g, int64_t, bool) {
            const int s = static_cast<int>(g % Cfg::NS);
            const uint32_t ph = (g / Cfg::NS) & 1;
            if (!mbar_wait_warp(&bar[Cfg::B_GFULL + s], ph, abort_flag, tmo, 0x630 + s)) return false;
            if (!mbar_wait_warp(&bar[Cfg::B_FULL + s], ph, abort_flag, tmo, 0x638 + s)) return false;
            const uint32_t x = sbase + s * Cfg::STAGE, y = x + Cfg::TILE;
            const uint32_t* w = reinterpret_cast<const uint32_t*>(smem + Cfg::OFF_W + (g % Cfg::NW) * 3 * C * 2);
            // w x = hi + mid + lo for two values at a time, in paired bf16 arithmetic.  A product of two 8-bit
            // significands has 16 bits, so w0 x = hi + r exactly; mid = r + p with p = w1 x rounded, and m - r is
            // exact, so w1 x - (m - r) is what both roundings lost.  A state is 1e-7 of itself off; 2.4e-6 where lo
            // takes only (w1 + w2) x, which saves three operations and 5 % of the time.
            auto split = [](uint32_t x2, uint32_t w0, uint32_t w1, uint32_t w2, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
                auto b = [](uint32_t u) { return *reinterpret_cast<__nv_bfloat162*>(&u); };
                auto u = [](__nv_bfloat162 v) { return *reinterpret_cast<uint32_t*>(&v); };
                const __nv_bfloat162 x = b(x2), h = __hmul2_rn(b(w0), x), r = __hfma2(b(w0), x, __hneg2(h)),
                                     m = __hadd2_rn(r, __hmul2_rn(b(w1), x)), q = __hsub2_rn(m, r);
                hi = u(h);
                mid = u(m);
                lo = u(__hfma2(b(w2), x, __hfma2(b(w1), x, __hneg2(q))));
            };
            const bool lofree = g < Cfg::NL;
            const uint32_t loph = ((g / Cfg::NL) + 1) & 1;
            if constexpr (Cfg::TS) {
                // lanes = columns of X: this warp's 32 of them, in two groups of 16, and 64 of the tokens
                const int sub = warp & 3, half = (warp - 4) >> 2;
                if (nv < C)
                    for (int row = nv + (warp - 4); row < C; row += 8)
                        if (lane < 16) st_shared_v4(y + (lane >> 3) * kPanel + row * 128 + (lane & 7) * 16, 0u, 0u, 0u, 0u);
                if (!lofree && !mbar_wait_warp(&bar[Cfg::B_LOEMPTY + g % Cfg::NL], loph, abort_flag, tmo, 0x648))
                    return false;
                tc_fence_after();
                const uint32_t tp = tmem + Cfg::tm_part(g % Cfg::NL, 0) + half * 32 + (static_cast<uint32_t>(sub * 32) << 16);
#pragma unroll 1
                for (int kk = 0; kk < 4; kk += 2) {  // 32 tokens
                    uint32_t part[2][3][8];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t wr[2][3];  // decays of token pairs t0, t0 + 1 and t0 + 8, t0 + 9
                        const int t0 = 64 * half + 16 * (kk + k) + 2 * (lane & 3);
#pragma unroll
                        for (int r = 0; r < 2; ++r)
#pragma unroll
                            for (int e = 0; e < 3; ++e) wr[r][e] = w[64 * e + (t0 >> 1) + 4 * r];
#pragma unroll
                        for (int grp = 0; grp < 2; ++grp) {
                            const int c0 = 4 * sub + 2 * grp;  // first 16-byte piece of the 16 columns
                            const int tok = 64 * half + 16 * (kk + k) + (lane & 7) + ((lane >> 4) << 3),
                                      ch = (c0 & 7) + ((lane >> 3) & 1);
                            uint32_t a[4];
                            ldmatrix_x4_trans(x + (c0 >> 3) * kPanel + sw128_off(tok, ch), a[0], a[1], a[2], a[3]);
                            if (nv < C) {
#pragma unroll
                                for (int r = 0; r < 4; ++r) {
                                    const int t = t0 + 8 * (r >> 1);
                                    a[r] &= (t < nv ? 0xffffu : 0u) | (t + 1 < nv ? 0xffff0000u : 0u);
                                }
                            }
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                split(a[r], wr[r >> 1][0], wr[r >> 1][1], wr[r >> 1][2], part[grp][0][4 * k + r],
                                      part[grp][1][4 * k + r], part[grp][2][4 * k + r]);
                        }
                    }
#pragma unroll
                    for (int grp = 0; grp < 2; ++grp)
#pragma unroll
                        for (int e = 0; e < 3; ++e)
                            tmem_st_16x128b_x4(tp + e * 64 + kk * 8 + (static_cast<uint32_t>(grp * 16) << 16), part[grp][e]);
                }
                tmem_wait_st();
                tc_fence_before();
            } else {
                const uint32_t lo = sbase + Cfg::OFF_LO + (g % Cfg::NL) * 2 * Cfg::TILE;
                if (!lofree && !mbar_wait_warp(&bar[Cfg::B_LOEMPTY + g % Cfg::NL], loph, abort_flag, tmo, 0x648))
                    return false;
                // warp w takes rows 16 (w - 4) ..; its lanes four rows of eight 16-byte pieces at a time
                const int r0 = (warp - 4) * 16 + (lane >> 3);
                uint32_t a[4][4];
#pragma unroll
                for (int it = 0; it < 4; ++it)
                    ld_shared_v4(x + (r0 + 4 * it) * 128 + (lane & 7) * 16, a[it][0], a[it][1], a[it][2], a[it][3]);
#pragma unroll
                for (int it = 0; it < 4; ++it) {
                    const int row = r0 + 4 * it;
                    const uint32_t at = row * 128 + (lane & 7) * 16;
                    uint32_t hi[4], l[4], l2[4], wr[3];
#pragma unroll
                    for (int k = 0; k < 3; ++k) {  // the row's decay in both halves
                        const uint32_t both = w[64 * k + (row >> 1)];
                        wr[k] = __byte_perm(both, 0u, row & 1 ? 0x3232 : 0x1010);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        split(row < nv ? a[it][e] : 0u, wr[0], wr[1], wr[2], hi[e], l[e], l2[e]);
                    if (row >= nv) st_shared_v4(y + at, 0u, 0u, 0u, 0u);
                    st_shared_v4(x + at, hi[0], hi[1], hi[2], hi[3]);
                    st_shared_v4(lo + at, l[0], l[1], l[2], l[3]);
                    st_shared_v4(lo + Cfg::TILE + at, l2[0], l2[1], l2[2], l2[3]);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[Cfg::B_SCALED + s]);
            return true;
        });
    } else if (warp >= 12 && warp < 12 + 4 * Cfg::NPAN) {
        const int sub = warp & 3, half = (warp - 12) >> 2;
        const int row = D == 128 ? sub * 32 + lane : (lane < 16 ? sub * 16 + lane : -1);
        const uint32_t lane_off = (static_cast<uint32_t>(sub * 32) << 16) + half * 64;
        uint8_t* panel = smem + Cfg::OFF_SB + half * Cfg::SB_PANEL;
        constexpr int kRows = D / 4;  // rows of this warp
        float S[64];
        int64_t g = 0;
        auto count_stored = [&] {  // this warp's parts of g chunks are in global memory
            asm volatile("st.release.cta.shared.u32 [%0], %1;" ::"r"(stored + 4 * (warp - 12)), "r"(static_cast<unsigned int>(g))
                         : "memory");
        };
        items(kWarp, [&](const GatedUnit& un, int64_t u, bool rev, int seg, int nch, int cc0, int cc1) {
            const int64_t item = ((rev ? p.n_units : 0) + u) * p.segs + seg;
            const float* in = rev ? p.dstate : (p.state ? p.state : p.s0);
            float* out = rev ? p.dstate : p.state;
            if (p.segs > 1) {
                // offset so that the indices of `at` below hold
                float* start = p.seg_states + (item - u) * D * D;
                in = p.sums ? nullptr : start;
                out = p.sums ? start : (cc1 == nch ? out : nullptr);
            }
            const int64_t at = u * D * D + static_cast<int64_t>(row < 0 ? 0 : row) * D + half * 64;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const float4 f = in && row >= 0 ? reinterpret_cast<const float4*>(in + at)[j] : make_float4(0, 0, 0, 0);
                S[4 * j] = f.x;
                S[4 * j + 1] = f.y;
                S[4 * j + 2] = f.z;
                S[4 * j + 3] = f.w;
            }
            uint8_t* slots = static_cast<uint8_t*>(rev ? p.e_states : p.s_states) + un.slot0 * Cfg::SB;
            for (int cc = cc0; cc < cc1; ++cc, ++g) {
                const int c = rev ? nch - 1 - cc : cc;
                const int b = static_cast<int>(g % Cfg::NU);
                if (!p.sums) {  // the state before this chunk, as bf16, to its slot
                    if (lane == 0) bulk_wait_group_read<0>();
                    __syncwarp();
                    if (row >= 0) {
#pragma unroll
                        for (int ch = 0; ch < 8; ++ch)
                            st_shared_v4(smem_u32(panel) + sw128_off(row, ch), pack_bf16x2(S[8 * ch], S[8 * ch + 1]),
                                         pack_bf16x2(S[8 * ch + 2], S[8 * ch + 3]),
                                         pack_bf16x2(S[8 * ch + 4], S[8 * ch + 5]),
                                         pack_bf16x2(S[8 * ch + 6], S[8 * ch + 7]));
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        const int off = half * Cfg::SB_PANEL + sub * kRows * 128;
                        bulk_store(slots + static_cast<int64_t>(c) * Cfg::SB + off, smem + Cfg::OFF_SB + off, kRows * 128);
                        bulk_commit_group();
                        if (g > 0) {  // the part of the chunk before is in global memory
                            bulk_wait_group<1>();
                            count_stored();
                        }
                    }
                }
                if (!mbar_wait_warp(&bar[Cfg::B_UFULL + b], (g / Cfg::NU) & 1, abort_flag, tmo, 0x640 + b)) return false;
                tc_fence_after();
                const float gamma = gam[g % Cfg::kGam];
                if (ALONE && rev && nch == 1) {
                    // The unit's only chunk: its states, E and S_0, are both at hand in fp32.  Half of the decay on either side.
                    float dot = 0.f;
                    const float half_decay = sqrtf(gamma);
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (p.s0 != nullptr && row >= 0) x = reinterpret_cast<const float4*>(p.s0 + at)[j];
                        dot = fmaf(half_decay * x.x, half_decay * S[4 * j], dot);
                        dot = fmaf(half_decay * x.y, half_decay * S[4 * j + 1], dot);
                        dot = fmaf(half_decay * x.z, half_decay * S[4 * j + 2], dot);
                        dot = fmaf(half_decay * x.w, half_decay * S[4 * j + 3], dot);
                        __syncwarp();  // one load at a time: sixteen would take the registers of S
                    }
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
                    if (lane == 0) alone_sums<D>(p, un.row0)[warp - 12] = dot;
                }
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    float x[16];
                    ld16f(tmem + lane_off + b * D + h * 16, x);
#pragma unroll
                    for (int j = 0; j < 16; ++j) S[h * 16 + j] = fmaf(gamma, S[h * 16 + j], x[j]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[Cfg::B_UEMPTY + b]);
            }
            if (out && row >= 0) {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    reinterpret_cast<float4*>(out + at)[j] =
                        make_float4(S[4 * j], S[4 * j + 1], S[4 * j + 2], S[4 * j + 3]);
            }
            // The last chunk too, here and not at the next item's first: the publisher waits for it before it looks at another
            // item, and the items behind may be empty ones, more of them than the producer may be ahead of the publisher.
            if (lane == 0 && !p.sums) {
                bulk_wait_group<0>();
                count_stored();
            }
            return true;
        });
        if (lane == 0) bulk_wait_group<0>();
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x == 0)
        for (int b = 0; b < Cfg::NBAR; ++b) mbar_inval(&bar[b]);
    __syncthreads();
}

// ---------------------------------------------------------------------------
// Output of the chunks.  Per chunk
//     A = Q K^T,  P_ij = e^{G_i - G_j} A_ij (j <= i),  O = e^{G_i} (Q S) + P V.
// The decay of a whole 32 x 32 block left of the diagonal is the product of a
// column's factor, e^{R - G_j} with R the prefix at the block's end, and a
// row's, e^{G_i - R}; only the diagonal blocks take an exponential per element.
//   warp 0       TMA producer        warps 1, 3  MMA issuers (output; scores,
//                which must not wait behind the output of the chunk before)
//   warp 2       decays; zeroes the rows behind a sequence's end in V
//   warps 4-11   scores -> P (bf16, over the scores in tensor memory); two warps
//                share 32 rows, 64 keys each
//   warps 12-19  (12-15 at D = 64) O -> bf16, staged in the chunk's Q tile -> TMA store
// ---------------------------------------------------------------------------
template <int D>
struct OutCfg {
    static constexpr int kThreads = 640;
    static constexpr int NPAN = D / 64;
    static constexpr int TILE = C * D * 2;
    static constexpr int STAGE = 3 * TILE;
    static constexpr int NS = D == 128 ? 2 : 4;
    static constexpr int SB = D * D * 2, SB_PANEL = D * 128;
    static constexpr int OFF_SB = NS * STAGE;
    static constexpr int OFF_G = OFF_SB + SB;  // [NS]: 128 prefix sums, 96 column factors (the last block needs none)
    static constexpr int G_BYTES = (C + 96) * 4;
    static constexpr int kRing = NS;  // published chunks
    static constexpr int OFF_RING = OFF_G + NS * G_BYTES;
    static constexpr int OFF_BAR = OFF_RING + kRing * 16;
    static constexpr int B_FULL = 0, B_EMPTY = NS, B_GFULL = 2 * NS, B_SFULL = 3 * NS, B_SEMPTY = 3 * NS + 1,
                         B_AFULL = 3 * NS + 2, B_PFULL = 3 * NS + 4, B_OFULL = 3 * NS + 6, B_OEMPTY = 3 * NS + 7,
                         B_DONE = 3 * NS + 8, B_PEMPTY = 3 * NS + 10, B_UFULL = 3 * NS + 12, B_UEMPTY = B_UFULL + NS,
                         NBAR = B_UEMPTY + NS;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
    static constexpr int SMEM = OFF_MISC + 16 + 1024;
    static constexpr int TM_A = 0, TM_O1 = 256, TM_O2 = 256 + D;
    static_assert(SMEM <= 232448, "shared memory");
};

template <int D>
__device__ __forceinline__ void gated_out_body(const GatedMaps& m, const GatedProblem& p, uint8_t* smem, uint32_t tmem) {
    using Cfg = OutCfg<D>;
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + Cfg::OFF_BAR);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::OFF_MISC);
    volatile int4* ring = reinterpret_cast<volatile int4*>(smem + Cfg::OFF_RING);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint64_t tmo = p.timeout_ns;
    const uint32_t sbase = smem_u32(smem);

    if (threadIdx.x == 0) {
        for (int s = 0; s < Cfg::NS; ++s) {
            mbar_init(&bar[Cfg::B_FULL + s], 1);
            mbar_init(&bar[Cfg::B_EMPTY + s], 4 * Cfg::NPAN);
            mbar_init(&bar[Cfg::B_GFULL + s], 1);
        }
        mbar_init(&bar[Cfg::B_SFULL], 1);
        mbar_init(&bar[Cfg::B_SEMPTY], 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&bar[Cfg::B_AFULL + b], 1);
            mbar_init(&bar[Cfg::B_PFULL + b], 8);
            mbar_init(&bar[Cfg::B_PEMPTY + b], 1);
        }
        mbar_init(&bar[Cfg::B_OFULL], 1);
        mbar_init(&bar[Cfg::B_OEMPTY], 4 * Cfg::NPAN);
        mbar_init(&bar[Cfg::B_DONE], 1);
        mbar_init(&bar[Cfg::B_DONE + 1], 1);
        for (int r = 0; r < Cfg::kRing; ++r) {
            mbar_init(&bar[Cfg::B_UFULL + r], 1);
            mbar_init(&bar[Cfg::B_UEMPTY + r], 3 + 8 + 4 * Cfg::NPAN);
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    __syncthreads();

    // Calls f(chunk, chunks before it) for every chunk that the producer publishes in the ring (`one`: by lane 0 alone).
    auto walk = [&](bool one, auto&& f) -> bool {
        for (int64_t g = 0;; ++g) {
            const int r = static_cast<int>(g % Cfg::kRing);
            const uint32_t ph = static_cast<uint32_t>(g / Cfg::kRing) & 1;
            if (!(one ? mbar_wait(&bar[Cfg::B_UFULL + r], ph, abort_flag, tmo, 0x770)
                      : mbar_wait_warp(&bar[Cfg::B_UFULL + r], ph, abort_flag, tmo, 0x771)))
                return false;
            const int row = ring[r].x, group = ring[r].y, nv = ring[r].z;
            if (!one) __syncwarp();
            if (lane == 0) mbar_arrive(&bar[Cfg::B_UEMPTY + r]);
            if (nv <= 0) return true;
            if (!f(GatedChunk{group * p.rows + row, group, row, nv, false}, g)) return false;
        }
    };

    if (warp == 0) {
        if (lane == 0) {
            int64_t started = 0, loaded = 0;  // chunks whose tiles, whose state are under way
            const int64_t total = p.cu ? static_cast<int64_t>(p.queue[2]) * p.H : p.groups * p.nc;
            const bool ok = [&] {
                for (int64_t g = 0;; ++g) {
                    // the next chunk in the order in which the states come to be
                    const unsigned int at = atomicAdd(&p.queue[1], 1u);
                    unsigned int entry = 0;
                    GatedChunk ch = {0, 0, 0, 0, false};
                    if (at < total) {
                        if (!wait_until(tmo, abort_flag, 0x772, [&] {
                                asm volatile("ld.acquire.gpu.global.u32 %0, [%1];"
                                             : "=r"(entry)
                                             : "l"(p.queue + kQueueHead + at)
                                             : "memory");
                                if (entry == 0) __nanosleep(40);
                                return entry != 0;
                            }))
                            return false;
                        asm volatile("fence.proxy.async;" ::: "memory");  // the state: another SM's writes, read by a copy
                        ch = gated_chunk(p, entry - 1, C);
                    }
                    const int r = static_cast<int>(g % Cfg::kRing), s = static_cast<int>(g % Cfg::NS);
                    if (g >= Cfg::kRing &&
                        !mbar_wait(&bar[Cfg::B_UEMPTY + r], ((g / Cfg::kRing) + 1) & 1, abort_flag, tmo, 0x773))
                        return false;
                    ring[r].x = ch.row;
                    ring[r].y = ch.group;
                    ring[r].z = ch.nv;
                    mbar_arrive(&bar[Cfg::B_UFULL + r]);
                    if (ch.nv <= 0) return true;
                    const uint8_t* state = static_cast<const uint8_t*>(p.s_states) + static_cast<int64_t>(entry - 1) * Cfg::SB;
                    if (g >= Cfg::NS) {
                        // into L2 while the stage is still in use
#pragma unroll
                        for (int pn = 0; pn < Cfg::NPAN; ++pn) {
                            tma_prefetch_l2_3d(&m.q, pn * 64, ch.row, ch.group);
                            tma_prefetch_l2_3d(&m.k, pn * 64, ch.row, ch.group);
                            tma_prefetch_l2_3d(&m.v, pn * 64, ch.row, ch.group);
                        }
                        if (!mbar_wait(&bar[Cfg::B_EMPTY + s], ((g / Cfg::NS) + 1) & 1, abort_flag, tmo, 0x700 + s))
                            return false;
                    }
                    mbar_arrive_expect_tx(&bar[Cfg::B_FULL + s], 3 * Cfg::TILE);
                    uint8_t* st = smem + s * Cfg::STAGE;
#pragma unroll
                    for (int pn = 0; pn < Cfg::NPAN; ++pn) {
                        tma_load_3d(st + pn * kPanel, &m.q, &bar[Cfg::B_FULL + s], pn * 64, ch.row, ch.group);
                        tma_load_3d(st + Cfg::TILE + pn * kPanel, &m.k, &bar[Cfg::B_FULL + s], pn * 64, ch.row, ch.group);
                        tma_load_3d(st + 2 * Cfg::TILE + pn * kPanel, &m.v, &bar[Cfg::B_FULL + s], pn * 64, ch.row,
                                    ch.group);
                    }
                    started = g + 1;
                    if (g >= 1 && !mbar_wait(&bar[Cfg::B_SEMPTY], (g + 1) & 1, abort_flag, tmo, 0x708)) return false;
                    mbar_arrive_expect_tx(&bar[Cfg::B_SFULL], Cfg::SB);
                    bulk_load(smem + Cfg::OFF_SB, state, Cfg::SB, &bar[Cfg::B_SFULL]);
                    loaded = g + 1;
                }
            }();
            if (!ok || *abort_flag) {
                for (int64_t g = started > Cfg::NS ? started - Cfg::NS : 0; g < started; ++g)
                    mbar_wait_drain(&bar[Cfg::B_FULL + g % Cfg::NS], (g / Cfg::NS) & 1, tmo);
                if (loaded >= 1) mbar_wait_drain(&bar[Cfg::B_SFULL], (loaded - 1) & 1, tmo);
            }
        }
    } else if (warp == 1 || warp == 3) {
        if (lane == 0) {
            constexpr uint32_t kIdA = idesc_bf16_f32(C, C, false, false);
            constexpr uint32_t kIdO = idesc_bf16_f32(C, D, false, true);
            bool issued = false;
            auto scores = [&](int64_t g) -> bool {
                const int s = static_cast<int>(g % Cfg::NS), b = static_cast<int>(g & 1);
                if (!mbar_wait(&bar[Cfg::B_FULL + s], (g / Cfg::NS) & 1, abort_flag, tmo, 0x710 + s)) return false;
                // the buffer's last P, of chunk g - 2, is used up
                if (g >= 2 && !mbar_wait(&bar[Cfg::B_PEMPTY + b], ((g >> 1) + 1) & 1, abort_flag, tmo, 0x718)) return false;
                tc_fence_after();
                const uint32_t q = sbase + s * Cfg::STAGE, k = q + Cfg::TILE;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    mma_bf16_ss(tmem + Cfg::TM_A + b * C, sdesc_sw128(tile_k(q, ks, kPanel), 16, 1024),
                                sdesc_sw128(tile_k(k, ks, kPanel), 16, 1024), kIdA, ks > 0);
                mma_commit(&bar[Cfg::B_AFULL + b]);
                issued = true;
                return true;
            };
            auto output = [&](int64_t g) -> bool {
                const int s = static_cast<int>(g % Cfg::NS), b = static_cast<int>(g & 1);
                if (g >= 1 && !mbar_wait(&bar[Cfg::B_OEMPTY], (g + 1) & 1, abort_flag, tmo, 0x720)) return false;
                if (!mbar_wait(&bar[Cfg::B_FULL + s], (g / Cfg::NS) & 1, abort_flag, tmo, 0x724)) return false;
                if (!mbar_wait(&bar[Cfg::B_SFULL], g & 1, abort_flag, tmo, 0x728)) return false;
                tc_fence_after();
                const uint32_t q = sbase + s * Cfg::STAGE, v = q + 2 * Cfg::TILE, sb = sbase + Cfg::OFF_SB;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    mma_bf16_ss(tmem + Cfg::TM_O1, sdesc_sw128(tile_k(q, ks, kPanel), 16, 1024),
                                sdesc_sw128(sb + ks * 2048, Cfg::SB_PANEL, 1024), kIdO, ks > 0);
                mma_commit(&bar[Cfg::B_SEMPTY]);
                issued = true;
                if (!mbar_wait(&bar[Cfg::B_PFULL + b], (g >> 1) & 1, abort_flag, tmo, 0x730 + b)) return false;
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < C / 16; ++ks)
                    mma_bf16_ts(tmem + Cfg::TM_O2, tmem + Cfg::TM_A + b * C + (ks >> 2) * 64 + (ks & 3) * 8,
                                sdesc_sw128(v + ks * 2048, kPanel, 1024), kIdO, ks > 0);
                mma_commit(&bar[Cfg::B_PEMPTY + b]);
                mma_commit(&bar[Cfg::B_OFULL]);
                return true;
            };
            if (warp == 3)
                walk(true, [&](const GatedChunk&, int64_t g) { return scores(g); });
            else
                walk(true, [&](const GatedChunk&, int64_t g) { return output(g); });
            if (issued) {
                mma_commit(&bar[Cfg::B_DONE + (warp == 3)]);
                mbar_wait_drain(&bar[Cfg::B_DONE + (warp == 3)], 0, tmo);
            }
        }
        __syncwarp();
    } else if (warp == 2) {
        walk(false, [&](const GatedChunk& ch, int64_t g) {
            const int s = static_cast<int>(g % Cfg::NS);
            float x[4], G[4];
            load_gates(p, ch.row0, ch.nv, x);
            scan_up(x, G);
            const float R = __shfl_sync(0xffffffffu, G[3], lane | 7);  // prefix at the end of the 32-token block
            // tiles landed: the slot's last readers are done
            if (!mbar_wait_warp(&bar[Cfg::B_FULL + s], (g / Cfg::NS) & 1, abort_flag, tmo, 0x740 + s)) return false;
            float4* o = reinterpret_cast<float4*>(smem + Cfg::OFF_G + s * Cfg::G_BYTES);
            o[lane] = make_float4(G[0], G[1], G[2], G[3]);
            if (lane < 24) o[32 + lane] = make_float4(ex2(R - G[0]), ex2(R - G[1]), ex2(R - G[2]), ex2(R - G[3]));
            if (ch.nv < C) {
                zero_rows<D>(sbase + s * Cfg::STAGE + 2 * Cfg::TILE, ch.nv);
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[Cfg::B_GFULL + s]);
            return true;
        });
    } else if (warp >= 4 && warp < 12) {
        const int sub = warp & 3, half = (warp - 4) >> 2, row = sub * 32 + lane;
        walk(false, [&](const GatedChunk&, int64_t g) {
            const int s = static_cast<int>(g % Cfg::NS), b = static_cast<int>(g & 1);
            if (!mbar_wait_warp(&bar[Cfg::B_GFULL + s], (g / Cfg::NS) & 1, abort_flag, tmo, 0x750 + s)) return false;
            if (!mbar_wait_warp(&bar[Cfg::B_AFULL + b], (g >> 1) & 1, abort_flag, tmo, 0x758 + b)) return false;
            tc_fence_after();
            const float* G = reinterpret_cast<const float*>(smem + Cfg::OFF_G + s * Cfg::G_BYTES);
            const float* F = G + C;
            // scores of this half's keys in columns 64 half ..; P goes to the first 32 of them
            const uint32_t tm = tmem + Cfg::TM_A + b * C + half * 64 + (static_cast<uint32_t>(sub * 32) << 16);
            const float Gi = G[row];
#pragma unroll 1
            for (int pc = 0; pc < 4; ++pc) {  // 16 keys; warp-uniform cases
                const int jb = 2 * half + (pc >> 1), j0 = jb * 32 + (pc & 1) * 16;
                uint32_t w[8];
                if (jb > sub) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = 0u;
                } else {
                    float a[16];
                    ld16f(tm + pc * 16, a);
                    if (jb < sub) {
                        const float f = ex2(Gi - G[jb * 32 + 31]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float4 c = reinterpret_cast<const float4*>(F + j0)[e];
                            w[2 * e] = pack_bf16x2(a[4 * e] * (f * c.x), a[4 * e + 1] * (f * c.y));
                            w[2 * e + 1] = pack_bf16x2(a[4 * e + 2] * (f * c.z), a[4 * e + 3] * (f * c.w));
                        }
                    } else {
                        const int last = lane - (pc & 1) * 16;  // keys up to the row's own
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float4 c = reinterpret_cast<const float4*>(G + j0)[e];
                            const float d[4] = {c.x, c.y, c.z, c.w};
                            float y[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) y[k] = 4 * e + k <= last ? a[4 * e + k] * ex2(Gi - d[k]) : 0.f;
                            w[2 * e] = pack_bf16x2(y[0], y[1]);
                            w[2 * e + 1] = pack_bf16x2(y[2], y[3]);
                        }
                    }
                }
                tmem_st8(tm + pc * 8, w);  // over scores that are read
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[Cfg::B_PFULL + b]);
            return true;
        });
    } else if (warp >= 12 && warp < 12 + 4 * Cfg::NPAN) {
        const int sub = warp & 3, half = (warp - 12) >> 2, row = sub * 32 + lane;
        const uint32_t lane_off = (static_cast<uint32_t>(sub * 32) << 16) + half * 64;
        walk(false, [&](const GatedChunk& ch, int64_t g) {
            const int s = static_cast<int>(g % Cfg::NS);
            if (!mbar_wait_warp(&bar[Cfg::B_GFULL + s], (g / Cfg::NS) & 1, abort_flag, tmo, 0x760 + s)) return false;
            const float f = ex2(reinterpret_cast<const float*>(smem + Cfg::OFF_G + s * Cfg::G_BYTES)[row]);
            if (!mbar_wait_warp(&bar[Cfg::B_OFULL], g & 1, abort_flag, tmo, 0x768)) return false;
            tc_fence_after();
            const uint32_t panel = sbase + s * Cfg::STAGE + half * kPanel;  // Q, read by both of its products
            uint16_t* out = static_cast<uint16_t*>(p.o) + (ch.row0 + row) * D + half * 64;
#pragma unroll 1
            for (int h = 0; h < 4; ++h) {
                float x[16], y[16];
                ld16f2(tmem + Cfg::TM_O1 + lane_off + h * 16, tmem + Cfg::TM_O2 + lane_off + h * 16, x, y);
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] = fmaf(f, x[e], y[e]);
                if (ch.nv == C)
                    put_row16(panel, row, 2 * h, x);
                else if (row < ch.nv)
                    put_row16(out + h * 16, x);
            }
            tc_fence_before();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bar[Cfg::B_OEMPTY]);
                if (ch.nv == C) {
                    tma_store_3d(&m.o, smem + s * Cfg::STAGE + half * kPanel + sub * 32 * 128, half * 64,
                                 ch.row + sub * 32, ch.group);
                    bulk_commit_group();
                    bulk_wait_group_read<0>();
                }
                mbar_arrive(&bar[Cfg::B_EMPTY + s]);
            }
            return true;
        });
        if (lane == 0) bulk_wait_group<0>();
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
}

// Shared memory of a kernel, 1 KB aligned, and all of its tensor memory.
__device__ __forceinline__ uint8_t* aligned_smem(uint8_t* raw) {
    return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
}
__device__ __forceinline__ uint32_t take_tmem(uint8_t* smem) {
    uint32_t* slot = reinterpret_cast<uint32_t*>(smem);
    if (threadIdx.x < 32) {
        tmem_alloc(slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *slot;
    __syncthreads();
    return tmem;
}
__device__ __forceinline__ void give_tmem(uint32_t tmem) {
    if (threadIdx.x < 32) tmem_dealloc(tmem, 512);
}

// The states of the gradient, both directions; the sums of segments.
template <int D, bool ALONE>
__global__ void __launch_bounds__(640, 1)
    gated_states_tc_kernel(const __grid_constant__ GatedMaps m, const GatedProblem p, int64_t n_items, bool grad) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = aligned_smem(smem_raw);
    const uint32_t tmem = take_tmem(smem);
    gated_states_body<D, ALONE>(m, p, n_items, grad, smem, tmem, blockIdx.x, gridDim.x);
    give_tmem(tmem);
}

// Whether any CTA has claimed a unit of the prefill yet; waits for it, but not longer than it takes the first CTAs of a
// launch to begin.  Every thread gets the same answer.
constexpr uint64_t kBeginNs = 20000;
__device__ __forceinline__ bool walk_begun(const GatedProblem& p) {
    int begun = 0;
    if (threadIdx.x == 0) {
        const uint64_t t0 = globaltimer_ns();
        do {
            unsigned int claims;
            asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(claims) : "l"(p.queue + 3) : "memory");
            begun = claims != 0;
        } while (!begun && globaltimer_ns() - t0 < kBeginNs);
    }
    return __syncthreads_or(begun) != 0;
}

// The prefill in one launch: the first n_state CTAs make the states and publish each chunk as its state is stored; the
// others, and those when they are done, take the chunks in that order.  So K, V and the states come from L2 the second
// time, and the serial phase of few long sequences overlaps the other.
// A CTA takes chunks, and so may wait for them, only after it has seen a unit claimed: whoever claimed it is running, waits
// for nobody and claims on until no unit is left.  A CTA that sees none claimed makes states itself.  So it matters neither
// how many of the CTAs are on the device at once nor in which order they start.  (Roles by order of arrival at a counter
// instead of by index: 445 us, not 362, at B8 H16 T8192, since the first to arrive sit close together.)
template <int D>
__global__ void __launch_bounds__(640, 1)
    gated_prefill_tc_kernel(const __grid_constant__ GatedMaps m, const GatedProblem p, int64_t n_items, int n_state) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = aligned_smem(smem_raw);
    const uint32_t tmem = take_tmem(smem);
    if (static_cast<int>(blockIdx.x) < n_state || !walk_begun(p))
        gated_states_body<D, false>(m, p, n_items, false, smem, tmem, blockIdx.x, n_state);
    gated_out_body<D>(m, p, smem, tmem);
    give_tmem(tmem);
}

// ---------------------------------------------------------------------------
// Gradient of the chunks.  With j the lane (row) of an accumulator, per chunk
//     T0 = K Q^T, T1 = V dO^T            -> P^T, W^T (decayed, i >= j; bf16 over T0)
//     T2 = e^{G_i} (dO S^T) + W K        -> dq
//     T3 = e^{G_C - G_j} (V E^T) + W^T Q -> dk
//     T1 = e^{G_C - G_j} (K E) + P^T dO  -> dv
// Each decayed part is scaled in tensor memory before its second product is
// accumulated onto it.  dg comes from the results, before they are rounded:
// with cj = e^{G_C - G_j} k_j . (E v_j), taken when T3 is scaled,
//     dg_t = e^{G_C} <E, S> + sum_{i >= t} (q_i . dq_i - k_i . dk_i + cj_i) + sum_{j < t} cj_j.
// The pairs on one side of gate t are in both sums and cancel: dq and dk are
// sums of the same rounded W_ij, so they do to fp32 of their size, over the 128
// tokens of a chunk at most.  That is dg's error where a gate lets little
// through; behind one that lets nothing through dg is set to zero.
//   warp 0       producer            warp 1  MMA issuer
//   warp 2       decays; zeroes the rows behind a sequence's end; stores dv
//   warp 3       dg; stores dq and dk
//   warps 4-19   everything else: four warps share 32 rows, 32 columns each (at
//                D = 64 two of them work on the D-wide tiles)
// Tiles are loaded once each (one stage at D = 128: 192 KB), reloaded for the
// next chunk as each dies; W^T lies over V, and dq, dk, dv are staged for their
// stores in the tiles of q, k and dO.
// ---------------------------------------------------------------------------
template <int D>
struct GrCfg {
    static constexpr int kThreads = 640;
    static constexpr int NPAN = D / 64;
    static constexpr int TILE = C * D * 2;
    static constexpr int SB = D * D * 2, SB_PANEL = D * 128;
    static constexpr int NS = D == 128 ? 1 : 2;
    static constexpr int STAGE = 4 * TILE + 2 * SB;
    // tiles of a stage
    static constexpr int Q = 0, K = TILE, V = 2 * TILE, O = 3 * TILE, S = 4 * TILE, E = 4 * TILE + SB;
    static constexpr int W_BYTES = C * C * 2;
    // W^T: over V at D = 128 (V is dead by then), a tile of its own at D = 64
    static constexpr int OFF_W = D == 128 ? V : NS * STAGE;
    static constexpr int OFF_G = NS * STAGE + (D == 128 ? 0 : W_BYTES);
    // [2][4][128]: prefix sums; e^{G_i}; e^{G_C - G_j}; e^{G_i - R}, R the prefix before i's block
    static constexpr int NQ = D / 32;                       // warps with columns of the D-wide tiles, per 32 rows
    static constexpr int OFF_U = OFF_G + 2 * 4 * C * 4;  // q_i . dq_i - k_i . dk_i by 32 columns [NQ][128]
    static constexpr int OFF_CJ = OFF_U + NQ * C * 4;    // e^{G_C - G_j} k_j . E v_j by 32 columns [NQ][128]
    static constexpr int OFF_ES = OFF_CJ + NQ * C * 4;   // e^{G_C} <E, S> by warp [16]
    static constexpr int OFF_BAR = OFF_ES + 64;
    // per stage: loads and releases of Q, K, V, dO, S, E
    static constexpr int F_Q = 0, F_K = 1, F_V = 2, F_O = 3, F_S = 4, F_E = 5;
    static constexpr int B_FULL = 0, B_EMPTY = 6 * NS, B_GFULL = 12 * NS, B_ABFULL = 12 * NS + NS, B_Y = B_ABFULL + 2, B_Z = B_ABFULL + 3, B_P = B_ABFULL + 4, B_XYS = B_ABFULL + 5,
                         B_ZS = B_ABFULL + 6, B_DK = B_ABFULL + 8, B_DV = B_ABFULL + 9,
                         B_FREE = B_ABFULL + 10 /* T2, T3, T1 read out */, B_SUMS = B_ABFULL + 13,
                         B_SUMFREE = B_ABFULL + 14, B_DONE = B_ABFULL + 15, B_READ = B_ABFULL + 16,
                         B_STAGED = B_ABFULL + 17 /* dq, dk, dv */, NBAR = B_ABFULL + 20;
    static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
    static constexpr int SMEM = OFF_MISC + 16 + 1024;
    static constexpr int T0 = 0, T1 = 128, T2 = 256, T3 = 384;
    static_assert(SMEM <= 232448, "shared memory");
};

// x . (the row's 16 bf16 values in two 16-byte pieces of a swizzled panel row).
__device__ __forceinline__ float row_dot16(const float (&x)[16], uint32_t panel, int row, int chunk0) {
    float2 d[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
    for (int ch = 0; ch < 2; ++ch) {
        uint32_t a[4];
        ld_shared_v4(panel + sw128_off(row, chunk0 + ch), a[0], a[1], a[2], a[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            d[e & 1] = __ffma2_rn(make_float2(x[8 * ch + 2 * e], x[8 * ch + 2 * e + 1]),
                                  make_float2(bf16_lo(a[e]), bf16_hi(a[e])), d[e & 1]);
    }
    return (d[0].x + d[0].y) + (d[1].x + d[1].y);
}

// x *= f, and back to tensor memory.
__device__ __forceinline__ void scale16(uint32_t taddr, float f, float (&x)[16]) {
    uint32_t w[16];
    const float2 ff = make_float2(f, f);
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        const float2 y = __fmul2_rn(make_float2(x[i], x[i + 1]), ff);
        x[i] = y.x;
        x[i + 1] = y.y;
        w[i] = __float_as_uint(y.x);
        w[i + 1] = __float_as_uint(y.y);
    }
    tmem_st16(taddr, w);
}

// Start the TMA store of a staged [128][D] tile (one thread; its own bulk group).
template <int D>
__device__ __forceinline__ void store_tile(const CUtensorMap* map, const uint8_t* tile, const GatedChunk& ch) {
#pragma unroll
    for (int pn = 0; pn < D / 64; ++pn) tma_store_3d(map, tile + pn * kPanel, pn * 64, ch.row, ch.group);
    bulk_commit_group();
}

template <int D>
__global__ void __launch_bounds__(640, 1)
    gated_grad_tc_kernel(const __grid_constant__ GatedMaps m, const GatedProblem p, int64_t n_slots) {
    using Cfg = GrCfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + Cfg::OFF_BAR);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::OFF_MISC + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint64_t tmo = p.timeout_ns;
    const uint32_t sbase = smem_u32(smem);
    if (threadIdx.x == 0) {
        for (int s = 0; s < Cfg::NS; ++s) {
            for (int t = 0; t < 6; ++t) {
                mbar_init(&bar[Cfg::B_FULL + 6 * s + t], 1);
                // S and E are read by the products and by every warp
                mbar_init(&bar[Cfg::B_EMPTY + 6 * s + t], t == Cfg::F_S || t == Cfg::F_E ? 17 : 1);
            }
            mbar_init(&bar[Cfg::B_GFULL + s], 1);
        }
        for (int b : {Cfg::B_ABFULL, Cfg::B_Y, Cfg::B_Z, Cfg::B_DK, Cfg::B_DV, Cfg::B_SUMFREE,
                      Cfg::B_DONE})
            mbar_init(&bar[b], 1);
        for (int b : {Cfg::B_P, Cfg::B_XYS, Cfg::B_ZS, Cfg::B_FREE, Cfg::B_FREE + 1, Cfg::B_FREE + 2, Cfg::B_SUMS, Cfg::B_READ})
            mbar_init(&bar[b], 16);
        for (int b = 0; b < 3; ++b) mbar_init(&bar[Cfg::B_STAGED + b], 4 * Cfg::NQ);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    auto walk = [&](auto&& f) -> bool {
        int64_t g = 0;
        for (int64_t i = blockIdx.x; i < n_slots; i += gridDim.x) {
            const GatedChunk ch = gated_chunk(p, i, C);
            if (ch.nv <= 0) continue;
            if (!f(ch, i, g)) return false;
            ++g;
        }
        return true;
    };
    auto full = [&](int s, int t) { return &bar[Cfg::B_FULL + 6 * s + t]; };
    auto empty = [&](int s, int t) { return &bar[Cfg::B_EMPTY + 6 * s + t]; };

    if (warp == 0) {
        if (lane == 0) {
            int64_t started[6] = {0, 0, 0, 0, 0, 0};
            const bool ok = walk([&](const GatedChunk& ch, int64_t slot, int64_t g) {
                const int s = static_cast<int>(g % Cfg::NS);
                uint8_t* st = smem + s * Cfg::STAGE;
                // in the order in which the tiles of the chunk before die
                constexpr int order[6] = {Cfg::F_V, Cfg::F_S, Cfg::F_E, Cfg::F_Q, Cfg::F_K, Cfg::F_O};
#pragma unroll
                for (int k = 0; k < 6; ++k) {
                    const int t = order[k];
                    if (g >= Cfg::NS && !mbar_wait(empty(s, t), ((g / Cfg::NS) + 1) & 1, abort_flag, tmo, 0x800 + t))
                        return false;
                    if (t == Cfg::F_S || t == Cfg::F_E) {
                        mbar_arrive_expect_tx(full(s, t), Cfg::SB);
                        bulk_load(st + (t == Cfg::F_S ? Cfg::S : Cfg::E),
                                  static_cast<const uint8_t*>(t == Cfg::F_S ? p.s_states : p.e_states) + slot * Cfg::SB,
                                  Cfg::SB, full(s, t));
                    } else {
                        const CUtensorMap* map =
                            t == Cfg::F_Q ? &m.q : (t == Cfg::F_K ? &m.k : (t == Cfg::F_V ? &m.v : &m.d_o));
                        mbar_arrive_expect_tx(full(s, t), Cfg::TILE);
#pragma unroll
                        for (int pn = 0; pn < Cfg::NPAN; ++pn)
                            tma_load_3d(st + t * Cfg::TILE + pn * kPanel, map, full(s, t), pn * 64, ch.row, ch.group);
                    }
                    started[t] = g + 1;
                }
                // the next chunk's tiles into L2 while this one is computed
                const int64_t next = slot + gridDim.x;
                if (next < n_slots) {
                    const GatedChunk c2 = gated_chunk(p, next, C);
                    if (c2.nv > 0) {
#pragma unroll
                        for (int pn = 0; pn < Cfg::NPAN; ++pn) {
                            tma_prefetch_l2_3d(&m.q, pn * 64, c2.row, c2.group);
                            tma_prefetch_l2_3d(&m.k, pn * 64, c2.row, c2.group);
                            tma_prefetch_l2_3d(&m.v, pn * 64, c2.row, c2.group);
                            tma_prefetch_l2_3d(&m.d_o, pn * 64, c2.row, c2.group);
                        }
                        bulk_prefetch_l2(static_cast<const uint8_t*>(p.s_states) + next * Cfg::SB, Cfg::SB);
                        bulk_prefetch_l2(static_cast<const uint8_t*>(p.e_states) + next * Cfg::SB, Cfg::SB);
                    }
                }
                return true;
            });
            if (!ok || *abort_flag)
                for (int t = 0; t < 6; ++t)
                    for (int64_t g = started[t] > Cfg::NS ? started[t] - Cfg::NS : 0; g < started[t]; ++g)
                        mbar_wait_drain(full(static_cast<int>(g % Cfg::NS), t), (g / Cfg::NS) & 1, tmo);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t kIdT = idesc_bf16_f32(C, C, false, false);   // scores: both operands K-major
            constexpr uint32_t kIdS = idesc_bf16_f32(C, D, false, false);   // .. S^T, .. E^T
            constexpr uint32_t kIdB = idesc_bf16_f32(C, D, false, true);    // .. E, P^T dO, W^T Q
            constexpr uint32_t kIdW = idesc_bf16_f32(C, D, true, true);     // W K, W held transposed
            bool issued = false;
            auto wait = [&](int b, int64_t phase, unsigned where) {
                return mbar_wait(&bar[b], static_cast<uint32_t>(phase & 1), abort_flag, tmo, where);
            };
            walk([&](const GatedChunk& ch, int64_t, int64_t g) {
                const int s = static_cast<int>(g % Cfg::NS);
                const int64_t k = g / Cfg::NS;
                const uint32_t st = sbase + s * Cfg::STAGE;
                const uint32_t q = st + Cfg::Q, kk = st + Cfg::K, v = st + Cfg::V, o = st + Cfg::O, sb = st + Cfg::S,
                               eb = st + Cfg::E, wt = sbase + Cfg::OFF_W;
                auto loaded = [&](int t) { return wait(Cfg::B_FULL + 6 * s + t, k, 0x810 + t); };
                // T0, T1: scores (T0 and T1 of the chunk before are consumed and read)
                if (!loaded(Cfg::F_Q) || !loaded(Cfg::F_K)) return false;
                // the scores of a part-filled chunk need its zeroed rows
                if (ch.nv < C && !wait(Cfg::B_GFULL + s, k, 0x817)) return false;
                if (g >= 1 && (!wait(Cfg::B_DV, g - 1, 0x818) || !wait(Cfg::B_FREE + 2, g - 1, 0x819))) return false;
                tc_fence_after();
                issued = true;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    mma_bf16_ss(tmem + Cfg::T0, sdesc_sw128(tile_k(kk, ks, kPanel), 16, 1024),
                                sdesc_sw128(tile_k(q, ks, kPanel), 16, 1024), kIdT, ks > 0);
                if (!loaded(Cfg::F_V) || !loaded(Cfg::F_O)) return false;
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    mma_bf16_ss(tmem + Cfg::T1, sdesc_sw128(tile_k(v, ks, kPanel), 16, 1024),
                                sdesc_sw128(tile_k(o, ks, kPanel), 16, 1024), kIdT, ks > 0);
                mma_commit(&bar[Cfg::B_ABFULL]);
                // T2 = dO S^T
                if (!loaded(Cfg::F_S)) return false;
                if (g >= 1 && !wait(Cfg::B_FREE + 0, g - 1, 0x81a)) return false;
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    mma_bf16_ss(tmem + Cfg::T2, sdesc_sw128(tile_k(o, ks, kPanel), 16, 1024),
                                sdesc_sw128(tile_k(sb, ks, Cfg::SB_PANEL), 16, 1024), kIdS, ks > 0);
                mma_commit(empty(s, Cfg::F_S));
                // T3 = V E^T
                if (!loaded(Cfg::F_E)) return false;
                if (g >= 1 && !wait(Cfg::B_FREE + 1, g - 1, 0x81b)) return false;
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    mma_bf16_ss(tmem + Cfg::T3, sdesc_sw128(tile_k(v, ks, kPanel), 16, 1024),
                                sdesc_sw128(tile_k(eb, ks, Cfg::SB_PANEL), 16, 1024), kIdS, ks > 0);
                mma_commit(&bar[Cfg::B_Y]);
                if (D == 64) mma_commit(empty(s, Cfg::F_V));
                // T1 = K E once the scores there are read
                if (!wait(Cfg::B_P, g, 0x81c)) return false;
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    mma_bf16_ss(tmem + Cfg::T1, sdesc_sw128(tile_k(kk, ks, kPanel), 16, 1024),
                                sdesc_sw128(eb + ks * 2048, Cfg::SB_PANEL, 1024), kIdB, ks > 0);
                mma_commit(&bar[Cfg::B_Z]);
                mma_commit(empty(s, Cfg::F_E));
                // onto the scaled parts
                if (!wait(Cfg::B_XYS, g, 0x81d)) return false;
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < C / 16; ++ks)
                    mma_bf16_ss(tmem + Cfg::T2, sdesc_sw128(wt + ks * 2048, kPanel, 1024),
                                sdesc_sw128(kk + ks * 2048, kPanel, 1024), kIdW, 1);
                if (D == 128) mma_commit(empty(s, Cfg::F_V));
#pragma unroll
                for (int ks = 0; ks < C / 16; ++ks)
                    mma_bf16_ts(tmem + Cfg::T3, tmem + Cfg::T0 + 64 + ks * 8,
                                sdesc_sw128(q + ks * 2048, kPanel, 1024), kIdB, 1);
                mma_commit(&bar[Cfg::B_DK]);
                if (!wait(Cfg::B_ZS, g, 0x81e)) return false;
                tc_fence_after();
#pragma unroll
                for (int ks = 0; ks < C / 16; ++ks)
                    mma_bf16_ts(tmem + Cfg::T1, tmem + Cfg::T0 + ks * 8, sdesc_sw128(o + ks * 2048, kPanel, 1024),
                                kIdB, 1);
                mma_commit(&bar[Cfg::B_DV]);
                return true;
            });
            if (issued) {
                mma_commit(&bar[Cfg::B_DONE]);
                mbar_wait_drain(&bar[Cfg::B_DONE], 0, tmo);
            }
        }
        __syncwarp();
    } else if (warp == 2) {
        walk([&](const GatedChunk& ch, int64_t, int64_t g) {
            const int s = static_cast<int>(g % Cfg::NS);
            const uint32_t ph = (g / Cfg::NS) & 1;
            float x[4], G[4], B[4], all;
            load_gates(p, ch.row0, ch.nv, x);
            scan_up(x, G);
            scan_down(x, B, all);
            float R = __shfl_sync(0xffffffffu, G[3], ((lane >> 3) * 8 + 31) & 31);  // prefix before the block
            if (lane < 8) R = 0.f;
            // (S: its tile was given back behind the last use of these decays' place.  V is waited for only where its
            // rows are zeroed: a full chunk's V may be given back, and loaded again, before this warp looks at it)
            for (int t : {Cfg::F_Q, Cfg::F_K, Cfg::F_O, Cfg::F_S, Cfg::F_V})
                if ((t != Cfg::F_V || ch.nv < C) && !mbar_wait_warp(full(s, t), ph, abort_flag, tmo, 0x820 + t)) return false;
            float4* o = reinterpret_cast<float4*>(smem + Cfg::OFF_G + (g & 1) * 4 * C * 4);
            o[lane] = make_float4(G[0], G[1], G[2], G[3]);
            o[32 + lane] = make_float4(ex2(G[0]), ex2(G[1]), ex2(G[2]), ex2(G[3]));
            o[64 + lane] = make_float4(ex2(B[0]), ex2(B[1]), ex2(B[2]), ex2(B[3]));
            o[96 + lane] = make_float4(ex2(G[0] - R), ex2(G[1] - R), ex2(G[2] - R), ex2(G[3] - R));
            if (ch.nv < C) {
                for (int t : {Cfg::F_Q, Cfg::F_K, Cfg::F_V, Cfg::F_O})
                    zero_rows<D>(sbase + s * Cfg::STAGE + t * Cfg::TILE, ch.nv);
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[Cfg::B_GFULL + s]);
            // dv, the last result of the chunk
            if (!mbar_wait_warp(&bar[Cfg::B_STAGED + 2], static_cast<uint32_t>(g & 1), abort_flag, tmo, 0x834)) return false;
            if (lane == 0) {
                if (ch.nv == C) {
                    store_tile<D>(&m.dv, smem + s * Cfg::STAGE + Cfg::O, ch);
                    bulk_wait_group_read<0>();
                }
                mbar_arrive(empty(s, Cfg::F_O));
            }
            __syncwarp();
            return true;
        });
        if (lane == 0) bulk_wait_group<0>();
    } else if (warp == 3) {
        walk([&](const GatedChunk& ch, int64_t, int64_t g) {
            const int s = static_cast<int>(g % Cfg::NS);
            const uint32_t gp = static_cast<uint32_t>(g & 1);
            // a gate at the floor, or one that no path of the chunk crosses with a weight of 2^-126, even with all of its
            // positive gates
            bool closed[4];
            {
                float x[4], up = 0.f;
                load_gates(p, ch.row0, ch.nv, x);
#pragma unroll
                for (int e = 0; e < 4; ++e) up += fmaxf(x[e], 0.f);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) up += __shfl_xor_sync(0xffffffffu, up, o);
#pragma unroll
                for (int e = 0; e < 4; ++e) closed[e] = x[e] <= kGateFloor * kLog2e || x[e] + up < -126.f;
            }
            auto store = [&](int n, int tile, const CUtensorMap* map) {
                if (!mbar_wait_warp(&bar[Cfg::B_STAGED + n], gp, abort_flag, tmo, 0x832 + n)) return false;
                if (lane == 0 && ch.nv == C) store_tile<D>(map, smem + s * Cfg::STAGE + tile * Cfg::TILE, ch);
                return true;
            };
            // what lies in dq's first row is read (every warp gives S back behind that)
            if (ch.alone && !mbar_wait_warp(empty(s, Cfg::F_S), (g / Cfg::NS) & 1, abort_flag, tmo, 0x835)) return false;
            if (!store(0, Cfg::F_Q, &m.dq) || !store(1, Cfg::F_K, &m.dk)) return false;
            if (lane == 0) {  // hand each tile back as soon as its store has read it
                if (ch.nv == C) bulk_wait_group_read<1>();
                mbar_arrive(empty(s, Cfg::F_Q));
                bulk_wait_group_read<0>();
                mbar_arrive(empty(s, Cfg::F_K));
            }
            __syncwarp();
            if (!mbar_wait_warp(&bar[Cfg::B_SUMS], gp, abort_flag, tmo, 0x830)) return false;
            const float* es = reinterpret_cast<const float*>(smem + Cfg::OFF_ES);
            auto get = [&](int off, float (&x)[4]) {
                const float4* a = reinterpret_cast<const float4*>(smem + off);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = 0.f;
#pragma unroll
                for (int k = 0; k < Cfg::NQ; ++k) {
                    const float4 f = a[32 * k + lane];
                    x[0] += f.x;
                    x[1] += f.y;
                    x[2] += f.z;
                    x[3] += f.w;
                }
            };
            float u[4], d[4], e0 = 0.f;
            get(Cfg::OFF_U, u);
            get(Cfg::OFF_CJ, d);
#pragma unroll
            for (int k = 0; k < 16; ++k) e0 += es[k];
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[Cfg::B_SUMFREE]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (4 * lane + e >= ch.nv) u[e] = d[e] = 0.f;
                u[e] += d[e];
            }
            float after[4], all, upto[4];
            scan_down(u, after, all);  // over i > t
            scan_up(d, upto);          // over j <= t
            if (p.dg != nullptr) {
                __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.dg) + ch.row0 + 4 * lane;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (4 * lane + e < ch.nv)
                        out[e] = __float2bfloat16_rn(closed[e] ? 0.f : e0 + after[e] + u[e] + (upto[e] - d[e]));
            }
            return true;
        });
        if (lane == 0) bulk_wait_group<0>();
    } else {
        const int sub = warp & 3, quarter = (warp - 4) >> 2, row = sub * 32 + lane;
        const bool wide = quarter < Cfg::NQ;  // has columns of the D-wide tiles
        const uint32_t lanes = static_cast<uint32_t>(sub * 32) << 16;
        const uint32_t dcol = lanes + quarter * 32;
        const int pan = quarter >> 1, ch0 = 4 * (quarter & 1);  // panel and first 16-byte piece of these columns
        float* us = reinterpret_cast<float*>(smem + Cfg::OFF_U);
        float* cj = reinterpret_cast<float*>(smem + Cfg::OFF_CJ);
        float* es = reinterpret_cast<float*>(smem + Cfg::OFF_ES);
        walk([&](const GatedChunk& ch, int64_t, int64_t g) {
            const int s = static_cast<int>(g % Cfg::NS);
            const uint32_t ph = (g / Cfg::NS) & 1, gp = static_cast<uint32_t>(g & 1);
            const uint32_t st = sbase + s * Cfg::STAGE;
            auto wait = [&](int b, uint32_t parity, unsigned where) {
                return mbar_wait_warp(&bar[b], parity, abort_flag, tmo, where);
            };
            auto arrive = [&](int b) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[b]);
            };
            if (!wait(Cfg::B_GFULL + s, ph, 0x840)) return false;
            const float* G = reinterpret_cast<const float*>(smem + Cfg::OFF_G + gp * 4 * C * 4);
            const float *Pre = G + C, *Suf = G + 2 * C, *F = G + 3 * C;
            for (int t : {Cfg::F_Q, Cfg::F_K, Cfg::F_S, Cfg::F_E})  // read here too
                if (!wait(Cfg::B_FULL + 6 * s + t, ph, 0x842)) return false;
            // decayed scores of key row j = row, readers i in block ib; warp-uniform cases
            if (!wait(Cfg::B_ABFULL, gp, 0x844)) return false;
            tc_fence_after();
            const int ib = quarter;
            uint32_t pw[16], ww[16];
            if (ib < sub) {
#pragma unroll
                for (int e = 0; e < 16; ++e) pw[e] = ww[e] = 0u;
            } else {
                const float Gj = G[row], fj = ib > sub ? ex2(G[ib * 32 - 1] - Gj) : 0.f;
                const uint32_t ta = tmem + Cfg::T0 + lanes + ib * 32, tb = tmem + Cfg::T1 + lanes + ib * 32;
#pragma unroll
                for (int hb = 0; hb < 2; ++hb) {
                    float a[16], b[16];
                    ld16f2(ta + hb * 16, tb + hb * 16, a, b);
                    if (ib > sub) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float4 f = reinterpret_cast<const float4*>(F + ib * 32 + hb * 16)[e];
                            const float w[4] = {fj * f.x, fj * f.y, fj * f.z, fj * f.w};
#pragma unroll
                            for (int h = 0; h < 4; ++h) {
                                a[4 * e + h] *= w[h];
                                b[4 * e + h] *= w[h];
                            }
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            const float w = ex2(G[ib * 32 + hb * 16 + c] - Gj);
                            const bool in = hb * 16 + c >= lane;
                            a[c] = in ? w * a[c] : 0.f;
                            b[c] = in ? w * b[c] : 0.f;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        pw[8 * hb + e] = pack_bf16x2(a[2 * e], a[2 * e + 1]);
                        ww[8 * hb + e] = pack_bf16x2(b[2 * e], b[2 * e + 1]);
                    }
                }
            }
            // every thread has read T0 and T1, and the products with V are done: the results take their place
            tc_fence_before();
            arrive(Cfg::B_READ);
            if (!wait(Cfg::B_Y, gp, 0x846) || !wait(Cfg::B_READ, gp, 0x848)) return false;
            tc_fence_after();
            tmem_st16(tmem + Cfg::T0 + lanes + ib * 16, pw);
            tmem_st16(tmem + Cfg::T0 + lanes + 64 + ib * 16, ww);
            {
                const uint32_t panel = sbase + Cfg::OFF_W + (ib >> 1) * kPanel;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    st_shared_v4(panel + sw128_off(row, 4 * (ib & 1) + c), ww[4 * c], ww[4 * c + 1], ww[4 * c + 2],
                                 ww[4 * c + 3]);
            }
            tmem_wait_st();
            tc_fence_before();
            fence_proxy_async_smem();
            arrive(Cfg::B_P);
            // scale the parts through the states (T2 before T3 was committed)
            tc_fence_after();
            // the sums of the chunk before are read
            if (g >= 1 && !wait(Cfg::B_SUMFREE, gp ^ 1u, 0x841)) return false;
            if (wide) {
                float dot = 0.f;
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    float x[16], y[16];
                    ld16f2(tmem + Cfg::T2 + dcol + h * 16, tmem + Cfg::T3 + dcol + h * 16, x, y);
                    scale16(tmem + Cfg::T2 + dcol + h * 16, Pre[row], x);
                    scale16(tmem + Cfg::T3 + dcol + h * 16, Suf[row], y);
                    dot += row_dot16(y, st + Cfg::K + pan * kPanel, row, ch0 + 2 * h);
                }
                cj[quarter * C + row] = dot;
            }
            tmem_wait_st();
            tc_fence_before();
            arrive(Cfg::B_XYS);
            if (!wait(Cfg::B_Z, gp, 0x847)) return false;
            tc_fence_after();
            if (wide) {
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    float x[16];
                    ld16f(tmem + Cfg::T1 + dcol + h * 16, x);
                    scale16(tmem + Cfg::T1 + dcol + h * 16, Suf[row], x);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            arrive(Cfg::B_ZS);
            // e^{G_C} <E, S>, a share of the elements per thread; half of the decay on either side: behind a memory that grew,
            // ahead of one that will, E S alone may leave fp32
            {
                float2 sum = make_float2(0.f, 0.f);
                const float half = Pre[C - 1] == 0.f ? 0.f : ex2(0.5f * G[C - 1]);
                const float2 hh = make_float2(half, half);
#pragma unroll 2
                for (int i = (threadIdx.x - 128) * 16; i < Cfg::SB && !ch.alone; i += 512 * 16) {
                    uint32_t a[4], b[4];
                    ld_shared_v4(st + Cfg::S + i, a[0], a[1], a[2], a[3]);
                    ld_shared_v4(st + Cfg::E + i, b[0], b[1], b[2], b[3]);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sum = __ffma2_rn(__fmul2_rn(hh, make_float2(bf16_lo(a[e]), bf16_hi(a[e]))),
                                         __fmul2_rn(hh, make_float2(bf16_lo(b[e]), bf16_hi(b[e]))), sum);
                }
                float acc = sum.x + sum.y;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
                if (lane == 0) {
                    if (ch.alone) acc = warp < 4 + 4 * Cfg::NPAN ? alone_sums<D>(p, ch.row0)[warp - 4] : 0.f;
                    es[warp - 4] = acc;
                    mbar_arrive(empty(s, Cfg::F_S));
                    mbar_arrive(empty(s, Cfg::F_E));
                }
            }
            // results: into the tile of q, k or dO, whose last reader is done; returns the dot product with what it held
            auto result = [&](int tm, int n, int tile, void* dst, bool dot) -> float {
                float sum = 0.f;
                if (wide) {
                    const uint32_t panel = st + tile * Cfg::TILE + pan * kPanel;
                    uint16_t* out = static_cast<uint16_t*>(dst) + (ch.row0 + row) * D + quarter * 32;
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {
                        float x[16];
                        ld16f(tmem + tm + dcol + h * 16, x);
                        if (dot) sum += row_dot16(x, panel, row, ch0 + 2 * h);
                        if (ch.nv == C)
                            put_row16(panel, row, ch0 + 2 * h, x);
                        else if (row < ch.nv)
                            put_row16(out + h * 16, x);
                    }
                    fence_proxy_async_smem();
                }
                tc_fence_before();
                arrive(Cfg::B_FREE + n);
                if (wide && lane == 0) mbar_arrive(&bar[Cfg::B_STAGED + n]);
                return sum;
            };
            if (!wait(Cfg::B_DK, gp, 0x850)) return false;
            // before any row is written: what lies in dq's first one is read
            if (ch.alone && !wait(Cfg::B_EMPTY + 6 * s + Cfg::F_S, ph, 0x852)) return false;
            tc_fence_after();
            float u = 0.f;
#pragma unroll 1
            for (int n = 0; n < 2; ++n)
                u += n == 0 ? result(Cfg::T2, 0, Cfg::F_Q, p.dq, true) : -result(Cfg::T3, 1, Cfg::F_K, p.dk_, true);
            if (wide) us[quarter * C + row] = u;
            arrive(Cfg::B_SUMS);
            if (!wait(Cfg::B_DV, gp, 0x851)) return false;
            tc_fence_after();
            result(Cfg::T1, 2, Cfg::F_O, p.dv_, false);
            return true;
        });
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <typename F>
cudaError_t raise_smem(PerDeviceOnce& once, F kern, int bytes) {
    return once.run([&] { return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes); });
}
unsigned grid_for(int64_t items, int num_sms) { return static_cast<unsigned>(items < num_sms ? items : num_sms); }

template <int D, bool ALONE>
cudaError_t states_d(const GatedProblem& p, const GatedMaps& m, bool grad, int num_sms, cudaStream_t s) {
    static PerDeviceOnce once;
    cudaError_t e = raise_smem(once, gated_states_tc_kernel<D, ALONE>, StCfg<D>::SMEM);
    if (e != cudaSuccess) return e;
    const int64_t items = p.n_units * p.segs * (grad ? 2 : 1);
    gated_states_tc_kernel<D, ALONE><<<grid_for(items, num_sms), StCfg<D>::kThreads, StCfg<D>::SMEM, s>>>(m, p, items, grad);
    return cudaGetLastError();
}
template <int D>
cudaError_t prefill_d(const GatedProblem& p, const GatedMaps& m, int num_sms, cudaStream_t s) {
    constexpr int kSmem = StCfg<D>::SMEM > OutCfg<D>::SMEM ? StCfg<D>::SMEM : OutCfg<D>::SMEM;
    static PerDeviceOnce once;
    cudaError_t e = raise_smem(once, gated_prefill_tc_kernel<D>, kSmem);
    if (e != cudaSuccess) return e;
    // As many CTAs as make the states in the fewest rounds on three quarters of the device.  Measured at 30, 45, 60, 75,
    // 90 and 100 %: B8 H16 T8192 466 369 369 369 382 382 us, B16 H32 T256 137 102 86 80 82 81, B4 H32 T512 59 46 46 46 43
    // 43, 24 packed sequences 288 233 239 225 231 209 (all d 128).
    const int most = std::max(1, num_sms * 75 / 100);
    const int64_t items = p.n_units * p.segs, rounds = (items + most - 1) / most;
    const int n_state = static_cast<int>((items + rounds - 1) / rounds);
    const int64_t slots = p.groups * p.nc;
    const dim3 grid(static_cast<unsigned>(std::min<int64_t>(num_sms, n_state + slots)));
    gated_prefill_tc_kernel<D><<<grid, OutCfg<D>::kThreads, kSmem, s>>>(m, p, items, n_state);
    return cudaGetLastError();
}
template <int D>
cudaError_t grad_d(const GatedProblem& p, const GatedMaps& m, int num_sms, cudaStream_t s) {
    static PerDeviceOnce once;
    cudaError_t e = raise_smem(once, gated_grad_tc_kernel<D>, GrCfg<D>::SMEM);
    if (e != cudaSuccess) return e;
    const int64_t slots = p.groups * p.nc;
    gated_grad_tc_kernel<D><<<grid_for(slots, num_sms), GrCfg<D>::kThreads, GrCfg<D>::SMEM, s>>>(m, p, slots);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gated_states_tc(const GatedProblem& p, const GatedMaps& m, bool grad, int num_sms, cudaStream_t s) {
    const bool alone = grad && !p.sums && (p.cu != nullptr || p.rows <= C);
    if (p.dk == 128) return alone ? states_d<128, true>(p, m, grad, num_sms, s) : states_d<128, false>(p, m, grad, num_sms, s);
    return alone ? states_d<64, true>(p, m, grad, num_sms, s) : states_d<64, false>(p, m, grad, num_sms, s);
}
cudaError_t launch_gated_prefill_tc(const GatedProblem& p, const GatedMaps& m, int num_sms, cudaStream_t s) {
    return p.dk == 128 ? prefill_d<128>(p, m, num_sms, s) : prefill_d<64>(p, m, num_sms, s);
}
cudaError_t launch_gated_grad_tc(const GatedProblem& p, const GatedMaps& m, int num_sms, cudaStream_t s) {
    return p.dk == 128 ? grad_d<128>(p, m, num_sms, s) : grad_d<64>(p, m, num_sms, s);
}

}  // namespace la
