// decode_few_sm103.cu -- paged MLA decode for at most 32 heads, one SM per unit.
//
// What it computes is what the decode kernels do for a unit: one query row, tokens [j0, j1). Those
// kernels put the heads on the tensor core's M side (128 rows, of which 16 heads use an eighth) and
// need two SMs for the 128 x 512 accumulator. With few heads the operands are swapped: the tokens
// and the latent dims are the M side, the heads the N side (N = 16 or 32):
//     S^T[token, head] = K Q^T     36 MMAs a page, M = 128 (the page's 64 rows; the other 64 are
//                                  whatever follows in shared memory, and their results unused)
//     O^T[dim, head] += V^T P^T    4 blocks of 128 dims x 4 steps of 16 tokens, V^T read from the same
//                                  tile as K (MN-major), so that a page is loaded once
// O^T takes 4 N columns of tensor memory and S^T two buffers of N, so everything fits one SM, P
// never leaves it, and 152 units run at once.
//
// Bound, bf16 cache: 74 KB a page from memory against about 52 MMAs of 50 cycles: at 152 units the cache
// stream is the limit. Measured over 64 rows of 128 selected pages of 16 heads: 122 us, 5.0 TB/s of pages
// (one row of 16 pages: 12 us, latency; the decode kernel takes 160 and 20). Prefetching further ahead
// of the ring was slower (6 pages instead of 3: 144 us). 16 KB pairs of 64-dim panels go through a
// ring of 10 or 11 slots (two pages and more), the rope panels through one of their own; one thread
// loads, one warp issues, and eight warps do the rest: the 64 tokens are lanes 0-63 of S^T (two lane
// quarters), each of two warp sets taking half of the heads.
// A thread holds one token's scores of its heads; the row maximum over tokens is only formed when some
// score passes its head's running maximum by 2^8 (one barrier with an OR tells), so that a page
// usually needs no reduction across threads. Sums are kept per thread and reduced once at the end:
// l of the bf16-rounded weights normalises O (as the MMA sees them), lt of the unrounded ones gives
// the LSE.
//
// FP8 cache: eight more warps load a page's codes straight into registers, one page ahead, and widen
// them into the same ring (a page is widened once for both products, where the decode kernel's two SMs
// widen it once each). A token's k_scale multiplies the scores of the thread that holds it, its
// v_scale the weight before its one rounding; both sums are of the unscaled weights. Bound: the widening
// warps and the 1.4 us of MMAs a page: 64 rows of 128 pages of 16 heads 135 us, of 32 heads 150 (the decode
// kernel: 230), one row of 16 pages 12.6 (19.5). Waiting for a page's slots pair by pair in a loop cost
// 149 and 175 us, a ring of two pages 147 and 163, without the L2 prefetch 173.
//
// All waits are bounded (see sm103_ptx.cuh).
#include <cuda.h>
#include <math_constants.h>

#include <cstring>

#include "decode_common.cuh"
#include "internal.h"
#include "sm103_ptx.cuh"

namespace mla {

cudaError_t encode_tmap(CUtensorMap* map, CUtensorMapDataType dtype, int rank, const void* base,
                        const uint64_t* dims, const uint64_t* strides_bytes, const uint32_t* box, bool swizzle128);

namespace {

using namespace ptx;
using namespace dec;

// warp 0 TMA, 1 MMA, 2-3 L2 prefetch, 4-11 softmax and epilogue, FP8: 12-19 converters
constexpr int threads_of(bool fp8) { return fp8 ? 640 : 384; }
constexpr int kWork = 256;
constexpr int kConvWarps = 8;
constexpr int kPanel = kPage * 128;     // one page's rows of one 64-dim panel (8 KB)
constexpr int kPair = 2 * kPanel;
constexpr int kCtrl = 4096;
constexpr int kSmemLimit = 232448;
constexpr int kMaxPairs = 11, kMaxRopes = 2;
constexpr float kRescaleThreshold = 8.0f;  // log2 units
// pages between the softmax's progress and the page prefetched into L2
constexpr int ahead_of(bool fp8) { return fp8 ? 2 : 3; }

// Shared memory for N = 2 NH heads: the rings first, since an MMA of M = 128 reads 8 KB past a panel.
template <int NH>
struct Layout {
    static constexpr int N = 2 * NH;
    static constexpr int kQPanel = N * 128;  // N heads x 64 dims
    static constexpr int kP = N * 128;       // N heads x 64 tokens
    static constexpr int kRopes = 2;
    static constexpr int kPBufs = 2;
    static constexpr int kPairs = (kSmemLimit - kCtrl - 9 * kQPanel - kPBufs * kP - kRopes * kPanel) / kPair;
    static constexpr int kRing = kCtrl;
    static constexpr int kRope = kRing + kPairs * kPair;
    static constexpr int kQ = kRope + kRopes * kPanel;
    static constexpr int kPBuf = kQ + 9 * kQPanel;
    static constexpr int kBytes = kPBuf + kPBufs * kP;
    // a page's scores are issued before the previous page's output: both pages' pairs are held
    static_assert(kPairs >= 8 && kPairs <= 11 && kPairs <= kMaxPairs && kRopes <= kMaxRopes && kBytes <= kSmemLimit, "ring");
    static_assert(9 * kQPanel >= kPanel, "the last rope panel's MMA reads 8 KB on, into Q");
    static constexpr uint32_t kCols = 6 * N <= 128 ? 128 : 256;  // a power of two
    static constexpr uint32_t kO = 2 * N;  // S^T buffers at 0 and N, O^T blocks from here
};

enum : int {
    B_KF = 0,                   // pair landed
    B_RF = B_KF + kMaxPairs,    // rope panel landed
    B_Q = B_RF + kMaxRopes,     // Q landed
    B_SF,                       // [2] S^T of the page (by its parity) ready: its rope slot is free
    B_SE = B_SF + 2,            // [2] S^T read (one arrival of each of the four token warps)
    B_PF = B_SE + 2,            // [2] P written, O^T rescaled, V rows past the last token zeroed (256)
    B_PE = B_PF + 2,            // [2] PV MMAs of the page completed: its pair slots are free
    B_COUNT = B_PE + 2
};
static_assert(8 * B_COUNT <= 512, "barrier slots");
constexpr int OFF_TMEM = 512, OFF_ABORT = 516;
constexpr int OFF_PROG = 520;    // pages whose softmax is done (paces the L2 prefetch)
constexpr int OFF_MX = 1024;     // f32 [2][64] maxima of the two token quarters; at the end sums of l
constexpr int OFF_LT = 1536;     // f32 [2][64] sums of lt
constexpr int OFF_ALPHA = 2048;  // f32 [64]
constexpr int OFF_M = 2304;      // f32 [64] final running maxima (log2 units)
constexpr uint32_t kBarOr = 1, kBarWork = 2;

// The maximum or sum over the warp of each of v[0 .. NH), NH 8 or 16: in each step a lane
// keeps half of its values and gives the other half away, so that it ends with the value of index
// reduced_index<NH>(lane) in v[0] after 9 or 16 exchanges (one value at a time takes 5 NH).
template <int NH, bool kMax, int O = 16, int n = NH>
__device__ __forceinline__ void warp_reduce(float (&v)[NH], int lane) {
    auto op = [](float a, float b) { return kMax ? fmaxf(a, b) : a + b; };
    if constexpr (n > 1) {
        const bool up = (lane & O) != 0;
#pragma unroll
        for (int k = 0; k < n / 2; ++k) {
            const float other = __shfl_xor_sync(0xffffffffu, up ? v[k] : v[k + n / 2], O);
            v[k] = op(up ? v[k + n / 2] : v[k], other);
        }
    } else {
        v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], O));
    }
    if constexpr (O > 1) warp_reduce<NH, kMax, O / 2, (n > 1 ? n / 2 : 1)>(v, lane);
}
template <int NH>
__device__ __forceinline__ int reduced_index(int lane) {
    return NH == 16 ? lane >> 1 : lane >> 2;
}

// Eight e4m3 codes -> eight bf16 (exact), as one 16-byte chunk of a bf16 row.
__device__ __forceinline__ uint4 widen8(uint2 v) {
    uint4 o;
    e4m3x4_to_bf16x4(v.x, o.x, o.y);
    e4m3x4_to_bf16x4(v.y, o.z, o.w);
    return o;
}

// Hint: bring the 128-byte line at `ptr` into L2 (no effect on correctness).
__device__ __forceinline__ void prefetch_l2(const void* ptr) { asm volatile("prefetch.global.L2 [%0];" ::"l"(ptr)); }

template <int NH, bool kFp8>
__global__ void __launch_bounds__(threads_of(kFp8), 1)
    decode_few_kernel(const __grid_constant__ CUtensorMap pair_map, const __grid_constant__ CUtensorMap rope_map,
                      const __grid_constant__ CUtensorMap q_map, const DecodeArgs p) {
    using Lay = Layout<NH>;
    constexpr int N = Lay::N;
    constexpr uint32_t kIdescQK = idesc_bf16_f32(128, N, false, false);
    constexpr uint32_t kIdescPV = idesc_bf16_f32(128, N, true, false);
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_addr(smem);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    if (sbase & 1023u) {  // the swizzled layouts need 1024-byte aligned tiles; never expected
        if (tid == 0 && p.dev_status) atomicOr(p.dev_status, MLA_DEV_WAIT_TIMEOUT);
        return;
    }
    const int unit = (int)blockIdx.x;
    RowGeom g{};
    if (!p.plan_units && p.order != kOrderWaitFirst) g = row_geometry(p, unit, tid == 0);
    volatile int* abort = reinterpret_cast<volatile int*>(smem + OFF_ABORT);
    int32_t* ds = p.dev_status;
    auto bar = [&](int i) -> uint32_t { return sbase + 8u * (uint32_t)i; };
    if (tid == 0) {
        *abort = 0;
        *reinterpret_cast<volatile int*>(smem + OFF_PROG) = 0;
        for (int i = 0; i < B_COUNT; ++i) {
            uint32_t cnt = 1;
            if (i >= B_SE && i < B_SE + 2) cnt = 4;
            if (i >= B_PF && i < B_PF + 2) cnt = kWork;
            if (kFp8 && i < B_Q) cnt = kConvWarps;  // panels widened by the converter warps
            bar_init(bar(i), cnt);
        }
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(sbase + OFF_TMEM, Lay::kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(smem + OFF_TMEM), 0);
    if (tid == 0) griddep_launch_dependents();
    if (p.plan_units || p.order == kOrderWaitFirst) {
        if (p.order != kOrderFree) griddep_wait();
        if (p.plan_units && unit >= *p.plan_count) {
            if (warp == 1) tmem_dealloc(tmem, Lay::kCols);
            return;
        }
        g = row_geometry(p, unit, tid == 0);
    }
    const int npages = g.npages;

    if (kFp8 && warp == 0) {
        if (lane == 0 && npages > 0) {
            tma_prefetch_desc(&q_map);
            if (p.order != kOrderFree) griddep_wait();
            bar_arrive_expect_tx(bar(B_Q), 9 * Lay::kQPanel);
            for (int pn = 0; pn < 9; ++pn)
                tma_load_2d(sbase + Lay::kQ + pn * Lay::kQPanel, &q_map, bar(B_Q), pn * 64, g.r * p.H);
            volatile int dummy = 0;  // it has landed before the CTA can exit, also after an abort
            wait_bar(bar(B_Q), 0, &dummy, nullptr);
        }
    } else if (warp == 0) {
        if (lane == 0 && npages > 0) {
            tma_prefetch_desc(&pair_map);
            tma_prefetch_desc(&rope_map);
            tma_prefetch_desc(&q_map);
            const int oob = (int)(p.num_blocks * kPage);  // one past the cache: TMA fills zeros
            // A commit costs the issuing warp about 50 ns, so there are two a page: the slots are
            // freed page by page, and the thread follows the pages' barriers in order. Each wait is
            // for a phase at most one behind: a page's loads ask for the page two earlier (or a
            // later one), and no page after it can be scored or summed before it is loaded.
            bool q_issued = false, ok = true;
            int pairs = 0, ropes = 0;  // issued
            int scored = 0, summed = 0;  // pages whose QK, whose PV MMAs are known to have completed
            auto follow = [&](int& done, int upto, int bars) -> bool {
                for (; done <= upto; ++done)
                    if (!wait_bar(bar(bars + (done & 1)), (done >> 1) & 1, abort, ds)) return false;
                return true;
            };
            for (int i = 0; i < npages && ok; ++i) {
                const int blk = page_block(p, g.b, g.page0 + i);
                const int y = blk < 0 ? oob : blk * kPage;
                for (int b = 0; b < 4; ++b) {
                    const int m = 4 * i + b, slot = m % Lay::kPairs;
                    if (m >= Lay::kPairs && !(ok = follow(summed, (m - Lay::kPairs) / 4, B_PE))) break;
                    bar_arrive_expect_tx(bar(B_KF + slot), kPair);
                    tma_load_3d(sbase + Lay::kRing + slot * kPair, &pair_map, bar(B_KF + slot), 0, y, 2 * b);
                    ++pairs;
                }
                if (!ok) break;
                if (!q_issued) {  // behind the first page: q may be the preceding kernel's output
                    if (p.order != kOrderFree) griddep_wait();
                    bar_arrive_expect_tx(bar(B_Q), 9 * Lay::kQPanel);
                    for (int pn = 0; pn < 9; ++pn)
                        tma_load_2d(sbase + Lay::kQ + pn * Lay::kQPanel, &q_map, bar(B_Q), pn * 64, g.r * p.H);
                    q_issued = true;
                }
                const int slot = i % Lay::kRopes;
                if (i >= Lay::kRopes && !(ok = follow(scored, i - Lay::kRopes, B_SF))) break;
                bar_arrive_expect_tx(bar(B_RF + slot), kPanel);
                tma_load_3d(sbase + Lay::kRope + slot * kPanel, &rope_map, bar(B_RF + slot), 0, y, 8);
                ++ropes;
            }
            if (*abort) {  // let the copies in flight land before the CTA can exit
                volatile int dummy = 0;
                if (q_issued) wait_bar(bar(B_Q), 0, &dummy, nullptr);
                for (int m = max(0, pairs - Lay::kPairs); m < pairs; ++m) {
                    dummy = 0;
                    wait_bar(bar(B_KF + m % Lay::kPairs), (m / Lay::kPairs) & 1, &dummy, nullptr);
                }
                for (int m = max(0, ropes - Lay::kRopes); m < ropes; ++m) {
                    dummy = 0;
                    wait_bar(bar(B_RF + m % Lay::kRopes), (m / Lay::kRopes) & 1, &dummy, nullptr);
                }
            } else {  // teardown: the MMAs have read everything, no commit is on its way here
                follow(scored, npages - 1, B_SF);
                follow(summed, npages - 1, B_PE);
            }
        }
    } else if (warp == 1) {
        if (npages > 0) {
            const bool leader = elect_one();  // the whole warp runs the loop (see the decode kernel)
            bool ok = warp_wait(bar(B_Q), 0, abort, ds);
            const uint64_t q0 = smem_desc_sw128(sbase + Lay::kQ, 16, 1024);
            // page i's scores, then page i - 1's output: its softmax runs beside the scores' MMAs
            for (int i = 0; i <= npages && ok; ++i) {
                if (i < npages) {
                    const int buf = i & 1;
                    if (i >= 2) {
                        if (!(ok = warp_wait(bar(B_SE + buf), ((i >> 1) - 1) & 1, abort, ds))) break;
                        tc_fence_after();
                    }
                    const uint32_t d = tmem + (uint32_t)(buf * N);
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const int m = 4 * i + b, slot = m % Lay::kPairs;
                        if (!(ok = warp_wait(bar(B_KF + slot), (m / Lay::kPairs) & 1, abort, ds))) break;
                        if (kFp8) tc_fence_after();  // written by the converter warps
                        const uint64_t a0 = smem_desc_sw128(sbase + Lay::kRing + slot * kPair, 16, 1024);
#pragma unroll
                        for (int j = 0; j < 8; ++j)  // two panels of four steps
                            if (leader)
                                mma_ss(d, a0 + (uint64_t)(((j >> 2) * kPanel + 32 * (j & 3)) >> 4),
                                       q0 + (uint64_t)(((2 * b + (j >> 2)) * Lay::kQPanel + 32 * (j & 3)) >> 4), kIdescQK,
                                       (b | j) ? 1u : 0u);
                    }
                    if (!ok) break;
                    const int rs = i % Lay::kRopes;
                    if (!(ok = warp_wait(bar(B_RF + rs), (i / Lay::kRopes) & 1, abort, ds))) break;
                    if (kFp8) tc_fence_after();
                    const uint64_t a0 = smem_desc_sw128(sbase + Lay::kRope + rs * kPanel, 16, 1024);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (leader)
                            mma_ss(d, a0 + (uint64_t)(2 * j), q0 + (uint64_t)((8 * Lay::kQPanel + 32 * j) >> 4), kIdescQK, 1u);
                    if (leader) mma_commit(bar(B_SF + buf));
                }
                if (i > 0) {
                    const int j = i - 1, buf = j & 1;
                    if (!(ok = warp_wait(bar(B_PF + buf), (j >> 1) & 1, abort, ds))) break;
                    tc_fence_after();
                    const uint64_t b0 = smem_desc_sw128(sbase + Lay::kPBuf + (j % Lay::kPBufs) * Lay::kP, 16, 1024);
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const int slot = (4 * j + b) % Lay::kPairs;
                        const uint64_t a0 = smem_desc_sw128(sbase + Lay::kRing + slot * kPair, kPanel, 1024);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (leader)
                                mma_ss(tmem + Lay::kO + (uint32_t)(b * N), a0 + (uint64_t)((k * 2048) >> 4),
                                       b0 + (uint64_t)(2 * k), kIdescPV, k > 0 ? 1u : (j > 0 ? 1u : 0u));
                    }
                    if (leader) mma_commit(bar(B_PE + buf));
                }
            }
        }
    } else if (warp >= 4 && warp < 12) {
        const int quarter = warp & 3, set = (warp - 4) >> 2;
        const int h0 = set * NH;               // this set's heads [h0, h0 + NH)
        const bool tokens = quarter < 2;       // holds tokens 32 quarter + lane
        const int token = 32 * quarter + lane;
        const uint32_t lane_base = (uint32_t)(32 * quarter) << 16;
        const int wtid = tid - 128;
        float* mx = reinterpret_cast<float*>(smem + OFF_MX);
        float* lts = reinterpret_cast<float*>(smem + OFF_LT);
        float* alpha_s = reinterpret_cast<float*>(smem + OFF_ALPHA);
        float* m_s = reinterpret_cast<float*>(smem + OFF_M);
        const float sl2 = p.scale * 1.4426950408889634f;  // exp2 domain
        float m[NH], l[NH], lt[NH];
#pragma unroll
        for (int k = 0; k < NH; ++k) {
            m[k] = kNoMax;
            l[k] = lt[k] = 0.f;
        }
        // FP8: (k_scale, v_scale) of this thread's token, a page ahead; 0 where there is no token
        float2 scale = make_float2(0.f, 0.f), scale_next = scale;
        int blk_next = -1;  // the block two pages ahead
        auto block_of = [&](int i) -> int {
            if (i >= npages) return -1;
            const int32_t blk = *table_entry(p, g.b, g.page0 + i);
            return (int64_t)blk < p.num_blocks ? blk : -1;
        };
        auto scale_of = [&](int i, int blk) -> float2 {
            if (blk < 0 || token >= valid_rows(g, i)) return make_float2(0.f, 0.f);
            return __ldcg(reinterpret_cast<const float2*>(p.cache + ((size_t)blk * kPage + token) * kFp8RowBytes + kD));
        };
        if (kFp8 && tokens) {
            scale_next = scale_of(0, block_of(0));
            blk_next = block_of(1);
        }
        for (int i = 0; i < npages; ++i) {
            // No early exit: all 256 threads must pass the same named barriers (which cannot time
            // out); after an abort the waits return at once and the work is skipped.
            const int buf = i & 1, valid = valid_rows(g, i);
            if (kFp8 && tokens) {
                scale = scale_next;
                scale_next = scale_of(i + 1, blk_next);
                blk_next = block_of(i + 2);
            }
            const bool okS = warp_wait(bar(B_SF + buf), (i >> 1) & 1, abort, ds);
            uint32_t s[NH];
            bool need = false;
            if (tokens) {
                if (okS) {
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < NH; k += 8) tmem_ld8(tmem + lane_base + (uint32_t)(buf * N + h0 + k), s + k);
                    tmem_wait_ld();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) bar_arrive(bar(B_SE + buf));
                }
#pragma unroll
                for (int k = 0; k < NH; ++k) {  // tokens past the last and heads past H have no weight
                    if (kFp8) s[k] = __float_as_uint(__uint_as_float(s[k]) * scale.x);  // K = codes * k_scale
                    if (!okS || token >= valid || h0 + k >= p.H) s[k] = __float_as_uint(-CUDART_INF_F);
                    need |= __uint_as_float(s[k]) * sl2 > m[k] + kRescaleThreshold;
                }
            }
            const bool any = named_bar_or(kBarOr, kWork, need);
            if (any) {
                if (tokens) {
                    float x[NH];
#pragma unroll
                    for (int k = 0; k < NH; ++k) x[k] = __uint_as_float(s[k]);
                    warp_reduce<NH, true>(x, lane);
                    mx[64 * quarter + h0 + reduced_index<NH>(lane)] = x[0];
                }
                named_bar(kBarWork, kWork);
                if (tokens) {
#pragma unroll
                    for (int k = 0; k < NH; ++k) {
                        const float mt = fmaxf(mx[h0 + k], mx[64 + h0 + k]) * sl2;  // scale > 0
                        float a = 1.f;
                        if (mt > m[k] + kRescaleThreshold) {
                            a = fast_exp2(m[k] - mt);  // 0 the first time
                            m[k] = mt;
                        }
                        l[k] *= a;
                        lt[k] *= a;
                        if (quarter == 0 && lane == 0) alpha_s[h0 + k] = a;
                    }
                }
                named_bar(kBarWork, kWork);
                if (i > 0 && warp_wait(bar(B_PE + ((i - 1) & 1)), ((i - 1) >> 1) & 1, abort, ds)) {
                    // O^T holds every earlier page's product: rescale it, column by column
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < 2 * N; c += 8) {  // this set's two blocks of 128 dims
                        uint32_t v[8];
                        const uint32_t col = tmem + lane_base + Lay::kO + (uint32_t)(2 * set * N + c);
                        tmem_ld8(col, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            v[k] = __float_as_uint(__uint_as_float(v[k]) * alpha_s[(c + k) % N]);
                        tmem_st8(col, v);
                    }
                    tmem_wait_st();
                }
            }
            // the P buffer is free once the PV of the page that used it last has completed
            if (i >= Lay::kPBufs) {
                const int j = i - Lay::kPBufs;
                warp_wait(bar(B_PE + (j & 1)), (j >> 1) & 1, abort, ds);
            }
            if (tokens) {
                uint8_t* pb = smem + Lay::kPBuf + (i % Lay::kPBufs) * Lay::kP;
#pragma unroll
                for (int k = 0; k < NH; ++k) {
                    const int h = h0 + k;
                    const float e = fast_exp2(fmaf(__uint_as_float(s[k]), sl2, -m[k]));
                    // V = codes * v_scale: the scale multiplies the weight before its one rounding, and
                    // both sums are of the unscaled weights
                    const uint32_t r = pack_bf16x2(kFp8 ? e * scale.y : e, 0.f) & 0xffffu;
                    lt[k] += e;
                    if (!kFp8) l[k] += bf16_lo_f(r);
                    *reinterpret_cast<uint16_t*>(pb + h * 128 + (((token >> 3) ^ (h & 7)) << 4) + (token & 7) * 2) =
                        (uint16_t)r;
                }
            }
            if (!kFp8 && valid < kPage) {  // V rows past the last token may hold anything, also NaN: 0 * NaN
                for (int q = wtid; q < (kPage - valid) * 64; q += kWork) {
                    const int row = valid + q / 64, pn = (q >> 3) & 7, c = q & 7;
                    const int slot = (4 * i + (pn >> 1)) % Lay::kPairs;
                    *reinterpret_cast<uint4*>(smem + Lay::kRing + slot * kPair + (pn & 1) * kPanel + row * 128 + c * 16) =
                        make_uint4(0, 0, 0, 0);
                }
            }
            fence_proxy_async_cta();  // P and the zeros, before the MMAs read them
            tc_fence_before();
            bar_arrive(bar(B_PF + buf));
            if (wtid == 0) *reinterpret_cast<volatile int*>(smem + OFF_PROG) = i + 1;
        }
        // sums over the tokens; l and lt of the two quarters meet in shared memory
        named_bar(kBarWork, kWork);
        if (tokens) {
            if (quarter == 0 && lane == 0) {
#pragma unroll
                for (int k = 0; k < NH; ++k) m_s[h0 + k] = m[k];
            }
            if (!kFp8) warp_reduce<NH, false>(l, lane);
            warp_reduce<NH, false>(lt, lane);
            mx[64 * quarter + h0 + reduced_index<NH>(lane)] = kFp8 ? lt[0] : l[0];
            lts[64 * quarter + h0 + reduced_index<NH>(lane)] = lt[0];
        }
        output_wait(p, unit);
        const bool has_o = npages > 0 && !*abort;
        const bool o_ok = has_o && warp_wait(bar(B_PE + ((npages - 1) & 1)), ((npages - 1) >> 1) & 1, abort, ds);
        tc_fence_after();
        named_bar(kBarWork, kWork);
        if (wtid < N) {
            const float lv = mx[wtid] + mx[64 + wtid], ltv = lts[wtid] + lts[64 + wtid];
            const bool empty = !o_ok || lv == 0.f;  // no token has a weight; a NaN sum is a NaN result
            alpha_s[wtid] = empty ? 0.f : 1.f / lv;
            if (wtid < p.H) {
                const float lse = empty ? -CUDART_INF_F : (m_s[wtid] + log2f(ltv)) * 0.6931471805599453f;
                if (g.slot >= 0)
                    p.part_lse[(size_t)g.slot * p.H + wtid] = lse;
                else if (p.lse)
                    p.lse[(size_t)g.r * p.H + wtid] = lse;
            }
        }
        named_bar(kBarWork, kWork);
        // O^T / l: a warp's lanes are 32 consecutive dims of one head, so its stores are whole lines
        const bool f32 = g.slot >= 0 || p.o_dtype == MLA_DT_F32;
        const size_t row = (size_t)(g.slot >= 0 ? g.slot : g.r) * p.H;
        float* of = g.slot >= 0 ? p.part_o : (float*)p.o_latent;
        uint16_t* oh = (uint16_t*)p.o_latent;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int dim = 128 * (2 * set + b) + 32 * quarter + lane;
#pragma unroll
            for (int hb = 0; hb < N; hb += 16) {
                uint32_t v[16];
                const uint32_t col = tmem + lane_base + Lay::kO + (uint32_t)((2 * set + b) * N + hb);
                tmem_ld8(col, v);
                tmem_ld8(col + 8u, v + 8);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const int h = hb + k;
                    const float inv = alpha_s[h];
                    const float x = inv != 0.f ? __uint_as_float(v[k]) * inv : 0.f;  // an empty row: O may hold anything
                    if (h < p.H) {
                        if (f32)
                            of[(row + h) * kL + dim] = x;
                        else
                            oh[(row + h) * kL + dim] = (uint16_t)(pack_bf16x2(x, 0.f) & 0xffffu);
                    }
                }
            }
        }
    } else if (kFp8 && warp >= 12) {
        // ---------------- converter warps 12-19 (256 threads), FP8 ----------------
        // They load a page's codes from global memory into registers while they widen the page before
        // it, 8 codes a load: of pair b, row r0 + 16 k, chunk cc of its 16; of the rope panel, row
        // q0 + 32 k, chunk qc of 8. Rows past the last token and pages without a block are zero, so
        // that stale or NaN codes cannot leak through 0 * NaN.
        const int ctid = tid - 384;
        const int r0 = ctid >> 4, cc = ctid & 15, q0 = ctid >> 3, qc = ctid & 7;
        const uint32_t pair_dst = sbase + Lay::kRing + (cc >> 3) * kPanel + r0 * 128 + (((cc & 7) ^ (r0 & 7)) << 4);
        const uint32_t rope_dst = sbase + Lay::kRope + q0 * 128 + ((qc ^ (q0 & 7)) << 4);
        uint2 v[4][4], w[2];
        const uint8_t* src = nullptr;  // of the page being loaded
        int rows = 0;                  // its rows that hold tokens
        auto open = [&](int i) {
            rows = 0;
            if (i >= npages) return;
            const int blk = page_block(p, g.b, g.page0 + i);
            if (blk < 0) return;
            rows = valid_rows(g, i);
            src = p.cache + (size_t)blk * (kPage * kFp8RowBytes);
        };
        auto load_pair = [&](int b) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int row = r0 + 16 * k;
                v[b][k] = make_uint2(0u, 0u);
                if (row < rows) v[b][k] = __ldcg(reinterpret_cast<const uint2*>(src + row * kFp8RowBytes + 128 * b + 8 * cc));
            }
        };
        auto load_rope = [&]() {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int row = q0 + 32 * k;
                w[k] = make_uint2(0u, 0u);
                if (row < rows) w[k] = __ldcg(reinterpret_cast<const uint2*>(src + row * kFp8RowBytes + kL + 8 * qc));
            }
        };
        if (npages > 0) {
            open(0);
#pragma unroll
            for (int b = 0; b < 4; ++b) load_pair(b);
            load_rope();
        }
        // A page's first kWaitAt pairs go where pairs of the page three earlier were, which completed
        // before the page ahead of this one was written; the others wait for the page two earlier.
        constexpr int kWaitAt = Lay::kPairs - 8;
        static_assert(kWaitAt >= 0 && kWaitAt < 4 && Lay::kRopes == 2, "ring");
        bool ok = true;
        for (int i = 0; i < npages && ok; ++i) {
            open(i + 1);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                if (b == kWaitAt && i >= 2) ok = warp_wait(bar(B_PE + (i & 1)), ((i - 2) >> 1) & 1, abort, ds);
                if (!ok) break;
                const int slot = (4 * i + b) % Lay::kPairs;
#pragma unroll
                for (int k = 0; k < 4; ++k) sts_u4(pair_dst + slot * kPair + k * 16 * 128, widen8(v[b][k]));
                fence_proxy_async_cta();  // generic-proxy writes before the MMAs read them
                warp_arrive(bar(B_KF + slot), lane);
                load_pair(b);
            }
            if (!ok) break;
            const int rs = i % Lay::kRopes;
#pragma unroll
            for (int k = 0; k < 2; ++k) sts_u4(rope_dst + rs * kPanel + k * 32 * 128, widen8(w[k]));
            fence_proxy_async_cta();
            warp_arrive(bar(B_RF + rs), lane);
            load_rope();
        }
    } else {
        // Warps 2, 3: pages that the ring has no room for yet are brought into L2, kAhead pages
        // past the last one whose softmax is done. Only a hint: gives up quietly if it falls behind.
        const volatile int* prog = reinterpret_cast<const volatile int*>(smem + OFF_PROG);
        int spins = 0;
        for (int t = 2; t < npages; ++t) {
            bool go = true;
            while (*prog < t - ahead_of(kFp8)) {
                if (*abort || ++spins > (1 << 20)) {
                    go = false;
                    break;
                }
                __nanosleep(128);
            }
            if (!go) break;
            const int32_t blk = *table_entry(p, g.b, g.page0 + t);
            if (blk < 0 || (int64_t)blk >= p.num_blocks) continue;
            constexpr int kPageBytes = kPage * (kFp8 ? kFp8RowBytes : kBf16RowBytes);
            const uint8_t* page = p.cache + (size_t)blk * kPageBytes;
            for (int q = tid - 64; q < kPageBytes / 128; q += 64) prefetch_l2(page + 128 * q);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, Lay::kCols);
}

template <int NH, bool kFp8>
cudaError_t launch(const DecodeArgs& a, cudaStream_t s) {
    static int done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !done[dev]) {
        e = cudaFuncSetAttribute(decode_few_kernel<NH, kFp8>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<NH>::kBytes);
        if (e != cudaSuccess) return e;
        if (dev < 64) done[dev] = 1;
    }
    CUtensorMap pair_map, rope_map, q_map;
    memset(&pair_map, 0, sizeof pair_map);
    memset(&rope_map, 0, sizeof rope_map);
    memset(&q_map, 0, sizeof q_map);
    if (a.num_blocks > 0 && a.max_seq_len > 0) {
        if constexpr (!kFp8) {  // the cache's rows as [panel of 64 dims][row][64]
            const uint64_t dims[3] = {64, (uint64_t)a.num_blocks * kPage, (uint64_t)(kD / 64)};
            const uint64_t strides[2] = {(uint64_t)kBf16RowBytes, 128};
            uint32_t box[3] = {64, (uint32_t)kPage, 2};
            e = encode_tmap(&pair_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.cache, dims, strides, box, true);
            if (e != cudaSuccess) return e;
            box[2] = 1;
            e = encode_tmap(&rope_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.cache, dims, strides, box, true);
            if (e != cudaSuccess) return e;
        }
        const uint64_t qdims[2] = {(uint64_t)kD, (uint64_t)a.rows * a.H};
        const uint64_t qstrides[1] = {(uint64_t)kD * 2};
        const uint32_t qbox[2] = {64, 2 * NH};
        e = encode_tmap(&q_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.q, qdims, qstrides, qbox, true);
        if (e != cudaSuccess) return e;
    }
    const int64_t units = a.plan_units ? a.plan_max_units : (int64_t)a.rows * a.num_splits;
    return launch_pdl(decode_few_kernel<NH, kFp8>, dim3((unsigned)units), dim3(threads_of(kFp8)), Layout<NH>::kBytes, s, pair_map,
                      rope_map, q_map, a);
}

}  // namespace

cudaError_t launch_decode_few_sm103(const DecodeArgs& a, cudaStream_t s) {
    if (a.kv_dtype == MLA_KV_FP8_E4M3_SCALED) return a.H <= 16 ? launch<8, true>(a, s) : launch<16, true>(a, s);
    return a.H <= 16 ? launch<8, false>(a, s) : launch<16, false>(a, s);
}

}  // namespace mla
