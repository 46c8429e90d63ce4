// decode_prefix_sm103.cu -- the shared part of mla_decode_shared_prefix: every query row and head of
// the batch against the prefix pages, which all requests have in common.
//
// For a flat row f = (request, query position, head) of the batch's R*H rows and a range of the
// prefix tokens:  S = scale * q[f] K^T,  P = softmax(S),  o[f] = P V,  written as a partial state
// (o, lse) that the merge combines with the other ranges and with the row's own tokens.
//
// What bounds it. With the keys common to all rows the work is a plain matrix product: 2 * 256 * 64 *
// (576 + 512) flops per page and 256 rows, against 74 KB of keys that stay in L2. mla_decode's kernel
// takes 128 rows at a time; every key byte is then written to shared memory once and read by the
// tensor core once, and that traffic, not the tensor core, sets its pace (128 B/clk for full-rate
// MMAs of M = 128). Here two SMs work as a pair on 256 rows (tcgen05 cta_group::2, M = 256): each SM
// loads half of the keys and the tensor cores of both read both halves, which halves the
// shared-memory traffic per flop.
//
// One cluster of four CTAs per (256 flat rows, range of pages); CTA i of a pair holds rows
// [128 i, 128 i + 128):
//   CTAs 0, 1 ("scores")  Q: 512 latent dims in tensor memory (256 columns), 64 rope dims in shared
//       memory. Pages go two at a time ("groups" of 128 tokens): CTA i loads page 2 g + i, three
//       64-dim panels (24 KB) per ring slot and TMA copy. S = Q K^T per group: 36 pair MMAs of
//       M = 256 x N = 128 x K = 16 into one of two 128-column buffers, so that the next group's
//       run while this one's softmax reads. Softmax: sixteen warps, four per TMEM lane quarter, half a
//       page of the group each; fp32 online softmax whose running maximum moves only when it grows by
//       more than 2^8. One barrier a group tells whether any row's does; only then are the maxima
//       of the four parts exchanged. P (bf16, swizzled) and the rows' rescale factors are staged,
//       and a warp of its own sends them to the output CTA of the same rows, one bulk copy a page.
//   CTAs 2, 3 ("output")  hold the 256 x 512 fp32 output accumulators (all of both SMs' tensor
//       memory). CTA i loads dims [128 i, 128 i + 128) and [256 + 128 i, ...) of each page; per page
//       8 pair MMAs of M = 256 x N = 256 x K = 16, V read as an MN-major operand from the TMA tile.
//       Helper warps rescale O when a group's maximum moved. Epilogue: fp32 O / l by TMA stores.
//
// Measured: 2048 flat rows over 32768 tokens 96 us, 1.51 PFLOP/s; 8192 rows over 4096 tokens 55 us,
// 1.33 (32 units of one range each: 4 of 36 clusters idle, and the 9 us to the first weights, the 9 us from
// the last scores to the end and the 17 MB of partial states weigh more). Steady state is 1.2 us a group, against 1.11 of MMAs at full rate: the
// 64 or 72 KB of a group from L2 come in just behind them. What it took, on the first size with the requests' own
// tokens: sixteen softmax warps for eight 293 -> 258 us (the softmax was the longest stage); arrivals at a
// peer's barrier that publish nothing without the cluster-wide release, which takes 0.9 us, 258 -> 209;
// MMAs issued by one elected lane of a converged warp, 64 cycles each instead of 140, 209 -> 175.
//
// Rounding: P to bf16 (the MMA's operand), 2^-8 relative per weight at most; the sums l that normalise
// O and give the LSE are of the unrounded fp32 weights.
//
// FP8 cache: the prefix is widened once per call to bf16 (exactly: e4m3 codes are bf16 values) into the
// workspace; k_scale multiplies the fp32 scores and v_scale the weights before their rounding.
//
// All waits are bounded (see sm103_ptx.cuh); on a timeout the kernel winds down and reports
// MLA_DEV_WAIT_TIMEOUT instead of hanging.
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
using dec::store_rows;
using dec::warp_wait;

// warp 0 TMA, 1 MMA, 2-17 softmax / 2-5 helpers, 6-9 CTA 3's relay, 2-17 epilogue, 18 P copies
constexpr int kThreads = 608;
constexpr int kSoftThreads = 512;
constexpr int kTileRows = 256;
constexpr int kPPG = 2;                      // pages per group, one per scores CTA
constexpr int kPageBox = kPage * 128;        // one page's rows of one 64-dim panel (8 KB)
constexpr int kSlotPanels = 3;
constexpr int kSlotBytes = kSlotPanels * kPageBox;  // 24 KB
constexpr int kSlots = 5;                    // K ring of a scores CTA
constexpr int kQPanelBytes = 128 * 128;      // 128 rows x 64 dims of Q (16 KB)
constexpr int kPBufs = 5;                    // P buffers of an output CTA (one page each)
constexpr int kVStages = 4;                  // V ring of an output CTA: a page's 4 panels each
constexpr int kVStageBytes = 4 * kPageBox;   // 32 KB
constexpr int kPBytes = 128 * 128;           // P page: 128 rows x 64 tokens bf16
constexpr int kPMsgBytes = (kPBytes + 512 + 4 + 15) / 16 * 16;  // P + alpha[128] + flag
constexpr int kPBufStride = 17 * 1024;
constexpr int kCtrlBytes = 4096;
// scores CTA
constexpr int OFF_QROPE = kCtrlBytes;
constexpr int OFF_RING = OFF_QROPE + kQPanelBytes;
constexpr int kStages = 4;                   // P staging buffers: each of a group's pages has two
constexpr int OFF_STAGE = OFF_RING + kSlots * kSlotBytes;
constexpr int kSmem0 = OFF_STAGE + kStages * kPBufStride;
// output CTA
constexpr int OFF_V = kCtrlBytes;
constexpr int OFF_PB = OFF_V + kVStages * kVStageBytes;
constexpr int kSmem1 = OFF_PB + kPBufs * kPBufStride;
constexpr int kSmemBytes = kSmem0 > kSmem1 ? kSmem0 : kSmem1;
static_assert(kSmemBytes <= 232448, "over the per-CTA shared memory limit");
static_assert(kPMsgBytes <= kPBufStride, "P message");
static_assert(OFF_RING % 1024 == 0 && OFF_STAGE % 1024 == 0 && OFF_PB % 1024 == 0 && kPBufStride % 1024 == 0 &&
                  kSlotBytes % 1024 == 0,
              "128-byte swizzled tiles need 1024-byte alignment");
static_assert(OFF_V + 12 * dec::kTileBytes <= kSmem1, "epilogue tiles");
// Q's latent panels land in the four staging buffers (panels 0-3) and at the end of the ring
// (panels 4-7, over slots 2-4), so that the first keys can load into slots 0 and 1 at once.
static_assert(kSlots == 5 && kStages == 4 && 4 * kQPanelBytes <= 3 * kSlotBytes, "Q panel homes");
constexpr int OFF_Q47 = OFF_RING + kSlots * kSlotBytes - 4 * kQPanelBytes;
static_assert(OFF_Q47 % 1024 == 0 && OFF_Q47 >= OFF_RING + 2 * kSlotBytes, "Q panel homes");
__device__ __forceinline__ uint32_t q_panel_off(int pn) {
    return pn < 4 ? OFF_STAGE + pn * kPBufStride : OFF_Q47 + (pn - 4) * kQPanelBytes;
}

// Barrier slots, one layout for all four CTAs (multicast commits land at the same offset in each).
enum : int {
    B_SLOTFULL = 0,                     // [kSlots] CTA 0: slot landed in both scores CTAs (TMA tx)
    B_SLOTEMPTY = B_SLOTFULL + kSlots,  // [kSlots] CTAs 0, 1: slot's QK MMAs completed
    B_SFULL = B_SLOTEMPTY + kSlots,     // [2] CTAs 0, 1: S buffer ready
    B_SEMPTY = B_SFULL + 2,             // [2] CTA 0: S buffer read by the 32 softmax warps of the pair
    B_QFULL = B_SEMPTY + 2,             // CTAs 0, 1: Q landed in shared memory
    B_QREADY,                           // CTAs 0, 1: Q latent dims moved to TMEM (512 threads)
    B_QPEER,                            // CTA 0: CTA 1's Q moved
    B_STAGEFULL,                        // [4] CTAs 0, 1: staging buffer written by the page's 8 softmax warps
    B_STAGEFREE = B_STAGEFULL + kStages,  // [4] CTAs 0, 1: staging buffer's copy has landed
    B_PEMPTY = B_STAGEFREE + kStages,         // [kPBufs] all: PV MMAs of the page in P buffer b completed
    B_VFULL = B_PEMPTY + kPBufs,        // [kVStages] CTA 2: V stage landed in both output CTAs
    B_VEMPTY = B_VFULL + kVStages,      // [kVStages] CTAs 2, 3: V stage consumed
    B_PFULL = B_VEMPTY + kVStages,      // [kPBufs] CTAs 2, 3: P message landed
    B_READY = B_PFULL + kPBufs,         // [kPBufs] CTA 2: its 4 helper warps and CTA 3 are done with the page
    B_PEER = B_READY + kPBufs,          // [kPBufs] CTA 3: its 4 helper warps are done with the page
    B_STATS = B_PEER + kPBufs,          // CTAs 2, 3: final row statistics written, last P copy issued
    B_COUNT
};
static_assert(8 * B_COUNT <= 512, "barrier slots");
constexpr int kRelayWarps = 4;    // of CTA 3, from warp 6 on: pages announced to CTA 2 in turn
constexpr int OFF_TMEM = 512;
constexpr int OFF_ABORT = 516;
constexpr int OFF_MX = 1024;      // scores: f32 [4][128] exchange between the column quarters
constexpr int OFF_STAT_M = 2048;  // output: f32 [128] final running max (log2 units)
constexpr int OFF_STAT_L = 2560;  // output: f32 [128] row sum

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSCol = 256;  // scores: Q latent in columns [0, 256), S buffers at 256 and 384
constexpr uint32_t kIdescQK = idesc_bf16_f32(256, 128, false, false);
constexpr uint32_t kIdescPV = idesc_bf16_f32(256, 256, false, true);
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr uint32_t kBarMax = 1, kBarOr = 2, kBarQuarter0 = 3;
constexpr uint32_t kBarEpi = 1;  // [4] the epilogue's warp sets (output CTAs)

template <bool kScaled>
__global__ void __cluster_dims__(4, 1, 1) __launch_bounds__(kThreads, 1)
    decode_prefix_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                         const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap o_map,
                         const PrefixArgs p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_addr(smem);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // warp-uniform, also to the compiler
    const uint32_t rank = cluster_ctarank();
    const int side = (int)(rank & 1);  // which half of the tile's rows
    const bool scores = rank < 2;
    if (sbase & 1023u) {  // the swizzled layouts need 1024-byte aligned tiles; never expected
        if (tid == 0 && p.dev_status) atomicOr(p.dev_status, MLA_DEV_WAIT_TIMEOUT);
        return;  // all CTAs of the cluster see the same alignment and leave together
    }
    const int unit = (int)(blockIdx.x >> 2);
    const int tile = unit / p.splits, split = unit % p.splits;
    const int page0 = min(p.prefix_pages, split * p.pages_per_split);
    const int npages = min(p.prefix_pages, page0 + p.pages_per_split) - page0;
    const int ngroups = (npages + kPPG - 1) / kPPG;
    const int rows0 = tile * kTileRows + 128 * side;  // first flat row of this CTA
    volatile int* abort = reinterpret_cast<volatile int*>(smem + OFF_ABORT);
    int32_t* ds = p.dev_status;
    auto bar = [&](int i) -> uint32_t { return sbase + 8u * (uint32_t)i; };

    if (tid == 0) {
        *abort = 0;
        for (int i = 0; i < B_COUNT; ++i) {
            uint32_t cnt = 1;
            if (i >= B_SEMPTY && i < B_SEMPTY + 2) cnt = 32;
            if (i == B_QREADY) cnt = kSoftThreads;
            if (i == B_STATS) cnt = 2;
            if (i >= B_STAGEFULL && i < B_STAGEFULL + kStages) cnt = 8;
            if (i >= B_READY && i < B_READY + kPBufs) cnt = 5;
            if (i >= B_PEER && i < B_PEER + kPBufs) cnt = 4;
            bar_init(bar(i), cnt);
        }
        if (!scores)  // P buffers armed for their first message before a scores CTA can send one
            for (int b = 0; b < kPBufs; ++b) bar_arrive_expect_tx(bar(B_PFULL + b), kPMsgBytes);
        fence_barrier_init();
    }
    if (warp == 0) {
        tmem_alloc_pair(sbase + OFF_TMEM, kTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    cluster_sync();  // every CTA's barriers exist before any remote arrive or copy
    const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(smem + OFF_TMEM), 0);
    griddep_wait();  // q, the cache and the lengths may be earlier kernels' outputs
    if (tid == 0) griddep_launch_dependents();

    // First cache row of the unit's page i (out of range: TMA fills zeros).
    auto page_row = [&](int i) -> int {
        if (i >= npages) return p.key_rows;
        if (!p.block_table) return (page0 + i) * kPage;  // widened prefix: its pages in order
        const int32_t blk = p.block_table[page0 + i];
        if (blk < 0 || (int64_t)blk >= p.num_blocks) {
            if (ds) atomicOr(ds, MLA_DEV_BAD_BLOCK_ID);
            return p.key_rows;
        }
        return blk * kPage;
    };

    if (scores) {
        if (warp == 0) {
            if (lane == 0 && npages > 0) {
                tma_prefetch_desc(&k_map);
                tma_prefetch_desc(&q_map);
                bar_arrive_expect_tx(bar(B_QFULL), 9 * kQPanelBytes);
                for (int qn = 0; qn < 8; ++qn)
                    tma_load_2d(sbase + q_panel_off(qn), &q_map, bar(B_QFULL), qn * 64, rows0);
                tma_load_2d(sbase + OFF_QROPE, &q_map, bar(B_QFULL), 8 * 64, rows0);
                int issued = 0;
                bool ok = true;
                for (int gi = 0; gi < ngroups && ok; ++gi) {
                    const int y = page_row(kPPG * gi + side);
                    for (int t = 0; t < 3; ++t) {
                        const int m = 3 * gi + t, slot = m % kSlots, k = m / kSlots;
                        // first use of slots 2-4: Q's panels have been moved out to TMEM
                        ok = k > 0       ? wait_bar<true>(bar(B_SLOTEMPTY + slot), (k - 1) & 1, abort, ds)
                             : slot >= 2 ? wait_bar(bar(B_QREADY), 0, abort, ds)
                                         : true;
                        if (!ok) break;
                        // both CTAs' bytes are counted on CTA 0's barrier
                        if (side == 0) bar_arrive_expect_tx(bar(B_SLOTFULL + slot), 2 * kSlotBytes);
                        tma_load_3d_pair(sbase + OFF_RING + slot * kSlotBytes, &k_map,
                                         map_to_rank(bar(B_SLOTFULL + slot), 0), 0, y, kSlotPanels * t);
                        ++issued;
                    }
                }
                // Teardown: the MMAs have consumed the last slots, so every copy has landed and no
                // commit is still on its way here.
                for (int m = (issued > kSlots ? issued - kSlots : 0); m < issued; ++m) {
                    volatile int dummy = 0;
                    wait_bar<true>(bar(B_SLOTEMPTY + m % kSlots), (m / kSlots) & 1, *abort ? &dummy : abort, ds);
                }
            }
        } else if (warp == 1) {
            if (lane == 0 && npages > 0 && side == 1) {
                // tell the issuing CTA that this CTA's half of Q is in place
                wait_bar(bar(B_QREADY), 0, abort, ds);
                tc_fence_after();
                tc_fence_before();
                bar_arrive_remote(bar(B_QPEER), 0);
            }
            if (npages > 0 && side == 0) {
                // The whole warp runs the loop and one elected lane issues: descriptors and addresses
                // then live in uniform registers. Issued from a lane-0 branch, an MMA took 140 cycles
                // instead of the 64 that the tensor core needs.
                const bool leader = elect_one();
                bool ok = warp_wait(bar(B_QREADY), 0, abort, ds) && warp_wait<true>(bar(B_QPEER), 0, abort, ds);
                if (ok) tc_fence_after();
                const uint64_t rope0 = smem_desc_sw128(sbase + OFF_QROPE, 16, 1024);
                int slot = 0, phase = 0;
                for (int gi = 0; gi < ngroups && ok; ++gi) {
                    const int buf = gi & 1, use = gi >> 1;
                    if (use > 0) {  // both CTAs' softmax warps have read the buffer's previous S
                        if (!(ok = warp_wait<true>(bar(B_SEMPTY + buf), (use - 1) & 1, abort, ds))) break;
                        tc_fence_after();
                    }
                    const uint32_t d = tmem + kSCol + 128u * buf;
#pragma unroll
                    for (int t = 0; t < 3; ++t) {  // unrolled: every TMEM address and flag an immediate offset
                        if (!(ok = warp_wait<true>(bar(B_SLOTFULL + slot), phase, abort, ds))) break;
                        const uint64_t bd0 = smem_desc_sw128(sbase + OFF_RING + slot * kSlotBytes, 16, 1024);
#pragma unroll
                        for (int q = 0; q < kSlotPanels; ++q) {
                            const int pn = kSlotPanels * t + q;
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint64_t bd = bd0 + (uint64_t)((q * kPageBox + 32 * j) >> 4);
                                if (leader) {
                                    if (pn < 8)
                                        mma_pair_ts(d, tmem + 8u * (4 * pn + j), bd, kIdescQK, (pn | j) ? 1u : 0u);
                                    else
                                        mma_pair_ss(d, rope0 + (uint64_t)(2 * j), bd, kIdescQK, 1u);
                                }
                            }
                        }
                        if (leader) mma_pair_commit(bar(B_SLOTEMPTY + slot), 0x3);
                        if (++slot == kSlots) {
                            slot = 0;
                            phase ^= 1;
                        }
                    }
                    if (ok && leader) mma_pair_commit(bar(B_SFULL + buf), 0x3);
                }
            }
        } else if (warp == 18) {
            // ------------------------- P copies -------------------------
            // One thread sends each staged page, so that the softmax neither waits for the output
            // CTA's buffer nor for the issue.
            if (lane == 0) {
                const uint32_t pbuf_remote = map_to_rank(sbase + OFF_PB, 2u + (uint32_t)side);
                const uint32_t pfull_remote = map_to_rank(bar(B_PFULL), 2u + (uint32_t)side);
                int sent = 0;
                for (int page = 0; page < npages; ++page) {
                    const int sbi = page & 3, pb = page % kPBufs, up = page / kPBufs;
                    if (!wait_bar(bar(B_STAGEFULL + sbi), (page >> 2) & 1, abort, ds)) break;
                    if (up > 0 && !wait_bar<true>(bar(B_PEMPTY + pb), (up - 1) & 1, abort, ds)) break;
                    if (*abort) break;
                    ++sent;
                    bulk_copy_to_peer(pbuf_remote + pb * kPBufStride, sbase + OFF_STAGE + sbi * kPBufStride, kPMsgBytes,
                                      pfull_remote + 8u * pb);
                }
                // The output CTA may now wait for its last page: the page kPBufs earlier is done, so
                // a wait by parity cannot take that page's phase for the last one's. (The softmax
                // is past its last page before that, and must not give this arrival.)
                bar_arrive_remote(bar(B_STATS), 2u + (uint32_t)side);
                // nothing may still be on its way to this CTA when it exits: the last multicast
                // commits of the output pair
                for (int pg = (sent > kPBufs ? sent - kPBufs : 0); pg < sent; ++pg) {
                    volatile int dummy = 0;
                    wait_bar<true>(bar(B_PEMPTY + pg % kPBufs), (pg / kPBufs) & 1, *abort ? &dummy : abort, ds);
                }
            }
        } else {
            // ------------------------- softmax warps (512 threads) -------------------------
            // Quarter `quarter` of the warps owns 32 columns of each group's S: half of page `pg2`.
            const int quarter = (warp - 2) >> 2, pg2 = quarter >> 1, sub = quarter & 1;
            const int row = 32 * (warp & 3) + lane;
            const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
            float* mx = reinterpret_cast<float*>(smem + OFF_MX);
            // Whether the row sees all of this unit's tokens (rows past the batch: never stored). If not it
            // takes none of them here, and the decode of its own tokens starts with this range: a weight
            // of 0 would not keep what its unseen tokens hold out of the sum, should that be NaN.
            bool sees = true;
            const int64_t flat = (int64_t)rows0 + row;
            if (flat < p.flat_rows) {
                const int r = (int)(flat / p.H), b = r / p.Sq, t = r % p.Sq;
                const int seq = min(max(p.seq_lens[b], 0), p.max_seq_len);
                sees = seq - (p.Sq - 1 - t) >= (page0 + npages) * kPage;
            }
            const bool all_see = __all_sync(0xffffffffu, sees);
            if (npages > 0) {
                // Q latent dims: this quarter moves panels 2 quarter and 2 quarter + 1 into TMEM
                const bool okq = warp_wait(bar(B_QFULL), 0, abort, ds);
#pragma unroll 1
                for (int pn = 2 * quarter; pn < 2 * quarter + 2; ++pn) {
                    uint32_t v[32];
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        uint4 x = make_uint4(0, 0, 0, 0);
                        if (okq)
                            x = *reinterpret_cast<const uint4*>(smem + q_panel_off(pn) + row * 128 +
                                                                ((c ^ (row & 7)) << 4));
                        v[4 * c] = x.x;
                        v[4 * c + 1] = x.y;
                        v[4 * c + 2] = x.z;
                        v[4 * c + 3] = x.w;
                    }
                    tmem_st32(tmem + lane_base + 32u * pn, v);
                }
                tmem_wait_st();
                tc_fence_before();
                bar_arrive(bar(B_QREADY));
            }
            const float sl2 = p.scale * 1.4426950408889634f;  // exp2 domain
            float m_run = -CUDART_INF_F, l_run = 0.f;          // each quarter keeps its own sum
            const uint32_t out_rank = 2u + (uint32_t)side;
            for (int gi = 0; gi < ngroups; ++gi) {
                // No early exit from this loop: all 512 threads must pass the same named barriers
                // (which cannot time out); after an abort the waits return at once.
                const int page = kPPG * gi + pg2, buf = gi & 1;
                size_t sc = 0;               // the quarter's first token of the page, in float4 units
                float4 ks[kScaled ? 8 : 1];  // k_scale of its 32 tokens
                if constexpr (kScaled) {  // plain loads: the widening kernel wrote them while this one began
                    sc = ((size_t)(page0 + min(page, npages - 1)) * kPage + 32 * sub) / 4;
                    const float4* src = reinterpret_cast<const float4*>(p.k_scales) + sc;
#pragma unroll
                    for (int j = 0; j < 8; ++j) ks[j] = src[j];
                }
                const bool okS = warp_wait<true>(bar(B_SFULL + buf), (gi >> 1) & 1, abort, ds);
                uint32_t s[32];
                if (okS) {
                    tc_fence_after();
                    tmem_ld32(tmem + lane_base + kSCol + 128u * buf + 32u * quarter, s);
                    tmem_wait_ld();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) bar_arrive_remote_relaxed(bar(B_SEMPTY + buf), 0);
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) s[j] = __float_as_uint(-CUDART_INF_F);
                }
                auto pair = [&](int j) { return make_float2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1])); };
                float4 vs[kScaled ? 8 : 1];  // v_scale of this quarter's 32 tokens, on their way early
                if constexpr (kScaled) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float2 x = mul2(pair(j), j & 1 ? make_float2(ks[j >> 1].z, ks[j >> 1].w)
                                                             : make_float2(ks[j >> 1].x, ks[j >> 1].y));
                        s[2 * j] = __float_as_uint(x.x);
                        s[2 * j + 1] = __float_as_uint(x.y);
                    }
                    const float4* src = reinterpret_cast<const float4*>(p.v_scales) + sc;
#pragma unroll
                    for (int j = 0; j < 8; ++j) vs[j] = src[j];
                }
                // No row of the warp sees these tokens (an empty slot's heads): no weights to compute.
                // Masked like any other, three empty slots of 64 made their clusters the last to end, by 8 us
                // of 63. (Not with scales: it spills there, 265 against 249 us a call.)
                bool dead = false;
                if (page >= npages || !all_see) {
                    const bool none = page >= npages || !sees;
                    if constexpr (!kScaled) dead = __all_sync(0xffffffffu, none);
                    if (!dead) {
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (none) s[j] = __float_as_uint(-CUDART_INF_F);
                    }
                }
                float lm = -CUDART_INF_F;
                if (!dead) {
                    float lm4[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
                    for (int j = 0; j < 16; ++j) lm4[j & 3] = max3(lm4[j & 3], pair(j).x, pair(j).y);
                    lm = max3(lm4[0], lm4[1], fmaxf(lm4[2], lm4[3]));
                }
                // Does any row's part pass the threshold? The barrier also keeps the next exchange's
                // writes of mx behind this one's reads.
                const bool any = named_bar_or(kBarOr, kSoftThreads, lm * sl2 > m_run + kRescaleThreshold);
                float alpha = 1.f;
                if (any) {
                    mx[quarter * 128 + row] = lm;
                    named_bar(kBarMax, kSoftThreads);
                    const float mt = fmaxf(fmaxf(mx[row], mx[128 + row]), fmaxf(mx[256 + row], mx[384 + row])) * sl2;
                    if (mt > m_run + kRescaleThreshold) {
                        alpha = fast_exp2(m_run - mt);  // 0 while m_run = -inf
                        m_run = mt;
                    }
                    l_run *= alpha;
                }
                const float mref = m_run == -CUDART_INF_F ? 0.f : m_run;  // nothing seen yet: weights 0
                uint32_t pk[16];
                if (dead) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) pk[j] = 0u;
                } else {
                    float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float2 a = fma2(pair(j), make_float2(sl2, sl2), make_float2(-mref, -mref));
                        a = make_float2(fast_exp2(a.x), fast_exp2(a.y));
                        l2[j & 1] = add2(l2[j & 1], a);
                        if constexpr (kScaled)
                            a = mul2(a, j & 1 ? make_float2(vs[j >> 1].z, vs[j >> 1].w)
                                              : make_float2(vs[j >> 1].x, vs[j >> 1].y));
                        pk[j] = pack_bf16x2(a.x, a.y);
                    }
                    l2[0] = add2(l2[0], l2[1]);
                    l_run += l2[0].x + l2[0].y;
                }
                // the page's staging buffers take turns: this one is free once the copy of two groups
                // ago has landed
                const int sbi = 2 * (gi & 1) + pg2;
                uint8_t* stage = smem + OFF_STAGE + sbi * kPBufStride;
                if (page < npages) {  // a page past the end sends nothing
                    if (gi > 1) warp_wait<true>(bar(B_STAGEFREE + sbi), ((gi >> 1) - 1) & 1, abort, ds);
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        *reinterpret_cast<uint4*>(stage + row * 128 + (((4 * sub + c) ^ (row & 7)) << 4)) =
                            make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
                    // the group's first page carries the rescale that O needs before it
                    if (sub == 0) reinterpret_cast<float*>(stage + kPBytes)[row] = alpha;
                    if (sub == 0 && row == 0)
                        *reinterpret_cast<uint32_t*>(stage + kPBytes + 512) = (pg2 == 0 && any && gi > 0) ? 1u : 0u;
                    fence_proxy_async_cta();  // generic writes before the bulk copy reads them
                    __syncwarp();
                    if (lane == 0) bar_arrive(bar(B_STAGEFULL + sbi));
                }
            }
            // combine the quarters' sums, ship the final statistics
            named_bar(kBarMax, kSoftThreads);
            mx[quarter * 128 + row] = l_run;
            named_bar(kBarMax, kSoftThreads);
            if (quarter == 0) {
                l_run = (mx[row] + mx[128 + row]) + (mx[256 + row] + mx[384 + row]);
                st_cluster_u32(map_to_rank(sbase + OFF_STAT_M, out_rank) + 4u * row, __float_as_uint(m_run));
                st_cluster_u32(map_to_rank(sbase + OFF_STAT_L, out_rank) + 4u * row, __float_as_uint(l_run));
                named_bar(kBarQuarter0, 128);
                if (tid == 64) bar_arrive_remote(bar(B_STATS), out_rank);
            }
        }
    } else {
        // ============================== output CTAs ==============================
        if (warp == 0) {
            if (lane == 0 && npages > 0) {
                tma_prefetch_desc(&v_map);
                int issued = 0;
                for (int i = 0; i < npages; ++i) {
                    const int y = page_row(i);
                    const int st = i % kVStages, k = i / kVStages;
                    if (k > 0 && !wait_bar<true>(bar(B_VEMPTY + st), (k - 1) & 1, abort, ds)) break;
                    if (side == 0) bar_arrive_expect_tx(bar(B_VFULL + st), 2 * kVStageBytes);
                    const uint32_t full = map_to_rank(bar(B_VFULL + st), 2);
                    const uint32_t dst = sbase + OFF_V + st * kVStageBytes;
                    tma_load_3d_pair(dst, &v_map, full, 0, y, 2 * side);
                    tma_load_3d_pair(dst + 2 * kPageBox, &v_map, full, 0, y, 4 + 2 * side);
                    issued = i + 1;
                }
                for (int i = (issued > kVStages ? issued - kVStages : 0); i < issued; ++i) {  // teardown, as above
                    volatile int dummy = 0;
                    wait_bar<true>(bar(B_VEMPTY + i % kVStages), (i / kVStages) & 1, *abort ? &dummy : abort, ds);
                }
            }
        } else if (warp == 1) {
            if (side == 0) {
                const bool leader = elect_one();  // as for the scores
                bool ok = true;
                for (int i = 0; i < npages && ok; ++i) {
                    const int pb = i % kPBufs, st = i % kVStages;
                    if (!(ok = warp_wait<true>(bar(B_READY + pb), (i / kPBufs) & 1, abort, ds))) break;
                    if (!(ok = warp_wait<true>(bar(B_VFULL + st), (i / kVStages) & 1, abort, ds))) break;
                    tc_fence_after();  // after a rescale by the helper warps' tcgen05.st
                    const uint64_t ad0 = smem_desc_sw128(sbase + OFF_PB + pb * kPBufStride, 16, 1024);
                    const uint64_t bd0 = smem_desc_sw128(sbase + OFF_V + st * kVStageBytes, kPageBox, 1024);
#pragma unroll
                    for (int kk = 0; kk < kPage / 16; ++kk)
#pragma unroll
                        for (int nh = 0; nh < 2; ++nh)
                            if (leader)
                                mma_pair_ss(tmem + 256u * nh, ad0 + (uint64_t)((kk * 32) >> 4),
                                            bd0 + (uint64_t)((nh * 2 * kPageBox + kk * 2048) >> 4), kIdescPV,
                                            kk > 0 ? 1u : (i > 0 ? 1u : 0u));
                    if (leader) {
                        mma_pair_commit(bar(B_VEMPTY + st), 0xC);
                        mma_pair_commit(bar(B_PEMPTY + pb), 0xF);
                    }
                }
            }
            // teardown: the last commits have landed in this CTA (in CTA 3, which does not follow the
            // pages here, the epilogue's wait for the last page stands for it)
            for (int pg = side == 1 ? npages : (npages > kPBufs ? npages - kPBufs : 0); pg < npages; ++pg) {
                volatile int dummy = 0;
                wait_bar<true>(bar(B_PEMPTY + pg % kPBufs), (pg / kPBufs) & 1, *abort ? &dummy : abort, ds);
            }
        } else if (warp < 18) {
            // ------------- helper warps 2-5: P arrival, rescale; warps 2-17: the epilogue -------------
            const int row = 32 * (warp & 3) + lane;
            const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
            const int ctid = tid - 64;  // 0..511; 0..127 are the helper warps
            const int eset = (warp - 2) >> 2;
            int pages_ready = warp >= 6 ? npages : 0;
            for (int i = 0; i < npages && warp < 6; ++i) {
                const int pb = i % kPBufs;
                if (!warp_wait<true>(bar(B_PFULL + pb), (i / kPBufs) & 1, abort, ds)) break;
                if (ctid == 0) {
                    bar_arrive_expect_tx(bar(B_PFULL + pb), kPMsgBytes);           // re-arm for the next message
                    bar_arrive_remote_relaxed(bar(B_STAGEFREE + (i & 3)), (uint32_t)side);  // the sender's staging buffer
                }
                const uint8_t* pmsg = smem + OFF_PB + pb * kPBufStride;
                const bool fix = i > 0 && *reinterpret_cast<const volatile uint32_t*>(pmsg + kPBytes + 512) != 0;
                if (fix) {  // O must hold every earlier PV product before it is rescaled
                    if (!warp_wait<true>(bar(B_PEMPTY + (i - 1) % kPBufs), ((i - 1) / kPBufs) & 1, abort, ds)) break;
                    tc_fence_after();
                    const float a = reinterpret_cast<const volatile float*>(pmsg + kPBytes)[row];
#pragma unroll 1
                    for (int c = 0; c < kL / 32; ++c) {
                        uint32_t v[32];
                        tmem_ld32(tmem + lane_base + 32u * c, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * a);
                        tmem_st32(tmem + lane_base + 32u * c, v);
                    }
                    tmem_wait_st();
                }
                tc_fence_before();
                // P came through the async proxy into this CTA, and O may have been rescaled here; both
                // are read by MMAs that CTA 2 issues. CTA 2's warps tell its MMA warp themselves, CTA 3's
                // through the relay below.
                fence_proxy_async_cta();
                dec::warp_arrive(bar((side == 0 ? B_READY : B_PEER) + pb), lane);
                pages_ready = i + 1;
            }
            // CTA 3's pages are announced to CTA 2 by an arrival that releases at cluster scope, since it
            // publishes the helpers' writes. That takes most of a microsecond, so warps that have nothing
            // else to do before the epilogue take the pages in turn; the P buffers cover its latency (64 rows
            // of 128 heads over 4096 + 512 tokens 86 us, 128 rows of 16 heads over 32768 + 1000 120).
            if (side == 1 && warp >= 6 && warp < 6 + kRelayWarps && lane == 0) {
                for (int i = warp - 6; i < npages; i += kRelayWarps) {
                    const int pb = i % kPBufs;
                    if (!wait_bar(bar(B_PEER + pb), (i / kPBufs) & 1, abort, ds)) break;
                    tc_fence_after();
                    tc_fence_before();
                    bar_arrive_remote(bar(B_READY + pb), 2);
                }
            }
            __syncwarp();
            const bool has_o = npages > 0 && pages_ready == npages && !*abort;
            wait_bar<true>(bar(B_STATS), 0, abort, ds);
            const bool o_ok = has_o && wait_bar<true>(bar(B_PEMPTY + (npages - 1) % kPBufs),
                                                      ((npages - 1) / kPBufs) & 1, abort, ds);
            tc_fence_after();
            const float m = reinterpret_cast<volatile float*>(smem + OFF_STAT_M)[row];
            const float l = reinterpret_cast<volatile float*>(smem + OFF_STAT_L)[row];
            const bool use_o = __all_sync(0xffffffffu, o_ok);
            const bool empty = !use_o || l == 0.f;  // no token has a weight; a NaN sum is a NaN result
            const float inv = empty ? 0.f : 1.f / l;
            const int64_t flat = (int64_t)rows0 + row;
            if (eset == 0 && flat < p.flat_rows)
                p.part_lse[(size_t)split * p.flat_rows + flat] =
                    empty ? -CUDART_INF_F : (m + log2f(l)) * 0.6931471805599453f;
            // O / l leaves through TMA stores over the V ring and the P buffers; rows past the batch
            // are cut off by the tensor map
            store_rows<true, 4, 3, kBarEpi>(smem, sbase, OFF_V, tmem + lane_base, row, eset, (ctid & 127) == 0, true,
                                            empty, inv, &o_map, rows0, split, rows0 < p.flat_rows);
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (warp == 0) tmem_dealloc_pair(tmem, kTmemCols);
    cluster_sync();
}

// ------------------------------------------------------------------------------------------
// FP8 prefix -> bf16 rows (exact) and scales, once per call. One warp per token: lanes take
// 8-byte chunks of the 576 codes.
// ------------------------------------------------------------------------------------------
__global__ void __launch_bounds__(256) prefix_widen_kernel(PrefixArgs p, const uint8_t* cache, uint16_t* x,
                                                           float* k_scales, float* v_scales) {
    griddep_wait();
    griddep_launch_dependents();
    const int token = (int)blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (token >= p.prefix_pages * kPage) return;
    const int32_t blk = p.block_table[token / kPage];
    const bool bad = blk < 0 || (int64_t)blk >= p.num_blocks;
    if (bad && lane == 0 && p.dev_status) atomicOr(p.dev_status, MLA_DEV_BAD_BLOCK_ID);
    const uint8_t* src = cache + ((size_t)(bad ? 0 : blk) * kPage + token % kPage) * kFp8RowBytes;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const int c = lane + 32 * i;
        if (c >= kD / 8) continue;
        uint2 v = make_uint2(0u, 0u);
        if (!bad) v = *reinterpret_cast<const uint2*>(src + 8 * c);
        uint4 w;  // as the decode kernels read the codes
        e4m3x4_to_bf16x4(v.x, w.x, w.y);
        e4m3x4_to_bf16x4(v.y, w.z, w.w);
        *reinterpret_cast<uint4*>(x + (size_t)token * kD + 8 * c) = w;
    }
    if (lane == 0) {
        const float2 sc = bad ? make_float2(0.f, 0.f) : *reinterpret_cast<const float2*>(src + kD);
        k_scales[token] = sc.x;
        v_scales[token] = sc.y;
    }
}

int g_attr_done[2][64] = {};
int g_clusters[64] = {};

cudaError_t set_attr(int dev, bool scaled) {
    if (dev < 64 && g_attr_done[scaled][dev]) return cudaSuccess;
    const cudaError_t e =
        scaled ? cudaFuncSetAttribute(decode_prefix_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes)
               : cudaFuncSetAttribute(decode_prefix_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e == cudaSuccess && dev < 64) g_attr_done[scaled][dev] = 1;
    return e;
}

}  // namespace

int prefix_clusters() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return -1;
    if (dev < 64 && g_clusters[dev] > 0) return g_clusters[dev];
    if (set_attr(dev, false) != cudaSuccess) return -1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(4);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 4;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, decode_prefix_kernel<false>, &cfg) != cudaSuccess || n < 1) return -1;
    if (dev < 64) g_clusters[dev] = n;
    return n;
}

// The split of a prefix of `pages` pages over `flat_rows` rows: S ranges of an even number of pages.
void prefix_split(int64_t flat_rows, int pages, int clusters, int* splits, int* pages_per_split) {
    // Time of S splits: waves of clusters, each a range of pages and a fixed part, and the partial
    // states written and read back. In page-times of one cluster (about 0.9 us).
    constexpr double kUnitPages = 14.0;
    const int64_t tiles = (flat_rows + kTileRows - 1) / kTileRows;
    const double partial = (double)flat_rows * (kL + 1) * 8.0 / 5.0e6 / 0.9;  // bytes / (bytes per page-time)
    double best = 1e300;
    *splits = 1;
    *pages_per_split = (pages + 1) / 2 * 2;
    for (int S = 1; S <= (pages + 1) / 2 && S <= 3 * clusters; ++S) {  // more never fill waves better
        const int per = ((pages + S - 1) / S + 1) / 2 * 2;
        const int used = (pages + per - 1) / per;  // ranges that hold pages
        if (used < S && S > 1) continue;
        const int64_t waves = (tiles * S + clusters - 1) / clusters;
        const double t = (double)waves * (per + kUnitPages) + S * partial;
        if (t < best * 0.999) {
            best = t;
            *splits = S;
            *pages_per_split = per;
        }
    }
}

cudaError_t launch_prefix_widen(const PrefixArgs& a, const uint8_t* cache, uint16_t* widened, float* scales,
                                cudaStream_t s) {
    return launch_pdl(prefix_widen_kernel, dim3((unsigned)(a.prefix_pages * kPage / 8)), dim3(256), 0, s, a, cache,
                      widened, scales, scales + (size_t)a.prefix_pages * kPage);
}

cudaError_t launch_decode_prefix(const PrefixArgs& in, const uint8_t* cache, const uint16_t* widened,
                                 const float* scales, cudaStream_t s) {
    PrefixArgs a = in;
    const bool fp8 = widened != nullptr;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = set_attr(dev, fp8);
    if (e != cudaSuccess) return e;
    const void* base = cache;
    uint64_t rows = (uint64_t)a.num_blocks * kPage;
    if (fp8) {
        a.block_table = nullptr;
        a.k_scales = scales;
        a.v_scales = scales + (size_t)a.prefix_pages * kPage;
        base = widened;
        rows = (uint64_t)a.prefix_pages * kPage;
    }
    a.key_rows = (int)rows;
    CUtensorMap k_map, v_map, q_map, o_map;
    memset(&k_map, 0, sizeof k_map);
    memset(&v_map, 0, sizeof v_map);
    memset(&q_map, 0, sizeof q_map);
    memset(&o_map, 0, sizeof o_map);
    {
        // the rows as [panel of 64 dims][row][64]: one box is several panels of a page
        const uint64_t dims[3] = {64, rows, (uint64_t)(kD / 64)};
        const uint64_t strides[2] = {(uint64_t)kBf16RowBytes, 128};
        const uint32_t kbox[3] = {64, (uint32_t)kPage, (uint32_t)kSlotPanels};
        e = encode_tmap(&k_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, kbox, true);
        if (e != cudaSuccess) return e;
        const uint32_t vbox[3] = {64, (uint32_t)kPage, 2};
        e = encode_tmap(&v_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, vbox, true);
        if (e != cudaSuccess) return e;
    }
    {
        const uint64_t dims[2] = {(uint64_t)kD, (uint64_t)a.flat_rows};
        const uint64_t strides[1] = {(uint64_t)kD * 2};
        const uint32_t box[2] = {64, 128};
        e = encode_tmap(&q_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.q, dims, strides, box, true);
        if (e != cudaSuccess) return e;
    }
    {
        const uint64_t dims[3] = {(uint64_t)kL, (uint64_t)a.flat_rows, (uint64_t)a.splits};
        const uint64_t strides[2] = {(uint64_t)kL * 4, (uint64_t)a.flat_rows * kL * 4};
        const uint32_t box[3] = {32, 128, 1};
        e = encode_tmap(&o_map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, a.part_o, dims, strides, box, true);
        if (e != cudaSuccess) return e;
    }
    const int64_t tiles = ((int64_t)a.flat_rows + kTileRows - 1) / kTileRows;
    const dim3 grid((unsigned)(4 * tiles * a.splits));
    return fp8 ? launch_pdl(decode_prefix_kernel<true>, grid, dim3(kThreads), kSmemBytes, s, k_map, v_map, q_map,
                            o_map, a)
               : launch_pdl(decode_prefix_kernel<false>, grid, dim3(kThreads), kSmemBytes, s, k_map, v_map, q_map,
                            o_map, a);
}

}  // namespace mla
