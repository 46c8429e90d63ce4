// decode_tree_sm103.cu -- mla_decode_tree of more than 32 (draft, head) pairs a request, or 128 over an FP8 cache:
// all pairs of a request against its own pages, 256 at a time.
//
// For a flat row f = (draft t, head) of request b and its pages, or a part of them:  S = scale * q[b, f] K^T over the
// tokens that draft t sees,  P = softmax(S),  o[f] = P V,  written to the outputs or, of a part, as a partial state
// (o, lse) that the merge below combines.
//
// What bounds it: the drafts of a request read the same keys, so that this is the matrix product of the
// prefix kernel (decode_prefix_sm103.cu, whose pipeline this one follows): two SMs work as a pair on 256 rows
// (tcgen05 cta_group::2, M = 256) and each loads half of the keys, 1.1 us of MMAs for a group of two pages. One
// cluster of four CTAs:
//   CTAs 0, 1 ("scores")  Q: 512 latent dims in tensor memory, 64 rope dims in shared memory; S of a group of
//       128 tokens into one of two buffers; sixteen softmax warps with a running maximum that moves only when it
//       grows by more than 2^8; P (bf16) staged and sent to the output CTA of the same rows, a page a copy.
//   CTAs 2, 3 ("output")  hold the 256 x 512 fp32 accumulators (all of both SMs' tensor memory) and add P V;
//       helper warps rescale O when a group's maximum moved. Epilogue: O / l by TMA stores.
//
// Clusters stay for all of their units (request, tile of 256 rows). While the output CTAs
// finish one, the scores CTAs load the next one's queries, score and weigh its first two groups. Barriers
// are used on by group numbers that run through all units; a unit's odd last page is followed by one of zeros,
// so that a group is always two pages.
//
// Balance. Many units go to the clusters whole, longest request first, back and forth: no counter, and (simulated)
// within 2% of giving each next unit to the cluster with the least work. A few units are cut (kCut): every cluster takes an
// equal share of all requests' groups, wherever it begins and ends. Which of the two is the host's guess from the
// longest length possible (tree_shares); the cuts are made on the device from the lengths. Against ranges of a fixed
// number of pages, which the host chose before: 20 requests x 256 rows over 8000 to 16,000 tokens 134 -> 101 us, 8 x 1024
// over up to 32,768 325 -> 272, 5 x 320 over up to 100,000 307 -> 236, 1 x 1024 over 131,072 the same.
//
// Measured: 16 requests x 32 drafts x 128 heads over up to 8192 tokens 550 us, 1.59 PFLOP/s (FP8 551 with the
// widening, 1.73), 29 x 8 over up to 4096 147 us, 1.38; 64 x 7 drafts of 16 heads over up
// to 8192 tokens 137 to 145 us: less than half of the rows are in use there. A group takes 1.28 us, its 2304 cycles
// of scores MMAs at the clock that the power leaves; a unit's change 6 us, the first scores 9 after the start.
// What it took, on the 32 x 8 drafts: one launch a unit 174 us; clusters that stay, longest first 154; first keys
// beside Q, lengths in shared memory 152; an arrival without a release, no 64-bit divisions 148; a later unit's Q loaded
// when the last scores are done, not the last weights, 146 (FP8, 16 x 32: 562 -> 552). FP8 scales from
// shared memory instead of global, 16 x 32 drafts: 614 -> 564 us.
//
// What hides drafts: the pages that hold any (two at most) are masked token by token. Their V rows are looked
// over when they land, since a hidden token's NaN would pass a weight of 0 (decode_common.cuh).
//
// Rounding: as the prefix kernel: P to bf16, the sums l of the unrounded fp32 weights. FP8 cache: the
// requests' rows are widened once per call to bf16 (exactly), and k_scale multiplies the fp32 scores, v_scale the
// weights before their rounding.
//
// All waits are bounded (see sm103_ptx.cuh).
#include <cuda.h>
#include <math_constants.h>

#include <algorithm>
#include <cmath>
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

// scores: warp 0 TMA, 1 MMA, 2-17 softmax, 18 P copies
// output: warp 0 TMA, 1 MMA, 2-5 helpers, 6-9 CTA 3's relay, 10-17 drafted pages' V, 2-17 epilogue, 18 L2 prefetch
constexpr int kThreads = 608;
constexpr int kSoftThreads = 512;
constexpr int kTileRows = 256;
constexpr int kPPG = 2;                      // pages per group, one per scores CTA
constexpr int kPageBox = kPage * 128;        // one page's rows of one 64-dim panel (8 KB)
constexpr int kSlotPanels = 3;
constexpr int kSlotBytes = kSlotPanels * kPageBox;  // 24 KB
constexpr int kSlots = 5;                    // K ring of a scores CTA
constexpr int kQPanelBytes = 128 * 128;      // 128 rows x 64 dims of Q (16 KB), loaded as two halves of 64 rows
constexpr int kQHalfBytes = kQPanelBytes / 2;
constexpr int kPBufs = 5;                    // P buffers of an output CTA (one page each)
constexpr int kVStages = 4;                  // V ring of an output CTA: a page's 4 panels each
constexpr int kVStageBytes = 4 * kPageBox;   // 32 KB
constexpr int kPBytes = 128 * 128;           // P page: 128 rows x 64 tokens bf16
constexpr int kPMsgBytes = (kPBytes + 512 + 4 + 15) / 16 * 16;  // P + alpha[128] + flag
constexpr int kPBufStride = 17 * 1024;
constexpr int kAuxWarp0 = 10, kAuxWarps = 8;
constexpr int kRelayWarps = 4;               // of CTA 3, from warp 6 on
constexpr int kAhead = 10, kInRings = 6;     // pages between the helpers' progress and the one prefetched; in the rings
constexpr int kCtrlBytes = 7168;
constexpr int kUnitGroups = 5;               // what a unit's start and end cost (7 us), in groups
constexpr int kEdgeGroups = 3;               // no part of a unit is shorter, unless the shares are short
// scores CTA
constexpr int OFF_QROPE = kCtrlBytes;
constexpr int OFF_RING = OFF_QROPE + kQPanelBytes;
constexpr int kStages = 4;                   // P staging buffers: each of a group's pages has two
constexpr int OFF_STAGE = OFF_RING + kSlots * kSlotBytes;
constexpr int OFF_QX = OFF_STAGE + kStages * kPBufStride;  // one panel of Q
constexpr int kSmem0 = OFF_QX + kQPanelBytes;
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
static_assert(8 * dec::kTileBytes <= kVStages * kVStageBytes, "epilogue tiles");
// Q's sixteen latent half panels land where nothing else is. The first unit's: in the four staging buffers, a place of
// their own and the two ring slots that its keys need last, so that its first group loads beside Q. A later unit's, whose
// load begins when the last scores of the one before are done: in the two staging buffers that are not those of that
// group, their own place and all ring slots but the first, so that a third of the first group loads beside it.
static_assert(kSlots == 5 && kStages == 4 && 3 * kQHalfBytes == kSlotBytes && kPBufStride >= kQPanelBytes, "Q panel homes");
static_assert(OFF_QX % 1024 == 0, "Q panel homes");
__device__ __forceinline__ uint32_t q_half_off(int h, uint32_t g0) {  // g0: groups of the units before
    const int staged = g0 == 0 ? 8 : 4, slot0 = g0 == 0 ? 3 : (int)(3 * g0 + 1) % kSlots, stage0 = g0 == 0 ? 0 : 2 * (int)(g0 & 1);
    if (h < staged) return OFF_STAGE + (stage0 + (h >> 1)) * kPBufStride + (h & 1) * kQHalfBytes;
    h -= staged;
    if (h < 2) return OFF_QX + h * kQHalfBytes;
    h -= 2;
    return OFF_RING + (slot0 + h / 3) % kSlots * kSlotBytes + h % 3 * kQHalfBytes;
}

// Barrier slots, one layout for all four CTAs (multicast commits land at the same offset in each).
enum : int {
    B_SLOTFULL = 0,                     // [kSlots] CTA 0: slot landed in both scores CTAs (TMA tx)
    B_SLOTEMPTY = B_SLOTFULL + kSlots,  // [kSlots] CTAs 0, 1: slot's QK MMAs completed
    B_SFULL = B_SLOTEMPTY + kSlots,     // [2] CTAs 0, 1: S buffer ready
    B_SEMPTY = B_SFULL + 2,             // [2] CTA 0: S buffer read by the 32 softmax warps of the pair
    B_QFULL = B_SEMPTY + 2,             // CTAs 0, 1: the unit's Q landed in shared memory
    B_QREADY,                           // CTAs 0, 1: its latent dims moved to TMEM (16 warps)
    B_QPEER,                            // CTA 0: CTA 1's Q moved
    B_STAGEFULL,                        // [4] CTAs 0, 1: staging buffer written by the page's 8 softmax warps
    B_STAGEFREE = B_STAGEFULL + kStages,  // [4] CTAs 0, 1: staging buffer's copy has landed
    B_PEMPTY = B_STAGEFREE + kStages,         // [kPBufs] all: PV MMAs of the page in P buffer b completed
    B_VFULL = B_PEMPTY + kPBufs,        // [kVStages] CTA 2: V stage landed in both output CTAs
    B_VEMPTY = B_VFULL + kVStages,      // [kVStages] CTAs 2, 3: V stage consumed
    B_PFULL = B_VEMPTY + kVStages,      // [kPBufs] CTAs 2, 3: P message landed
    B_READY = B_PFULL + kPBufs,         // [kPBufs] CTA 2: its 4 helper warps and CTA 3 are done with the page
    B_PEER = B_READY + kPBufs,          // [kPBufs] CTA 3: its 4 helper warps are done with the page
    B_STATS = B_PEER + kPBufs,          // CTAs 2, 3: the unit's row statistics written, last P copy issued
    B_DONE,                             // all: the output CTA of the same rows (or this one) has stored the unit
    B_VLAND,                            // [2] CTAs 2, 3: this CTA's half of a drafted page's V landed
    B_VCLEAN = B_VLAND + 2,             // [2] CTA 2: both halves looked over (16 warps)
    B_COUNT = B_VCLEAN + 2
};
static_assert(8 * B_COUNT <= 512, "barrier slots");
constexpr int OFF_TMEM = 512;
constexpr int OFF_ABORT = 516;
constexpr int OFF_PROG = 520;     // CTA 2: pages of all units that its helper warps have seen (paces the prefetch)
constexpr int OFF_MX = 1024;      // scores: f32 [4][128] exchange between the column quarters
constexpr int OFF_STAT_M = 2048;  // output: f32 [128] final running max (log2 units)
constexpr int OFF_STAT_L = 2560;  // output: f32 [128] row sum
// Requests whose lengths are kept and, for more units than clusters, sorted: what the control block has room for. More are
// taken in the caller's order and their lengths read from global memory: 7 to 8% slower (2 x 64 pairs over up to 2000 tokens,
// us per million tokens: 240 requests 414, 241 446).
constexpr int kMaxSorted = 240;
constexpr int OFF_ORDER = 544;    // u16 [kMaxSorted] requests, longest first; or the cuts:
constexpr int OFF_CUTS = OFF_ORDER;          // Place [2] where the cluster's part begins and ends
constexpr int OFF_BEFORE = OFF_CUTS + 32;    // u32 [kTreeMaxCut] weights of the requests before
constexpr int OFF_LENS = OFF_STAT_L + 512;  // s32 [kMaxSorted] tokens of each request
constexpr int OFF_SCALES = 4096;  // scores, FP8: f32 [3][2][128] k_scales and v_scales of three groups in turn
constexpr int kScaleBytes = 2 * kPPG * kPage * 4;
static_assert(OFF_ORDER + 2 * kMaxSorted <= OFF_MX && OFF_BEFORE + 4 * kTreeMaxCut <= OFF_MX && kTreeMaxCut <= kMaxSorted &&
                  OFF_LENS + 4 * kMaxSorted <= OFF_SCALES &&
                  OFF_SCALES + 3 * kScaleBytes <= kCtrlBytes,
              "control block");

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSCol = 256;  // scores: Q latent in columns [0, 256), S buffers at 256 and 384
constexpr uint32_t kIdescQK = idesc_bf16_f32(256, 128, false, false);
constexpr uint32_t kIdescPV = idesc_bf16_f32(256, 256, false, true);
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr uint32_t kBarMax = 1, kBarOr = 2, kBarQuarter0 = 3;
constexpr uint32_t kBarEpi = 1;  // [4] the epilogue's warp sets (output CTAs)
constexpr uint32_t kBarStored = 5;

// After an abort: copies in flight, at most a few microseconds' worth, land before the CTA can exit.
__device__ __forceinline__ void settle() {
    for (int i = 0; i < 1000; ++i) __nanosleep(1000);
}

// A place in the row of all groups: group `group` of entry `entry` (request entry % B of round entry / B).
struct Place {
    int entry, group;
};
__device__ __forceinline__ bool before(const Place& a, const Place& b) {
    return a.entry < b.entry || (a.entry == b.entry && a.group < b.group);
}

// One unit of a cluster's list, or a part of one.
struct Unit {
    int entry, req, tile;  // entry: of the row, where units are cut
    int slab;              // the request, of a part its partial state
    bool part;
    int page0, npages, ngroups;
    int drafts0;           // the request's tokens before its drafts (below 0: the first are not there)
    int drafted;           // the first of the unit's pages that holds drafts (npages: none)
};

// The cuts. The requests stand in a row, each as long as its groups and kUnitGroups for a unit's start and
// end; the row is cut into equal shares. `lanes` clusters side by side go through one share for as many tiles (and find
// its pages in L2); with fewer lanes than tiles the row has a round of all requests for each set of them. A cut that falls
// into a unit's fixed part, or leaves a few groups before or behind it, moves to the unit's edge.
__device__ __forceinline__ uint32_t unit_groups(int len) {
    return ((uint32_t)((len + kPage - 1) / kPage) + kPPG - 1) / kPPG;
}
__device__ __forceinline__ uint32_t unit_weight(int len) { return len > 0 ? unit_groups(len) + kUnitGroups : 1u; }
__device__ Place cut_of(const TreeArgs& p, const int* lens, const uint32_t* weights, int share) {
    if (share == 0) return Place{0, 0};
    const uint32_t rounds = (uint32_t)(p.tiles / p.lanes), round = weights[p.B - 1] + unit_weight(lens[p.B - 1]);
    if (share == p.shares) return Place{p.B * (int)rounds, 0};
    const uint64_t all = (uint64_t)round * rounds;
    // every share has a start of its own: the first request's is not counted
    const uint64_t free = min(all - 1, (uint64_t)kUnitGroups), rest = all - free;
    uint64_t at = free;
    uint32_t nth;
    if (all < 1u << 26) {  // 64 shares at most
        at += (uint32_t)rest * (uint32_t)share / (uint32_t)p.shares;
        nth = (uint32_t)at / round;
    } else {
        at += rest * (uint32_t)share / (uint32_t)p.shares;
        nth = (uint32_t)(at / round);
    }
    const uint32_t in = (uint32_t)(at - (uint64_t)nth * round);
    const int edge = (int)min((uint32_t)min(rest, (uint64_t)UINT32_MAX) / (4u * (uint32_t)p.shares), (uint32_t)kEdgeGroups);
    int lo = 0, hi = p.B - 1;  // the last request that begins at or before `in`
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (weights[mid] <= in)
            lo = mid;
        else
            hi = mid - 1;
    }
    const int groups = (int)unit_groups(lens[lo]), group = (int)(in - weights[lo]) - kUnitGroups;
    const int entry = (int)nth * p.B + lo;
    return group <= edge ? Place{entry, 0} : groups - group > edge ? Place{entry, group} : Place{entry + 1, 0};
}

// kCut: units are cut (see cut_of). Instances of their own: with both in one, FP8's softmax spilled (562 -> 600 us).
template <bool kScaled, bool kCut>
__global__ void __cluster_dims__(4, 1, 1) __launch_bounds__(kThreads, 1)
    decode_tree_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                       const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap o_map,
                       const __grid_constant__ CUtensorMap part_map, const TreeArgs p) {
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
    volatile int* abort = reinterpret_cast<volatile int*>(smem + OFF_ABORT);
    int32_t* ds = p.dev_status;
    auto bar = [&](int i) -> uint32_t { return sbase + 8u * (uint32_t)i; };
    auto length = [&](int b, bool report = false) -> int {
        const int n = p.seq_lens[b];
        if (report && ds && (n < 0 || n > p.max_seq_len)) atomicOr(ds, MLA_DEV_SEQ_TOO_LONG);
        return min(max(n, 0), p.max_seq_len);
    };

    // Lengths, and the requests in their order (ties by number), every thread placing one. The lengths are read ahead of the
    // wait for the kernels in front, by the rule of the decode kernels: no kernel that writes lengths lets the next one start
    // early (internal.h, launch_pdl). The roles of the cluster's CTAs, each of which reads them for itself, agree by that alone.
    const int clusters = (int)(gridDim.x >> 2), cluster = (int)(blockIdx.x >> 2);
    const bool kept = p.B <= kMaxSorted, sorted = kept && !kCut && p.units > (int64_t)clusters;
    int* lens = reinterpret_cast<int*>(smem + OFF_LENS);
    if (kept && tid < p.B) lens[tid] = length(tid, blockIdx.x == 0);
    if (tid == kThreads - 1) {
        *abort = 0;
        *reinterpret_cast<volatile uint32_t*>(smem + OFF_PROG) = 0;
    }
    if (tid < B_COUNT) {
        const int i = tid;
        uint32_t cnt = 1;
        if (i >= B_SEMPTY && i < B_SEMPTY + 2) cnt = 32;
        if (i == B_QREADY) cnt = kSoftThreads / 32;
        if (i == B_STATS) cnt = 2;
        if (i >= B_STAGEFULL && i < B_STAGEFULL + kStages) cnt = 8;
        if (i >= B_READY && i < B_READY + kPBufs) cnt = 5;
        if (i >= B_PEER && i < B_PEER + kPBufs) cnt = 4;
        if (i >= B_VCLEAN && i < B_VCLEAN + 2) cnt = 2 * kAuxWarps;
        bar_init(bar(i), cnt);
        // P buffers armed for their first message before a scores CTA can send one
        if (!scores && i >= B_PFULL && i < B_PFULL + kPBufs) bar_arrive_expect_tx(bar(i), kPMsgBytes);
        fence_barrier_init();
    }
    if (warp == 0) {
        tmem_alloc_pair(sbase + OFF_TMEM, kTmemCols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (sorted && tid < p.B) {
        const int mine = lens[tid];
        int place = 0;
        for (int b = 0; b < p.B; ++b) place += lens[b] > mine || (lens[b] == mine && b < tid);
        reinterpret_cast<uint16_t*>(smem + OFF_ORDER)[place] = (uint16_t)tid;
    }
    Place* cuts = reinterpret_cast<Place*>(smem + OFF_CUTS);
    if constexpr (kCut) {
        uint32_t* weights = reinterpret_cast<uint32_t*>(smem + OFF_BEFORE);
        if (tid < p.B) {
            uint32_t sum = 0;
            for (int b = 0; b < tid; ++b) sum += unit_weight(lens[b]);
            weights[tid] = sum;
        }
        __syncthreads();
        if (tid < 2) cuts[tid] = cut_of(p, lens, weights, cluster / p.lanes + tid);
    }
    cluster_sync();  // every CTA's barriers (and the order) exist before any remote arrive or copy
    const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(smem + OFF_TMEM), 0);
    // q, the masks, the cache, the table and, where they were not kept above, the lengths may be earlier kernels' outputs
    griddep_wait();
    if (tid == 0) griddep_launch_dependents();

    // The cluster's unit number k (u: the one before). Whole units: in the order (request by length, tile), so that a
    // request's tiles run side by side and read its pages from L2. Cut ones: what lies between the cluster's cuts.
    auto unit_of = [&](int k, Unit& u) -> bool {
        Place at{};
        if constexpr (kCut) {
            at = k > 0 ? Place{u.entry + 1, 0} : cuts[0];
            if (!before(at, cuts[1])) return false;
            u.entry = at.entry;
            u.req = at.entry % p.B;
            u.tile = at.entry / p.B * p.lanes + cluster % p.lanes;
        } else {
            const uint32_t i = (uint32_t)k * clusters + (uint32_t)(k & 1 ? clusters - 1 - cluster : cluster);
            if (i >= (uint32_t)p.units) return false;
            u.req = (int)(i / (uint32_t)p.tiles);
            u.tile = (int)(i - (uint32_t)u.req * (uint32_t)p.tiles);
            if (sorted) u.req = (int)reinterpret_cast<const uint16_t*>(smem + OFF_ORDER)[u.req];
        }
        const int seq = kept ? lens[u.req] : length(u.req), pages = (seq + kPage - 1) / kPage;
        u.page0 = kPPG * at.group;
        int end = pages;
        if (kCut && cuts[1].entry == u.entry) end = min(pages, kPPG * cuts[1].group);
        u.npages = end - u.page0;
        u.part = kCut && u.npages < pages;
        u.slab = u.part ? 2 * cluster + (at.group == 0) : u.req;
        u.ngroups = (u.npages + kPPG - 1) / kPPG;
        u.drafts0 = seq - p.Sq;
        u.drafted = min(u.npages, max(0, max(u.drafts0, 0) / kPage - u.page0));
        return true;
    };
    auto rows_of = [&](const Unit& u) -> int { return u.tile * kTileRows + 128 * side; };  // first flat row of this CTA
    // First row of the unit's page i behind the keys' tensor map (out of range: TMA fills zeros).
    auto page_row = [&](const Unit& u, int i) -> int {
        if (i >= u.npages) return p.key_rows;
        if (kScaled) return (u.req * p.wide_pages + u.page0 + i) * kPage;
        const int32_t blk = p.block_table[(size_t)u.req * p.max_blocks + u.page0 + i];
        if (blk < 0 || (int64_t)blk >= p.num_blocks) {
            if (ds) atomicOr(ds, MLA_DEV_BAD_BLOCK_ID);
            return p.key_rows;
        }
        return blk * kPage;
    };

    // All roles walk the same units. `n` counts those with pages, whose barriers have one phase a unit; `g0` their
    // groups and `d0` their drafted pages before the current one.
    Unit u{};
    uint32_t n = 0, g0 = 0, d0 = 0;
    auto next = [&]() {
        ++n;
        g0 += (uint32_t)u.ngroups;
        d0 += (uint32_t)(u.npages - u.drafted);
    };
    if (scores) {
        if (warp == 0) {
            if (lane == 0) {
                tma_prefetch_desc(&k_map);
                tma_prefetch_desc(&q_map);
                bool ok = true;
                // The K ring's slots and the staging buffers (of the last group too) as the groups before g0 left them. A wait
                // by parity needs the phase before the awaited one to be over. With the last MMAs done, the softmax warps have
                // read the scores of group g0 - 3, so that g0 - 4 is staged but may not be sent (the output CTAs can be
                // an epilogue behind): group g0 - 2 is awaited as staged first, which group g0 - 4's copies precede.
                auto drained = [&](bool all) -> bool {
                    for (uint32_t m = 3 * g0 > kSlots ? 3 * g0 - kSlots : 0; m < 3 * g0; ++m)
                        if (!wait_bar<true>(bar(B_SLOTEMPTY + (int)(m % kSlots)), (m / kSlots) & 1, abort, ds)) return false;
                    for (uint32_t g = g0 > 2 ? g0 - 2 : 0; g + !all < g0; ++g)
                        for (int q = 0; q < kPPG; ++q) {
                            const int sbi = 2 * (int)(g & 1) + q;
                            if (!wait_bar(bar(B_STAGEFULL + sbi), (g >> 1) & 1, abort, ds) ||
                                !wait_bar<true>(bar(B_STAGEFREE + sbi), (g >> 1) & 1, abort, ds))
                                return false;
                        }
                    return true;
                };
                for (int k = 0; ok && unit_of(k, u); ++k) {
                    if (!kept) length(u.req, rank == 0);
                    if (u.npages == 0) continue;
                    int y = page_row(u, side);  // looked up ahead of the waits
                    if (!(ok = drained(false))) break;
                    bar_arrive_expect_tx(bar(B_QFULL), 9 * kQPanelBytes);
                    auto load_q = [&](uint32_t groups) {
#pragma unroll
                        for (int h = 0; h < 18; ++h)
                            tma_load_3d(sbase + (h < 16 ? q_half_off(h, groups) : OFF_QROPE + (h - 16) * kQHalfBytes), &q_map,
                                        bar(B_QFULL), (h >> 1) * 64, rows_of(u) + 64 * (h & 1), u.req);
                    };
                    if (g0 == 0)
                        load_q(0);  // constants
                    else
                        load_q(g0);
                    for (int gi = 0; gi < u.ngroups && ok; ++gi) {
                        if (gi > 0) y = page_row(u, kPPG * gi + side);
                        for (int t = 0; t < 3; ++t) {
                            // behind what loads beside Q: its panels have been moved out to TMEM
                            if (3 * gi + t == (n == 0 ? 3 : 1) && !(ok = wait_bar(bar(B_QREADY), n & 1, abort, ds))) break;
                            const uint32_t m = 3 * (g0 + (uint32_t)gi) + (uint32_t)t;
                            const int slot = (int)(m % kSlots);
                            if (m >= kSlots && !(ok = wait_bar<true>(bar(B_SLOTEMPTY + slot), (m / kSlots - 1) & 1, abort, ds))) break;
                            // both CTAs' bytes are counted on CTA 0's barrier
                            if (side == 0) bar_arrive_expect_tx(bar(B_SLOTFULL + slot), 2 * kSlotBytes);
                            tma_load_3d_pair(sbase + OFF_RING + slot * kSlotBytes, &k_map,
                                             map_to_rank(bar(B_SLOTFULL + slot), 0), 0, y, kSlotPanels * t);
                        }
                    }
                    next();
                }
                // Teardown: the MMAs have consumed the last slots, so every copy has landed and no commit is
                // still on its way here.
                if (!ok || !drained(true)) settle();
            }
        } else if (warp == 1) {
            if (lane == 0 && side == 1) {
                // tell the issuing CTA that this CTA's half of Q is in place
                for (int k = 0; unit_of(k, u); ++k) {
                    if (u.npages == 0) continue;
                    if (!wait_bar(bar(B_QREADY), n & 1, abort, ds)) break;
                    tc_fence_after();
                    tc_fence_before();  // tensor memory alone is published: no release is needed
                    bar_arrive_remote_relaxed(bar(B_QPEER), 0);
                    next();
                }
            }
            if (side == 0) {
                // The whole warp runs the loop and one elected lane issues: descriptors and addresses then live
                // in uniform registers (from a lane-0 branch an MMA took 140 cycles instead of 64).
                const bool leader = elect_one();
                const uint64_t rope0 = smem_desc_sw128(sbase + OFF_QROPE, 16, 1024);
                bool ok = true;
                int slot = 0, phase = 0;
                for (int k = 0; ok && unit_of(k, u); ++k) {
                    if (u.npages == 0) continue;
                    ok = warp_wait(bar(B_QREADY), n & 1, abort, ds) && warp_wait<true>(bar(B_QPEER), n & 1, abort, ds);
                    if (ok) tc_fence_after();
                    for (int gi = 0; gi < u.ngroups && ok; ++gi) {
                        const uint32_t g = g0 + (uint32_t)gi;
                        const int buf = (int)(g & 1);
                        if (g > 1) {  // both CTAs' softmax warps have read the buffer's previous S
                            if (!(ok = warp_wait<true>(bar(B_SEMPTY + buf), ((g >> 1) - 1) & 1, abort, ds))) break;
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
                    next();
                }
            }
        } else if (warp == 18) {
            // ------------------------- P copies -------------------------
            // One thread sends each staged page, so that the softmax neither waits for the output CTA's
            // buffer nor for the issue.
            if (lane == 0) {
                const uint32_t out_rank = 2u + (uint32_t)side;
                const uint32_t pbuf_remote = map_to_rank(sbase + OFF_PB, out_rank);
                const uint32_t pfull_remote = map_to_rank(bar(B_PFULL), out_rank);
                bool ok = true;
                for (int k = 0; ok && unit_of(k, u); ++k) {
                    if (u.npages == 0) continue;
                    for (uint32_t page = 2 * g0; page < 2 * (g0 + (uint32_t)u.ngroups) && ok; ++page) {
                        const int sbi = (int)(page & 3), pb = (int)(page % kPBufs);
                        ok = wait_bar(bar(B_STAGEFULL + sbi), (page >> 2) & 1, abort, ds) &&
                             (page < kPBufs || wait_bar<true>(bar(B_PEMPTY + pb), (page / kPBufs - 1) & 1, abort, ds)) && !*abort;
                        if (!ok) break;
                        bulk_copy_to_peer(pbuf_remote + pb * kPBufStride, sbase + OFF_STAGE + sbi * kPBufStride, kPMsgBytes,
                                          pfull_remote + 8u * pb);
                    }
                    // The output CTA may now wait for its last page: the page kPBufs earlier is done, so a wait
                    // by parity cannot take that page's phase for the last one's.
                    if (ok) bar_arrive_remote(bar(B_STATS), out_rank);
                    next();
                }
                // nothing may still be on its way to this CTA when it exits: the last multicast commits of the
                // output pair, its last announcement
                if (ok) {
                    for (uint32_t page = 2 * g0 > kPBufs ? 2 * g0 - kPBufs : 0; page < 2 * g0; ++page)
                        wait_bar<true>(bar(B_PEMPTY + (int)(page % kPBufs)), (page / kPBufs) & 1, abort, ds);
                    if (n > 0) wait_bar<true>(bar(B_DONE), (n - 1) & 1, abort, ds);
                }
            }
        } else {
            // ------------------------- softmax warps (512 threads) -------------------------
            // Quarter `quarter` of the warps owns 32 columns of each group's S: half of page `pg2`.
            const int quarter = (warp - 2) >> 2, pg2 = quarter >> 1, sub = quarter & 1;
            const int row = 32 * (warp & 3) + lane;
            const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
            const uint32_t out_rank = 2u + (uint32_t)side;
            float* mx = reinterpret_cast<float*>(smem + OFF_MX);
            const float sl2 = p.scale * 1.4426950408889634f;  // exp2 domain
            for (int k = 0; unit_of(k, u); ++k) {
                if (u.npages == 0) continue;
                uint64_t mask = 0;  // the drafts that the row sees
                if (rows_of(u) + row < p.flat_rows) {
                    mask = __ldcg(reinterpret_cast<const unsigned long long*>(p.masks) + (size_t)u.req * p.Sq +
                                  (rows_of(u) + row) / p.H);
                    if (p.Sq < 64) mask &= (1ull << p.Sq) - 1;
                }
                {
                    // Q latent dims: this quarter moves panels 2 quarter and 2 quarter + 1 into TMEM. (Q was
                    // loaded after the last MMA that reads the unit before's.)
                    const bool okq = warp_wait(bar(B_QFULL), n & 1, abort, ds);
#pragma unroll 1
                    for (int pn = 2 * quarter; pn < 2 * quarter + 2; ++pn) {
                        const uint32_t home = q_half_off(2 * pn + (row >> 6), g0) + (row & 63) * 128;
                        uint32_t v[32];
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            uint4 x = make_uint4(0, 0, 0, 0);
                            if (okq)
                                x = *reinterpret_cast<const uint4*>(smem + home + ((c ^ (row & 7)) << 4));
                            v[4 * c] = x.x;
                            v[4 * c + 1] = x.y;
                            v[4 * c + 2] = x.z;
                            v[4 * c + 3] = x.w;
                        }
                        tmem_st32(tmem + lane_base + 32u * pn, v);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    dec::warp_arrive(bar(B_QREADY), lane);
                }
                // FP8: half of the threads bring one scale each of a group into shared memory, two groups ahead of
                // its use. (Read from global memory by every thread they cost 0.2 us a group and spilled.)
                const int ft = tid - 64;
                float sc = 0.f;
                auto scale_of = [&](int gi) -> float {
                    const int page = min(kPPG * gi + (ft >> 6 & 1), u.npages - 1);
                    const float* src = ft < kPPG * kPage ? p.k_scales : p.v_scales;
                    return src[((size_t)u.req * p.wide_pages + u.page0 + page) * kPage + (ft & 63)];
                };
                auto put_scale = [&](uint32_t g, float x) {
                    reinterpret_cast<float*>(smem + OFF_SCALES + g % 3 * kScaleBytes)[ft] = x;
                };
                if (kScaled) {
                    if (ft < 2 * kPPG * kPage) {
                        const float first = scale_of(0);
                        sc = scale_of(1);
                        put_scale(g0, first);
                    }
                    named_bar(kBarMax, kSoftThreads);
                }
                float m_run = -CUDART_INF_F, l_run = 0.f;  // each quarter keeps its own sum
                for (int gi = 0; gi < u.ngroups; ++gi) {
                    // No early exit from this loop: all 512 threads must pass the same named barriers (which
                    // cannot time out); after an abort the waits return at once.
                    const uint32_t g = g0 + (uint32_t)gi;
                    const int page = kPPG * gi + pg2, buf = (int)(g & 1);
                    if (kScaled && ft < 2 * kPPG * kPage) {  // visible to all behind this group's barrier
                        put_scale(g + 1, sc);
                        sc = scale_of(gi + 2);
                    }
                    const float4* scales = reinterpret_cast<const float4*>(smem + OFF_SCALES + g % 3 * kScaleBytes) + 8 * quarter;
                    const bool okS = warp_wait<true>(bar(B_SFULL + buf), (g >> 1) & 1, abort, ds);
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
                    auto pair = [&](int j) {
                        return make_float2(__uint_as_float(s[2 * j]), __uint_as_float(s[2 * j + 1]));
                    };
                    if constexpr (kScaled) {
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            const float4 k = scales[j >> 1];
                            const float2 a = mul2(pair(j), make_float2(k.x, k.y)), b = mul2(pair(j + 1), make_float2(k.z, k.w));
                            s[2 * j] = __float_as_uint(a.x);
                            s[2 * j + 1] = __float_as_uint(a.y);
                            s[2 * j + 2] = __float_as_uint(b.x);
                            s[2 * j + 3] = __float_as_uint(b.y);
                        }
                    }
                    // bit c: the row sees token 32 sub + c of the page; none of the page behind the last
                    uint32_t seen = 0xffffffffu;
                    if (page >= u.drafted) {
                        seen = page < u.npages ? seen_tokens(mask, (u.page0 + page) * kPage + 32 * sub - u.drafts0) : 0u;
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (!(seen >> j & 1u)) s[j] = __float_as_uint(-CUDART_INF_F);
                    }
                    float lm4[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
                    for (int j = 0; j < 16; ++j) lm4[j & 3] = max3(lm4[j & 3], pair(j).x, pair(j).y);
                    const float lm = max3(lm4[0], lm4[1], fmaxf(lm4[2], lm4[3]));
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
                    {
                        float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            float2 a = fma2(pair(j), make_float2(sl2, sl2), make_float2(-mref, -mref));
                            a = make_float2(fast_exp2(a.x), fast_exp2(a.y));
                            l2[j & 1] = add2(l2[j & 1], a);
                            if constexpr (kScaled)
                                a = mul2(a, reinterpret_cast<const float2*>(scales + kPPG * kPage / 4)[j]);
                            pk[j] = pack_bf16x2(a.x, a.y);
                        }
                        if (kScaled && page >= u.drafted) {  // a hidden token has no weight, whatever its scale is
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                pk[j] &= (seen >> (2 * j) & 1u ? 0xffffu : 0u) | (seen >> (2 * j + 1) & 1u ? 0xffff0000u : 0u);
                        }
                        l2[0] = add2(l2[0], l2[1]);
                        l_run += l2[0].x + l2[0].y;
                    }
                    // the page's staging buffers take turns: this one is free once the copy of two groups ago
                    // has landed
                    const int sbi = 2 * buf + pg2;
                    uint8_t* stage = smem + OFF_STAGE + sbi * kPBufStride;
                    if (g > 1) warp_wait<true>(bar(B_STAGEFREE + sbi), ((g >> 1) - 1) & 1, abort, ds);
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
                // combine the quarters' sums, ship the unit's statistics (the unit before's have been read once
                // it is stored)
                named_bar(kBarMax, kSoftThreads);
                mx[quarter * 128 + row] = l_run;
                named_bar(kBarMax, kSoftThreads);
                if (quarter == 0) {
                    if (n > 0) warp_wait<true>(bar(B_DONE), (n - 1) & 1, abort, ds);
                    l_run = (mx[row] + mx[128 + row]) + (mx[256 + row] + mx[384 + row]);
                    st_cluster_u32(map_to_rank(sbase + OFF_STAT_M, out_rank) + 4u * row, __float_as_uint(m_run));
                    st_cluster_u32(map_to_rank(sbase + OFF_STAT_L, out_rank) + 4u * row, __float_as_uint(l_run));
                    named_bar(kBarQuarter0, 128);
                    if (tid == 64) bar_arrive_remote(bar(B_STATS), out_rank);
                }
                next();
            }
        }
    } else {
        // ============================== output CTAs ==============================
        if (warp == 0) {
            if (lane == 0) {
                tma_prefetch_desc(&v_map);
                bool ok = true;
                for (int k = 0; ok && unit_of(k, u); ++k) {
                    if (u.npages == 0) continue;
                    int y = page_row(u, 0);  // looked up ahead of the wait
                    // the ring holds the unit before's output tiles until it is stored
                    if (n > 0 && !(ok = wait_bar(bar(B_DONE), (n - 1) & 1, abort, ds))) break;
                    for (int i = 0; i < kPPG * u.ngroups; ++i) {
                        if (i > 0) y = page_row(u, i);
                        const uint32_t v = kPPG * g0 + (uint32_t)i;
                        const int st = (int)(v % kVStages);
                        if (v >= kVStages && !(ok = wait_bar<true>(bar(B_VEMPTY + st), (v / kVStages - 1) & 1, abort, ds))) break;
                        uint32_t full = map_to_rank(bar(B_VFULL + st), 2);
                        if (!kScaled && i >= u.drafted && i < u.npages) {  // to be looked over in each CTA first
                            const int land = B_VLAND + (int)((d0 + (uint32_t)(i - u.drafted)) & 1);
                            bar_arrive_expect_tx(bar(land), kVStageBytes);
                            full = map_to_rank(bar(land), rank);
                        } else if (side == 0) {
                            bar_arrive_expect_tx(bar(B_VFULL + st), 2 * kVStageBytes);
                        }
                        const uint32_t dst = sbase + OFF_V + st * kVStageBytes;
                        tma_load_3d_pair(dst, &v_map, full, 0, y, 2 * side);
                        tma_load_3d_pair(dst + 2 * kPageBox, &v_map, full, 0, y, 4 + 2 * side);
                    }
                    next();
                }
                // teardown, as above
                const uint32_t end = kPPG * g0;
                for (uint32_t v = end > kVStages ? end - kVStages : 0; ok && v < end; ++v)
                    ok = wait_bar<true>(bar(B_VEMPTY + (int)(v % kVStages)), (v / kVStages) & 1, abort, ds);
                if (!ok) settle();
            }
        } else if (warp == 1) {
            bool ok = true;
            const bool leader = elect_one();  // as for the scores
            for (int k = 0; ok && unit_of(k, u); ++k) {
                if (u.npages == 0) continue;
                for (int i = 0; i < kPPG * u.ngroups && ok && side == 0; ++i) {
                    const uint32_t v = kPPG * g0 + (uint32_t)i;
                    const int pb = (int)(v % kPBufs), st = (int)(v % kVStages);
                    if (!(ok = warp_wait<true>(bar(B_READY + pb), (v / kPBufs) & 1, abort, ds))) break;
                    if (!kScaled && i >= u.drafted && i < u.npages) {
                        const uint32_t d = d0 + (uint32_t)(i - u.drafted);
                        ok = warp_wait<true>(bar(B_VCLEAN + (int)(d & 1)), (d >> 1) & 1, abort, ds);
                        if (leader) bar_arrive(bar(B_VFULL + st));  // the stage's own barrier keeps pace
                    } else {
                        ok = warp_wait<true>(bar(B_VFULL + st), (v / kVStages) & 1, abort, ds);
                    }
                    if (!ok) break;
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
                next();
            }
            const uint32_t end = kPPG * g0;  // the last commits have landed in this CTA
            for (uint32_t v = end > kPBufs ? end - kPBufs : 0; ok && v < end; ++v)
                ok = warp_wait<true>(bar(B_PEMPTY + (int)(v % kPBufs)), (v / kPBufs) & 1, abort, ds);
        } else if (warp < 18) {
            // ------------- helper warps 2-5: P arrival, rescale; warps 2-17: the epilogue -------------
            const int row = 32 * (warp & 3) + lane;
            const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
            const int ctid = tid - 64;  // 0..511; 0..127 are the helper warps
            const int eset = (warp - 2) >> 2;
            if (kCut && eset == 0 && cuts[0].group > 0 && !before(cuts[0], cuts[1]))  // a share of no groups amid a unit
                p.part_lse[(size_t)2 * cluster * kTileRows + 128 * side + row] = -CUDART_INF_F;
            for (int k = 0; unit_of(k, u); ++k) {
                const int rows0 = rows_of(u);
                float* lse_out = u.part ? p.part_lse : p.lse;
                const size_t out_row =
                    u.part ? (size_t)u.slab * kTileRows + 128 * side + row : (size_t)u.slab * p.flat_rows + rows0 + row;
                const bool live = rows0 + row < p.flat_rows;
                if (u.npages == 0) {  // no token
                    if (eset == 0 && live && lse_out) lse_out[out_row] = -CUDART_INF_F;
                    if (live) {
                        const int bytes = p.o_bf16 ? 2 * kL / 4 : 4 * kL / 4;  // of this warp set's quarter of the row
                        uint4* dst = reinterpret_cast<uint4*>((uint8_t*)p.o + out_row * 4 * bytes + (size_t)eset * bytes);
                        for (int c = 0; c < bytes / 16; ++c) dst[c] = make_uint4(0u, 0u, 0u, 0u);
                    }
                    continue;
                }
                const int pages = kPPG * u.ngroups;
                bool ready = true;
                for (int i = 0; i < pages && warp < 6; ++i) {
                    const uint32_t v = kPPG * g0 + (uint32_t)i;
                    const int pb = (int)(v % kPBufs);
                    if (!(ready = warp_wait<true>(bar(B_PFULL + pb), (v / kPBufs) & 1, abort, ds))) break;
                    if (ctid == 0) {
                        bar_arrive_expect_tx(bar(B_PFULL + pb), kPMsgBytes);           // re-arm for the next message
                        bar_arrive_remote_relaxed(bar(B_STAGEFREE + (int)(v & 3)), (uint32_t)side);  // the sender's staging buffer
                    }
                    const uint8_t* pmsg = smem + OFF_PB + pb * kPBufStride;
                    const bool fix = i > 0 && *reinterpret_cast<const volatile uint32_t*>(pmsg + kPBytes + 512) != 0;
                    if (fix) {  // O must hold every earlier PV product before it is rescaled
                        if (!(ready = warp_wait<true>(bar(B_PEMPTY + (int)((v - 1) % kPBufs)), ((v - 1) / kPBufs) & 1, abort, ds))) break;
                        tc_fence_after();
                        const float a = reinterpret_cast<const volatile float*>(pmsg + kPBytes)[row];
#pragma unroll 1
                        for (int c = 0; c < kL / 32; ++c) {
                            uint32_t x[32];
                            tmem_ld32(tmem + lane_base + 32u * c, x);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 32; ++j) x[j] = __float_as_uint(__uint_as_float(x[j]) * a);
                            tmem_st32(tmem + lane_base + 32u * c, x);
                        }
                        tmem_wait_st();
                    }
                    tc_fence_before();
                    // P came through the async proxy into this CTA, and O may have been rescaled here; both are
                    // read by MMAs that CTA 2 issues. CTA 2's warps tell its MMA warp themselves, CTA 3's
                    // through the relay below.
                    fence_proxy_async_cta();
                    dec::warp_arrive(bar((side == 0 ? B_READY : B_PEER) + pb), lane);
                    if (ctid == 0) *reinterpret_cast<volatile uint32_t*>(smem + OFF_PROG) = v + 1;
                }
                // CTA 3's pages are announced to CTA 2 by an arrival that releases at cluster scope, since it
                // publishes the helpers' writes. That takes most of a microsecond, so warps that have nothing else
                // to do before the epilogue take the pages in turn.
                if (side == 1 && warp >= 6 && warp < 6 + kRelayWarps && lane == 0) {
                    for (int i = warp - 6; i < pages; i += kRelayWarps) {
                        const uint32_t v = kPPG * g0 + (uint32_t)i;
                        const int pb = (int)(v % kPBufs);
                        if (!wait_bar(bar(B_PEER + pb), (v / kPBufs) & 1, abort, ds)) break;
                        tc_fence_after();
                        tc_fence_before();
                        bar_arrive_remote(bar(B_READY + pb), 2);
                    }
                }
                if (!kScaled && warp >= kAuxWarp0) {
                    // drafts and the cache rows behind them: hidden from some rows, see dec::zero_nonfinite
                    for (int i = u.drafted; i < u.npages; ++i) {
                        const uint32_t d = d0 + (uint32_t)(i - u.drafted);
                        if (!warp_wait(bar(B_VLAND + (int)(d & 1)), (d >> 1) & 1, abort, ds)) break;
                        const uint32_t v = sbase + OFF_V + ((kPPG * g0 + (uint32_t)i) % kVStages) * kVStageBytes +
                                           16u * (uint32_t)(tid - 32 * kAuxWarp0);
#pragma unroll
                        for (int c = 0; c < kVStageBytes; c += 32 * kAuxWarps * 16) dec::zero_nonfinite(v + c);
                        fence_proxy_async_cta();
                        __syncwarp();
                        if (lane == 0) bar_arrive_remote(bar(B_VCLEAN + (int)(d & 1)), 2);
                    }
                }
                __syncwarp();
                const uint32_t last = kPPG * g0 + (uint32_t)pages - 1;
                wait_bar<true>(bar(B_STATS), n & 1, abort, ds);
                const bool o_ok = ready && !*abort &&
                                  wait_bar<true>(bar(B_PEMPTY + (int)(last % kPBufs)), (last / kPBufs) & 1, abort, ds);
                tc_fence_after();
                const float m = reinterpret_cast<volatile float*>(smem + OFF_STAT_M)[row];
                const float l = reinterpret_cast<volatile float*>(smem + OFF_STAT_L)[row];
                const bool use_o = __all_sync(0xffffffffu, o_ok);
                const bool empty = !use_o || l == 0.f;  // no token has a weight; a NaN sum is a NaN result
                const float inv = empty ? 0.f : 1.f / l;
                if (eset == 0 && live && lse_out)
                    lse_out[out_row] = empty ? -CUDART_INF_F : (m + log2f(l)) * 0.6931471805599453f;
                // O / l leaves through TMA stores over the V ring; rows past the request's are
                // cut off by the tensor map
                const bool store = rows0 < p.flat_rows;
                if (p.o_bf16 && !u.part)
                    store_rows<false, 4, 2, kBarEpi, false>(smem, sbase, OFF_V, tmem + lane_base, row, eset, (ctid & 127) == 0, true,
                                                     empty, inv, &o_map, rows0, u.slab, store);
                else
                    store_rows<true, 4, 2, kBarEpi, false>(smem, sbase, OFF_V, tmem + lane_base, row, eset, (ctid & 127) == 0, true,
                                                    empty, inv, u.part ? &part_map : &o_map, u.part ? 128 * side : rows0,
                                                    u.slab, store);
                // O, the statistics and the tiles have been read: the next unit's may come
                tc_fence_before();
                fence_proxy_async_cta();
                named_bar(kBarStored, kSoftThreads);
                if (ctid == 0) {
                    bar_arrive(bar(B_DONE));
                    bar_arrive_remote(bar(B_DONE), (uint32_t)side);
                }
                next();
            }
            if ((ctid & 127) == 0) bulk_wait_group<0>();  // the stores are complete before the CTA exits
        } else if (kCut && side == 1) {
            // Warp 18 of CTA 3: for the merge, the unit that ends in the cluster's share, and the share it begins in.
            if (lane == 0) {
                const Place from = cuts[0];
                int share = -1;
                if (from.group > 0 && cuts[1].entry > from.entry) {
                    const uint32_t* weights = reinterpret_cast<const uint32_t*>(smem + OFF_BEFORE);
                    share = cluster / p.lanes - 1;
                    while (before(Place{from.entry, 0}, cut_of(p, lens, weights, share))) --share;
                }
                p.pieces[cluster] = make_int2(from.entry, share);
            }
        } else if (!kScaled && side == 0 && lane == 0 && p.tiles == 1) {
            // Warp 18: the pages that the rings have no room for yet are brought into L2, the next unit's first ones
            // too (64 requests of up to 8192 tokens, 112 pairs: 146 -> 139 us; with several tiles a request the others
            // mostly find them there, and line by line it cost 5 to 8%). Only a hint: it gives up quietly.
            const volatile uint32_t* prog = reinterpret_cast<const volatile uint32_t*>(smem + OFF_PROG);
            bool go = true;
            for (int k = 0; go && unit_of(k, u); next(), ++k)
                for (int i = n == 0 ? kInRings : 0; i < u.npages && go; ++i) {
                    for (int spins = 0; (int32_t)(*prog + kAhead - (kPPG * g0 + (uint32_t)i)) < 0; ++spins) {
                        if (*abort || spins > (1 << 16)) {
                            go = false;
                            break;
                        }
                        __nanosleep(128);
                    }
                    const int y = page_row(u, i);
                    if (go && y < p.key_rows) bulk_prefetch_l2(p.keys + (size_t)y * kBf16RowBytes, kPage * kBf16RowBytes);
                }
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (warp == 0) tmem_dealloc_pair(tmem, kTmemCols);
    cluster_sync();
}

// ------------------------------------------------------------------------------------------
// FP8 pages -> bf16 rows (exact) and scales, every request's, once per call. One block per page; a thread
// takes nine chunks of 8 codes, all of their loads first (36 requests of 4 pages: 28 -> 24 us a call against two
// rounds of 256 threads). A request's last page is widened whole: what is behind its end is not seen.
// ------------------------------------------------------------------------------------------
constexpr int kWidenThreads = 512, kChunks = kPage * kD / 8, kBatch = 9;
static_assert(kChunks % (kWidenThreads * kBatch) == 0, "a page's chunks");
__global__ void __launch_bounds__(kWidenThreads) tree_widen_kernel(TreeArgs p, const uint8_t* cache, uint16_t* x,
                                                                   float* k_scales, float* v_scales) {
    griddep_wait();
    griddep_launch_dependents();
    const int req = (int)(blockIdx.x / (unsigned)p.wide_pages), page = (int)(blockIdx.x % (unsigned)p.wide_pages), tid = threadIdx.x;
    if (page >= (min(max(p.seq_lens[req], 0), p.max_seq_len) + kPage - 1) / kPage) return;
    const int32_t blk = p.block_table[(size_t)req * p.max_blocks + page];
    const bool bad = blk < 0 || (int64_t)blk >= p.num_blocks;
    if (bad && tid == 0 && p.dev_status) atomicOr(p.dev_status, MLA_DEV_BAD_BLOCK_ID);
    const uint8_t* src = cache + (size_t)(bad ? 0 : blk) * (kPage * kFp8RowBytes);
    const size_t row0 = ((size_t)req * p.wide_pages + page) * kPage;
    uint4* dst = reinterpret_cast<uint4*>(x + row0 * kD);
    float2 sc = make_float2(0.f, 0.f);
    if (tid < kPage && !bad) sc = *reinterpret_cast<const float2*>(src + tid * kFp8RowBytes + kD);
#pragma unroll
    for (int k0 = 0; k0 < kChunks; k0 += kWidenThreads * kBatch) {
        uint2 v[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int c = k0 + k * kWidenThreads + tid;
            v[k] = make_uint2(0u, 0u);
            if (!bad) v[k] = *reinterpret_cast<const uint2*>(src + 8 * (c + c / (kD / 8)));  // a row's chunks, then its scales
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            uint4 w;  // as the decode kernels read the codes
            e4m3x4_to_bf16x4(v[k].x, w.x, w.y);
            e4m3x4_to_bf16x4(v[k].y, w.z, w.w);
            dst[k0 + k * kWidenThreads + tid] = w;
        }
    }
    if (tid < kPage) {
        k_scales[row0 + tid] = sc.x;
        v_scales[row0 + tid] = sc.y;
    }
}

// ------------------------------------------------------------------------------------------
// The states of a cut unit's parts -> its rows:  o = sum_i w_i o_i / sum_i w_i,  lse = M + log sum_i w_i,  w_i =
// exp(lse_i - M), M the largest lse. Half a row a warp, four rows a block and turn. Up to two parts of 512 KB a cluster,
// 37 MB, are read once, 6 to 9 us with the launch. Four blocks an SM, of which three run at once (76 registers): with one for
// every cluster and four rows (2304) 3 x 256 rows over up to 3000 tokens took 24.8 us a call, 23.5 so.
// ------------------------------------------------------------------------------------------
constexpr int kMergeThreads = 256, kMergeRows = kMergeThreads / 64, kMergeBatch = 3, kMergeBlocks = 608;
__global__ void __launch_bounds__(kMergeThreads) tree_merge_kernel(const TreeArgs p) {
    griddep_launch_dependents();
    griddep_wait();
    static_assert(kTreeMaxClusters == 64, "two a lane");
    __shared__ int3 units_s[kTreeMaxClusters];  // (entry, its first share, cluster of its last one)
    __shared__ int n_s;
    const int tid = threadIdx.x, lane = tid & 31, clusters = p.shares * p.lanes;
    if (tid < 32) {
        int found = 0;
        int2 u[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) u[h] = 32 * h + lane < clusters ? p.pieces[32 * h + lane] : make_int2(0, -1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t cut = __ballot_sync(0xffffffffu, u[h].y >= 0);
            if (u[h].y >= 0) units_s[found + __popc(cut & ((1u << lane) - 1u))] = make_int3(u[h].x, u[h].y, 32 * h + lane);
            found += __popc(cut);
        }
        if (lane == 0) n_s = found;
    }
    __syncthreads();
    const int chunks = (p.slab_rows + kMergeRows - 1) / kMergeRows, tasks = n_s * chunks, dim = (tid & 63) * 8;
    for (int task = (int)blockIdx.x; task < tasks; task += (int)gridDim.x) {
        const int3 unit = units_s[task / chunks];
        const int row = task % chunks * kMergeRows + (tid >> 6), side = unit.z % p.lanes;
        const int flat = (unit.x / p.B * p.lanes + side) * kTileRows + row;
        if (flat >= p.flat_rows) continue;
        // the unit's first part is its share's last one, the others their shares' first
        const int n = unit.z / p.lanes - unit.y + 1;
        auto slab_of = [&](int i) -> size_t { return 2 * (size_t)((unit.y + i) * p.lanes + side) + (i == 0); };
        float4 v[kMergeBatch][2];
        float x[kMergeBatch];
        auto load = [&](int i0) {
#pragma unroll
            for (int k = 0; k < kMergeBatch; ++k) {
                x[k] = -CUDART_INF_F;
                v[k][0] = v[k][1] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i0 + k >= n) continue;
                const size_t slab = slab_of(i0 + k);
                x[k] = p.part_lse[slab * kTileRows + row];
                const float4* src = reinterpret_cast<const float4*>(p.part_o + (slab * p.slab_rows + row) * kL + dim);
                v[k][0] = src[0];
                v[k][1] = src[1];
            }
        };
        load(0);
        // a NaN state counts as the largest: its weight, the sum and the result are NaN then
        float M = -CUDART_INF_F;
        for (int i = lane; i < n; i += 32) {
            const float y = p.part_lse[slab_of(i) * kTileRows + row];
            M = fmaxf(M, y != y ? CUDART_INF_F : y);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        float acc[8] = {}, sum = 0.f;
        for (int i0 = 0; i0 < n && M != -CUDART_INF_F; i0 += kMergeBatch) {
            if (i0 > 0) load(i0);
#pragma unroll
            for (int k = 0; k < kMergeBatch; ++k) {
                if (x[k] == -CUDART_INF_F) continue;
                const float w = __expf(x[k] - M);
                sum += w;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    acc[4 * h] = fmaf(w, v[k][h].x, acc[4 * h]);
                    acc[4 * h + 1] = fmaf(w, v[k][h].y, acc[4 * h + 1]);
                    acc[4 * h + 2] = fmaf(w, v[k][h].z, acc[4 * h + 2]);
                    acc[4 * h + 3] = fmaf(w, v[k][h].w, acc[4 * h + 3]);
                }
            }
        }
        const float inv = M == -CUDART_INF_F ? 0.f : 1.f / sum;
        const size_t out = (size_t)(unit.x % p.B) * p.flat_rows + flat;
        if ((tid & 63) == 0 && p.lse) p.lse[out] = M == -CUDART_INF_F ? M : M + logf(sum);
        if (p.o_bf16) {
            *reinterpret_cast<uint4*>((uint16_t*)p.o + out * kL + dim) =
                make_uint4(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv),
                           pack_bf16x2(acc[4] * inv, acc[5] * inv), pack_bf16x2(acc[6] * inv, acc[7] * inv));
        } else {
            float4* dst = reinterpret_cast<float4*>((float*)p.o + out * kL + dim);
            dst[0] = make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
            dst[1] = make_float4(acc[4] * inv, acc[5] * inv, acc[6] * inv, acc[7] * inv);
        }
    }
}

int g_attr_done[2][2][64] = {};
int g_clusters[64] = {};

using TreeKernel = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, TreeArgs);
const TreeKernel kKernels[2][2] = {{decode_tree_kernel<false, false>, decode_tree_kernel<false, true>},
                                   {decode_tree_kernel<true, false>, decode_tree_kernel<true, true>}};  // [FP8][cut]

cudaError_t set_attr(int dev, bool scaled, bool cut) {
    if (dev < 64 && g_attr_done[scaled][cut][dev]) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kKernels[scaled][cut], cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e == cudaSuccess && dev < 64) g_attr_done[scaled][cut][dev] = 1;
    return e;
}

}  // namespace

int tree_clusters() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return -1;
    if (dev < 64 && g_clusters[dev] > 0) return g_clusters[dev];
    if (set_attr(dev, false, false) != cudaSuccess) return -1;
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
    if (cudaOccupancyMaxActiveClusters(&n, kKernels[0][0], &cfg) != cudaSuccess || n < 1) return -1;
    n = std::min(n, kTreeMaxClusters);
    if (dev < 64) g_clusters[dev] = n;
    return n;
}

int tree_shares(int B, int tiles, int slab_rows, int pages, int clusters, int* lanes) {
    // Times in groups (1.28 us), of requests half to all as long as the longest. Whole units: the balanced time, and
    // the rest of the last turn.
    if (B < 1 || B > kTreeMaxCut || pages < 2 * kPPG) return 0;
    const double longest = (pages + kPPG - 1) / kPPG, usual = 0.75 * longest, units = (double)B * tiles;
    const double turns = std::ceil(units / clusters), even = units / clusters * (usual + kUnitGroups);
    double best = turns == 1 ? longest + kUnitGroups : even + 0.4 * (turns - units / clusters) * (longest + kUnitGroups);
    // Cut: a request of few groups into fewer parts. One more takes G / n^2 of its G groups off each of n, and costs a
    // third of a group of the merge's time, or its rows written and read (5 TB/s).
    const double parts = std::min(std::sqrt(units * longest * 1562.0 / slab_rows) / units, 1.7 * std::sqrt(longest));
    const double part = std::max(1.0, std::ceil(longest / parts));
    int found = 0;
    for (int n = 1; n <= tiles && n <= clusters; ++n) {
        if (tiles % n) continue;
        const double requests = (double)B * (tiles / n);
        const double shares = std::min(std::floor((double)clusters / n),
                                       std::max(requests, std::ceil((requests * (longest + kUnitGroups) - kUnitGroups) / part)));
        if (shares < 2) continue;
        // beside a share of the groups: a start of its own, the merge's launch, and the partial rows written and read (12
        // groups for 36 x 256 rows);
        // tiles that do not go through a share side by side find less of it in L2 (1 lane for 4 tiles: 10%)
        const double merge = 2.0 + 12.0 / (36 * kTileRows) * shares * n * slab_rows;
        const double cut = requests * (usual + kUnitGroups) / shares * (1.0 + 0.05 * std::log2((double)tiles / n)) + kUnitGroups + merge;
        if (cut < best) {
            best = cut;
            found = (int)shares;
            *lanes = n;
        }
    }
    return found;
}

cudaError_t launch_decode_tree(const TreeArgs& in, bool fp8, const uint8_t* cache, uint16_t* widened, float* scales,
                               cudaStream_t s) {
    TreeArgs a = in;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = set_attr(dev, fp8, a.pieces != nullptr);
    if (e != cudaSuccess) return e;
    const int clusters = tree_clusters();
    if (clusters < 1) return cudaErrorUnknown;
    // with a bound of 0 no request has a page, and cache, table and workspace may be null
    uint64_t rows = a.max_seq_len > 0 ? (uint64_t)a.num_blocks * kPage : 0;
    if (fp8) {
        rows = a.max_seq_len > 0 ? (uint64_t)a.B * a.wide_pages * kPage : 0;
        a.k_scales = scales;
        a.v_scales = scales + rows;
        if (rows > 0) {
            e = launch_pdl(tree_widen_kernel, dim3((unsigned)(rows / kPage)), dim3(kWidenThreads), 0, s, a, cache,
                           widened, scales, scales + rows);
            if (e != cudaSuccess) return e;
        }
    }
    a.key_rows = (int)rows;
    a.keys = fp8 ? (const uint8_t*)widened : cache;
    CUtensorMap k_map, v_map, q_map, o_map, part_map;
    memset(&k_map, 0, sizeof k_map);
    memset(&v_map, 0, sizeof v_map);
    memset(&q_map, 0, sizeof q_map);
    memset(&o_map, 0, sizeof o_map);
    memset(&part_map, 0, sizeof part_map);
    if (rows > 0) {
        // the rows as [panel of 64 dims][row][64]: one box is several panels of a page
        const void* base = fp8 ? (const void*)widened : cache;
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
        const uint64_t dims[3] = {(uint64_t)kD, (uint64_t)a.flat_rows, (uint64_t)a.B};
        const uint64_t strides[2] = {(uint64_t)kD * 2, (uint64_t)a.flat_rows * kD * 2};
        const uint32_t box[3] = {64, 64, 1};
        e = encode_tmap(&q_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.q, dims, strides, box, true);
        if (e != cudaSuccess) return e;
    }
    {
        const bool f32 = !a.o_bf16;
        const uint64_t size = f32 ? 4 : 2;
        const uint64_t dims[3] = {(uint64_t)kL, (uint64_t)a.flat_rows, (uint64_t)a.B};
        const uint64_t strides[2] = {(uint64_t)kL * size, (uint64_t)a.flat_rows * kL * size};
        const uint32_t box[3] = {f32 ? 32u : 64u, 128, 1};
        e = encode_tmap(&o_map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                        a.o, dims, strides, box, true);
        if (e != cudaSuccess) return e;
    }
    if (a.pieces) {
        const uint64_t dims[3] = {(uint64_t)kL, (uint64_t)a.slab_rows, 2 * (uint64_t)a.shares * a.lanes};
        const uint64_t strides[2] = {(uint64_t)kL * 4, (uint64_t)a.slab_rows * kL * 4};
        const uint32_t box[3] = {32u, 128, 1};
        e = encode_tmap(&part_map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, a.part_o, dims, strides, box, true);
        if (e != cudaSuccess) return e;
    }
    a.units = (int64_t)a.B * a.tiles;
    const int64_t used = a.pieces ? (int64_t)a.shares * a.lanes : std::min<int64_t>(a.units, clusters);
    e = launch_pdl(kKernels[fp8][a.pieces != nullptr], dim3(4u * (unsigned)used), dim3(kThreads), kSmemBytes, s, k_map, v_map,
                   q_map, o_map, part_map, a);
    if (e != cudaSuccess || !a.pieces) return e;
    return launch_pdl(tree_merge_kernel, dim3(kMergeBlocks), dim3(kMergeThreads), 0, s, a);
}

}  // namespace mla
