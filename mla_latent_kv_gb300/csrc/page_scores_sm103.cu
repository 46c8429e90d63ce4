// page_scores_sm103.cu -- the cheap score of every page for every query row:
//     score[r, j] = max_h scale * <q[r, h, 0:576], kbar[block_table[b, j], 0:576]>
// One page is scored once for all heads, since all heads read the same rows; a page matters if it
// matters to any of them.
//
// One CTA per (row, 128 pages), on the tensor cores "swapped": the pages are the M side and the
// heads the N side (16..128 of them), so that a thread of the epilogue owns one page and takes the
// maximum over heads in its own registers. The keys of the 128 pages are scattered rows of 1152
// bytes: four warps gather them with 16-byte asynchronous copies straight into the nine swizzled
// 64-dim panels (147 KB, all in flight at once), while q's panels come by TMA through a ring of
// four. Products of bf16 are exact in fp32, and the sums are fp32.
// Bound by latency: 8 rows of 2048 pages of 128 heads (128 CTAs) take 7.5 us, of which the gather's two
// dependent loads, nine panels of MMAs as they land and the launch are nearly all; 64 rows of 64 pages
// 7.1 us. The keys are 9 MB there, 1.4 us of memory bandwidth.
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

constexpr int kTile = 128;                     // pages of a CTA
constexpr int kPanels = kD / 64;               // 9 panels of 64 dims
constexpr int kPanelBytes = kTile * 128;       // 16 KB
constexpr int kQSlots = 4;
constexpr int kThreads = 192;                  // warps 0-3: gather, epilogue; 4: q by TMA; 5: MMA
constexpr int OFF_A = 1024;
constexpr int OFF_Q = OFF_A + kPanels * kPanelBytes;
constexpr int kSmem = OFF_Q + kQSlots * kPanelBytes;
static_assert(kSmem <= 232448, "over the per-CTA shared memory limit");
enum : int { B_AFULL = 0, B_QFULL = B_AFULL + kPanels, B_QEMPTY = B_QFULL + kQSlots, B_DONE = B_QEMPTY + kQSlots, B_COUNT };
constexpr int OFF_TMEM = 512, OFF_ABORT = 516;
constexpr uint32_t kTmemCols = 128;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16u : 0u) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// The larger of two values, NaN if either is one: a NaN key or query must not look like a number.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Panel P of this thread's key rows has landed: publish it to the MMA (async proxy).
template <int P>
__device__ __forceinline__ void publish_panels(uint32_t sbase) {
    if constexpr (P < kPanels) {
        cp_async_wait<kPanels - 1 - P>();
        fence_proxy_async_cta();
        bar_arrive(sbase + 8u * (B_AFULL + P));
        publish_panels<P + 1>(sbase);
    }
}

__global__ void __launch_bounds__(kThreads, 1)
    page_scores_kernel(const __grid_constant__ CUtensorMap q_map, const PageScoresArgs p, int tiles, uint32_t idesc) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_addr(smem);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int r = (int)(blockIdx.x / tiles), tile = (int)(blockIdx.x % tiles);
    const int b = r / p.Sq, t = r % p.Sq;
    volatile int* abort = reinterpret_cast<volatile int*>(smem + OFF_ABORT);
    int32_t* ds = p.dev_status;
    auto bar = [&](int i) -> uint32_t { return sbase + 8u * (uint32_t)i; };
    if (warp == 4 && lane == 0) {
        tma_prefetch_desc(&q_map);
        *abort = 0;
        for (int i = 0; i < B_COUNT; ++i) bar_init(bar(i), i < B_QFULL ? 128u : 1u);
        fence_barrier_init();
    }
    if (warp == 5) {
        tmem_alloc(sbase + OFF_TMEM, kTmemCols);
        tmem_relinquish();
    }
    griddep_wait();  // q, the keys and the lengths may be earlier kernels' outputs
    griddep_launch_dependents();
    int seq = p.seq_lens[b];
    if (seq < 0 || seq > p.max_seq_len) {
        if (tid == 0 && tile == 0 && p.dev_status) atomicOr(p.dev_status, MLA_DEV_SEQ_TOO_LONG);
        seq = seq < 0 ? 0 : p.max_seq_len;
    }
    const int n = max(0, seq - (p.Sq - 1 - t));
    const int np = (n + kPage - 1) / kPage;
    const int first = tile * kTile;
    float* out = p.scores + (size_t)r * p.width;
    const bool misplaced = (sbase & 1023u) != 0;  // the swizzled tiles need 1024-byte alignment; never expected
    if (first >= np || misplaced) {                // no page in sight
        for (int i = first + tid; i < min(p.width, first + kTile); i += kThreads) out[i] = -CUDART_INF_F;
        if (misplaced && tid == 0 && ds) atomicOr(ds, MLA_DEV_WAIT_TIMEOUT);
        __syncthreads();
        if (warp == 5) tmem_dealloc(*reinterpret_cast<volatile uint32_t*>(smem + OFF_TMEM), kTmemCols);
        return;
    }
    const int live = min(kTile, np - first);
    uint32_t bad = 0;  // bit i: row i of this thread has no block
    if (warp < 4) {
        // eight threads cover a 128-byte panel row; this thread's rows are tid / 8 + 16 i
        const int c = tid & 7, row0 = tid >> 3;
        const uint16_t* src[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int row = row0 + 16 * i;
            int blk = row < live ? p.block_table[(size_t)b * p.max_blocks + first + row] : -1;
            if (blk < 0 || (int64_t)blk >= p.num_blocks) {
                if (row < live && ds) atomicOr(ds, MLA_DEV_BAD_BLOCK_ID);
                bad |= 1u << i;
                blk = 0;
            }
            src[i] = p.page_keys + (size_t)blk * kD + 8 * c;
        }
#pragma unroll 1
        for (int pn = 0; pn < kPanels; ++pn) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int row = row0 + 16 * i;
                cp_async16(sbase + OFF_A + pn * kPanelBytes + row * 128 + ((c ^ (row & 7)) << 4), src[i] + 64 * pn,
                           !((bad >> i) & 1u));
            }
            cp_async_commit();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(smem + OFF_TMEM), 0);
    const int nq = (p.H + 15) / 16 * 16;  // rows of a q panel: the heads, rounded up to the MMA's N
    if (warp == 4) {
        if (lane == 0) {
            bool ok = true;
            int issued = 0;
            for (int pn = 0; pn < kPanels && ok; ++pn) {
                const int slot = pn % kQSlots;
                if (pn >= kQSlots && !(ok = wait_bar(bar(B_QEMPTY + slot), (pn / kQSlots - 1) & 1, abort, ds))) break;
                bar_arrive_expect_tx(bar(B_QFULL + slot), (uint32_t)nq * 128u);
                tma_load_2d(sbase + OFF_Q + slot * kPanelBytes, &q_map, bar(B_QFULL + slot), pn * 64, r * p.H);
                ++issued;
            }
            if (*abort)  // let the copies in flight land before the CTA can exit
                for (int m = max(0, issued - kQSlots); m < issued; ++m) {
                    volatile int dummy = 0;
                    wait_bar(bar(B_QFULL + m % kQSlots), (m / kQSlots) & 1, &dummy, nullptr);
                }
        }
    } else if (warp == 5) {
        // the whole warp runs the loop and one elected lane issues (see the decode kernel)
        const bool leader = elect_one();
        bool ok = true;
        int done = 0;
#pragma unroll
        for (int pn = 0; pn < kPanels; ++pn) {
            constexpr int kStep = 32 >> 4;  // of a descriptor, 16 dims on
            const int slot = pn % kQSlots;
            if (ok) ok = dec::warp_wait(bar(B_QFULL + slot), (pn / kQSlots) & 1, abort, ds);
            if (ok) ok = dec::warp_wait(bar(B_AFULL + pn), 0, abort, ds);
            if (!ok) continue;
            const uint64_t a0 = smem_desc_sw128(sbase + OFF_A + pn * kPanelBytes, 16, 1024);
            const uint64_t b0 = smem_desc_sw128(sbase + OFF_Q + slot * kPanelBytes, 16, 1024);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (leader) mma_ss(tmem, a0 + (uint64_t)(kStep * k), b0 + (uint64_t)(kStep * k), idesc, (pn | k) ? 1u : 0u);
            if (leader) mma_commit(bar(B_QEMPTY + slot));
            ++done;
        }
        if (leader) mma_commit(bar(B_DONE));
        for (int m = max(0, done - kQSlots); m < done; ++m) {  // the last commits land before teardown
            volatile int dummy = 0;
            dec::warp_wait(bar(B_QEMPTY + m % kQSlots), (m / kQSlots) & 1, &dummy, nullptr);
        }
    } else {
        publish_panels<0>(sbase);
        const bool ok = __all_sync(0xffffffffu, wait_bar(bar(B_DONE), 0, abort, ds));
        tc_fence_after();
        float best = -CUDART_INF_F;
        const uint32_t lane_base = (uint32_t)(32 * warp) << 16;
        for (int h0 = 0; h0 < p.H; h0 += 32) {
            uint32_t v[32];
            tmem_ld32(tmem + lane_base + (uint32_t)h0, v);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (h0 + j < p.H) best = max_nan(best, __uint_as_float(v[j]));
        }
        // page `row` of the tile was gathered by threads 8 (row % 16) ..: its validity again
        const int row = tid;
        float s = -CUDART_INF_F;
        if (row < live && ok) {
            const int blk = p.block_table[(size_t)b * p.max_blocks + first + row];
            if (blk >= 0 && (int64_t)blk < p.num_blocks) s = best * p.scale;
        }
        if (first + row < p.width) out[first + row] = s;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 5) tmem_dealloc(tmem, kTmemCols);
}

int g_attr_done[64] = {};

}  // namespace

cudaError_t launch_page_scores(const PageScoresArgs& a, cudaStream_t s) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !g_attr_done[dev]) {
        e = cudaFuncSetAttribute(page_scores_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        if (dev < 64) g_attr_done[dev] = 1;
    }
    const int nq = (a.H + 15) / 16 * 16;
    CUtensorMap q_map;
    memset(&q_map, 0, sizeof q_map);
    const uint64_t dims[2] = {(uint64_t)kD, (uint64_t)a.B * a.Sq * a.H};
    const uint64_t strides[1] = {(uint64_t)kD * 2};
    const uint32_t box[2] = {64, (uint32_t)nq};
    e = encode_tmap(&q_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.q, dims, strides, box, true);
    if (e != cudaSuccess) return e;
    const int tiles = (a.width + kTile - 1) / kTile;
    return launch_pdl(page_scores_kernel, dim3((unsigned)((int64_t)a.B * a.Sq * tiles)), dim3(kThreads), kSmem, s,
                      q_map, a, tiles, idesc_bf16_f32(128, nq, false, false));
}

}  // namespace mla
