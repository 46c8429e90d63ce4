// decode_common.cuh -- pieces shared by the two decode kernels (bf16 cache and FP8 cache):
// which query row and token range a work unit covers, and the per-page bookkeeping.
#pragma once

#include "internal.h"
#include "sm103_ptx.cuh"

namespace mla {
namespace dec {

// A running maximum before any score. Finite, so that the weight of a masked score (-inf) is
// exp2(-inf) = 0 from the start and only that of a NaN score is NaN.
constexpr float kNoMax = -3.402823466e38f;

struct RowGeom {
    int r, b, t, j0, j1, npages, page0;
    int slot;  // partial-output slot, or -1: this unit writes the row's final output
};

// Unit -> (query row, token range [j0, j1), partial slot). With a device-built schedule the
// unit list is the preceding kernel's output; otherwise unit = row * S + split and the range
// follows split_range.
__device__ __forceinline__ RowGeom row_geometry(const DecodeArgs& p, int unit, bool report) {
    RowGeom g;
    if (p.plan_units) {  // device-built schedule
        const int4 u = p.plan_units[unit];
        g.r = u.x;
        g.j0 = u.y;
        g.j1 = u.z;
        g.slot = u.w;
    } else {  // uniform splits: unit = row * S + split
        const int S = p.num_splits;
        int base;
        g.r = unit / S;
        split_range(visible_tokens(p, g.r, report, &base), S, unit % S, &g.j0, &g.j1);
        g.j0 += base;
        g.j1 += base;
        g.slot = S > 1 || p.all_partial ? unit : -1;
    }
    int q_len;
    row_request(p, g.r, &g.b, &g.t, &q_len);
    g.npages = (g.j1 - g.j0 + kPage - 1) / kPage;
    g.page0 = g.j0 / kPage;
    return g;
}

// Physical block of page `pg` of request b, or -1 (reported as MLA_DEV_BAD_BLOCK_ID) if the block-table
// entry is outside the cache.
__device__ __forceinline__ int page_block(const DecodeArgs& p, int b, int pg) {
    const int32_t blk = *table_entry(p, b, pg);
    if (blk < 0 || (int64_t)blk >= p.num_blocks) {
        if (p.dev_status) atomicOr(p.dev_status, MLA_DEV_BAD_BLOCK_ID);
        return -1;
    }
    return blk;
}

// Before a unit's output is written. By default the kernel ahead in the stream may still read the
// buffers, so its end is awaited. With kOrderFree nothing in flight touches them, and only the last
// unit waits: the grid must not end before the kernel ahead does, since the kernel behind waits for
// this grid alone and reads the other's output too.
__device__ __forceinline__ void output_wait(const DecodeArgs& p, int unit) {
    if (p.order == kOrderFree) {
        const int last = p.plan_units ? *p.plan_count - 1 : p.rows * p.num_splits - 1;
        if (unit != last) return;
    }
    ptx::griddep_wait();
}

// A bounded mbarrier wait taken by a whole warp: true only if every lane's wait succeeded.
template <bool kCluster = false>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort, int32_t* ds) {
    bool ok = ptx::wait_bar<kCluster>(bar, parity, abort, ds);
    return __all_sync(0xffffffffu, ok);
}

// One arrival for the whole warp, after what its lanes did (a lane each would be serialised at the barrier).
__device__ __forceinline__ void warp_arrive(uint32_t bar, int lane) {
    __syncwarp();
    if (lane == 0) ptx::bar_arrive(bar);
}

// A unit's output rows, O * inv from tensor memory, to global memory: 128 rows of 512 columns as
// panels of 128 bytes a row (32 fp32 or 64 bf16 columns), each written to a swizzled shared tile and
// stored by TMA as one box, so that global writes are whole lines. kSets sets of four warps (one
// warp per TMEM lane quarter) take the panels in turn; each set has kBufs tiles of its own, its own
// named barrier (kBar0 + set) and its own storing thread, so a set never waits for another and its
// stores overlap its next panels. (Two rounds of eight panels with a barrier of all warps and one
// storing thread took 6.3 us of a 22 us unit.) `off`: the tiles' place in shared memory, idle by now;
// rows with `zero` are written as 0, rows that are not `live` and panels without `store` not at all. The stores
// are complete at the end, without kComplete only their reads of the tiles.
constexpr int kTileBytes = 128 * 128;
template <bool kF32, int kSets, int kBufs, uint32_t kBar0, bool kComplete = true>
__device__ __forceinline__ void store_rows(uint8_t* smem, uint32_t sbase, int off, uint32_t taddr, int row, int set,
                                           bool issuer, bool live, bool zero, float inv, const void* map, int y, int z,
                                           bool store) {
    constexpr int kPanels = (kF32 ? 16 : 8) / kSets;
    uint32_t v[2][32];
    if (kF32) ptx::tmem_ld32(taddr + 32u * set, v[0]);
#pragma unroll
    for (int i = 0; i < kPanels; ++i) {
        const int panel = i * kSets + set;
        const int buf = off + (set * kBufs + i % kBufs) * kTileBytes;
        if (!kF32) {
            ptx::tmem_ld32(taddr + 64u * panel, v[0]);
            ptx::tmem_ld32(taddr + 64u * panel + 32u, v[1]);
        }
        ptx::tmem_wait_ld();
        if (kF32 && i + 1 < kPanels) ptx::tmem_ld32(taddr + 32u * (panel + kSets), v[(i + 1) & 1]);
        if (i >= kBufs) {  // the tile's previous store has read it
            if (issuer) ptx::bulk_wait_group_read<kBufs - 1>();
            ptx::named_bar(kBar0 + set, 128);
        }
        if (live) {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                if (!zero) {
                    if (kF32) {
                        const uint32_t* w = &v[i & 1][4 * c];
                        x = make_uint4(__float_as_uint(__uint_as_float(w[0]) * inv),
                                       __float_as_uint(__uint_as_float(w[1]) * inv),
                                       __float_as_uint(__uint_as_float(w[2]) * inv),
                                       __float_as_uint(__uint_as_float(w[3]) * inv));
                    } else {
                        const uint32_t* w = &v[c >> 2][8 * (c & 3)];
                        x = make_uint4(ptx::pack_bf16x2(__uint_as_float(w[0]) * inv, __uint_as_float(w[1]) * inv),
                                       ptx::pack_bf16x2(__uint_as_float(w[2]) * inv, __uint_as_float(w[3]) * inv),
                                       ptx::pack_bf16x2(__uint_as_float(w[4]) * inv, __uint_as_float(w[5]) * inv),
                                       ptx::pack_bf16x2(__uint_as_float(w[6]) * inv, __uint_as_float(w[7]) * inv));
                    }
                }
                *reinterpret_cast<uint4*>(smem + buf + row * 128 + ((c ^ (row & 7)) << 4)) = x;
            }
        }
        ptx::fence_proxy_async_cta();
        ptx::named_bar(kBar0 + set, 128);
        if (issuer && store) ptx::tma_store_3d(map, sbase + buf, panel * (kF32 ? 32 : 64), y, z);
        if (issuer) ptx::bulk_commit_group();
    }
    if (issuer) {
        if (kComplete)
            ptx::bulk_wait_group<0>();  // the stores are complete before the CTA exits
        else
            ptx::bulk_wait_group_read<0>();
    }
}

// Visible rows of the unit's page `page` (0 past its last page).
__device__ __forceinline__ int valid_rows(const RowGeom& g, int page) {
    return page < g.npages ? min(kPage, g.j1 - (g.j0 + kPage * page)) : 0;
}

// Infinities and NaNs among the eight bf16 at shared address `addr` become 0. For V rows of tokens that a row
// may not see: a weight of 0 would not keep them out of its sum. A row that does see such a token has a NaN
// score (or an infinite one that takes no part) and needs no help from V.
__device__ __forceinline__ void zero_nonfinite(uint32_t addr) {
    auto bad = [](uint32_t& w) -> bool {
        uint32_t x = w;
        if ((w & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
        if ((w & 0x7f800000u) == 0x7f800000u) x &= 0xffffu;
        const bool found = x != w;
        w = x;
        return found;
    };
    uint4 v = ptx::lds_u4(addr);
    if (bad(v.x) | bad(v.y) | bad(v.z) | bad(v.w)) ptx::sts_u4(addr, v);
}

}  // namespace dec
}  // namespace mla
