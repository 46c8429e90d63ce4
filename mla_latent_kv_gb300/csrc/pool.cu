// pool.cu -- the page pool between decode steps: accepted drafts moved to the front of their request
// (mla_accept_tokens), and one state of the pool made from another (mla_fork_pages).
//
// Both are copies of whole cache rows with a little bookkeeping on the device, so that a step that decides
// there (how many drafts were accepted, which beams go on) needs no host in between. Bound: latency; the
// rows moved are a few per request and layer. Measured, one call after another: 64 accepted branches in sixteen
// layers 2.5 us; a beam search's step of 128 rows in sixteen layers, 23 MB moved, 11.5 us (its two kernels 5.5
// and 6), four answers from one request 8.6. In a pool of which 95% is held the search adds: 60,000 pages 12 us
// in all, a million 62, 3.8 million 210 (one step's counts at a time 18.5, 189 and 696; small pools 0.7 less).
//
// No kernel that writes cache rows, block tables or lengths signals its dependents early: a decode reads them
// before its own wait.
#include <climits>

#include "internal.h"
#include "sm103_ptx.cuh"

namespace mla {
namespace {

// ------------------------------------------------------------------------------------------
// Accepted drafts. Draft path[i] of a request moves to place i behind the tokens before its drafts. The path
// ascends, so place i <= path[i]: rows are read and written in order, and no row is overwritten before it
// was read. One block per (request, layer); a thread owns one column chunk of the rows and moves eight rows
// at a time, all of their loads first.
// ------------------------------------------------------------------------------------------
constexpr int kAcceptThreads = 96;  // >= 73 chunks and >= 64 drafts
constexpr int kAcceptBatch = 8;

template <class Chunk, int kRowBytes>
__global__ void __launch_bounds__(kAcceptThreads) accept_kernel(const AcceptArgs p) {
    constexpr int kChunks = kRowBytes / (int)sizeof(Chunk);
    static_assert(kChunks * (int)sizeof(Chunk) == kRowBytes && kChunks <= kAcceptThreads, "chunks of a row");
    ptx::griddep_wait();
    const int b = (int)blockIdx.x, layer = (int)blockIdx.y, tid = threadIdx.x;
    __shared__ int n_s;
    __shared__ int64_t src_s[kTreeMaxDrafts], dst_s[kTreeMaxDrafts];  // rows of the cache
    const int cap = p.max_blocks * kPage;
    int seq = p.seq_lens[b];
    const bool bad_len = seq < 0 || seq > cap;
    seq = min(max(seq, 0), cap);
    const int first = max(seq - p.Sq, 0);       // tokens before the drafts
    const int gone = max(p.Sq - seq, 0);        // drafts that are not there: the first ones
    const int want = p.counts[b];
    if (tid == 0) n_s = min(max(want, 0), p.Sq);
    __syncthreads();
    int place = -1;
    if (tid < p.Sq && tid < want) {
        place = p.path[(size_t)b * p.Sq + tid];
        const int before = tid > 0 ? p.path[(size_t)b * p.Sq + tid - 1] : gone - 1;
        if (place <= before || place >= p.Sq) atomicMin(&n_s, tid);
    }
    __syncthreads();
    const int n = n_s;
    bool bad_block = false;
    if (tid < n) {
        auto row_of = [&](int token) -> int64_t {
            const int32_t blk = p.block_table[(size_t)b * p.max_blocks + token / kPage];
            return blk < 0 || (int64_t)blk >= p.num_blocks ? -1 : (int64_t)blk * kPage + token % kPage;
        };
        const int64_t s = row_of(seq - p.Sq + place), d = row_of(first + tid);
        bad_block = s < 0 || d < 0;
        src_s[tid] = s;
        dst_s[tid] = bad_block || s == d ? -1 : d;
    }
    __syncthreads();
    if (layer == 0) {
        if (tid == 0) {
            p.new_lens[b] = first + n;
            int bits = (bad_len ? MLA_DEV_SEQ_TOO_LONG : 0) | (n != want ? MLA_DEV_BAD_BRANCH : 0);
            if (bits && p.dev_status) atomicOr(p.dev_status, bits);
        }
        if (bad_block && p.dev_status) atomicOr(p.dev_status, MLA_DEV_BAD_BLOCK_ID);
    }
    if (tid >= kChunks) return;
    uint8_t* base = p.cache + (size_t)layer * p.num_blocks * (kPage * kRowBytes) + tid * sizeof(Chunk);
    for (int i0 = 0; i0 < n; i0 += kAcceptBatch) {
        Chunk v[kAcceptBatch];
#pragma unroll
        for (int u = 0; u < kAcceptBatch; ++u)
            if (i0 + u < n && dst_s[i0 + u] >= 0) v[u] = *reinterpret_cast<const Chunk*>(base + src_s[i0 + u] * kRowBytes);
#pragma unroll
        for (int u = 0; u < kAcceptBatch; ++u)
            if (i0 + u < n && dst_s[i0 + u] >= 0) *reinterpret_cast<Chunk*>(base + dst_s[i0 + u] * kRowBytes) = v[u];
    }
}

// ------------------------------------------------------------------------------------------
// The pool's next state. The plan kernel's block 0 finds each old row's heir (its first child), counts the
// pages every new row has to take and finds that many free ones, lowest first; its other blocks copy the
// reference counts. The second kernel writes the new rows, applies the changes of the counts (sums of +1
// and -1, in any order) and copies the rows of pages that are held in part by more than one.
// ------------------------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;
constexpr int kRefsPerThread = 8;  // of a step of the free-page search
constexpr int kSteps = 4;          // steps whose counts are on their way
constexpr int kFewPages = 4;       // pages behind a row's whole ones that one thread looks at
constexpr int kForkThreads = 256;
constexpr int kCopyBatch = 5;  // 16-byte loads of a thread in flight

// Whether the heir of an old row keeps the row's page j: the pages full of tokens that it may share, and of
// the others those that nobody else holds (tokens will be written there).
__device__ __forceinline__ bool heir_keeps(const ForkArgs& p, const int32_t* row, int j, int whole, int held, int need) {
    if (j < whole) return true;
    if (j >= held || j >= need) return false;
    const int32_t page = row[j];
    return page >= 0 && (int64_t)page < p.num_blocks && p.refs[page] == 1;
}

// Exclusive prefix sum of v over the block's threads, and the total.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = (int)blockDim.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int s = lane < warps ? warp_sums[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        if (lane < warps) warp_sums[lane] = s;
    }
    __syncthreads();
    const int base = warp > 0 ? warp_sums[warp - 1] : 0;
    *total = warp_sums[warps - 1];
    __syncthreads();
    return base + x - v;
}

__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const ForkArgs p) {
    ptx::griddep_wait();
    // The second kernel waits for this one before anything else, and the kernel behind it for that one, which
    // signals nothing: it may be scheduled now.
    ptx::griddep_launch_dependents();
    const int tid = threadIdx.x;
    if (blockIdx.x > 0) {
        const int64_t step = (int64_t)(gridDim.x - 1) * kPlanThreads;
        for (int64_t i = (int64_t)(blockIdx.x - 1) * kPlanThreads + tid; i < p.num_blocks; i += step) p.new_refs[i] = p.refs[i];
        return;
    }
    __shared__ int heir_s[kMaxPoolRows];
    __shared__ int sums[kPlanThreads / 32];
    __shared__ int bits_s, long_s;
    // The counts of the thread's pages of a step, and a bit for each that is free. The first step's are loaded here, so
    // that they have arrived when they are needed.
    const bool wide = (reinterpret_cast<uintptr_t>(p.refs) & 15u) == 0;
    struct Counts {
        int4 a, b;
    };
    auto load_counts = [&](int64_t step) -> Counts {
        const int64_t i = (step * kPlanThreads + tid) * kRefsPerThread;
        Counts c;
        c.a = c.b = make_int4(1, 1, 1, 1);
        if (wide && i + kRefsPerThread <= p.num_blocks) {
            c.a = reinterpret_cast<const int4*>(p.refs + i)[0];
            c.b = reinterpret_cast<const int4*>(p.refs + i)[1];
        } else if (i < p.num_blocks) {
            int* x[kRefsPerThread] = {&c.a.x, &c.a.y, &c.a.z, &c.a.w, &c.b.x, &c.b.y, &c.b.z, &c.b.w};
#pragma unroll
            for (int k = 0; k < kRefsPerThread; ++k)
                if (i + k < p.num_blocks) *x[k] = p.refs[i + k];
        }
        return c;
    };
    auto free_pages = [](const Counts& c) -> uint32_t {
        return (uint32_t)((c.a.x == 0) | (c.a.y == 0) << 1 | (c.a.z == 0) << 2 | (c.a.w == 0) << 3 | (c.b.x == 0) << 4 |
                          (c.b.y == 0) << 5 | (c.b.z == 0) << 6 | (c.b.w == 0) << 7);
    };
    const Counts first_step = load_counts(0);
    if (tid == 0) bits_s = long_s = 0;
    for (int b = tid; b < p.B; b += kPlanThreads) heir_s[b] = INT_MAX;
    __syncthreads();
    for (int r = tid; r < p.B2; r += kPlanThreads) {
        const int parent = p.parents[r];
        if (parent >= p.B || parent < -1)
            atomicOr(&bits_s, MLA_DEV_BAD_PARENT);
        else if (parent >= 0)
            atomicMin(&heir_s[parent], r);
    }
    __syncthreads();
    for (int b = tid; b < p.B; b += kPlanThreads) {
        p.heirs[b] = heir_s[b] == INT_MAX ? -1 : heir_s[b];
        const int n = p.lens[b], held = p.counts[b];
        if (n < 0 || held < 0 || held > p.max_blocks || (n + (int64_t)kPage - 1) / kPage > held)
            atomicOr(&bits_s, MLA_DEV_SEQ_TOO_LONG);
    }
    __syncthreads();
    if (bits_s == 0) {  // parents and lengths are good
        for (int r = tid; r < p.B2; r += kPlanThreads) {
            const int parent = p.parents[r], room = p.room[r];
            const int n = parent >= 0 ? p.lens[parent] : 0, held = parent >= 0 ? p.counts[parent] : 0;
            const int whole = n / kPage;
            const int64_t want = ((int64_t)max(n, room) + kPage - 1) / kPage;
            const int need = (int)min(want, (int64_t)p.max_blocks);
            if (want > p.max_blocks) atomicOr(&bits_s, MLA_DEV_SEQ_TOO_LONG);
            const bool heir = parent >= 0 && heir_s[parent] == r;
            const int32_t* row = p.table + (size_t)max(parent, 0) * p.max_blocks;
            int take = need - whole;
            bool first = false;  // the page behind the whole ones is kept
            // usually one or two pages: the one held in part, and room
            const int behind = heir ? min(held, need) - whole : 0;
            if (behind > kFewPages) long_s = 1;
            for (int j = whole; behind <= kFewPages && j < whole + behind; ++j)
                if (heir_keeps(p, row, j, whole, held, need)) {
                    --take;
                    first |= j == whole;
                }
            if (behind > kFewPages) first = heir_keeps(p, row, whole, whole, held, need);
            const bool copy = n % kPage && !first;
            p.rows[r] = make_int4(parent, need, take, heir ? 1 : 0);
            // where its rows come from; where they go is known later
            p.copies[r] = make_int4(copy ? row[whole] : -1, 0, copy ? n % kPage : 0, 0);
        }
    }
    __syncthreads();
    if (bits_s == 0 && long_s)  // rows with much room: a warp each (2000 pages by one thread take milliseconds)
        for (int r = tid >> 5; r < p.B2; r += kPlanThreads / 32) {
            const int4 rec = p.rows[r];
            if (!rec.w) continue;
            const int held = p.counts[rec.x], whole = p.lens[rec.x] / kPage, end = min(held, rec.y);
            if (end - whole <= kFewPages) continue;
            const int32_t* row = p.table + (size_t)rec.x * p.max_blocks;
            int kept = 0;
            for (int j = whole + (tid & 31); j < end; j += 32) kept += heir_keeps(p, row, j, whole, held, rec.y);
            kept = __reduce_add_sync(0xffffffffu, kept);
            if ((tid & 31) == 0) p.rows[r].z -= kept;
        }
    __syncthreads();
    int total = 0;
    if (bits_s == 0) {
        for (int r0 = 0; r0 < p.B2; r0 += kPlanThreads) {  // takes -> first of the taken pages
            const int r = r0 + tid;
            int sum;
            const int at = total + block_scan(r < p.B2 ? p.rows[r].z : 0, sums, &sum);
            if (r < p.B2) p.rows[r].z = at;
            // more than there are pages, at the latest after this many rows: no overflow below
            total = (int)min((int64_t)total + sum, (int64_t)INT_MAX / 2);
        }
        int got = 0;
        const int64_t steps = (p.num_blocks + kPlanThreads * kRefsPerThread - 1) / (kPlanThreads * kRefsPerThread);
        uint32_t ahead[kSteps] = {free_pages(first_step), 0u, 0u, 0u};
        static_assert(kSteps == 4, "the lists of four");
        for (int64_t s0 = 0; s0 < steps && got < total; s0 += kSteps) {
            uint32_t now[kSteps];
#pragma unroll
            for (int k = 0; k < kSteps; ++k) now[k] = ahead[k];
            if (s0 == 0 && steps > 1) {
#pragma unroll
                for (int k = 1; k < kSteps; ++k) now[k] = free_pages(load_counts(k));
            }
            if (s0 + kSteps < steps) {
#pragma unroll
                for (int k = 0; k < kSteps; ++k) ahead[k] = free_pages(load_counts(s0 + k + kSteps));
            }
#pragma unroll 1
            for (int k = 0; k < kSteps && got < total; ++k) {
                uint32_t free = k == 0 ? now[0] : k == 1 ? now[1] : k == 2 ? now[2] : now[3];
                if (!__syncthreads_or((int)free)) continue;  // all held
                int sum;
                int to = got + block_scan(__popc(free), sums, &sum);
                const int64_t first = ((s0 + k) * kPlanThreads + tid) * kRefsPerThread;
                for (; free; free &= free - 1, ++to)
                    if (to < total) p.fresh[to] = (int32_t)(first + __ffs(free) - 1);
                got += sum;
            }
        }
        if (tid == 0 && got < total) atomicOr(&bits_s, MLA_DEV_NO_PAGES);
        __syncthreads();
        // a copied page is the first that its row takes
        for (int r = tid; r < p.B2 && bits_s == 0; r += kPlanThreads)
            if (p.copies[r].z > 0) p.copies[r].y = p.fresh[p.rows[r].z];
    }
    __syncthreads();
    if (tid == 0) {
        p.head[0] = bits_s != 0;
        if (bits_s && p.dev_status) atomicOr(p.dev_status, bits_s);
    }
}

template <int kRowBytes>
__global__ void __launch_bounds__(kForkThreads) fork_apply_kernel(const ForkArgs p) {
    ptx::griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool failed = p.head[0] != 0;
    int64_t u = blockIdx.x;
    auto in_pool = [&](int32_t page) -> bool {
        const bool ok = page >= 0 && (int64_t)page < p.num_blocks;
        if (!ok && p.dev_status) atomicOr(p.dev_status, MLA_DEV_BAD_BLOCK_ID);
        return ok;
    };
    if (u < p.B2) {  // ---- a new row
        __shared__ int counts[kForkThreads / 32];
        const int r = (int)u;
        int32_t* to = p.new_table + (size_t)r * p.max_blocks;
        const int4 rec = failed ? make_int4(-1, 0, 0, 0) : p.rows[r];
        const int n = rec.x >= 0 ? p.lens[rec.x] : 0, held = rec.x >= 0 ? p.counts[rec.x] : 0;
        const int whole = n / kPage, need = rec.y;
        const bool heir = rec.w != 0;
        const int32_t* from = p.table + (size_t)max(rec.x, 0) * p.max_blocks;
        int taken = rec.z;
        for (int j0 = 0; j0 < p.max_blocks; j0 += kForkThreads) {
            const int j = j0 + tid;
            const bool keep = j < need && (heir ? heir_keeps(p, from, j, whole, held, need) : j < whole);
            const bool take = j < need && !keep;
            // this page's place among the taken ones
            const uint32_t takes = __ballot_sync(0xffffffffu, take);
            if (lane == 0) counts[warp] = __popc(takes);
            __syncthreads();
            int at = taken + __popc(takes & ((1u << lane) - 1u));
            for (int w = 0; w < kForkThreads / 32; ++w) {
                if (w < warp) at += counts[w];
                taken += counts[w];
            }
            __syncthreads();
            if (j >= p.max_blocks) continue;
            int32_t page = -1;
            if (keep) page = from[j];
            if (take) page = p.fresh[at];
            // the heir's kept pages were looked at by nobody else: reported here, and counted already
            if ((take || keep) && in_pool(page) && !(keep && heir)) atomicAdd(p.new_refs + page, 1);
            to[j] = page;
        }
        if (tid == 0) {
            p.new_counts[r] = need;
            p.new_lens[r] = n;
        }
        return;
    }
    if (failed) return;
    u -= p.B2;
    if (u < p.B) {  // ---- an old row: what its heir does not keep is given back
        const int b = (int)u, r = p.heirs[b];
        const int held = p.counts[b], whole = r >= 0 ? p.lens[b] / kPage : 0, need = r >= 0 ? p.rows[r].y : 0;
        const int32_t* row = p.table + (size_t)b * p.max_blocks;
        for (int j = (r >= 0 ? whole : 0) + tid; j < held; j += kForkThreads)
            if (!(r >= 0 && heir_keeps(p, row, j, whole, held, need)) && in_pool(row[j])) atomicSub(p.new_refs + row[j], 1);
        return;
    }
    u -= p.B;  // ---- a new row's copied page, in one layer
    const int r = (int)(u / p.layers), layer = (int)(u % p.layers);
    const int4 rec = p.copies[r];
    const int bytes = rec.z * kRowBytes;
    if (bytes == 0 || !in_pool(rec.x)) return;
    constexpr size_t kPageBytes = (size_t)kPage * kRowBytes;
    const uint8_t* src = p.cache + ((size_t)layer * p.num_blocks + rec.x) * kPageBytes;
    uint8_t* dst = p.cache + ((size_t)layer * p.num_blocks + rec.y) * kPageBytes;
    for (int at = tid * 16; at + 16 <= bytes; at += kForkThreads * kCopyBatch * 16) {
        uint4 v[kCopyBatch];
#pragma unroll
        for (int k = 0; k < kCopyBatch; ++k)
            if (at + k * kForkThreads * 16 + 16 <= bytes) v[k] = *reinterpret_cast<const uint4*>(src + at + k * kForkThreads * 16);
#pragma unroll
        for (int k = 0; k < kCopyBatch; ++k)
            if (at + k * kForkThreads * 16 + 16 <= bytes) *reinterpret_cast<uint4*>(dst + at + k * kForkThreads * 16) = v[k];
    }
    if (kRowBytes % 16 && tid == 0 && bytes % 16)  // rows of 584 bytes: an odd number of 8-byte words
        *reinterpret_cast<uint2*>(dst + bytes - 8) = *reinterpret_cast<const uint2*>(src + bytes - 8);
}

}  // namespace

cudaError_t launch_accept_tokens(const AcceptArgs& a, bool fp8, cudaStream_t s) {
    return launch_pdl(fp8 ? accept_kernel<uint2, kFp8RowBytes> : accept_kernel<uint4, kBf16RowBytes>,
                      dim3((unsigned)a.B, (unsigned)a.layers), dim3(kAcceptThreads), 0, s, a);
}

cudaError_t launch_fork_pages(const ForkArgs& a, bool fp8, cudaStream_t s) {
    const int64_t refs = (a.num_blocks + kPlanThreads - 1) / kPlanThreads;
    cudaError_t e = launch_pdl(fork_plan_kernel, dim3((unsigned)(1 + (refs < 64 ? refs : 64))), dim3(kPlanThreads), 0, s, a);
    if (e != cudaSuccess) return e;
    const int64_t blocks = (int64_t)a.B2 + a.B + (int64_t)a.B2 * a.layers;
    if (blocks == 0) return cudaSuccess;  // the counts alone were copied
    return launch_pdl(fp8 ? fork_apply_kernel<kFp8RowBytes> : fork_apply_kernel<kBf16RowBytes>, dim3((unsigned)blocks),
                      dim3(kForkThreads), 0, s, a);
}

}  // namespace mla
