// pages.cu -- the page-level steps of sparse decode: mean keys of cache pages, the choice of pages
// from their scores, and the page tables that the decode kernels read.
#include "internal.h"
#include "sm103_ptx.cuh"

namespace mla {
namespace {

// ------------------------------------------------------------------------------------------
// Mean key of every page that holds new tokens:
//     kbar[block, d] = 1/c sum_{i < c} K[block, i, d],   c = valid tokens of the page (1..64)
// One CTA per page. The 64 rows are read once: 72 threads cover a row (8 elements each), four
// such row groups take 16 rows each, and a thread's 16 row loads are all issued before any is
// used, so that a CTA keeps its whole page (74 KB) in flight. Sums in fp32 in a fixed order
// (rows of a group ascending, then the four groups), one rounding to bf16: the keys are a tensor-core
// operand of the score, and bf16 halves what that has to read. Bound by memory: 64 requests of 64 pages
// (238 MB) take 40 us, 5.9 TB/s; one new token in each of 128 requests takes 4.4 us, latency.
// ------------------------------------------------------------------------------------------
constexpr int kChunks = kD / 8;                   // 72 chunks of 8 elements in a row
constexpr int kGroups = 4;                        // row groups
constexpr int kRowsPer = kPage / kGroups;         // 16 rows of a group
constexpr int kKeyThreads = kChunks * kGroups;    // 288

template <bool kFp8>
__global__ void __launch_bounds__(kKeyThreads) page_keys_kernel(PageKeysArgs p) {
    __shared__ float part[kGroups - 1][kD];
    ptx::griddep_wait();  // the cache rows and lengths may be an earlier kernel's output
    ptx::griddep_launch_dependents();
    const int b = (int)(blockIdx.x / p.pages_per_req);
    const int off = (int)(blockIdx.x % p.pages_per_req);
    const int tid = threadIdx.x;
    int seq = p.seq_lens[b];
    int start = p.start_lens ? p.start_lens[b] : 0;
    const int64_t cap = (int64_t)p.max_blocks * kPage;
    if (start < 0) start = 0;
    if (seq < 0 || seq > cap || (int64_t)seq - start > p.max_new_len) {
        if (tid == 0 && off == 0 && p.dev_status) atomicOr(p.dev_status, MLA_DEV_SEQ_TOO_LONG);
        seq = seq < 0 ? 0 : (seq > cap ? (int)cap : seq);
    }
    const int page = start / kPage + off;
    if (seq <= start || page > (seq - 1) / kPage) return;
    const int valid = min(kPage, seq - page * kPage);
    const int32_t blk = p.block_table[(size_t)b * p.max_blocks + page];
    if (blk < 0 || (int64_t)blk >= p.num_blocks) {
        if (tid == 0 && p.dev_status) atomicOr(p.dev_status, MLA_DEV_BAD_BLOCK_ID);
        return;
    }
    const int chunk = tid % kChunks, grp = tid / kChunks;
    const int row0 = grp * kRowsPer;
    float acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.f;
    if constexpr (kFp8) {
        const uint8_t* src = p.cache + ((size_t)blk * kPage + row0) * kFp8RowBytes;
        uint2 v[kRowsPer];
        float ks[kRowsPer];
#pragma unroll
        for (int i = 0; i < kRowsPer; ++i) {
            v[i] = make_uint2(0u, 0u);
            ks[i] = 0.f;
            if (row0 + i < valid) {  // rows past the last token are not read: they may hold anything
                v[i] = *reinterpret_cast<const uint2*>(src + (size_t)i * kFp8RowBytes + 8 * chunk);
                ks[i] = *reinterpret_cast<const float*>(src + (size_t)i * kFp8RowBytes + kD);
            }
        }
#pragma unroll
        for (int i = 0; i < kRowsPer; ++i) {
            uint32_t h[4];  // as the decode kernels read the codes
            ptx::e4m3x4_to_bf16x4(v[i].x, h[0], h[1]);
            ptx::e4m3x4_to_bf16x4(v[i].y, h[2], h[3]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (row0 + i < valid) {
                    acc[2 * j] += ptx::bf16_lo_f(h[j]) * ks[i];
                    acc[2 * j + 1] += ptx::bf16_hi_f(h[j]) * ks[i];
                }
            }
        }
    } else {
        const uint8_t* src = p.cache + ((size_t)blk * kPage + row0) * kBf16RowBytes;
        uint4 v[kRowsPer];
#pragma unroll
        for (int i = 0; i < kRowsPer; ++i) {
            v[i] = make_uint4(0u, 0u, 0u, 0u);
            if (row0 + i < valid) v[i] = *reinterpret_cast<const uint4*>(src + (size_t)i * kBf16RowBytes + 16 * chunk);
        }
#pragma unroll
        for (int i = 0; i < kRowsPer; ++i) {
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[2 * j] += ptx::bf16_lo_f(w[j]);
                acc[2 * j + 1] += ptx::bf16_hi_f(w[j]);
            }
        }
    }
    if (grp > 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) part[grp - 1][8 * chunk + j] = acc[j];
    }
    __syncthreads();
    if (grp == 0) {
#pragma unroll
        for (int g = 0; g < kGroups - 1; ++g)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] += part[g][8 * chunk + j];
        const float c = (float)valid;
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = __fdiv_rn(acc[j], c);
        *reinterpret_cast<uint4*>(p.page_keys + (size_t)blk * kD + 8 * chunk) =
            make_uint4(ptx::pack_bf16x2(acc[0], acc[1]), ptx::pack_bf16x2(acc[2], acc[3]),
                       ptx::pack_bf16x2(acc[4], acc[5]), ptx::pack_bf16x2(acc[6], acc[7]));
    }
}

// ------------------------------------------------------------------------------------------
// Choice of pages. A row that sees n tokens has np = ceil(n / 64) pages. With np <= K all are
// taken; else the first `sink`, the last `local` and, of the others, the K - sink - local best
// scores (equal scores: the lower page; NaN below everything). The list is ascending, -1 behind.
//
// One CTA per row. Scores become order-preserving 32-bit keys, and the key T of the last page taken
// is found bit by bit from the top: T keeps a bit if at least `need` keys are >= T with it. Counting
// has no atomics (a histogram's would collide: scores share their exponents) and gives the same
// answer in any order. Bits that all keys share are skipped, and the search ends as soon as exactly
// `need` keys are >= T. A thread keeps kPer consecutive keys in registers: a pass is then mostly
// compares, where with four keys a thread its reductions and barriers took three times as long
// (256 rows of 2048 pages: 21 us, now 9.8, or 7.5 in a captured graph; 64 rows of 64 pages 2.5). Bound by
// the search's chain of up to 32 reductions and barriers; two bits a round, three counts each, gained 5 %
// there and lost 15 % on rows of 16384 pages. One scan then places the pages.
__device__ __forceinline__ uint32_t score_key(float x) {
    const uint32_t u = __float_as_uint(x);
    if ((u & 0x7fffffffu) > 0x7f800000u) return 0u;       // NaN
    const uint32_t z = (u << 1) == 0u ? 0u : u;           // -0 equals +0
    return (z & 0x80000000u) ? ~z : (z | 0x80000000u);    // never 0
}

// The sum of a warp-uniform-per-warp count over the block. `slot` alternates between two buffers, so that
// one barrier a call is enough.
__device__ __forceinline__ int block_count(int c, int (*buf)[32], int slot, int nw, int warp, int lane) {
    c = __reduce_add_sync(0xffffffffu, c);
    if (nw == 1) return c;
    if (lane == 0) buf[slot][warp] = c;
    __syncthreads();
    return __reduce_add_sync(0xffffffffu, lane < nw ? buf[slot][lane] : 0);
}

template <int kPer>
__global__ void __launch_bounds__(1024) select_pages_kernel(SelectArgs p) {
    __shared__ int s_cnt[2][32];
    __shared__ uint32_t s_and[32], s_or[32];
    __shared__ int2 s_scan[32];
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    const int r = (int)blockIdx.x, b = r / p.Sq, t = r % p.Sq;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x, nw = nt >> 5;
    int seq = p.seq_lens[b];
    if (seq < 0 || (int64_t)seq > (int64_t)p.width * kPage) {
        if (tid == 0 && p.dev_status) atomicOr(p.dev_status, MLA_DEV_SEQ_TOO_LONG);
        seq = seq < 0 ? 0 : p.width * kPage;
    }
    const int n = max(0, seq - (p.Sq - 1 - t));
    const int np = (n + kPage - 1) / kPage;
    int32_t* out = p.pages + (size_t)r * p.K;
    if (np <= p.K) {
        for (int i = tid; i < p.K; i += nt) out[i] = i < np ? i : -1;
        return;
    }
    const int c0 = p.sink, c1 = np - p.local;  // candidates [c0, c1): c1 - c0 > need
    const int need = p.K - p.sink - p.local;
    const float* src = p.scores + (size_t)r * p.stride;
    // This thread's pages i0 .. i0 + kPer - 1. Pages that are no candidates have key 0, which no trial
    // value counts (trials are > 0); a NaN candidate's key is 0 too, and T = 0 takes those last.
    const int i0 = tid * kPer;
    static_assert(kPer <= 32, "a bit a page below");
    uint32_t key[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int i = i0 + k;
        key[k] = i >= c0 && i < c1 ? score_key(src[i]) : 0u;
    }
    uint32_t T = 0;
    if (need > 0) {
        uint32_t all_and = 0xffffffffu, all_or = 0u;  // of the candidates' keys
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int i = i0 + k;
            if (i >= c0 && i < c1) {
                all_and &= key[k];
                all_or |= key[k];
            }
        }
        all_and = __reduce_and_sync(0xffffffffu, all_and);
        all_or = __reduce_or_sync(0xffffffffu, all_or);
        if (nw > 1) {
            if (lane == 0) {
                s_and[warp] = all_and;
                s_or[warp] = all_or;
            }
            __syncthreads();
            all_and = __reduce_and_sync(0xffffffffu, lane < nw ? s_and[lane] : 0xffffffffu);
            all_or = __reduce_or_sync(0xffffffffu, lane < nw ? s_or[lane] : 0u);
        }
        const uint32_t differ = all_and ^ all_or;
        const int top = differ ? 31 - __clz(differ) : -1;  // the highest bit in which two keys differ
        T = differ ? all_and & ~(0xffffffffu >> __clz(differ)) : all_and;  // what is above it
        for (int bit = top; bit >= 0; --bit) {
            const uint32_t trial = T | (1u << bit);
            int c = 0;
#pragma unroll
            for (int k = 0; k < kPer; ++k) c += key[k] >= trial ? 1 : 0;
            c = block_count(c, s_cnt, bit & 1, nw, warp, lane);
            if (c >= need) T = trial;
            if (c == need) break;
        }
    }
    // Pages above T (or forced) and those equal to T, in this thread's run of pages.
    uint32_t forced = 0, above = 0, equal = 0;  // one bit a page
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int i = i0 + k;
        if (i < np && (i < c0 || i >= c1)) forced |= 1u << k;
        if (need > 0 && i >= c0 && i < c1) {
            if (key[k] > T) above |= 1u << k;
            if (key[k] == T) equal |= 1u << k;
        }
    }
    above |= forced;
    const int na = __popc(above), ne = __popc(equal);
    int2 inc = make_int2(na, ne);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc.x, o), y = __shfl_up_sync(0xffffffffu, inc.y, o);
        if (lane >= o) {
            inc.x += x;
            inc.y += y;
        }
    }
    if (lane == 31) s_scan[warp] = inc;
    __syncthreads();
    int2 before = make_int2(inc.x - na, inc.y - ne), all = make_int2(0, 0);
    for (int w = 0; w < nw; ++w) {
        const int2 v = s_scan[w];
        if (w < warp) {
            before.x += v.x;
            before.y += v.y;
        }
        all.x += v.x;
    }
    const int ties = p.K - all.x;  // pages equal to T that are taken, the lowest first
    int at = before.x + min(before.y, ties), eq = before.y;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        bool take = (above >> k) & 1u;
        if ((equal >> k) & 1u) take = eq++ < ties;
        if (take) out[at++] = i0 + k;
    }
}

// ------------------------------------------------------------------------------------------
// Page tables of a sparse decode: row r's selected pages become the block table of a one-row
// request and its token count. An entry is taken if it is above every entry before it and inside
// the row's pages; -1 ends nothing and is skipped, any other entry is skipped and reported. The
// entries stay ascending, so only the last page can be a partial one. One warp a row: 128 rows of 32
// entries take 3.6 us, the latency of two dependent loads and a launch.
// ------------------------------------------------------------------------------------------
__global__ void __launch_bounds__(128) sparse_table_kernel(SparseTableArgs p) {
    const int r = (int)blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const bool live = r < p.B * p.Sq;
    const int b = live ? r / p.Sq : 0, t = live ? r % p.Sq : 0;
    ptx::griddep_wait();  // the lengths, too, may be a caller's kernel's output
    ptx::griddep_launch_dependents();
    if (!live) return;
    int seq = p.seq_lens[b];
    int next = lane < p.K ? p.pages[(size_t)r * p.K + lane] : -1;
    const int64_t cap = (int64_t)p.max_blocks * kPage;
    if (seq < 0 || seq > cap) {
        if (lane == 0 && p.dev_status) atomicOr(p.dev_status, MLA_DEV_SEQ_TOO_LONG);
        seq = seq < 0 ? 0 : (int)cap;
    }
    const int n = max(0, seq - (p.Sq - 1 - t));
    const int np = (n + kPage - 1) / kPage;
    int top = -1, count = 0;  // largest entry so far; entries taken
    for (int k0 = 0; k0 < p.K; k0 += 32) {
        const int e = next;
        next = lane < p.K - k0 - 32 ? p.pages[(size_t)r * p.K + k0 + 32 + lane] : -1;
        const int in = e < np ? e : -1;  // an entry outside the row's pages shadows none behind it
        int m = in;                      // inclusive running maximum
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, m, o);
            if (lane >= o) m = max(m, y);
        }
        int below = __shfl_up_sync(0xffffffffu, m, 1);
        below = lane == 0 ? top : max(top, below);
        const bool ok = in > below;  // below >= -1
        if (e != -1 && !ok && p.dev_status) atomicOr(p.dev_status, MLA_DEV_BAD_PAGE);
        const uint32_t mask = __ballot_sync(0xffffffffu, ok);
        if (ok)
            p.table[(size_t)r * p.K + count + __popc(mask & ((1u << lane) - 1u))] =
                p.block_table[(size_t)b * p.max_blocks + in];
        top = max(top, __shfl_sync(0xffffffffu, m, 31));
        count += __popc(mask);
    }
    if (lane == 0) p.lens[r] = count == 0 ? 0 : (count - 1) * kPage + (top == np - 1 ? n - (np - 1) * kPage : kPage);
}

}  // namespace

cudaError_t launch_page_keys(const PageKeysArgs& a, bool fp8, cudaStream_t s) {
    const dim3 grid((unsigned)((int64_t)a.B * a.pages_per_req));
    return fp8 ? launch_pdl(page_keys_kernel<true>, grid, dim3(kKeyThreads), 0, s, a)
               : launch_pdl(page_keys_kernel<false>, grid, dim3(kKeyThreads), 0, s, a);
}

cudaError_t launch_select_pages(const SelectArgs& a, cudaStream_t s) {
    // Two pages a thread while a row fits two warps, else 16, and 32 once 1024 threads do not reach.
    const int per = a.width <= 128 ? 2 : a.width <= 16384 ? 16 : 32;
    int threads = ((a.width + per - 1) / per + 31) / 32 * 32;
    if (threads < 32) threads = 32;
    auto* kernel = per == 2    ? select_pages_kernel<2>
                   : per == 16 ? select_pages_kernel<16>
                               : select_pages_kernel<32>;
    return launch_pdl(kernel, dim3((unsigned)(a.B * a.Sq)), dim3(threads), 0, s, a);
}

cudaError_t launch_sparse_table(const SparseTableArgs& a, cudaStream_t s) {
    return launch_pdl(sparse_table_kernel, dim3((unsigned)((a.B * a.Sq + 3) / 4)), dim3(128), 0, s, a);
}

}  // namespace mla
