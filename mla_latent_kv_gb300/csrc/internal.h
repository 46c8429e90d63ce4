// internal.h -- shared declarations of the CUDA library (not part of the public ABI).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "mla_latent_kv.h"

namespace mla {

constexpr int kL = MLA_KV_LORA_RANK;  // 512 latent dims (also the V width)
constexpr int kR = MLA_ROPE_DIM;      // 64 rope dims
constexpr int kD = MLA_HEAD_DIM;      // 576 = one cached row / one absorbed query
constexpr int kP = MLA_NOPE_DIM;      // 128
constexpr int kV = MLA_V_DIM;         // 128
constexpr int kPage = MLA_PAGE_SIZE;  // 64 tokens per page
constexpr int kBf16RowBytes = 2 * kD; // 1152
constexpr int kFp8RowBytes = kD + 8;  // 584

// What a decode kernel may read before the kernel ahead of it in the stream has ended: cache, block
// table and lengths (the default: no kernel of the library that signals early writes them; q and a
// device-built schedule wait), nothing (the one ahead writes the lengths and the block table), or everything
// (the one ahead began only after all before it had ended, and writes nothing that is read here:
// the second of two kernels that run side by side).
enum { kOrderDefault = 0, kOrderWaitFirst = 1, kOrderFree = 2 };

// Everything a decode launch needs, resolved and validated on the host.
struct DecodeArgs {
    const uint16_t* q;          // bf16 [B, Sq, H, 576]
    const uint8_t* cache;       // [num_blocks, 64, row_bytes]
    int kv_dtype;
    int64_t num_blocks;
    const int32_t* block_table; // [B, max_blocks]
    int max_blocks;
    const int32_t* seq_lens;    // [B]
    int max_seq_len;
    int B, Sq, H;               // requests, uniform query rows per request (1 for packed rows), heads
    int rows;                   // query rows: B * Sq, or the packed total
    const int32_t* qsl;         // packed rows: request b owns rows [qsl[b], qsl[b + 1]); else null
    float scale;
    int num_splits;             // resolved, >= 1
    int shared_pages;           // the first pages of every request are those of block_table's row 0
    int base;                   // tokens (whole pages) at the front of every request that are left out;
    int base_step;              // a row that sees only a part of them leaves out whole multiples of this
    int all_partial;            // every unit writes a partial state, also the only one of its row
    int order;                  // kOrder*: what the kernel may read before the preceding one ends
    const float* pre_o;         // partial states of every row over the base tokens, merged with the
    const float* pre_lse;       // row's own: [pre_splits, rows, H, 512] and [pre_splits, rows, H]
    int pre_splits;             // (0: none)
    float* part_o;              // [B*Sq, S, H, 512] fp32 (num_splits > 1)
    float* part_lse;            // [B*Sq, S, H]     fp32 (num_splits > 1)
    void* o_latent;             // [B, Sq, H, 512]
    int o_dtype;                // mla_dtype
    float* lse;                 // [B, Sq, H] or null
    int32_t* dev_status;        // or null
    // Device-built schedule (num_splits == -2): unit u covers tokens [y, z) of query row x and
    // writes partial slot w (-1: the row's final output); row r's partials are slots
    // [rows[r].x, rows[r].x + rows[r].y) when rows[r].y > 1. Null in the uniform-split modes.
    const int4* plan_units;
    const int2* plan_rows;
    const int* plan_count;      // [0] units actually planned, [1] split rows (rows with partials)
    const int* plan_split_rows; // the split rows' indices, plan_count[1] of them
    int plan_max_units;         // the grid is sized for this many units
};

// Request b, position t and query length of query row r: uniform rows are r = b * Sq + t;
// packed rows belong to the last request whose first row is <= r (binary search of qsl).
__device__ __forceinline__ void row_request(const DecodeArgs& p, int r, int* b, int* t, int* q_len) {
    if (p.qsl == nullptr) {
        *b = r / p.Sq;
        *t = r % p.Sq;
        *q_len = p.Sq;
        return;
    }
    int lo = 0, hi = p.B - 1;  // invariant: qsl[lo] <= r
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.qsl[mid] <= r)
            lo = mid;
        else
            hi = mid - 1;
    }
    *b = lo;
    *t = r - p.qsl[lo];
    *q_len = p.qsl[lo + 1] - p.qsl[lo];
}

// Visible tokens of query row r past its base, and that base in *base: the row sees
// n = seq_len - (q_len - 1 - t) tokens, clamped at 0, with seq_len clamped to what the block table can
// hold, and leaves out the first p.base of them or, if it sees fewer, the ranges of base_step tokens that
// it sees whole. An out-of-range seq_len sets MLA_DEV_SEQ_TOO_LONG when `report`.
__device__ __forceinline__ int visible_tokens(const DecodeArgs& p, int r, bool report, int* base) {
    int b, t, q_len;
    row_request(p, r, &b, &t, &q_len);
    int seq = p.seq_lens[b];
    const int cap = p.max_blocks * MLA_PAGE_SIZE;
    if (seq > cap || seq > p.max_seq_len || seq < 0) {
        if (report && p.dev_status) atomicOr(p.dev_status, MLA_DEV_SEQ_TOO_LONG);
        seq = seq < 0 ? 0 : (seq > cap ? cap : seq);
    }
    const int n = max(0, seq - (q_len - 1 - t));
    *base = n >= p.base ? p.base : n / p.base_step * p.base_step;
    return n - *base;
}

// The block-table entry of page `page` of request b.
__device__ __forceinline__ const int32_t* table_entry(const DecodeArgs& p, int b, int page) {
    return p.block_table + (page < p.shared_pages ? (size_t)page : (size_t)b * p.max_blocks + page);
}

// Upper bound of planned units (num_splits == -2) for B * Sq query rows on `pairs` SM pairs.
inline int64_t plan_max_units(int64_t rows, int pairs) { return rows + 2 * (int64_t)pairs; }

// Workspace carve-up of a decode call (the same for both cache formats): the device-built
// schedule, then the split-KV partials; every region starts on a 256-byte boundary.
struct WorkspaceLayout {
    size_t plan, part_o, part_lse, total;
    int64_t partial_slots;  // rows of part_o / part_lse
};
// `rows` query rows (split partials per row); B, kv_dtype and max_seq_len do not change it.
// `all_partial`: one uniform split has its partial state too.
WorkspaceLayout workspace_layout(int kv_dtype, int B, int64_t rows, int H, int num_splits, int max_seq_len,
                                 bool all_partial = false);

// Token range [j0, j1) of split s of a row with n visible tokens: the row is cut into
// num_splits page-aligned chunks of round_up(ceil(n / S), 64) tokens; trailing splits may be
// empty. The same rule is used by every decode kernel.
__host__ __device__ inline void split_range(int n, int S, int s, int* j0, int* j1) {
    int per = (n + S - 1) / S;
    int chunk = ((per + kPage - 1) / kPage) * kPage;
    int a = s * chunk;
    int e = a + chunk;
    *j0 = a < n ? a : n;
    *j1 = e < n ? e : n;
}

// Launch with programmatic stream serialization: the kernel may start while the preceding
// kernel of the stream finishes, once that kernel has signalled (griddepcontrol); every kernel
// of this library calls ptx::griddep_wait() before it touches data another of its kernels writes. (The
// decode kernels read cache pages before that: cache_write, which writes them, does not signal early.)
template <typename... Params, typename... Args>
cudaError_t launch_pdl(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                       Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---- page keys, page scores, page choice and sparse decode ----------------------------------
struct PageKeysArgs {
    const uint8_t* cache;       // [num_blocks, 64, row_bytes]
    int64_t num_blocks;
    const int32_t* block_table; // [B, max_blocks]
    int max_blocks;
    const int32_t* start_lens;  // [B] or null (0): tokens whose pages have their keys
    const int32_t* seq_lens;    // [B]
    int max_new_len, pages_per_req, B;
    uint16_t* page_keys;        // bf16 [num_blocks, 576]
    int32_t* dev_status;        // or null
};
struct PageScoresArgs {
    const uint16_t* q;          // bf16 [B, Sq, H, 576]
    const uint16_t* page_keys;  // bf16 [num_blocks, 576]
    int64_t num_blocks;
    const int32_t* block_table; // [B, max_blocks]
    int max_blocks;
    const int32_t* seq_lens;    // [B]
    int max_seq_len, B, Sq, H;
    float scale;
    float* scores;              // fp32 [B * Sq, width]
    int width;                  // ceil(max_seq_len / 64)
    int32_t* dev_status;        // or null
};
struct SelectArgs {
    const float* scores;        // row r at scores + r * stride, `width` entries
    int64_t stride;
    int width;
    const int32_t* seq_lens;    // [B]
    int B, Sq, K, sink, local;
    int32_t* pages;             // [B * Sq, K]
    int32_t* dev_status;        // or null
};
struct SparseTableArgs {
    const int32_t* pages;       // [B * Sq, K] ascending page numbers, -1 behind
    int K;
    const int32_t* block_table; // [B, max_blocks]
    int max_blocks;
    const int32_t* seq_lens;    // [B]
    int B, Sq;
    int32_t* table;             // [B * Sq, K] blocks of the selected pages
    int32_t* lens;              // [B * Sq] their tokens
    int32_t* dev_status;        // or null
};
constexpr int kMaxSelectWidth = 32768;  // pages of a row: 32 keys a thread in one CTA
cudaError_t launch_page_keys(const PageKeysArgs& a, bool fp8, cudaStream_t s);
cudaError_t launch_page_scores(const PageScoresArgs& a, cudaStream_t s);
cudaError_t launch_select_pages(const SelectArgs& a, cudaStream_t s);
cudaError_t launch_sparse_table(const SparseTableArgs& a, cudaStream_t s);

// What the body of a decode call does beyond mla_decode (its own call by default).
struct DecodeExtra {
    const char* who = "mla_decode";  // the entry point, for messages
    bool few = false;                // the kernel for few heads, one SM a unit, see below
    bool check_only = false;         // return after the argument checks that need no device
    int shared_pages = 0;            // see DecodeArgs
    int base = 0, base_step = 0;
    bool all_partial = false;
    int order = kOrderDefault;
    // launched between the schedule and the decode (null: nothing); its error ends the call
    cudaError_t (*between)(void*) = nullptr;
    void* between_arg = nullptr;
    const float* pre_o = nullptr;
    const float* pre_lse = nullptr;
    int pre_splits = 0;
};
mla_status decode_impl(const void* q, const void* kv_cache, mla_kv_dtype kv_dtype, int64_t num_blocks,
                       const int32_t* block_table, int max_blocks, const int32_t* seq_lens, const int32_t* qsl,
                       int max_seq_len, int B, int Sq, int64_t rows, int H, float scale, int num_splits,
                       void* workspace, size_t workspace_bytes, void* o_latent, mla_dtype o_dtype, float* lse,
                       int32_t* dev_status, mla_stream_t stream, const DecodeExtra& x);

// Whether a decode takes the kernel for few heads, and the split count of its units (as
// mla_resolve_num_splits, which counts pairs of SMs). At 32 heads it took 25 against 33 us (32 rows of
// 32 pages), 71 against 121 (128 rows of 32), 134 against 160 (64 rows of 128); with room for 64 heads
// 37 against 36, 92 against 121 and 176 against 160: the ring then holds two pages only. FP8 cache, 32
// heads: 27 against 44, 77 against 149, 150 against 230.
inline bool few_heads(int H) { return H <= 32; }
int resolve_splits(bool few, int num_splits, int rows, int H, int max_seq_len);

// Clear the detail string and return MLA_OK.
mla_status set_ok();

// ---- decode over a prefix that the batch shares ------------------------------------------------
struct PrefixArgs {
    const uint16_t* q;          // bf16 [flat_rows, 576]: (request, query position, head)
    int flat_rows;              // B * Sq * H
    const int32_t* block_table; // the prefix pages' blocks (row 0 of the table); null: rows in order
    int64_t num_blocks;
    int key_rows;               // rows behind the keys' tensor map
    int prefix_pages, splits, pages_per_split;
    const float* k_scales;      // FP8: per prefix token
    const float* v_scales;
    const int32_t* seq_lens;    // [B]
    int max_seq_len, Sq, H;
    float scale;
    float* part_o;              // fp32 [splits, flat_rows, 512]
    float* part_lse;            // fp32 [splits, flat_rows]
    int32_t* dev_status;        // or null
};
int prefix_clusters();  // clusters of the prefix kernel that run at once on the current device, or -1
void prefix_split(int64_t flat_rows, int pages, int clusters, int* splits, int* pages_per_split);
// FP8: launch_prefix_widen first writes the prefix's rows to `widened` [prefix tokens, 576] and
// their scales to `scales` [2, prefix tokens].
cudaError_t launch_prefix_widen(const PrefixArgs& a, const uint8_t* cache, uint16_t* widened, float* scales,
                                cudaStream_t s);
cudaError_t launch_decode_prefix(const PrefixArgs& a, const uint8_t* cache, const uint16_t* widened,
                                 const float* scales, cudaStream_t s);

int device_sm_count();  // of the current device, or -1

// Record an error for mla_last_error_detail() and return `st` (printf-style message).
mla_status set_error(mla_status st, const char* fmt, ...);

cudaError_t launch_decode_sm103(const DecodeArgs& a, cudaStream_t s);
cudaError_t launch_decode_fp8_sm103(const DecodeArgs& a, cudaStream_t s);
cudaError_t launch_decode_few_sm103(const DecodeArgs& a, cudaStream_t s);  // H <= 32
cudaError_t launch_merge(const DecodeArgs& a, cudaStream_t s);
cudaError_t launch_plan(const DecodeArgs& a, int pairs, cudaStream_t s);
cudaError_t launch_cache_write(const uint16_t* kv_c, int64_t st_c, const uint16_t* k_pe, int64_t st_pe,
                               const int64_t* slots, int T, uint8_t* cache, int kv_dtype, int64_t num_blocks,
                               float kv_scale, int32_t* dev_status, cudaStream_t s);
cudaError_t launch_absorb_sm103(const uint16_t* q_nope, int64_t snt, int64_t snh, const uint16_t* q_pe,
                                int64_t spt, int64_t sph, const uint16_t* w_uk_t, uint16_t* q_out, int T, int H,
                                cudaStream_t s);
cudaError_t launch_out_proj_sm103(const void* o_latent, int in_dtype, const uint16_t* w_uv, void* o,
                                  int out_dtype, int T, int H, cudaStream_t s);
cudaError_t launch_up_proj_sm103(const uint16_t* x, int64_t x_st, int rows, const uint16_t* w, bool w_is_uk,
                                 uint16_t* out, int H, cudaStream_t s);

// ---- prefill, the compute-friendly route ---------------------------------------------------
// Rows of one segment gathered into a contiguous workspace: the latent part x [rows, 512] and the
// rope part kpe [rows, 64], both bf16 holding the stored values exactly (FP8 codes are not scaled
// here), plus per-row (k_scale, v_scale) for an FP8 cache (1 for rows taken from kv_c / k_pe).
// Segments: the new tokens (kPrefillNew), one context chunk (kPrefillChunk), or every request's
// context followed by its new tokens (kPrefillAll: request b's rows start at cu_ctx[b] + qsl[b]).
enum { kPrefillChunk = 0, kPrefillNew = 1, kPrefillAll = 2 };
struct PrefillGather {
    int mode;
    const int32_t* qsl;         // [B + 1] (kPrefillAll)
    const uint16_t* kv_c;       // new tokens' rows (row strides st_c, st_pe)
    int64_t st_c;
    const uint16_t* k_pe;
    int64_t st_pe;
    const uint8_t* cache;       // context chunk: packed context rows [c0, c0 + rows)
    int kv_dtype;
    int64_t num_blocks;
    const int32_t* block_table;
    int max_blocks;
    const int32_t* cu_ctx;      // [B + 1] prefix sums of the context lengths
    int B;
    int64_t c0;
    int rows;
    uint16_t* x;
    uint16_t* kpe;
    float2* scales;             // FP8 only
    int32_t* dev_status;
};

// One attention segment: every query row of the requests attends to its keys in the segment.
// kPrefillNew: the keys are the request's own new tokens (key i visible to query row t iff
// i <= t). kPrefillChunk: the request's rows of the context chunk [c0, c1), all visible.
// kPrefillAll: the request's context and then its new tokens (key p visible to query row t iff
// p <= ctx + t). The result is written (merge = 0) or merged by LSE into o / lse (merge = 1).
struct PrefillAttn {
    const uint16_t* q;          // [T, H, 192]
    const uint16_t* kn;         // [H, key_rows, 128] up-projected k_nope (head-major)
    const uint16_t* v;          // [H, key_rows, 128] up-projected v (head-major)
    const uint16_t* kpe;        // [key_rows, 64]
    const float2* scales;       // FP8 only: per key row (k_scale, v_scale)
    int key_rows;
    const int32_t* qsl;         // [B + 1]
    const int32_t* cu_ctx;      // [B + 1]
    int B, H, T, max_q_len;
    int mode;
    int64_t c0, c1;
    float scale;
    int merge;
    float* o;                   // [T, H, 128]
    float* lse;                 // [T, H]
    int32_t* dev_status;
};
cudaError_t launch_prefill_cu_ctx(const int32_t* ctx_lens, int B, int32_t* cu_ctx, int32_t* dev_status,
                                  cudaStream_t s);
cudaError_t launch_prefill_gather(const PrefillGather& g, cudaStream_t s);
cudaError_t launch_prefill_attn(const PrefillAttn& a, cudaStream_t s);

}  // namespace mla
