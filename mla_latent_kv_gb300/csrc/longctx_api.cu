// longctx_api.cu -- the entry points for long contexts: decode of a batch that shares a prefix, and
// the steps of decode over selected pages (mean page keys, page scores, page choice, attention).
// Host-side validation and launches, by the rules of mla_api.cu: nothing is allocated, freed or
// synchronised, and every argument is checked before the first launch.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "internal.h"

namespace {

using mla::set_error;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t up256(size_t x) { return (x + 255) / 256 * 256; }
bool known_kv(mla_kv_dtype d) { return d == MLA_KV_BF16 || d == MLA_KV_FP8_E4M3_SCALED; }

mla_status cuda_error(cudaError_t e, const char* who) {
    return set_error(MLA_ERR_CUDA, "%s launch: %s (%s)", who, cudaGetErrorName(e), cudaGetErrorString(e));
}

// Checks that the calls share. B == 0 is allowed.
mla_status check_shape(const char* who, int B, int Sq, int64_t num_blocks, int max_blocks, int max_seq_len) {
    if (B < 0 || Sq < 1) return set_error(MLA_ERR_INVALID_ARG, "%s: B=%d, Sq=%d", who, B, Sq);
    if (max_seq_len < 0 || max_blocks < 0 || num_blocks < 0)
        return set_error(MLA_ERR_INVALID_ARG, "%s: negative length, max_blocks or num_blocks", who);
    if ((int64_t)max_seq_len > (int64_t)max_blocks * mla::kPage)
        return set_error(MLA_ERR_INVALID_ARG, "%s: max_seq_len=%d exceeds max_blocks*64=%lld", who, max_seq_len,
                         (long long)max_blocks * mla::kPage);
    if (num_blocks > (int64_t)(INT32_MAX / mla::kPage))
        return set_error(MLA_ERR_UNSUPPORTED, "%s: num_blocks=%lld too large (max %d)", who, (long long)num_blocks,
                         INT32_MAX / mla::kPage);
    if ((int64_t)B * Sq > INT32_MAX / MLA_MAX_HEADS)
        return set_error(MLA_ERR_UNSUPPORTED, "%s: %lld query rows too many", who, (long long)B * Sq);
    return MLA_OK;
}

// The split count of a sparse decode. Its rows are mostly of max_sel pages each, so that the default is the
// uniform split with the least modelled time, in us: waves of units, each of its pages and a fixed part,
// then the merge. (Fitted to 100..300 rows of 16..128 pages. mla_decode's default, the schedule built on
// the device for more rows than units that run at once, costs its 11 us here: 128 rows of 32 pages,
// 128 heads 130 us against 107, FP8 153 against 139; 160 rows of 128 pages of 16 heads 440 against 316;
// it gains only where waves do not fill and rows are long: 100 rows of 128 pages, FP8, 367 against 381.)
int sparse_splits(mla_kv_dtype kv, int num_splits, int rows, int H, int pages) {
    const bool few = mla::few_heads(H), fp8 = kv == MLA_KV_FP8_E4M3_SCALED;
    if (num_splits != -1) return mla::resolve_splits(few, num_splits, rows, H, pages * mla::kPage);
    const int sms = mla::device_sm_count();
    if (sms < 2) return -1;
    const int slots = few ? sms : sms / 2;
    const double page = few ? (fp8 ? 1.9 : 1.6) : fp8 ? 1.7 : 1.1, fixed = few ? 6 : 14;
    int best = 1;
    double least = 1e300;
    for (int S = 1; S <= std::min(pages, 2 * slots); ++S) {
        const double waves = (double)(((int64_t)rows * S + slots - 1) / slots);
        const double states = (double)rows * H * S * (mla::kL + 1) * 8 / 5e6;  // written and read
        const double t = waves * (page * ((pages + S - 1) / S) + fixed) + (S > 1 ? 3 + 0.1 * S + states : 0);
        if (t < least * 0.999) {
            least = t;
            best = S;
        }
    }
    return best;
}

// Workspace of a sparse decode: the rows' tables and lengths, then that of their decode.
struct SparseLayout {
    size_t table, lens, decode, total;
};
SparseLayout sparse_layout(mla_kv_dtype kv, int64_t rows, int H, int K, int S) {
    SparseLayout w{};
    w.table = 0;
    w.lens = up256((size_t)rows * K * sizeof(int32_t));
    w.decode = w.lens + up256((size_t)rows * sizeof(int32_t));
    w.total = w.decode + mla::workspace_layout(kv, (int)rows, rows, H, S, K * mla::kPage).total;
    return w;
}

// How a shared-prefix call runs, and its workspace: the widened prefix (FP8), the prefix's partial
// states, then what the decode of the requests' own tokens needs.
struct PrefixPlan {
    int pages, splits, pages_per_split;  // of the prefix kernel; splits == 0: the decode kernels do it all
    int own_splits;                      // resolved, of the requests' own tokens
    size_t widened, scales, part_o, part_lse, decode, total;
};
// The prefix kernel's launches, as a step of the decode that follows them.
struct PrefixLaunch {
    mla::PrefixArgs a;
    const uint8_t* cache;
    uint16_t* widened;  // null: the cache is bf16
    float* scales;
    cudaStream_t stream;
    static cudaError_t run(void* self) {
        const PrefixLaunch& l = *static_cast<const PrefixLaunch*>(self);
        if (l.widened) {
            const cudaError_t e = mla::launch_prefix_widen(l.a, l.cache, l.widened, l.scales, l.stream);
            if (e != cudaSuccess) return e;
        }
        return mla::launch_decode_prefix(l.a, l.cache, l.widened, l.scales, l.stream);
    }
};
// Whether the prefix kernel is worth its launch, its partial states and their merge: estimated times in
// us of the call with it and of the decode kernels alone, fitted to graph replays of both at 1..128
// requests, 8..128 heads, 64..16384 prefix tokens and 64 or 512 own ones. Measured at the border, with
// and without: 128 rows of 16 heads, 256 + 64 tokens 21 and 12, 1024 + 64 tokens 29 and 31; 32 rows of
// 128 heads, 4096 + 64 tokens 56 and 56, 16384 + 64 tokens 103 and 166; 8 rows of 16 heads, 4096 + 64
// tokens 26 and 15, 16384 + 64 tokens 30 and 31. FP8 cache: 128 rows of 16 heads, 1024 + 64 tokens 32 and
// 37, 4096 + 64 tokens 41 and 128; 32 rows of 128 heads, 1024 + 64 tokens 44 and 36, 4096 + 64 60 and 77.
bool prefix_pays(bool fp8, int rows, int H, int pages, int own_pages, int clusters, int splits, int per) {
    // of one row's page on one of 76 SM pairs, the machine full
    const bool few = mla::few_heads(H);
    const double page = fp8 ? (!few ? 2.1 : H > 16 ? 1.2 : 1.0) : few ? 1.15 : 1.6;
    const int pairs = 76;
    const double alone = 12 + (rows > (few ? 2 * pairs : pairs) ? 11 : 0) + page * rows * (pages + own_pages) / pairs;
    const int64_t units = ((int64_t)rows * H + 255) / 256 * splits;
    const double waves = (double)((units + clusters - 1) / clusters);
    const double prefix = waves * (per * (fp8 ? 0.75 : 0.62) + 9) + (fp8 ? 3 : 0);
    const double states = (splits + 1.0) * rows * H * (mla::kL + 1) * 8 / 5e6;  // written and read
    return prefix + 12 + page * rows * own_pages / pairs + 4 + states < alone;
}

bool plan_prefix(mla_kv_dtype kv, int rows, int H, int prefix_len, int num_splits, int max_seq_len, PrefixPlan* w) {
    // tokens past max_seq_len are no request's; a page that it cuts is left to the requests' own tokens
    const int seen = (max_seq_len + mla::kPage - 1) / mla::kPage;
    const int pages = std::min(prefix_len, max_seq_len) / mla::kPage;
    const int64_t flat = (int64_t)rows * H;
    const bool fp8 = kv == MLA_KV_FP8_E4M3_SCALED;
    if (pages > 0) {
        const int clusters = mla::prefix_clusters();
        if (clusters < 1) return false;
        int splits, per;
        mla::prefix_split(flat, pages, clusters, &splits, &per);
        if (prefix_pays(fp8, rows, H, pages, seen - pages, clusters, splits, per)) {
            w->pages = pages;
            w->splits = splits;
            w->pages_per_split = per;
            size_t off = 0;
            if (fp8) {
                w->widened = off;
                off += up256((size_t)pages * mla::kPage * mla::kBf16RowBytes);
                w->scales = off;
                off += up256((size_t)pages * mla::kPage * 2 * sizeof(float));
            }
            w->part_o = off;
            off += up256((size_t)splits * flat * mla::kL * sizeof(float));
            w->part_lse = off;
            off += up256((size_t)splits * flat * sizeof(float));
            w->decode = off;
        }
    }
    const int own_len = std::max(0, max_seq_len - w->pages * mla::kPage);
    // With more rows than SM pairs mla_decode's default builds a schedule on the device, about 10 us
    // ahead of everything else. Behind a prefix the requests' own tokens are usually few: up to 32
    // pages each row is one unit instead (128 rows of 16 heads, up to 1000 own tokens: 150 -> 140 us), or two
    // for few heads and more than 12 pages, which shortens the tail behind the prefix (the same 74 -> 68 us
    // over 8192 shared tokens, FP8 83 -> 78, up to 2000 tokens 99 -> 89 and 115 -> 99; up to 300 tokens of 32
    // heads one unit takes 68 and two 71, and 256 rows up to 1000 tokens 104 and 105).
    if (num_splits == -1 && w->splits > 0 && own_len <= 32 * mla::kPage && rows > 76)
        num_splits = mla::few_heads(H) && own_len > 12 * mla::kPage ? 2 : 1;
    w->own_splits = mla::resolve_splits(mla::few_heads(H), num_splits, rows, H, own_len);
    if (w->own_splits < 1 && w->own_splits != -2) return false;
    w->total = w->decode + mla::workspace_layout(kv, rows, rows, H, w->own_splits, own_len, w->splits > 0).total;
    return true;
}

}  // namespace

extern "C" {

mla_status mla_page_keys(const void* kv_cache, mla_kv_dtype kv_dtype, int64_t num_blocks, const int32_t* block_table,
                         int max_blocks, const int32_t* start_lens, const int32_t* seq_lens, int max_new_len, int B,
                         void* page_keys, int32_t* dev_status, mla_stream_t stream) {
    const char* who = "mla_page_keys";
    if (!known_kv(kv_dtype)) return set_error(MLA_ERR_INVALID_ARG, "%s: unknown kv_dtype %d", who, (int)kv_dtype);
    const mla_status st = check_shape(who, B, 1, num_blocks, max_blocks, max_new_len);
    if (st != MLA_OK) return st;
    if (B == 0 || max_new_len == 0) return mla::set_ok();
    if (!kv_cache || !block_table || !seq_lens || !page_keys)
        return set_error(MLA_ERR_INVALID_ARG, "%s: null pointer", who);
    if (!aligned16(kv_cache) || !aligned16(page_keys))
        return set_error(MLA_ERR_UNSUPPORTED, "%s: kv_cache and page_keys must be 16-byte aligned", who);
    mla::PageKeysArgs a{};
    a.cache = (const uint8_t*)kv_cache;
    a.num_blocks = num_blocks;
    a.block_table = block_table;
    a.max_blocks = max_blocks;
    a.start_lens = start_lens;
    a.seq_lens = seq_lens;
    a.max_new_len = max_new_len;
    // new tokens that start inside a page touch one page more than their number fills
    const int full = (max_new_len + mla::kPage - 1) / mla::kPage;
    a.pages_per_req = std::min(start_lens ? full + 1 : full, max_blocks);
    a.B = B;
    a.page_keys = (uint16_t*)page_keys;
    a.dev_status = dev_status;
    if ((int64_t)B * a.pages_per_req > INT32_MAX)
        return set_error(MLA_ERR_UNSUPPORTED, "%s: %lld pages too many", who, (long long)B * a.pages_per_req);
    const cudaError_t e = mla::launch_page_keys(a, kv_dtype == MLA_KV_FP8_E4M3_SCALED, (cudaStream_t)stream);
    return e == cudaSuccess ? mla::set_ok() : cuda_error(e, who);
}

mla_status mla_page_scores(const void* q, const void* page_keys, int64_t num_blocks, const int32_t* block_table,
                           int max_blocks, const int32_t* seq_lens, int max_seq_len, int B, int Sq, int H, float scale,
                           float* scores, int32_t* dev_status, mla_stream_t stream) {
    const char* who = "mla_page_scores";
    if (H < 1 || H > MLA_MAX_HEADS)
        return set_error(MLA_ERR_UNSUPPORTED, "%s: H=%d outside [1, %d]", who, H, MLA_MAX_HEADS);
    const mla_status st = check_shape(who, B, Sq, num_blocks, max_blocks, max_seq_len);
    if (st != MLA_OK) return st;
    if (!std::isfinite(scale) || scale <= 0.f)
        return set_error(MLA_ERR_INVALID_ARG, "%s: scale must be finite and > 0", who);
    if (B == 0 || max_seq_len == 0) return mla::set_ok();
    if (!q || !page_keys || !block_table || !seq_lens || !scores)
        return set_error(MLA_ERR_INVALID_ARG, "%s: null pointer", who);
    if (!aligned16(q) || !aligned16(page_keys))
        return set_error(MLA_ERR_UNSUPPORTED, "%s: q and page_keys must be 16-byte aligned", who);
    mla::PageScoresArgs a{};
    a.q = (const uint16_t*)q;
    a.page_keys = (const uint16_t*)page_keys;
    a.num_blocks = num_blocks;
    a.block_table = block_table;
    a.max_blocks = max_blocks;
    a.seq_lens = seq_lens;
    a.max_seq_len = max_seq_len;
    a.B = B;
    a.Sq = Sq;
    a.H = H;
    a.scale = scale;
    a.scores = scores;
    a.width = (max_seq_len + mla::kPage - 1) / mla::kPage;
    a.dev_status = dev_status;
    if ((int64_t)B * Sq * ((a.width + 127) / 128) > INT32_MAX)
        return set_error(MLA_ERR_UNSUPPORTED, "%s: B*Sq*max_seq_len too large", who);
    const cudaError_t e = mla::launch_page_scores(a, (cudaStream_t)stream);
    return e == cudaSuccess ? mla::set_ok() : cuda_error(e, who);
}

mla_status mla_select_pages(const float* scores, int64_t scores_stride, int num_pages, const int32_t* seq_lens, int B,
                            int Sq, int max_sel, int sink_pages, int local_pages, int32_t* pages, int32_t* dev_status,
                            mla_stream_t stream) {
    const char* who = "mla_select_pages";
    if (B < 0 || Sq < 1 || num_pages < 0 || max_sel < 1)
        return set_error(MLA_ERR_INVALID_ARG, "%s: B=%d, Sq=%d, num_pages=%d, max_sel=%d", who, B, Sq, num_pages,
                         max_sel);
    if (sink_pages < 0 || local_pages < 0 || (int64_t)sink_pages + local_pages > max_sel)
        return set_error(MLA_ERR_INVALID_ARG, "%s: sink_pages=%d and local_pages=%d do not fit max_sel=%d", who,
                         sink_pages, local_pages, max_sel);
    if (scores_stride < num_pages)
        return set_error(MLA_ERR_INVALID_ARG, "%s: scores_stride=%lld < num_pages=%d", who, (long long)scores_stride,
                         num_pages);
    if (num_pages > mla::kMaxSelectWidth)
        return set_error(MLA_ERR_UNSUPPORTED, "%s: num_pages=%d above %d", who, num_pages, mla::kMaxSelectWidth);
    if ((int64_t)B * Sq > INT32_MAX)
        return set_error(MLA_ERR_UNSUPPORTED, "%s: %lld query rows too many", who, (long long)B * Sq);
    if (B == 0) return mla::set_ok();
    if (!seq_lens || !pages || (num_pages > 0 && !scores))
        return set_error(MLA_ERR_INVALID_ARG, "%s: null pointer", who);
    mla::SelectArgs a{};
    a.scores = scores;
    a.stride = scores_stride;
    a.width = num_pages;
    a.seq_lens = seq_lens;
    a.B = B;
    a.Sq = Sq;
    a.K = max_sel;
    a.sink = sink_pages;
    a.local = local_pages;
    a.pages = pages;
    a.dev_status = dev_status;
    const cudaError_t e = mla::launch_select_pages(a, (cudaStream_t)stream);
    return e == cudaSuccess ? mla::set_ok() : cuda_error(e, who);
}

size_t mla_decode_sparse_workspace_bytes(mla_kv_dtype kv_dtype, int B, int Sq, int H, int max_sel, int num_splits) {
    if (!known_kv(kv_dtype) || B < 1 || Sq < 1 || H < 1 || H > MLA_MAX_HEADS || max_sel < 1 ||
        max_sel > INT32_MAX / mla::kPage || (int64_t)B * Sq > INT32_MAX / MLA_MAX_HEADS)
        return 0;
    const int rows = B * Sq;
    const int S = sparse_splits(kv_dtype, num_splits, rows, H, max_sel);
    if (S < 1 && S != -2) return 0;
    return sparse_layout(kv_dtype, rows, H, max_sel, S).total;
}

mla_status mla_decode_sparse(const void* q, const void* kv_cache, mla_kv_dtype kv_dtype, int64_t num_blocks,
                             const int32_t* block_table, int max_blocks, const int32_t* seq_lens, const int32_t* pages,
                             int max_sel, int B, int Sq, int H, float scale, int num_splits, void* workspace,
                             size_t workspace_bytes, void* o_latent, mla_dtype o_dtype, float* lse,
                             int32_t* dev_status, mla_stream_t stream) {
    const char* who = "mla_decode_sparse";
    if (!known_kv(kv_dtype)) return set_error(MLA_ERR_INVALID_ARG, "%s: unknown kv_dtype %d", who, (int)kv_dtype);
    if (H < 1 || H > MLA_MAX_HEADS)
        return set_error(MLA_ERR_UNSUPPORTED, "%s: H=%d outside [1, %d]", who, H, MLA_MAX_HEADS);
    const mla_status st = check_shape(who, B, Sq, num_blocks, max_blocks, 0);
    if (st != MLA_OK) return st;
    if ((int64_t)max_blocks * mla::kPage > INT32_MAX)
        return set_error(MLA_ERR_UNSUPPORTED, "%s: max_blocks=%d too large", who, max_blocks);
    if (max_sel < 1 || max_sel > INT32_MAX / mla::kPage)
        return set_error(MLA_ERR_INVALID_ARG, "%s: max_sel=%d outside [1, %d]", who, max_sel, INT32_MAX / mla::kPage);
    if (num_splits < -2) return set_error(MLA_ERR_INVALID_ARG, "%s: num_splits=%d < -2", who, num_splits);
    if (o_dtype != MLA_DT_F32 && o_dtype != MLA_DT_BF16)
        return set_error(MLA_ERR_INVALID_ARG, "%s: unknown o_dtype %d", who, (int)o_dtype);
    if (!std::isfinite(scale) || scale <= 0.f)
        return set_error(MLA_ERR_INVALID_ARG, "%s: scale must be finite and > 0", who);
    if (B == 0) return mla::set_ok();
    if (!q || !o_latent || !seq_lens || !pages || !kv_cache || !block_table)
        return set_error(MLA_ERR_INVALID_ARG, "%s: null pointer", who);
    if (!aligned16(q) || !aligned16(kv_cache) || !aligned16(o_latent))
        return set_error(MLA_ERR_UNSUPPORTED, "%s: q, kv_cache and o_latent must be 16-byte aligned", who);
    const int rows = B * Sq;
    const int S = sparse_splits(kv_dtype, num_splits, rows, H, max_sel);
    if (S < 1 && S != -2) return set_error(MLA_ERR_CUDA, "%s: could not resolve num_splits (no CUDA device?)", who);
    const SparseLayout w = sparse_layout(kv_dtype, rows, H, max_sel, S);
    if (!workspace || workspace_bytes < w.total)
        return set_error(MLA_ERR_WORKSPACE_TOO_SMALL, "%s: workspace %zu bytes < %zu needed", who,
                         workspace ? workspace_bytes : (size_t)0, w.total);
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return set_error(MLA_ERR_UNSUPPORTED, "%s: workspace must be 256-byte aligned", who);
    mla::SparseTableArgs t{};
    t.pages = pages;
    t.K = max_sel;
    t.block_table = block_table;
    t.max_blocks = max_blocks;
    t.seq_lens = seq_lens;
    t.B = B;
    t.Sq = Sq;
    t.table = (int32_t*)((char*)workspace + w.table);
    t.lens = (int32_t*)((char*)workspace + w.lens);
    t.dev_status = dev_status;
    const cudaError_t e = mla::launch_sparse_table(t, (cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_error(e, who);
    mla::DecodeExtra x;
    x.who = who;
    x.few = mla::few_heads(H);
    x.order = mla::kOrderWaitFirst;
    return mla::decode_impl(q, kv_cache, kv_dtype, num_blocks, t.table, max_sel, t.lens, nullptr, max_sel * mla::kPage,
                            rows, 1, rows, H, scale, S, (char*)workspace + w.decode, w.total - w.decode, o_latent,
                            o_dtype, lse, dev_status, stream, x);
}

size_t mla_decode_shared_prefix_workspace_bytes(mla_kv_dtype kv_dtype, int B, int Sq, int H, int prefix_len,
                                                int num_splits, int max_seq_len) {
    if (!known_kv(kv_dtype) || B < 1 || Sq < 1 || H < 1 || H > MLA_MAX_HEADS || prefix_len < 0 ||
        prefix_len % mla::kPage || max_seq_len < 0 || (int64_t)B * Sq > INT32_MAX / MLA_MAX_HEADS)
        return 0;
    PrefixPlan w{};
    return plan_prefix(kv_dtype, B * Sq, H, prefix_len, num_splits, max_seq_len, &w) ? w.total : 0;
}

mla_status mla_decode_shared_prefix(const void* q, const void* kv_cache, mla_kv_dtype kv_dtype, int64_t num_blocks,
                                    const int32_t* block_table, int max_blocks, const int32_t* seq_lens,
                                    int max_seq_len, int prefix_len, int B, int Sq, int H, float scale,
                                    int num_splits, void* workspace, size_t workspace_bytes, void* o_latent,
                                    mla_dtype o_dtype, float* lse, int32_t* dev_status, mla_stream_t stream) {
    const char* who = "mla_decode_shared_prefix";
    const mla_status st = check_shape(who, B, Sq, num_blocks, max_blocks, max_seq_len);
    if (st != MLA_OK) return st;
    if (prefix_len < 0 || prefix_len % mla::kPage)
        return set_error(MLA_ERR_INVALID_ARG, "%s: prefix_len=%d is not a multiple of 64", who, prefix_len);
    if ((int64_t)prefix_len > (int64_t)max_blocks * mla::kPage)
        return set_error(MLA_ERR_INVALID_ARG, "%s: prefix_len=%d exceeds max_blocks*64=%lld", who, prefix_len,
                         (long long)max_blocks * mla::kPage);
    mla::DecodeExtra x;
    x.who = who;
    x.few = mla::few_heads(H);
    x.shared_pages = prefix_len / mla::kPage;
    auto decode = [&](int splits, void* ws, size_t bytes) {
        return mla::decode_impl(q, kv_cache, kv_dtype, num_blocks, block_table, max_blocks, seq_lens, nullptr,
                                max_seq_len, B, Sq, (int64_t)B * Sq, H, scale, splits, ws, bytes, o_latent, o_dtype,
                                lse, dev_status, stream, x);
    };
    // What mla_decode refuses is refused by the same checks before anything is launched (and a
    // batch that launches nothing ends there).
    x.check_only = true;
    const mla_status checked = decode(1, nullptr, 0);
    if (checked != MLA_OK || B == 0) return checked;
    x.check_only = false;
    if (num_splits < -2) return set_error(MLA_ERR_INVALID_ARG, "%s: num_splits=%d < -2", who, num_splits);
    PrefixPlan w{};
    if (!plan_prefix(kv_dtype, B * Sq, H, prefix_len, num_splits, max_seq_len, &w))
        return set_error(MLA_ERR_CUDA, "%s: could not plan the call (no CUDA device?)", who);
    if (w.splits > 0 && num_blocks == 0)
        return set_error(MLA_ERR_INVALID_ARG, "%s: prefix_len=%d in a cache without blocks", who, prefix_len);
    if (w.total > 0 && (!workspace || workspace_bytes < w.total))
        return set_error(MLA_ERR_WORKSPACE_TOO_SMALL, "%s: workspace %zu bytes < %zu needed", who,
                         workspace ? workspace_bytes : (size_t)0, w.total);
    if (w.total > 0 && (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return set_error(MLA_ERR_UNSUPPORTED, "%s: workspace must be 256-byte aligned", who);
    char* ws = (char*)workspace;
    PrefixLaunch launch{};
    if (w.splits > 0) {
        mla::PrefixArgs& a = launch.a;
        a.q = (const uint16_t*)q;
        a.flat_rows = B * Sq * H;
        a.block_table = block_table;
        a.num_blocks = num_blocks;
        a.prefix_pages = w.pages;
        a.splits = w.splits;
        a.pages_per_split = w.pages_per_split;
        a.seq_lens = seq_lens;
        a.max_seq_len = max_seq_len;
        a.Sq = Sq;
        a.H = H;
        a.scale = scale;
        a.part_o = (float*)(ws + w.part_o);
        a.part_lse = (float*)(ws + w.part_lse);
        a.dev_status = dev_status;
        x.base = w.pages * mla::kPage;
        x.base_step = w.pages_per_split * mla::kPage;
        x.all_partial = true;
        // The prefix kernel goes between the schedule and the decode of the requests' own tokens. It
        // lets that one start once all of its clusters run, which is after everything ahead of this
        // call has ended: the decode takes the SMs that the prefix leaves and reads what it likes.
        // (The other way round, with the prefix filling up behind the short units, those took longer:
        // 64 rows of 128 heads over 4096 + 512 tokens 97 us instead of 88.)
        launch.cache = (const uint8_t*)kv_cache;
        const bool fp8 = kv_dtype == MLA_KV_FP8_E4M3_SCALED;
        launch.widened = fp8 ? (uint16_t*)(ws + w.widened) : nullptr;
        launch.scales = (float*)(ws + w.scales);
        launch.stream = (cudaStream_t)stream;
        x.between = &PrefixLaunch::run;
        x.between_arg = &launch;
        x.order = mla::kOrderFree;
        x.pre_o = a.part_o;
        x.pre_lse = a.part_lse;
        x.pre_splits = w.splits;
    }
    return decode(w.own_splits, ws ? ws + w.decode : nullptr, w.total - w.decode);
}

}  // extern "C"
