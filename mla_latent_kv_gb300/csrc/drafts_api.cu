// drafts_api.cu -- the entry points of a serving step with drafted tokens: rotary positions, decode of a
// tree of drafts, and the page pool between steps. Host-side validation and launches, by the rules of
// mla_api.cu: nothing is allocated, freed or synchronised, and every argument is checked before the first
// launch.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "internal.h"

namespace {

using mla::set_error;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t up256(size_t x) { return (x + 255) / 256 * 256; }
// Whether the buffers of m and n int32 have an element in common.
bool overlap(const int32_t* a, int64_t m, const int32_t* b, int64_t n) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && x < y + 4 * (uintptr_t)n && y < x + 4 * (uintptr_t)m;
}
bool known_kv(mla_kv_dtype d) { return d == MLA_KV_BF16 || d == MLA_KV_FP8_E4M3_SCALED; }

mla_status cuda_error(cudaError_t e, const char* who) {
    return set_error(MLA_ERR_CUDA, "%s launch: %s (%s)", who, cudaGetErrorName(e), cudaGetErrorString(e));
}

// ------------------------------------------------------------------------------------ positions
// w / 2 pi, modulo whole turns, in units of 2^-64: rounded once. A double's quotient alone is off by 2^-56 of a turn
// for the fast pairs, 2^-25 after 2^31 positions, so that the product with 1 / 2 pi is taken in two doubles.
uint64_t step_of(double w) {
    constexpr double kHigh = 0x1.45f306dc9c883p-3, kLow = -0x1.6b01ec5417056p-57;  // 1 / 2 pi
    const double high = std::fma(w, kHigh, 0.0);  // (as an fma: not to be contracted with the difference below)
    const double low = std::fma(w, kLow, std::fma(w, kHigh, -high));
    // without their whole turns, which leaves no error, in units of 2^-64: 2^63 at most
    const double a = (high - std::nearbyint(high)) * 0x1p64, b = (low - std::nearbyint(low)) * 0x1p64;
    auto integer = [](double x) { return x < 0 ? -(uint64_t)(-x) : (uint64_t)x; };
    const double whole = std::nearbyint(a);
    return integer(whole) + integer(std::nearbyint(b + (a - whole)));
}

// The checks and arguments that the two rotary calls share; x == null: no heads.
mla_status rope_args(const char* who, const void* x, int64_t x_t, int64_t x_n, const int32_t* positions,
                     const double* inv_freq, float mscale, int adjacent, void* out, int64_t out_t, int64_t out_n, int T,
                     int N, mla::RopeArgs* a) {
    if (T < 0 || N < 1) return set_error(MLA_ERR_INVALID_ARG, "%s: T=%d, %d heads", who, T, N);
    if (!inv_freq) return set_error(MLA_ERR_INVALID_ARG, "%s: null inv_freq", who);
    if (adjacent != 0 && adjacent != 1) return set_error(MLA_ERR_INVALID_ARG, "%s: adjacent=%d", who, adjacent);
    if (!std::isfinite(mscale)) return set_error(MLA_ERR_INVALID_ARG, "%s: mscale is not finite", who);
    for (int i = 0; i < mla::kPairs; ++i) {
        if (!std::isfinite(inv_freq[i])) return set_error(MLA_ERR_INVALID_ARG, "%s: inv_freq[%d] is not finite", who, i);
        a->step[i] = step_of(inv_freq[i]);
    }
    if (T == 0) return MLA_OK;
    if (!positions) return set_error(MLA_ERR_INVALID_ARG, "%s: null pointer", who);
    if (x || out) {
        if (!x || !out) return set_error(MLA_ERR_INVALID_ARG, "%s: null pointer", who);
        // (strides over a single token or head have no meaning)
        if (!aligned16(x) || !aligned16(out) || (T > 1 && (x_t % 8 || out_t % 8)) || (N > 1 && (x_n % 8 || out_n % 8)))
            return set_error(MLA_ERR_UNSUPPORTED, "%s: 16-byte aligned pointers and strides of multiples of 8 needed", who);
        if ((T > 1 && out_t == 0) || (N > 1 && out_n == 0))
            return set_error(MLA_ERR_INVALID_ARG, "%s: the result's rows overlap", who);
    }
    if ((int64_t)T * (N / 8 + 2) > (int64_t)INT32_MAX)
        return set_error(MLA_ERR_UNSUPPORTED, "%s: %d tokens of %d heads too many", who, T, N);
    a->mscale = mscale;
    a->adjacent = adjacent;
    a->positions = positions;
    a->T = T;
    a->x = (const uint16_t*)x;
    a->x_t = x_t;
    a->x_n = x_n;
    a->out = (uint16_t*)out;
    a->out_t = out_t;
    a->out_n = out_n;
    a->N = N;
    return MLA_OK;
}

// ------------------------------------------------------------------------------------ tree
// How a tree call runs, and its workspace. At most 32 (draft, head) pairs, or 128 over an FP8 cache, are one row
// of so many heads for the decode kernels (splits: theirs). More go through a kernel of their own, 256 at a time;
// its workspace is the widened rows (FP8), then, if units are cut, their parts' states. The widened rows have room for the
// bound on the lengths, not for the lengths, which the host does not know. Both sides of the border: 64 requests of up to
// 8192 tokens, bf16, 32 pairs 131 us as a row and 147 by the tree kernel; 112 pairs 157 and 146, FP8 233 and 303;
// 128 requests of up to 1000 tokens, 128 pairs, bf16 80 and 66, FP8 74 and 107.
struct TreePlan {
    bool rows;
    int splits, tiles, shares, lanes, slab_rows, wide_pages;  // shares: that the requests are cut into, or 0
    size_t scales, part_o, part_lse, pieces, total;
};
bool plan_tree(mla_kv_dtype kv, int B, int Sq, int H, int max_seq_len, TreePlan* w) {
    const int64_t flat = (int64_t)Sq * H;
    const int pages = (max_seq_len + mla::kPage - 1) / mla::kPage;
    w->rows = mla::few_heads((int)std::min<int64_t>(flat, INT32_MAX)) || (kv == MLA_KV_FP8_E4M3_SCALED && flat <= MLA_MAX_HEADS);
    if (w->rows) {
        const bool few = mla::few_heads((int)flat);
        // Over an FP8 cache with more than 32 pairs: short requests one unit each where there are more of them than SM
        // pairs (128 of up to 1000 tokens 74 us, by the schedule built on the device 85); much work by the schedule
        // (64 of up to 8192 tokens 223 us, ranges of a fixed length 233; 30 of up to 6000 91 and 102; 40 of up to 20,000 288
        // and 327), little by ranges, which need no plan (5 of up to 12,000 42 us, by the schedule 60). The borders lie
        // where the two cost the same (112 pairs, us per 1000 pages: 3 and 4 requests of up to 60,000 tokens 45.6 and 46.1;
        // 29 requests of up to 89 and 90 pages 48.7 and 45.2, 60 of them 40.4 both).
        const bool much = pages >= 90 && B >= 4 && (int64_t)B * pages > 2500;
        const int splits = few ? -1 : pages <= 32 && B > mla::device_sm_count() / 2 ? 1 : much ? -2 : -1;
        w->splits = mla::resolve_splits(few, splits, B, (int)flat, max_seq_len);
        if (w->splits < 1 && w->splits != -2) return false;
        w->total = mla::workspace_layout(kv, B, B, (int)flat, w->splits, max_seq_len).total;
        return true;
    }
    const int clusters = mla::tree_clusters();
    if (clusters < 1) return false;
    w->tiles = (int)((flat + 255) / 256);
    w->slab_rows = (int)std::min<int64_t>(flat, 256);
    w->shares = mla::tree_shares(B, w->tiles, w->slab_rows, pages, clusters, &w->lanes);
    size_t off = 0;
    if (kv == MLA_KV_FP8_E4M3_SCALED) {
        w->wide_pages = pages;
        const size_t rows = (size_t)B * pages * mla::kPage;
        off += up256(rows * mla::kBf16RowBytes);
        w->scales = off;
        off += up256(rows * 2 * sizeof(float));
    }
    if (w->shares > 0) {
        const size_t slabs = (size_t)2 * w->shares * w->lanes;
        w->part_o = off;
        off += up256(slabs * w->slab_rows * mla::kL * sizeof(float));
        w->part_lse = off;
        off += up256(slabs * 256 * sizeof(float));
        w->pieces = off;
        off += up256(slabs / 2 * sizeof(int2));
    }
    w->total = off;
    return true;
}
bool tree_shape(int B, int Sq, int H) {
    return B >= 0 && Sq >= 1 && Sq <= mla::kTreeMaxDrafts && H >= 1 && H <= MLA_MAX_HEADS &&
           (int64_t)B * Sq <= INT32_MAX / MLA_MAX_HEADS;
}

// ------------------------------------------------------------------------------------ pool
mla_status check_pool(const char* who, const void* cache, mla_kv_dtype kv, int layers, int64_t num_blocks, int max_blocks) {
    if (!known_kv(kv)) return set_error(MLA_ERR_INVALID_ARG, "%s: unknown kv_dtype %d", who, (int)kv);
    if (layers < 0 || num_blocks < 0 || max_blocks < 0)
        return set_error(MLA_ERR_INVALID_ARG, "%s: layers=%d, num_blocks=%lld, max_blocks=%d", who, layers,
                         (long long)num_blocks, max_blocks);
    if (num_blocks > (int64_t)(INT32_MAX / mla::kPage) || max_blocks > INT32_MAX / mla::kPage || layers > 65535)
        return set_error(MLA_ERR_UNSUPPORTED, "%s: num_blocks=%lld, max_blocks=%d or layers=%d too large", who,
                         (long long)num_blocks, max_blocks, layers);
    if (layers > 0 && num_blocks > 0 && !cache) return set_error(MLA_ERR_INVALID_ARG, "%s: null pointer", who);
    if (!aligned16(cache)) return set_error(MLA_ERR_UNSUPPORTED, "%s: kv_cache must be 16-byte aligned", who);
    return MLA_OK;
}

struct ForkLayout {
    size_t rows, copies, heirs, fresh, total;
};
ForkLayout fork_layout(int B, int B2, int64_t num_blocks) {
    ForkLayout w{};
    w.rows = 256;
    w.copies = w.rows + up256((size_t)B2 * sizeof(int4));
    w.heirs = w.copies + up256((size_t)B2 * sizeof(int4));
    w.fresh = w.heirs + up256((size_t)B * sizeof(int32_t));
    w.total = w.fresh + up256((size_t)num_blocks * sizeof(int32_t));
    return w;
}

}  // namespace

extern "C" {

mla_status mla_rope_frequencies(double base, double factor, int trained, double beta_fast, double beta_slow, double* inv_freq) {
    const char* who = "mla_rope_frequencies";
    if (!inv_freq) return set_error(MLA_ERR_INVALID_ARG, "%s: null pointer", who);
    if (!std::isfinite(base) || base <= 1.0 || !std::isfinite(factor) || factor < 1.0)
        return set_error(MLA_ERR_INVALID_ARG, "%s: base=%g must be above 1 and factor=%g at least 1", who, base, factor);
    const bool scaled = factor > 1.0;
    if (scaled && (trained < 1 || !(beta_slow > 0.0) || !(beta_fast >= beta_slow) || !std::isfinite(beta_fast)))
        return set_error(MLA_ERR_INVALID_ARG, "%s: trained=%d, beta_fast=%g, beta_slow=%g", who, trained, beta_fast, beta_slow);
    // the pair (not a whole number) that makes `turns` turns over the trained positions
    auto pair_of = [&](double turns) {
        return mla::kR * std::log(trained / (turns * 6.283185307179586476925286766559)) / (2.0 * std::log(base));
    };
    const double low = scaled ? std::max(std::floor(pair_of(beta_fast)), 0.0) : 0.0;
    const double high = scaled ? std::min(std::ceil(pair_of(beta_slow)), mla::kR - 1.0) : 0.0;
    for (int i = 0; i < mla::kPairs; ++i) {
        const double w = std::pow(base, -2.0 * i / mla::kR);
        const double ramp = scaled ? std::min(1.0, std::max(0.0, (i - low) / std::max(high - low, 0.001))) : 0.0;
        inv_freq[i] = w / factor * ramp + w * (1.0 - ramp);
    }
    return mla::set_ok();
}

mla_status mla_rope(const void* x, int64_t x_stride_t, int64_t x_stride_n, const int32_t* positions, const double* inv_freq,
                    float mscale, int adjacent, void* out, int64_t out_stride_t, int64_t out_stride_n, int T, int N,
                    mla_stream_t stream) {
    const char* who = "mla_rope";
    mla::RopeArgs a{};
    const mla_status st = rope_args(who, x, x_stride_t, x_stride_n, positions, inv_freq, mscale, adjacent, out, out_stride_t,
                                    out_stride_n, T, N, &a);
    if (st != MLA_OK) return st;
    if (T == 0) return mla::set_ok();
    if (!x) return set_error(MLA_ERR_INVALID_ARG, "%s: null pointer", who);
    const cudaError_t e = mla::launch_rope(a, (cudaStream_t)stream);
    return e == cudaSuccess ? mla::set_ok() : cuda_error(e, who);
}

mla_status mla_rope_cache_write(const void* kv_c, int64_t kv_c_stride_t, const void* k_pe, int64_t k_pe_stride_t,
                                const void* q_pe, int64_t q_pe_stride_t, int64_t q_pe_stride_h, void* q_out,
                                int64_t q_out_stride_t, int64_t q_out_stride_h, const int32_t* positions,
                                const double* inv_freq, float mscale, int adjacent, const int64_t* slot_mapping, int T, int H,
                                void* kv_cache, mla_kv_dtype kv_dtype, int64_t num_blocks, float kv_scale,
                                int32_t* dev_status, mla_stream_t stream) {
    const char* who = "mla_rope_cache_write";
    if (!known_kv(kv_dtype)) return set_error(MLA_ERR_INVALID_ARG, "%s: unknown kv_dtype %d", who, (int)kv_dtype);
    if (num_blocks < 0) return set_error(MLA_ERR_INVALID_ARG, "%s: negative num_blocks", who);
    if (num_blocks > (int64_t)1 << 40) return set_error(MLA_ERR_UNSUPPORTED, "%s: num_blocks too large", who);
    if (!(kv_scale >= 0.f) || std::isinf(kv_scale))
        return set_error(MLA_ERR_INVALID_ARG, "%s: kv_scale must be finite and >= 0 (0 = per-token)", who);
    mla::RopeArgs a{};
    const mla_status st = rope_args(who, q_pe, q_pe_stride_t, q_pe_stride_h, positions, inv_freq, mscale, adjacent, q_out,
                                    q_out_stride_t, q_out_stride_h, T, q_pe ? H : 1, &a);
    if (st != MLA_OK) return st;
    if (T == 0) return mla::set_ok();
    if (!kv_c || !k_pe || !slot_mapping || !kv_cache) return set_error(MLA_ERR_INVALID_ARG, "%s: null pointer", who);
    if (!aligned16(kv_c) || !aligned16(k_pe) || !aligned16(kv_cache) ||
        (T > 1 && (kv_c_stride_t % 8 || k_pe_stride_t % 8)))
        return set_error(MLA_ERR_UNSUPPORTED, "%s: 16-byte aligned pointers and strides of multiples of 8 needed", who);
    mla::RopeRows r{};
    r.kv_c = (const uint16_t*)kv_c;
    r.st_c = kv_c_stride_t;
    r.k_pe = (const uint16_t*)k_pe;
    r.st_pe = k_pe_stride_t;
    r.slots = slot_mapping;
    r.cache = (uint8_t*)kv_cache;
    r.num_blocks = num_blocks;
    r.kv_scale = kv_scale;
    r.dev_status = dev_status;
    const cudaError_t e = mla::launch_rope_cache_write(a, r, kv_dtype == MLA_KV_FP8_E4M3_SCALED, (cudaStream_t)stream);
    return e == cudaSuccess ? mla::set_ok() : cuda_error(e, who);
}

size_t mla_decode_tree_workspace_bytes(mla_kv_dtype kv_dtype, int B, int Sq, int H, int max_seq_len) {
    TreePlan w{};
    if (!known_kv(kv_dtype) || !tree_shape(B, Sq, H) || B < 1 || max_seq_len < 0 || max_seq_len > INT32_MAX - mla::kPage)
        return 0;
    return plan_tree(kv_dtype, B, Sq, H, max_seq_len, &w) ? w.total : 0;
}

mla_status mla_decode_tree(const void* q, const void* kv_cache, mla_kv_dtype kv_dtype, int64_t num_blocks,
                           const int32_t* block_table, int max_blocks, const int32_t* seq_lens, const uint64_t* tree_mask,
                           int max_seq_len, int B, int Sq, int H, float scale, void* workspace, size_t workspace_bytes,
                           void* o_latent, mla_dtype o_dtype, float* lse, int32_t* dev_status, mla_stream_t stream) {
    const char* who = "mla_decode_tree";
    if (Sq > mla::kTreeMaxDrafts)
        return set_error(MLA_ERR_UNSUPPORTED, "%s: Sq=%d drafts, at most %d", who, Sq, mla::kTreeMaxDrafts);
    if (B < 0 || Sq < 1) return set_error(MLA_ERR_INVALID_ARG, "%s: B=%d, Sq=%d", who, B, Sq);
    // What mla_decode refuses is refused by the same checks.
    mla::DecodeExtra x;
    x.who = who;
    x.check_only = true;
    const mla_status checked = mla::decode_impl(q, kv_cache, kv_dtype, num_blocks, block_table, max_blocks, seq_lens, nullptr,
                                                max_seq_len, B, Sq, (int64_t)B * Sq, H, scale, 1, nullptr, 0, o_latent,
                                                o_dtype, lse, dev_status, stream, x);
    if (checked != MLA_OK || B == 0) return checked;
    if (!tree_mask) return set_error(MLA_ERR_INVALID_ARG, "%s: null pointer", who);
    if (max_seq_len > INT32_MAX - mla::kPage)
        return set_error(MLA_ERR_UNSUPPORTED, "%s: max_seq_len=%d too large", who, max_seq_len);
    if (!tree_shape(B, Sq, H)) return set_error(MLA_ERR_UNSUPPORTED, "%s: %lld query rows too many", who, (long long)B * Sq);
    TreePlan w{};
    if (!plan_tree(kv_dtype, B, Sq, H, max_seq_len, &w))
        return set_error(MLA_ERR_CUDA, "%s: could not plan the call (no CUDA device?)", who);
    if (!w.rows && ((int64_t)B * w.tiles > INT32_MAX / 4 || (int64_t)B * w.wide_pages > INT32_MAX / mla::kPage))
        return set_error(MLA_ERR_UNSUPPORTED, "%s: %d requests of %d tokens too many", who, B, max_seq_len);
    if (w.total > 0 && (!workspace || workspace_bytes < w.total))
        return set_error(MLA_ERR_WORKSPACE_TOO_SMALL, "%s: workspace %zu bytes < %zu needed", who,
                         workspace ? workspace_bytes : (size_t)0, w.total);
    if (w.total > 0 && (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return set_error(MLA_ERR_UNSUPPORTED, "%s: workspace must be 256-byte aligned", who);
    if (w.rows) {
        x.check_only = false;
        x.few = mla::few_heads(Sq * H);
        x.masks = tree_mask;
        x.tree_drafts = Sq;
        x.tree_heads = H;
        return mla::decode_impl(q, kv_cache, kv_dtype, num_blocks, block_table, max_blocks, seq_lens, nullptr, max_seq_len, B, 1,
                                B, Sq * H, scale, w.splits, workspace, workspace_bytes, o_latent, o_dtype, lse, dev_status,
                                stream, x);
    }
    const bool fp8 = kv_dtype == MLA_KV_FP8_E4M3_SCALED;
    char* ws = (char*)workspace;
    mla::TreeArgs a{};
    a.q = (const uint16_t*)q;
    a.flat_rows = Sq * H;
    a.B = B;
    a.Sq = Sq;
    a.H = H;
    a.tiles = w.tiles;
    a.block_table = block_table;
    a.max_blocks = max_blocks;
    a.num_blocks = num_blocks;
    a.seq_lens = seq_lens;
    // no cache: no request sees a token, and a positive length is reported as too long
    a.max_seq_len = num_blocks > 0 ? max_seq_len : 0;
    a.masks = tree_mask;
    a.scale = scale;
    a.wide_pages = w.wide_pages;
    a.o = o_latent;
    a.lse = lse;
    a.o_bf16 = o_dtype == MLA_DT_BF16;
    if (w.shares > 0) {
        a.shares = w.shares;
        a.lanes = w.lanes;
        a.slab_rows = w.slab_rows;
        a.part_o = (float*)(ws + w.part_o);
        a.part_lse = (float*)(ws + w.part_lse);
        a.pieces = (int2*)(ws + w.pieces);
    }
    a.dev_status = dev_status;
    cudaStream_t s = (cudaStream_t)stream;
    const cudaError_t e = mla::launch_decode_tree(a, fp8, (const uint8_t*)kv_cache, fp8 ? (uint16_t*)ws : nullptr,
                                                  fp8 ? (float*)(ws + w.scales) : nullptr, s);
    return e == cudaSuccess ? mla::set_ok() : cuda_error(e, who);
}

mla_status mla_accept_tokens(void* kv_cache, mla_kv_dtype kv_dtype, int layers, int64_t num_blocks, const int32_t* block_table,
                             int max_blocks, const int32_t* seq_lens, const int32_t* path, const int32_t* counts, int B, int Sq,
                             int32_t* new_lens, int32_t* dev_status, mla_stream_t stream) {
    const char* who = "mla_accept_tokens";
    if (B < 0 || Sq < 1) return set_error(MLA_ERR_INVALID_ARG, "%s: B=%d, Sq=%d", who, B, Sq);
    if (Sq > mla::kTreeMaxDrafts)
        return set_error(MLA_ERR_UNSUPPORTED, "%s: Sq=%d drafts, at most %d", who, Sq, mla::kTreeMaxDrafts);
    const mla_status st = check_pool(who, kv_cache, kv_dtype, layers, num_blocks, max_blocks);
    if (st != MLA_OK) return st;
    if (B == 0) return mla::set_ok();
    if (layers < 1) return set_error(MLA_ERR_INVALID_ARG, "%s: layers=%d", who, layers);
    if (!seq_lens || !path || !counts || !new_lens || (max_blocks > 0 && !block_table))
        return set_error(MLA_ERR_INVALID_ARG, "%s: null pointer", who);
    // (every layer's blocks read the inputs)
    if (overlap(new_lens, B, seq_lens, B) || overlap(new_lens, B, counts, B) || overlap(new_lens, B, path, (int64_t)B * Sq) ||
        overlap(new_lens, B, block_table, (int64_t)B * max_blocks))
        return set_error(MLA_ERR_INVALID_ARG, "%s: new_lens must not be seq_lens, nor overlap another input", who);
    mla::AcceptArgs a{};
    a.cache = (uint8_t*)kv_cache;
    a.layers = layers;
    a.num_blocks = num_blocks;
    a.block_table = block_table;
    a.max_blocks = max_blocks;
    a.seq_lens = seq_lens;
    a.path = path;
    a.counts = counts;
    a.B = B;
    a.Sq = Sq;
    a.new_lens = new_lens;
    a.dev_status = dev_status;
    const cudaError_t e = mla::launch_accept_tokens(a, kv_dtype == MLA_KV_FP8_E4M3_SCALED, (cudaStream_t)stream);
    return e == cudaSuccess ? mla::set_ok() : cuda_error(e, who);
}

size_t mla_fork_pages_workspace_bytes(int B, int B2, int64_t num_blocks) {
    if (B < 0 || B2 < 0 || num_blocks < 0 || num_blocks > (int64_t)(INT32_MAX / mla::kPage)) return 0;
    return fork_layout(B, B2, num_blocks).total;
}

mla_status mla_fork_pages(void* kv_cache, mla_kv_dtype kv_dtype, int layers, int64_t num_blocks, const int32_t* block_table,
                          int max_blocks, const int32_t* page_counts, const int32_t* seq_lens, const int32_t* refs, int B,
                          const int32_t* parents, const int32_t* room, int B2, int32_t* new_table, int32_t* new_counts,
                          int32_t* new_lens, int32_t* new_refs, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                          mla_stream_t stream) {
    const char* who = "mla_fork_pages";
    if (B < 0 || B2 < 0) return set_error(MLA_ERR_INVALID_ARG, "%s: B=%d, B2=%d", who, B, B2);
    const mla_status st = check_pool(who, kv_cache, kv_dtype, layers, num_blocks, max_blocks);
    if (st != MLA_OK) return st;
    if (B > mla::kMaxPoolRows || B2 > mla::kMaxPoolRows || (int64_t)std::max(B, B2) * max_blocks > INT32_MAX)
        return set_error(MLA_ERR_UNSUPPORTED, "%s: %d and %d rows of %d pages (at most %d rows)", who, B, B2, max_blocks,
                         mla::kMaxPoolRows);
    if (B == 0 && B2 == 0 && num_blocks == 0) return mla::set_ok();
    if ((num_blocks > 0 && (!refs || !new_refs)) || (B > 0 && (!page_counts || !seq_lens)) ||
        (B2 > 0 && (!parents || !room || !new_counts || !new_lens)) || (B > 0 && max_blocks > 0 && !block_table) ||
        (B2 > 0 && max_blocks > 0 && !new_table))
        return set_error(MLA_ERR_INVALID_ARG, "%s: null pointer", who);
    struct Buffer {
        const int32_t* at;
        int64_t n;
    };
    const Buffer before[4] = {{block_table, (int64_t)B * max_blocks}, {page_counts, B}, {seq_lens, B}, {refs, num_blocks}};
    const Buffer after[4] = {{new_table, (int64_t)B2 * max_blocks}, {new_counts, B2}, {new_lens, B2}, {new_refs, num_blocks}};
    for (const Buffer& x : before)
        for (const Buffer& y : after)
            if (overlap(x.at, x.n, y.at, y.n))
                return set_error(MLA_ERR_INVALID_ARG, "%s: the new state must not be the old one's buffers, nor overlap them", who);
    if ((int64_t)B2 * (1 + (int64_t)layers) + B > (int64_t)INT32_MAX)
        return set_error(MLA_ERR_UNSUPPORTED, "%s: %d rows of %d layers too many", who, B2, layers);
    const ForkLayout w = fork_layout(B, B2, num_blocks);
    if (!workspace || workspace_bytes < w.total)
        return set_error(MLA_ERR_WORKSPACE_TOO_SMALL, "%s: workspace %zu bytes < %zu needed", who,
                         workspace ? workspace_bytes : (size_t)0, w.total);
    if (reinterpret_cast<uintptr_t>(workspace) & 255u)
        return set_error(MLA_ERR_UNSUPPORTED, "%s: workspace must be 256-byte aligned", who);
    char* ws = (char*)workspace;
    mla::ForkArgs a{};
    a.cache = (uint8_t*)kv_cache;
    a.layers = layers;
    a.num_blocks = num_blocks;
    a.table = block_table;
    a.counts = page_counts;
    a.lens = seq_lens;
    a.refs = refs;
    a.B = B;
    a.max_blocks = max_blocks;
    a.parents = parents;
    a.room = room;
    a.B2 = B2;
    a.new_table = new_table;
    a.new_counts = new_counts;
    a.new_lens = new_lens;
    a.new_refs = new_refs;
    a.head = (int32_t*)ws;
    a.rows = (int4*)(ws + w.rows);
    a.copies = (int4*)(ws + w.copies);
    a.heirs = (int32_t*)(ws + w.heirs);
    a.fresh = (int32_t*)(ws + w.fresh);
    a.dev_status = dev_status;
    const cudaError_t e = mla::launch_fork_pages(a, kv_dtype == MLA_KV_FP8_E4M3_SCALED, (cudaStream_t)stream);
    return e == cudaSuccess ? mla::set_ok() : cuda_error(e, who);
}

}  // extern "C"
