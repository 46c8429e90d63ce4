// merge.cu -- split-KV stage 2: combine the per-split partial states of every (row, head).
//
// [vLLM-MLA, Triton MLA section]: stage 1 writes a partial output and LSE per split into an
// fp32 buffer (B, N, splits, 512 + 1); stage 2 reduces them by LSE. [vLLM-MLA, Prefill
// section], merge_attn_states: partials are re-weighted by exp(lse - max_lse); an empty partial
// (o = 0, lse = -inf) has no weight.
//     M = max_s lse_s,  w_s = exp(lse_s - M),  lse = M + ln sum_s w_s,  o = sum_s w_s o_s / sum_s w_s
// One warp per (row, head, half of the latent dims); lane i owns 8 dims of its half. The partial
// states are read once, coalesced, four splits at a time (two behind a prefix) so that each lane has
// eight 16-byte loads in flight, and the result is written once.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "internal.h"
#include "sm103_ptx.cuh"

namespace mla {
namespace {

constexpr int kWarps = 8;
// States that are loaded together. Behind a prefix there are many rows of few states, and two leave room
// for more warps (128 rows of 128 heads, FP8: 249 -> 246 us a call); else four (8 rows of 9 splits of 128
// heads: 35.6 -> 35.1).
constexpr int batch_of(bool pre) { return pre ? 2 : 4; }

template <bool kPre>
__device__ __forceinline__ void merge_item(const DecodeArgs& p, int64_t r, int h, int half, int lane);

// kPre: the row's states over the base tokens (pre_o, pre_lse) come before its own.
template <bool kPre>
__global__ void __launch_bounds__(kWarps * 32) merge_kernel(DecodeArgs p) {
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();  // the partials are the preceding kernel's output
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    // grid-stride over (row, head, half) of the rows with partials: every row with uniform
    // splits, the listed split rows with a device-built schedule (none: the kernel ends here)
    const int64_t n_rows = p.plan_rows ? (int64_t)p.plan_count[1] : (int64_t)p.rows;
    const int64_t n_tasks = n_rows * p.H * 2;
    for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < n_tasks; t += (int64_t)gridDim.x * kWarps) {
        const int64_t item = t >> 1;
        const int64_t i = item / p.H;
        const int64_t r = p.plan_rows ? (int64_t)p.plan_split_rows[i] : i;
        merge_item<kPre>(p, r, (int)(item % p.H), (int)(t & 1), lane);
    }
}

template <bool kPre>
__device__ __forceinline__ void merge_item(const DecodeArgs& p, int64_t r, int h, int half, int lane) {
    // the row's partials are slots [slot0, slot0 + S): uniform splits put row r at r * S; a
    // device-built schedule lists them per row (a row with one unit already wrote its output)
    int S, slot0;
    if (p.plan_rows) {
        const int2 ri = p.plan_rows[r];
        S = ri.y;
        slot0 = ri.x;
        if (!kPre && S <= 1) return;
    } else {
        S = p.num_splits;
        slot0 = (int)(r * S);
    }
    // The row's states in order: those over the base tokens (kPre), then its own.
    const size_t heads = (size_t)p.rows * p.H, rh = (size_t)r * p.H + h;
    const int npre = kPre ? p.pre_splits : 0, total = npre + S;
    const int dim = half * (kL / 2) + lane * 8;
    auto state_lse = [&](int s) -> float {
        return kPre && s < npre ? p.pre_lse[(size_t)s * heads + rh]
                                : p.part_lse[((size_t)slot0 + (s - npre)) * p.H + h];
    };
    auto state_o = [&](int s) -> const float4* {
        return reinterpret_cast<const float4*>(kPre && s < npre
                                                   ? p.pre_o + ((size_t)s * heads + rh) * kL + dim
                                                   : p.part_o + (((size_t)slot0 + (s - npre)) * p.H + h) * kL + dim);
    };

    // A NaN state counts as the largest: its weight, the sum and the result are NaN then.
    auto top = [](float a, float b) { return fmaxf(a, b != b ? CUDART_INF_F : b); };
    constexpr int kBatch = batch_of(kPre);
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    float wsum = 0.f, M = -CUDART_INF_F;
    float ls[kBatch];
    float4 v[kBatch][2];
    auto load = [&](int s0) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            ls[u] = -CUDART_INF_F;
            v[u][0] = v[u][1] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (s0 + u < total) {
                ls[u] = state_lse(s0 + u);
                const float4* src = state_o(s0 + u);
                v[u][0] = src[0];
                v[u][1] = src[1];
            }
        }
    };
    auto add = [&]() {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (ls[u] == -CUDART_INF_F) continue;  // an empty split has no weight
            const float w = __expf(ls[u] - M);
            wsum += w;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                acc[4 * i + 0] = fmaf(w, v[u][i].x, acc[4 * i + 0]);
                acc[4 * i + 1] = fmaf(w, v[u][i].y, acc[4 * i + 1]);
                acc[4 * i + 2] = fmaf(w, v[u][i].z, acc[4 * i + 2]);
                acc[4 * i + 3] = fmaf(w, v[u][i].w, acc[4 * i + 3]);
            }
        }
    };
    if (total <= kBatch) {  // one batch: the maximum comes from the loads that are on their way anyway
        load(0);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) M = top(M, ls[u]);
        add();
    } else {
        for (int s = lane; s < total; s += 32) M = top(M, state_lse(s));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
        if (M != -CUDART_INF_F)
            for (int s0 = 0; s0 < total; s0 += kBatch) {
                // all loads of the batch first, then the arithmetic in split order
                load(s0);
                add();
            }
    }
    const float inv = wsum != 0.f ? 1.f / wsum : 0.f;
    const size_t base = ((size_t)r * p.H + h) * kL + half * (kL / 2) + lane * 8;
    if (p.o_dtype == MLA_DT_F32) {
        float4* dst = reinterpret_cast<float4*>((float*)p.o_latent + base);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            dst[i] = make_float4(acc[4 * i] * inv, acc[4 * i + 1] * inv, acc[4 * i + 2] * inv, acc[4 * i + 3] * inv);
    } else {
        __nv_bfloat162* dst = reinterpret_cast<__nv_bfloat162*>((__nv_bfloat16*)p.o_latent + base);
#pragma unroll
        for (int i = 0; i < 4; ++i) dst[i] = __floats2bfloat162_rn(acc[2 * i] * inv, acc[2 * i + 1] * inv);
    }
    if (half == 0 && lane == 0 && p.lse) p.lse[(size_t)r * p.H + h] = wsum != 0.f ? M + __logf(wsum) : -CUDART_INF_F;
}

}  // namespace

cudaError_t launch_merge(const DecodeArgs& a, cudaStream_t s) {
    const int64_t n_tasks = (int64_t)a.rows * a.H * 2;
    int64_t blocks = (n_tasks + kWarps - 1) / kWarps;
    // grid-stride over the split rows: enough warps that each takes about one (row, head, half),
    // since a task is a chain of dependent loads; with no split row every block ends at once
    if (a.plan_rows && blocks > 1216) blocks = 1216;
    return launch_pdl(a.pre_splits > 0 ? merge_kernel<true> : merge_kernel<false>, dim3((unsigned)blocks),
                      dim3(kWarps * 32), 0, s, a);
}

}  // namespace mla
