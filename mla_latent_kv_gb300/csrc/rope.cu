// rope.cu -- rotary positions of queries and keys, alone or together with the cache write.
//
// A rope part's 64 values are 32 pairs; pair i of a token at position m turns by m * w_i:
//     u' = mscale (u cos(m w_i) - v sin(m w_i)),   v' = mscale (v cos(m w_i) + u sin(m w_i))
// The angle is only needed modulo a turn, so the host gives each pair's step w_i / 2 pi as a fraction of
// 2^64 and the product m * step, which wraps at 2^64, is the turn's fraction: exact for any position but
// for the step's own 2^-65 (2^-34 of a turn at 2^31 tokens). Its leading bits go to sincospi in fp32.
// (In fp32, m * w_i alone is off by 0.004 rad at 131072 tokens.)
//
// One warp per 32 heads of a token (8 or 16 where there are few): each lane computes one pair's cosine and sine, four lanes share a head's
// row (pairs 8 c .. 8 c + 7 are lane c's, in both layouts) and get theirs by shuffles; up to four rows' loads are
// in flight before the first is used. A thread writes what it read and no more, so that the result may
// replace its input. Bound: memory, 256 bytes a head.
#include "internal.h"
#include "sm103_ptx.cuh"

namespace mla {
namespace {

constexpr int kWarps = 8;
// Head rows of a lane: a warp has eight times as many heads of a token.
constexpr int rows_per_lane(int heads) { return heads > 16 ? 4 : heads > 8 ? 2 : 1; }

// (cos, sin) of this lane's pair at position m, times mscale.
__device__ __forceinline__ float2 turn_of(const RopeArgs& p, int m, int lane) {
    const uint64_t turns = (uint64_t)(int64_t)m * p.step[lane];
    float s, c;
    sincospif((float)(int32_t)(uint32_t)(turns >> 32) * 4.6566128730773926e-10f, &s, &c);  // 2^-31: half turns
    return make_float2(c * p.mscale, s * p.mscale);
}

__device__ __forceinline__ void rotate(float& u, float& v, float2 t) {
    const float a = u * t.x - v * t.y;
    v = v * t.x + u * t.y;
    u = a;
}

__device__ __forceinline__ uint4 pack8(const float* x) {
    return make_uint4(ptx::pack_bf16x2(x[0], x[1]), ptx::pack_bf16x2(x[2], x[3]), ptx::pack_bf16x2(x[4], x[5]),
                      ptx::pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void unpack8(uint4 w, float* x) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = ptx::bf16_lo_f(v[i]);
        x[2 * i + 1] = ptx::bf16_hi_f(v[i]);
    }
}

// Heads [8 kRows part, ...) of token t, by one warp.
template <int kRows>
__device__ __forceinline__ void rope_heads(const RopeArgs& p, int t, int part, int lane) {
    const float2 mine = turn_of(p, p.positions[t], lane);
    const int c = lane & 3;
    // the lane's 16 values: two chunks of 8, side by side or half a row apart
    const int c0 = p.adjacent ? 2 * c : c, c1 = p.adjacent ? 2 * c + 1 : c + 4;
    uint4 w[kRows][2];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int n = 8 * kRows * part + 8 * r + (lane >> 2);
        if (n >= p.N) continue;
        const uint16_t* src = p.x + t * p.x_t + n * p.x_n;
        w[r][0] = *reinterpret_cast<const uint4*>(src + 8 * c0);
        w[r][1] = *reinterpret_cast<const uint4*>(src + 8 * c1);
    }
    float2 tr[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
        tr[k] = make_float2(__shfl_sync(0xffffffffu, mine.x, 8 * c + k), __shfl_sync(0xffffffffu, mine.y, 8 * c + k));
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const int n = 8 * kRows * part + 8 * r + (lane >> 2);
        if (n >= p.N) continue;
        float x[16];
        unpack8(w[r][0], x);
        unpack8(w[r][1], x + 8);
        if (p.adjacent) {
#pragma unroll
            for (int k = 0; k < 8; ++k) rotate(x[2 * k], x[2 * k + 1], tr[k]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) rotate(x[k], x[8 + k], tr[k]);
        }
        uint16_t* dst = p.out + t * p.out_t + n * p.out_n;
        *reinterpret_cast<uint4*>(dst + 8 * c0) = pack8(x);
        *reinterpret_cast<uint4*>(dst + 8 * c1) = pack8(x + 8);
    }
}

// Two binary32 values -> two OCP E4M3 bytes (lo at the lower address), nearest even, saturating.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// The cache row of token t, by one warp: its 72 chunks of 8 values, chunks 64-71 (lanes 0-7) turned. A value
// is rounded once, to bf16 or, from the fp32 of the rotation, to e4m3.
template <bool kFp8>
__device__ __forceinline__ void rope_row(const RopeArgs& p, const RopeRows& r, int t, int lane) {
    const int64_t slot = r.slots[t];
    if (slot < 0) return;  // padding
    if (slot >= r.num_blocks * kPage) {
        if (lane == 0 && r.dev_status) atomicOr(r.dev_status, MLA_DEV_BAD_SLOT);
        return;
    }
    uint4 w[3];
    w[2] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < 2; ++i) w[i] = *reinterpret_cast<const uint4*>(r.kv_c + t * r.st_c + 8 * (lane + 32 * i));
    if (lane < 8) w[2] = *reinterpret_cast<const uint4*>(r.k_pe + t * r.st_pe + 8 * lane);
    const float2 mine = turn_of(p, p.positions[t], lane);
    float x[8], y[8];
    unpack8(w[2], x);
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = __shfl_xor_sync(0xffffffffu, x[k], 4);  // the pairs' other half
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const int pair = p.adjacent ? 4 * (lane & 7) + (k >> 1) : 8 * (lane & 3) + k;
        const float2 tr = make_float2(__shfl_sync(0xffffffffu, mine.x, pair), __shfl_sync(0xffffffffu, mine.y, pair));
        if (!p.adjacent) {
            if (lane & 4)
                rotate(y[k], x[k], tr);
            else
                rotate(x[k], y[k], tr);
        } else if (k & 1) {
            rotate(x[k - 1], x[k], tr);
        }
    }
    if constexpr (!kFp8) {
        uint4* dst = reinterpret_cast<uint4*>(r.cache + slot * kBf16RowBytes);
        dst[lane] = w[0];
        dst[lane + 32] = w[1];
        if (lane < 8) dst[lane + 64] = pack8(x);
    } else {
        float z[16];
        unpack8(w[0], z);
        unpack8(w[1], z + 8);
        float amax = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) amax = fmaxf(amax, fabsf(z[k]));
#pragma unroll
        for (int k = 0; k < 8; ++k) amax = fmaxf(amax, lane < 8 ? fabsf(x[k]) : 0.f);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
        const float scale = r.kv_scale > 0.f ? r.kv_scale : (amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f);
        const float inv = __frcp_rn(scale);
        uint8_t* dst = r.cache + slot * kFp8RowBytes;  // 584-byte rows are 8-byte aligned
        auto store = [&](int chunk, const float* v) {
            uint32_t b[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] = f32x2_to_e4m3x2(__fmul_rn(v[2 * j], inv), __fmul_rn(v[2 * j + 1], inv));
            reinterpret_cast<uint2*>(dst)[chunk] = make_uint2(b[0] | (b[1] << 16), b[2] | (b[3] << 16));
        };
        store(lane, z);
        store(lane + 32, z + 8);
        if (lane < 8) store(lane + 64, x);
        if (lane == 8) *reinterpret_cast<float2*>(dst + kD) = make_float2(scale, scale);
    }
}

template <int kRows>
__global__ void __launch_bounds__(kWarps * 32) rope_kernel(const RopeArgs p) {
    // No early signal to the kernels behind: the result may be a part of a cache, which a decode reads
    // before its own wait.
    ptx::griddep_wait();
    const int parts = (p.N + 8 * kRows - 1) / (8 * kRows);
    const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (w < (int64_t)p.T * parts) rope_heads<kRows>(p, (int)(w / parts), (int)(w % parts), threadIdx.x & 31);
}

template <bool kFp8, int kRows>
__global__ void __launch_bounds__(kWarps * 32) rope_cache_write_kernel(const RopeArgs p, const RopeRows r) {
    ptx::griddep_wait();  // no early signal, as above
    const int parts = p.x ? (p.N + 8 * kRows - 1) / (8 * kRows) : 0;
    const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (w < p.T)
        rope_row<kFp8>(p, r, (int)w, lane);
    else if (w < (int64_t)p.T * (parts + 1))
        rope_heads<kRows>(p, (int)((w - p.T) / parts), (int)((w - p.T) % parts), lane);
}

unsigned blocks_of(int64_t warps) { return (unsigned)((warps + kWarps - 1) / kWarps); }

template <int kRows>
cudaError_t launch(const RopeArgs& a, cudaStream_t s) {
    const int64_t parts = (a.N + 8 * kRows - 1) / (8 * kRows);
    return launch_pdl(rope_kernel<kRows>, dim3(blocks_of(a.T * parts)), dim3(kWarps * 32), 0, s, a);
}
template <bool kFp8, int kRows>
cudaError_t launch(const RopeArgs& a, const RopeRows& r, cudaStream_t s) {
    const int64_t parts = a.x ? (a.N + 8 * kRows - 1) / (8 * kRows) : 0;
    return launch_pdl(rope_cache_write_kernel<kFp8, kRows>, dim3(blocks_of(a.T * (parts + 1))), dim3(kWarps * 32), 0, s, a, r);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s) {
    const int rows = rows_per_lane(a.N);
    return rows == 4 ? launch<4>(a, s) : rows == 2 ? launch<2>(a, s) : launch<1>(a, s);
}

cudaError_t launch_rope_cache_write(const RopeArgs& a, const RopeRows& r, bool fp8, cudaStream_t s) {
    const int rows = rows_per_lane(a.N);
    if (fp8) return rows == 4 ? launch<true, 4>(a, r, s) : rows == 2 ? launch<true, 2>(a, r, s) : launch<true, 1>(a, r, s);
    return rows == 4 ? launch<false, 4>(a, r, s) : rows == 2 ? launch<false, 2>(a, r, s) : launch<false, 1>(a, r, s);
}

}  // namespace mla
