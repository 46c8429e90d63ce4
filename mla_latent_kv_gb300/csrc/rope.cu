// rope.cu -- rotary positions of queries and keys, alone or together with the cache write.
//
// A rope part's 64 values are 32 pairs; pair i of a token at position m turns by m * w_i:
//     u' = mscale (u cos(m w_i) - v sin(m w_i)),   v' = mscale (v cos(m w_i) + u sin(m w_i))
// The angle is only needed modulo a turn, so the host gives each pair's step w_i / 2 pi as a fraction of
// 2^64, rounded once, and the product m * step, which wraps at 2^64, is the turn's fraction: exact for any position
// but for the step's rounding (2^-34 of a turn at 2^31 tokens). Its leading 32 bits go to sincospi in fp32.
// (In fp32, m * w_i alone is off by 0.004 rad at 131072 tokens.)
//
// Queries: one warp per 32 heads of a token (8 or 16 where there are few). Each lane computes one pair's cosine
// and sine, four lanes share a head's row (pairs 8 c .. 8 c + 7 are lane c's, in both layouts) and get theirs by
// shuffles; up to four rows' loads are in flight before the first is used. For fewer than eight heads a warp
// takes eight head rows of as many tokens, and each lane computes the eight pairs that it turns. A thread writes
// what it read and no more, so that the result may replace its input.
// Cache rows: one warp per four tokens, whose rope parts are turned together, eight lanes each.
//
// Bound: memory, 256 bytes a head: 8192 tokens of 128 heads 44 us, 6.1 TB/s; 32768 of 16 heads with their FP8 rows
// 34 us, 5.6 TB/s (a row a warp 38.5 us: its rope part alone kept 24 lanes idle; fewer registers a thread spilled).
#include "internal.h"
#include "sm103_ptx.cuh"

namespace mla {
namespace {

constexpr int kWarps = 8;
constexpr int kTokens = 4;  // cache rows of a warp
// Head rows of a lane: a warp has eight times as many heads of a token (0: fewer than eight heads, see above).
constexpr int rows_per_lane(int heads) { return heads > 16 ? 4 : heads > 8 ? 2 : heads == 8 ? 1 : 0; }

// (cos, sin) of a pair at position m, times mscale.
__device__ __forceinline__ float2 turn_of(const RopeArgs& p, int m, int pair) {
    const uint64_t turns = (uint64_t)(int64_t)m * p.step[pair];
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

// The same for fewer than eight heads: rows [8 w, 8 w + 8) of all tokens' rows.
template <>
__device__ __forceinline__ void rope_heads<0>(const RopeArgs& p, int w, int, int lane) {
    const int64_t row = (int64_t)w * 8 + (lane >> 2);
    const int t = (int)(row / p.N), n = (int)(row % p.N), c = lane & 3;
    if (row >= (int64_t)p.T * p.N) return;
    const int c0 = p.adjacent ? 2 * c : c, c1 = p.adjacent ? 2 * c + 1 : c + 4;
    const uint16_t* src = p.x + t * p.x_t + n * p.x_n;
    const uint4 w0 = *reinterpret_cast<const uint4*>(src + 8 * c0), w1 = *reinterpret_cast<const uint4*>(src + 8 * c1);
    const int m = p.positions[t];
    float x[16];
    unpack8(w0, x);
    unpack8(w1, x + 8);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float2 tr = turn_of(p, m, 8 * c + k);
        if (p.adjacent)
            rotate(x[2 * k], x[2 * k + 1], tr);
        else
            rotate(x[k], x[8 + k], tr);
    }
    uint16_t* dst = p.out + t * p.out_t + n * p.out_n;
    *reinterpret_cast<uint4*>(dst + 8 * c0) = pack8(x);
    *reinterpret_cast<uint4*>(dst + 8 * c1) = pack8(x + 8);
}

// Warps that the heads take.
template <int kRows>
__host__ __device__ __forceinline__ int64_t head_warps(const RopeArgs& p) {
    if (!p.x) return 0;
    return kRows == 0 ? ((int64_t)p.T * p.N + 7) / 8 : (int64_t)p.T * ((p.N + 8 * kRows - 1) / (kRows == 0 ? 1 : 8 * kRows));
}

// The cache rows of tokens [kTokens w, ...), by one warp. Each row is 72 chunks of 8 values: 64 of kv_c, two a
// lane, and 8 of the turned k_pe, which lane 8 u + c holds for token u. A value is rounded once, to bf16 or, from
// the fp32 of the rotation, to e4m3.
template <bool kFp8>
__device__ __forceinline__ void rope_rows(const RopeArgs& p, const RopeRows& r, int64_t w, int lane) {
    static_assert(kTokens * 8 == 32, "eight lanes a token");
    const int64_t t0 = w * kTokens, mine = t0 + (lane >> 3);
    uint4 pe = make_uint4(0u, 0u, 0u, 0u);
    int m = 0;
    int64_t slot = -1;  // of this lane's token; below 0: padding
    if (mine < p.T) {
        slot = r.slots[mine];
        m = p.positions[mine];
        pe = *reinterpret_cast<const uint4*>(r.k_pe + mine * r.st_pe + 8 * (lane & 7));
    }
    uint4 v[2][2];  // kv_c of two tokens at a time
    auto load = [&](int u, uint4 (&x)[2]) {
        if (t0 + u >= p.T) return;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            x[i] = *reinterpret_cast<const uint4*>(r.kv_c + (t0 + u) * r.st_c + 8 * (lane + 32 * i));
    };
    load(0, v[0]);
    load(1, v[1]);
    if (slot >= r.num_blocks * kPage) {
        if ((lane & 7) == 0 && r.dev_status) atomicOr(r.dev_status, MLA_DEV_BAD_SLOT);
        slot = -1;
    }
    float x[8];
    unpack8(pe, x);
    {
        // chunk c has pairs 4 c .. 4 c + 3 or, in halves, one side of pairs 8 (c & 3) ..: then this lane and the one
        // four further compute four pairs each and exchange them, with their values
        const int c = lane & 7, pair0 = p.adjacent ? 4 * c : 8 * (c & 3) + 4 * (c >> 2);
        float2 tr[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) tr[k] = turn_of(p, m, pair0 + k);
        if (p.adjacent) {
#pragma unroll
            for (int k = 0; k < 4; ++k) rotate(x[2 * k], x[2 * k + 1], tr[k]);
        } else {
            const bool up = c & 4;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float other = __shfl_xor_sync(0xffffffffu, x[k], 4);
                const float2 got = make_float2(__shfl_xor_sync(0xffffffffu, tr[k & 3].x, 4), __shfl_xor_sync(0xffffffffu, tr[k & 3].y, 4));
                const float2 q = (k >= 4) == up ? tr[k & 3] : got;
                x[k] = up ? x[k] * q.x + other * q.y : x[k] * q.x - other * q.y;
            }
        }
    }
#pragma unroll
    for (int u = 0; u < kTokens; ++u) {
        const int64_t at = __shfl_sync(0xffffffffu, slot, 8 * u);
        const bool rope = (lane >> 3) == u;
        const int chunk = 64 + (lane & 7);
        uint4 kv[2] = {v[u & 1][0], v[u & 1][1]};
        if (u + 2 < kTokens) load(u + 2, v[u & 1]);
        if (at < 0) continue;
        if constexpr (!kFp8) {
            uint4* dst = reinterpret_cast<uint4*>(r.cache + at * kBf16RowBytes);
            dst[lane] = kv[0];
            dst[lane + 32] = kv[1];
            if (rope) dst[chunk] = pack8(x);
        } else {
            float z[16], amax = 0.f;
            unpack8(kv[0], z);
            unpack8(kv[1], z + 8);
#pragma unroll
            for (int k = 0; k < 16; ++k) amax = fmaxf(amax, fabsf(z[k]));
#pragma unroll
            for (int k = 0; k < 8; ++k) amax = fmaxf(amax, rope ? fabsf(x[k]) : 0.f);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
            const float scale = r.kv_scale > 0.f ? r.kv_scale : (amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f);
            const float inv = __frcp_rn(scale);
            uint8_t* dst = r.cache + at * kFp8RowBytes;  // 584-byte rows are 8-byte aligned
            auto store = [&](int c, const float* y) {
                uint32_t b[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) b[j] = ptx::f32x2_to_e4m3x2(__fmul_rn(y[2 * j], inv), __fmul_rn(y[2 * j + 1], inv));
                reinterpret_cast<uint2*>(dst)[c] = make_uint2(b[0] | (b[1] << 16), b[2] | (b[3] << 16));
            };
            store(lane, z);
            store(lane + 32, z + 8);
            if (rope) store(chunk, x);
            if (lane == 0) *reinterpret_cast<float2*>(dst + kD) = make_float2(scale, scale);
        }
    }
}

template <int kRows>
__device__ __forceinline__ void head_warp(const RopeArgs& p, int64_t w, int lane) {
    if (w >= head_warps<kRows>(p)) return;
    const int parts = kRows == 0 ? 1 : (p.N + 8 * kRows - 1) / (kRows == 0 ? 1 : 8 * kRows);
    rope_heads<kRows>(p, (int)(w / parts), (int)(w % parts), lane);
}

template <int kRows>
__global__ void __launch_bounds__(kWarps * 32) rope_kernel(const RopeArgs p) {
    // No early signal to the kernels behind: the result may be a part of a cache, which a decode reads
    // before its own wait.
    ptx::griddep_wait();
    const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    head_warp<kRows>(p, w, threadIdx.x & 31);
}

template <bool kFp8, int kRows>
__global__ void __launch_bounds__(kWarps * 32) rope_cache_write_kernel(const RopeArgs p, const RopeRows r) {
    ptx::griddep_wait();  // no early signal, as above
    const int64_t rows = ((int64_t)p.T + kTokens - 1) / kTokens, w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (w < rows)
        rope_rows<kFp8>(p, r, w, threadIdx.x & 31);
    else
        head_warp<kRows>(p, w - rows, threadIdx.x & 31);
}

unsigned blocks_of(int64_t warps) { return (unsigned)((warps + kWarps - 1) / kWarps); }

template <int kRows>
cudaError_t launch(const RopeArgs& a, cudaStream_t s) {
    return launch_pdl(rope_kernel<kRows>, dim3(blocks_of(head_warps<kRows>(a))), dim3(kWarps * 32), 0, s, a);
}
template <bool kFp8, int kRows>
cudaError_t launch(const RopeArgs& a, const RopeRows& r, cudaStream_t s) {
    const int64_t rows = ((int64_t)a.T + kTokens - 1) / kTokens;
    return launch_pdl(rope_cache_write_kernel<kFp8, kRows>, dim3(blocks_of(rows + head_warps<kRows>(a))), dim3(kWarps * 32), 0, s,
                      a, r);
}
template <bool kFp8>
cudaError_t launch_write(const RopeArgs& a, const RopeRows& r, cudaStream_t s) {
    switch (rows_per_lane(a.N)) {
        case 4: return launch<kFp8, 4>(a, r, s);
        case 2: return launch<kFp8, 2>(a, r, s);
        case 1: return launch<kFp8, 1>(a, r, s);
        default: return launch<kFp8, 0>(a, r, s);
    }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s) {
    switch (rows_per_lane(a.N)) {
        case 4: return launch<4>(a, s);
        case 2: return launch<2>(a, s);
        case 1: return launch<1>(a, s);
        default: return launch<0>(a, s);
    }
}

cudaError_t launch_rope_cache_write(const RopeArgs& a, const RopeRows& r, bool fp8, cudaStream_t s) {
    return fp8 ? launch_write<true>(a, r, s) : launch_write<false>(a, r, s);
}

}  // namespace mla
