// rope.hip - rotary positions on gfx950.
//
// Pair p of a head, (x[2p], x[2p+1]) in the interleaved layout and (x[p], x[p + dim/2]) in the half
// one, is turned by the angle position * inv_freq[p] and scaled by the amplitude:
//     (a, b) -> (a cos - b sin, a sin + b cos)
//
// HBM bound: 4 bytes an element.  What would not be is the angles: a sine and a cosine with 64-bit
// range reduction take some 60 instructions, as much time as the memory of a pair in 32 heads.  A
// workgroup therefore takes whole tokens, or many heads of one, forms their angles once, one per
// thread, and keeps them in LDS for all heads.  8192 tokens of 32 heads of 128 take 27.6 us, 4.9 TB/s, what
// a large copy reaches; 64 tokens of 128 heads of 64 take 4.0 us, which is latency.
#include "device_codec.hpp"
#include "internal.hpp"
#include "rotary.hpp"

namespace bfp8 {

constexpr int kRopeThreads = 256;

static_assert(kRopeMaxDim / 2 * sizeof(float2) <= 65536 && kRopeMaxDim / 2 <= 65536, "a token's angles fit LDS");

struct RopeArgs {
    const uint16_t* x;
    int64_t x_ts, x_hs;
    const int32_t* positions;
    const float* inv_freq;
    uint16_t* out;
    int64_t o_ts, o_hs;
    int64_t T;
    int heads, pairs;
    float amplitude;
    int tokens, block_heads;                 // of a workgroup
    Divisor by_pairs, by_groups, by_heads;   // pairs; groups of a head; heads of a workgroup
};

// kVec: a thread's group is eight elements (interleaved) or twice eight (half layout), 16-byte loads
// and stores; otherwise it is a pair.
template <bool kInterleaved, bool kVec>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeArgs a) {
    extern __shared__ float2 angles[];       // [tokens][pairs]
    const int tid = threadIdx.x;
    const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
    const int n = (int)min((int64_t)a.tokens, a.T - t0);
    const int h0 = blockIdx.y * a.block_heads, heads = min(a.block_heads, a.heads - h0);
    for (int i = tid; i < n * a.pairs; i += kRopeThreads) {
        int p;
        const int t = a.by_pairs.of(i, p);
        angles[i] = rotary(a.positions[t0 + t], a.inv_freq[p], a.amplitude);
    }
    __syncthreads();
    const int groups = a.by_groups.d, all = n * (int)a.by_heads.d * groups;
    for (int i = tid; i < all; i += kRopeThreads) {
        int g, h;
        const int t = a.by_heads.of(a.by_groups.of(i, g), h);
        if (h >= heads || a.positions[t0 + t] < 0) continue;
        const uint16_t* const x = a.x + (t0 + t) * a.x_ts + (int64_t)(h0 + h) * a.x_hs;
        uint16_t* const y = a.out + (t0 + t) * a.o_ts + (int64_t)(h0 + h) * a.o_hs;
        if constexpr (!kVec) {
            const float2 cs = angles[t * a.pairs + g];
            const int i0 = kInterleaved ? 2 * g : g, i1 = kInterleaved ? 2 * g + 1 : g + a.pairs;
            float p = bf16_lo(x[i0]), q = bf16_lo(x[i1]);
            turn(p, q, cs);
            const uint32_t w = pack_bf16x2(p, q);
            y[i0] = (uint16_t)w;
            y[i1] = (uint16_t)(w >> 16);
        } else if constexpr (kInterleaved) {
            const float4* const cs = (const float4*)(angles + t * a.pairs + 4 * g);
            const uint4 v = *(const uint4*)(x + 8 * g);
            const float4 c0 = cs[0], c1 = cs[1];
            const float2 c[4] = {{c0.x, c0.y}, {c0.z, c0.w}, {c1.x, c1.y}, {c1.z, c1.w}};
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float p = bf16_lo(w[k]), q = bf16_hi(w[k]);
                turn(p, q, c[k]);
                o[k] = pack_bf16x2(p, q);
            }
            *(uint4*)(y + 8 * g) = make_uint4(o[0], o[1], o[2], o[3]);
        } else {
            const float4* const cs = (const float4*)(angles + t * a.pairs + 8 * g);
            const uint4 u = *(const uint4*)(x + 8 * g), v = *(const uint4*)(x + a.pairs + 8 * g);
            const uint32_t uw[4] = {u.x, u.y, u.z, u.w}, vw[4] = {v.x, v.y, v.z, v.w};
            uint32_t p[4], q[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float4 c = cs[k];
                float a0 = bf16_lo(uw[k]), a1 = bf16_hi(uw[k]), b0 = bf16_lo(vw[k]), b1 = bf16_hi(vw[k]);
                turn(a0, b0, make_float2(c.x, c.y));
                turn(a1, b1, make_float2(c.z, c.w));
                p[k] = pack_bf16x2(a0, a1);
                q[k] = pack_bf16x2(b0, b1);
            }
            *(uint4*)(y + 8 * g) = make_uint4(p[0], p[1], p[2], p[3]);
            *(uint4*)(y + a.pairs + 8 * g) = make_uint4(q[0], q[1], q[2], q[3]);
        }
    }
}

hipError_t launch_rope(const void* x, int64_t x_ts, int64_t x_hs, const int32_t* positions,
                       const float* inv_freq, void* out, int64_t o_ts, int64_t o_hs, int64_t T,
                       int32_t heads, int32_t dim, bool interleaved, float amplitude,
                       hipStream_t stream) {
    const int pairs = dim / 2;
    const bool vec = dim % (interleaved ? 8 : 16) == 0 && ((uintptr_t)x | (uintptr_t)out) % 16 == 0 &&
                     (x_ts | x_hs | o_ts | o_hs) % 8 == 0;
    const int groups = !vec ? pairs : dim / (interleaved ? 8 : 16);
    // About four groups a thread, to pay for the angles: tokens with few heads share a workgroup
    // where there are workgroups enough, one with many is divided.
    constexpr int kGroups = 4 * kRopeThreads;
    int block_heads = heads, tokens = 1;
    if ((int64_t)heads * groups > kGroups) {
        block_heads = (kGroups + groups - 1) / groups;
    } else {
        tokens = kGroups / (heads * groups);
        while (tokens > 1 && (T + tokens - 1) / tokens < 1024) tokens /= 2;
        while (tokens > 1 && tokens * pairs > 2048) tokens /= 2;
    }
    RopeArgs a;
    a.x = (const uint16_t*)x;
    a.x_ts = x_ts;
    a.x_hs = x_hs;
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.out = (uint16_t*)out;
    a.o_ts = o_ts;
    a.o_hs = o_hs;
    a.T = T;
    a.heads = heads;
    a.pairs = pairs;
    a.amplitude = amplitude;
    a.tokens = tokens;
    a.block_heads = block_heads;
    a.by_pairs = Divisor::by(pairs);
    a.by_groups = Divisor::by(groups);
    a.by_heads = Divisor::by(block_heads);
    const dim3 grid((unsigned)((T + tokens - 1) / tokens), (unsigned)((heads + block_heads - 1) / block_heads));
    const size_t lds = (size_t)tokens * pairs * sizeof(float2);
    auto* const kernel = interleaved ? (vec ? rope_kernel<true, true> : rope_kernel<true, false>)
                                     : (vec ? rope_kernel<false, true> : rope_kernel<false, false>);
    hipLaunchKernelGGL(kernel, grid, dim3(kRopeThreads), lds, stream, a);
    return hipGetLastError();
}

}  // namespace bfp8
