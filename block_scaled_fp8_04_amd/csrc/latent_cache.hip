// latent_cache.hip - the paged cache of shared latents on gfx950: quantizing append and read back.
//
// A token's row in the cache is 512 e4m3 codes, one power-of-two scale (fp32) and 64 rotated bf16:
// 644 bytes.  The scale is the token's own, so a token is written without a look at its page and
// never touched again.
//
// append: one wave per two tokens, eight latent elements of each a lane.
//     y = c * rsqrt(mean c^2 + eps) * w        (or y = c), fp32, not rounded in between
//     s = 2^ceil(log2(max(amax |y|, 1e-4) / 448)),   code = e4m3_rne(y / s)
// Each half of the wave turns one token's key, a pair a lane: an angle's sine and cosine take some 60
// instructions.  17312 tokens take 11.6 us alone, 10.6 among other calls (2.9 TB/s read and written), of
// which a launch that fills no SIMD twice, 64 tokens, takes 3.8: 8656 waves are little more than the eight a SIMD
// that are resident at once, so nearly all of them load, sum twice over the wave and store at the same time.
//
// gather: one wave per eight or four rows: a row's codes are eight a lane, its key eight elements of
// eight lanes.  194700 rows take 82 us, 4.3 TB/s; 1600 take 6.4: offsets, table, row, one behind the other.
#include "attn_common.hpp"
#include "device_codec.hpp"
#include "internal.hpp"
#include "rotary.hpp"

namespace bfp8 {

constexpr int kLatentThreads = 256;
constexpr int kLatentWaves = kLatentThreads / 64;

// Over the 64 lanes, to all of them: lanes of four, of eight, of a row of 16, of two rows, of both halves.
template <typename F>
__device__ __forceinline__ uint32_t over_wave(uint32_t x, F join) {
    x = join(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xF, 0xF, true));
    x = join(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 0xF, 0xF, true));
    x = join(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x141, 0xF, 0xF, true));
    x = join(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x140, 0xF, 0xF, true));
    const auto rows = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    x = join(rows[0], rows[1]);
    const auto halves = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return join(halves[0], halves[1]);
}
__device__ __forceinline__ float wave_add(float x) {
    return __uint_as_float(over_wave(__float_as_uint(x), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}
__device__ __forceinline__ uint32_t wave_most(uint32_t x) {
    return over_wave(x, [](uint32_t a, uint32_t b) { return max(a, b); });
}

// Eight bf16 (kVec: 16-byte aligned).
template <bool kVec>
__device__ __forceinline__ void widen8_bf16(const uint16_t* p, float (&y)[8]) {
    if constexpr (kVec) {
        const uint4 v = *(const uint4*)p;
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y[2 * i] = bf16_lo(w[i]);
            y[2 * i + 1] = bf16_hi(w[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = bf16_lo(p[i]);
    }
}

template <bool kVec>
__global__ __launch_bounds__(kLatentThreads) void latent_append_kernel(
    const uint16_t* __restrict__ kv, int64_t kv_ts, const uint16_t* __restrict__ norm_weight, float eps,
    const int32_t* __restrict__ slot_map, const int32_t* __restrict__ positions,
    const float* __restrict__ inv_freq, int interleaved, float amplitude, int64_t T,
    uint8_t* __restrict__ codes, float* __restrict__ scales, uint16_t* __restrict__ rope, int64_t slots) {
    const int lane = threadIdx.x & 63, pair = lane & 31, half = lane >> 5;
    const int64_t t0 = ((int64_t)blockIdx.x * kLatentWaves + (threadIdx.x >> 6)) * 2;
    if (t0 >= T) return;
    const int64_t t[2] = {t0, min(t0 + 1, T - 1)};
    const int at[2] = {positions[t[0]], positions[t[1]]};
    // a token without a position is skipped, as one without a slot
    const int64_t slot[2] = {at[0] < 0 ? -1 : slot_map[t0], t0 + 1 == T || at[1] < 0 ? -1 : slot_map[t[1]]};
    float y[2][8], w[8];
#pragma unroll
    for (int j = 0; j < 2; ++j) widen8_bf16<kVec>(kv + t[j] * kv_ts + 8 * lane, y[j]);
    if (norm_weight) widen8_bf16<kVec>(norm_weight + 8 * lane, w);
    // each half of the wave turns a token's key
    const uint16_t* const key = kv + (half ? t[1] : t[0]) * kv_ts + kLatent;
    const int i0 = interleaved ? 2 * pair : pair, i1 = interleaved ? 2 * pair + 1 : pair + kLatentRope / 2;
    float a = bf16_lo(key[i0]), b = bf16_lo(key[i1]);
    const float2 cs = rotary(half ? at[1] : at[0], inv_freq[pair], amplitude);
    turn(a, b, cs);
    const uint32_t rot = pack_bf16x2(a, b);
    const uint64_t odd = __ballot((rot & 0x7F80u) == 0x7F80u || (rot >> 16 & 0x7F80u) == 0x7F80u);
    if (norm_weight) {
        float mean[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(y[j][i], y[j][i], sum);
            mean[j] = wave_add(sum) * (1.f / kLatent) + eps;
        }
        // squares that may have left fp32's range: those of the rows over a power of two near the largest
        // element, or near eps's root.  (Means are those of all lanes; NaN stays NaN, infinity becomes it.)
        if (!(fminf(mean[0], mean[1]) >= 0x1p-90f && fmaxf(mean[0], mean[1]) <= 0x1p120f)) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t top = __float_as_uint(__builtin_sqrtf(eps));
#pragma unroll
                for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(y[j][i]) & 0x7FFFFFFFu);
                const int down = 127 - (int)(wave_most(top) >> 23);
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    y[j][i] = __builtin_ldexpf(y[j][i], down);
                    sum = __builtin_fmaf(y[j][i], y[j][i], sum);
                }
                mean[j] = wave_add(sum) * (1.f / kLatent) + __builtin_ldexpf(eps, 2 * down);
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float f = 1.f / __builtin_sqrtf(mean[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[j][i] = y[j][i] * f * w[i];
        }
    }
    bool bad[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        // by bit patterns: infinities and NaN are the largest
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) most = max(most, __float_as_uint(y[j][i]) & 0x7FFFFFFFu);
        most = wave_most(most);
        // not finite, or 2^127 and more: codes times the scale would pass bf16
        bad[j] = most >= 0x7F000000u || (uint32_t)(odd >> 32 * j) != 0;
        if (slot[j] < 0 || slot[j] >= slots) continue;
        const float s = pow2_scale(__uint_as_float(most));
        const float inv = __uint_as_float((254u << 23) - __float_as_uint(s));
        uint2 q = make_uint2(e4m3_encode4<true>(y[j][0] * inv, y[j][1] * inv, y[j][2] * inv, y[j][3] * inv),
                             e4m3_encode4<true>(y[j][4] * inv, y[j][5] * inv, y[j][6] * inv, y[j][7] * inv));
        if (bad[j]) q = make_uint2(0, 0);
        *(uint2*)(codes + slot[j] * kLatent + 8 * lane) = q;
        if (lane == 0) scales[slot[j]] = bad[j] ? __uint_as_float(0x7FC00000u) : s;
    }
    const int64_t mine = half ? slot[1] : slot[0];
    if (mine >= 0 && mine < slots) {
        const bool none = half ? bad[1] : bad[0];
        uint16_t* const to = rope + mine * kLatentRope;
        if (interleaved) {
            *(uint32_t*)(to + i0) = none ? 0u : rot;
        } else {
            to[i0] = none ? 0 : (uint16_t)rot;
            to[i1] = none ? 0 : (uint16_t)(rot >> 16);
        }
    }
}

hipError_t launch_latent_append(const void* kv, int64_t kv_ts, const void* norm_weight, float eps,
                                const int32_t* slot_map, const int32_t* positions,
                                const float* inv_freq, bool interleaved, float amplitude, int64_t T,
                                void* codes, float* scales, void* rope, int64_t slots,
                                hipStream_t stream) {
    const bool vec = ((uintptr_t)kv | (uintptr_t)norm_weight) % 16 == 0 && kv_ts % 8 == 0;
    const unsigned grid = (unsigned)((T + 2 * kLatentWaves - 1) / (2 * kLatentWaves));
    hipLaunchKernelGGL(vec ? latent_append_kernel<true> : latent_append_kernel<false>, dim3(grid), dim3(kLatentThreads),
                       0, stream, (const uint16_t*)kv, kv_ts, (const uint16_t*)norm_weight, eps, slot_map, positions,
                       inv_freq, (int)interleaved, amplitude, T, (uint8_t*)codes, scales, (uint16_t*)rope, slots);
    return hipGetLastError();
}

// ------------------------------------------------------------------ gather

// Rows of a wave, whose loads are all on their way at once: eight where there are few, as what counts is
// latency (16000 rows of 8 requests: 11.0 us, and 18.3 with four), four where there are many, as what
// counts is how many waves a CU holds (64000 rows of 16 requests: 31 us, and 27 with four).
constexpr int kGatherFew = 40000;

struct GatherArgs {
    const uint8_t* codes;
    const float* scales;
    const uint16_t* rope;
    int64_t pages;
    int log_b;
    const int32_t* block_table;
    int64_t width;
    const int32_t *row_offsets, *starts;
    int R;
    int64_t rows;
    uint16_t* latent;
    int64_t l_ts;
    uint16_t* rope_out;
    int64_t r_ts;
};

template <int ROWS>
__global__ __launch_bounds__(kLatentThreads) void latent_gather_kernel(GatherArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t row0 = ((int64_t)blockIdx.x * kLatentWaves + (threadIdx.x >> 6)) * ROWS;
    if (row0 >= a.rows) return;
    const int each64 = a.row_offsets[min(lane * 64, a.R)];
    int ends = a.row_offsets[min(1 + lane, a.R)];                 // of request from + lane
    if (row0 >= a.row_offsets[a.R]) return;
    // the request of the first row, in two steps of 64; those of the others follow
    int from = 0;
    if (a.R > 64) {
        from = last_of(lane * 64 < a.R && each64 <= row0) * 64;
        ends = a.row_offsets[min(from + 1 + lane, a.R)];
    }
    int r = a.R;                                                  // lane j < ROWS: row j's
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
        int before = __popcll(__ballot(from + lane < a.R && ends <= row0 + j));
        while (before == 64 && from + 64 < a.R) {
            from += 64;
            ends = a.row_offsets[min(from + 1 + lane, a.R)];
            before = __popcll(__ballot(from + lane < a.R && ends <= row0 + j));
        }
        if (lane == j) r = from + before;
    }
    // where it lies in the pool, -1 for nowhere: rows in front of the first request have its number, too
    int64_t at = -1;
    if (r < a.R && row0 + lane < a.rows) {
        const int64_t in = row0 + lane - a.row_offsets[r], pos = in + (a.starts ? a.starts[r] : 0);
        if (in >= 0 && pos >= 0 && pos < a.width << a.log_b) {
            const int64_t page = a.block_table[r * a.width + (pos >> a.log_b)];
            at = min(max(page, (int64_t)0), a.pages - 1) << a.log_b | (pos & ((1 << a.log_b) - 1));
        }
    }
    const int64_t mine = max(at, (int64_t)0);
    const float scale = lane < ROWS ? a.scales[mine] : 0.f;
    uint2 c[ROWS];
    uint4 k[ROWS];
    int64_t slot[ROWS];
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
        slot[j] = (int64_t)(uint32_t)__builtin_amdgcn_readlane((int)at, j) |
                  (int64_t)__builtin_amdgcn_readlane((int)(at >> 32), j) << 32;
        const int64_t s = max(slot[j], (int64_t)0);
        c[j] = *(const uint2*)(a.codes + s * kLatent + 8 * lane);
        k[j] = *(const uint4*)(a.rope + s * kLatentRope + 8 * (lane & 7));
    }
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
        if (slot[j] < 0) continue;
        const float e = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(scale), j));
        *(uint4*)(a.latent + (row0 + j) * a.l_ts + 8 * lane) =
            __builtin_bit_cast(uint4, widen8((int)c[j].x, (int)c[j].y, e));
        if (lane < 8) *(uint4*)(a.rope_out + (row0 + j) * a.r_ts + 8 * lane) = k[j];
    }
}

hipError_t launch_latent_gather(const void* codes, const float* scales, const void* rope,
                                int64_t pages, int32_t page, const int32_t* block_table,
                                int64_t width, const int32_t* row_offsets, const int32_t* starts,
                                int64_t R, int64_t rows, void* latent, int64_t l_ts, void* rope_out,
                                int64_t r_ts, hipStream_t stream) {
    const GatherArgs a = {(const uint8_t*)codes, scales, (const uint16_t*)rope, pages, __builtin_ctz(page), block_table,
                          width, row_offsets, starts, (int)R, rows, (uint16_t*)latent, l_ts, (uint16_t*)rope_out, r_ts};
    const bool few = rows < kGatherFew;
    const int64_t each = kLatentWaves * (few ? 8 : 4);
    hipLaunchKernelGGL(few ? latent_gather_kernel<8> : latent_gather_kernel<4>,
                       dim3((unsigned)((rows + each - 1) / each)), dim3(kLatentThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace bfp8
