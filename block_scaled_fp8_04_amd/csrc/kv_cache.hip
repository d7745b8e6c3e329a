// kv_cache.hip - the paged e4m3 cache of attention on gfx950: a step's block
// tables and slot maps from its request lengths (kv_plan), and the quantizing
// append of its keys and values (kv_append).
#include "device_codec.hpp"
#include "internal.hpp"

namespace bfp8 {

// ------------------------------------------------------------------ kv_plan
//
// With B tokens per page, have = ceil(ctx / B), want = ceil((ctx + new) / B):
// request r needs want - have pages, and the running sum of needs over the
// requests up to r says whether it fits (upto <= pages left) and where its
// pages lie in the free list (upto - need).  A refusal leaves no gap: once the
// sum has passed the pages left, every later request that needs a page is
// refused too.  The other outputs are prefix sums of the same rows.
//
// One launch: every workgroup scans all requests itself (at most 4096, two
// loads each from L2) and then fills its own share of the token arrays and
// of the block table; the first one also writes the per-request arrays.
//
// All latency: 64 requests take 6.5 us, 1024 requests with 85000 new tokens 8.5, of which about 2
// are the launch.  Sums within a wave go by row operations and cached lengths stay in LDS (through
// cross-lane loads, and read again for every token: 7.2 and 9.4).
constexpr int kPlanThreads = 512;
constexpr int kPlanTokens = 1024;       // tokens per workgroup
constexpr int kPlanPer = kKvMaxRequests / kPlanThreads;

// x of the lanes that a row operation names, 0 where there is none.
template <int kCtrl, int kRows>
__device__ __forceinline__ int64_t dpp64(int64_t x) {
    const int lo = __builtin_amdgcn_update_dpp(0, (int)x, kCtrl, kRows, 0xF, false);
    const int hi = __builtin_amdgcn_update_dpp(0, (int)(x >> 32), kCtrl, kRows, 0xF, false);
    return (int64_t)(uint32_t)lo | (int64_t)hi << 32;
}

// Inclusive sums over the workgroup of one value per thread, in thread order.
template <int NV>
__device__ __forceinline__ void block_scan(int64_t (&v)[NV], int64_t (&wsum)[NV][kPlanThreads / 64],
                                           int tid) {
    const int lane = tid & 63, wave = tid >> 6;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        v[k] += dpp64<0x111, 0xF>(v[k]);                         // rows of 16 lanes: one, two, four, eight back
        v[k] += dpp64<0x112, 0xF>(v[k]);
        v[k] += dpp64<0x114, 0xF>(v[k]);
        v[k] += dpp64<0x118, 0xF>(v[k]);
        v[k] += dpp64<0x142, 0xA>(v[k]);                         // a row's last lane to the next row
        v[k] += dpp64<0x143, 0xC>(v[k]);                         // and to the upper two
    }
    if (lane == 63) {
#pragma unroll
        for (int k = 0; k < NV; ++k) wsum[k][wave] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < NV; ++k)
        for (int w = 0; w < wave; ++w) v[k] += wsum[k][w];
    __syncthreads();
}

__global__ __launch_bounds__(kPlanThreads) void kv_plan_kernel(
    const int32_t* __restrict__ ctx_lens, const int32_t* __restrict__ new_lens, int R,
    const int32_t* __restrict__ free_pages, int64_t n_free, const int32_t* __restrict__ free_head,
    int32_t* block_table, int64_t width, int log_b, int32_t* __restrict__ q_offsets,
    int32_t* __restrict__ kv_lens, int32_t* __restrict__ tile_offsets,
    int32_t* __restrict__ slot_map, int32_t* __restrict__ positions, int64_t T,
    int32_t* __restrict__ counts) {
    extern __shared__ int32_t lds[];
    int32_t* qoff = lds;                       // [R + 1]
    int32_t* first = lds + R + 1;              // [R] first free-list entry, -1: refused
    int32_t* cached = lds + 2 * R + 1;         // [R] ctx_lens
    __shared__ int64_t wsum[2][kPlanThreads / 64];
    __shared__ int64_t wtot[3][kPlanThreads / 64];
    const int tid = threadIdx.x;
    const int64_t B = (int64_t)1 << log_b;
    const int64_t head = free_head ? max((int64_t)*free_head, (int64_t)0) : 0;
    const int64_t left = max(n_free - head, (int64_t)0);

    const int per = (R + kPlanThreads - 1) / kPlanThreads;   // consecutive requests per thread
    const int r0 = tid * per;
    int64_t ctx[kPlanPer], neu[kPlanPer], need[kPlanPer];
    int64_t sums[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
        const int r = r0 + i;
        ctx[i] = neu[i] = need[i] = 0;
        if (i < per && r < R) {
            ctx[i] = ctx_lens[r];
            neu[i] = new_lens[r];
            const int64_t want = (ctx[i] + neu[i] + B - 1) >> log_b;
            if (ctx[i] < 0 || neu[i] < 0 || want > width) need[i] = -1;   // refused for itself
            else need[i] = want - ((ctx[i] + B - 1) >> log_b);
            sums[0] += max(neu[i], (int64_t)0);
            sums[1] += max(need[i], (int64_t)0);
        }
    }
    const int64_t own[2] = {sums[0], sums[1]};
    block_scan(sums, wsum, tid);
    int64_t q = sums[0] - own[0], upto = sums[1] - own[1];
    int64_t tally[3] = {0, 0, 0};              // tiles, requests not refused, pages taken
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
        const int r = r0 + i;
        if (i < per && r < R) {
            qoff[r] = (int32_t)min(q, T);
            cached[r] = (int32_t)ctx[i];
            q += max(neu[i], (int64_t)0);
            upto += max(need[i], (int64_t)0);
            const bool ok = need[i] >= 0 && q <= T && (need[i] == 0 || upto <= left);
            first[r] = !ok ? -1 : (need[i] ? (int32_t)(head + upto - need[i]) : 0);
            const int64_t kv = ok && neu[i] > 0 ? ctx[i] + neu[i] : 0;
            ctx[i] = kv;                       // from here on: the request's kv length
            tally[0] += (kv + kKvTile - 1) / kKvTile;
            tally[1] += ok;
            if (ok) tally[2] += need[i];
        }
    }
    if (tid == kPlanThreads - 1) qoff[R] = (int32_t)min(sums[0], T);
    if (blockIdx.x == 0) {
        const int64_t mine = tally[0];
        block_scan(tally, wtot, tid);
        int64_t tiles = tally[0] - mine;
#pragma unroll
        for (int i = 0; i < kPlanPer; ++i) {
            const int r = r0 + i;
            if (i < per && r < R) {
                tile_offsets[r] = (int32_t)tiles;
                kv_lens[r] = (int32_t)ctx[i];
                q_offsets[r] = qoff[r];
                tiles += (ctx[i] + kKvTile - 1) / kKvTile;
            }
        }
        if (tid == kPlanThreads - 1) {
            tile_offsets[R] = (int32_t)tally[0];
            q_offsets[R] = (int32_t)min(sums[0], T);
            counts[0] = (int32_t)min(sums[0], T);
            counts[1] = (int32_t)(head + tally[2]);
            counts[2] = (int32_t)tally[1];
            counts[3] = (int32_t)min(sums[1], (int64_t)INT32_MAX);
        }
    }
    __syncthreads();

    // newly taken pages, one wave per request
    const int lane = tid & 63;
    const int waves = gridDim.x * (kPlanThreads / 64);
    for (int r = blockIdx.x * (kPlanThreads / 64) + (tid >> 6); r < R; r += waves) {
        const int32_t f = first[r];
        if (f < 0) continue;
        const int64_t c = cached[r], have = (c + B - 1) >> log_b;
        const int64_t want = (c + qoff[r + 1] - qoff[r] + B - 1) >> log_b;   // (all its tokens fit T)
        for (int64_t j = have + lane; j < want; j += 64)
            block_table[r * width + j] = free_pages[f + j - have];
    }
    // tokens: the last request that starts at or before t (idle ones own none)
    const int64_t t_end = min(T, ((int64_t)blockIdx.x + 1) * kPlanTokens);
    for (int64_t t = (int64_t)blockIdx.x * kPlanTokens + tid; t < t_end; t += kPlanThreads) {
        int32_t slot = -1, pos = -1;
        if (t < qoff[R]) {
            int lo = 0, hi = R;                // qoff[lo] <= t < qoff[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (qoff[mid] <= t) lo = mid;
                else hi = mid;
            }
            const int32_t f = first[lo];
            if (f >= 0) {
                const int64_t c = cached[lo], p = c + t - qoff[lo];
                const int64_t j = p >> log_b, have = (c + B - 1) >> log_b;
                // entries this launch takes are read from the free list: the table's
                // may not be written yet
                const int64_t page = j < have ? block_table[lo * width + j] : free_pages[f + j - have];
                pos = (int32_t)p;
                slot = (int32_t)((page << log_b) + (p & (B - 1)));
            }
        }
        slot_map[t] = slot;
        positions[t] = pos;
    }
}

hipError_t launch_kv_plan(const int32_t* ctx_lens, const int32_t* new_lens, int64_t R,
                          const int32_t* free_pages, int64_t n_free, const int32_t* free_head,
                          int32_t* block_table, int64_t width, int32_t page, int32_t* q_offsets,
                          int32_t* kv_lens, int32_t* tile_offsets, int32_t* slot_map,
                          int32_t* positions, int64_t T, int32_t* counts, hipStream_t stream) {
    const int64_t grid = T > 0 ? (T + kPlanTokens - 1) / kPlanTokens : 1;
    const size_t lds = (3 * (size_t)R + 1) * sizeof(int32_t);
    kv_plan_kernel<<<dim3((unsigned)grid), dim3(kPlanThreads), lds, stream>>>(
        ctx_lens, new_lens, (int)R, free_pages, n_free, free_head, block_table, width,
        __builtin_ctz(page), q_offsets, kv_lens, tile_offsets, slot_map, positions, T, counts);
    return hipGetLastError();
}

// ---------------------------------------------------------------- kv_append
//
// One workgroup takes one head of a short run of tokens, finds the tokens in
// it that lead a page (the slot before is not the same page's previous one)
// and writes each such page whole: its new tokens are the ones that follow in
// ascending slots.  The page's maximum, the scale, the codes and the older
// tokens' re-encoding so need no second pass and no atomics.  Slots outside
// the pool are passed over, up to 63 in a row: looking further would make the
// last token of a padded step walk its whole padding.
//
// Keys keep the layout they come in.  Values are turned token-contiguous:
// their codes meet in LDS as [Dv][B] bytes, each thread then stores words of
// the rows that are new.
//
// Scale: the power of two at or above max(amax, floor) / 448 (as act_quant's
// power-of-two form): x / s is exact and below 448, and re-encoding an older
// code by old / s is exact but for values that fall under the format's normal
// range, so a page's growing scale does not wear its codes down.
//
// Bound by latency more than by bytes: 13240 tokens x 8 heads of 128 + 128 elements (54 MB read,
// 27 MB written) take 25.4 us in pages of 64, 3.2 TB/s, 64 tokens x 8 heads 4.9 us.  A workgroup's
// slots, loads, maximum and stores follow one another, and its registers, which hold the row
// slices of a page, let four share a compute unit at 128/128 in pages of 64 (120 registers; 33.5 us
// with registers for 128 tokens throughout): 1656 workgroups are one round and a second that is 60 %
// full.  The same tokens in other forms, with the workgroups that share a unit:
//                 pages of 32    of 64          of 128
//     64/64       23.3 us (4)    16.5 us (5)    16.3 us (4)
//     128/128     26.0 us (5)    25.1 us (4)    30.3 us (2)
//     192/128     33.6 us (4)    35.0 us (3)    36.4 us (2)
// Values turned by words instead of bytes bought the most (121 us); 512 threads take 28.9 and 5.6 us.
constexpr int kAppendThreads = 256;

__device__ __forceinline__ float append_scale(float amax) {
    const float y = fmaxf(amax, kAmaxFloor) / kE4m3Max;      // correctly rounded
    uint32_t e = __float_as_uint(y) >> 23;
    if (__float_as_uint(y) & 0x7FFFFFu) e += 1;
    return __uint_as_float(e << 23);
}

// Eight bf16 of a token's row; kVec: one 16-byte load.
template <bool kVec>
__device__ __forceinline__ uint4 load8(const uint16_t* p) {
    if constexpr (kVec) {
        return *(const uint4*)p;
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = (uint32_t)p[2 * i] | ((uint32_t)p[2 * i + 1] << 16);
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
}

typedef short s2v __attribute__((ext_vector_type(2)));
typedef unsigned short u2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf2v __attribute__((ext_vector_type(2)));

// Largest finite |element| of eight bf16 (as an fp32 bit pattern's upper half), and
// whether any is not finite.
__device__ __forceinline__ uint32_t amax8(const uint4 v, bool& odd) {
    const uint32_t w[4] = {v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu, v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu};
    const u2v m = __builtin_elementwise_max(
        __builtin_elementwise_max(__builtin_bit_cast(u2v, w[0]), __builtin_bit_cast(u2v, w[1])),
        __builtin_elementwise_max(__builtin_bit_cast(u2v, w[2]), __builtin_bit_cast(u2v, w[3])));
    uint32_t most = max((uint32_t)m.x, (uint32_t)m.y);
    if (most >= 0x7F80u) {
        odd = true;
        most = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = w[i] & 0xFFFFu, hi = w[i] >> 16;
            most = max(most, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
        }
    }
    return most;
}

// e4m3 codes of eight bf16 over s; `bad` is the code of an element that is not finite.  The
// conversion takes s, a power of two, by its exponent and rounds once, to nearest even; no
// finite element of the page passes 448 s.
__device__ __forceinline__ uint2 encode8(const uint4 v, float s, bool odd, uint32_t bad) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t c[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        s2v r = {0, 0};
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf2v, w[2 * i]), s, false);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf2v, w[2 * i + 1]), s, true);
        c[i] = __builtin_bit_cast(uint32_t, r);
    }
    if (odd) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t x = (w[i >> 1] >> (16 * (i & 1))) & 0x7FFFu;
            const uint32_t sh = 8 * (i & 3);
            if (x >= 0x7F80u) c[i >> 2] = (c[i >> 2] & ~(0xFFu << sh)) | (bad << sh);
        }
    }
    return make_uint2(c[0], c[1]);
}

// Four older codes re-encoded for a scale that grew: e4m3(value * ratio); NaN codes stay
// as they are.
__device__ __forceinline__ uint32_t reencode4(uint32_t w, float ratio) {
    float a, b, c, d;
    e4m3_decode2<false>(w, a, b);
    e4m3_decode2<true>(w, c, d);
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(a * ratio, b * ratio, 0, false);
    r = __builtin_amdgcn_cvt_pk_fp8_f32(c * ratio, d * ratio, r, true);
    // bytes of w that are 0x7F but for the sign
    const uint32_t nan = (((w & 0x7F7F7F7Fu) + 0x01010101u) >> 7 & 0x01010101u) * 0xFFu;
    return ((uint32_t)r & ~nan) | (w & nan);
}

// The first `keep` bytes of a piece re-encoded.
__device__ __forceinline__ uint4 reencode16(const uint4 v, float ratio, int keep) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int b = keep - 4 * i;
        const uint32_t m = b >= 4 ? ~0u : b <= 0 ? 0u : (1u << (8 * b)) - 1;
        r[i] = (reencode4(w[i], ratio) & m) | (w[i] & ~m);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

template <int DK, int DV, int B, bool kVec>
__global__ __launch_bounds__(kAppendThreads) void kv_append_kernel(
    const uint16_t* __restrict__ k, int64_t k_ts, int64_t k_hs, const uint16_t* __restrict__ v,
    int64_t v_ts, int64_t v_hs, const int32_t* __restrict__ slot_map, int64_t T, int run,
    uint8_t* __restrict__ k_cache, float* __restrict__ k_scales, uint8_t* __restrict__ v_cache,
    float* __restrict__ v_scales, int64_t slots, int H) {
    constexpr int KC = DK / 8, VC = DV / 8;                       // 8-element chunks per row
    constexpr int KP = (B * KC + kAppendThreads - 1) / kAppendThreads;
    constexpr int VP = (B / 4 * VC + kAppendThreads - 1) / kAppendThreads;   // items of 4 slots, 8 dims
    constexpr int vrow = B + 4;
    __shared__ uint32_t vt[DV * vrow / 4];                         // [DV][B + 4] bytes
    __shared__ uint32_t red[2][kAppendThreads / 64];
    __shared__ uint32_t poison[B];
    __shared__ int32_t token[B];                                   // of each new slot
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int h = blockIdx.y;
    k += h * k_hs;
    v += h * v_hs;

    // which of this run's tokens lead a page: in the pool, and the nearest slot before that is in
    // the pool is not the one in front of it in the same page
    const int64_t t0 = (int64_t)blockIdx.x * run;
    const int64_t behind = t0 - 64 + lane, ahead = t0 + lane;
    const int32_t prior = behind >= 0 ? slot_map[behind] : -1;
    const int32_t mine = lane < run && ahead < T ? slot_map[ahead] : -1;
    const bool valid = mine >= 0 && mine < slots;
    const uint64_t priors = __ballot(prior >= 0 && prior < slots) >> lane << lane;   // 64 back at most
    const uint64_t before = __ballot(valid) & ((1ull << lane) - 1);
    const uint64_t from = before ? before : priors;
    const int nearest = from ? 63 - __clzll((long long)from) : lane;
    const int32_t in_run = __shfl(mine, nearest), in_prior = __shfl(prior, nearest);
    const bool follows = from && (before ? in_run : in_prior) == mine - 1;
    const bool leads = valid && ((mine & (B - 1)) == 0 || !follows);
    for (uint64_t leaders = __ballot(leads); leaders; leaders &= leaders - 1) {
        const int which = __ffsll((unsigned long long)leaders) - 1;
        const int64_t t = t0 + which;
        const uint32_t s0 = __shfl(mine, which);
        const int off = (int)(s0 & (B - 1));
        const int64_t page = s0 / B;
        uint8_t* const kc = k_cache + (page * H + h) * ((int64_t)B * DK);
        uint8_t* const vc = v_cache + (page * H + h) * ((int64_t)B * DV);

        __syncthreads();                                           // the last page's LDS reads
        if (tid < B) poison[tid] = 0;
        // the tokens that follow in ascending slots of this page
        int n = 0;
        for (int64_t from = t; off + n < B;) {
            const int64_t i = from + lane;
            const int64_t s = i < T ? slot_map[i] : -1;
            const bool in = s >= 0 && s < slots;
            const uint64_t ins = __ballot(in);
            const int at = n + __popcll(ins & ((1ull << lane) - 1));
            const uint64_t end = __ballot(in && (s != s0 + at || off + at >= B));
            const uint64_t ours = end ? ins & ((end & -end) - 1) : ins;
            if (wave == 0 && (ours >> lane & 1)) token[at] = (int32_t)i;
            n += __popcll(ours);
            if (end || !ours) break;
            from += 64 - __clzll((long long)ours);
        }
        __syncthreads();
        // keys: a thread takes 8 elements of a token at a time; values: 8 of each of the four
        // tokens that share words of the turned rows.  One token alone (a decode step) is a few
        // lanes' work and branches over the rest, whose straight code costs more to fetch than
        // to run: 64 tokens x 8 heads take 4.3 us through here, 5.3 us through the quads.
        uint4 kx[KP], vx[VP][4];
        uint32_t km = 0, vm = 0;
        bool k_odd = false, v_odd = false;
        const int q0 = off >> 2, quads = ((off + n + 3) >> 2) - q0;
        const float ko = off > 0 ? k_scales[page * H + h] : 0.0f;
        const float vo = off > 0 ? v_scales[page * H + h] : 0.0f;
        if (n == 1) {
            if (tid < KC) kx[0] = load8<kVec>(k + t * k_ts + tid * 8);
            if (tid < VC) vx[0][0] = load8<kVec>(v + t * v_ts + tid * 8);
            if (tid < KC) km = amax8(kx[0], k_odd);
            if (tid < VC) vm = amax8(vx[0][0], v_odd);
            if (v_odd) poison[0] = 1;
        } else {
#pragma unroll
            for (int p = 0; p < KP; ++p) {
                const int c = p * kAppendThreads + tid, i = c / KC;
                if (i < n) kx[p] = load8<kVec>(k + token[i] * k_ts + (c % KC) * 8);
            }
#pragma unroll
            for (int p = 0; p < VP; ++p) {
                const int c = p * kAppendThreads + tid, i0 = 4 * (q0 + c / VC) - off;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    vx[p][b] = make_uint4(0, 0, 0, 0);
                    if (c / VC < quads && i0 + b >= 0 && i0 + b < n)
                        vx[p][b] = load8<kVec>(v + token[i0 + b] * v_ts + (c % VC) * 8);
                }
            }
#pragma unroll
            for (int p = 0; p < KP; ++p)
                if ((p * kAppendThreads + tid) / KC < n) km = max(km, amax8(kx[p], k_odd));
#pragma unroll
            for (int p = 0; p < VP; ++p) {
                const int i0 = 4 * (q0 + (p * kAppendThreads + tid) / VC) - off;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    bool odd = false;
                    vm = max(vm, amax8(vx[p][b], odd));         // zeros where there is no token
                    if (odd) poison[i0 + b] = 1;
                    v_odd |= odd;
                }
            }
        }
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            km = max(km, (uint32_t)__shfl_xor((int)km, d));
            vm = max(vm, (uint32_t)__shfl_xor((int)vm, d));
        }
        if (lane == 0) {
            red[0][wave] = km;
            red[1][wave] = vm;
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kAppendThreads / 64; ++w) {
            km = max(km, red[0][w]);
            vm = max(vm, red[1][w]);
        }
        float ks = append_scale(__uint_as_float(km << 16));
        float vs = append_scale(__uint_as_float(vm << 16));
        if (off > 0) {
            if (ks > ko) {
                const float ratio = ko / ks;
#pragma unroll 4
                for (int w = tid; w < off * (DK / 16); w += kAppendThreads)
                    ((uint4*)kc)[w] = reencode16(((uint4*)kc)[w], ratio, 16);
            } else {
                ks = ko;
            }
            if (vs > vo) {
                const int pieces = (off + 15) >> 4;                 // of 16 tokens per row
                const float ratio = vo / vs;
#pragma unroll 4
                for (int e = tid; e < DV * pieces; e += kAppendThreads) {
                    const int w = e % pieces;
                    uint4* const at = (uint4*)(vc + e / pieces * B + 16 * w);
                    *at = reencode16(*at, ratio, off - 16 * w);     // later bytes stay
                }
            } else {
                vs = vo;
            }
        }
        __syncthreads();                                           // old scales are read
        if (tid == 0) {
            k_scales[page * H + h] = ks;
            v_scales[page * H + h] = vs;
        }
        if (n == 1) {
            if (tid < KC) {
                uint2 w = encode8(kx[0], ks, k_odd, 0x7Fu);
                if (poison[0]) w = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
                *(uint2*)(kc + off * DK + tid * 8) = w;
            }
            if (tid < VC) {
                const uint2 w = encode8(vx[0][0], vs, v_odd, 0u);
#pragma unroll
                for (int y = 0; y < 8; ++y)
                    vc[(tid * 8 + y) * B + off] = (uint8_t)((y < 4 ? w.x : w.y) >> (8 * (y & 3)));
            }
            continue;
        }
#pragma unroll
        for (int p = 0; p < KP; ++p) {
            const int c = p * kAppendThreads + tid, i = c / KC;
            if (i < n) {
                uint2 w = encode8(kx[p], ks, k_odd, 0x7Fu);
                if (poison[i]) w = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
                *(uint2*)(kc + (int64_t)off * DK + (int64_t)c * 8) = w;
            }
        }
#pragma unroll
        for (int p = 0; p < VP; ++p) {
            const int c = p * kAppendThreads + tid, q = q0 + c / VC, d = (c % VC) * 8;
            if (c / VC < quads) {
                uint2 w[4];
#pragma unroll
                for (int b = 0; b < 4; ++b) w[b] = encode8(vx[p][b], vs, v_odd, 0u);
                // byte y of the four tokens' codes is row d + y's word
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                    const uint32_t sel = (y & 3) * 0x0101u + 0x0400u;     // bytes y of two codes
                    const uint32_t lo = y < 4 ? __builtin_amdgcn_perm(w[1].x, w[0].x, sel)
                                              : __builtin_amdgcn_perm(w[1].y, w[0].y, sel);
                    const uint32_t hi = y < 4 ? __builtin_amdgcn_perm(w[3].x, w[2].x, sel)
                                              : __builtin_amdgcn_perm(w[3].y, w[2].y, sel);
                    vt[((d + y) * vrow >> 2) + q] = (lo & 0xFFFFu) | hi << 16;
                }
            }
        }
        __syncthreads();
        for (int e = tid; e < DV * quads; e += kAppendThreads) {
            const int d = e / quads, w = q0 + (e - d * quads);
            const uint32_t c = vt[(d * vrow >> 2) + w];
            uint8_t* const at = vc + d * B + 4 * w;
            if (4 * w >= off && 4 * w + 4 <= off + n) {
                *(uint32_t*)at = c;
            } else {
                for (int b = 0; b < 4; ++b)
                    if (4 * w + b >= off && 4 * w + b < off + n) at[b] = (uint8_t)(c >> (8 * b));
            }
        }
    }
}

template <int DK, int DV, int B, bool kVec>
static hipError_t append_launch(const void* k, int64_t k_ts, int64_t k_hs, const void* v,
                                int64_t v_ts, int64_t v_hs, const int32_t* slot_map, int64_t T,
                                void* k_cache, float* k_scales, void* v_cache, float* v_scales,
                                int64_t pages, int32_t heads, hipStream_t stream) {
    // tokens per workgroup: one, until the launch would pass 2048 workgroups.  13240 tokens x 8
    // heads of 128 + 128: 25.1 us so, the same with up to 1024 or 4096, 35.4 with 8192; in pages of 128
    // 30.3 us, and 32.5 with 4096.
    int run = 1;
    while (run < 64 && (T + run - 1) / run * heads > 2048) run *= 2;
    const dim3 grid((unsigned)((T + run - 1) / run), (unsigned)heads);
    kv_append_kernel<DK, DV, B, kVec><<<grid, dim3(kAppendThreads), 0, stream>>>(
        (const uint16_t*)k, k_ts, k_hs, (const uint16_t*)v, v_ts, v_hs, slot_map, T, run,
        (uint8_t*)k_cache, k_scales, (uint8_t*)v_cache, v_scales, pages * B, heads);
    return hipGetLastError();
}

hipError_t launch_kv_append(const void* k, int64_t k_ts, int64_t k_hs, const void* v, int64_t v_ts,
                            int64_t v_hs, const int32_t* slot_map, int64_t T, void* k_cache,
                            float* k_scales, void* v_cache, float* v_scales, int64_t pages,
                            int32_t page, int32_t heads, int32_t dk, int32_t dv,
                            hipStream_t stream) {
    const bool vec = ((uintptr_t)k | (uintptr_t)v) % 16 == 0 && ((k_ts | k_hs | v_ts | v_hs) % 8) == 0;
#define BFP8_APPEND(DK, DV, B)                                                                     \
    if (dk == DK && dv == DV && page == B)                                                         \
        return vec ? append_launch<DK, DV, B, true>(k, k_ts, k_hs, v, v_ts, v_hs, slot_map, T,     \
                                                    k_cache, k_scales, v_cache, v_scales, pages,   \
                                                    heads, stream)                                 \
                   : append_launch<DK, DV, B, false>(k, k_ts, k_hs, v, v_ts, v_hs, slot_map, T,    \
                                                     k_cache, k_scales, v_cache, v_scales, pages,  \
                                                     heads, stream);
#define BFP8_APPEND_PAGES(DK, DV) BFP8_APPEND(DK, DV, 32) BFP8_APPEND(DK, DV, 64) BFP8_APPEND(DK, DV, 128)
    BFP8_APPEND_PAGES(64, 64)
    BFP8_APPEND_PAGES(128, 128)
    BFP8_APPEND_PAGES(192, 128)
#undef BFP8_APPEND_PAGES
#undef BFP8_APPEND
    return hipErrorInvalidValue;
}

}  // namespace bfp8
