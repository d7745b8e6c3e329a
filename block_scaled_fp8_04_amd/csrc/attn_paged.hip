// attn_paged.hip - attention over the paged e4m3 cache on gfx950.
//
//     out = sum_t p_t v_t / sum_t p_t,   p_t = exp(scale q . k_t - max)
//
// Both products are taken transposed, keys and values as the first operand:
//     S^T [token, query] = K Q^T,     O^T [d, query] += V^T P^T
// A group of lanes takes the same run of a tile's tokens in both: the rows of K enter the first
// product in the order that leaves those tokens' results in that group's lanes, where they are
// the second product's P^T operand as they stand.  P never moves between lanes, and with values
// stored token-contiguous neither product's operands need a transposition.
//
// Precision.  Codes are widened to bf16 with their page's scale on the way to the matrix
// cores (exact: four significant bits and a power of two) and q is bf16 as it comes.  p
// enters as two bf16 terms, p rounded and the remainder, sixteen bits at any size of p: one
// term alone would be off by 2^-8, as much as the rounding of the output.  The fp8 product
// would take the codes as they are, but it drops what lies 2^-14 below the largest product of
// a 16-element group (measured), which moves a logit by 1e-5 of that product, and p as two
// e4m3 terms loses what lies 2^-22 below a tile's largest.  Logits, maxima,
// norms and sums are fp32.  Codes are widened with half their scale, because the largest value,
// 256 * 2^120 for an element of 248 * 2^120 or more, would be infinite, and its token's zero weight in
// the rows that do not see it NaN; logits and outputs get the factor of two back, so no result changes.
// Running maxima are rounded up to integers (in units of log 2), so that rescaling by 2^(old - new)
// is exact.
#include <algorithm>

#include "attn_common.hpp"
#include "device_codec.hpp"
#include "internal.hpp"
#include "tile_common.hpp"

namespace bfp8 {

constexpr int kAttnThreads = 256;
constexpr int kAttnWaves = kAttnThreads / 64;
constexpr int kCols = 16;                     // query columns of a wave
// Most query columns (new tokens times heads per KV head) of the kernels for few of them; the
// others widen the codes once for 128 or 256 columns.  32 requests x 4096 tokens x 8 heads of 128:
// 64 columns take 174 us by the former and 178 by the latter, 96 columns 260 and 182.
constexpr int kSplitMaxCols = 64;
// Eight fp32 as bf16 and the remainders as bf16.
__device__ __forceinline__ void split8(const float (&p)[8], bf8v& hi, bf8v& lo) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        hi[j] = (__bf16)p[j];
        lo[j] = (__bf16)(p[j] - (float)hi[j]);
    }
}

// Reads through the scalar cache (uniform addresses): page numbers and scales.
typedef const __attribute__((address_space(4))) int32_t* scalar_i32;
typedef const __attribute__((address_space(4))) float* scalar_f32;

// A value that is the same in all lanes, in scalar registers (where the compiler cannot see it).
__device__ __forceinline__ int64_t uniform(int64_t x) {
    return (int64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)x) |
           (int64_t)__builtin_amdgcn_readfirstlane((int)(x >> 32)) << 32;
}

// Lengths reach 2^31 - 32 (pages of 32 tokens).  Pieces of `per` tokens that hold `tokens`, and the
// table entry of a token `ahead` of a tile's first one, which may lie beyond the length: both pass
// 31 bits on the way.
constexpr int pieces(int tokens, int per) { return (int)(((uint32_t)tokens + per - 1) / per); }
constexpr uint32_t entry_ahead(int tile, int per, int ahead, int log_b) {
    return ((uint32_t)tile * per + ahead) >> log_b;
}
static_assert(pieces(INT32_MAX - 31, 64) == 1 << 25 && pieces(INT32_MAX - 31, 256) == 1 << 23 && pieces(0, 64) == 0,
              "the largest length's pieces");
static_assert(entry_ahead((1 << 25) + 24, 64, 63 * 32, 5) == (1u << 26) + 48 + 63,
              "an entry past the largest length");

// What an item's columns are: shared by all kernels.
struct Item {
    int64_t q0;
    int n, cols, kv_len, G;
    static __device__ __forceinline__ Item of(const AttnArgs& a, int from, int to, int kv_len) {
        Item it;
        it.G = a.heads_q / a.heads_kv;
        it.q0 = min(max((int64_t)from, (int64_t)0), a.T);
        const int64_t q1 = min(max((int64_t)to, it.q0), a.T);
        it.n = (int)(q1 - it.q0);
        it.cols = (int)min((int64_t)it.n, a.max_new) * it.G;
        it.kv_len = (int)min(max((int64_t)kv_len, (int64_t)0), a.width << a.log_b);
        return it;
    }
    static __device__ __forceinline__ Item of(const AttnArgs& a, int r) {
        return of(a, a.q_offsets[r], a.q_offsets[r + 1], a.kv_lens[r]);
    }
    // tokens that column c sees
    __device__ __forceinline__ int limit(int c) const {
        return min(kv_len, max(kv_len - n + c / G + 1, 0));
    }
    __device__ __forceinline__ const uint16_t* row(const AttnArgs& a, int h, int c) const {
        return a.q + (q0 + c / G) * a.q_ts + (int64_t)(h * G + c % G) * a.q_hs;
    }
};

// 64 consecutive requests, one per lane: what a workgroup has to know of the requests it meets,
// read at once.  Reads that follow one another, each for the next one's address, are what a short
// call spends its time on.
struct Requests {
    int base;                                        // the first one
    int tiles0, tiles1, q0, q1, kv_len;              // of request base + lane
    __device__ __forceinline__ void load(const AttnArgs& a, int from) {
        base = from;
        const int r = min(base + (int)(threadIdx.x & 63), a.R - 1);
        tiles0 = a.tile_offsets[r];
        tiles1 = a.tile_offsets[r + 1];
        q0 = a.q_offsets[r];
        q1 = a.q_offsets[r + 1];
        kv_len = a.kv_lens[r];
    }
    // of request r, in scalar registers
    __device__ __forceinline__ int tiles_from(int r) const { return __builtin_amdgcn_readlane(tiles0, r - base); }
    __device__ __forceinline__ int tiles_to(int r) const { return __builtin_amdgcn_readlane(tiles1, r - base); }
    __device__ __forceinline__ Item item(const AttnArgs& a, int r) const {
        return Item::of(a, __builtin_amdgcn_readlane(q0, r - base), __builtin_amdgcn_readlane(q1, r - base),
                        __builtin_amdgcn_readlane(kv_len, r - base));
    }
};
static_assert(kKvMaxRequests <= 64 * 64, "a request is found in two steps of 64");

__device__ __forceinline__ bool q_vec(const AttnArgs& a) {
    return ((uintptr_t)a.q % 16) == 0 && ((a.q_ts | a.q_hs) % 8) == 0;
}
// The factor of half the logits that makes them exponents of two.
__device__ __forceinline__ float exp2_scale(const AttnArgs& a) {
    return 2.f * fmaxf(__builtin_fabsf(a.scale) * kLog2e, 0x1p-126f);     // -inf times 0 is NaN
}
// Twice 1 / l for sums over half the values; 0 for a row that sees nothing.
__device__ __forceinline__ float out_factor(float l) { return l == 0.f ? 0.f : 2.0f / l; }

// A run of tiles of one item that a workgroup walks; its waves take every fourth one.
struct Segment {
    int r, h, ct;
    int t0, t1;                                      // tiles of TT tokens
    int whole;                                       // the item's only run
};

// One wave's attention of kCols query columns over TT-token tiles, page size B.
//
// Each wave brings its own tiles to LDS, by loads that bypass the registers, and reads them
// back as fragments; nothing is shared between waves, so there is no barrier in the loop.  A
// fragment's lanes take sixteen different rows, and read straight from memory that way every
// 16 bytes are an access of their own: 3.8 instead of 5.1 TB/s (64 requests, 180k tokens, 8
// heads of 128).  The next tile's keys are requested when this tile's have been multiplied,
// its values when this tile's have: one of the two is always on its way while the wave
// computes, and the keys also while the waves of a finished item are joined.  The loads are
// non-temporal (without the hint 4.8 TB/s).
//
// Lane group g = lane / 16 holds tokens TT / 4 * g .. of a tile.  In LDS a row's 16-byte
// chunks are permuted (by exclusive or with k_swz, v_swz of the row), so that the sixteen
// rows that lanes read together lie in different banks.
template <int DK, int DV, int B, int TT>
struct AttnWave {
    static constexpr int LT = TT / 4;                // tokens per lane group
    static constexpr int KT = TT / 16;               // 16-row tiles of S^T
    static constexpr int PM = TT / 32;               // matrix instructions per 16 rows of O^T
    static constexpr int KF = DK / 32;               // matrix instructions per 16 keys
    static constexpr int DT = DV / 16;               // 16-row tiles of O^T
    static constexpr int NP = TT > B ? TT / B : 1;   // pages of a tile
    static constexpr int VB = TT > B ? B : TT;       // bytes of a value row in one page
    static constexpr int K_BYTES = TT * DK, V_BYTES = TT * DV;
    static constexpr int NK = K_BYTES / 1024, NV = V_BYTES / 1024;      // loads per tile
    static_assert(kCols * DV * 4 <= V_BYTES, "results fit the wave's values");

    bf8v q[KF];                                      // lane group g: dims DK / 4 * g + 8 i ..
    v4f o[DT];
    float m, l;                                      // l: this lane's tokens only
    int entry[NP];                                   // table entries of the tile after the next
    int64_t page[NP];                                // page * heads + head of the tile loaded last
    float ks[NP], vs[NP];                            // and its scales

    // bits 4 .. of a chunk's place that depend on the row
    static __device__ __forceinline__ int k_swz(int token) {
        const int x = token / LT & 3;
        return DK == 128 ? ((token >> 1 & 1) | x << 1) << 4 : x << 4;
    }
    static __device__ __forceinline__ int v_swz(int d) {
        return (VB == 128 ? d >> 1 & 7 : VB == 64 ? d >> 2 & 3 : d >> 3 & 1) << 4;
    }

    // column `lane & 15` is this query row (NULL: an unused column)
    __device__ __forceinline__ void load_q(const uint16_t* row, bool vec, bool negate, int g) {
#pragma unroll
        for (int i = 0; i < KF; ++i)
            q[i] = row ? load_q8(row + DK / 4 * g + 8 * i, vec, negate) : bf8v{0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d] = v4f{0.f, 0.f, 0.f, 0.f};
        m = neg_inf();
        l = 0.f;
#pragma unroll
        for (int p = 0; p < NP; ++p) entry[p] = 0;
    }

    __device__ __forceinline__ void read_table(const AttnArgs& a, int r, int tile, int kv_len) {
        const scalar_i32 table = (scalar_i32)(uintptr_t)(a.block_table + r * a.width);
#pragma unroll
        for (int p = 0; p < NP; ++p)
            entry[p] = table[max(min((tile * TT + p * B) / B, (kv_len - 1) / B), 0)];
    }
    __device__ __forceinline__ void find_pages(const AttnArgs& a, int h) {
        const scalar_f32 k_scales = (scalar_f32)(uintptr_t)a.k_scales;
        const scalar_f32 v_scales = (scalar_f32)(uintptr_t)a.v_scales;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            page[p] = min(max((int64_t)entry[p], (int64_t)0), a.pages - 1) * a.heads_kv + h;
            ks[p] = k_scales[page[p]];
            vs[p] = v_scales[page[p]];
        }
    }
    // real: otherwise the loads are out of their resource's range and read nothing
    __device__ __forceinline__ void load_k(const AttnArgs& a, uint8_t* lds_k, int tile, bool real) {
        const int lane = threadIdx.x & 63;
        const int row = lane / (DK / 16), at = lane % (DK / 16);
        const int in_page = TT < B ? tile * TT & (B - 1) : 0;
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            const int p = i * 1024 / DK / B;                    // all of a load's rows are in one page
            const __amdgpu_buffer_rsrc_t src =
                make_rsrc(a.k_cache + uniform(page[p]) * ((int64_t)B * DK), real ? (uint64_t)B * DK : 0);
            int voff;
            if constexpr (DK == 192) {
                const int x = i % 3 * 64 + lane;                // 16 rows are three loads
                voff = ((x / 12) * 192 + x % 12 * 16) ^ (i / 3 * 16 / LT & 3) << 4;
            } else {
                voff = (row * DK + at * 16) ^ k_swz(i * (1024 / DK) + row);
            }
            const int from = (DK == 192 ? i / 3 * 3072 : i * 1024) - p * B * DK + in_page * DK;
            buf_lds16_nt(src, voff, from, lds_k + i * 1024);
        }
    }
    __device__ __forceinline__ void load_v(const AttnArgs& a, uint8_t* lds_v, int tile) {
        constexpr int PER = DV * VB / 1024, RI = 1024 / VB;     // loads per page, rows per load
        const int lane = threadIdx.x & 63;
        const int row = lane / (VB / 16), at = lane % (VB / 16);
        const int in_page = TT < B ? tile * TT & (B - 1) : 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int p = i / PER;
            const __amdgpu_buffer_rsrc_t src =
                make_rsrc(a.v_cache + uniform(page[p]) * ((int64_t)B * DV), (uint64_t)B * DV);
            const int voff = row * B + (at * 16 ^ v_swz(i * RI + row));
            buf_lds16_nt(src, voff, i % PER * RI * B + in_page, lds_v + i * 1024);
        }
    }
    static __device__ __forceinline__ float pick(const float (&x)[NP], int token) {
        float y = x[0];                                         // the scale of a lane's tokens
#pragma unroll
        for (int p = 1; p < NP; ++p)
            if (token / B == p) y = x[p];
        return y;
    }

    // This wave's tiles of segment s.  lds_k, lds_v: its LDS bytes, of two arrays (so that reads of
    // the one are seen not to wait for loads into the other).  limit: this column sees tokens
    // below it; free_limit: every column sees those below.  next (NULL: none) is the segment
    // after this one, in which the wave's first tile is n0 < next->t1: its keys are requested here.
    // ready: the first tile's keys were requested by the walk before.  Everything but limit is
    // uniform.
    __device__ __forceinline__ void walk(const AttnArgs& a, uint8_t* lds_k, uint8_t* lds_v,
                                         const Segment& s, int t0, int kv_len, int limit,
                                         int free_limit, float c, bool ready, bool has_next,
                                         const Segment& next, int n0, int n_kv_len) {
        const int lane = threadIdx.x & 63, g = lane >> 4, lr = lane & 15;
        const int t1 = __builtin_amdgcn_readfirstlane(s.t1);
        t0 = __builtin_amdgcn_readfirstlane(t0);
        n0 = __builtin_amdgcn_readfirstlane(n0);
        // fragments: this lane's K rows are tokens ktok + 4 t, its V rows lr + 16 d
        const int ktok = LT * (lr >> 2) + (lr & 3);
        const uint8_t* kf[DK / 64];
#pragma unroll
        for (int x = 0; x < DK / 64; ++x)
            kf[x] = lds_k + ktok * DK + ((DK / 64 * g + x) * 16 ^ k_swz(ktok));
        const uint8_t* vf[LT / 16];
#pragma unroll
        for (int y = 0; y < LT / 16; ++y) {
            const int tok = LT * g + 16 * y;
            vf[y] = lds_v + tok / VB * (DV * VB) + lr * VB + (tok % VB ^ v_swz(lr));
        }
        if (!ready) {
            read_table(a, s.r, t0, kv_len);
            find_pages(a, s.h);
            load_k(a, lds_k, t0, true);
        }
        load_v(a, lds_v, t0);
        const auto read_after = [&](int tile) {                 // the entry of the tile after `tile`
            if (tile + kAttnWaves < t1) read_table(a, s.r, tile + kAttnWaves, kv_len);
            else if (has_next) read_table(a, next.r, n0, n_kv_len);
        };
        read_after(t0);
        // one tile; kMore: this wave has another one in the segment
        const auto tile_step = [&](auto more, int tile) {
            constexpr bool kMore = decltype(more)::value != 0;
            const int base = tile * TT;
            wait_vmcnt<NV>();                                   // this tile's keys have landed
            __builtin_amdgcn_sched_barrier(0);
            const float ke = 0.5f * pick(ks, LT * (lr >> 2)), ve = 0.5f * pick(vs, LT * g);
            v4f x[KT];
#pragma unroll
            for (int t = 0; t < KT; ++t) x[t] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < DK / 64; ++i) {
#pragma unroll
                for (int t = 0; t < KT; ++t) {
                    const uint4 w = *(const uint4*)(kf[i] + 4 * t * DK);
                    x[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8((int)w.x, (int)w.y, ke), q[2 * i],
                                                                   x[t], 0, 0, 0);
                    x[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8((int)w.z, (int)w.w, ke),
                                                                   q[2 * i + 1], x[t], 0, 0, 0);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
            // the next tile's keys; with none left, loads that read nothing: a branch around them
            // would make the waits below cover the shorter path, which is too much
            find_pages(a, kMore ? s.h : next.h);
            load_k(a, lds_k, kMore ? tile + kAttnWaves : n0, kMore || has_next);
            if constexpr (kMore) read_after(tile + kAttnWaves);
            __builtin_amdgcn_sched_barrier(0);
            uint32_t mask[LT / 4];
#pragma unroll
            for (int w = 0; w < LT / 4; ++w) mask[w] = 0xFFFFFFFFu;
            if (base > free_limit - TT) {
                const int seen = limit - base - LT * g;         // this lane's tokens: the first `seen`
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (4 * t + i >= seen) x[t][i] = neg_inf();
                // bytes behind the last token may hold anything: 0 * NaN is NaN
                const int live = kv_len - base - LT * g;
#pragma unroll
                for (int w = 0; w < LT / 4; ++w) {
                    const int n = min(max(live - 4 * w, 0), 4);
                    mask[w] = n == 4 ? 0xFFFFFFFFu : (1u << (8 * n)) - 1;
                }
            }
            bf8v ph[PM], pl[PM];
            softmax(x, c, ph, pl);
            wait_vmcnt<NK>();                                   // this tile's values have landed
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int y = 0; y < LT / 16; ++y)
#pragma unroll
                for (int d = 0; d < DT; ++d) {
                    const uint4 w = *(const uint4*)(vf[y] + 16 * d * VB);
                    const bf8v x0 = widen8((int)(w.x & mask[4 * y]), (int)(w.y & mask[4 * y + 1]), ve);
                    o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x0, ph[2 * y], o[d], 0, 0, 0);
                    o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x0, pl[2 * y], o[d], 0, 0, 0);
                    const bf8v x1 = widen8((int)(w.z & mask[4 * y + 2]), (int)(w.w & mask[4 * y + 3]), ve);
                    o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x1, ph[2 * y + 1], o[d], 0, 0, 0);
                    o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x1, pl[2 * y + 1], o[d], 0, 0, 0);
                }
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (kMore) load_v(a, lds_v, tile + kAttnWaves);
            __builtin_amdgcn_sched_barrier(0);
        };
        int tile = t0;
        for (; tile + kAttnWaves < t1; tile += kAttnWaves) tile_step(StageId<1>{}, tile);
        tile_step(StageId<0>{}, tile);
    }

    // S^T of one tile to P^T, with this lane's tokens 8 i .. 8 i + 7 in ph[i] (rounded) and pl[i]
    // (the remainder); rescales o and l to the new running maximum.
    __device__ __forceinline__ void softmax(v4f (&s)[KT], float c, bf8v (&ph)[PM], bf8v (&pl)[PM]) {
        float mx = s[0][0];
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) mx = fmaxf(mx, s[t][i]);
        mx = fmaxf(mx, __shfl_xor(mx, 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        const float m_new = fmaxf(m, __builtin_ceilf(mx * c));
        // logits so large that fp32 cannot hold s c - m to a unit: round s c alone, as m was, so
        // that the largest keeps p = 1
        if (__any(__builtin_fabsf(m_new) > 4194304.f && m_new != neg_inf())) {
#pragma unroll
            for (int t = 0; t < KT; ++t) s[t] *= c;
            c = 1.f;
        }
        const float sub = m_new == neg_inf() ? 0.f : -m_new;    // nothing seen yet: every p is 0
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < PM; ++i) {
            float p[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                p[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[2 * i + (j >> 2)][j & 3], c, sub));
                sum += p[j];
            }
            split8(p, ph[i], pl[i]);
        }
        if (m != m_new) {
            const float alpha = __builtin_amdgcn_exp2f(m - m_new);
            l *= alpha;
#pragma unroll
            for (int d = 0; d < DT; ++d) o[d] *= alpha;
            m = m_new;
        }
        l += sum;
    }
};

// Barrier behind finished LDS accesses, leaving the loads that are on their way alone.
__device__ __forceinline__ void barrier_ds() {
    __builtin_amdgcn_s_waitcnt(0xC07F);                         // lgkmcnt(0)
    barrier_lds();
}

// Joins the four waves' results of one 16-column item in their bytes of lds_v (the keys' bytes
// may be receiving the next item's): first m and l, then each wave's O times 2^(m_w - m), its
// four-dim groups permuted by the column against bank conflicts.  Thread x gets column x / 16,
// dims 4 (x % 16) + 64 j of the sum, in wave order, and that column's m and l.
template <class W, int DV>
__device__ __forceinline__ void join_waves(const W& w, uint8_t* lds_v, float (&part)[DV / 16], float& m,
                                           float& l) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, col = lane & 15;
    float ll = w.l + __shfl_xor(w.l, 16);
    ll += __shfl_xor(ll, 32);
    float* const mine = (float*)(lds_v + wave * W::V_BYTES);
    if (g == 0) {
        mine[col] = w.m;
        mine[kCols + col] = ll;
    }
    barrier_ds();
    const int oc = tid >> 4;
    float mw[kAttnWaves], m_col = neg_inf();
    m = neg_inf();
#pragma unroll
    for (int x = 0; x < kAttnWaves; ++x) {
        const float* const theirs = (const float*)(lds_v + x * W::V_BYTES);
        mw[x] = theirs[oc];
        m = fmaxf(m, mw[x]);
        m_col = fmaxf(m_col, theirs[col]);
    }
    l = 0.f;
#pragma unroll
    for (int x = 0; x < kAttnWaves; ++x) {
        const float lw = ((const float*)(lds_v + x * W::V_BYTES))[kCols + oc];
        if (mw[x] != neg_inf() || lw != 0.f) l = __builtin_fmaf(lw, __builtin_amdgcn_exp2f(mw[x] - m), l);
    }
    barrier_ds();
    // a wave that saw nothing in the column has zeros there
    const float f = w.m == neg_inf() ? 1.f : __builtin_amdgcn_exp2f(w.m - m_col);
#pragma unroll
    for (int d = 0; d < DV / 16; ++d) *(v4f*)(mine + col * DV + ((4 * d + g) ^ col) * 4) = w.o[d] * f;
    barrier_ds();
#pragma unroll
    for (int j = 0; j < DV / 16; ++j) part[j] = 0.f;
#pragma unroll
    for (int x = 0; x < kAttnWaves; ++x) {
        const float* const theirs = (const float*)(lds_v + x * W::V_BYTES);
#pragma unroll
        for (int j = 0; j < DV / 64; ++j) {
            const v4f v = *(const v4f*)(theirs + oc * DV + (((tid & 15) + 16 * j) ^ oc) * 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) part[4 * j + i] += v[i];
        }
    }
    barrier_ds();                                            // before the next item's values
}

template <int DV>
__device__ __forceinline__ void store_row(const AttnArgs& a, int64_t row, int head, int od,
                                          const float (&part)[DV / 16], float m, float l) {
    const float r = out_factor(l);
    uint16_t* const out = a.out + (row * a.heads_q + head) * DV + od;
#pragma unroll
    for (int j = 0; j < DV / 64; ++j) {
        const uint2 w = make_uint2(pack_bf16x2(part[4 * j] * r, part[4 * j + 1] * r),
                                   pack_bf16x2(part[4 * j + 2] * r, part[4 * j + 3] * r));
        *(uint2*)(out + 64 * j) = w;
    }
    if (a.lse && od == 0)
        a.lse[row * a.heads_q + head] = l == 0.f ? neg_inf() : (m + __builtin_log2f(l)) * kLn2;
}

// Few query columns (a decode step, drafts): the 128-token tiles of all items, an item being
// (request, KV head, 16 columns), form one row of units that the workgroups divide evenly, so
// that ragged lengths and few long caches load the chip alike.  A workgroup walks its units
// item by item; an item that lies within one workgroup is finished there, the others leave
// partial sums (at most two of them per workgroup: its first and its last item) that
// attn_join_kernel adds in token order.
//
// Bound by reading the cache: 64 requests, 180k tokens, 8 heads of 128 (370 MB) take 70 + 5 us, 5.3
// TB/s, where a large copy's reads take 63 us.  One token over 1030: 7.3 + 4 us, which is latency:
// four dependent reads, one tile, the join.  There a workgroup takes a single 128-token tile; with
// four tiles, one for each wave twice, it is 13.2 us.  The kernel has more uniform values than scalar
// registers: the compiler keeps 28 to 79 of them in lanes of vector registers.

// Workgroups: at 128/128 and 192/128 as many as the CUs hold at once, two each (16 and 20 KB of LDS a
// wave): 64 requests, 180k tokens, 64 heads on 8 of 128 take 74.5 us, with 768 workgroups 79.5, with
// 1024 75.3.  At 64/64 the registers (137) let three a CU run, and 1024 workgroups are more than that:
// the same requests take 47.1 us at 64/64, with 768 44.7, with 512 46.5; 24 requests of four drafts 17.2,
// 16.6 and 16.4.
constexpr int split_groups(int dv) { return dv == 64 ? 1024 : 512; }

struct SplitPlan {
    int64_t units;      // tiles of all items
    int64_t per;        // tiles per workgroup
};

template <int DV>
__device__ __forceinline__ SplitPlan split_plan(const AttnArgs& a, int tiles, int col_tiles) {
    const int64_t units = (int64_t)max(tiles, 0) * a.heads_kv * col_tiles;
    return {units, max((units + split_groups(DV) - 1) / split_groups(DV), (int64_t)1)};
}

// One workgroup per (request, KV head, 16 query columns): its waves take every fourth tile.
template <int DK, int DV, int B, int TT>
__global__ __launch_bounds__(kAttnThreads) void attn_item_kernel(AttnArgs a, int col_tiles) {
    using W = AttnWave<DK, DV, B, TT>;
    __shared__ __attribute__((aligned(1024))) uint8_t lds_k[kAttnWaves * W::K_BYTES];
    __shared__ __attribute__((aligned(1024))) uint8_t lds_v[kAttnWaves * W::V_BYTES];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    uint32_t item = blockIdx.x;
    const int ct = (int)(item % col_tiles);
    item /= col_tiles;
    const int h = (int)(item % a.heads_kv);
    const int r = __builtin_amdgcn_readfirstlane((int)(item / a.heads_kv));
    const Item it = Item::of(a, r);
    if (ct * kCols >= it.cols) return;
    const int col = ct * kCols + (lane & 15);
    const bool used = col < it.cols;
    W w;
    w.load_q(used ? it.row(a, h, col) : nullptr, q_vec(a), a.scale < 0.f, lane >> 4);
    Segment seg;
    seg.r = r;
    seg.h = h;
    seg.ct = ct;
    seg.t0 = 0;
    seg.t1 = pieces(it.limit(min(ct * kCols + kCols, it.cols) - 1), TT);
    seg.whole = 1;
    if (wave < seg.t1)
        w.walk(a, lds_k + wave * W::K_BYTES, lds_v + wave * W::V_BYTES, seg, wave, it.kv_len,
               used ? it.limit(col) : 0, it.limit(ct * kCols), exp2_scale(a), false, false, seg, 0, 0);
    float part[DV / 16], m, l;
    join_waves<W, DV>(w, lds_v, part, m, l);
    const int oc = ct * kCols + (tid >> 4);
    if (oc < it.cols)
        store_row<DV>(a, it.q0 + oc / it.G, h * it.G + oc % it.G, (tid & 15) * 4, part, m, l);
    wait_vmcnt<0>();                                            // no load outlives its LDS
}

template <int DK, int DV, int B, int TT>
__global__ __launch_bounds__(kAttnThreads) void attn_split_kernel(AttnArgs a, int col_tiles) {
    using W = AttnWave<DK, DV, B, TT>;
    __shared__ __attribute__((aligned(1024))) uint8_t lds_k[kAttnWaves * W::K_BYTES];
    __shared__ __attribute__((aligned(1024))) uint8_t lds_v[kAttnWaves * W::V_BYTES];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    Requests reqs;
    reqs.load(a, 0);
    const int each64 = a.tile_offsets[min(lane * 64, a.R)];
    const SplitPlan sp = split_plan<DV>(a, __builtin_amdgcn_readfirstlane(a.tile_offsets[a.R]), col_tiles);
    int64_t u = (int64_t)blockIdx.x * sp.per;
    const int64_t end = min(u + sp.per, sp.units);
    if (u >= end) return;
    const int64_t items = (int64_t)a.heads_kv * col_tiles;   // of one request
    // the request of the first unit
    const int64_t ut = quotient(u, items);
    const int from = last_of(lane * 64 < a.R && each64 <= ut) * 64;
    if (from > 0) reqs.load(a, from);
    int r = __builtin_amdgcn_readfirstlane(from + last_of(from + lane < a.R && reqs.tiles0 <= ut));
    // the workgroup's next run of tiles, from unit u on
    const auto advance = [&](Segment& s, Item& it) {
        for (; r < a.R && u < end; ++r) {
            if (r - reqs.base >= 64) reqs.load(a, r);
            const int64_t f = reqs.tiles_from(r);
            const int nt = (int)min(max((int64_t)reqs.tiles_to(r) - f, (int64_t)0), (int64_t)1 << 24);
            const int64_t local = max(u - f * items, (int64_t)0);
            if (nt <= 0 || local >= (int64_t)nt * items) continue;
            const int item = __builtin_amdgcn_readfirstlane((int)quotient(local, nt));
            const int tile0 = (int)(local - (int64_t)item * nt);
            const int count = (int)min((int64_t)(nt - tile0), end - u);
            u += count;
            s.r = r;
            s.h = __builtin_amdgcn_readfirstlane(item / col_tiles);
            s.ct = item - s.h * col_tiles;
            s.t0 = tile0 * (kKvTile / TT);
            s.t1 = (tile0 + count) * (kKvTile / TT);
            s.whole = count == nt;
            it = reqs.item(a, r);
            return true;
        }
        return false;
    };
    bool first = true, ready = false;
    int64_t page[W::NP] = {};                                  // of the keys that are on their way
    float ks[W::NP] = {}, vs[W::NP] = {};
    Segment cur, next;
    Item it = {}, nit;
    bool valid = advance(cur, it);
    while (valid) {
        next = cur;                                             // defined, and inside the pool, if there is none
        nit = it;
        const bool has = advance(next, nit);
        W w;
        const int col = cur.ct * kCols + (lane & 15);
        const bool used = col < it.cols;
        if (cur.ct * kCols < it.cols) {
            cur.t1 = min(cur.t1, pieces(it.kv_len, TT));
            const int n1 = next.ct * kCols < nit.cols ? min(next.t1, pieces(nit.kv_len, TT)) : 0;
            const bool chain = has && next.t0 + wave < n1;
            w.load_q(used ? it.row(a, cur.h, col) : nullptr, q_vec(a), a.scale < 0.f, lane >> 4);
            if (cur.t0 + wave < cur.t1) {
#pragma unroll
                for (int p = 0; p < W::NP; ++p) {
                    w.page[p] = page[p];
                    w.ks[p] = ks[p];
                    w.vs[p] = vs[p];
                }
                w.walk(a, lds_k + wave * W::K_BYTES, lds_v + wave * W::V_BYTES, cur, cur.t0 + wave,
                       it.kv_len, used ? it.limit(col) : 0, it.limit(cur.ct * kCols), exp2_scale(a), ready,
                       chain, next, next.t0 + wave, nit.kv_len);
#pragma unroll
                for (int p = 0; p < W::NP; ++p) {
                    page[p] = w.page[p];
                    ks[p] = w.ks[p];
                    vs[p] = w.vs[p];
                }
                ready = chain;
            }
            float part[DV / 16], m, l;
            join_waves<W, DV>(w, lds_v, part, m, l);
            const int x = tid >> 4, oc = cur.ct * kCols + x, od = (tid & 15) * 4;
            if (oc < it.cols) {
                if (cur.whole) {
                    store_row<DV>(a, it.q0 + oc / it.G, cur.h * it.G + oc % it.G, od, part, m, l);
                } else {
                    const int64_t slot = ((int64_t)blockIdx.x * 2 + (first ? 0 : 1)) * kCols + x;
                    float* const ws = a.ws + slot * DV + od;
#pragma unroll
                    for (int j = 0; j < DV / 64; ++j)
                        *(v4f*)(ws + 64 * j) = v4f{part[4 * j], part[4 * j + 1], part[4 * j + 2],
                                                   part[4 * j + 3]};
                    if (od == 0) {
                        float* const ml = a.ws + (int64_t)split_groups(DV) * 2 * kCols * DV + slot * 2;
                        ml[0] = m;
                        ml[1] = l;
                    }
                }
            }
        }
        first = false;
        cur = next;
        it = nit;
        valid = has;
    }
    wait_vmcnt<0>();                                            // no load outlives its LDS
}

// Partial sums of one row, or of a strand of it: O, l and the maximum they refer to.
struct Part {
    v4f acc = {0.f, 0.f, 0.f, 0.f};
    float m = neg_inf(), l = 0.f;
    __device__ __forceinline__ void add(const v4f& v, float mw, float lw) {
        const float top = fmaxf(m, mw);
        const float f0 = m == top ? 1.f : __builtin_amdgcn_exp2f(m - top);
        const float f1 = mw == top ? 1.f : __builtin_amdgcn_exp2f(mw - top);
        m = top;
        l = __builtin_fmaf(lw, f1, l * f0);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(v[i], f1, acc[i] * f0);
    }
    __device__ __forceinline__ void store(const AttnArgs& a, int64_t row, int dv, int d4) const {
        const float rl = out_factor(l);
        *(uint2*)(a.out + row * dv + d4) =
            make_uint2(pack_bf16x2(acc[0] * rl, acc[1] * rl), pack_bf16x2(acc[2] * rl, acc[3] * rl));
        if (a.lse && d4 == 0) a.lse[row] = l == 0.f ? neg_inf() : (m + __builtin_log2f(l)) * kLn2;
    }
};

// Adds the partial sums of the workgroups that shared an item, one row (item column) by STRANDS
// strands of DV / 4 lanes each: every strand takes its workgroups in token order, then the strands
// are added in order.  Rows of a request without tokens get their zeros here.
template <int DV, int STRANDS>
__global__ __launch_bounds__(kAttnThreads) void attn_join_kernel(AttnArgs a, int col_tiles, int max_cols) {
    constexpr int L = DV / 4, ROWS = kAttnThreads / (L * STRANDS), GROUPS = split_groups(DV);
    __shared__ float red[kAttnThreads / L][DV + 4];
    __shared__ float red_m[kAttnThreads / L], red_l[kAttnThreads / L];
    const int tid = threadIdx.x, strand = tid / L % STRANDS, d4 = tid % L * 4;
    const int64_t x = (int64_t)blockIdx.x * ROWS + tid / (L * STRANDS);
    const int64_t rh = quotient(x, max_cols);                   // request and KV head
    const int col = (int)(x - rh * max_cols);
    const int64_t rq = quotient(rh, a.heads_kv);
    const int h = (int)(rh - rq * a.heads_kv);
    const int r = (int)min(rq, (int64_t)a.R - 1);
    const int tiles = a.tile_offsets[a.R], from = a.tile_offsets[r], to = a.tile_offsets[r + 1];
    const Item it = Item::of(a, r);
    const bool live = rq < a.R && col < it.cols;
    const int64_t t0 = max(from, 0), nt = (int64_t)to - t0;
    const int64_t row = (it.q0 + col / it.G) * a.heads_q + h * it.G + col % it.G;
    const SplitPlan sp = split_plan<DV>(a, tiles, col_tiles);
    const int64_t begin = t0 * a.heads_kv * col_tiles + ((int64_t)h * col_tiles + col / kCols) * nt;
    const int wa = (int)min(quotient(begin, sp.per), (int64_t)GROUPS);
    const int wb = (int)min(quotient(begin + max(nt, (int64_t)1) - 1, sp.per), (int64_t)GROUPS - 1);
    const bool joins = live && nt > 0 && wa < wb;               // else finished by one workgroup
    Part part;
    if (joins) {
        const float* const ml = a.ws + (int64_t)GROUPS * 2 * kCols * DV;
#pragma unroll 4
        for (int w = wa + strand; w <= wb; w += STRANDS) {
            const int64_t slot = ((int64_t)w * 2 + (w * sp.per >= begin ? 0 : 1)) * kCols + col % kCols;
            const float2 mw = *(const float2*)(ml + slot * 2);
            part.add(*(const v4f*)(a.ws + slot * DV + d4), mw.x, mw.y);
        }
    }
    const int mine = tid / L;
    *(v4f*)&red[mine][d4] = part.acc;
    if (tid % L == 0) {
        red_m[mine] = part.m;
        red_l[mine] = part.l;
    }
    __syncthreads();
    if (strand != 0 || !live || (nt > 0 && !joins)) return;
#pragma unroll
    for (int i = 1; i < STRANDS; ++i) part.add(*(const v4f*)&red[mine + i][d4], red_m[mine + i], red_l[mine + i]);
    part.store(a, row, DV, d4);
}

// ---------------------------------------------------------------- many query columns
//
// Prompts and chunks: a workgroup takes 32 columns a wave of one request and KV head and walks
// the tokens they see.  The products and the softmax beside them bound this, so the codes are
// widened with their scales once per workgroup on their way into LDS, and every wave reads its
// fragments from there.
//
// p enters its product as two bf16 terms here too, for the same fragment of values; p may pass 1,
// up to 2^kSlack: a maximum over 32 columns that is followed at once moves in every second step
// (2048 tokens over 32k), and O has to be rescaled each time.
//
// A step forms the logits of 32 tokens, does the softmax of the 32 before and adds the values of
// the 32 before those: three independent streams, written out so that each matrix instruction
// (32 cycles) is followed by the vector work that fits beside it and by the LDS read of a fragment
// three instructions on.  S^T's rows are the tokens
// with bits 2 and 3 exchanged, which makes its registers the second product's operand as they
// stand.
//
// 2048 tokens behind 30000, 32 heads of 192/128: 1.52 to 1.55 ms, 0.85 PFLOP/s of the operator's own
// products (the matrix cores also multiply the remainders of p: 1.2 PFLOP/s).  The two waves of
// a SIMD keep the matrix cores 61 % busy (counters): an element has 56 cycles of matrix instructions
// and 10.6 vector instructions, at least 42 cycles, of the softmax, of splitting p and of staging the
// next tile; and the clock falls to 1.85 GHz under this load.  One f16 term of p takes 1.21 ms and
// loses weights under
// 2^-32 of the largest, which show where the largest one's value is zero.  64 columns a wave (one
// wave a SIMD) 1.47 ms against 1.24 at that time, four waves a workgroup 1.32 against 1.21.
typedef float v16f __attribute__((ext_vector_type(16)));

constexpr int kBlockTile = 64;                // tokens in LDS at a time
// Workgroups that a split launch aims at: two a CU.  1024: 215 us against 203 (256 tokens behind 30k,
// 32 heads on 8); behind 2k, 8 heads on 2, both 24.
constexpr int kBlockSlots = 512;
constexpr int kBlockMaxSplits = 16;
// Tokens that are not split further.  24 requests, decodes and chunks of up to 700 tokens: 44.3 us
// so, 43.6 with 512, 45.4 with 1024.
constexpr int kPartTokens = 256;
constexpr float kSlack = 8.f;

// Sum and maximum of the wave's values, in scalar registers.
template <int kCtrl, int kRows>
__device__ __forceinline__ int dpp(int x) { return __builtin_amdgcn_update_dpp(0, x, kCtrl, kRows, 0xF, false); }
template <class F>
__device__ __forceinline__ int wave_reduce(int x, F f) {
    x = f(x, dpp<0x111, 0xF>(x));                               // shifts within rows of 16 lanes
    x = f(x, dpp<0x112, 0xF>(x));
    x = f(x, dpp<0x114, 0xF>(x));
    x = f(x, dpp<0x118, 0xF>(x));
    x = f(x, dpp<0x142, 0xA>(x));                               // a row's last lane to the next row
    x = f(x, dpp<0x143, 0xC>(x));                               // and to the upper two rows
    return __builtin_amdgcn_readlane(x, 63);
}
// (of values that are not negative: lanes without a partner take 0)
__device__ __forceinline__ int wave_sum(int x) { return wave_reduce(x, [](int a, int b) { return a + b; }); }
__device__ __forceinline__ int wave_max(int x) { return wave_reduce(x, [](int a, int b) { return max(a, b); }); }

// Level of a request's first block of cb columns by the tokens that it sees beside its own, in units
// of a block's own; beyond kTopLevel (2^36 tokens times heads) blocks keep no order.
constexpr int kTopLevel = 1 << 29;
constexpr int first_level(int before, int G, int cb) {
    const uint64_t level = (uint64_t)before * G / cb;
    return level < kTopLevel ? (int)level : kTopLevel;
}
static_assert(first_level(INT32_MAX, 65535, 128) >= 0 && kTopLevel + ((INT32_MAX >> 7) + 1) < 1 << 30,
              "a level and the search's step above it fit 32 bits");

// A block of cb columns of a launch.  Request r's blocks are numbered from q_offsets[r] * G / cb + r
// on, where there is room for all of them.
struct Block {
    Item it;
    int r, c0, seen;                                 // first column; tokens that the last column sees
    __device__ __forceinline__ bool find(const AttnArgs& a, int b, int cb) {
        const int lane = threadIdx.x & 63, G = a.heads_q / a.heads_kv;
        const auto start = [&](int q, int r) {
            return (int64_t)((uint64_t)min(max((int64_t)q, (int64_t)0), a.T) * G / cb) + r;
        };
        Requests reqs;
        reqs.load(a, 0);
        const int each64 = a.q_offsets[min(lane * 64, a.R)];
        const int from = last_of(lane * 64 < a.R && start(each64, lane * 64) <= b) * 64;
        if (from > 0) reqs.load(a, from);
        r = __builtin_amdgcn_readfirstlane(
            from + last_of(from + lane < a.R && start(reqs.q0, from + lane) <= b));
        it = reqs.item(a, r);
        c0 = (int)min(b - start((int)it.q0, r), (int64_t)1 << 22) * cb;
        if (c0 < 0 || c0 >= it.cols) return false;
        seen = it.limit(min(c0 + cb, it.cols) - 1);
        return true;
    }
    // The block of this rank by the tokens that it sees, most first (in steps of a block's own
    // tokens); one request per lane, so for R <= 64.
    __device__ __forceinline__ bool ranked(const AttnArgs& a, int rank, int cb) {
        const int lane = threadIdx.x & 63;
        Requests reqs;
        reqs.load(a, 0);
        const Item mine = Item::of(a, reqs.q0, reqs.q1, reqs.kv_len);
        // level of a block: the level of its request's first one, and one more for each further
        const int count = lane < a.R ? (mine.cols + cb - 1) / cb : 0;
        const int low = first_level(max(mine.kv_len - mine.n, 0), mine.G, cb), high = low + count;
        const auto above = [&](int level) { return wave_sum(min(max(high - level, 0), count)); };
        if (above(0) <= rank) return false;
        int level = 0;                               // the highest with more than `rank` blocks from it on
        for (int step = 1 << (31 - __builtin_clz(wave_max(high) | 1)); step > 0; step >>= 1)
            if (above(level + step) > rank) level += step;
        const uint64_t here = __ballot(low <= level && level < high);
        const int nth = rank - above(level + 1);
        r = __ffsll((unsigned long long)__ballot((here >> lane & 1) &&
                                                 __popcll(here & ((1ull << lane) - 1)) == nth)) - 1;
        it = reqs.item(a, r);
        c0 = (level - __builtin_amdgcn_readlane(low, r)) * cb;
        seen = it.limit(min(c0 + cb, it.cols) - 1);
        return true;
    }
    // workgroups that share its tokens
    __device__ __forceinline__ int parts(int splits) const {
        return min(splits, max(pieces(seen, kPartTokens), 1));
    }
};

template <int DK, int DV, int WAVES>
__global__ __launch_bounds__(WAVES * 64, 2) void attn_block_kernel(AttnArgs a, int blocks, int splits) {
    constexpr int CB = 32 * WAVES, NT = 64 * WAVES;        // columns and threads of a workgroup
    constexpr int KS = DK / 16, DT = DV / 32;        // steps of the products, 32-row tiles of O^T
    constexpr int K_CHUNKS = kBlockTile * DK / 16, V_CHUNKS = kBlockTile * DV / 16;
    constexpr int KCH = (K_CHUNKS + NT - 1) / NT, VCH = (V_CHUNKS + NT - 1) / NT;
    constexpr int K_ROW = DK * 2, V_ROW = kBlockTile * 2;
    constexpr int K_BUF = kBlockTile * K_ROW, V_BUF = DV * V_ROW;
    __shared__ __attribute__((aligned(1024))) uint8_t lds_k[2 * K_BUF];
    __shared__ __attribute__((aligned(1024))) uint8_t lds_v[2 * V_BUF];
    const int tid = threadIdx.x, lane = tid & 63, hh = lane >> 5, lr = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int G = a.heads_q / a.heads_kv;

    // blocks that see the most tokens go first, for the last ones to end together: by rank (eight
    // prompts of 296 to 1662 tokens: 119 us, 122 by number), or by number from the last one down
    // where there are more requests than lanes, or the launch is split and runs all at once
    int idx = blockIdx.x;
    const int z = idx % splits;
    idx /= splits;
    const int h = idx % a.heads_kv, nth = idx / a.heads_kv;
    Block k;
    if (!(a.R <= 64 && splits == 1 ? k.ranked(a, nth, CB) : k.find(a, blocks - 1 - nth, CB))) return;
    const Item& it = k.it;
    const int r = k.r, c0 = k.c0, parts = k.parts(splits);
    if (z >= parts) return;
    const int seen_by_all = it.limit(c0);
    const int tiles = pieces(k.seen, kBlockTile);
    static_assert(kBlockMaxSplits <= 32, "2^25 tiles at most, so 32 bits will do");
    const int t_first = __builtin_amdgcn_readfirstlane(tiles * z / parts);
    const int t_end = __builtin_amdgcn_readfirstlane(tiles * (z + 1) / parts);
    const int n = t_end - t_first;
    const int kv_len = it.kv_len, last = max(kv_len - 1, 0) >> a.log_b, B = 1 << a.log_b;
    const float c = exp2_scale(a);

    bf8v q[KS];
    v16f o[DT];
    float m, l;
    const int col = c0 + wave * 32 + lr;
    const bool used = col < it.cols;
    const int limit = used ? it.limit(col) : 0;
    const uint16_t* const row = it.row(a, h, used ? col : c0);
    const bool vec = q_vec(a), negate = a.scale < 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) q[ks] = load_q8(row + 16 * ks + 8 * hh, vec, negate);
    m = neg_inf();
    l = 0.f;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] = 0.f;

    if (n > 0) {
        // staging: global codes of one tile in registers, widened into LDS later.  Page numbers and
        // scales of 64 groups of 32 tokens are held by the wave's lanes, the next 64 fetched while
        // these are in use: scalar loads in the loop would have every LDS wait behind them wait
        // for them too (they share a counter).
        uint4 kr[KCH], vr[VCH];
        struct Pages {                                           // of a tile's two 32-token groups
            int64_t page0, page1;
            float ks0, ks1, vs0, vs1;
        };
        int entry, entry_n = 0;
        float ks_l, vs_l, ks_n = 0.f, vs_n = 0.f;
        const auto fetch_table = [&](int tile) {                 // the lanes' entries from `tile` on
            const int j = (int)min(entry_ahead(tile, kBlockTile, 32 * lane, a.log_b), (uint32_t)last);
            return (int)min(max((int64_t)a.block_table[(int64_t)r * a.width + j], (int64_t)0), a.pages - 1);
        };
        const auto fetch_scale = [&](const float* x, int e) { return x[(int64_t)e * a.heads_kv + h]; };
        entry = fetch_table(t_first);
        ks_l = 0.5f * fetch_scale(a.k_scales, entry);
        vs_l = 0.5f * fetch_scale(a.v_scales, entry);
        const auto pages_at = [&](Pages& x, int at) {
            x.page0 = (int64_t)__builtin_amdgcn_readlane(entry, at) * a.heads_kv + h;
            x.page1 = (int64_t)__builtin_amdgcn_readlane(entry, at + 1) * a.heads_kv + h;
        };
        const auto scales_at = [&](Pages& x, int at) {
            const auto lane_of = [&](float x, int l) {
                return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(x), l));
            };
            x.ks0 = lane_of(ks_l, at);
            x.ks1 = lane_of(ks_l, at + 1);
            x.vs0 = lane_of(vs_l, at);
            x.vs1 = lane_of(vs_l, at + 1);
        };
        // of tile t_first + i, for i = 3, 4, 5, ... in order
        const auto pages_of = [&](int i) {
            const int at = 2 * i & 63;
            if (at == 0 && i > 0) {
                entry = entry_n;
                ks_l = 0.5f * ks_n;                              // (halved here: at the load, it would wait)
                vs_l = 0.5f * vs_n;
            }
            if (at == 16) entry_n = fetch_table(t_first + i + 24);
            if (at == 40) {
                ks_n = fetch_scale(a.k_scales, entry_n);
                vs_n = fetch_scale(a.v_scales, entry_n);
            }
            Pages x;
            pages_at(x, at);
            scales_at(x, at);
            return x;
        };
        const auto load_k = [&](uint4 (&kr)[KCH], int tile, const Pages& pg) {
            const int base = min(tile, t_end - 1) * kBlockTile;
#pragma unroll
            for (int e = 0; e < KCH; ++e) {
                const int x = e * NT + tid, token = x / (DK / 16), at = x % (DK / 16);
                // 64 chunks lie in one group: the page is the wave's
                const bool second = e * NT + wave * 64 >= K_CHUNKS / 2;
                const uint8_t* const page = a.k_cache + uniform(second ? pg.page1 : pg.page0) * ((int64_t)B * DK);
                if (K_CHUNKS % NT == 0 || x < K_CHUNKS)
                    kr[e] = *(const uint4*)(page + (uint32_t)(((base + token) & (B - 1)) * DK + 16 * at));
            }
        };
        const auto load_v = [&](int tile, const Pages& pg) {
            const int base = min(tile, t_end - 1) * kBlockTile;
#pragma unroll
            for (int e = 0; e < VCH; ++e) {
                const int x = e * NT + tid, d = x >> 2, token = (x & 3) * 16;
                const uint8_t* const page = a.v_cache + (token < 32 ? pg.page0 : pg.page1) * ((int64_t)B * DV);
                if (V_CHUNKS % NT == 0 || x < V_CHUNKS)
                    vr[e] = *(const uint4*)(page + (uint32_t)(d * B + ((base + token) & (B - 1))));
            }
        };
        // a row's 16-byte chunks are permuted so that the rows that lanes read together lie in
        // different banks
        const auto k_swz = [](int row) { return DK == 128 ? (row & 15) : (row >> 1 & 7); };
        const auto store_k = [&](const uint4 (&kr)[KCH], int buf, const Pages& pg) {
#pragma unroll
            for (int e = 0; e < KCH; ++e) {
                const int x = e * NT + tid, token = x / (DK / 16), at = x % (DK / 16);
                if (K_CHUNKS % NT != 0 && x >= K_CHUNKS) break;
                const float s = e * NT + wave * 64 >= K_CHUNKS / 2 ? pg.ks1 : pg.ks0;
                uint8_t* const to = lds_k + buf * K_BUF + token * K_ROW;
                *(bf8v*)(to + ((2 * at) ^ k_swz(token)) * 16) = widen8((int)kr[e].x, (int)kr[e].y, s);
                *(bf8v*)(to + ((2 * at + 1) ^ k_swz(token)) * 16) = widen8((int)kr[e].z, (int)kr[e].w, s);
            }
        };
        const auto store_v = [&](int tile, int buf, const Pages& pg) {
            const int live = kv_len - min(tile, t_end - 1) * kBlockTile;
#pragma unroll
            for (int e = 0; e < VCH; ++e) {
                const int x = e * NT + tid, d = x >> 2, token = (x & 3) * 16;
                if (V_CHUNKS % NT != 0 && x >= V_CHUNKS) break;
                uint32_t w[4] = {vr[e].x, vr[e].y, vr[e].z, vr[e].w};
                if (live < kBlockTile) {
                    // bytes behind the last token may hold anything: 0 * NaN is NaN
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const int k = min(max(live - token - 4 * y, 0), 4);
                        w[y] &= k == 4 ? 0xFFFFFFFFu : (1u << (8 * k)) - 1;
                    }
                }
                const int f = d >> 1 & 7;
                const float s = token < 32 ? pg.vs0 : pg.vs1;
                uint8_t* const to = lds_v + buf * V_BUF + d * V_ROW;
                *(bf8v*)(to + (((x & 3) * 2) ^ f) * 16) = widen8((int)w[0], (int)w[1], s);
                *(bf8v*)(to + (((x & 3) * 2 + 1) ^ f) * 16) = widen8((int)w[2], (int)w[3], s);
            }
        };
        // fragment places: K rows are tokens with bits 2 and 3 exchanged, V rows are lr + 32 d
        const int krow = (lr & 0x13) | (lr & 4) << 1 | (lr & 8) >> 1;
        constexpr int KA = DK == 128 ? 8 : 4;                    // k_swz takes 2 KA chunks: then it repeats
        int kat[KA], vat[4];
#pragma unroll
        for (int ks = 0; ks < KA; ++ks) kat[ks] = krow * K_ROW + (((2 * ks) ^ (k_swz(krow) ^ hh)) * 16);
#pragma unroll
        for (int x = 0; x < 4; ++x) vat[x] = lr * V_ROW + (((2 * x) ^ ((lr >> 1 & 7) ^ hh)) * 16);

        v16f s_even, s_odd;                              // logits of even and odd subtiles
        uint4 p_even[4], p_odd[4];                       // and their p: rounded, remainders
#pragma unroll
        for (int i = 0; i < 4; ++i) p_odd[i] = make_uint4(0, 0, 0, 0);
        // one step: values of subtile j - 1 (half VSUB of buffer VBUF), softmax of j, logits of j + 1
        // (half KSUB of buffer KBUF).  The values go first: their p make room for the new ones.
        constexpr int NV = 2 * DT, NM = NV + KS;                 // fragments, of values and in all
        constexpr int AHEAD = 3;
        const auto step = [&](int j, v16f& s, v16f& next, const uint4 (&p)[4], uint4 (&p_new)[4], auto kbuf_,
                              auto ksub_, auto vbuf_, auto vsub_) __attribute__((always_inline)) {
            constexpr int KBUF = decltype(kbuf_)::value, KSUB = decltype(ksub_)::value;
            constexpr int VBUF = decltype(vbuf_)::value, VSUB = decltype(vsub_)::value;
            uint4 ring[AHEAD + 1];
            const auto read = [&](auto y_) __attribute__((always_inline)) {
                constexpr int Y = decltype(y_)::value, K = Y - NV;
                if constexpr (Y < NV)
                    ring[Y % (AHEAD + 1)] = *(const uint4*)(lds_v + vat[2 * VSUB + Y / DT] + VBUF * V_BUF +
                                                           Y % DT * 32 * V_ROW);
                else if constexpr (Y < NM)
                    ring[Y % (AHEAD + 1)] = *(const uint4*)(lds_k + kat[K % KA] + K / KA * KA * 32 + KBUF * K_BUF +
                                                           KSUB * 32 * K_ROW);
            };
            read(StageId<0>{});
            read(StageId<1>{});
            read(StageId<2>{});
            const int base = t_first * kBlockTile + 32 * j;
            if (base > seen_by_all - 32) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (base + 16 * (i >> 3) + 8 * hh + (i & 7) >= limit) s[i] = neg_inf();
            }
            float top, alpha, add, sum[2] = {0.f, 0.f}, y_last, cc = c;
            bool grew;
            uint32_t w[8], rest[8];
            __builtin_amdgcn_sched_barrier(0);
            const auto slot = [&](auto y_) __attribute__((always_inline)) {
                constexpr int Y = decltype(y_)::value;
                // elements of the softmax that are done before slot y: they start in slot FIRST and
                // spread over the matrix instructions from there on, two a slot of values
                constexpr int FIRST = DT == 2 ? 2 : 3;
                constexpr auto at = [](int y) { return y < NV ? 2 * y : NV + y; };
                constexpr auto done = [at](int y) {
                    return y <= FIRST ? 0 : 16 * (at(y) - at(FIRST)) / (at(NM) - at(FIRST));
                };
                read(StageId<Y + AHEAD>{});
                const uint4 f = ring[Y % (AHEAD + 1)];
                if constexpr (Y < NV) {
                    constexpr int U = Y / DT, D = Y % DT;
                    o[D] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                        __builtin_bit_cast(bf8v, f), __builtin_bit_cast(bf8v, p[U]), o[D], 0, 0, 0);
                    o[D] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                        __builtin_bit_cast(bf8v, f), __builtin_bit_cast(bf8v, p[2 + U]), o[D], 0, 0, 0);
                } else {
                    if constexpr (Y == NV) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) next[i] = 0.f;
                    }
                    next = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf8v, f), q[Y - NV], next, 0,
                                                                   0, 0);
                }
                if constexpr (Y > 0 && Y < FIRST) {              // the maximum
                    constexpr int N = FIRST - 1, X = Y - 1;
                    if constexpr (X == 0) top = s[0];
#pragma unroll
                    for (int i = 16 * X / N; i < 16 * (X + 1) / N; ++i) top = fmaxf(top, s[i]);
                }
                if constexpr (Y == FIRST - 1) {
                    // the reference follows the maximum only where it would be passed by over 2^kSlack
                    const float x = __builtin_ceilf(half_max(top) * c);
                    const float m_new = x > m + kSlack ? x : m;
                    alpha = m == neg_inf() ? 0.f : __builtin_amdgcn_exp2f(m - m_new);
                    add = m_new == neg_inf() ? 0.f : -m_new;
                    grew = m_new != m;
                    if (__any(__builtin_fabsf(m_new) > 4194304.f && m_new != neg_inf())) {
                        asm volatile("" ::: "memory");           // a branch: see AttnWave::softmax
                        s *= c;
                        cc = 1.f;
                    }
                    m = m_new;
                }
#pragma unroll
                for (int i = done(Y); i < done(Y + 1); ++i) {
                    const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], cc, add));
                    sum[i & 1] += y;
                    if (i & 1) {
                        uint32_t hi = __builtin_bit_cast(uint32_t, bf2v{(__bf16)y_last, (__bf16)y});
                        asm("" : "+v"(hi));                      // not rounded again for the remainder
                        w[i >> 1] = hi;
                        rest[i >> 1] = __builtin_bit_cast(uint32_t, bf2v{(__bf16)(y_last - bf16_lo(hi)),
                                                                         (__bf16)(y - bf16_hi(hi))});
                        // computed here
                        asm volatile("" : "+v"(w[i >> 1]), "+v"(rest[i >> 1]), "+v"(sum[0]), "+v"(sum[1]));
                    }
                    y_last = y;
                }
                __builtin_amdgcn_sched_barrier(0);
            };
            __builtin_amdgcn_s_setprio(1);                       // before a wave that is between its steps
            slot(StageId<0>{}); slot(StageId<1>{}); slot(StageId<2>{}); slot(StageId<3>{});
            slot(StageId<4>{}); slot(StageId<5>{}); slot(StageId<6>{}); slot(StageId<7>{});
            if constexpr (NM > 8) {
                slot(StageId<8>{}); slot(StageId<9>{}); slot(StageId<10>{}); slot(StageId<11>{});
                slot(StageId<12>{}); slot(StageId<13>{}); slot(StageId<14>{}); slot(StageId<15>{});
            }
            if constexpr (NM > 16) {
                slot(StageId<16>{}); slot(StageId<17>{}); slot(StageId<18>{}); slot(StageId<19>{});
            }
            __builtin_amdgcn_s_setprio(0);
            l = __builtin_fmaf(l, alpha, sum[0] + sum[1]);
            p_new[0] = make_uint4(w[0], w[1], w[2], w[3]);
            p_new[1] = make_uint4(w[4], w[5], w[6], w[7]);
            p_new[2] = make_uint4(rest[0], rest[1], rest[2], rest[3]);
            p_new[3] = make_uint4(rest[4], rest[5], rest[6], rest[7]);
            if (__any(grew)) {                                   // O holds the values up to j - 1
#pragma unroll
                for (int d = 0; d < DT; ++d) o[d] *= alpha;
            }
        };
        static_assert(NM == 8 || NM == 16 || NM == 20, "slots written out");

        Pages p0, p1, p2, p3;                                    // of tile 0 and tiles i + 1 .. i + 3
        uint4 kr1[KCH];
        pages_at(p0, 0);
        pages_at(p1, 2);
        pages_at(p2, 4);
        load_k(kr, t_first, p0);
        load_v(t_first, p0);
        load_k(kr1, t_first + 1, p1);
        scales_at(p0, 0);
        scales_at(p1, 2);
        scales_at(p2, 4);
        store_k(kr, 0, p0);
        store_v(t_first, 0, p0);
        store_k(kr1, 1, p1);
        // the values "before the first" meet p = 0: zeros, since LDS may hold anything
        for (int x = tid; x < V_BUF / 16; x += NT) ((uint4*)(lds_v + V_BUF))[x] = make_uint4(0, 0, 0, 0);
        load_k(kr, t_first + 2, p2);
        load_v(t_first + 1, p1);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 16; ++i) s_even[i] = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
            s_even = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                *(const bf8v*)(lds_k + kat[ks % KA] + ks / KA * KA * 32), q[ks], s_even, 0, 0, 0);
        // tile i: buffers i & 1.  Between its two steps every wave is done with the keys of tile i
        // and the values of tile i - 1, and their buffers take those of i + 2 and i + 1.  Half of
        // the waves stage before their step, half behind it: the two that share a SIMD then do
        // not both leave its matrix unit idle at a time.
        const bool early = WAVES < 8 || wave < WAVES / 2;
        const auto stage = [&](int i, auto par) __attribute__((always_inline)) {
            constexpr int P = decltype(par)::value;
            store_k(kr, P, p2);
            store_v(t_first + i + 1, 1 - P, p1);
            p3 = pages_of(i + 3);
            load_k(kr, t_first + i + 3, p3);
            load_v(t_first + i + 2, p2);
        };
        const auto tile_pair = [&](int i, auto par) __attribute__((always_inline)) {
            constexpr int P = decltype(par)::value;
            step(2 * i, s_even, s_odd, p_odd, p_even, StageId<P>{}, StageId<1>{}, StageId<1 - P>{},
                 StageId<1>{});
            __syncthreads();
            if (early) stage(i, par);
            step(2 * i + 1, s_odd, s_even, p_even, p_odd, StageId<1 - P>{}, StageId<0>{}, StageId<P>{},
                 StageId<0>{});
            if (!early) stage(i, par);
            p1 = p2;
            p2 = p3;
        };
        for (int i = 0; i < n; i += 2) {
            tile_pair(i, StageId<0>{});
            if (i + 1 < n) tile_pair(i + 1, StageId<1>{});
        }
        const uint8_t* const at = lds_v + (n - 1 & 1) * V_BUF;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                const bf8v f = *(const bf8v*)(at + vat[2 + u] + d * 32 * V_ROW);
#pragma unroll
                for (int x = u; x < 4; x += 2)
                    o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, __builtin_bit_cast(bf8v, p_odd[x]), o[d], 0,
                                                                   0, 0);
            }
    }

    // results: lane half hh holds dims 32 d + 8 (i / 4) + 4 hh + i % 4 of its columns
    const float ll = half_sum(l);
    if (!used) return;
    if (parts == 1) {
        const float rl = out_factor(ll);
        const int64_t at = (it.q0 + col / G) * a.heads_q + h * G + col % G;
        uint16_t* const out = a.out + at * DV + 4 * hh;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int y = 0; y < 4; ++y)
                *(uint2*)(out + 32 * d + 8 * y) =
                    make_uint2(pack_bf16x2(o[d][4 * y] * rl, o[d][4 * y + 1] * rl),
                               pack_bf16x2(o[d][4 * y + 2] * rl, o[d][4 * y + 3] * rl));
        if (a.lse && hh == 0)
            a.lse[at] = ll == 0.f ? neg_inf() : (m + __builtin_log2f(ll)) * kLn2;
    } else {
        const int64_t slot = (int64_t)blockIdx.x * CB + wave * 32 + lr;
        float* const ws = a.ws + slot * DV + 4 * hh;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int y = 0; y < 4; ++y)
                *(v4f*)(ws + 32 * d + 8 * y) = v4f{o[d][4 * y], o[d][4 * y + 1], o[d][4 * y + 2],
                                                   o[d][4 * y + 3]};
        if (hh == 0) {
            float* const ml = a.ws + (int64_t)gridDim.x * CB * DV + slot * 2;
            ml[0] = m;
            ml[1] = ll;
        }
    }
}

// Adds the parts of a split block, in token order: DV / 4 lanes a row, a workgroup 32 rows.
constexpr int kJoinRows = 32;
template <int DV, int CB>
__global__ __launch_bounds__(kAttnThreads) void attn_block_join_kernel(AttnArgs a, int blocks, int splits) {
    constexpr int L = DV / 4, ROWS = kAttnThreads / L;
    const int tid = threadIdx.x, d4 = tid % L * 4;
    const int piece = blockIdx.x % (CB / kJoinRows), block = blockIdx.x / (CB / kJoinRows);
    const int h = block % a.heads_kv;
    Block k;
    if (!k.find(a, blocks - 1 - block / a.heads_kv, CB)) return;
    const int parts = k.parts(splits);
    if (parts == 1) return;                                     // finished by its workgroup
    const int64_t first = (int64_t)block * splits * CB;
    const float* const ml = a.ws + (int64_t)blocks * a.heads_kv * splits * CB * DV;
#pragma unroll
    for (int y = 0; y < kJoinRows / ROWS; ++y) {
        const int x = piece * kJoinRows + y * ROWS + tid / L, col = k.c0 + x;
        if (col >= k.it.cols) continue;
        Part part;
#pragma unroll 4
        for (int z = 0; z < parts; ++z) {
            const int64_t slot = first + z * CB + x;
            const float2 mw = *(const float2*)(ml + slot * 2);
            part.add(*(const v4f*)(a.ws + slot * DV + d4), mw.x, mw.y);
        }
        part.store(a, (k.it.q0 + col / k.it.G) * a.heads_q + h * k.it.G + col % k.it.G, DV, d4);
    }
}

constexpr int kSplitTile = 64;                // tokens of a wave's tile
static bool splits(int64_t max_new, int32_t heads_q, int32_t heads_kv) {
    return max_new * (heads_q / heads_kv) <= kSplitMaxCols;
}

// How a launch of many columns divides: eight waves a workgroup, or four where that leaves CUs
// idle, and the tokens of a block over several workgroups where even those are few.  Behind 8k
// tokens, 32 heads of 128: a chunk of 1024 tokens takes 244 us by four waves and 309 by eight, one
// of 2048 442 and 429.
struct BlockPlan {
    int waves;
    int64_t blocks, splits;                          // per KV head; parts of each
};
static BlockPlan block_plan(int64_t T, int64_t R, int heads_q, int heads_kv) {
    const int64_t G = heads_q / heads_kv;
    BlockPlan p{8, T * G / 256 + R, 1};
    if (p.blocks * heads_kv < 256) {
        p.waves = 4;
        p.blocks = T * G / 128 + R;
        const int64_t n = p.blocks * heads_kv;
        p.splits = n * 2 <= kBlockSlots ? kBlockSlots / n : 1;
        if (p.splits > kBlockMaxSplits) p.splits = kBlockMaxSplits;
    }
    return p;
}

size_t attn_paged_workspace_bytes(int64_t R, int64_t max_new, int32_t heads_q, int32_t heads_kv,
                                  int32_t dk, int32_t dv) {
    if (splits(max_new, heads_q, heads_kv))
        return (size_t)split_groups(dv) * 2 * kCols * (dv + 2) * sizeof(float);
    // more tokens make more blocks: what one token in all does not split, nothing does
    if (block_plan(1, R, heads_q, heads_kv).splits == 1) return 0;
    // any number of tokens up to R * max_new: at most kBlockSlots parts of 128 columns
    const BlockPlan p = block_plan(R * max_new, R, heads_q, heads_kv);
    const int64_t most = p.waves == 4 ? p.blocks * heads_kv * kBlockMaxSplits : kBlockSlots;
    return (size_t)(most < kBlockSlots ? most : kBlockSlots) * 128 * (dv + 2) * sizeof(float);
}

template <int DK, int DV, int B>
static hipError_t split_launch(const AttnArgs& a, hipStream_t stream) {
    const int max_cols = (int)(a.max_new * (a.heads_q / a.heads_kv));
    const int64_t col_tiles = (max_cols + kCols - 1) / kCols;
    const int64_t items = (int64_t)a.R * a.heads_kv * col_tiles;
    if (!a.ws) {
        attn_item_kernel<DK, DV, B, kSplitTile>
            <<<dim3((unsigned)items), dim3(kAttnThreads), 0, stream>>>(a, (int)col_tiles);
        return hipGetLastError();
    }
    constexpr int groups = split_groups(DV);
    attn_split_kernel<DK, DV, B, kSplitTile><<<dim3(groups), dim3(kAttnThreads), 0, stream>>>(a, (int)col_tiles);
    const int64_t rows = (int64_t)a.R * a.heads_kv * max_cols;
    // where items are many, an item has few parts (about groups / items + 1) and two strands (128
    // wide: one wave) take a row; where they are few, a workgroup of eight strands does.  64 requests
    // x 8 heads: 74.5 us by the former, 79 by the latter; 3 requests, 195k tokens, 2 heads: 36 and 29.
    constexpr int FEW = 256 / DV;                               // a wave's strands
    if (items * 4 >= groups) {
        attn_join_kernel<DV, FEW><<<dim3((unsigned)((rows + 3) / 4)), dim3(kAttnThreads), 0, stream>>>(
            a, (int)col_tiles, max_cols);
    } else {
        attn_join_kernel<DV, 4 * FEW><<<dim3((unsigned)rows), dim3(kAttnThreads), 0, stream>>>(
            a, (int)col_tiles, max_cols);
    }
    return hipGetLastError();
}

template <int DK, int DV, int WAVES>
static hipError_t block_launch(const AttnArgs& a, const BlockPlan& p, hipStream_t stream) {
    // as many parts as the workspace holds: it is sized for R * max_new tokens, T may be padded
    const int64_t hold = a.ws ? (int64_t)(a.ws_bytes / (32 * WAVES * (DV + 2) * sizeof(float))) : 0;
    const int64_t splits = std::max<int64_t>(1, std::min(p.splits, hold / (p.blocks * a.heads_kv)));
    const unsigned grid = (unsigned)(p.blocks * a.heads_kv * splits);
    attn_block_kernel<DK, DV, WAVES><<<dim3(grid), dim3(64 * WAVES), 0, stream>>>(a, (int)p.blocks, (int)splits);
    if (splits > 1) {
        constexpr int CB = 32 * WAVES;
        attn_block_join_kernel<DV, CB>
            <<<dim3((unsigned)(p.blocks * a.heads_kv * (CB / kJoinRows))), dim3(kAttnThreads), 0, stream>>>(
                a, (int)p.blocks, (int)splits);
    }
    return hipGetLastError();
}

template <int DK, int DV>
static hipError_t attn_launch(const AttnArgs& a, hipStream_t stream) {
    if (splits(a.max_new, a.heads_q, a.heads_kv))
        return a.log_b == 5   ? split_launch<DK, DV, 32>(a, stream)
               : a.log_b == 6 ? split_launch<DK, DV, 64>(a, stream)
                              : split_launch<DK, DV, 128>(a, stream);
    const BlockPlan p = block_plan(a.T, a.R, a.heads_q, a.heads_kv);
    return p.waves == 4 ? block_launch<DK, DV, 4>(a, p, stream) : block_launch<DK, DV, 8>(a, p, stream);
}

hipError_t launch_attn_paged(const AttnArgs& a, int32_t dk, int32_t dv, hipStream_t stream) {
    if (dk == 64 && dv == 64) return attn_launch<64, 64>(a, stream);
    if (dk == 128 && dv == 128) return attn_launch<128, 128>(a, stream);
    if (dk == 192 && dv == 128) return attn_launch<192, 128>(a, stream);
    return hipErrorInvalidValue;
}

}  // namespace bfp8
