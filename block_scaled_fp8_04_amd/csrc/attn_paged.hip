// attn_paged.hip - attention over the paged e4m3 cache on gfx950.
//
//     out = sum_t p_t v_t / sum_t p_t,   p_t = exp(scale q . k_t - max)
//
// Both products are taken transposed, keys and values as the first operand:
//     S^T [token, query] = K Q^T,     O^T [d, query] += V^T P^T
// Lane group g = lane / 16 takes tokens 32 g .. 32 g + 31 of a 128-token tile in both: the
// rows of K enter the first product in the order that leaves those tokens' results in that
// group's lanes, where they are the second product's P^T operand as they stand.  P never
// moves between lanes, and with values stored token-contiguous neither product's operands
// need a transposition.
//
// Precision.  Codes are widened to bf16 with their page's scale on the way to the matrix
// cores (exact: four significant bits and a power of two) and q is bf16 as it comes.  p
// enters as two bf16 terms, p rounded and the remainder, sixteen bits at any size of p: one
// term alone would be off by 2^-8, as much as the rounding of the output.  The fp8 product
// would take the codes as they are, but it drops what lies 2^-14 below the largest product of
// a 16-element group (measured), which moves a logit by 1e-5 of that product, and p as two
// e4m3 terms loses what lies 2^-22 below a tile's largest.  Logits, maxima,
// norms and sums are fp32.  Running maxima are rounded up to integers (in units of log 2),
// so that rescaling by 2^(old - new) is exact.
#include <algorithm>

#include "device_codec.hpp"
#include "internal.hpp"
#include "tile_common.hpp"

namespace bfp8 {

constexpr int kAttnThreads = 256;
constexpr int kAttnWaves = kAttnThreads / 64;
constexpr int kCols = 16;                     // query columns of a wave
constexpr int kSplitMaxCols = 64;             // most query columns of a split item
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float neg_inf() { return __uint_as_float(0xFF800000u); }

typedef __bf16 bf8v __attribute__((ext_vector_type(8)));
typedef __bf16 bf2v __attribute__((ext_vector_type(2)));

// Eight e4m3 codes (two registers) times a power of two, as bf16 (exact).
__device__ __forceinline__ bf8v widen8(int w0, int w1, float scale) {
    const bf2v a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, scale, false);
    const bf2v b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, scale, true);
    const bf2v c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, scale, false);
    const bf2v d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, scale, true);
    return bf8v{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Eight fp32 as bf16 and the remainders as bf16.
__device__ __forceinline__ void split8(const float (&p)[8], bf8v& hi, bf8v& lo) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        hi[j] = (__bf16)p[j];
        lo[j] = (__bf16)(p[j] - (float)hi[j]);
    }
}

// Eight elements of a bf16 query row (negated for a negative scale).
__device__ __forceinline__ bf8v load_q8(const uint16_t* p, bool vec, bool negate) {
    uint4 x;
    if (vec) {
        x = *(const uint4*)p;
    } else {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = (uint32_t)p[2 * j] | ((uint32_t)p[2 * j + 1] << 16);
        x = make_uint4(w[0], w[1], w[2], w[3]);
    }
    const uint32_t f = negate ? 0x80008000u : 0u;
    return __builtin_bit_cast(bf8v, make_uint4(x.x ^ f, x.y ^ f, x.z ^ f, x.w ^ f));
}

// Reads through the scalar cache (uniform addresses): page numbers and scales.
typedef const __attribute__((address_space(4))) int32_t* scalar_i32;
typedef const __attribute__((address_space(4))) float* scalar_f32;

// A value that is the same in all lanes, in scalar registers (where the compiler cannot see it).
__device__ __forceinline__ int64_t uniform(int64_t x) {
    return (int64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)x) |
           (int64_t)__builtin_amdgcn_readfirstlane((int)(x >> 32)) << 32;
}

// What an item's columns are: shared by the three kernels.  kUniform: r is the same for the wave,
// and so is then all of this, in scalar registers.
struct Item {
    int64_t q0;
    int n, cols, kv_len, G;
    template <bool kUniform>
    static __device__ __forceinline__ int32_t at(const int32_t* p, int i) {
        return kUniform ? ((scalar_i32)(uintptr_t)p)[i] : p[i];
    }
    template <bool kUniform>
    static __device__ __forceinline__ Item of(const AttnArgs& a, int r) {
        Item it;
        it.G = a.heads_q / a.heads_kv;
        it.q0 = min(max((int64_t)at<kUniform>(a.q_offsets, r), (int64_t)0), a.T);
        const int64_t q1 = min(max((int64_t)at<kUniform>(a.q_offsets, r + 1), it.q0), a.T);
        it.n = (int)(q1 - it.q0);
        it.cols = (int)min((int64_t)it.n, a.max_new) * it.G;
        it.kv_len = (int)min(max((int64_t)at<kUniform>(a.kv_lens, r), (int64_t)0), a.width << a.log_b);
        return it;
    }
    // tokens that column c sees
    __device__ __forceinline__ int limit(int c) const {
        return min(kv_len, max(kv_len - n + c / G + 1, 0));
    }
    __device__ __forceinline__ const uint16_t* row(const AttnArgs& a, int h, int c) const {
        return a.q + (q0 + c / G) * a.q_ts + (int64_t)(h * G + c % G) * a.q_hs;
    }
};

__device__ __forceinline__ bool q_vec(const AttnArgs& a) {
    return ((uintptr_t)a.q % 16) == 0 && ((a.q_ts | a.q_hs) % 8) == 0;
}
__device__ __forceinline__ float exp2_scale(const AttnArgs& a) {
    return fmaxf(__builtin_fabsf(a.scale) * kLog2e, 0x1p-126f);     // -inf times 0 is NaN
}

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
// 16 bytes are an access of their own: 3.8 instead of 5.2 TB/s (64 requests, 180k tokens, 8
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
            const float ke = pick(ks, LT * (lr >> 2)), ve = pick(vs, LT * g);
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
            if (base + TT > free_limit) {
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

// Joins the four waves' results of one 16-column item in their bytes of lds_v (the keys' bytes
// may be receiving the next item's): first m and l, then each wave's O times 2^(m_w - m), its
// four-dim groups permuted by the column against bank conflicts.  Thread x gets column x / 16,
// dims 4 (x % 16) + 64 j of the sum, in wave order, and that column's m and l.
// Barrier behind finished LDS accesses, leaving the loads that are on their way alone.
__device__ __forceinline__ void barrier_ds() {
    __builtin_amdgcn_s_waitcnt(0xC07F);                         // lgkmcnt(0)
    barrier_lds();
}

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
    const float r = l == 0.f ? 0.f : 1.0f / l;
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
constexpr int kSplitMinUnits = kAttnWaves;    // tiles per workgroup, at least one for each wave

struct SplitPlan {
    int64_t units;      // tiles of all items
    int64_t per;        // tiles per workgroup
};

__device__ __forceinline__ SplitPlan split_plan(const AttnArgs& a, int col_tiles, int groups) {
    const int64_t units = (int64_t)max(a.tile_offsets[a.R], 0) * a.heads_kv * col_tiles;
    return {units, max((units + groups - 1) / groups, (int64_t)kSplitMinUnits)};
}

// One workgroup per (request, KV head, 16 query columns): its waves take every fourth tile.
template <int DK, int DV, int B, int TT>
__global__ __launch_bounds__(kAttnThreads) void attn_item_kernel(AttnArgs a, int col_tiles) {
    using W = AttnWave<DK, DV, B, TT>;
    __shared__ __attribute__((aligned(1024))) uint8_t lds_k[kAttnWaves * W::K_BYTES];
    __shared__ __attribute__((aligned(1024))) uint8_t lds_v[kAttnWaves * W::V_BYTES];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int64_t item = blockIdx.x;
    const int ct = (int)(item % col_tiles);
    item /= col_tiles;
    const int h = (int)(item % a.heads_kv);
    const Item it = Item::of<true>(a, (int)(item / a.heads_kv));
    if (ct * kCols >= it.cols) return;
    const int col = ct * kCols + (lane & 15);
    const bool used = col < it.cols;
    W w;
    w.load_q(used ? it.row(a, h, col) : nullptr, q_vec(a), a.scale < 0.f, lane >> 4);
    Segment seg;
    seg.r = (int)(item / a.heads_kv);
    seg.h = h;
    seg.ct = ct;
    seg.t0 = 0;
    seg.t1 = (it.limit(min(ct * kCols + kCols, it.cols) - 1) + TT - 1) / TT;
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
    const SplitPlan sp = split_plan(a, col_tiles, gridDim.x);
    int64_t u = (int64_t)blockIdx.x * uniform(sp.per);
    const int64_t end = min(u + uniform(sp.per), uniform(sp.units));
    if (u >= end) return;
    const int64_t items = (int64_t)a.heads_kv * col_tiles;   // of one request
    // the request of the first unit: how many offsets lie at or below it, counted by 64 lanes on
    // every 64th offset and then on the 64 behind the last of those
    static_assert(kKvMaxRequests <= 64 * 64, "two steps");
    const int64_t ut = uniform(u / items);
    const int lo64 = __popcll(__ballot(lane * 64 < a.R && a.tile_offsets[min(lane * 64, a.R)] <= ut)) - 1;
    const int at = max(lo64, 0) * 64 + lane;
    const int lo = max(lo64, 0) * 64 +
                   max(__popcll(__ballot(at < a.R && a.tile_offsets[min(at, a.R)] <= ut)) - 1, 0);
    const scalar_i32 offs = (scalar_i32)(uintptr_t)a.tile_offsets;
    int r = __builtin_amdgcn_readfirstlane(lo);
    // the workgroup's next run of tiles, from unit u on
    const auto advance = [&](Segment& s) {
        for (; r < a.R && u < end; ++r) {
            const int64_t f = offs[r];
            const int nt = (int)min(max((int64_t)offs[r + 1] - f, (int64_t)0), (int64_t)1 << 24);
            const int64_t local = max(u - f * items, (int64_t)0);
            if (nt <= 0 || local >= (int64_t)nt * items) continue;
            const int item = __builtin_amdgcn_readfirstlane((int)(local / nt));
            const int tile0 = (int)(local - (int64_t)item * nt);
            const int count = (int)min((int64_t)(nt - tile0), end - u);
            u += count;
            s.r = r;
            s.h = __builtin_amdgcn_readfirstlane(item / col_tiles);
            s.ct = item - s.h * col_tiles;
            s.t0 = tile0 * (kKvTile / TT);
            s.t1 = (tile0 + count) * (kKvTile / TT);
            s.whole = count == nt;
            return true;
        }
        return false;
    };
    bool first = true, ready = false;
    int64_t page[W::NP] = {};                                  // of the keys that are on their way
    float ks[W::NP] = {}, vs[W::NP] = {};
    Segment cur, next;
    bool valid = advance(cur);
    Item it = Item::of<true>(a, valid ? cur.r : 0);
    while (valid) {
        next = cur;                                             // defined, and inside the pool, if there is none
        const bool has = advance(next);
        const Item nit = Item::of<true>(a, has ? next.r : 0);
        W w;
        const int col = cur.ct * kCols + (lane & 15);
        const bool used = col < it.cols;
        if (cur.ct * kCols < it.cols) {
            cur.t1 = min(cur.t1, (it.kv_len + TT - 1) / TT);
            const int n1 = next.ct * kCols < nit.cols ? min(next.t1, (nit.kv_len + TT - 1) / TT) : 0;
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
                        float* const ml = a.ws + (int64_t)gridDim.x * 2 * kCols * DV + slot * 2;
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

// Adds the partial sums of the workgroups that shared an item, one row (item column) by STRANDS
// strands of DV / 4 lanes each: every strand takes its workgroups in token order, then the strands
// are added in order.  Rows of a request without tokens get their zeros here.
//
// Where items are many, an item has few parts and two strands (128 wide: one wave) take a row;
// where they are few, a workgroup of eight strands does.
template <int DV, int STRANDS>
__global__ __launch_bounds__(kAttnThreads) void attn_join_kernel(AttnArgs a, int col_tiles,
                                                                 int groups, int max_cols) {
    constexpr int L = DV / 4, ROWS = kAttnThreads / (L * STRANDS);
    __shared__ float red[kAttnThreads / L][DV + 4];
    __shared__ float red_l[kAttnThreads / L];
    const int tid = threadIdx.x, strand = tid / L % STRANDS, d4 = tid % L * 4;
    int64_t x = (int64_t)blockIdx.x * ROWS + tid / (L * STRANDS);
    const int col = (int)(x % max_cols);
    x /= max_cols;
    const int h = (int)(x % a.heads_kv);
    const int r = (int)min(x / a.heads_kv, (int64_t)a.R - 1);
    const Item it = Item::of<false>(a, r);
    const bool live = x / a.heads_kv < a.R && col < it.cols;
    const int ct = col / kCols;
    const int64_t items = (int64_t)a.heads_kv * col_tiles;
    const int64_t t0 = max(a.tile_offsets[r], 0), nt = (int64_t)a.tile_offsets[r + 1] - t0;
    const int64_t row = it.q0 + col / it.G;
    const int head = h * it.G + col % it.G;
    const SplitPlan sp = split_plan(a, col_tiles, groups);
    const int64_t begin = t0 * items + ((int64_t)h * col_tiles + ct) * nt;
    const int wa = (int)min(begin / sp.per, (int64_t)groups);
    const int wb = (int)min((begin + nt - 1) / sp.per, (int64_t)groups - 1);
    const bool joins = live && nt > 0 && wa < wb;               // else finished by one workgroup
    const auto slot_of = [&](int w) {
        return ((int64_t)w * 2 + (w * sp.per >= begin ? 0 : 1)) * kCols + col % kCols;
    };
    const float* const ml = a.ws + (int64_t)groups * 2 * kCols * DV;
    float m = neg_inf(), l = 0.f;
    v4f acc = {0.f, 0.f, 0.f, 0.f};
    if (joins) {
        // the row's lanes (64, or all 256 of the workgroup's waves alike) look at every part's m
        for (int w = wa + (tid & 63); w <= wb; w += 64) m = fmaxf(m, ml[slot_of(w) * 2]);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
    if (joins) {
#pragma unroll 4
        for (int w = wa + strand; w <= wb; w += STRANDS) {
            const int64_t slot = slot_of(w);
            const float mw = ml[slot * 2], lw = ml[slot * 2 + 1];
            const v4f v = *(const v4f*)(a.ws + slot * DV + d4);
            const bool saw = mw != neg_inf() || lw != 0.f;      // otherwise its sums are zeros
            const float f = saw ? __builtin_amdgcn_exp2f(mw - m) : 0.f;
            l = __builtin_fmaf(lw, f, l);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(v[i], f, acc[i]);
        }
    }
    const int mine = tid / L;
    *(v4f*)&red[mine][d4] = acc;
    if (tid % L == 0) red_l[mine] = l;
    __syncthreads();
    if (strand != 0 || !live) return;
    uint16_t* const out = a.out + (row * a.heads_q + head) * DV + d4;
    if (nt <= 0) {
        *(uint2*)out = make_uint2(0, 0);
        if (a.lse && d4 == 0) a.lse[row * a.heads_q + head] = neg_inf();
    } else if (joins) {
#pragma unroll
        for (int i = 1; i < STRANDS; ++i) {
            l += red_l[mine + i];
            acc += *(const v4f*)&red[mine + i][d4];
        }
        const float rl = l == 0.f ? 0.f : 1.0f / l;
        *(uint2*)out =
            make_uint2(pack_bf16x2(acc[0] * rl, acc[1] * rl), pack_bf16x2(acc[2] * rl, acc[3] * rl));
        if (a.lse && d4 == 0)
            a.lse[row * a.heads_q + head] = l == 0.f ? neg_inf() : (m + __builtin_log2f(l)) * kLn2;
    }
}

// ---------------------------------------------------------------- many query columns
//
// Prompts and chunks: a workgroup takes 32 columns a wave of one request and KV head and walks
// the tokens they see.  The products and the softmax beside them bound this, so the codes are
// widened once per workgroup on their way into LDS, keys to bf16 with their scale, values to f16
// without it, and every wave reads its fragments from there.
//
// p enters its product as one f16 term (eleven bits).  Its range is kept by the value page's
// scale 2^e: with m' within kSlack of the running maximum of x + e over the tokens (x the logit
// in units of log 2), p' = 2^(x + e - m' + 15 - kSlack) lies in (0, 2^15], is exact to 2^-11
// down to 2^-21 of the largest weighted token and to 2^-32 of it below that.  O sums p' times
// the codes, l sums p' 2^-e: their quotient is the result.  The slack is there because a
// maximum over 32 columns that is followed at once moves in every second step (2048 tokens
// over 32k), and O has to be rescaled each time.
//
// A step forms the logits of 32 tokens, does the softmax of the 32 before and adds the values of
// the 32 before those: three independent streams, written out so that each matrix instruction
// is followed by the vector work that fits beside it (a softmax element takes 26 of its 32
// cycles) and by the LDS read of a fragment three instructions on.  S^T's rows are the tokens
// with bits 2 and 3 exchanged, which makes its registers the second product's operand as they
// stand.
typedef float v16f __attribute__((ext_vector_type(16)));
typedef _Float16 h8v __attribute__((ext_vector_type(8)));
typedef _Float16 h2v __attribute__((ext_vector_type(2)));

constexpr int kBlockTile = 64;                // tokens in LDS at a time
constexpr int kBlockSlots = 512;              // workgroups that a split launch aims at
constexpr int kBlockMaxSplits = 16;
constexpr float kSlack = 8.f;

__device__ __forceinline__ h8v widen8h(uint32_t w0, uint32_t w1) {
    const h2v a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w0, 1.f, false);
    const h2v b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w0, 1.f, true);
    const h2v c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w1, 1.f, false);
    const h2v d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w1, 1.f, true);
    return h8v{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// x of the two halves of the wave: their maximum, their sum
__device__ __forceinline__ float half_max(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float half_sum(float x) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

template <int DK, int DV, int WAVES, int NC>
__global__ __launch_bounds__(WAVES * 64, 2 / NC) void attn_block_kernel(AttnArgs a, int blocks, int splits) {
    constexpr int CB = 32 * NC * WAVES, NT = 64 * WAVES;        // columns and threads of a workgroup
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

    // block b of the launch: request r's blocks start at q_offsets[r] * G / CB + r, where there
    // is room for all of them; the last ones, which see the most tokens, go first
    int idx = blockIdx.x;
    const int z = idx % splits;
    idx /= splits;
    const int h = idx % a.heads_kv, b = blocks - 1 - idx / a.heads_kv;
    const auto start_of = [&](int r) {
        return (int64_t)min(max((int64_t)a.q_offsets[r], (int64_t)0), a.T) * G / CB + r;
    };
    int r = 0;
    {
        const int hi = __popcll(__ballot(lane * 64 < a.R && start_of(min(lane * 64, a.R)) <= b)) - 1;
        const int at = max(hi, 0) * 64 + lane;
        r = max(hi, 0) * 64 +
            max(__popcll(__ballot(at < a.R && start_of(min(at, a.R)) <= b)) - 1, 0);
        r = __builtin_amdgcn_readfirstlane(r);
    }
    const Item it = Item::of<true>(a, r);
    const int c0 = __builtin_amdgcn_readfirstlane((int)min(b - start_of(r), (int64_t)1 << 22)) * CB;
    if (c0 < 0 || c0 >= it.cols) return;
    const int c1 = min(c0 + CB, it.cols) - 1;                   // last column
    const int seen_by_all = it.limit(c0), seen = it.limit(c1);
    const int tiles = (seen + kBlockTile - 1) / kBlockTile;
    const int t_first = (int)((int64_t)tiles * z / splits), t_end = (int)((int64_t)tiles * (z + 1) / splits);
    const int n = t_end - t_first;
    const int kv_len = it.kv_len, last = max(kv_len - 1, 0) >> a.log_b, B = 1 << a.log_b;
    const float c = exp2_scale(a);

    // this lane's columns: 32 t + lr of the wave's
    int limit[NC];
    bf8v q[NC][KS];
    v16f o[NC][DT];
    float m[NC], l[NC];
#pragma unroll
    for (int t = 0; t < NC; ++t) {
        const int col = c0 + (wave * NC + t) * 32 + lr;
        const bool used = col < it.cols;
        limit[t] = used ? it.limit(col) : 0;
        const uint16_t* const row = it.row(a, h, used ? col : c0);
        const bool vec = q_vec(a), negate = a.scale < 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) q[t][ks] = load_q8(row + 16 * ks + 8 * hh, vec, negate);
        m[t] = neg_inf();
        l[t] = 0.f;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[t][d][i] = 0.f;
    }

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
            const int j = min((tile * kBlockTile + 32 * lane) >> a.log_b, last);
            return (int)min(max((int64_t)a.block_table[(int64_t)r * a.width + j], (int64_t)0), a.pages - 1);
        };
        const auto fetch_scale = [&](const float* x, int e) { return x[(int64_t)e * a.heads_kv + h]; };
        entry = fetch_table(t_first);
        ks_l = fetch_scale(a.k_scales, entry);
        vs_l = fetch_scale(a.v_scales, entry);
        // of tile t_first + i, for i = 0, 1, 2, ... in order
        const auto pages_of = [&](int i) {
            const int at = 2 * i & 63;
            if (at == 0 && i > 0) {
                entry = entry_n;
                ks_l = ks_n;
                vs_l = vs_n;
            }
            if (at == 16) entry_n = fetch_table(t_first + i + 24);
            if (at == 40) {
                ks_n = fetch_scale(a.k_scales, entry_n);
                vs_n = fetch_scale(a.v_scales, entry_n);
            }
            const auto lane_of = [&](float x, int l) {
                return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(x), l));
            };
            Pages x;
            x.page0 = (int64_t)__builtin_amdgcn_readlane(entry, at) * a.heads_kv + h;
            x.page1 = (int64_t)__builtin_amdgcn_readlane(entry, at + 1) * a.heads_kv + h;
            x.ks0 = lane_of(ks_l, at);
            x.ks1 = lane_of(ks_l, at + 1);
            x.vs0 = lane_of(vs_l, at);
            x.vs1 = lane_of(vs_l, at + 1);
            return x;
        };
        const auto load_k = [&](int tile, const Pages& pg) {
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
        const auto store_k = [&](int buf, const Pages& pg) {
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
        const auto store_v = [&](int tile, int buf) {
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
                uint8_t* const to = lds_v + buf * V_BUF + d * V_ROW;
                *(h8v*)(to + (((x & 3) * 2) ^ f) * 16) = widen8h(w[0], w[1]);
                *(h8v*)(to + (((x & 3) * 2 + 1) ^ f) * 16) = widen8h(w[2], w[3]);
            }
        };
        // fragment places: K rows are tokens with bits 2 and 3 exchanged, V rows are lr + 32 d
        const int krow = (lr & 0x13) | (lr & 4) << 1 | (lr & 8) >> 1;
        int kat[KS], vat[4];
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) kat[ks] = krow * K_ROW + (((2 * ks) ^ (k_swz(krow) ^ hh)) * 16);
#pragma unroll
        for (int x = 0; x < 4; ++x) vat[x] = lr * V_ROW + (((2 * x) ^ ((lr >> 1 & 7) ^ hh)) * 16);

        v16f s_even[NC], s_odd[NC];                              // logits of even and odd subtiles
        uint4 p_even[NC][2], p_odd[NC][2];                       // and their p'
        float top[NC];                                           // maximum of the current ones
#pragma unroll
        for (int t = 0; t < NC; ++t) p_odd[t][0] = p_odd[t][1] = make_uint4(0, 0, 0, 0);
        // one step: softmax of subtile j, logits of j + 1 (half KSUB of buffer KBUF) and their
        // maximum, values of j - 1 (half VSUB of buffer VBUF)
        constexpr int NM = KS + 2 * DT;                          // fragments, matrix instructions a column tile
        constexpr int AHEAD = 3;
        const auto step = [&](int j, float vs, v16f (&s)[NC], v16f (&next)[NC], const uint4 (&p)[NC][2],
                              uint4 (&p_new)[NC][2], auto kbuf_, auto ksub_, auto vbuf_,
                              auto vsub_) __attribute__((always_inline)) {
            constexpr int KBUF = decltype(kbuf_)::value, KSUB = decltype(ksub_)::value;
            constexpr int VBUF = decltype(vbuf_)::value, VSUB = decltype(vsub_)::value;
            uint4 ring[AHEAD + 1];
            const auto read = [&](auto y_) __attribute__((always_inline)) {
                constexpr int Y = decltype(y_)::value;
                if constexpr (Y < KS)
                    ring[Y % (AHEAD + 1)] = *(const uint4*)(lds_k + kat[Y] + KBUF * K_BUF + KSUB * 32 * K_ROW);
                else if constexpr (Y < NM)
                    ring[Y % (AHEAD + 1)] = *(const uint4*)(lds_v + vat[2 * VSUB + (Y - KS) / DT] + VBUF * V_BUF +
                                                           (Y - KS) % DT * 32 * V_ROW);
            };
            read(StageId<0>{});
            read(StageId<1>{});
            read(StageId<2>{});
            const int base = t_first * kBlockTile + 32 * j;
            if (base + 32 > seen_by_all) {
#pragma unroll
                for (int t = 0; t < NC; ++t) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (base + 16 * (i >> 3) + 8 * hh + (i & 7) >= limit[t]) s[t][i] = neg_inf();
                    top[t] = s[t][0];
#pragma unroll
                    for (int i = 1; i < 16; ++i) top[t] = fmaxf(top[t], s[t][i]);
                }
            }
            const int e = (int)(__float_as_uint(vs) >> 23) - 127;
            float alpha[NC], add[NC], sum[NC][2], y_last[NC];
            bool grew = false, far = false;
#pragma unroll
            for (int t = 0; t < NC; ++t) {
                // the reference follows the maximum only where it would be passed by over 2^kSlack
                const float x = __builtin_ceilf(half_max(top[t]) * c) + (float)e;
                const float m_new = x > m[t] + kSlack ? x : m[t];
                alpha[t] = m[t] == neg_inf() ? 0.f : __builtin_amdgcn_exp2f(m[t] - m_new);
                add[t] = m_new == neg_inf() ? 0.f : (float)(e + 15 - (int)kSlack) - m_new;
                grew |= m_new != m[t];
                far |= __builtin_fabsf(m_new) > 4194304.f && m_new != neg_inf();
                m[t] = m_new;
                sum[t][0] = sum[t][1] = 0.f;
            }
            float cc = c;
            if (__any(far)) {                                    // see AttnWave::softmax
                asm volatile("" ::: "memory");                   // a branch: it is hardly ever taken
#pragma unroll
                for (int t = 0; t < NC; ++t) s[t] *= c;
                cc = 1.f;
            }
            uint32_t w[NC][8];
            __builtin_amdgcn_sched_barrier(0);
            const auto slot = [&](auto y_) __attribute__((always_inline)) {
                constexpr int Y = decltype(y_)::value;
                read(StageId<Y + AHEAD>{});
                const uint4 f = ring[Y % (AHEAD + 1)];
#pragma unroll
                for (int t = 0; t < NC; ++t) {
                    if constexpr (Y < KS) {
                        if constexpr (Y == 0) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) next[t][i] = 0.f;
                        }
                        next[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf8v, f), q[t][Y],
                                                                          next[t], 0, 0, 0);
                    } else {
                        constexpr int U = (Y - KS) / DT, D = (Y - KS) % DT;
                        o[t][D] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
                            __builtin_bit_cast(h8v, f), __builtin_bit_cast(h8v, p[t][U]), o[t][D], 0, 0, 0);
                    }
                    // this slot's softmax elements
#pragma unroll
                    for (int i = 16 * Y / NM; i < 16 * (Y + 1) / NM; ++i) {
                        const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][i], cc, add[t]));
                        sum[t][i & 1] += y;
                        if (i & 1) {
                            w[t][i >> 1] = __builtin_bit_cast(uint32_t, h2v{(_Float16)y_last[t], (_Float16)y});
                            asm volatile("" : "+v"(w[t][i >> 1]), "+v"(sum[t][0]), "+v"(sum[t][1]));  // computed here
                        }
                        y_last[t] = y;
                    }
                    // and of the next step's maximum, once its logits are there
                    if constexpr (Y > KS) {
                        constexpr int N = 2 * DT - 1, X = Y - KS - 1;
                        if constexpr (X == 0) top[t] = next[t][0];
#pragma unroll
                        for (int i = 16 * X / N; i < 16 * (X + 1) / N; ++i) top[t] = fmaxf(top[t], next[t][i]);
                        asm volatile("" : "+v"(top[t]));
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
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
#pragma unroll
            for (int t = 0; t < NC; ++t) {
                if (t == 0) __builtin_amdgcn_s_setprio(0);
                l[t] = __builtin_fmaf(sum[t][0] + sum[t][1], __uint_as_float((uint32_t)(127 - e) << 23), l[t] * alpha[t]);
                p_new[t][0] = make_uint4(w[t][0], w[t][1], w[t][2], w[t][3]);
                p_new[t][1] = make_uint4(w[t][4], w[t][5], w[t][6], w[t][7]);
            }
            if (__any(grew)) {                                   // O holds the values up to j - 1
#pragma unroll
                for (int t = 0; t < NC; ++t)
#pragma unroll
                    for (int d = 0; d < DT; ++d) o[t][d] *= alpha[t];
            }
        };
        static_assert(NM == 8 || NM == 16 || NM == 20, "slots written out");

        Pages p0 = pages_of(0);                                  // of tiles i .. i + 3
        load_k(t_first, p0);
        load_v(t_first, p0);
        Pages p1 = pages_of(1);
        store_k(0, p0);
        store_v(t_first, 0);
        load_k(t_first + 1, p1);
        Pages p2 = pages_of(2), p3;
        store_k(1, p1);
        // the values "before the first" meet p = 0: zeros, since LDS may hold anything
        for (int x = tid; x < V_BUF / 16; x += NT) ((uint4*)(lds_v + V_BUF))[x] = make_uint4(0, 0, 0, 0);
        __syncthreads();
        load_k(t_first + 2, p2);
        load_v(t_first + 1, p1);
#pragma unroll
        for (int t = 0; t < NC; ++t) {
#pragma unroll
            for (int i = 0; i < 16; ++i) s_even[t][i] = 0.f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
                s_even[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(*(const bf8v*)(lds_k + kat[ks]), q[t][ks],
                                                                    s_even[t], 0, 0, 0);
            top[t] = s_even[t][0];
#pragma unroll
            for (int i = 1; i < 16; ++i) top[t] = fmaxf(top[t], s_even[t][i]);
        }
        // tile i: buffers i & 1.  Between its two steps every wave is done with the keys of tile i
        // and the values of tile i - 1, and their buffers take those of i + 2 and i + 1.  Half of
        // the waves stage before their step, half behind it: the two that share a SIMD then do
        // not both leave its matrix unit idle at a time.
        const bool early = WAVES < 8 || wave < WAVES / 2;
        const auto stage = [&](int i, auto par) __attribute__((always_inline)) {
            constexpr int P = decltype(par)::value;
            store_k(P, p2);
            store_v(t_first + i + 1, 1 - P);
            p3 = pages_of(i + 3);
            load_k(t_first + i + 3, p3);
            load_v(t_first + i + 2, p2);
        };
        const auto tile_pair = [&](int i, auto par) __attribute__((always_inline)) {
            constexpr int P = decltype(par)::value;
            step(2 * i, p0.vs0, s_even, s_odd, p_odd, p_even, StageId<P>{}, StageId<1>{}, StageId<1 - P>{},
                 StageId<1>{});
            __syncthreads();
            if (early) stage(i, par);
            step(2 * i + 1, p0.vs1, s_odd, s_even, p_even, p_odd, StageId<1 - P>{}, StageId<0>{}, StageId<P>{},
                 StageId<0>{});
            if (!early) stage(i, par);
            p0 = p1;
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
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int t = 0; t < NC; ++t)
                    o[t][d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(*(const h8v*)(at + vat[2 + u] + d * 32 * V_ROW),
                                                                     __builtin_bit_cast(h8v, p_odd[t][u]), o[t][d], 0, 0, 0);
    }

    // results: lane half hh holds dims 32 d + 8 (i / 4) + 4 hh + i % 4 of its columns
#pragma unroll
    for (int t = 0; t < NC; ++t) {
        const float ll = half_sum(l[t]) * 0x1p-7f;
        const int x = (wave * NC + t) * 32 + lr, col = c0 + x;
        if (col >= it.cols) continue;
        if (splits == 1) {
            const float rl = ll == 0.f ? 0.f : 0x1p-7f / ll;
            const int64_t row = it.q0 + col / G;
            const int head = h * G + col % G;
            uint16_t* const out = a.out + (row * a.heads_q + head) * DV + 4 * hh;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    *(uint2*)(out + 32 * d + 8 * y) =
                        make_uint2(pack_bf16x2(o[t][d][4 * y] * rl, o[t][d][4 * y + 1] * rl),
                                   pack_bf16x2(o[t][d][4 * y + 2] * rl, o[t][d][4 * y + 3] * rl));
            if (a.lse && hh == 0)
                a.lse[row * a.heads_q + head] = ll == 0.f ? neg_inf() : (m[t] + __builtin_log2f(ll)) * kLn2;
        } else {
            const int64_t slot = (int64_t)blockIdx.x * CB + x;
            float* const ws = a.ws + slot * DV + 4 * hh;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    *(v4f*)(ws + 32 * d + 8 * y) = v4f{o[t][d][4 * y], o[t][d][4 * y + 1], o[t][d][4 * y + 2],
                                                       o[t][d][4 * y + 3]} * 0x1p-7f;
            if (hh == 0) {
                float* const ml = a.ws + (int64_t)gridDim.x * CB * DV + slot * 2;
                ml[0] = m[t];
                ml[1] = ll;
            }
        }
    }
}

// Adds the parts of a split launch, in token order: one row per DV / 4 lanes.
template <int DV, int CB>
__global__ __launch_bounds__(kAttnThreads) void attn_block_join_kernel(AttnArgs a, int blocks, int splits) {
    constexpr int L = DV / 4, ROWS = kAttnThreads / L;
    const int tid = threadIdx.x, d4 = tid % L * 4;
    const int G = a.heads_q / a.heads_kv;
    const int64_t row = (int64_t)blockIdx.x * ROWS + tid / L;   // of T * heads_q
    const int64_t t = row / a.heads_q;
    const int head = (int)(row % a.heads_q), h = head / G;
    if (t >= a.T) return;
    int lo = 0, hi = a.R;                                      // the request of token t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.q_offsets[mid] <= t) lo = mid;
        else hi = mid;
    }
    const Item it = Item::of<false>(a, lo);
    const int64_t col = (t - it.q0) * G + head % G;
    if (t < it.q0 || col >= it.cols) return;
    const int b = (int)(it.q0 * G / CB + lo + col / CB);
    const int64_t first = ((int64_t)(blocks - 1 - b) * a.heads_kv + h) * splits;
    const float* const ml = a.ws + (int64_t)blocks * a.heads_kv * splits * CB * DV;
    float m = neg_inf();
    for (int z = 0; z < splits; ++z) m = fmaxf(m, ml[((first + z) * CB + col % CB) * 2]);
    v4f acc = {0.f, 0.f, 0.f, 0.f};
    float l = 0.f;
    for (int z = 0; z < splits; ++z) {
        const int64_t slot = (first + z) * CB + col % CB;
        const float mw = ml[slot * 2], lw = ml[slot * 2 + 1];
        const float f = mw != neg_inf() || lw != 0.f ? __builtin_amdgcn_exp2f(mw - m) : 0.f;
        const v4f v = *(const v4f*)(a.ws + slot * DV + d4);
        l = __builtin_fmaf(lw, f, l);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(v[i], f, acc[i]);
    }
    const float rl = l == 0.f ? 0.f : 1.0f / l;
    *(uint2*)(a.out + (t * a.heads_q + head) * DV + d4) =
        make_uint2(pack_bf16x2(acc[0] * rl, acc[1] * rl), pack_bf16x2(acc[2] * rl, acc[3] * rl));
    if (a.lse && d4 == 0) a.lse[t * a.heads_q + head] = l == 0.f ? neg_inf() : (m + __builtin_log2f(l)) * kLn2;
}

// Tile of a wave, and workgroups of a split launch: as many as the CUs hold at once (16 KB of
// LDS a wave at 128/128, 20 at 192/128: two workgroups; four at 64/64).
constexpr int kSplitTile = 64;
static int split_groups(int dk) { return dk == 64 ? 1024 : 512; }
static bool splits(int64_t max_new, int32_t heads_q, int32_t heads_kv) {
    return max_new * (heads_q / heads_kv) <= kSplitMaxCols;
}

// How a launch of many columns divides: eight waves a workgroup, or four where that leaves CUs
// idle, and the tokens of a block over several workgroups where even those are few.
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
        return (size_t)split_groups(dk) * 2 * kCols * (dv + 2) * sizeof(float);
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
    const int groups = split_groups(DK);
    attn_split_kernel<DK, DV, B, kSplitTile><<<dim3(groups), dim3(kAttnThreads), 0, stream>>>(a, (int)col_tiles);
    const int64_t rows = (int64_t)a.R * a.heads_kv * max_cols;
    // parts per item, about groups / items + 1
    constexpr int FEW = 256 / DV;                               // a wave's strands
    if (items * 4 >= groups) {
        attn_join_kernel<DV, FEW><<<dim3((unsigned)((rows + 3) / 4)), dim3(kAttnThreads), 0, stream>>>(
            a, (int)col_tiles, groups, max_cols);
    } else {
        attn_join_kernel<DV, 4 * FEW><<<dim3((unsigned)rows), dim3(kAttnThreads), 0, stream>>>(
            a, (int)col_tiles, groups, max_cols);
    }
    return hipGetLastError();
}

template <int DK, int DV, int WAVES, int NC>
static hipError_t block_launch(const AttnArgs& a, const BlockPlan& p, hipStream_t stream) {
    // as many parts as the workspace holds
    const int64_t hold = a.ws ? (int64_t)(a.ws_bytes / (32 * NC * WAVES * (DV + 2) * sizeof(float))) : 0;
    const int64_t splits = std::max<int64_t>(1, std::min(p.splits, hold / (p.blocks * a.heads_kv)));
    const unsigned grid = (unsigned)(p.blocks * a.heads_kv * splits);
    attn_block_kernel<DK, DV, WAVES, NC><<<dim3(grid), dim3(64 * WAVES), 0, stream>>>(a, (int)p.blocks, (int)splits);
    if (splits > 1) {
        const int64_t rows = a.T * a.heads_q, per = kAttnThreads / (DV / 4);
        attn_block_join_kernel<DV, 32 * NC * WAVES><<<dim3((unsigned)((rows + per - 1) / per)), dim3(kAttnThreads), 0, stream>>>(
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
    return p.waves == 4 ? block_launch<DK, DV, 4, 1>(a, p, stream) : block_launch<DK, DV, 8, 1>(a, p, stream);
}

hipError_t launch_attn_paged(const AttnArgs& a, int32_t dk, int32_t dv, hipStream_t stream) {
    if (dk == 64 && dv == 64) return attn_launch<64, 64>(a, stream);
    if (dk == 128 && dv == 128) return attn_launch<128, 128>(a, stream);
    if (dk == 192 && dv == 128) return attn_launch<192, 128>(a, stream);
    return hipErrorInvalidValue;
}

}  // namespace bfp8
