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
#include "device_codec.hpp"
#include "internal.hpp"
#include "tile_common.hpp"

namespace bfp8 {

constexpr int kAttnThreads = 256;
constexpr int kAttnWaves = kAttnThreads / 64;
constexpr int kCols = 16;                     // query columns of a wave
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

// 32 elements of a bf16 query row (negated for a negative scale); p == nullptr: zeros.
__device__ __forceinline__ void load_q32(const uint16_t* p, bool vec, bool negate, bf8v (&q)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (p != nullptr) {
            if (vec) {
                x = ((const uint4*)p)[i];
            } else {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[j] = (uint32_t)p[8 * i + 2 * j] | ((uint32_t)p[8 * i + 2 * j + 1] << 16);
                x = make_uint4(w[0], w[1], w[2], w[3]);
            }
            const uint32_t f = negate ? 0x80008000u : 0u;
            x = make_uint4(x.x ^ f, x.y ^ f, x.z ^ f, x.w ^ f);
        }
        q[i] = __builtin_bit_cast(bf8v, x);
    }
}

// One wave's attention of kCols query columns over 128-token tiles
// tile0, tile0 + step, ... < tile1 of one request and KV head.
template <int DK, int DV>
struct AttnWave {
    static constexpr int KS = (DK + 127) / 128;      // 128-wide steps of the first product
    static constexpr int DT = DV / 16;               // 16-row tiles of O^T
    bf8v q[KS][4];                                   // lane group g: dims 128 s + 32 g ..
    v4f o[DT];
    float m, l;                                      // l: this lane's tokens only

    // column `lane & 15` is this query row (NULL: an unused column)
    __device__ __forceinline__ void load_q(const uint16_t* row, bool vec, bool negate, int g) {
#pragma unroll
        for (int s = 0; s < KS; ++s)
            load_q32(row != nullptr && 128 * s + 32 * g < DK ? row + 128 * s + 32 * g : nullptr, vec,
                     negate, q[s]);
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d] = v4f{0.f, 0.f, 0.f, 0.f};
        m = neg_inf();
        l = 0.f;
    }

    __device__ __forceinline__ void walk(const AttnArgs& a, int r, int h, int tile0, int tile1,
                                         int step, int kv_len, int limit, int free_limit, float c) {
        // limit: this column sees tokens below it; free_limit: every column sees those below
        if (tile0 >= tile1) return;
        const int lane = threadIdx.x & 63, g = lane >> 4, lr = lane & 15;
        const int log_b = a.log_b, B = 1 << log_b;
        const int last = (kv_len - 1) >> log_b;                 // last page that is read
        const int32_t* const table = a.block_table + (int64_t)r * a.width;
        // this lane's K rows are tokens ktok + 4 t, its P^T and V^T elements tokens 32 g + j
        const int ktok = 32 * (lr >> 2) + (lr & 3);
        const auto page_of = [&](int token) {
            const int j = min(token >> log_b, last);
            return min(max((int64_t)table[j], (int64_t)0), a.pages - 1) * a.heads_kv + h;
        };
        for (int tile = tile0; tile < tile1; tile += step) {
            const int base = tile * kKvTile;
            const int64_t kp = page_of(base + ktok), vp = page_of(base + 32 * g);
            const float ke = a.k_scales[kp], ve = a.v_scales[vp];
            const uint8_t* const kb = a.k_cache + kp * ((int64_t)B * DK) +
                                      ((base + ktok) & (B - 1)) * DK + 32 * g;
            const uint8_t* const vb = a.v_cache + vp * ((int64_t)B * DV) + lr * B + (32 * g & (B - 1));
            v4f s[8];
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                s[t] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    v8i kf = {0, 0, 0, 0, 0, 0, 0, 0};
                    if (128 * ks + 128 <= DK || 128 * ks + 32 * g < DK) {
                        const uint4* p = (const uint4*)(kb + 4 * t * DK + 128 * ks);
                        kf = frag_from(p[0], p[1]);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        s[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            widen8(kf[2 * i], kf[2 * i + 1], ke), q[ks][i], s[t], 0, 0, 0);
                }
            }
            v8i vf[DT];
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                const uint4* p = (const uint4*)(vb + 16 * d * B);
                vf[d] = frag_from(p[0], p[1]);
            }
            if (base + kKvTile > free_limit) {
                const int seen = limit - base - 32 * g;         // this lane's tokens: the first `seen`
#pragma unroll
                for (int t = 0; t < 8; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (4 * t + i >= seen) s[t][i] = neg_inf();
                // bytes behind the last token may hold anything: 0 * NaN is NaN
                if (base + kKvTile > kv_len) {
                    const int live = kv_len - base - 32 * g;
#pragma unroll
                    for (int w = 0; w < 8; ++w) {
                        const int nb = min(max(live - 4 * w, 0), 4);
                        const int mask = nb == 4 ? -1 : (1 << (8 * nb)) - 1;
#pragma unroll
                        for (int d = 0; d < DT; ++d) vf[d][w] &= mask;
                    }
                }
            }
            bf8v ph[4], pl[4];
            softmax(s, c, ph, pl);
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const bf8v x = widen8(vf[d][2 * i], vf[d][2 * i + 1], ve);
                    o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, ph[i], o[d], 0, 0, 0);
                    o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, pl[i], o[d], 0, 0, 0);
                }
        }
    }

    // S^T of one tile to P^T, with this lane's tokens 8 i .. 8 i + 7 in ph[i] (rounded) and pl[i]
    // (the remainder); rescales o and l to the new running maximum.
    __device__ __forceinline__ void softmax(v4f (&s)[8], float c, bf8v (&ph)[4], bf8v (&pl)[4]) {
        float mx = s[0][0];
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) mx = fmaxf(mx, s[t][i]);
        mx = fmaxf(mx, __shfl_xor(mx, 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        const float m_new = fmaxf(m, __builtin_ceilf(mx * c));
        // logits so large that fp32 cannot hold s c - m to a unit: round s c alone, as m was, so
        // that the largest keeps p = 1
        if (__any(__builtin_fabsf(m_new) > 4194304.f && m_new != neg_inf())) {
#pragma unroll
            for (int t = 0; t < 8; ++t) s[t] *= c;
            c = 1.f;
        }
        const float sub = m_new == neg_inf() ? 0.f : -m_new;    // nothing seen yet: every p is 0
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
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

// Joins the four waves' results of one 16-column item in LDS.  Every wave ends up knowing
// the column's (m, l); lane (column, dims) results are left in `part` as
// sum over waves of O 2^(m_w - m), [kCols][DV] fp32 spread over the threads: thread x owns
// column x / 16, dims 4 (x % 16) + 64 j.
template <int DK, int DV>
__device__ __forceinline__ void join_waves(AttnWave<DK, DV>& w, float* lds_o, float* lds_ml,
                                           float (&part)[DV / 16], float& m, float& l) {
    constexpr int ROW = DV + 4;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, col = lane & 15;
    float ll = w.l + __shfl_xor(w.l, 16);
    ll += __shfl_xor(ll, 32);
    __syncthreads();                                            // the last item's reads
    if (g == 0) {
        lds_ml[wave * kCols + col] = w.m;
        lds_ml[(kAttnWaves + wave) * kCols + col] = ll;
    }
#pragma unroll
    for (int d = 0; d < DV / 16; ++d)
        *(v4f*)(lds_o + (wave * kCols + col) * ROW + 16 * d + 4 * g) = w.o[d];
    __syncthreads();
    const int oc = tid >> 4, od = (tid & 15) * 4;
    m = neg_inf();
#pragma unroll
    for (int x = 0; x < kAttnWaves; ++x) m = fmaxf(m, lds_ml[x * kCols + oc]);
    l = 0.f;
#pragma unroll
    for (int j = 0; j < DV / 16; ++j) part[j] = 0.f;
#pragma unroll
    for (int x = 0; x < kAttnWaves; ++x) {
        const float mw = lds_ml[x * kCols + oc];
        if (mw == neg_inf() && lds_ml[(kAttnWaves + x) * kCols + oc] == 0.f) continue;
        const float f = __builtin_amdgcn_exp2f(mw - m);
        l = __builtin_fmaf(lds_ml[(kAttnWaves + x) * kCols + oc], f, l);
#pragma unroll
        for (int j = 0; j < DV / 64; ++j) {
            const v4f v = *(const v4f*)(lds_o + (x * kCols + oc) * ROW + od + 64 * j);
#pragma unroll
            for (int i = 0; i < 4; ++i) part[4 * j + i] = __builtin_fmaf(v[i], f, part[4 * j + i]);
        }
    }
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

// One workgroup per (request, KV head, 16 query columns): its waves take every fourth tile.
template <int DK, int DV>
__global__ __launch_bounds__(kAttnThreads, 1) void attn_item_kernel(AttnArgs a, int col_tiles) {
    __shared__ float lds_o[kAttnWaves * kCols * (DV + 4)];
    __shared__ float lds_ml[2 * kAttnWaves * kCols];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int64_t item = blockIdx.x;
    const int ct = (int)(item % col_tiles);
    item /= col_tiles;
    const int h = (int)(item % a.heads_kv), r = (int)(item / a.heads_kv);
    const int G = a.heads_q / a.heads_kv;
    const int64_t q0 = min(max((int64_t)a.q_offsets[r], (int64_t)0), a.T);
    const int64_t q1 = min(max((int64_t)a.q_offsets[r + 1], q0), a.T);
    const int n = (int)(q1 - q0);
    const int cols = (int)min((int64_t)n, a.max_new) * G;
    if (ct * kCols >= cols) return;
    const int kv_len = (int)min(max((int64_t)a.kv_lens[r], (int64_t)0), a.width << a.log_b);

    const auto col_limit = [&](int c) { return min(kv_len, max(kv_len - n + c / G + 1, 0)); };
    const int col = ct * kCols + (lane & 15), g = lane >> 4;
    const bool used = col < cols;
    const bool vec = ((uintptr_t)a.q % 16) == 0 && ((a.q_ts | a.q_hs) % 8) == 0;
    AttnWave<DK, DV> w;
    w.load_q(used ? a.q + (q0 + col / G) * a.q_ts + (int64_t)(h * G + col % G) * a.q_hs : nullptr, vec,
             a.scale < 0.f, g);
    const int last_col = min(ct * kCols + kCols, cols) - 1;
    const int tiles = (col_limit(last_col) + kKvTile - 1) / kKvTile;
    w.walk(a, r, h, wave, tiles, kAttnWaves, kv_len, used ? col_limit(col) : 0, col_limit(ct * kCols),
           fmaxf(__builtin_fabsf(a.scale) * kLog2e, 0x1p-126f));     // -inf times 0 is NaN
    float part[DV / 16], m, l;
    join_waves<DK, DV>(w, lds_o, lds_ml, part, m, l);
    const int oc = ct * kCols + (tid >> 4);
    if (oc < cols) store_row<DV>(a, q0 + oc / G, h * G + oc % G, (tid & 15) * 4, part, m, l);
}

size_t attn_paged_workspace_bytes(int64_t, int64_t, int32_t, int32_t, int32_t, int32_t) { return 0; }

template <int DK, int DV>
static hipError_t attn_launch(const AttnArgs& a, hipStream_t stream) {
    const int64_t col_tiles = (a.max_new * (a.heads_q / a.heads_kv) + kCols - 1) / kCols;
    const int64_t items = (int64_t)a.R * a.heads_kv * col_tiles;
    attn_item_kernel<DK, DV><<<dim3((unsigned)items), dim3(kAttnThreads), 0, stream>>>(a, (int)col_tiles);
    return hipGetLastError();
}

hipError_t launch_attn_paged(const AttnArgs& a, int32_t dk, int32_t dv, hipStream_t stream) {
    if (dk == 64 && dv == 64) return attn_launch<64, 64>(a, stream);
    if (dk == 128 && dv == 128) return attn_launch<128, 128>(a, stream);
    if (dk == 192 && dv == 128) return attn_launch<192, 128>(a, stream);
    return hipErrorInvalidValue;
}

}  // namespace bfp8
