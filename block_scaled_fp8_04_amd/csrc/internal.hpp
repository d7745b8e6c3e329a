// internal.hpp - launchers behind the C ABI (include/bfp8.h).  Each launcher
// assumes its arguments were validated by the ABI layer and only enqueues
// kernels on `stream`.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>

namespace bfp8 {

// Largest number of local experts the MoE dispatch handles (LDS counters).
constexpr int kMoeMaxGroups = 1024;

// Compute units of the current device (cached per device).
int device_cu_count();

hipError_t launch_act_quant(const void* x, void* q, float* s, int64_t M, int64_t K,
                            hipStream_t stream);
hipError_t launch_act_quant_pow2(const void* x, void* q, float* s, int64_t M, int64_t K,
                                 hipStream_t stream);
hipError_t launch_gemm_ue8m0(const void* a, const float* as, const void* b, const float* bs,
                             void* c, int64_t M, int64_t N, int64_t K, void* workspace,
                             size_t workspace_bytes, hipStream_t stream);
size_t gemm_ue8m0_workspace_bytes(int64_t M, int64_t N, int64_t K);
hipError_t launch_act_quant_rows(const void* x, int64_t T, const int32_t* row_token,
                                 const int32_t* num_rows, void* q, float* s, int64_t M, int64_t K,
                                 hipStream_t stream);
hipError_t launch_encode_range(uint32_t first, int64_t count, void* out, int variant,
                               hipStream_t stream);
hipError_t launch_bf16_round_range(uint32_t first, int64_t count, void* out, int variant,
                                   hipStream_t stream);
hipError_t launch_weight_dequant(const void* w, const float* s, void* out, int64_t N, int64_t K,
                                 hipStream_t stream);
size_t gemm_workspace_bytes(int64_t M, int64_t N, int64_t K);

// The split last round of large GEMMs on 256 x 256 tiles (the fp8, power-of-two
// scale and bf16 GEMMs share it): when the tiles fill whole rounds of the 256 CUs
// and a last round at most half full of whole tile columns, the nt_tail last
// columns of tiles run as `splits` K ranges of kb_per 128-wide blocks each into
// an fp32 workspace [splits][M][N - 256 nt_main], then one ordered reduction.
struct TailPlan {
    int nt_main = 0, nt_tail = 0, splits = 0;
    int64_t kb_per = 0;
};
TailPlan tail_plan(int64_t M, int64_t N, int64_t K);
size_t tail_workspace_bytes(int64_t M, int64_t N, int64_t K);
// Adds the K ranges' partial sums in order and writes bf16 columns [n1, N) of c.
hipError_t launch_tail_reduce(const float* ws, void* c, int64_t M, int64_t N, int64_t n1,
                              int splits, hipStream_t stream);

enum class GemmConfig { kBig256x256, kBig256x128, kBig128x128 };
GemmConfig gemm_config(int64_t M, int64_t N, int64_t K);
const char* gemm_config_name(GemmConfig cfg);
hipError_t launch_gemm(const void* a, const float* as, const void* b, const float* bs, void* c,
                       int64_t M, int64_t N, int64_t K, void* workspace, size_t workspace_bytes,
                       hipStream_t stream);
hipError_t launch_gemm_quant(const void* a, const float* as, const void* b, const float* bs,
                             void* q, float* qs, int64_t M, int64_t N, int64_t K,
                             hipStream_t stream);
hipError_t launch_gemm_swiglu_quant(const void* a, const float* as, const void* w13,
                                    const float* s13, void* q, float* qs, int64_t M, int64_t n_out,
                                    int64_t K, hipStream_t stream);
size_t linear_workspace_bytes(int64_t M, int64_t N, int64_t K);
// Size of the library-owned device scratch array behind the no-allocation GEMM
// entry point (one per GPU, resident until the process ends).
constexpr size_t kNoAllocScratchBytes = (size_t)64 << 20;
hipError_t launch_gemm_noalloc(const void* a, const float* as, const void* b, const float* bs,
                               void* c, int64_t M, int64_t N, int64_t K, hipStream_t stream);
hipError_t launch_linear_fp8(const void* x, const void* b, const float* bs, void* c, int64_t M,
                             int64_t N, int64_t K, void* workspace, hipStream_t stream);
hipError_t launch_gemm_grouped(const void* a, const float* as, const void* b, const float* bs,
                               void* c, const int32_t* off, int32_t G, int64_t total_M,
                               int64_t N, int64_t K, hipStream_t stream);

hipError_t launch_gemm_bf16(const void* a, const void* b, void* c, int64_t M, int64_t N, int64_t K,
                            void* workspace, size_t workspace_bytes, hipStream_t stream);
const char* gemm_bf16_config_name(int64_t M, int64_t N, int64_t K);

size_t moe_dispatch_workspace_bytes(int64_t T, int32_t k, int32_t G);
hipError_t launch_moe_dispatch(const int32_t* topk, int64_t T, int32_t k, int32_t lo, int32_t G,
                               int32_t* off, int32_t* row_token, int32_t* slot_row, void* ws,
                               hipStream_t stream);
hipError_t launch_moe_combine(const void* out, int64_t rows_cap, const int32_t* slot_row,
                              const float* weight, void* y, int64_t T, int32_t k, int64_t N,
                              hipStream_t stream);

// Requests of one step, and tokens per tile of the plan's tile offsets (kv_cache.hip,
// attn_paged.hip).
constexpr int kKvMaxRequests = 4096;
constexpr int kKvTile = 128;
hipError_t launch_kv_plan(const int32_t* ctx_lens, const int32_t* new_lens, int64_t R,
                          const int32_t* free_pages, int64_t n_free, const int32_t* free_head,
                          int32_t* block_table, int64_t width, int32_t page, int32_t* q_offsets,
                          int32_t* kv_lens, int32_t* tile_offsets, int32_t* slot_map,
                          int32_t* positions, int64_t T, int32_t* counts, hipStream_t stream);
hipError_t launch_kv_append(const void* k, int64_t k_ts, int64_t k_hs, const void* v, int64_t v_ts,
                            int64_t v_hs, const int32_t* slot_map, int64_t T, void* k_cache,
                            float* k_scales, void* v_cache, float* v_scales, int64_t pages,
                            int32_t page, int32_t heads, int32_t dk, int32_t dv,
                            hipStream_t stream);

// Arguments of one paged-attention call (validated by the ABI layer).
struct AttnArgs {
    const uint16_t* q;
    int64_t q_ts, q_hs;
    const uint8_t* k_cache;
    const float* k_scales;
    const uint8_t* v_cache;
    const float* v_scales;
    int64_t pages;
    const int32_t* block_table;
    int64_t width;
    const int32_t* q_offsets;
    const int32_t* kv_lens;
    const int32_t* tile_offsets;
    int R, heads_q, heads_kv, log_b;
    int64_t T, max_new;
    float scale;
    uint16_t* out;
    float* lse;
    float* ws;
    size_t ws_bytes;
};
size_t attn_paged_workspace_bytes(int64_t R, int64_t max_new, int32_t heads_q, int32_t heads_kv,
                                  int32_t dk, int32_t dv);
hipError_t launch_attn_paged(const AttnArgs& a, int32_t dk, int32_t dv, hipStream_t stream);

// Rotary positions (rope.hip) and the latent cache (latent_cache.hip, attn_latent.hip): a token's
// latent and the rotated dims of its key.
constexpr int kLatent = 512;
constexpr int kLatentRope = 64;
constexpr int kRopeMaxDim = 1024;
hipError_t launch_rope(const void* x, int64_t x_ts, int64_t x_hs, const int32_t* positions,
                       const float* inv_freq, void* out, int64_t o_ts, int64_t o_hs, int64_t T,
                       int32_t heads, int32_t dim, bool interleaved, float amplitude,
                       hipStream_t stream);
hipError_t launch_latent_append(const void* kv, int64_t kv_ts, const void* norm_weight, float eps,
                                const int32_t* slot_map, const int32_t* positions,
                                const float* inv_freq, bool interleaved, float amplitude, int64_t T,
                                void* codes, float* scales, void* rope, int64_t slots,
                                hipStream_t stream);
hipError_t launch_latent_gather(const void* codes, const float* scales, const void* rope,
                                int64_t pages, int32_t page, const int32_t* block_table,
                                int64_t width, const int32_t* row_offsets, const int32_t* starts,
                                int64_t R, int64_t rows, void* latent, int64_t l_ts, void* rope_out,
                                int64_t r_ts, hipStream_t stream);

// Quotient and remainder by a number that is the same for a whole launch: the quotient by
// m = 2^32 / d rounded down is short by one at most.
struct Divisor {
    uint32_t d, m;
    static Divisor by(int32_t d) { return {(uint32_t)d, (uint32_t)std::min<uint64_t>(((uint64_t)1 << 32) / d, UINT32_MAX)}; }
    __device__ __forceinline__ int of(int x, int& rest) const {
        uint32_t q = __umulhi((uint32_t)x, m), r = (uint32_t)x - q * d;
        if (r >= d) {
            q += 1;
            r -= d;
        }
        rest = (int)r;
        return (int)q;
    }
    __device__ __forceinline__ int of(int x) const {
        int rest;
        return of(x, rest);
    }
};

// Arguments of one call of attention over the latent cache (validated by the ABI layer).
struct LatentArgs {
    const uint16_t* q_latent;
    int64_t ql_ts, ql_hs;
    const uint16_t* q_rope;
    int64_t qr_ts, qr_hs;
    const uint8_t* codes;
    const float* scales;
    const uint16_t* rope;
    int64_t pages;
    const int32_t* block_table;
    int64_t width;
    const int32_t* q_offsets;
    const int32_t* kv_lens;
    int R, heads, log_b;
    Divisor by_heads;
    int64_t T, max_new;
    float scale;
    uint16_t* out;
    int64_t o_ts, o_hs;
    float* lse;
    float* ws;
    bool q_near;             // set by the launcher: queries are aligned and rows' offsets small
};
size_t attn_latent_workspace_bytes(int64_t R, int64_t max_new, int32_t heads);
hipError_t launch_attn_latent(LatentArgs a, hipStream_t stream);

}  // namespace bfp8
