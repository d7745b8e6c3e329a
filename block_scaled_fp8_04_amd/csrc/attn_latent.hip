// attn_latent.hip - attention whose keys and values are one shared latent per token (the absorbed
// form of latent attention) over the paged latent cache, on gfx950.
//
//     x_t = scale (q_latent . c_t + q_rope . r_t),   out = sum_t p_t c_t / sum_t p_t,  p_t = exp(x_t - max)
//
// with c_t = 2^e_t times 512 e4m3 codes and r_t 64 bf16.  A query row is a (new token, head) pair:
// every row of a request reads the same tokens, so a token is brought to LDS once and serves all
// rows of a workgroup, as key and as value: 2176 operations per row for its 644 bytes.
//
// Both products are taken transposed, the cache as the first operand:
//     S^T [token, row] = C Q^T + R Qr^T,     O^T [dim, row] += C^T P^T
// so a lane holds one row's logits (lane & 31, tokens 8 i + 4 (lane / 32) + 0 .. 3 of 32), the softmax
// needs one exchange between the wave's halves, and its results are the second product's operand
// where they stand: that product sums over the tokens in the order in which the lanes hold them.
// C^T comes from the same bytes of LDS through transposing reads (8 tokens of one dim a lane), whose
// rows are given by address, so in that order too.
//
// Precision.  As keys, codes are widened to bf16 with their token's scale, exactly, and q is bf16 as
// it comes.  As values they are widened to fp16 without it, exactly as well, and the scale goes into
// the weight: the maximum is taken over x_t + e_t (in units of log 2), w_t = 2^(x_t + e_t - reference) is
// rounded to fp16 once (2^-11 of it, where a bf16 weight would lose 2^-8, as much as the rounding of
// the output), and the norm sums w_t 2^-e_t before that rounding.  So a weight's size is that of the
// token's contribution, and as the reference lies 2^7 below the largest, all of fp16's range is used: below
// its normal numbers a weight loses 2^-31 of the largest
// contribution.  Logits, maxima, norms and sums are fp32; maxima are rounded up to integers, so that
// rescaling by 2^(old - new) is exact.  (The fp8 matrix product would take the codes as they are, but it
// drops what lies 13 bits below the largest product it adds: 2^-12.3 of the sum of their sizes, measured.)
//
// What bounds it.  64 requests of 512 to 8192 tokens: with 16 heads their 118 MB, which the main kernel
// brings at 3.3 TB/s in 36 us (4.9 is what a large copy reaches), its tiles alone at 5.1; about 5 us are a
// workgroup's first loads, one behind the other.  With 128 heads their 50 GFLOP, which take 77 us, 0.65
// PFLOP/s (1.2 is what a large matrix product reaches), and 11 us for the join, at 4.5 TB/s.  The matrix
// units are busy for 28 % of that: a wave has its SIMD to itself, as accumulators and queries take up its
// registers, so nothing covers the softmax (800 of a tile's 5000 cycles), the trade of weights (700) and
// the first reads behind each barrier.
#include <algorithm>

#include "attn_common.hpp"
#include "device_codec.hpp"
#include "internal.hpp"
#include "tile_common.hpp"

namespace bfp8 {

typedef _Float16 h8v __attribute__((ext_vector_type(8)));
typedef _Float16 h2v __attribute__((ext_vector_type(2)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef int v2i __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) v2i* lds_v2i;

constexpr int kLatThreads = 256;
constexpr int kLatGroups = 256;               // most workgroups of a split launch: one a CU (LDS, registers)
// What an item's queries and results cost, in tiles: 64 requests of 128 heads take 80.1 us if shares
// count 2 for them, 76.8 with 3, 77.8 with 4, and 12 us more with none.
constexpr int kLatItemCost = 3;
// Items of a split launch are fewer than this, by the bound that the host knows; as many fill the chip.
// 600 of 300 requests of 128 heads over 512 to 8192 tokens take 347 us split and 495 if not, 1008 by the
// bound of 24 requests with 1 to 60 new tokens 59 and 90; but 1600 of 8 requests with 100 new tokens each
// 239 and 189, as a split item's tiles are all of its request's, also those that its rows do not see, and
// 700 of a tile or two 30 and 24.
constexpr int kLatItems = 1024;
constexpr int kLatTile = 64;                  // tokens of a tile
constexpr int kLatCodes = kLatTile * kLatent; // its bytes of codes and of rotated keys
constexpr int kLatStage = kLatCodes + kLatTile * kLatentRope * 2;
// A row's reference is the largest exponent of two that it met, rounded up, less kLatRise, and follows one
// that passes it by more than kLatTop.  So weights reach 2^15, and the largest is 2^6 or more: fp16's last
// step, 2^-24, is 2^-30 of it or less.  (kLatTop 14: 64 requests of 128 heads 85.6 us instead of 84.4.)
constexpr float kLatRise = 7.f;
constexpr float kLatTop = 15.f;

// The permutation of a row's 16-byte chunks in LDS: chunk c of row r lies at c ^ lat_swz(r).  Key
// reads take the same chunk of 16 rows, all different here; transposing reads take two neighbouring
// chunks of rows with equal bit 2, so that bit is the lowest and the other three keep pairs apart.
__device__ __forceinline__ constexpr int lat_swz(int r) {
    return (r & 3) << 1 | (r >> 3 & 1) << 3 | (r >> 2 & 1);
}
__device__ __forceinline__ constexpr int rope_swz(int r) { return r >> 1 & 7; }

// Eight e4m3 codes as fp16 (exact).
__device__ __forceinline__ h8v widen8_f16(int w0, int w1) {
    const h2v a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.f, false);
    const h2v b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.f, true);
    const h2v c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.f, false);
    const h2v d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.f, true);
    return h8v{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// The workspace: parts of kLatSlots runs, (maximum, norm) of their rows, and the items' notes.
constexpr int64_t kLatSlots = 2 * kLatGroups;
__device__ __forceinline__ float2* latent_ml(const LatentArgs& a, int rows) {
    return (float2*)(a.ws + kLatSlots * rows * kLatent);
}
__device__ __forceinline__ int2* latent_info(const LatentArgs& a, int rows) {
    return (int2*)(latent_ml(a, rows) + kLatSlots * rows);
}

// Barrier behind everything that this wave wrote to LDS or has on its way there.
__device__ __forceinline__ void barrier_all() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(7 << 4);                          // vmcnt 0, lgkmcnt 0
    barrier_lds();
}

// Barrier behind what this wave wrote to LDS, but not behind its loads that are on their way there.
__device__ __forceinline__ void barrier_written() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(15 | 7 << 4 | 3 << 14);           // lgkmcnt 0
    barrier_lds();
}

// A request's part in the launch: its first new token, its query rows and cached tokens.
struct LatentItem {
    int q0, n, rows, kv_len;
    static __device__ __forceinline__ LatentItem of(const LatentArgs& a, int from, int to, int kv_len) {
        LatentItem it;
        it.q0 = min(max(from, 0), (int)a.T);                     // (T has 29 bits)
        it.n = min(max(to, it.q0), (int)a.T) - it.q0;
        it.rows = (int)min((int64_t)it.n, a.max_new) * a.heads;
        it.kv_len = (int)min(max((int64_t)kv_len, (int64_t)0), a.width << a.log_b);
        return it;
    }
    // tokens that new token i sees
    __device__ __forceinline__ int limit(int i) const { return min(kv_len, max(kv_len - n + i + 1, 0)); }
};

// Tiles of kLatTile tokens that hold this many (lengths reach 2^31 - 32).
__device__ __forceinline__ int latent_tiles(int tokens) {
    return (int)(((uint32_t)tokens + kLatTile - 1) / kLatTile);
}

// 64 consecutive requests, one per lane, and the cost of their work before each: for each item its tiles
// and kLatItemCost.
template <int ROWS>
struct LatentRequests {
    int base, q0, q1, kv_len;
    int64_t before, cost;                            // before the lane's request; of it
    __device__ __forceinline__ void load(const LatentArgs& a, int from) {
        base = from;
        const int mine = base + (int)(threadIdx.x & 63), r = min(mine, a.R - 1);
        q0 = a.q_offsets[r];
        q1 = a.q_offsets[r + 1];
        kv_len = a.kv_lens[r];
        const LatentItem it = LatentItem::of(a, q0, q1, kv_len);
        cost = mine < a.R && it.kv_len > 0
                   ? (int64_t)((it.rows + ROWS - 1) / ROWS) * (latent_tiles(it.kv_len) + kLatItemCost) : 0;
    }
    // sums up the costs, with `start` before the 64 requests; returns what comes before the next
    __device__ __forceinline__ int64_t scan(int64_t start) {
        int64_t sum = cost;
        add<0x111, 0xF>(sum);                                    // rows of 16 lanes: from 1, 2, 4, 8 before
        add<0x112, 0xF>(sum);
        add<0x114, 0xF>(sum);
        add<0x118, 0xF>(sum);
        add<0x142, 0xA>(sum);                                    // row 1, 3: from the last of the one before
        add<0x143, 0xC>(sum);                                    // row 2, 3: from the last of row 1
        before = start + sum - cost;
        return start + from_lane(sum, 63);
    }
    template <int CONTROL, int LANES>
    static __device__ __forceinline__ void add(int64_t& sum) {
        const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)sum, CONTROL, LANES, 0xF, false);
        const int hi = __builtin_amdgcn_update_dpp(0, (int)(sum >> 32), CONTROL, LANES, 0xF, false);
        sum += (int64_t)hi << 32 | lo;
    }
    static __device__ __forceinline__ int64_t from_lane(int64_t x, int lane) {
        return (int64_t)(uint32_t)__builtin_amdgcn_readlane((int)x, lane) |
               (int64_t)__builtin_amdgcn_readlane((int)(x >> 32), lane) << 32;
    }
    __device__ __forceinline__ LatentItem item(const LatentArgs& a, int r) const {
        return LatentItem::of(a, __builtin_amdgcn_readlane(q0, r - base), __builtin_amdgcn_readlane(q1, r - base),
                              __builtin_amdgcn_readlane(kv_len, r - base));
    }
};

// The lane, in a form that keeps what is computed from it at a run's ends from being held in registers
// over its tiles.
__device__ __forceinline__ int fresh_lane() {
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    return lane;
}

// An item, that is a request's row tile, and its tiles.  Uniform.
struct LatentJob {
    int r, rt, tiles;
    LatentItem it;
};

// A workgroup's share of the work: runs of tiles, each of one item.
template <int ROWS>
struct LatentShare {
    LatentRequests<ROWS> reqs;
    LatentJob job;
    int tile;                                        // the run's first
    int64_t at, to;                                  // cost before it; at the share's end

    // From cost `from` on, in request r (one of reqs); false: no tile begins there.
    __device__ __forceinline__ bool begin(const LatentArgs& a, int r, int64_t from, int64_t end) {
        take(a, r);
        const int64_t local = from - reqs.from_lane(reqs.before, r - reqs.base);
        const int per = job.tiles + kLatItemCost;
        job.rt = __builtin_amdgcn_readfirstlane((int)quotient(local, per));
        const int x = (int)(local - (int64_t)job.rt * per);
        tile = max(x - kLatItemCost, 0);
        at = from + tile + kLatItemCost - x;
        to = end;
        return at < to;
    }
    __device__ __forceinline__ void take(const LatentArgs& a, int r) {
        job.r = r;
        job.rt = 0;
        job.it = reqs.item(a, r);
        job.tiles = latent_tiles(job.it.kv_len);
    }
    // the tile behind the run's last
    __device__ __forceinline__ int end() const { return (int)min((int64_t)job.tiles, tile + (to - at)); }
    // To the next run; false: there is none.
    __device__ __forceinline__ bool next(const LatentArgs& a) {
        at += job.tiles - tile + kLatItemCost;
        tile = 0;
        if (at >= to) return false;
        if (++job.rt * ROWS < job.it.rows) return true;
        uint64_t later = __ballot(reqs.cost > 0) & ~((2ull << (job.r - reqs.base)) - 1);
        while (later == 0 && reqs.base + 64 < a.R) {
            reqs.load(a, reqs.base + 64);
            later = __ballot(reqs.cost > 0);
        }
        if (later == 0) return false;                            // (not with cost left)
        take(a, reqs.base + __ffsll((unsigned long long)later) - 1);
        return true;
    }
};

struct LatentLds {
    float2* scales;                                  // this wave's [64 tokens] exponents and inverses
    uint4* trade;                                    // [row half][token half][2][64 lanes] weights
    float* refs;                                     // [row half][token half][2][64 lanes] references, norms
};

// One workgroup's way through its tiles.  Its four waves form weights two by two, each for 32 rows and
// half tg of a tile's tokens, trade them through LDS, and each sums its rows' values over all of the
// tile's tokens for its share of the dims:
//   RW == 2 (64 rows): wave (rg, x) has 32 rows, token half x and dim half x.
//   RW == 1 (32 rows): wave x has all rows, token half x & 1 and dim quarter x; two waves form the
//     same weights, which is work twice done, but with so few rows the cache's bytes are what counts.
// (A wave with 32 rows and all dims would keep 256 registers of O next to 144 of q, which the compiler
// does not manage without spills.  Eight waves of 256 registers, which share the dims of the logits as
// well and widen each code once for 64 rows, take 87 us where these take 77: a second exchange for each
// tile, and twice as many waves to read all weights.)
// A wave alone on its SIMD issues an instruction every five cycles and a matrix instruction takes 32, so
// the four conversions that each needs stand before it or after it, not eight of them before two.
template <int RW>
struct LatentWalk {
    static constexpr int DT = RW == 2 ? 8 : 4;       // blocks of 32 dims of a wave
    static constexpr int ROWS = 32 * RW;

    v16f o[DT];
    float m, l;                                      // l: over this wave's tokens of this lane only
    bf8v q[36];                                      // 32 of the latent, 4 of the rotated part
    int rg, tg, dw;                                  // this wave's rows, tokens, dims
    bool gives;                                      // its weights are the ones that are traded
    int limit, free_limit;                           // tokens that this lane's row sees; that all rows see
    int from, kv_len;                                // the run's first tile; cached tokens

    __device__ __forceinline__ void init() {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        rg = RW == 2 ? wave & 1 : 0;
        tg = RW == 2 ? wave >> 1 : wave & 1;
        dw = RW == 2 ? wave >> 1 : wave;
        gives = RW == 2 || wave < 2;
    }
    // this lane's row, counted in the item
    __device__ __forceinline__ int row(int rt) const { return rt * ROWS + rg * 32 + (threadIdx.x & 31); }

    // An item's queries come by way of a free stage, 512 / RW dims of all rows at a time, as whole rows,
    // and go from there into accumulation registers, where the matrix instructions take them from.
    // (Straight from memory a wave's lanes read 32 bytes of 32 rows at a time: 14000 cycles for 64 rows.)
    // Rows behind the item's last are copies of that one: nothing of them is stored.  Rows that are not
    // 16-byte aligned, or far apart, are read by elements.
    static constexpr int QROW = 1024 / RW;           // bytes of a staged row; the rotated dims come last
    // (chunk c of row r lies at c ^ (r & 15), or at rope_swz(r): sixteen rows' same chunk is spread)
    template <int X>
    static __device__ __forceinline__ void stage_q(const LatentArgs& a, const LatentJob& u, uint8_t* st) {
        constexpr int MINE = ROWS / 4, C = QROW / 16;            // rows of a wave; chunks of a row
        const int lane = fresh_lane(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int first = u.rt * ROWS + wave * MINE, last = u.it.rows - 1;
        if (!a.q_near) {                                         // by elements
            constexpr int N = X == RW - 1 ? C + 8 : C;
#pragma unroll 1
            for (int i = lane; i < MINE * N; i += 64) {
                const int r = i / N, c = i % N, at = wave * MINE + r;
                int j;
                const int64_t t = u.it.q0 + a.by_heads.of(min(first + r, last), j);
                const uint16_t* const from = c < C ? a.q_latent + t * a.ql_ts + j * a.ql_hs + X * 256 + c * 8
                                                   : a.q_rope + t * a.qr_ts + j * a.qr_hs + (c - C) * 8;
                *(bf8v*)(c < C ? st + at * QROW + ((c ^ (at & 15)) << 4)
                               : st + kLatCodes + at * 128 + ((c - C ^ rope_swz(at)) << 4)) = load_q8(from, false, false);
            }
            return;
        }
        const int t0 = a.by_heads.of(min(first, last));
        const int64_t t = u.it.q0 + t0;
        // a lane's row steps by `by`; offsets from the first row's token have 32 bits (a.q_near)
        const auto rows = [&](uint32_t ts, uint32_t hs, int r, int by, int n, auto&& put) {
            int j, dj, lj;
            const uint32_t end = (a.by_heads.of(last, lj) - t0) * ts + lj * hs;
            uint32_t at = (a.by_heads.of(min(first + r, last), j) - t0) * ts;
            at += j * hs;
            const int dt = a.by_heads.of(by, dj);
            const uint32_t step = dt * ts + dj * hs, wrap = ts - a.heads * hs;
#pragma unroll
            for (int k = 0; k < n; ++k) {
                put(k, r, first + r < last ? at : end);
                r += by;
                j += dj;
                at += step;
                if (j >= a.heads) {
                    j -= a.heads;
                    at += wrap;
                }
            }
        };
        const __amdgpu_buffer_rsrc_t latents = make_rsrc(a.q_latent + t * a.ql_ts, ~0ull);
        rows((uint32_t)a.ql_ts * 2, (uint32_t)a.ql_hs * 2, lane / C, RW, MINE / RW,
             [&](int k, int r, uint32_t at) __attribute__((always_inline)) {
                 buf_lds16(latents, at + ((lane % C ^ (wave * MINE + r & 15)) << 4),
                           X * 512, st + wave * (MINE * QROW) + k * 1024);
             });
        const __amdgpu_buffer_rsrc_t ropes = make_rsrc(a.q_rope + t * a.qr_ts, ~0ull);
        if (X == RW - 1)
            rows((uint32_t)a.qr_ts * 2, (uint32_t)a.qr_hs * 2, lane / 8, 8, MINE / 8,
                 [&](int k, int r, uint32_t at) __attribute__((always_inline)) {
                     buf_lds16(ropes, at + ((lane % 8 ^ rope_swz(wave * MINE + r)) << 4),
                               0, st + kLatCodes + wave * (MINE * 128) + k * 1024);
                 });
    }
    template <int X>
    __device__ __forceinline__ void read_q(const uint8_t* st) {
        const int lane = fresh_lane(), h = lane >> 5, r = rg * 32 + (lane & 31);
        // operand s: dims 32 (s / 2) + 16 h + 8 (s % 2) .., as a 16-byte read of codes feeds two
#pragma unroll
        for (int s = X * 16; s < X * 16 + 32 / RW; ++s) {
            const int chunk = s / 2 * 4 + 2 * h + s % 2 - X * 32;
            q[s] = *(const bf8v*)(st + r * QROW + ((chunk ^ (r & 15)) << 4));
        }
        if (X == RW - 1) {
#pragma unroll
            for (int s = 0; s < 4; ++s)
                q[32 + s] = *(const bf8v*)(st + kLatCodes + r * 128 + (((2 * s + h) ^ rope_swz(r)) << 4));
        }
#pragma unroll
        for (int s = X * 16; s < (X == RW - 1 ? 36 : X * 16 + 32 / RW); ++s) asm volatile("" : "+a"(q[s]));
    }
    __device__ __forceinline__ void begin(const LatentArgs& a, const LatentJob& u, int tile) {
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
        m = neg_inf();
        l = 0.f;
        const int mine = row(u.rt);
        limit = mine < u.it.rows ? u.it.limit(a.by_heads.of(mine)) : 0;
        free_limit = u.it.limit(a.by_heads.of(u.rt * ROWS));
        from = tile;
        kv_len = u.it.kv_len;
    }

    // The table entry of the page that holds token `lane` of a tile (of the last page, behind the end).
    static __device__ __forceinline__ int entry(const LatentArgs& a, const LatentJob& u, int tile) {
        const uint32_t pos = min((uint32_t)tile * kLatTile + (threadIdx.x & 63), (uint32_t)u.it.kv_len - 1);
        return (a.block_table + u.r * a.width)[pos >> a.log_b];
    }

    // A tile's way to LDS: each wave brings 16 of its tokens, by ten loads that bypass the registers.
    // not real: the loads lie outside their resource and read nothing.
    struct Fetch {
        __amdgpu_buffer_rsrc_t codes, rope;
        const float* scale;                          // of token `lane`
        __device__ __forceinline__ Fetch(const LatentArgs& a, int tile, int entry, bool real) {
            const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
            const uint32_t in_page = (1u << a.log_b) - 1, first = (uint32_t)tile * kLatTile;
            const uint32_t page = (uint32_t)min(max(entry, 0), (int)a.pages - 1);        // slots have 31 bits
            const uint32_t own = (uint32_t)__builtin_amdgcn_readlane((int)page, 16 * wave) << a.log_b |
                                 (first + 16 * wave & in_page);
            codes = make_rsrc(a.codes + (uint64_t)own * kLatent, real ? 16 * kLatent : 0);
            rope = make_rsrc(a.rope + (uint64_t)own * kLatentRope, real ? 16 * kLatentRope * 2 : 0);
            scale = a.scales + (page << a.log_b | (first + lane & in_page));
        }
        __device__ __forceinline__ void load(uint8_t* st, int k) const {
            const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
            if (k < 8) {
                // row 2 k + hi of the wave's sixteen; the lane's place in LDS holds this chunk of it
                const int hi = lane >> 5, at = hi * kLatent + (((lane & 31) ^ lat_swz(hi)) << 4);
                buf_lds16(codes, at ^ lat_swz(2 * k) << 4, k * 1024, st + wave * 8192 + k * 1024);
            } else {
                const int row = 8 * (k - 8) + (lane >> 3);
                buf_lds16(rope, row * (kLatentRope * 2) + (((lane & 7) ^ rope_swz(row)) << 4), 0,
                          st + kLatCodes + wave * 2048 + (k - 8) * 1024);
            }
        }
    };
    static constexpr int FETCHES = 10;

    // S^T of 32 tokens: rows of C are widened with their token's scale.  Codes are read four chunks
    // ahead and widened one ahead of the matrix instructions that take them, which would otherwise wait
    // for the conversion; between them, the loads of a tile to come.
    // tokens: exponents and inverses of the scales of this lane's tokens, read when there is room.
    __device__ __forceinline__ v16f logits(const uint8_t* st, int b, float scale, const Fetch& fetch, uint8_t* to,
                                           const float2* scales, v4f (&tokens)[8]) const {
        const int lane = threadIdx.x & 63, h = lane >> 5, row = 32 * b + (lane & 31);
        const uint8_t* const c = st + row * kLatent;
        const uint8_t* const r = st + kLatCodes + row * (kLatentRope * 2);
        const int cs = lat_swz(row & 15), rs = rope_swz(row);
        v16f s;
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = 0.f;
        constexpr int N = 20, AHEAD = 4;                         // reads, those on their way
        uint4 w[N];
        const auto read = [&](int p) {
            return *(const uint4*)(p < 16 ? c + (((2 * p + h) ^ cs) << 4) : r + (((2 * (p - 16) + h) ^ rs) << 4));
        };
#pragma unroll
        for (int p = 0; p < AHEAD; ++p) w[p] = read(p);
        __builtin_amdgcn_sched_barrier(0);
        bf8v lo = widen8((int)w[0].x, (int)w[0].y, scale), hi = widen8((int)w[0].z, (int)w[0].w, scale);
        const auto mfma = [&](bf8v x, int k) __attribute__((always_inline)) {
            __builtin_amdgcn_sched_barrier(0);
            s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, q[k], s, 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        };
#pragma unroll
        for (int p = 0; p < 16; ++p) {
            bf8v next = lo;
            mfma(lo, 2 * p);
            if (p + 1 < 16) next = widen8((int)w[p + 1].x, (int)w[p + 1].y, scale);
            w[p + AHEAD] = read(p + AHEAD);
            mfma(hi, 2 * p + 1);
            if (p + 1 < 16) hi = widen8((int)w[p + 1].z, (int)w[p + 1].w, scale);
            if (p < FETCHES) fetch.load(to, p);
            lo = next;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) tokens[i] = *(const v4f*)(scales + 8 * (i >> 1) + 4 * h + 2 * (i & 1));
#pragma unroll
        for (int k = 0; k < 4; ++k) mfma(__builtin_bit_cast(bf8v, w[16 + k]), 32 + k);
        return s;
    }

    // Logits to exponents of two, with the tokens' scale exponents added; tokens from `seen` on are
    // hidden.  Returns the reference that this wave's next weights need.
    __device__ __forceinline__ float exponents(v16f& s, const v4f (&tokens)[8], float c, int seen, bool masked) const {
        const int h = (threadIdx.x & 63) >> 5;
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = __builtin_fmaf(s[i], c, tokens[i >> 1][2 * (i & 1)]);
        if (masked) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (8 * (i >> 2) + 4 * h + (i & 3) >= seen) s[i] = neg_inf();
        }
        float top[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) top[i] = fmaxf(fmaxf(s[i], s[i + 4]), fmaxf(s[i + 8], s[i + 12]));
        const float x = __builtin_ceilf(half_max(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]))));
        return x - m > kLatTop ? x - kLatRise : m;               // (m + kLatTop may be rounded up)
    }

    // 2^(from - to) for references; 0 where there was none.
    static __device__ __forceinline__ float shrink(float from, float to) {
        return from == neg_inf() ? 0.f : __builtin_amdgcn_exp2f(from - to);
    }

    // Weights against `from` as weights against `to`, in two steps: one fp16 factor ends at 2^-24, where a
    // weight of 2^15 still is 2^-9.
    static __device__ __forceinline__ void lower(h8v& x, h8v& y, float from, float to) {
        const float d = from == neg_inf() ? -64.f : from - to;   // (or all is 0)
        const _Float16 a = (_Float16)__builtin_amdgcn_exp2f(fmaxf(d, -14.f));
        const _Float16 b = (_Float16)__builtin_amdgcn_exp2f(fminf(d + 14.f, 0.f));
        x *= a;
        y *= a;
        if (__any(d < -14.f)) {
            x *= b;
            y *= b;
        }
    }

    // Weights of 32 tokens against the reference m, and their share of the norm.
    __device__ __forceinline__ void weights(const v16f& s, const v4f (&tokens)[8], h8v (&w)[2]) {
        const float ref = m == neg_inf() ? 0.f : m;
        // summed up before they meet l: one by one, weights under its last step would be lost
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float y = __builtin_amdgcn_exp2f(s[i] - ref);
            sum[i & 3] = __builtin_fmaf(y, tokens[i >> 1][2 * (i & 1) + 1], sum[i & 3]);
            w[i >> 3][i & 7] = (_Float16)y;
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    }

    // Codes of a tile as values: read n is of 16 tokens (n / DT) and 32 dims (n % DT), 8 tokens of a dim a
    // lane; reads are AHEAD of their use, and the first ones are asked for before the weights are there.
    struct Codes {
        static constexpr int N = 4 * DT, AHEAD = 6;
        v2i x[N];
        const uint8_t* c;
        int cs;
        __device__ __forceinline__ Codes(const uint8_t* st) {
            const int lane = threadIdx.x & 63, h = lane >> 5, g = lane >> 4 & 1, i = lane >> 1 & 7;
            // this lane's address is that of token T, 8 of 16 dims; it gets 8 tokens of dim lane & 31
            const int T = (i & 3) + 8 * (i >> 2) + 4 * h;
            c = st + T * kLatent + (lane & 1) * 8;
            cs = lat_swz(T) ^ g;
        }
        __device__ __forceinline__ void read(int n, int dw) {
            const int chunk = 2 * (dw * DT + n % DT) ^ cs;
            x[n] = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i)(c + n / DT * 16 * kLatent + (chunk << 4)));
        }
    };

    // O^T += C^T P^T over a tile's tokens, 16 at a time; widened two ahead.
    __device__ __forceinline__ void values(Codes& k, const h8v (&w)[4]) {
        __builtin_amdgcn_sched_barrier(0);
        h8v f = widen8_f16(k.x[0][0], k.x[0][1]), next = widen8_f16(k.x[1][0], k.x[1][1]);
#pragma unroll
        for (int n = 0; n < k.N; ++n) {
            h8v last = next;
            if (n + 2 < k.N) last = widen8_f16(k.x[n + 2][0], k.x[n + 2][1]);
            if (n + k.AHEAD < k.N) k.read(n + k.AHEAD, dw);
            __builtin_amdgcn_sched_barrier(0);
            o[n % DT] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f, w[n / DT], o[n % DT], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
            f = next;
            next = last;
        }
    }

    // Bytes behind the last token may hold anything, and 0 * NaN is NaN.
    __device__ __forceinline__ void clear_tail(uint8_t* st, int base) const {
        if (base <= kv_len - kLatTile) return;
        for (int x = (kv_len - base) * (kLatent / 16) + threadIdx.x; x < kLatCodes / 16; x += kLatThreads)
            *(uint4*)(st + x * 16) = make_uint4(0, 0, 0, 0);
        barrier_written();
    }

    // One tile, which has landed in st.
    __device__ __forceinline__ void work(const LatentLds& lds, int tile, uint8_t* st, float sc, float c,
                                         const Fetch& fetch, uint8_t* to) {
        const int base = tile * kLatTile;
        const int lane = threadIdx.x & 63, pair = (rg * 2 + tg) * 128 + lane, first = rg * 256 + lane;
        clear_tail(st, base);
        // 255: a token that is not finite.  A scale of zero would pass fp32 in the norm: of scales below 2^-90
        // the values, nothing next to any other, count as if it were that.
        const uint32_t ex = max(__float_as_uint(sc) >> 23 & 255, 127u - 90u);
        lds.scales[lane] = make_float2(ex == 255 ? __uint_as_float(0x7FC00000u) : (float)((int)ex - 127),
                                       ex == 255 ? 0.f : __uint_as_float((254 - ex) << 23));
        __builtin_amdgcn_wave_barrier();
        const auto both = __builtin_amdgcn_permlane32_swap(__float_as_uint(sc), __float_as_uint(sc), false, false);
        v4f tokens[8];
        v16f s = logits(st, tg, __uint_as_float(tg == 0 ? both[0] : both[1]), fetch, to, lds.scales + 32 * tg, tokens);
        const float m_new = exponents(s, tokens, c, limit - base - 32 * tg, base > free_limit - kLatTile);
        const float before = m;
        l *= m == m_new ? 1.f : shrink(m, m_new);
        m = m_new;
        h8v w[4];
        {
            h8v mine[2];
            weights(s, tokens, mine);
            if (gives) {
                lds.trade[pair] = __builtin_bit_cast(uint4, mine[0]);
                lds.trade[pair + 64] = __builtin_bit_cast(uint4, mine[1]);
                lds.refs[pair] = m;
            }
        }
        Codes codes(st);
#pragma unroll
        for (int n = 0; n < codes.AHEAD; ++n) codes.read(n, dw);
        barrier_written();
        const float m0 = lds.refs[first], m1 = lds.refs[first + 128];
#pragma unroll
        for (int x = 0; x < 4; ++x) w[x] = __builtin_bit_cast(h8v, lds.trade[first + 64 * x]);
        // the rows' reference is that of O in all waves: the larger of the two
        if (__any(m0 != m1 || m0 != before)) {
            const float top = fmaxf(m0, m1), alpha = shrink(before, top);
            lower(w[0], w[1], m0, top);
            lower(w[2], w[3], m1, top);
#pragma unroll
            for (int d = 0; d < DT; ++d) o[d] *= alpha;
            l *= m == top ? 1.f : shrink(m, top);
            m = top;
        }
        values(codes, w);
    }

    // The rows' norms, over both halves of the tokens (which have one reference).
    __device__ __forceinline__ void join(const LatentLds& lds) {
        l = half_sum(l);
        const int at = rg * 256 + (threadIdx.x & 63);
        if (gives) lds.refs[at + 128 * tg + 64] = l;
        barrier_written();
        l = lds.refs[at + 64] + lds.refs[at + 192];
    }

    // Rows that see nothing.
    __device__ __forceinline__ void nothing() {
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
        m = neg_inf();
        l = 0.f;
    }

    // The rows' results to out and lse.
    __device__ __forceinline__ void store(const LatentArgs& a, const LatentItem& it, int row) const {
        if (row >= it.rows) return;
        const int h = (threadIdx.x & 63) >> 5;
        int j;
        const int64_t t = it.q0 + a.by_heads.of(row, j);
        const float f = l == 0.f ? 0.f : 1.f / l;
        uint16_t* const out = a.out + t * a.o_ts + (int64_t)j * a.o_hs + dw * (32 * DT) + 4 * h;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *(uint2*)(out + 32 * d + 8 * i) =
                    make_uint2(pack_bf16x2(o[d][4 * i] * f, o[d][4 * i + 1] * f),
                               pack_bf16x2(o[d][4 * i + 2] * f, o[d][4 * i + 3] * f));
        if (a.lse && h == 0 && dw == 0)
            a.lse[t * a.heads + j] = l == 0.f ? neg_inf() : (m + __builtin_log2f(l)) * kLn2;
    }

    // Partial results of a slot: [RW][16 dims blocks][4][64 lanes] of four floats, then (m, l) a row.
    __device__ __forceinline__ void store_part(const LatentArgs& a, const LatentJob& u, int64_t slot) const {
        const int lane = fresh_lane();
        if (row(u.rt) >= u.it.rows) return;
        v4f* const ws = (v4f*)a.ws + ((slot * RW + rg) * 16 + dw * DT) * 256 + lane;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                ws[(d * 4 + i) * 64] = v4f{o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
        if (lane < 32 && dw == 0) {
            latent_ml(a, ROWS)[slot * ROWS + rg * 32 + lane] = make_float2(m, l);
        }
    }
};

// A split launch's cost is shared evenly by this many workgroups (no share is empty).
__device__ __forceinline__ int latent_groups(int64_t cost) {
    return (int)min(cost, (int64_t)kLatGroups);
}
// Where workgroup w's share begins, and the workgroup whose share holds position `at`.
__device__ __forceinline__ int64_t latent_first(int64_t cost, int groups, int w) { return quotient(cost * w, groups); }
__device__ __forceinline__ int latent_owner(int64_t cost, int groups, int64_t at) {
    return (int)quotient((at + 1) * groups - 1, cost);
}

// A workgroup's runs, of items whose rows it stores, or whose parts.  While a tile is worked on the
// next is on its way to LDS, and the one after that is asked for.  A run begins with all of its first
// loads at once: its queries, its first tile, whose page the run before asked for; the results of the
// run before are stored while they come.
template <int RW, bool kSplit>
__device__ __forceinline__ void latent_walk(const LatentArgs& a, LatentShare<32 * RW>& share, int64_t cost, int groups,
                                            int row_tiles) {
    using W = LatentWalk<RW>;
    __shared__ __attribute__((aligned(1024))) uint8_t st0[kLatStage];
    __shared__ __attribute__((aligned(1024))) uint8_t st1[kLatStage];
    __shared__ __attribute__((aligned(1024))) uint8_t st2[kLatStage];
    __shared__ __attribute__((aligned(16))) float2 scales[4][kLatTile];
    __shared__ uint4 trade[RW * 256];
    __shared__ float refs[RW * 256];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const LatentLds lds = {scales[wave], trade, refs};
    const float c = a.scale * kLog2e;
    W w;
    w.init();
    LatentJob job = share.job, done;
    int tile = share.tile, end = share.end(), slot = -1;
    bool whole = false;
    int ent0 = w.entry(a, job, tile), ent1 = w.entry(a, job, tile + 1);
    for (;;) {
        w.template stage_q<0>(a, job, st1);
        if constexpr (RW == 2) w.template stage_q<1>(a, job, st2);
        const typename W::Fetch f0(a, tile, ent0, true), f1(a, tile + 1, ent1, tile + 1 < end);
        float sc0 = *f0.scale, sc1 = *f1.scale, sc2 = 0.f;
#pragma unroll
        for (int k = 0; k < W::FETCHES; ++k) f0.load(st0, k);
        int ent2 = w.entry(a, job, tile + 2);
        if (slot >= 0) {                                         // the run before
            if (whole) w.store(a, done.it, w.row(done.rt));
            else w.store_part(a, done, slot);
        }
        barrier_all();
        w.template read_q<0>(st1);
        if constexpr (RW == 2) w.template read_q<1>(st2);
        barrier_written();
#pragma unroll
        for (int k = 0; k < W::FETCHES; ++k) f1.load(st1, k);
        w.begin(a, job, tile);
        whole = !kSplit || (tile == 0 && end == job.tiles);
        slot = (int)blockIdx.x * 2 + (slot < 0 ? 0 : 1);
        if (kSplit && tile == 0 && threadIdx.x == 0)
            latent_info(a, W::ROWS)[job.r * row_tiles + job.rt] =
                make_int2(slot, whole ? 0 : latent_owner(cost, groups, share.at + job.tiles - 1) - (int)blockIdx.x);
        const bool more = kSplit && share.next(a);
        ent0 = w.entry(a, share.job, 0);
        ent1 = w.entry(a, share.job, 1);
        const auto step = [&](uint8_t* st, uint8_t* ahead, float sc, float& sc_ahead) __attribute__((always_inline)) {
            wait_vmcnt<W::FETCHES>();                            // all but the next tile's loads
            barrier_lds();
            __builtin_amdgcn_sched_barrier(0);
            const typename W::Fetch fetch(a, tile + 2, ent2, tile + 2 < end);
            ent2 = w.entry(a, job, tile + 3);
            sc_ahead = *fetch.scale;
            __builtin_amdgcn_sched_barrier(0);
            w.work(lds, tile, st, sc, c, fetch, ahead);
            return ++tile < end;
        };
        while (step(st0, st2, sc0, sc2) && step(st1, st0, sc1, sc0) && step(st2, st1, sc2, sc1)) {
        }
        wait_vmcnt<0>();                                         // no load outlives its use of LDS
        w.join(lds);                                             // and all waves are done with their stages
        done = job;
        if (!more) break;
        job = share.job;
        tile = 0;
        end = share.end();
    }
    if (whole) w.store(a, done.it, w.row(done.rt));
    else w.store_part(a, done, slot);
}

// Every workgroup takes an even share of the cost of all items, in their order.  Where it begins an
// item it notes for the join where the item's parts are: its own slot (of the two that a workgroup has:
// its first run's and its last one's) and how many workgroups follow.
template <int RW>
__global__ __launch_bounds__(kLatThreads, 1) void attn_latent_split_kernel(LatentArgs a, int row_tiles) {
    const int lane = threadIdx.x & 63;
    LatentShare<32 * RW> share;
    auto& reqs = share.reqs;
    int64_t cost = 0;
    for (int from = 0; from < a.R; from += 64) {
        reqs.load(a, from);
        cost = reqs.scan(cost);
    }
    const int groups = latent_groups(cost);
    if ((int)blockIdx.x >= groups || cost == 0) return;
    const int64_t from = latent_first(cost, groups, blockIdx.x), to = latent_first(cost, groups, blockIdx.x + 1);
    if (a.R > 64) {                                              // back to the requests where it begins
        int64_t next = 0;
        for (int x = 0; x < a.R && next <= from; x += 64) {
            reqs.load(a, x);
            next = reqs.scan(next);
        }
    }
    const int in = last_of(reqs.base + lane < a.R && reqs.before <= from);
    if (share.begin(a, __builtin_amdgcn_readfirstlane(reqs.base + in), from, to))
        latent_walk<RW, true>(a, share, cost, groups, row_tiles);
}

// One workgroup per item: enough of them to fill the chip, or no workspace.  Request r's items are
// numbered from q_offsets[r] * heads / ROWS + r on, where there is room for all of them.
template <int RW>
__global__ __launch_bounds__(kLatThreads, 1) void attn_latent_item_kernel(LatentArgs a) {
    using W = LatentWalk<RW>;
    const int lane = threadIdx.x & 63;
    const int64_t b = blockIdx.x;
    const auto start = [&](int q, int r) {
        return min(max((int64_t)q, (int64_t)0), a.T) * a.heads / W::ROWS + r;
    };
    const int each64 = a.q_offsets[min(lane * 64, a.R)];
    const int from = last_of(lane * 64 < a.R && start(each64, lane * 64) <= b) * 64;
    LatentShare<W::ROWS> share;
    share.reqs.load(a, from);
    const int r = __builtin_amdgcn_readfirstlane(from + last_of(from + lane < a.R && start(share.reqs.q0, from + lane) <= b));
    const LatentItem it = share.reqs.item(a, r);
    const int64_t at = b - start((int)it.q0, r);
    if (at < 0 || at * W::ROWS >= it.rows) return;
    const int rt = __builtin_amdgcn_readfirstlane((int)at);
    const int last = min((rt + 1) * W::ROWS, it.rows) - 1;
    const int tiles = latent_tiles(it.limit(a.by_heads.of(last)));         // that its rows see
    if (tiles == 0) {
        W w;
        w.init();
        w.nothing();
        w.store(a, it, w.row(rt));
        return;
    }
    share.job = {r, rt, tiles, it};
    share.tile = 0;
    share.at = 0;
    share.to = tiles;
    latent_walk<RW, false>(a, share, 0, 0, 0);
}
static_assert(kKvMaxRequests <= 64 * 64, "a request is found in two steps of 64");

// Adds the parts of items that several workgroups shared, and gives the rows of a request without
// tokens their zeros.  A workgroup takes 32 rows x 32 dims; each of its WAVES waves takes every
// WAVES-th part, in token order, then the waves' sums are added in order.
template <int RW, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void attn_latent_join_kernel(LatentArgs a, int row_tiles) {
    constexpr int ROWS = 32 * RW;
    __shared__ v4f sums[WAVES][4][64];
    __shared__ float2 stats[WAVES][32];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, d = blockIdx.y;
    const int rg = blockIdx.x % RW, item = blockIdx.x / RW;
    const int r = item / row_tiles, rt = item % row_tiles;
    const int2 info = latent_info(a, ROWS)[item];                // of no meaning where there are no tokens
    const LatentItem it = LatentItem::of(a, a.q_offsets[r], a.q_offsets[r + 1], a.kv_lens[r]);
    if (rt * ROWS + rg * 32 >= it.rows) return;
    v4f o[4] = {};
    float m = neg_inf(), l = 0.f;
    if (it.kv_len > 0 && info.y == 0) return;                    // finished by its workgroup
    if (it.kv_len > 0 && rt * ROWS + rg * 32 + (lane & 31) < it.rows) {
        const v4f* const ws = (const v4f*)a.ws + (rg * 16 + d) * 256 + lane;
        const float2* const ml = latent_ml(a, ROWS) + rg * 32 + (lane & 31);
#pragma unroll 2
        for (int g = wave; g <= info.y; g += WAVES) {
            const int64_t slot = g == 0 ? info.x : (info.x / 2 + g) * 2;
            const float2 part = ml[slot * ROWS];
            v4f x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = ws[slot * (RW * 16 * 256) + i * 64];
            const float top = fmaxf(m, part.x);
            const float old = m == neg_inf() ? 0.f : __builtin_amdgcn_exp2f(m - top);
            const float add = part.x == neg_inf() ? 0.f : __builtin_amdgcn_exp2f(part.x - top);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = o[i] * old + x[i] * add;
            l = l * old + part.y * add;
            m = top;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[wave][i][lane] = o[i];
    if (lane < 32) stats[wave][lane] = make_float2(m, l);
    __syncthreads();
    if (wave >= 4) return;
    const int i = wave, row = rt * ROWS + rg * 32 + (lane & 31);
    if (row >= it.rows) return;
    float2 part[WAVES];
    m = neg_inf();
#pragma unroll
    for (int z = 0; z < WAVES; ++z) {
        part[z] = stats[z][lane & 31];
        m = fmaxf(m, part[z].x);
    }
    v4f sum = {0.f, 0.f, 0.f, 0.f};
    l = 0.f;
#pragma unroll
    for (int z = 0; z < WAVES; ++z) {
        const float f = part[z].x == neg_inf() ? 0.f : __builtin_amdgcn_exp2f(part[z].x - m);
        sum += sums[z][i][lane] * f;
        l += part[z].y * f;
    }
    int j;
    const int64_t t = it.q0 + a.by_heads.of(row, j);
    const float f = l == 0.f ? 0.f : 1.f / l;
    *(uint2*)(a.out + t * a.o_ts + (int64_t)j * a.o_hs + 32 * d + 8 * i + 4 * (lane >> 5)) =
        make_uint2(pack_bf16x2(sum[0] * f, sum[1] * f), pack_bf16x2(sum[2] * f, sum[3] * f));
    if (a.lse && d == 0 && i == 0 && lane < 32)
        a.lse[t * a.heads + j] = l == 0.f ? neg_inf() : (m + __builtin_log2f(l)) * kLn2;
}

// How a launch divides its rows: the 32-row groups of a workgroup, and the row tiles of a request.  With
// one group where a request's rows are no more (64 requests of 16 heads: 39 us, and 47 with two), with two
// otherwise (128 heads: 84 us, and 117 with one; only where the tokens are few, too, one is ahead: 24
// requests of 60 rows over 100 to 6000 tokens 24 us, and 26 with two).
struct LatentPlan {
    int rw;
    int64_t row_tiles;
    bool split;
};
static LatentPlan latent_plan(int64_t R, int64_t max_new, int32_t heads) {
    const int64_t rows = max_new * heads;
    LatentPlan p;
    p.rw = rows <= 32 ? 1 : 2;
    p.row_tiles = (rows + 32 * p.rw - 1) / (32 * p.rw);
    p.split = R * p.row_tiles < kLatItems;
    return p;
}

size_t attn_latent_workspace_bytes(int64_t R, int64_t max_new, int32_t heads) {
    const LatentPlan p = latent_plan(R, max_new, heads);
    if (!p.split) return 0;
    return (size_t)kLatSlots * 32 * p.rw * (kLatent + 2) * sizeof(float) + (size_t)kLatItems * sizeof(int2);
}

template <int RW>
static hipError_t latent_launch(const LatentArgs& a, const LatentPlan& p, hipStream_t stream) {
    const int rt = (int)p.row_tiles;
    if (!p.split || !a.ws) {
        const int64_t items = a.T * a.heads / (32 * RW) + a.R;
        attn_latent_item_kernel<RW><<<dim3((unsigned)items), dim3(kLatThreads), 0, stream>>>(a);
        return hipGetLastError();
    }
    attn_latent_split_kernel<RW><<<dim3(kLatGroups), dim3(kLatThreads), 0, stream>>>(a, rt);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t joins = a.R * p.row_tiles * RW;
    // with few items of many parts, eight waves (two long requests of 128 heads 63.8 -> 62.3 us, 24 drafts
    // 27.0 -> 26.4); with many of few, four (64 requests of 128 heads 75.9 us, and 79.0 with eight)
    if (joins < 64)
        attn_latent_join_kernel<RW, 8><<<dim3((unsigned)joins, 16), dim3(512), 0, stream>>>(a, rt);
    else
        attn_latent_join_kernel<RW, 4><<<dim3((unsigned)joins, 16), dim3(256), 0, stream>>>(a, rt);
    return hipGetLastError();
}

hipError_t launch_attn_latent(LatentArgs a, hipStream_t stream) {
    LatentPlan p = latent_plan(a.R, a.max_new, a.heads);
    // costs that quotient() takes: a split launch's are below 2^31
    const int64_t tiles = ((a.width << a.log_b) + kLatTile - 1) / kLatTile;
    p.split = p.split && a.R * p.row_tiles * (tiles + kLatItemCost) < (int64_t)1 << 31;
    // sixteen rows of queries, in memory, span at most so many tokens
    const auto near = [&](int64_t ts, int64_t hs) {
        return ts < (1 << 26) && hs < ((int64_t)1 << 30) / a.heads && (ts | hs) % 8 == 0;
    };
    a.q_near = ((uintptr_t)a.q_latent | (uintptr_t)a.q_rope) % 16 == 0 && near(a.ql_ts, a.ql_hs) && near(a.qr_ts, a.qr_hs);
    if (p.rw == 1) return latent_launch<1>(a, p, stream);
    return latent_launch<2>(a, p, stream);
}

}  // namespace bfp8
