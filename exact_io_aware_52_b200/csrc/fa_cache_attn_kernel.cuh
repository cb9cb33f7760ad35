// fa_cache_attn_kernel.cuh -- attention of a few query tokens for each
// sequence over the paged 8-bit cache (fa_cache_attn), and the merge of its
// parts.
//
// Mathematics.  With k = ks * k', v = vs * v' (codes times the scale of their
// page), x_j = q . k'_j * ks * scale * log2(e):
//     O = sum_j 2^x_j vs_j v'_j / sum_j 2^x_j,   lse = ln 2 * log2(sum_j 2^x_j)
// in one pass over the keys.  Two references per row, raised only when a
// value lies more than 2^8 above them: m for l = sum_j 2^(x_j - m), and n for
// acc = sum_j 2^(x_j + log2(vs_j) - n + 7) v'_j.  The second keeps the weights of
// the product with the codes inside fp16 whatever the pages' scales are (largest
// 2^15, and 2^-24 the step of the smallest: a weight errs by 2^-25 too, where the largest is
// 2^7 or more, that is by 2^-32 of it); O = acc * 2^(n - m - 7) / l.
//
// Tiles.  A warp takes 16 tokens of one key/value head at a time.  S^T = K Q^T and
// O^T = V^T P^T are computed transposed (tokens or components
// on the 16 side, query rows on the 8 side), so that the 4 to 8 query rows
// that share a key fill the tensor core's narrow side and the codes are the
// A operand.  (tcgen05 could have 128 tokens or components on its large side in the same way, with the query rows as
// its narrow one.  It takes its operands from shared or tensor memory, so that the codes of 128 tokens, 8 boxes of 16, would
// have to be written there as fp16 first.  Up to 8 rows the reads bound the kernel as it is; for more the form is untried.)
// Both run on fp16 (mma m16n8k16), to which the codes convert exactly.  (The E4M3 form of
// mma, with the queries in two parts, took more instructions: 408 for each tile of d = 128 against 334.)
// Every warp works by itself: it has a ring of tiles that TMA fills (one lane issues),
// with an mbarrier for each, and no barrier is shared between warps.  Which token
// or component a row of a matrix stands for is free; it is chosen such that a
// lane reads its operands from the 128-byte-swizzled tile as whole 16-byte runs (8 for
// the values of d = 64) without bank conflicts: row r of K is token tau(r) (8 + tau(r - 8)).
//
// Bound by memory: 2 d bytes per token and key/value head, read once for all
// query rows that share it.  The same tiles fetched by 16-byte cp.async (64 bytes
// of a key for each group of 4 lanes) stopped at 4.8 TB/s whatever was done with
// them; TMA's requests reach the copy rate.  Measured, 32 query heads on 8 of d = 128, one token each: 64 ragged
// sequences of up to 8192 tokens (547 MB) 96 us, 8 of 16384 to 131072 (1451 MB) 235 us or 6.2 TB/s, one of
// 500 tokens 6.7 us.  About 8 us of the split form are its start (lengths, plan, page table, first tiles) and
// the merge.  With 16 rows for each key (96 us for 394 MB) and at d = 64 (49 us for 198 MB, 8 rows) neither memory nor a
// pipe is full: the instructions of a tile (conversions, scores and weights, 235 at d = 64) wait for one
// another, and 12 to 16 warps an SM fill 38 to 47 % of the issue slots.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "fa.h"
#include "fa_cache_kernels.cuh"

namespace fa {
namespace cattn {

constexpr int kWarps = 4;         // of a CTA when the keys are split
// Of a CTA that takes a whole pair: as many as its registers and rings allow, since one warp for
// each scheduler takes 0.9 us for a tile, which more warps hide.
template <int D, int NT> constexpr int kDirectWarps = D <= 128 && NT < 2 ? 16 : 8;
constexpr int kTile = 16;         // tokens a warp takes at a time; divides every page size
constexpr int kMaxWorkers = 2560;  // warps that take work, at most
// What a warp spends on a (sequence, head) pair besides its tiles (the table, the queries, the
// first copies, the result), in tiles.
constexpr int kPairCost = 6;
constexpr int kMinRun = 4;        // of one worker, in tiles

// Tiles of one step (two: their chains of products and the softmax's reductions overlap)
// and of the ring.
template <int D> constexpr int kStep = D == 64 ? 2 : 1;
template <int D> constexpr int kStages = D == 64 ? 4 : 3;
// CTAs for each SM.  More tiles in flight are not better: d = 128 with one CTA more or a tile
// more in the ring took 5 to 15 % longer.
template <int D, int NT> constexpr int kResident = D == 64 ? (NT == 2 ? 3 : 4) : (D == 128 ? 3 : 2);
template <int D> constexpr int kStageBytes = 2 * kTile * D;  // codes of K and V
template <int D> constexpr int kRingBytes = kStages<D> * kStageBytes<D>;
// 16 rows of d = 128 leave too few registers for the queries: they are read from shared memory for each tile.
template <int D, int NT> constexpr int kQueryBytes = D == 128 && NT == 2 ? NT * (D / 16) * 256 : 0;
template <int D, int NT> constexpr int kWarpBytes = kRingBytes<D> + kQueryBytes<D, NT>;
template <int D, int NT, int WARPS>
constexpr int kSmemBytes = WARPS * kWarpBytes<D, NT> + 1024;  // the rings begin on a swizzle atom
// tau(r) in four bits for each of 8 rows r: found by trying the orders for one in which neither the
// lanes' reads of K (16 bytes) nor those of V (16, or 8 for d = 64) meet in a bank.  d = 64 has two
// tokens in a 128-byte line, d = 256 half a token.
template <int D> constexpr uint32_t kTau = D == 64 ? 0x65217430u : 0x37621540u;
template <int D>
__device__ __forceinline__ int tau(int r) { return (kTau<D> >> (4 * r)) & 7; }
// Byte b of a tile of 128-byte lines under the 128-byte swizzle.
__device__ __forceinline__ uint32_t swizzled(uint32_t b) { return b ^ (((b >> 7) & 7) << 4); }
// Query rows that one warp handles: 8 NT, or 4 for NT = 0.
__host__ __device__ constexpr int rows_of(int nt) { return nt ? 8 * nt : 4; }

struct Params {
    CUtensorMap tm_k, tm_v;  // codes as [tiles][16 d / line][line], line = 128 bytes (256 for d = 256), swizzled
    CacheView c;
    const uint16_t *q;
    void *o;
    float *lse;
    const int32_t *k_len;
    int32_t *status;
    float *o_part;        // [chunk][worker][2][rows][D]
    float2 *ml_part;      // [chunk][worker][2][rows] (m, l)
    int N, rows;          // query tokens; rows that share a key/value head: group * N
    int chunks, workers;  // blocks of rows; warps for each of them
    int cluster;          // CTAs for each pair (direct)
    int causal, o_bf16;
    float scale_log2;
    uint64_t timeout_ns;
    int drop_load;        // test: the first warp never issues its n-th tile
};

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

__device__ __forceinline__ int seq_len(const Params &p, int b) {
    const long long cap = (long long)p.c.max_pages << p.c.page_log2;
    const int n = max(__ldg(p.k_len + b), 0);
    return (int)min((long long)n, cap);
}
__device__ __forceinline__ int seq_tiles(const Params &p, int b) { return (seq_len(p, b) + kTile - 1) / kTile; }

// All threads of a cluster's CTAs; what they wrote to shared memory before is visible to the others after.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// Two floats of CTA `rank` of the cluster, at the place of this CTA's shared-memory address.
__device__ __forceinline__ float2 peer_float2(uint32_t addr, int rank) {
    float2 r;
    asm volatile("{\n\t.reg .b32 a;\n\t"
                 "mapa.shared::cluster.u32 a, %2, %3;\n\t"
                 "ld.shared::cluster.v2.f32 {%0, %1}, [a];\n\t}"
                 : "=f"(r.x), "=f"(r.y)
                 : "r"(addr), "r"(rank)
                 : "memory");
    return r;
}

// What turns acc into O, 2^(n - m - 7) / sum, as two factors, each near its square root: for value scales far
// below 1 the whole is below the normal fp32 values, which ex2.approx.ftz makes 0, although O is not.
__device__ __forceinline__ float2 out_factor(float m, float n, float sum) {
    if (sum == 0.f) return make_float2(0.f, 0.f);
    const float half = ex2_approx(0.5f * (n - m - 7.f));
    return make_float2(half / sum, half);
}

__device__ __forceinline__ float row_lse(float m, float l) {
    return l == 0.f ? neg_inf() : ((m == neg_inf() ? 0.f : m) + log2f(l)) * 0.693147180559945f;
}

__device__ __forceinline__ void store_out(const Params &p, long long at, float4 o) {
    if (p.o_bf16)
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.o) + at) = make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
    else
        *reinterpret_cast<float4 *>(static_cast<float *>(p.o) + at) = o;
}

// The plan: all (sequence, key/value head) pairs with tiles, in that order, lie on a line,
// each kPairCost + its tiles long, and the line is cut into runs of `per`, one
// for each worker (kMinRun at least).  Its length is below 2^31.
__device__ __forceinline__ int pair_cost(int tiles) { return tiles ? tiles + kPairCost : 0; }

// Lanes' lengths on the line of sequences b0 .. b0 + 31, and their running sum.
__device__ __forceinline__ void scan_costs(const Params &p, int b0, int &own, int &sum) {
    const int lane = threadIdx.x & 31;
    own = b0 + lane < p.c.B ? pair_cost(seq_tiles(p, b0 + lane)) * p.c.H_kv : 0;
    sum = own;
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, sum, i);
        if (lane >= i) sum += o;
    }
}

struct Plan {
    int total, per;
    int own, sum;  // scan_costs of the first 32 sequences
};
__device__ __forceinline__ Plan make_plan(const Params &p) {
    Plan r;
    scan_costs(p, 0, r.own, r.sum);
    r.total = __shfl_sync(0xffffffffu, r.sum, 31);
    for (int b0 = 32; b0 < p.c.B; b0 += 32) {
        const int b = b0 + (threadIdx.x & 31);
        const int own = b < p.c.B ? pair_cost(seq_tiles(p, b)) * p.c.H_kv : 0;
        r.total += __reduce_add_sync(0xffffffffu, own);
    }
    r.per = max((int)(((unsigned)r.total + p.workers - 1) / (unsigned)p.workers), kMinRun);
    return r;
}

// The sequence that holds place x < total of the line, and where it begins.
__device__ __forceinline__ void locate(const Params &p, const Plan &plan, int x, int &b, int &first) {
    int before = 0, own = plan.own, sum = plan.sum;
    first = 0;
    for (b = 0;; b += 32) {
        const unsigned hit = __ballot_sync(0xffffffffu, before + sum > x);
        if (hit) {
            const int l = __ffs(hit) - 1;
            b += l;
            first = before + __shfl_sync(0xffffffffu, sum - own, l);
            return;
        }
        before += __shfl_sync(0xffffffffu, sum, 31);
        scan_costs(p, b + 32, own, sum);
        if (b + 32 >= p.c.B) return;  // (x < total: not reached)
    }
}

// tma_load_3d with the destination as a shared-memory address.
__device__ __forceinline__ void tma_load_3d_at(uint32_t dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1,
                                               int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 r;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
    return r;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
    uint2 r;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
    return r;
}

// The four E4M3 codes of a word as two fp16 pairs (exact).
__device__ __forceinline__ void half4(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed8x8(uint32_t a) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}

// A value's first 11 bits, which fp16 holds (from 2^-14 on).
__device__ __forceinline__ float upper11(float x) { return __uint_as_float(__float_as_uint(x) & 0xffffe000u); }

// The sums of the weights' two parts, of the even and the odd columns.
template <int D>
__device__ __forceinline__ void join_halves(float (&acc)[D / 16][4]) {
#pragma unroll
    for (int d = 0; d < D / 16; ++d) acc[d][0] += acc[d][1], acc[d][2] += acc[d][3];
}

// Words of V codes of one lane: [token][word], tokens tau(2c), tau(2c + 1) of the tile and those 8 further on.
template <int D> using VWords = uint32_t[4][D / 32];

// The A operands of word w: matrix tile 2 w + i has the components 4 w + 2 i
// (rows 0..7) and 4 w + 2 i + 1 (rows 8..15) of each lane's run.
template <int D>
__device__ __forceinline__ void v_operands(uint32_t (&a)[2][4], const VWords<D> &v, int w) {
    half4(__byte_perm(v[0][w], v[1][w], 0x5140), a[0][0], a[0][1]);
    half4(__byte_perm(v[0][w], v[1][w], 0x7362), a[1][0], a[1][1]);
    half4(__byte_perm(v[2][w], v[3][w], 0x5140), a[0][2], a[0][3]);
    half4(__byte_perm(v[2][w], v[3][w], 0x7362), a[1][2], a[1][3]);
}

__device__ __forceinline__ bool has_nan_code(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

// Split (WARPS = kWarps): one warp takes a run of the line, pair by pair.
// Direct (kDirectWarps): a cluster of CTAs takes one pair, its warps parts of the pair's
// tiles, which are merged in shared memory, the CTA's first and then the cluster's: one launch and
// no partial results in memory, for lengths at which that counts.
//
// A weight is fp32 until its product with the codes, which takes fp16.  FINE: it goes there as the sum of two
// fp16 numbers, its first 11 bits and the rest, so that O keeps fp32's precision (2^-20 of a weight instead of 2^-11).
// Up to 4 rows that costs nothing (the rests are the columns that are empty otherwise) and is always so.  With more rows the
// rests have products of their own, for fp32 outputs only: a bf16 output is itself off by 8 times 2^-11.
// Measured, fp32 outputs with and without, us: 16 rows of d = 128 105 / 96 and of d = 64 76 / 70, 8 rows of d = 64 52 / 49,
// of d = 128 78 / 80 and of d = 256 92 / 87, 56 rows of d = 128 326 / 286.
template <int D, int NT, int WARPS, bool FINE>
__global__ void __launch_bounds__(32 * WARPS, WARPS == kWarps ? kResident<D, NT> : 1)
fa_cache_attn_kernel(const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) uint64_t s_bar[WARPS][kStages<D>];
    __shared__ int s_abort[WARPS];
    constexpr bool DIRECT = WARPS != kWarps;
    constexpr int KJ = D / 64;               // 16-byte runs of a key for each lane
    constexpr int T = kStep<D>, S = kStages<D>;
    // NT = 0: at most 4 rows, in the products' even columns: one for each lane of a group of 4, so that the
    // softmax has no idle half.  Else 8 NT rows, two for each lane of a group and product.
    constexpr int CH = T == 1 ? 2 : 1;       // sums that a tile's scores are split into
    constexpr bool PACK = NT == 0, TWICE = FINE && !PACK, QS = kQueryBytes<D, NT> > 0;
    constexpr int G = PACK ? 1 : NT, RL = PACK ? 1 : 2, R = rows_of(NT);
    static_assert(S % T == 0 && 32 % T == 0, "steps do not straddle the ring's end or a window's");

    if (!DIRECT) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        prefetch_tensormap(&p.tm_k);
        prefetch_tensormap(&p.tm_v);
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    // split: neighbours on the line are on different SMs, so that few workers still use them all
    const int rank = DIRECT ? blockIdx.x % p.cluster : 0;  // of a cluster's CTAs
    const int id = DIRECT ? blockIdx.x / p.cluster : warp * gridDim.x + blockIdx.x;
    if (!DIRECT && id >= p.chunks * p.workers) return;
    const int chunk = id % p.chunks, worker = id / p.chunks;
    const int row0 = chunk * R;
    int per = 0, at = 0, end = 0, b = 0, first = 0;
    if constexpr (!DIRECT) {
        const Plan plan = make_plan(p);
        per = plan.per;
        if ((long long)worker * per >= plan.total) return;
        at = worker * per;
        end = at + min(plan.total - at, per);
        locate(p, plan, at, b, first);
    }

    const uint32_t ring = ((smem_u32(smem_raw) + 1023) & ~1023u) + warp * kWarpBytes<D, NT>;
    const uint32_t q_at = ring + kRingBytes<D> + 8 * lane;  // QS: [row block][step][lane] operands
    uint64_t *bar = s_bar[warp];
    if (lane == 0) {
        for (int i = 0; i < S; ++i) mbar_init(&bar[i], 1);
        fence_mbar_init();
        s_abort[warp] = 0;
    }
    __syncwarp();
    const CacheView &cv = p.c;
    // This lane's places in a tile: its first run of key tau(g), and its run of the values tau(2c) and
    // tau(2c + 1).  8 tokens further on are 8 lines (d = 64: 4 lines, which flips a bit of the swizzle).
    const uint32_t k_at = ring + swizzled(tau<D>(g) * (D == 64 ? 64 : 128) + 16 * c);
    const uint32_t v_at0 = ring + kTile * D + swizzled(tau<D>(2 * c) * (D == 64 ? 64 : 128) + (D == 64 ? 8 : 16) * g);
    const uint32_t v_at1 = ring + kTile * D + swizzled(tau<D>(2 * c + 1) * (D == 64 ? 64 : 128) + (D == 64 ? 8 : 16) * g);
    const int tile_shift = cv.page_log2 - 4;
    int slot0 = 0;        // slot of the next step's first tile, and the parity of its phase
    uint32_t parity = 0;

    // The pair at hand: its first row of q, o and lse, its tokens, its page table, and the tiles
    // t0 .. t0 + n_own of its nb that are this warp's.
    long long q_row = 0;
    const int32_t *table = nullptr;
    int len = 0, nb = 0, h = 0, t0 = 0, n_own = 0, n_pad = 0;
    // windows of 32 own tiles: lane i has tile i's place in the pool (in tiles) and scales;
    // the copies run ahead of the products, so the window before is kept
    int w_tile = -1;
    float w_ks = -1.f, w_lv = 0.f, w_ks_old = -1.f, w_lv_old = 0.f;
    auto window = [&](int i) {
        w_ks_old = w_ks;
        w_lv_old = w_lv;
        w_tile = -1;
        w_ks = -1.f;  // marks a page outside the pool
        w_lv = 0.f;
        if (i + lane < n_own) {
            const int t = t0 + i + lane;
            const int page_id = __ldg(table + (t >> tile_shift));
            if (page_id >= 0 && page_id < cv.n_pages) {
                const int unit = page_id * cv.H_kv + h;
                w_tile = (unit << tile_shift) + (t & ((1 << tile_shift) - 1));
                w_ks = cv.k_scale[unit];
                w_lv = __log2f(cv.v_scale[unit]);
            } else {
                report_bad_page(p.status);
            }
        }
    };
    // Copies of own tile i into the slot at `st`.  A page outside the pool, and the place of a
    // missing second tile of the last step, have nothing to copy: their phase
    // completes all the same.
    auto load = [&](int i, int slot) {
        const int tile = __shfl_sync(0xffffffffu, w_tile, i & 31);
        if (lane == 0) {
            const uint32_t dst = ring + slot * kStageBytes<D>;
            if (tile < 0) {
                mbar_arrive(&bar[slot]);
            } else if (p.drop_load <= 0 || i != p.drop_load - 1 || id != 0 || (DIRECT && warp + rank != 0)) {
                mbar_arrive_expect_tx(&bar[slot], kStageBytes<D>);
                tma_load_3d_at(dst, &p.tm_k, &bar[slot], 0, 0, tile);
                if constexpr (D == 256) tma_load_3d_at(dst + kTile * 128, &p.tm_k, &bar[slot], 128, 0, tile);
                tma_load_3d_at(dst + kTile * D, &p.tm_v, &bar[slot], 0, 0, tile);
                if constexpr (D == 256) tma_load_3d_at(dst + kTile * (D + 128), &p.tm_v, &bar[slot], 128, 0, tile);
            }
        }
    };
    auto begin_pair = [&]() {
        n_pad = (n_own + T - 1) / T * T;
        q_row = ((long long)b * cv.H_kv + h) * p.rows + row0;
        table = cv.table + b * cv.table_stride;
        window(0);
#pragma unroll
        for (int i = 0; i < S; ++i)
            if (i < n_pad) load(i, slot0 + i < S ? slot0 + i : slot0 + i - S);
    };
    // Takes the next pair of the run and starts its copies; false at the run's end.
    auto next_pair = [&]() -> bool {
        while (at < end) {
            len = seq_len(p, b);
            nb = (len + kTile - 1) / kTile;
            const int cost = pair_cost(nb);
            if (at - first >= cost * cv.H_kv) {  // next sequence (this one may be empty)
                first += cost * cv.H_kv;
                ++b;
                continue;
            }
            h = (at - first) / cost;
            const int from = at - first - h * cost;
            const int to = min(cost, from + (end - at));
            at += to - from;
            t0 = max(from - kPairCost, 0);
            n_own = max(to - kPairCost, 0) - t0;
            if (n_own > 0) break;  // else the run has none of the pair's tiles, only its begin
        }
        if (n_own <= 0) return false;
        begin_pair();
        return true;
    };

    bool more = true;
    if constexpr (DIRECT) {
        b = worker / cv.H_kv;
        h = worker - b * cv.H_kv;
        len = seq_len(p, b);
        nb = (len + kTile - 1) / kTile;
        const int part = rank * WARPS + warp, parts = p.cluster * WARPS;
        t0 = (nb * part + parts - 1) / parts;  // a few tiles for each of up to 128 warps: no overflow
        n_own = (nb * (part + 1) + parts - 1) / parts - t0;
        begin_pair();
    } else {
        more = next_pair();
    }
    while (more) {
        // ---- queries: fp16 of each row times a power of two that brings its largest magnitude
        // to [2^14, 2^15); bf16's 8 bits stay exact but for components 2^-28 below the row's largest
        uint32_t qf[QS ? 1 : G][QS ? 1 : D / 16][2];
        float rs[G][RL];   // of this lane's rows: scale * log2(e) / that power
        int lim[G][RL];    // and their number of keys
#pragma unroll
        for (int t = 0; t < G; ++t) {
            const int r = PACK ? g >> 1 : 8 * t + g;
            const bool live = row0 + r < p.rows && !(PACK && (g & 1));  // PACK: odd columns are zero
            const uint16_t *q = p.q + (q_row + r) * D + 16 * c;
            uint32_t raw[KJ][8];
            uint32_t mag = 0;
#pragma unroll
            for (int j = 0; j < KJ; ++j) {
                uint4 x = make_uint4(0, 0, 0, 0), y = x;
                if (live) {
                    x = __ldg(reinterpret_cast<const uint4 *>(q + 64 * j));
                    y = __ldg(reinterpret_cast<const uint4 *>(q + 64 * j) + 1);
                }
                const uint32_t z[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    raw[j][i] = z[i];
                    const uint32_t lo = z[i] & 0x7fffu, hi = (z[i] >> 16) & 0x7fffu;
                    if (lo < 0x7f80u) mag = max(mag, lo);
                    if (hi < 0x7f80u) mag = max(mag, hi);
                }
            }
            mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 1));
            mag = max(mag, __shfl_xor_sync(0xffffffffu, mag, 2));
            // 2^126 at most: a row of subnormal values stays below 2^14
            const int e = min(max(14 - ((int)(mag >> 7) - 127), -126), 126);
            const float up = __uint_as_float((uint32_t)(e + 127) << 23);
#pragma unroll
            for (int j = 0; j < KJ; ++j)
#pragma unroll
                for (int w = 0; w < 4; ++w)
                {
                    const uint32_t z0 = raw[j][2 * w], z1 = raw[j][2 * w + 1];
                    const uint32_t a = pack_half2(bf16x2_lo(z0) * up, bf16x2_hi(z0) * up);
                    const uint32_t b2 = pack_half2(bf16x2_lo(z1) * up, bf16x2_hi(z1) * up);
                    if constexpr (QS) {  // read by this lane alone
                        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(q_at + (t * (D / 16) + 4 * j + w) * 256),
                                     "r"(a), "r"(b2)
                                     : "memory");
                    } else {
                        qf[t][4 * j + w][0] = a;
                        qf[t][4 * j + w][1] = b2;
                    }
                }
            const float f = __uint_as_float((uint32_t)(127 - e) << 23) * p.scale_log2;
#pragma unroll
            for (int i = 0; i < RL; ++i) {
                rs[t][i] = __shfl_sync(0xffffffffu, f, 8 * c + 4 * i);
                const int row = row0 + (PACK ? c : 8 * t + 2 * c + i);
                lim[t][i] = p.causal ? len - p.N + row % p.N + 1 : len;
            }
        }
        const int all = p.causal ? len - p.N + 1 : len;  // keys that every row sees

        float acc[G][D / 16][4];
        float m[G][RL], n[G][RL], l[G][RL];
        float m0[G][RL], n0[G][RL];  // what is added to a score: -m, and 7 - n (0 and 7 while nothing is seen)
#pragma unroll
        for (int t = 0; t < G; ++t) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i) acc[t][i][0] = acc[t][i][1] = acc[t][i][2] = acc[t][i][3] = 0.f;
#pragma unroll
            for (int i = 0; i < RL; ++i) {
                m[t][i] = n[t][i] = neg_inf();
                l[t][i] = m0[t][i] = 0.f;
                n0[t][i] = 7.f;
            }
        }

        bool failed = false;
        for (int i = 0; i < n_own; i += T) {
#pragma unroll
            for (int u = 0; u < T; ++u)
                if (!failed && !mbar_wait(&bar[slot0 + u], parity, &s_abort[warp], p.timeout_ns)) failed = true;
            failed = __any_sync(0xffffffffu, failed);
            if (failed) {
                // The copies in flight end (or their waits run out) before the ring is used otherwise.
                for (int k = i; k < min(i + S, n_pad); ++k) {
                    const int at_k = slot0 + (k - i);
                    const uint64_t since = globaltimer_ns();
                    while (!mbar_try_wait(smem_u32(&bar[at_k % S]), parity ^ (at_k >= S)) &&
                           globaltimer_ns() - since < p.timeout_ns) {
                    }
                }
                if (lane == 0 && p.status) atomicCAS(p.status, 0, (int)FA_ERR_DEVICE_TIMEOUT);
                break;
            }
            const uint32_t st = slot0 * kStageBytes<D>;
            // the copies have reached tile i + S - 1: its window is the current one
            const bool old = (min(i + S, n_pad) - 1) >> 5 != i >> 5;
            float ks[T], lv[T];
            bool bad[T], edge[T];
            int tok0[T];
#pragma unroll
            for (int u = 0; u < T; ++u) {
                ks[u] = __shfl_sync(0xffffffffu, old ? w_ks_old : w_ks, (i + u) & 31);
                lv[u] = __shfl_sync(0xffffffffu, old ? w_lv_old : w_lv, (i + u) & 31);
                tok0[u] = (t0 + i + u) * kTile;
                bad[u] = i + u >= n_own || ks[u] < 0.f;
                edge[u] = tok0[u] + kTile > all || bad[u];
            }

            // ---- S^T
            float s[T][G][CH][4];
#pragma unroll
            for (int u = 0; u < T; ++u)
#pragma unroll
                for (int t = 0; t < G; ++t)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int y = 0; y < CH; ++y) s[u][t][y][k] = 0.f;
#pragma unroll
            for (int j = 0; j < KJ; ++j) {
                uint4 ka[T], kb[T];
#pragma unroll
                for (int u = 0; u < T; ++u) {
                    // run j: for d >= 128 chunk c + 4 (j & 1) of the line, in half j / 2 of the tile
                    const uint32_t at_k = k_at + st + u * kStageBytes<D> + (j >> 1) * (kTile * 128);
                    ka[u] = lds16(at_k ^ ((j & 1) * 64));
                    kb[u] = D == 64 ? lds16((at_k + 512) ^ 64) : lds16((at_k + 1024) ^ ((j & 1) * 64));
                }
#pragma unroll
                for (int w = 0; w < 4; ++w)
#pragma unroll
                    for (int u = 0; u < T; ++u) {
                        const uint32_t aw[4] = {ka[u].x, ka[u].y, ka[u].z, ka[u].w};
                        const uint32_t bw[4] = {kb[u].x, kb[u].y, kb[u].z, kb[u].w};
                        uint32_t a0, a1, a2, a3;
                        half4(aw[w], a0, a2);
                        half4(bw[w], a1, a3);
#pragma unroll
                        for (int t = 0; t < G; ++t) {
                            uint2 q;
                            if constexpr (QS)
                                q = lds8(q_at + (t * (D / 16) + 4 * j + w) * 256);
                            else
                                q = make_uint2(qf[t][4 * j + w][0], qf[t][4 * j + w][1]);
                            mma16816(s[u][t][w % CH], a0, a1, a2, a3, q.x, q.y);
                        }
                    }
            }
            // ---- scores in units of log2 of this lane's rows: [i] of token tau(g), [RL + i] of tau(g) + 8
            float x[T][G][2 * RL];
            bool raise = false;
#pragma unroll
            for (int u = 0; u < T; ++u)
#pragma unroll
                for (int t = 0; t < G; ++t) {
#pragma unroll
                    for (int k = 0; k < 2 * RL; ++k) {
                        constexpr int step = PACK ? 2 : 1;  // PACK: the even columns
                        float y = s[u][t][0][step * k];
                        if constexpr (CH == 2) y += s[u][t][1][step * k];
                        x[u][t][k] = y * (rs[t][k % RL] * ks[u]);
                    }
                    if (edge[u]) {
#pragma unroll
                        for (int k = 0; k < 2 * RL; ++k)
                            if (bad[u] || tok0[u] + tau<D>(g) + 8 * (k / RL) >= lim[t][k % RL]) x[u][t][k] = neg_inf();
                    }
                    // n - lv is +inf for a scale of 0 (and NaN, which fminf leaves out, if nothing is seen)
#pragma unroll
                    for (int k = 0; k < RL; ++k)
                        raise |= fmaxf(x[u][t][k], x[u][t][k + RL]) > fminf(m[t][k], n[t][k] - lv[u]) + 8.f;
                }
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int t = 0; t < G; ++t)
#pragma unroll
                    for (int k = 0; k < RL; ++k) {
                        float mn = m[t][k], nn = n[t][k];
#pragma unroll
                        for (int u = 0; u < T; ++u) {
                            float top = fmaxf(x[u][t][k], x[u][t][k + RL]);
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                            mn = fmaxf(mn, top);
                            nn = fmaxf(nn, top + lv[u]);
                        }
                        // nothing seen yet (-inf): there is nothing to rescale
                        const float fl = m[t][k] == neg_inf() ? 1.f : ex2_approx(m[t][k] - mn);
                        const float fa = n[t][k] == neg_inf() ? 1.f : ex2_approx(n[t][k] - nn);
                        m[t][k] = mn;
                        n[t][k] = nn;
                        m0[t][k] = mn == neg_inf() ? 0.f : -mn;
                        n0[t][k] = nn == neg_inf() ? 7.f : 7.f - nn;
                        l[t][k] *= fl;
#pragma unroll
                        for (int d = 0; d < D / 16; ++d) {
                            acc[t][d][k] *= fa;
                            acc[t][d][k + 2] *= fa;
                            if constexpr (PACK) acc[t][d][1] *= fa, acc[t][d][3] *= fa;
                        }
                    }
            }
            uint32_t pb[T][G][2], pl[TWICE ? T : 1][TWICE ? G : 1][2];
#pragma unroll
            for (int u = 0; u < T; ++u)
#pragma unroll
                for (int t = 0; t < G; ++t) {
                    float w[2 * RL];
#pragma unroll
                    for (int k = 0; k < 2 * RL; ++k) {
                        l[t][k % RL] += ex2_approx(x[u][t][k] + m0[t][k % RL]);
                        w[k] = ex2_approx(x[u][t][k] + (lv[u] + n0[t][k % RL]));
                    }
                    if constexpr (PACK) {  // column 2 c has the first bits of row c, column 2 c + 1 the rest
                        pb[u][t][0] = transposed8x8(pack_half2(upper11(w[0]), w[0] - upper11(w[0])));
                        pb[u][t][1] = transposed8x8(pack_half2(upper11(w[1]), w[1] - upper11(w[1])));
                    } else {
                        if constexpr (TWICE) {
                            pl[u][t][0] = transposed8x8(pack_half2(w[0] - upper11(w[0]), w[1] - upper11(w[1])));
                            pl[u][t][1] = transposed8x8(pack_half2(w[2] - upper11(w[2]), w[3] - upper11(w[3])));
#pragma unroll
                            for (int k = 0; k < 4; ++k) w[k] = upper11(w[k]);
                        }
                        pb[u][t][0] = transposed8x8(pack_half2(w[0], w[1]));
                        pb[u][t][1] = transposed8x8(pack_half2(w[2], w[3]));
                    }
                }

            // ---- O^T
#pragma unroll
            for (int u = 0; u < T; ++u) {
                // nothing to add, and nothing was copied (a missing tile is the step's last)
                if (!bad[u]) {
                    const uint32_t st_v = st + u * kStageBytes<D>;
                    VWords<D> v;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        // token tau(2c + r % 2) + 8 (r / 2)
                        const uint32_t at_v = ((r & 1) ? v_at1 : v_at0) + st_v;
                        if constexpr (D == 64) {
                            const uint2 y = lds8(r < 2 ? at_v : (at_v + 512) ^ 64);
                            v[r][0] = y.x;
                            v[r][1] = y.y;
                        } else {
#pragma unroll
                            for (int j = 0; j < D / 128; ++j) {
                                const uint4 y = lds16(at_v + (r >> 1) * 1024 + j * (kTile * 128));
                                v[r][4 * j] = y.x;
                                v[r][4 * j + 1] = y.y;
                                v[r][4 * j + 2] = y.z;
                                v[r][4 * j + 3] = y.w;
                            }
                        }
                    }
                    if (edge[u]) {  // what lies behind the sequence's end may be anything
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            if (tok0[u] + tau<D>(2 * c + (r & 1)) + 8 * (r >> 1) >= len)
#pragma unroll
                                for (int w = 0; w < D / 32; ++w) v[r][w] = 0u;
                    }
                    // A NaN code among tokens that some rows do not see must not reach
                    // those rows (0 * NaN): then the product is taken for each query token by
                    // itself, with only the values that it sees.
                    bool special = false;
                    if (edge[u] && p.causal && p.N > 1) {
#pragma unroll
                        for (int r = 0; r < 4; ++r)
#pragma unroll
                            for (int w = 0; w < D / 32; ++w) special |= has_nan_code(v[r][w]);
                        special = __any_sync(0xffffffffu, special);
                    }
                    if (special) {
                        for (int tq = 0; tq < p.N; ++tq) {
                            const int seen = len - p.N + tq + 1 - tok0[u];
                            VWords<D> vm;
#pragma unroll
                            for (int r = 0; r < 4; ++r)
#pragma unroll
                                for (int w = 0; w < D / 32; ++w)
                                    vm[r][w] = tau<D>(2 * c + (r & 1)) + 8 * (r >> 1) < seen ? v[r][w] : 0u;
#pragma unroll
                            for (int w = 0; w < D / 32; ++w) {
                                uint32_t a[2][4];
                                v_operands<D>(a, vm, w);
#pragma unroll
                                for (int t = 0; t < G; ++t)
#pragma unroll
                                    for (int k = 0; k < 2; ++k) {
                                        float part[4] = {0.f, 0.f, 0.f, 0.f};
                                        mma16816(part, a[k][0], a[k][1], a[k][2], a[k][3], pb[u][t][0], pb[u][t][1]);
                                        if constexpr (TWICE)
                                            mma16816(part, a[k][0], a[k][1], a[k][2], a[k][3], pl[u][t][0], pl[u][t][1]);
#pragma unroll
                                        for (int j = 0; j < 4; ++j)
                                            if ((row0 + (PACK ? c : 8 * t + 2 * c + (j & 1))) % p.N == tq) acc[t][2 * w + k][j] += part[j];
                                    }
                            }
                        }
                    } else {
#pragma unroll
                        for (int w = 0; w < D / 32; ++w) {
                            uint32_t a[2][4];
                            v_operands<D>(a, v, w);
#pragma unroll
                            for (int t = 0; t < G; ++t)
#pragma unroll
                                for (int k = 0; k < 2; ++k)
                                    mma16816(acc[t][2 * w + k], a[k][0], a[k][1], a[k][2], a[k][3], pb[u][t][0], pb[u][t][1]);
                            if constexpr (TWICE) {
#pragma unroll
                                for (int t = 0; t < G; ++t)
#pragma unroll
                                    for (int k = 0; k < 2; ++k)
                                        mma16816(acc[t][2 * w + k], a[k][0], a[k][1], a[k][2], a[k][3], pl[u][t][0], pl[u][t][1]);
                            }
                        }
                    }
                }
                __syncwarp();  // every lane has taken its part of the tile
                if (i + u + S < n_pad) {
                    if (((i + u + S) & 31) == 0) window(i + u + S);
                    load(i + u + S, slot0 + u);
                }
            }
            slot0 += T;
            if (slot0 == S) slot0 = 0, parity ^= 1;
        }
        if constexpr (DIRECT) {
            // ---- the warps' parts, normalised, in their rings, and their merge
            constexpr int RS = D + 4;
            static_assert(R * RS * 4 <= kWarpBytes<D, NT>, "the rows lie in the warp's shared memory");
            __shared__ float2 s_ml[WARPS][R], s_row[R];
            __shared__ __align__(16) float s_o[R][D];
            uint8_t *const base = smem_raw + (((smem_u32(smem_raw) + 1023) & ~1023u) - smem_u32(smem_raw));
            float *rows = reinterpret_cast<float *>(base + warp * kWarpBytes<D, NT>);
            if constexpr (PACK) join_halves<D>(acc[0]);
            __syncwarp();  // every lane has read its last tile
#pragma unroll
            for (int t = 0; t < G; ++t)
#pragma unroll
                for (int k = 0; k < RL; ++k) {
                    float sum = l[t][k];
                    sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                    if (failed) sum = __int_as_float(0x7fffffff);
                    const float2 f = out_factor(m[t][k], n[t][k], sum);
                    const int r = PACK ? c : 8 * t + 2 * c + k;
                    if (g == 0) s_ml[warp][r] = make_float2(m[t][k], sum);
#pragma unroll
                    for (int w = 0; w < D / 32; ++w) {
                        const int d0 = D == 64 ? 8 * g + 4 * w : 128 * (w >> 2) + 16 * g + 4 * (w & 3);
                        *reinterpret_cast<float4 *>(rows + r * RS + d0) =
                            make_float4(acc[t][2 * w][k] * f.x * f.y, acc[t][2 * w][k + 2] * f.x * f.y,
                                        acc[t][2 * w + 1][k] * f.x * f.y, acc[t][2 * w + 1][k + 2] * f.x * f.y);
                    }
                }
            __syncthreads();
            for (int k = threadIdx.x; k < R * (D / 4); k += 32 * WARPS) {
                const int r = k / (D / 4), d0 = 4 * (k % (D / 4));
                if (row0 + r >= p.rows) break;
                float top = neg_inf();
#pragma unroll
                for (int w = 0; w < WARPS; ++w) top = fmaxf(top, s_ml[w][r].x);
                const float ref = top == neg_inf() ? 0.f : top;
                float sum = 0.f;
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < WARPS; ++w) {
                    const float a = ex2_approx(s_ml[w][r].x - ref) * s_ml[w][r].y;
                    const float4 y = *reinterpret_cast<const float4 *>(base + w * kWarpBytes<D, NT> + 4 * (r * RS + d0));
                    sum += a;
                    o.x += a * y.x, o.y += a * y.y, o.z += a * y.z, o.w += a * y.w;
                }
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
                if (p.cluster == 1) {
                    store_out(p, (q_row + r) * D + d0, o);
                    if (d0 == 0) p.lse[q_row + r] = row_lse(top, sum);
                } else {
                    *reinterpret_cast<float4 *>(&s_o[r][d0]) = o;
                    if (d0 == 0) s_row[r] = make_float2(top, sum);
                }
            }
            if (p.cluster == 1) return;
            // ---- the CTAs' parts: each CTA merges its share of the components
            cluster_sync();
            for (int k = threadIdx.x * p.cluster + rank; k < R * (D / 4); k += 32 * WARPS * p.cluster) {
                const int r = k / (D / 4), d0 = 4 * (k % (D / 4));
                if (row0 + r >= p.rows) break;
                const uint32_t row_at = smem_u32(&s_row[r]), o_at = smem_u32(&s_o[r][d0]);
                float top = neg_inf();
                for (int i = 0; i < p.cluster; ++i) top = fmaxf(top, peer_float2(row_at, i).x);
                const float ref = top == neg_inf() ? 0.f : top;
                float sum = 0.f;
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int i = 0; i < p.cluster; ++i) {
                    const float2 ml = peer_float2(row_at, i);
                    const float a = ex2_approx(ml.x - ref) * ml.y;
                    const float2 y = peer_float2(o_at, i), z = peer_float2(o_at + 8, i);
                    sum += a;
                    o.x += a * y.x, o.y += a * y.y, o.z += a * z.x, o.w += a * z.y;
                }
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
                store_out(p, (q_row + r) * D + d0, o);
                if (d0 == 0) p.lse[q_row + r] = row_lse(top, sum);
            }
            cluster_sync();  // no CTA ends while another reads its part
            return;
        }

        // ---- the next pair's copies start before this one's result is written
        const long long row = q_row;
        const bool whole = t0 == 0 && n_own == nb;
        const long long part = ((((long long)chunk * p.workers + worker) * 2) + (t0 == 0 ? 1 : 0)) * R;
        n_own = 0;
        if constexpr (PACK) join_halves<D>(acc[0]);
        more = !failed && next_pair();
#pragma unroll
        for (int t = 0; t < G; ++t)
#pragma unroll
            for (int k = 0; k < RL; ++k) {
                float sum = l[t][k];
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                if (failed) sum = __int_as_float(0x7fffffff);
                const float2 f = out_factor(m[t][k], n[t][k], sum);
                const int r = PACK ? c : 8 * t + 2 * c + k;
                if (row0 + r >= p.rows) continue;
                if (g == 0) {
                    if (whole)
                        p.lse[row + r] = row_lse(m[t][k], sum);
                    else
                        p.ml_part[part + r] = make_float2(m[t][k], sum);
                }
                // components 4 w .. 4 w + 3 of the lane's run
#pragma unroll
                for (int w = 0; w < D / 32; ++w) {
                    const int d0 = D == 64 ? 8 * g + 4 * w : 128 * (w >> 2) + 16 * g + 4 * (w & 3);
                    const float4 o = make_float4(acc[t][2 * w][k] * f.x * f.y, acc[t][2 * w][k + 2] * f.x * f.y,
                                                 acc[t][2 * w + 1][k] * f.x * f.y, acc[t][2 * w + 1][k + 2] * f.x * f.y);
                    if (whole)
                        store_out(p, (row + r) * D + d0, o);
                    else
                        *reinterpret_cast<float4 *>(p.o_part + (part + r) * D + d0) = o;
                }
            }
    }
}

// The rows whose keys several workers had, and those without keys.  WPR warps
// for each row share its parts (part i is warp i % WPR's); lane i has components
// [i D / 32, (i + 1) D / 32).  Bound by latency: the plan is found again while the
// first kernel still runs, then a warp reads the statistics of 32 parts at a
// time and their outputs, several in flight: about 4 us.  (One head of 131072 tokens, with 8 rows of 1776 parts,
// took 77 us with 8 warps a row that read all statistics first, 23 us now with the first kernel.)
template <int WPR> constexpr int kMergeWarps = WPR < 4 ? 4 : WPR;

template <int D, int WPR>
__global__ void __launch_bounds__(32 * kMergeWarps<WPR>) fa_cache_merge_kernel(const __grid_constant__ Params p, int rows_per) {
    constexpr int W = D / 32, WARPS = kMergeWarps<WPR>;
    __shared__ float s_o[WPR > 1 ? WARPS : 1][WPR > 1 ? D : 1];
    __shared__ float2 s_ml[WARPS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * (WARPS / WPR) + warp / WPR;
    const int sub = warp % WPR;
    const Plan plan = make_plan(p);
    const int unit = (int)(row / p.rows), r = (int)(row - (long long)unit * p.rows);
    const int b = unit / p.c.H_kv, h = unit - b * p.c.H_kv;
    const bool inside = b < p.c.B;
    int first = 0;
    for (int i = lane; i < min(b, p.c.B); i += 32) first += pair_cost(seq_tiles(p, i));
    first = __reduce_add_sync(0xffffffffu, first);
    const int nb = inside ? seq_tiles(p, b) : 0;
    const int s = first * p.c.H_kv + h * pair_cost(nb) + kPairCost;  // its first tile's place
    const int w0 = s / plan.per, w1 = nb ? (s + nb - 1) / plan.per : w0;
    // The results of the first kernel are complete from here on.  Every thread
    // waits, so that this grid does not end before the other.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!inside || (nb && w0 == w1)) return;  // the one worker that had it has written it
    const int n = nb ? w1 - w0 + 1 : 0;
    const int chunk = r / rows_per;
    // part i is worker w0 + i's; the first begins the pair, the others continue it
    const long long base = ((long long)chunk * p.workers + w0) * 2;
    const int rr = r - chunk * rows_per;
    auto index = [&](int i) { return (base + 2 * i + (i == 0 ? 1 : 0)) * rows_per + rr; };

    float o[W];
#pragma unroll
    for (int k = 0; k < W; ++k) o[k] = 0.f;
    float top = neg_inf(), sum = 0.f;
    for (int i0 = sub; i0 < n; i0 += 32 * WPR) {
        const int own = i0 + lane * WPR;
        const int m = min((n - i0 + WPR - 1) / WPR, 32);
        constexpr int UN = W > 4 ? 4 : 8;
        float y[UN][W];
        auto load = [&](int j0) {
#pragma unroll
            for (int u = 0; u < UN; ++u) {
                const float *src = p.o_part + index(i0 + min(j0 + u, m - 1) * WPR) * D + lane * W;
                if constexpr (W % 4 == 0) {
#pragma unroll
                    for (int k = 0; k < W; k += 4) {
                        const float4 z = *reinterpret_cast<const float4 *>(src + k);
                        y[u][k] = z.x, y[u][k + 1] = z.y, y[u][k + 2] = z.z, y[u][k + 3] = z.w;
                    }
                } else {
                    const float2 z = *reinterpret_cast<const float2 *>(src);
                    y[u][0] = z.x, y[u][1] = z.y;
                }
            }
        };
        float2 ml = make_float2(neg_inf(), 0.f);
        if (own < n) ml = p.ml_part[index(own)];
        load(0);  // in flight together with the statistics
        float t = fmaxf(ml.x, top);
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, i));
        if (t != neg_inf()) {  // else nothing has been seen: there is nothing to rescale
            const float f = ex2_approx(top - t);
            sum *= f;
#pragma unroll
            for (int k = 0; k < W; ++k) o[k] *= f;
        }
        top = t;
        const float a = ex2_approx(ml.x - (t == neg_inf() ? 0.f : t)) * ml.y;
        sum += a;  // this lane's parts; the lanes are added at the end
        for (int j0 = 0; j0 < m; j0 += UN) {
            if (j0 > 0) load(j0);
#pragma unroll
            for (int u = 0; u < UN; ++u) {
                if (j0 + u >= m) break;
                const float w = __shfl_sync(0xffffffffu, a, j0 + u);
#pragma unroll
                for (int k = 0; k < W; ++k) o[k] += w * y[u][k];
            }
        }
    }
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
    if constexpr (WPR > 1) {
#pragma unroll
        for (int k = 0; k < W; ++k) s_o[warp][lane * W + k] = o[k];
        if (lane == 0) s_ml[warp] = make_float2(top, sum);
        __syncthreads();
        if (warp) return;
        const float2 ml = lane < WPR ? s_ml[lane] : make_float2(neg_inf(), 0.f);
        top = ml.x;
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
        const float f = ex2_approx(ml.x - (top == neg_inf() ? 0.f : top));
        sum = f * ml.y;
#pragma unroll
        for (int i = 16; i > 0; i >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
#pragma unroll
        for (int k = 0; k < W; ++k) o[k] = 0.f;
        for (int w = 0; w < min(WPR, n); ++w) {
            const float fw = __shfl_sync(0xffffffffu, f, w);
#pragma unroll
            for (int k = 0; k < W; ++k) o[k] += fw * s_o[w][lane * W + k];
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const long long dst = row * D + lane * W;
#pragma unroll
    for (int k = 0; k < W; k += 2) {
        if (p.o_bf16)
            *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.o) + dst + k) = pack_bf16x2(o[k] * inv, o[k + 1] * inv);
        else
            *reinterpret_cast<float2 *>(static_cast<float *>(p.o) + dst + k) = make_float2(o[k] * inv, o[k + 1] * inv);
    }
    if (lane == 0) p.lse[row] = row_lse(top, sum);
}

}  // namespace cattn
}  // namespace fa
