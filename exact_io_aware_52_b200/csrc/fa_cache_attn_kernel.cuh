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
// 2^15, and 2^-24 the step of the smallest); O = acc * 2^(n - m - 7) / l.
//
// Tiles.  A warp takes 16 tokens of one key/value head at a time.  S^T = K Q^T and
// O^T = V^T P^T are computed transposed (mma m16n8k16, tokens or components
// on the 16 side, query rows on the 8 side), so that the 4 to 8 query rows
// that share a key fill the tensor core's narrow side and the codes are the
// A operand.  Which token or component a matrix row stands for is free, and it is
// chosen such that each lane's operands are whole 16-byte runs (8 for the values of
// d = 64) of the cache: every lane copies, by cp.async, what it will itself read, into
// its own slots of a ring in shared memory.  That needs no barrier, has no bank
// conflicts, and keeps the copies in flight out of the registers.
// tcgen05 would want 128 rows: at 8 rows 15/16 of it would be idle, and the codes would have to be
// written back to shared memory as fp16 for it.
//
// Bound by memory: 2 d bytes per token and key/value head, read once for
// all query rows that share it.
#pragma once

#include <cstdint>

#include "fa.h"
#include "fa_cache_kernels.cuh"

namespace fa {
namespace cattn {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 16;         // tokens a warp takes at a time; divides every page size
constexpr int kMaxWorkers = 640;  // CTAs that take work, at most

template <int D> constexpr int kStages = D == 64 ? 4 : (D == 128 ? 3 : 2);
template <int D> constexpr int kStageBytes = 2 * kTile * D;  // codes of K and V
template <int D> constexpr int kRingBytes = kStages<D> * kStageBytes<D>;
template <int D> constexpr int kSmemBytes = kWarps * kRingBytes<D>;
// query rows one CTA handles: 8 NT
template <int D> constexpr int kMaxNT = D == 256 ? 1 : 2;

struct Params {
    CacheView c;
    const uint16_t *q;
    void *o;
    float *lse;
    const int32_t *k_len;
    int32_t *status;
    float *o_part;        // [chunk][worker][2][8 NT][D]
    float2 *ml_part;      // [chunk][worker][2][8 NT] (m, l)
    int N, rows;          // query tokens; rows that share a key/value head: group * N
    int chunks, workers;  // blocks of 8 NT rows; CTAs for each of them
    int causal, o_bf16;
    float scale_log2;
};

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

__device__ __forceinline__ int seq_len(const Params &p, int b) {
    const long long cap = (long long)p.c.max_pages << p.c.page_log2;
    const int n = max(__ldg(p.k_len + b), 0);
    return (int)min((long long)n, cap);
}
__device__ __forceinline__ int seq_tiles(const Params &p, int b) { return (seq_len(p, b) + kTile - 1) / kTile; }

// The plan: the tiles of all (sequence, key/value head) pairs, in that order, are
// cut into runs of `per` tiles, one for each worker.  At least one tile for each
// warp; a multiple of the warps where a run is short enough for it to matter.
struct Plan {
    long long total;
    long long per;
};
__device__ __forceinline__ Plan make_plan(const Params &p) {
    const int lane = threadIdx.x & 31;
    long long t = 0;
    for (int b = lane; b < p.c.B; b += 32) t += seq_tiles(p, b);
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) t += __shfl_xor_sync(0xffffffffu, t, i);
    Plan r;
    r.total = t * p.c.H_kv;
    r.per = (r.total + p.workers - 1) / p.workers;
    if (r.per < 16 * kWarps) r.per = (r.per + kWarps - 1) / kWarps * kWarps;
    if (r.per < kWarps) r.per = kWarps;
    return r;
}

// The sequence that holds tile g < total, and its first tile.
__device__ __forceinline__ void locate(const Params &p, long long g, int &b, long long &first) {
    const int lane = threadIdx.x & 31;
    long long before = 0;
    for (int b0 = 0; b0 < p.c.B; b0 += 32) {
        const long long own = b0 + lane < p.c.B ? (long long)seq_tiles(p, b0 + lane) * p.c.H_kv : 0;
        long long inc = own;
#pragma unroll
        for (int i = 1; i < 32; i <<= 1) {
            const long long o = __shfl_up_sync(0xffffffffu, inc, i);
            if (lane >= i) inc += o;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, before + inc > g);
        if (hit) {
            const int l = __ffs(hit) - 1;
            b = b0 + l;
            first = before + __shfl_sync(0xffffffffu, inc - own, l);
            return;
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
    }
    b = p.c.B;
    first = before;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool take) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp8(uint32_t dst, const void *src, bool take) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(take ? 8 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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

// Words of V codes of one lane: [token][word], tokens 2c, 2c + 1, 2c + 8, 2c + 9 of the tile.
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

// One CTA: a run of tiles, segment by segment ((sequence, head) pairs).  The
// warps of the CTA take a segment's tiles in turn and merge at its end.
template <int D, int NT>
__global__ void __launch_bounds__(kThreads, D == 256 ? 2 : (NT == 2 ? 3 : 4))
fa_cache_attn_kernel(const __grid_constant__ Params p) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float2 s_ml[kWarps][8 * NT];
    constexpr int KJ = D / 64;               // 16-byte runs of a key for each lane
    constexpr int RS = D + 4;                // row stride of the merge's floats
    static_assert(8 * NT * RS * 4 <= kRingBytes<D>, "the merge's rows lie in the warp's ring");

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    const int chunk = blockIdx.x % p.chunks, worker = blockIdx.x / p.chunks;
    const int row0 = chunk * 8 * NT;
    const Plan plan = make_plan(p);
    long long at = worker * plan.per;
    const long long end = min(plan.total, at + plan.per);
    if (at >= end) return;
    int b;
    long long first;
    locate(p, at, b, first);

    uint8_t *ring = smem + warp * kRingBytes<D>;
    const uint32_t ring_u32 = smem_u32(ring);
    const uint32_t k_slot = ring_u32 + 16 * lane;
    const uint32_t v_slot = ring_u32 + kTile * D + (D == 64 ? 8 : 16) * lane;
    const int tile_shift = p.c.page_log2 - 4;
    const CacheView &cv = p.c;

    while (at < end) {
        const int len = seq_len(p, b);
        const int nb = (len + kTile - 1) / kTile;
        if (at - first >= (long long)nb * cv.H_kv) {  // next sequence (this one may be empty)
            first += (long long)nb * cv.H_kv;
            ++b;
            continue;
        }
        const int h = (int)((at - first) / nb);
        const int t0 = (int)(at - first - (long long)h * nb);
        const int t1 = (int)min((long long)nb, t0 + (end - at));
        at += t1 - t0;
        const long long q_row = ((long long)b * cv.H_kv + h) * p.rows + row0;  // first row of q, o, lse
        const int32_t *table = cv.table + b * cv.table_stride;

        // ---- this warp's tiles: t0 + warp + 4 i, i < n_own
        const int n_own = (t1 - t0 - warp + kWarps - 1) / kWarps;
        // windows of 32 own tiles: lane i has tile i's page and scales
        int w_page = -1;
        float w_ks = -1.f, w_vs = 0.f, w_ks_old = -1.f, w_vs_old = 0.f;
        auto load = [&](int i) {  // own tile i into its stage
            if ((i & 31) == 0) {
                w_ks_old = w_ks;
                w_vs_old = w_vs;
                w_page = -1;
                w_ks = -1.f;  // marks a page outside the pool
                w_vs = 0.f;
                if (i + lane < n_own) {
                    const int t = t0 + warp + kWarps * (i + lane);
                    const int page_id = __ldg(table + (t >> tile_shift));
                    if (page_id >= 0 && page_id < cv.n_pages) {
                        w_page = page_id;
                        const long long unit = (long long)page_id * cv.H_kv + h;
                        w_ks = cv.k_scale[unit];
                        w_vs = cv.v_scale[unit];
                    } else {
                        report_bad_page(p.status);
                    }
                }
            }
            const int page_id = __shfl_sync(0xffffffffu, w_page, i & 31);
            const int t = t0 + warp + kWarps * i;
            const int slot = (t & ((1 << tile_shift) - 1)) * kTile;
            const int left = page_id < 0 ? 0 : len - t * kTile;  // tokens of the tile to read
            const long long off = (((long long)max(page_id, 0) * cv.H_kv + h) * cv.page + slot) * D;
            const uint32_t st = (uint32_t)(i % kStages<D>) * kStageBytes<D>;
            const uint8_t *ks = cv.k + off + g * D + 16 * c;
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int j = 0; j < KJ; ++j)
                    cp16(k_slot + st + (r * KJ + j) * 512, ks + r * 8 * D + 64 * j, g + 8 * r < left);
            const uint8_t *vs = cv.v + off + 2 * c * D + (D == 64 ? 8 : 16) * g;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int tok = (r & 1) + 8 * (r >> 1);
                const bool take = 2 * c + tok < left;
                if constexpr (D == 64) {
                    cp8(v_slot + st + r * 256, vs + tok * D, take);
                } else {
#pragma unroll
                    for (int j = 0; j < D / 128; ++j)
                        cp16(v_slot + st + (r * (D / 128) + j) * 512, vs + tok * D + 128 * j, take);
                }
            }
        };
#pragma unroll
        for (int i = 0; i < kStages<D> - 1; ++i) {
            if (i < n_own) load(i);
            cp_commit();
        }

        // ---- queries: fp16 of each row times a power of two that brings its
        // largest magnitude to [2^14, 2^15); bf16's 8 bits stay exact but for
        // components 2^-29 below the row's largest
        uint32_t qf[NT][D / 16][2];
        float rs[NT][2];   // of rows 2c and 2c + 1: scale * log2(e) / that power
        int lim[NT][2];    // and their number of keys
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int r = 8 * t + g;
            const bool live = row0 + r < p.rows;
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
            // up = 2^(14 - E), E the exponent of the largest (2^126 at most: a row of subnormal
            // values stays below 2^14)
            const int e = min(max(14 - ((int)(mag >> 7) - 127), -126), 126);
            const float up = __uint_as_float((uint32_t)(e + 127) << 23);
#pragma unroll
            for (int j = 0; j < KJ; ++j)
#pragma unroll
                for (int w = 0; w < 4; ++w)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t z = raw[j][2 * w + i];
                        qf[t][4 * j + w][i] = pack_half2(bf16x2_lo(z) * up, bf16x2_hi(z) * up);
                    }
            const float f = __uint_as_float((uint32_t)(127 - e) << 23) * p.scale_log2;
            rs[t][0] = __shfl_sync(0xffffffffu, f, 8 * c);
            rs[t][1] = __shfl_sync(0xffffffffu, f, 8 * c + 4);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int row = row0 + 8 * t + 2 * c + i;
                lim[t][i] = p.causal ? len - p.N + row % p.N + 1 : len;
            }
        }
        const int all = p.causal ? len - p.N + 1 : len;  // keys that every row sees

        float acc[NT][D / 16][4];
        float m[NT][2], n[NT][2], l[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i) acc[t][i][0] = acc[t][i][1] = acc[t][i][2] = acc[t][i][3] = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) m[t][i] = n[t][i] = neg_inf(), l[t][i] = 0.f;
        }

        for (int i = 0; i < n_own; ++i) {
            if (i + kStages<D> - 1 < n_own) load(i + kStages<D> - 1);
            cp_commit();
            cp_wait<kStages<D> - 1>();
            const uint32_t st = (uint32_t)(i % kStages<D>) * kStageBytes<D>;
            const int tok0 = (t0 + warp + kWarps * i) * kTile;
            const bool old = (min(i + kStages<D> - 1, n_own - 1) >> 5) != (i >> 5);  // its window has been left
            const float ks = __shfl_sync(0xffffffffu, old ? w_ks_old : w_ks, i & 31);
            const float vs = __shfl_sync(0xffffffffu, old ? w_vs_old : w_vs, i & 31);
            const float lv = __log2f(vs);

            // ---- S^T, in two sums
            float s[NT][2][4];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int k = 0; k < 4; ++k) s[t][0][k] = s[t][1][k] = 0.f;
#pragma unroll
            for (int j = 0; j < KJ; ++j) {
                const uint4 a = lds16(k_slot + st + j * 512), bq = lds16(k_slot + st + (KJ + j) * 512);
                const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {bq.x, bq.y, bq.z, bq.w};
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint32_t a0, a1, a2, a3;
                    half4(aw[w], a0, a2);
                    half4(bw[w], a1, a3);
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        mma16816(s[t][w & 1], a0, a1, a2, a3, qf[t][4 * j + w][0], qf[t][4 * j + w][1]);
                }
            }
            VWords<D> v;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if constexpr (D == 64) {
                    const uint2 x = lds8(v_slot + st + r * 256);
                    v[r][0] = x.x;
                    v[r][1] = x.y;
                } else {
#pragma unroll
                    for (int j = 0; j < D / 128; ++j) {
                        const uint4 x = lds16(v_slot + st + (r * (D / 128) + j) * 512);
                        v[r][4 * j] = x.x;
                        v[r][4 * j + 1] = x.y;
                        v[r][4 * j + 2] = x.z;
                        v[r][4 * j + 3] = x.w;
                    }
                }
            }

            // ---- scores in units of log2; x[t][0..1] token g, x[t][2..3] token g + 8
            float x[NT][4];
            const bool bad = ks < 0.f;
            const bool edge = tok0 + kTile > all || bad;
            bool raise = false;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const float f[2] = {rs[t][0] * ks, rs[t][1] * ks};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    x[t][k] = (s[t][0][k] + s[t][1][k]) * f[k & 1];
                    if (edge && (bad || tok0 + g + 8 * (k >> 1) >= lim[t][k & 1])) x[t][k] = neg_inf();
                    raise |= x[t][k] > m[t][k & 1] + 8.f || x[t][k] + lv > n[t][k & 1] + 8.f;
                }
            }
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float top = fmaxf(x[t][k], x[t][k + 2]);
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                        const float mn = fmaxf(m[t][k], top), nn = fmaxf(n[t][k], top + lv);
                        // nothing seen yet (-inf): there is nothing to rescale
                        const float fl = m[t][k] == neg_inf() ? 1.f : ex2_approx(m[t][k] - mn);
                        const float fa = n[t][k] == neg_inf() ? 1.f : ex2_approx(n[t][k] - nn);
                        m[t][k] = mn;
                        n[t][k] = nn;
                        l[t][k] *= fl;
#pragma unroll
                        for (int d = 0; d < D / 16; ++d) {
                            acc[t][d][k] *= fa;
                            acc[t][d][k + 2] *= fa;
                        }
                    }
            }
            uint32_t pb[NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float mr = m[t][k & 1], nr = n[t][k & 1];
                    l[t][k & 1] += ex2_approx(x[t][k] - (mr == neg_inf() ? 0.f : mr));
                    w[k] = ex2_approx(x[t][k] + (lv - (nr == neg_inf() ? 0.f : nr) + 7.f));
                }
                pb[t][0] = transposed8x8(pack_half2(w[0], w[1]));
                pb[t][1] = transposed8x8(pack_half2(w[2], w[3]));
            }

            // ---- O^T.  A NaN code among tokens that some rows do not see must not
            // reach those rows (0 * NaN): then the product is taken for each query
            // token by itself, with only the values that it sees.
            bool special = false;
            if (edge && p.causal && p.N > 1) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int w = 0; w < D / 32; ++w) special |= has_nan_code(v[r][w]);
            }
            if (edge && __any_sync(0xffffffffu, special)) {
                for (int tq = 0; tq < p.N; ++tq) {
                    const int seen = len - p.N + tq + 1 - tok0;
                    VWords<D> vm;
#pragma unroll
                    for (int r = 0; r < 4; ++r)
#pragma unroll
                        for (int w = 0; w < D / 32; ++w)
                            vm[r][w] = 2 * c + (r & 1) + 8 * (r >> 1) < seen ? v[r][w] : 0u;
#pragma unroll
                    for (int w = 0; w < D / 32; ++w) {
                        uint32_t a[2][4];
                        v_operands<D>(a, vm, w);
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                float part[4] = {0.f, 0.f, 0.f, 0.f};
                                mma16816(part, a[k][0], a[k][1], a[k][2], a[k][3], pb[t][0], pb[t][1]);
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    if ((row0 + 8 * t + 2 * c + (j & 1)) % p.N == tq) acc[t][2 * w + k][j] += part[j];
                            }
                    }
                }
            } else {
#pragma unroll
                for (int w = 0; w < D / 32; ++w) {
                    uint32_t a[2][4];
                    v_operands<D>(a, v, w);
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            mma16816(acc[t][2 * w + k], a[k][0], a[k][1], a[k][2], a[k][3], pb[t][0], pb[t][1]);
                }
            }
        }
        cp_wait<0>();
        __syncwarp();  // every lane has read its last stage: the ring becomes the merge's rows

        // ---- this warp's part, normalised
        float *rows = reinterpret_cast<float *>(ring);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float sum = l[t][k];
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                const float f = sum == 0.f ? 0.f : ex2_approx(n[t][k] - m[t][k] - 7.f) / sum;
                const int r = 8 * t + 2 * c + k;
                if (g == 0) s_ml[warp][r] = make_float2(m[t][k], sum);
                // components 4 w .. 4 w + 3 of the lane's run
#pragma unroll
                for (int w = 0; w < D / 32; ++w) {
                    const int d0 = D == 64 ? 8 * g + 4 * w : 128 * (w >> 2) + 16 * g + 4 * (w & 3);
                    *reinterpret_cast<float4 *>(rows + r * RS + d0) =
                        make_float4(acc[t][2 * w][k] * f, acc[t][2 * w][k + 2] * f, acc[t][2 * w + 1][k] * f,
                                    acc[t][2 * w + 1][k + 2] * f);
                }
            }
        __syncthreads();

        // ---- merge the warps: 4 components of a row for each thread
        const bool whole = t0 == 0 && t1 == nb;
        const long long part = ((long long)chunk * p.workers + worker) * 2 + (t0 == 0 ? 1 : 0);
        for (int k = threadIdx.x; k < 8 * NT * (D / 4); k += kThreads) {
            const int r = k / (D / 4), d0 = 4 * (k % (D / 4));
            if (row0 + r >= p.rows) break;
            float2 ml[kWarps];
            float top = neg_inf();
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                ml[w] = s_ml[w][r];
                top = fmaxf(top, ml[w].x);
            }
            const float ref = top == neg_inf() ? 0.f : top;
            float sum = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float a = ex2_approx(ml[w].x - ref) * ml[w].y;
                const float4 y = *reinterpret_cast<const float4 *>(smem + w * kRingBytes<D> + 4 * (r * RS + d0));
                sum += a;
                o.x += a * y.x;
                o.y += a * y.y;
                o.z += a * y.z;
                o.w += a * y.w;
            }
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            o.x *= inv, o.y *= inv, o.z *= inv, o.w *= inv;
            if (!whole) {
                *reinterpret_cast<float4 *>(p.o_part + (part * 8 * NT + r) * D + d0) = o;
                if (d0 == 0) p.ml_part[part * 8 * NT + r] = make_float2(top, sum);
            } else {
                const long long at_o = (q_row + r) * D + d0;
                if (p.o_bf16)
                    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.o) + at_o) =
                        make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
                else
                    *reinterpret_cast<float4 *>(static_cast<float *>(p.o) + at_o) = o;
                if (d0 == 0) p.lse[q_row + r] = sum == 0.f ? neg_inf() : (ref + log2f(sum)) * 0.693147180559945f;
            }
        }
        __syncthreads();  // before the next segment's copies reach the rows
    }
}

constexpr int kMergeWarps = 8;

// The rows whose keys several workers had, and those without keys.  WPR warps
// for each row share its parts; lane i has components [i D / 32, (i + 1) D / 32).
// Bound by latency: the plan is found again while the first kernel still runs.
template <int D, int WPR>
__global__ void __launch_bounds__(32 * kMergeWarps) fa_cache_merge_kernel(const __grid_constant__ Params p, int nt8) {
    constexpr int W = D / 32;
    __shared__ float s_o[WPR > 1 ? kMergeWarps : 1][D];
    __shared__ float2 s_ml[kMergeWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * (kMergeWarps / WPR) + warp / WPR;
    const int sub = warp % WPR;
    const Plan plan = make_plan(p);
    const int unit = (int)(row / p.rows), r = (int)(row - (long long)unit * p.rows);
    const int b = unit / p.c.H_kv, h = unit - b * p.c.H_kv;
    const bool inside = b < p.c.B;
    long long first = 0;
    for (int i = lane; i < min(b, p.c.B); i += 32) first += seq_tiles(p, i);
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) first += __shfl_xor_sync(0xffffffffu, first, i);
    const int nb = inside ? seq_tiles(p, b) : 0;
    const long long s = first * p.c.H_kv + (long long)h * nb;
    const long long w0 = s / plan.per, w1 = nb ? (s + nb - 1) / plan.per : w0;
    // The results of the first kernel are complete from here on.  Every thread
    // waits, so that this grid does not end before the other.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!inside || (nb && w0 == w1)) return;  // the one worker that had it has written it
    const int n = nb ? (int)(w1 - w0) + 1 : 0;
    const int chunk = r / nt8;
    // part i is worker w0 + i's; the first begins the segment, the others continue it
    const long long base = ((long long)chunk * p.workers + w0) * 2;
    const int rr = r - chunk * nt8;
    auto index = [&](int i) { return (base + 2 * i + (i == 0 ? 1 : 0)) * nt8 + rr; };

    float top = neg_inf();
    for (int i = lane; i < n; i += 32) top = fmaxf(top, p.ml_part[index(i)].x);
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
    const float ref = top == neg_inf() ? 0.f : top;
    float o[W];
#pragma unroll
    for (int k = 0; k < W; ++k) o[k] = 0.f;
    float sum = 0.f;
    constexpr int UN = 4;
    for (int i0 = sub; i0 < n; i0 += UN * WPR) {
        float a[UN], y[UN][W];
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const int i = i0 + u * WPR;
            a[u] = 0.f;
#pragma unroll
            for (int k = 0; k < W; ++k) y[u][k] = 0.f;
            if (i < n) {
                const float2 ml = p.ml_part[index(i)];
                a[u] = ex2_approx(ml.x - ref) * ml.y;
                const float *src = p.o_part + index(i) * D + lane * W;
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
        }
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            sum += a[u];
#pragma unroll
            for (int k = 0; k < W; ++k) o[k] += a[u] * y[u][k];
        }
    }
    if constexpr (WPR > 1) {
#pragma unroll
        for (int k = 0; k < W; ++k) s_o[warp][lane * W + k] = o[k];
        if (lane == 0) s_ml[warp].y = sum;
        __syncthreads();
        if (warp) return;
        sum = 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) o[k] = 0.f;
        for (int w = 0; w < WPR; ++w) {
            sum += s_ml[w].y;
#pragma unroll
            for (int k = 0; k < W; ++k) o[k] += s_o[w][lane * W + k];
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
    if (lane == 0) p.lse[row] = sum == 0.f ? neg_inf() : (ref + log2f(sum)) * 0.693147180559945f;
}

}  // namespace cattn
}  // namespace fa
