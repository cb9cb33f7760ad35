// fa_cache_kernels.cuh -- writing the paged 8-bit key/value cache
// (fa_cache_append) and reading it as contiguous bf16 (fa_cache_gather).
//
// A page and head's scale is a power of two.  E4M3 is a floating type: its
// relative step is the same wherever in the range a value lies, so a power of
// two costs no precision against amax / 448, and it makes x / scale, the
// rescaling of a page that grows and code * scale in bf16 exact (the rescaling
// but for codes that become subnormal).
#pragma once

#include <cstdint>

#include "fa.h"
#include "fa_rotary.cuh"

namespace fa {

struct CacheView {
    uint8_t *k, *v;
    float *k_scale, *v_scale;
    const int32_t *table;
    long long table_stride;
    int n_pages, max_pages, B, H_kv, page, d;
    int page_log2;
};

// The first error of a launch wins.
__device__ __forceinline__ void report_bad_page(int32_t *status) {
    if (status) atomicCAS(status, 0, (int)FA_ERR_BAD_PAGE);
}

// ---------------------------------------------------------------- append
struct AppendParams {
    CacheView c;
    const uint16_t *x[2];       // new keys, new values
    long long xs[2][3];
    int N;
    int pages;                  // pages that N tokens can touch, at most
    int group;                  // heads that one block handles
    const int32_t *start, *n_new;
    int32_t *status;
    int dim, interleaved;       // dim 0: keys are not turned
    float amplitude;
    uint64_t step[FA_ROTARY_MAX_DIM / 2];
};

constexpr int kMinScaleExp = -100;

// The exponent field of the scale for values of magnitude amax (a float's bits): 2^e with the least
// e >= kMinScaleExp such that amax <= 448 * 2^e.  With amax = m * 2^E, 1 <= m < 2, and 448 = 1.75 * 2^8, e is
// E - 8 where m <= 1.75 and E - 7 else: adding what a mantissa just above 1.75 needs to carry gives that.
__device__ __forceinline__ uint32_t scale_field(uint32_t amax) {
    return (uint32_t)max((int)((amax + 0x1fffffu) >> 23) - 8, 127 + kMinScaleExp);
}

// Four values times inv as E4M3 codes.  NaN gives the code NaN; SPECIAL: infinities
// do so too (v * 0 is NaN for them and 0 for the others; the conversion would saturate them).
template <bool SPECIAL>
__device__ __forceinline__ uint32_t codes4(const float *v, float inv) {
    if constexpr (SPECIAL)
        return pack_e4m3x4(fmaf(v[0], inv, v[0] * 0.f), fmaf(v[1], inv, v[1] * 0.f), fmaf(v[2], inv, v[2] * 0.f),
                           fmaf(v[3], inv, v[3] * 0.f));
    else {
        const float2 i2 = make_float2(inv, inv);
        const float2 a = __fmul2_rn(make_float2(v[0], v[1]), i2), b = __fmul2_rn(make_float2(v[2], v[3]), i2);
        return pack_e4m3x4(a.x, a.y, b.x, b.y);
    }
}

// The four values of a word of E4M3 codes.
__device__ __forceinline__ void values4(uint32_t w, float *v) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(v[0]), "=f"(v[1])
        : "r"(lo));
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(v[2]), "=f"(v[3])
        : "r"(hi));
}

// One component of a key, turned, for layouts that do not fall into slots.  Not made for speed: the partner is loaded
// and the sine computed for each component.  Measured, 4 x 4096 tokens, 8 heads of d = 128: 20 turned components 68 us, 32, which
// fall into slots, 28 us.
__device__ __forceinline__ float key_component(const AppendParams &p, const uint16_t *x, int e, int pos) {
    const float v = load1(x + e);
    if (e >= p.dim) return v;
    const int half = p.dim >> 1;
    const int i = p.interleaved ? e >> 1 : (e < half ? e : e - half);
    const bool first = p.interleaved ? !(e & 1) : e < half;
    float a, b, c, s;
    a = first ? v : load1(x + (p.interleaved ? e - 1 : e - half));
    b = first ? load1(x + (p.interleaved ? e + 1 : e + half)) : v;
    rotary_cs(p.step[i], pos, p.amplitude, 1.f, c, s);
    rotary_turn(a, b, c, s);
    return first ? a : b;
}

// The scale of a page whose new values reach amax (bits), and its inverse; `held`: the page holds tokens
// from before, with the scale `before`.
struct ScaleUpdate {
    float now, inv;
    bool grows;  // the page's earlier codes have to follow
};
__device__ __forceinline__ ScaleUpdate update_scale(bool held, float before, uint32_t amax) {
    const uint32_t field = scale_field(amax);
    ScaleUpdate r;
    r.now = __uint_as_float(field << 23);
    r.inv = __uint_as_float((254u - field) << 23);
    r.grows = false;
    if (held) {  // the caller's own scale may be anything
        const float mine = r.now;
        r.now = fmaxf(before, mine);
        r.grows = r.now != before;
        if (r.now != mine) r.inv = 1.f / r.now;
    }
    return r;
}

// Where a block's (or warp's) new tokens lie: slots [s0, s1) of one page, the first of them
// the sequence's new token t0.
struct Touched {
    int page_id, s0, s1, t0;
    long long lo;  // position of the page's slot 0
};
// The pt-th page that sequence b's new tokens touch; false if there is none, or if it
// is bad, which is reported.  The same for all threads of a block.
__device__ __forceinline__ bool touched_page(const AppendParams &p, int b, int pt, bool reporter, Touched &r) {
    const CacheView &c = p.c;
    const int start = p.start[b];
    int n = p.n_new ? p.n_new[b] : p.N;
    n = n < 0 ? 0 : (n > p.N ? p.N : n);
    if (n == 0) return false;
    if (start < 0) {
        if (reporter) report_bad_page(p.status);
        return false;
    }
    const long long first = start, end = first + n;
    const long long page_i = (first >> c.page_log2) + pt;
    r.lo = page_i << c.page_log2;
    if (r.lo >= end) return false;
    r.page_id = page_i < c.max_pages ? c.table[b * c.table_stride + page_i] : -1;
    if (r.page_id < 0 || r.page_id >= c.n_pages) {
        if (reporter) report_bad_page(p.status);
        return false;
    }
    r.s0 = first > r.lo ? (int)(first - r.lo) : 0;
    r.s1 = end - r.lo < c.page ? (int)(end - r.lo) : c.page;
    r.t0 = (int)(r.lo + r.s0 - first);
    return true;
}

// A slot of 16 components in one piece.
__device__ __forceinline__ RotarySlot plain_slot(int s) { return RotarySlot{16 * s, 16 * s + 8, false}; }

// A slot's components as they come: 16 bf16.
struct Raw16 {
    uint32_t w[8];
    __device__ __forceinline__ void load(const uint16_t *row, const RotarySlot &at) {
        const uint4 x = *reinterpret_cast<const uint4 *>(row + at.a), y = *reinterpret_cast<const uint4 *>(row + at.b);
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w, w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
    }
    __device__ __forceinline__ void load_elements(const uint16_t *x) {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = (uint32_t)x[2 * j] | (uint32_t)x[2 * j + 1] << 16;
    }
    __device__ __forceinline__ void get(float (&v)[16]) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[2 * j] = bf16x2_lo(w[j]), v[2 * j + 1] = bf16x2_hi(w[j]);
    }
};

constexpr uint32_t kInfBits = 0x7f800000u;

// Largest magnitude as bits, which order as the magnitudes do; from kInfBits on there is an infinity
// (or, among values, NaN).  NaN among keys is left out.
__device__ __forceinline__ uint32_t key_amax(const float (&v)[16]) {
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 16; j += 2) asm("max.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(v[j]), "f"(v[j + 1]));
    return __float_as_uint(m);
}
__device__ __forceinline__ uint32_t value_amax(const Raw16 &x) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) asm("max.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(x.w[j]));
    m &= 0x7fff7fffu;  // (the signs are those of the products)
    return max(m << 16, m & 0xffff0000u);
}
// Of the finite ones.
__device__ __forceinline__ uint32_t amax_finite(const float (&v)[16]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        const uint32_t u = __float_as_uint(v[j]) & 0x7fffffffu;
        if (u < kInfBits) m = max(m, u);
    }
    return m;
}

__device__ __forceinline__ void store_slot(uint8_t *row, const RotarySlot &at, const float (&v)[16], float inv,
                                           bool special) {
    uint2 a, b;
    if (special) {
        a = make_uint2(codes4<true>(v, inv), codes4<true>(v + 4, inv));
        b = make_uint2(codes4<true>(v + 8, inv), codes4<true>(v + 12, inv));
    } else {
        a = make_uint2(codes4<false>(v, inv), codes4<false>(v + 4, inv));
        b = make_uint2(codes4<false>(v + 8, inv), codes4<false>(v + 12, inv));
    }
    if (at.b == at.a + 8) {
        *reinterpret_cast<uint4 *>(row + at.a) = make_uint4(a.x, a.y, b.x, b.y);
    } else {
        *reinterpret_cast<uint2 *>(row + at.a) = a;
        *reinterpret_cast<uint2 *>(row + at.b) = b;
    }
}

// 16 codes of a page that grows.
__device__ __forceinline__ void rescale_run(uint8_t *run, float ratio) {
    uint4 w = *reinterpret_cast<const uint4 *>(run);
    uint32_t *q = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float o[4];
        values4(q[j], o);
        q[j] = codes4<true>(o, ratio);
    }
    *reinterpret_cast<uint4 *>(run) = w;
}

// `runs` runs of 16 codes of a page that grows, by the whole block.  Rare, and kept out of the kernel's registers.
__device__ __noinline__ void rescale_codes(uint8_t *codes, int runs, float ratio) {
    for (int r = threadIdx.x; r < runs; r += blockDim.x) rescale_run(codes + 16 * r, ratio);
}

// One block per (sequence, touched page, group of heads): it owns the page's codes and scales of
// its heads, so that nothing in global memory needs atomics and no order of blocks changes the result.  The block's
// maxima go through atomics in shared memory, one for each warp (a maximum does not depend on their order).
// The sines and cosines, several times the work of the rest, are computed once for a group
// and lie in shared memory (registers would leave no room for the next
// head's loads, which are in flight while a head is finished).  A thread has the same slot
// (16 components) of a new token for every head; keys and values are read once and stay in
// registers between the maximum and the rounding.  TWO: a page's new tokens are two
// blocks' worth of slots; they are read again, from L2, after the maximum.  Bound by
// memory (2 bytes read and 1 written per component) as far as the issue slots allow.  Measured: 4 ragged
// prompts of up to 8192 tokens, 8 heads of d = 128, pages of 64 (154 MB), keys turned whole 40 us,
// as they are 31 us, two thirds of the issue slots used.  256 threads with two slots each took 49 to 60 us, 512
// with twice the registers 45 us.
template <bool VEC, bool TWO>
__global__ void __launch_bounds__(1024, 1) fa_cache_append_kernel(const __grid_constant__ AppendParams p) {
    extern __shared__ float4 s_cs[];  // [token][pair of entries][slot]: (cos, sin) of two of a slot's 8 entries
    __shared__ uint32_t s_max[3][2];  // of K and V, of three heads in turn
    constexpr bool AHEAD = VEC && !TWO;
    constexpr int CHUNKS = TWO ? 2 : 1;
    const CacheView &c = p.c;
    const int groups = (c.H_kv + p.group - 1) / p.group;
    const int h0 = (blockIdx.x % groups) * p.group, h1 = min(h0 + p.group, c.H_kv);
    const int u = blockIdx.x / groups;
    const int pt = u % p.pages, b = u / p.pages;
    Touched pg;
    if (!touched_page(p, b, pt, threadIdx.x == 0, pg)) return;
    if (threadIdx.x < 6) s_max[threadIdx.x >> 1][threadIdx.x & 1] = 0;
    const int dim = VEC ? p.dim : 0;
    const int per_row = c.d >> 4, row_log2 = 31 - __clz(per_row);
    const int turned = dim >> 4;  // slots of a token that are turned
    const int n_new = pg.s1 - pg.s0;
    // This thread's slot of new token i of the page (and of token i + dt), and where it lies in the inputs
    // and in the page.  All of it advances by a head at a time.
    const int i = threadIdx.x >> row_log2, dt = blockDim.x >> row_log2, slot = threadIdx.x & (per_row - 1);
    const RotarySlot at = VEC ? rotary_slot(slot, c.d, dim) : plain_slot(slot);
    const bool turns = slot < turned;
    const uint16_t *xk = p.x[0] + b * p.xs[0][0] + h0 * p.xs[0][1] + (pg.t0 + i) * p.xs[0][2];
    const uint16_t *xv = p.x[1] + b * p.xs[1][0] + h0 * p.xs[1][1] + (pg.t0 + i) * p.xs[1][2] + 16 * slot;
    int unit = pg.page_id * c.H_kv + h0;  // (page, head)
    long long off = ((long long)unit * c.page + pg.s0 + i) * c.d;

    Raw16 rk, rv;
    auto load = [&](int chunk) {
        if (i + chunk * dt >= n_new) return;
        if constexpr (VEC) {
            rk.load(xk + chunk * dt * p.xs[0][2], at);
            rv.load(xv + chunk * dt * p.xs[1][2], RotarySlot{0, 8, false});
        } else {
            rv.load_elements(xv + chunk * dt * p.xs[1][2]);
        }
    };
    load(0);
    if constexpr (VEC) {
        if (dim) {
            __shared__ uint64_t step[FA_ROTARY_MAX_DIM / 2];
            for (int j = threadIdx.x; j < (dim >> 1); j += blockDim.x) step[j] = p.step[j];
            __syncthreads();
            const unsigned n = n_new * 4 * turned;
            for (unsigned k = threadIdx.x; k < n; k += blockDim.x) {
                const unsigned q = k / (unsigned)turned, e = k - q * turned;
                const int pos = (int)(pg.lo + pg.s0 + (q >> 2)), j = 2 * (q & 3);
                float4 x;
                rotary_cs(step[rotary_pair(e, j, dim, p.interleaved)], pos, p.amplitude, 1.f, x.x, x.y);
                rotary_cs(step[rotary_pair(e, j + 1, dim, p.interleaved)], pos, p.amplitude, 1.f, x.z, x.w);
                s_cs[q * turned + e] = x;
            }
        }
    }
    __syncthreads();
    const float4 *my_cs = s_cs + i * 4 * turned + slot;
    // The key of this thread's slot, turned.
    auto key = [&](int chunk, float (&k)[16]) {
        if constexpr (VEC) {
            rk.get(k);
            if (turns) {
                float cs[8], sn[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 x = my_cs[(chunk * dt * 4 + j) * turned];
                    cs[2 * j] = x.x, sn[2 * j] = x.y, cs[2 * j + 1] = x.z, sn[2 * j + 1] = x.w;
                }
                rotary_turn_slot(k, cs, sn, p.interleaved);
            }
        } else {
            for (int j = 0; j < 16; ++j)
                k[j] = key_component(p, xk + chunk * dt * p.xs[0][2], 16 * slot + j, (int)(pg.lo + pg.s0 + i + chunk * dt));
        }
    };
    int turn = 0;

    for (int h = h0; h < h1; ++h) {
        float k[16];
        Raw16 v;
        uint32_t mk = 0, mv = 0;
#pragma unroll
        for (int chunk = 0; chunk < CHUNKS; ++chunk) {
            if (TWO || (!AHEAD && h > h0)) load(chunk);
            if (i + chunk * dt < n_new) {
                v = rv;
                key(chunk, k);
                mk = max(mk, key_amax(k));
                mv = max(mv, value_amax(v));
            }
        }
        if (AHEAD) {
            xk += p.xs[0][1];
            xv += p.xs[1][1];
            if (h + 1 < h1) load(0);
        }
        // the maximum of the block.  Its place was last read a barrier ago when it is cleared, and is
        // next used after the following barrier.
        auto block_max = [&]() {
            mk = __reduce_max_sync(0xffffffffu, mk);
            mv = __reduce_max_sync(0xffffffffu, mv);
            if ((threadIdx.x & 31) == 0) {
                atomicMax(&s_max[turn][0], mk);
                atomicMax(&s_max[turn][1], mv);
            }
            __syncthreads();
            mk = s_max[turn][0];
            mv = s_max[turn][1];
            const int before = turn == 0 ? 2 : turn - 1;
            if (threadIdx.x == 0) s_max[before][0] = s_max[before][1] = 0;
            turn = turn == 2 ? 0 : turn + 1;
        };
        // read by all before thread 0 writes them
        const float before_k = pg.s0 > 0 ? c.k_scale[unit] : 0.f, before_v = pg.s0 > 0 ? c.v_scale[unit] : 0.f;
        block_max();
        const bool special_k = mk >= kInfBits, special_v = mv >= kInfBits;
        if (special_k || special_v) {  // rare; the same for the whole block
            mk = mv = 0;
#pragma unroll
            for (int chunk = 0; chunk < CHUNKS; ++chunk) {
                if (i + chunk * dt >= n_new) continue;
                if constexpr (TWO) {
                    load(chunk);
                    v = rv;
                    key(chunk, k);
                }
                float y[16];
                v.get(y);
                mk = max(mk, amax_finite(k));
                mv = max(mv, amax_finite(y));
            }
            block_max();
        }
        const ScaleUpdate uk = update_scale(pg.s0 > 0, before_k, mk), uv = update_scale(pg.s0 > 0, before_v, mv);
#pragma unroll
        for (int chunk = 0; chunk < CHUNKS; ++chunk) {
            if (i + chunk * dt >= n_new) continue;
            if constexpr (TWO) {
                load(chunk);
                v = rv;
                key(chunk, k);
            }
            float y[16];
            v.get(y);
            store_slot(c.k + off + chunk * dt * c.d, at, k, uk.inv, special_k);
            store_slot(c.v + off + chunk * dt * c.d, plain_slot(slot), y, uv.inv, special_v);
        }
        // the tokens from before, by exact ratios for powers of two
        if (uk.grows) rescale_codes(c.k + (long long)unit * c.page * c.d, pg.s0 * per_row, before_k * uk.inv);
        if (uv.grows) rescale_codes(c.v + (long long)unit * c.page * c.d, pg.s0 * per_row, before_v * uv.inv);
        if (threadIdx.x == 0) {
            if (pg.s0 == 0 || uk.grows) c.k_scale[unit] = uk.now;
            if (pg.s0 == 0 || uv.grows) c.v_scale[unit] = uv.now;
        }
        if (!AHEAD) {
            xk += p.xs[0][1];
            xv += p.xs[1][1];
        }
        off += c.page * c.d;
        ++unit;
    }
}

// The same for so few tokens that a warp holds them (N * d / 16 <= 32): one warp per
// (sequence, head), lane (token, slot).  Bound by latency: one token for each of 64 sequences, 8 heads of
// d = 128, turned, 3.8 us; a block for each page and head took 12 us.
constexpr int kFewWarps = 4;
__global__ void __launch_bounds__(32 * kFewWarps) fa_cache_append_few_kernel(const __grid_constant__ AppendParams p) {
    const CacheView &c = p.c;
    const int lane = threadIdx.x & 31;
    const long long unit_i = (long long)blockIdx.x * kFewWarps + (threadIdx.x >> 5);
    const int b = (int)(unit_i / c.H_kv), h = (int)(unit_i - (long long)b * c.H_kv);
    if (b >= c.B) return;
    const int per_row = c.d >> 4, row_log2 = 31 - __clz(per_row);
    const int i = lane >> row_log2, slot = lane & (per_row - 1);  // new token i
    const RotarySlot at = rotary_slot(slot, c.d, p.dim);
    float k[16], v[16];
    Raw16 w;
#pragma unroll
    for (int j = 0; j < 16; ++j) k[j] = 0.f, w.w[j >> 1] = 0;
    const int start = p.start[b];
    const int n = max(0, min(p.n_new ? p.n_new[b] : p.N, p.N));
    if (i < n) {
        const uint16_t *xk = p.x[0] + b * p.xs[0][0] + h * p.xs[0][1] + i * p.xs[0][2];
        const uint16_t *xv = p.x[1] + b * p.xs[1][0] + h * p.xs[1][1] + i * p.xs[1][2];
        load8(xk + at.a, k);
        load8(xk + at.b, k + 8);
        w.load(xv, plain_slot(slot));
        if (at.rotated) {
            const int pos = (int)((unsigned)start + i);  // (past the table where this wraps)
            float cs[8], sn[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) rotary_cs(p.step[rotary_pair(slot, j, p.dim, p.interleaved)], pos, p.amplitude, 1.f, cs[j], sn[j]);
            rotary_turn_slot(k, cs, sn, p.interleaved);
        }
    }
    w.get(v);
    const bool first_of_seq = h == 0 && lane == 0;
    for (int pt = 0; pt < p.pages; ++pt) {
        Touched pg;
        if (!touched_page(p, b, pt, first_of_seq, pg)) continue;
        const int t = i < n ? (int)((long long)start + i - pg.lo) : -1;  // this lane's slot in the page
        const bool here = t >= pg.s0 && t < pg.s1;
        const long long unit = (long long)pg.page_id * c.H_kv + h;
        const float before_k = pg.s0 > 0 ? c.k_scale[unit] : 0.f, before_v = pg.s0 > 0 ? c.v_scale[unit] : 0.f;
        uint32_t mk = __reduce_max_sync(0xffffffffu, here ? key_amax(k) : 0u);
        uint32_t mv = __reduce_max_sync(0xffffffffu, here ? value_amax(w) : 0u);
        const bool special_k = mk >= kInfBits, special_v = mv >= kInfBits;
        if (special_k || special_v) {
            mk = __reduce_max_sync(0xffffffffu, here ? amax_finite(k) : 0u);
            mv = __reduce_max_sync(0xffffffffu, here ? amax_finite(v) : 0u);
        }
        const ScaleUpdate uk = update_scale(pg.s0 > 0, before_k, mk), uv = update_scale(pg.s0 > 0, before_v, mv);
        uint8_t *ck = c.k + unit * c.page * c.d, *cvv = c.v + unit * c.page * c.d;
        if (here) {
            store_slot(ck + t * c.d, at, k, uk.inv, special_k);
            store_slot(cvv + t * c.d, plain_slot(slot), v, uv.inv, special_v);
        }
        if (uk.grows)
            for (int r = lane; r < pg.s0 * per_row; r += 32) rescale_run(ck + 16 * r, before_k * uk.inv);
        if (uv.grows)
            for (int r = lane; r < pg.s0 * per_row; r += 32) rescale_run(cvv + 16 * r, before_v * uv.inv);
        if (lane == 0) {
            if (pg.s0 == 0 || uk.grows) c.k_scale[unit] = uk.now;
            if (pg.s0 == 0 || uv.grows) c.v_scale[unit] = uv.now;
        }
    }
}

// ---------------------------------------------------------------- gather
struct GatherParams {
    CacheView c;
    const int32_t *k_len;
    uint16_t *k, *v;
    int N_k;
    int row_blocks;             // blocks for the rows of one (sequence, head)
    int32_t *status;
};

constexpr int kGatherThreads = 256;
constexpr int kGatherItems = 4;  // runs of 8 codes a thread has in flight, of K and of V

// 8 codes times scale as bf16.
__device__ __forceinline__ void gather_store(uint16_t *dst, uint2 w, float scale) {
    float v[8];
    values4(w.x, v);
    values4(w.y, v + 4);
    *reinterpret_cast<uint4 *>(dst) =
        make_uint4(pack_bf16x2(v[0] * scale, v[1] * scale), pack_bf16x2(v[2] * scale, v[3] * scale),
                   pack_bf16x2(v[4] * scale, v[5] * scale), pack_bf16x2(v[6] * scale, v[7] * scale));
}

// Bound by memory: 1 byte read and 2 written per component.  One thread takes
// runs of 8 components of one (sequence, head), of the keys and the values at
// the same place (they share the page lookup), so that a warp's stores are 512 bytes in
// one piece; all its loads are issued before its stores.  Measured: 4 sequences of up to 32768 tokens, 8
// heads of d = 128 (727 MB), 116 us or 6.2 TB/s; 16 codes a lane, with stores 32 bytes apart, took 146 us.
__global__ void __launch_bounds__(kGatherThreads) fa_cache_gather_kernel(const __grid_constant__ GatherParams p) {
    const CacheView &c = p.c;
    const int bh = blockIdx.x / p.row_blocks, part = blockIdx.x - bh * p.row_blocks;
    const int b = bh / c.H_kv, h = bh - b * c.H_kv;
    const int runs = c.d >> 3, runs_log2 = 31 - __clz(runs);
    const long long cap = (long long)c.max_pages << c.page_log2;
    const int len = (int)min((long long)max(p.k_len[b], 0), cap);
    const int row0 = part * (kGatherThreads * kGatherItems / runs);  // below N_k
    const int32_t *table = c.table + b * c.table_stride;
    uint2 kw[kGatherItems], vw[kGatherItems];
    float ks[kGatherItems], vs[kGatherItems];
#pragma unroll
    for (int i = 0; i < kGatherItems; ++i) {
        const int k = threadIdx.x + i * kGatherThreads;
        const long long n = (long long)row0 + (k >> runs_log2);
        const int run = k & (runs - 1);
        kw[i] = vw[i] = make_uint2(0, 0);
        ks[i] = vs[i] = 0.f;
        if (n >= p.N_k || n >= len) continue;
        const int page_id = table[n >> c.page_log2];
        if (page_id < 0 || page_id >= c.n_pages) {
            if (run == 0) report_bad_page(p.status);
            continue;
        }
        const long long unit = (long long)page_id * c.H_kv + h;
        const long long off = (unit * c.page + (n & (c.page - 1))) * c.d + 8 * run;
        kw[i] = __ldcs(reinterpret_cast<const uint2 *>(c.k + off));
        vw[i] = __ldcs(reinterpret_cast<const uint2 *>(c.v + off));
        ks[i] = c.k_scale[unit];
        vs[i] = c.v_scale[unit];
    }
#pragma unroll
    for (int i = 0; i < kGatherItems; ++i) {
        const int k = threadIdx.x + i * kGatherThreads;
        const long long n = (long long)row0 + (k >> runs_log2);
        if (n >= p.N_k) continue;
        const long long off = ((long long)bh * p.N_k + n) * c.d + 8 * (k & (runs - 1));
        gather_store(p.k + off, kw[i], ks[i]);
        gather_store(p.v + off, vw[i], vs[i]);
    }
}

}  // namespace fa
