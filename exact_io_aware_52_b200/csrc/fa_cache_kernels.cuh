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
    const int32_t *start, *n_new;
    int32_t *status;
    int dim, interleaved;       // dim 0: keys are not turned
    float amplitude;
    uint64_t step[FA_ROTARY_MAX_DIM / 2];
};

constexpr int kMinScaleExp = -100;

// 2^e with the least e >= kMinScaleExp such that amax <= 448 * 2^e, for a finite
// amax >= 0: with amax = m * 2^E, 1 <= m < 2, and 448 = 1.75 * 2^8, e is E - 8
// where m <= 1.75 and E - 7 else.  E comes from the exponent field (a
// subnormal amax gives E = -127, under the limit either way).
__device__ __forceinline__ float page_scale(float amax) {
    const uint32_t u = __float_as_uint(amax);
    int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u);
    e = max(e, kMinScaleExp);
    return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Four values times inv as E4M3 codes; infinities and NaN give the code NaN
// (v * 0 is NaN for them and 0 for the others; the conversion would saturate
// an infinity).
__device__ __forceinline__ uint32_t codes4(const float *v, float inv) {
    return pack_e4m3x4(fmaf(v[0], inv, v[0] * 0.f), fmaf(v[1], inv, v[1] * 0.f), fmaf(v[2], inv, v[2] * 0.f),
                       fmaf(v[3], inv, v[3] * 0.f));
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

// One component of a key, turned, for layouts that do not fall into slots.
__device__ __forceinline__ float turned_component(const AppendParams &p, const uint64_t *step, const uint16_t *x, int e,
                                                  int pos) {
    const float v = load1(x + e);
    if (e >= p.dim) return v;
    const int half = p.dim >> 1;
    const int i = p.interleaved ? e >> 1 : (e < half ? e : e - half);
    const bool first = p.interleaved ? !(e & 1) : e < half;
    float a, b, c, s;
    a = first ? v : load1(x + (p.interleaved ? e - 1 : e - half));
    b = first ? load1(x + (p.interleaved ? e + 1 : e + half)) : v;
    rotary_cs(step[i], pos, p.amplitude, 1.f, c, s);
    rotary_turn(a, b, c, s);
    return first ? a : b;
}

// One block per (sequence, touched page, head, K or V).  Bound by memory: 2
// bytes read and 1 written per component.  The page's new values stay in
// registers between the maximum and the rounding (SPT slots of 16 components
// a thread), so they are read once; the block owns the page, so the scale needs
// no atomics and the result no order.
template <int SPT, bool VEC>
__global__ void __launch_bounds__(512) fa_cache_append_kernel(const __grid_constant__ AppendParams p) {
    __shared__ uint64_t step[FA_ROTARY_MAX_DIM / 2];
    __shared__ uint32_t s_max[16];
    const CacheView &c = p.c;
    const int kv = blockIdx.x & 1;
    int u = blockIdx.x >> 1;
    const int h = u % c.H_kv;
    u /= c.H_kv;
    const int pt = u % p.pages, b = u / p.pages;

    const int start = p.start[b];
    int n = p.n_new ? p.n_new[b] : p.N;
    n = n < 0 ? 0 : (n > p.N ? p.N : n);
    if (n == 0) return;
    if (start < 0) {
        if (threadIdx.x == 0) report_bad_page(p.status);
        return;
    }
    const long long first = start, end = first + n;                 // positions
    const long long page_i = (first >> c.page_log2) + pt;
    const long long lo = page_i << c.page_log2;                     // the page's first position
    if (lo >= end) return;
    const int page_id = page_i < c.max_pages ? c.table[b * c.table_stride + page_i] : -1;
    if (page_id < 0 || page_id >= c.n_pages) {
        if (threadIdx.x == 0) report_bad_page(p.status);
        return;
    }
    const int s0 = first > lo ? (int)(first - lo) : 0;              // new tokens are in slots [s0, s1)
    const int s1 = end - lo < c.page ? (int)(end - lo) : c.page;
    const int dim = kv ? 0 : p.dim;
    if (dim) {
        for (int i = threadIdx.x; i < (dim >> 1); i += blockDim.x) step[i] = p.step[i];
        __syncthreads();
    }

    const int per_row = c.d >> 4;                                   // slots of 16 components in a token
    const uint16_t *x = p.x[kv] + b * p.xs[kv][0] + h * p.xs[kv][1];
    float v[SPT][16];
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < SPT; ++i) {
        const int k = threadIdx.x + i * blockDim.x;
        const int t = k / per_row, slot = k - t * per_row;
        if (t < s0 || t >= s1) continue;
        const int pos = (int)(lo + t);
        const uint16_t *row = x + (lo + t - first) * p.xs[kv][2];
        if constexpr (VEC) {
            const RotarySlot at = rotary_slot(slot, dim, p.interleaved);
            load8(row + at.a, v[i]);
            load8(row + at.b, v[i] + 8);
            if (at.rotated) {
                float cs[8], sn[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) rotary_cs(step[8 * slot + j], pos, p.amplitude, 1.f, cs[j], sn[j]);
                rotary_turn_slot(v[i], cs, sn, p.interleaved);
            }
        } else {
            for (int j = 0; j < 16; ++j)
                v[i][j] = dim ? turned_component(p, step, row, 16 * slot + j, pos) : load1(row + 16 * slot + j);
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const uint32_t m = __float_as_uint(v[i][j]) & 0x7fffffffu;
            if (m < 0x7f800000u) amax = max(amax, m);               // finite magnitudes order as their bits
        }
    }
    amax = __reduce_max_sync(0xffffffffu, amax);
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = amax;
    float *scale = (kv ? c.v_scale : c.k_scale) + (long long)page_id * c.H_kv + h;
    const float before = s0 > 0 ? *scale : 0.f;                     // read by all before thread 0 writes it
    __syncthreads();
    for (int i = 0; i < (int)(blockDim.x >> 5); ++i) amax = max(amax, s_max[i]);
    const float now = fmaxf(before, page_scale(__uint_as_float(amax)));
    const float inv = 1.f / now;
    uint8_t *codes = (kv ? c.v : c.k) + ((long long)page_id * c.H_kv + h) * c.page * c.d;
    const bool grows = s0 > 0 && now != before;
    const float ratio = before * inv;                               // exact for powers of two
#pragma unroll
    for (int i = 0; i < SPT; ++i) {
        const int k = threadIdx.x + i * blockDim.x;
        const int t = k / per_row, slot = k - t * per_row;
        if (t >= s1) continue;
        uint8_t *row = codes + t * c.d;
        if (t >= s0) {
            const RotarySlot at = rotary_slot(slot, VEC ? dim : 0, p.interleaved);
            *reinterpret_cast<uint2 *>(row + at.a) = make_uint2(codes4(v[i], inv), codes4(v[i] + 4, inv));
            *reinterpret_cast<uint2 *>(row + at.b) = make_uint2(codes4(v[i] + 8, inv), codes4(v[i] + 12, inv));
        } else if (grows) {
            uint4 w = *reinterpret_cast<const uint4 *>(row + 16 * slot);
            uint32_t *q = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float o[4];
                values4(q[j], o);
                q[j] = codes4(o, ratio);
            }
            *reinterpret_cast<uint4 *>(row + 16 * slot) = w;
        }
    }
    if (threadIdx.x == 0) *scale = now;
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
constexpr int kGatherItems = 4;  // 16-byte runs of codes a thread has in flight, of K and of V

// 16 codes times scale as bf16.
__device__ __forceinline__ void gather_store(uint16_t *dst, uint4 w, float scale) {
    const uint32_t q[4] = {w.x, w.y, w.z, w.w};
    uint32_t r[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float v[4];
        values4(q[j], v);
        r[2 * j] = pack_bf16x2(v[0] * scale, v[1] * scale);
        r[2 * j + 1] = pack_bf16x2(v[2] * scale, v[3] * scale);
    }
    reinterpret_cast<uint4 *>(dst)[0] = make_uint4(r[0], r[1], r[2], r[3]);
    reinterpret_cast<uint4 *>(dst)[1] = make_uint4(r[4], r[5], r[6], r[7]);
}

// Bound by memory: 1 byte read and 2 written per component.  One thread takes
// runs of 16 components of one (sequence, head), of the keys and the values at
// the same place (they share the page lookup); all its loads are issued before
// its stores.
__global__ void __launch_bounds__(kGatherThreads) fa_cache_gather_kernel(const __grid_constant__ GatherParams p) {
    const CacheView &c = p.c;
    const int bh = blockIdx.x / p.row_blocks, part = blockIdx.x - bh * p.row_blocks;
    const int b = bh / c.H_kv, h = bh - b * c.H_kv;
    const int runs = c.d >> 4;
    const long long cap = (long long)c.max_pages << c.page_log2;
    const long long len = min((long long)max(p.k_len[b], 0), cap);
    const int per_block = kGatherThreads * kGatherItems / runs;     // rows
    uint4 kw[kGatherItems], vw[kGatherItems];
    float ks[kGatherItems], vs[kGatherItems];
#pragma unroll
    for (int i = 0; i < kGatherItems; ++i) {
        const int k = threadIdx.x + i * kGatherThreads;
        const int r = k / runs, run = k - r * runs;
        const long long n = (long long)part * per_block + r;
        kw[i] = vw[i] = make_uint4(0, 0, 0, 0);
        ks[i] = vs[i] = 0.f;
        if (n >= p.N_k || n >= len) continue;
        const int page_id = c.table[b * c.table_stride + (n >> c.page_log2)];
        if (page_id < 0 || page_id >= c.n_pages) {
            if (run == 0) report_bad_page(p.status);
            continue;
        }
        const long long unit = (long long)page_id * c.H_kv + h;
        const long long off = (unit * c.page + (n & (c.page - 1))) * c.d + 16 * run;
        kw[i] = *reinterpret_cast<const uint4 *>(c.k + off);
        vw[i] = *reinterpret_cast<const uint4 *>(c.v + off);
        ks[i] = c.k_scale[unit];
        vs[i] = c.v_scale[unit];
    }
#pragma unroll
    for (int i = 0; i < kGatherItems; ++i) {
        const int k = threadIdx.x + i * kGatherThreads;
        const int r = k / runs, run = k - r * runs;
        const long long n = (long long)part * per_block + r;
        if (n >= p.N_k) continue;
        const long long off = ((long long)bh * p.N_k + n) * c.d + 16 * run;
        gather_store(p.k + off, kw[i], ks[i]);
        gather_store(p.v + off, vw[i], vs[i]);
    }
}

}  // namespace fa
