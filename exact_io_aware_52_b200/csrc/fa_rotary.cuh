// fa_rotary.cuh -- the rotation of rotary positions, shared by fa_rope and
// fa_cache_append.
//
// The angle of pair i at position p is p * w_i.  A float (or a double, for a
// far position and fast pairs) would lose its fraction of a turn, so the
// table holds w_i as a 64-bit fraction of a turn and the product p * step is
// taken modulo 2^64: the wrap-around drops the whole turns exactly, and the
// error left is |p| * 2^-65 turns (2^-34 at p = 2^31).  The product's high
// word is the angle.
#pragma once

#include <cstdint>

#include "sm100_ptx.cuh"

namespace fa {

// cos and sin of position * step, times the amplitude.  The angle's nearest quarter
// turn leaves at most an eighth of a turn x, where sin x = x + x^3 S(x^2) and
// cos x = 1 - x^2 / 2 + x^4 C(x^2) with S and C of degree 2, fitted for this file on [0, pi / 4] by Lawson's
// iteration (weighted least squares towards the least maximum error), S for the error relative to the sine, C for
// the absolute one of the cosine.  Rounded to fp32 the coefficients leave 2^-26.8 of the sine (2^-27.3 of 1) and 2^-30.9;
// with every step in fp32, from the 32-bit angle on, both err by at most 2^-23.2 of 1.
// About 30 instructions for both, two thirds of what sincospif takes.
__device__ __forceinline__ void rotary_cs(uint64_t step, int pos, float amplitude, float sign, float &c, float &s) {
    const uint32_t angle = (uint32_t)((step * (uint64_t)(int64_t)pos) >> 32);  // in 2^-32 turns
    const uint32_t quarter = (angle + 0x20000000u) >> 30;
    const float x = (float)(int32_t)(angle - (quarter << 30)) * 1.4629180792671596e-09f;  // 2 pi 2^-32
    const float t = x * x;
    const float sp = fmaf(fmaf(-0.00019515282474458218f, t, 0.00833216030150652f), t, -0.16666655242443085f);
    const float cp = fmaf(fmaf(2.4438451873720624e-05f, t, -0.001388736767694354f), t, 0.04166664555668831f);
    const float sx = fmaf(x * t, sp, x);
    const float cx = fmaf(fmaf(cp, t, -0.5f), t, 1.f);
    // quarter turns: (c, s) -> (c, s), (-s, c), (-c, -s), (s, -c)
    const float cq = (quarter & 1) ? sx : cx, sq = (quarter & 1) ? cx : sx;
    c = __uint_as_float(__float_as_uint(cq) ^ (((quarter + 1) & 2) << 30)) * amplitude;
    s = __uint_as_float(__float_as_uint(sq) ^ ((quarter & 2) << 30)) * (amplitude * sign);
}

// (a, b) -> (a c - b s, b c + a s), the products in fp32.
__device__ __forceinline__ void rotary_turn(float &a, float &b, float c, float s) {
    const float x = a, y = b;
    a = fmaf(x, c, -(y * s));
    b = fmaf(y, c, x * s);
}
// Two pairs at once: the same roundings in half the instructions.
__device__ __forceinline__ void rotary_turn2(float *a, float *b, const float *c, const float *s) {
    const float2 x = make_float2(a[0], a[1]), y = make_float2(b[0], b[1]);
    const float2 cc = make_float2(c[0], c[1]), ss = make_float2(s[0], s[1]);
    const float2 ys = __fmul2_rn(y, ss), xs = __fmul2_rn(x, ss);
    const float2 p = __ffma2_rn(x, cc, make_float2(-ys.x, -ys.y)), q = __ffma2_rn(y, cc, xs);
    a[0] = p.x, a[1] = p.y, b[0] = q.x, b[1] = q.y;
}

// A head's components are handled in slots of 16: two runs of 8 components
// that hold whole pairs, so that one thread reads, turns and writes a slot by
// itself.  Needs d and dim to be multiples of 16.  The runs of neighbouring slots lie
// side by side, those of a rotated slot s < dim / 16 at 8 s and 8 s + dim / 2, those of the
// others likewise in what is left of the head: lanes along the slots read and write
// whole lines.  With the half layout a rotated slot has the pairs 8 s + j, with the
// interleaved one pairs 4 s + j and dim / 4 + 4 s + j, j < 4.
struct RotarySlot {
    int a, b;      // first component of each run
    bool rotated;
};
__device__ __forceinline__ RotarySlot rotary_slot(int s, int d, int dim) {
    RotarySlot r;
    r.rotated = s < (dim >> 4);
    const int first = r.rotated ? 0 : dim, size = r.rotated ? dim : d - dim;
    r.a = first + 8 * (s - (first >> 4));
    r.b = r.a + (size >> 1);
    return r;
}
// The pair that entry j of a rotated slot's sines and cosines belongs to.
__device__ __forceinline__ int rotary_pair(int s, int j, int dim, bool interleaved) {
    return interleaved ? 4 * s + (j & 3) + (j >> 2) * (dim >> 2) : 8 * s + j;
}

// Turns a slot's 16 components in place: pair j is (v[j], v[8 + j]) or (v[2 j], v[2 j + 1]).
__device__ __forceinline__ void rotary_turn_slot(float (&v)[16], const float (&c)[8], const float (&s)[8],
                                                 bool interleaved) {
    if (interleaved) {
#pragma unroll
        for (int j = 0; j < 8; ++j) rotary_turn(v[2 * j], v[2 * j + 1], c[j], s[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; j += 2) rotary_turn2(v + j, v + 8 + j, c + j, s + j);
    }
}

// 8 components at p (16-byte aligned for bf16, 32 bytes read for fp32).
__device__ __forceinline__ void load8(const uint16_t *p, float *v) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    v[0] = bf16x2_lo(u.x), v[1] = bf16x2_hi(u.x), v[2] = bf16x2_lo(u.y), v[3] = bf16x2_hi(u.y);
    v[4] = bf16x2_lo(u.z), v[5] = bf16x2_hi(u.z), v[6] = bf16x2_lo(u.w), v[7] = bf16x2_hi(u.w);
}
__device__ __forceinline__ void load8(const float *p, float *v) {
    const float4 x = *reinterpret_cast<const float4 *>(p), y = *reinterpret_cast<const float4 *>(p + 4);
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
}
__device__ __forceinline__ void store8(uint16_t *p, const float *v) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                               pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float *p, const float *v) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ float load1(const uint16_t *p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ void store1(uint16_t *p, float v) { *p = (uint16_t)pack_bf16x2(v, 0.f); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }

}  // namespace fa
