// fa_rope.cu -- rotary positions: the table (fa_rotary_init) and the kernels
// of fa_rope.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "fa.h"
#include "fa_internal.h"
#include "fa_rotary.cuh"

namespace fa {

struct RopeTensor {
    const void *x;
    void *y;
    long long xs[3], ys[3];
};

struct RopeParams {
    RopeTensor t[2];
    int heads0, heads;  // heads of t[0], and of both together
    int N, d, dim;
    int rows;           // B * N
    int interleaved;
    int chunk;          // heads that one thread handles
    const int32_t *pos;
    long long pos_stride;
    int pos0;
    float amplitude, sign;
    int copy_tail;      // 0: in place, the components from dim on are there already
    uint64_t step[FA_ROTARY_MAX_DIM / 2];
};

constexpr int kRopeThreads = 256;

template <typename T>
__device__ __forceinline__ const T *rope_src(const RopeParams &p, int h, int b, int n) {
    const RopeTensor &t = p.t[h >= p.heads0];
    return static_cast<const T *>(t.x) + b * t.xs[0] + (h >= p.heads0 ? h - p.heads0 : h) * t.xs[1] + n * t.xs[2];
}
template <typename T>
__device__ __forceinline__ T *rope_dst(const RopeParams &p, int h, int b, int n) {
    const RopeTensor &t = p.t[h >= p.heads0];
    return static_cast<T *>(t.y) + b * t.ys[0] + (h >= p.heads0 ? h - p.heads0 : h) * t.ys[1] + n * t.ys[2];
}

// A slot's 16 components as they are read: kept so while their loads are in flight, which takes half
// the registers of fp32 for bf16.
template <typename T> struct RawSlot;
template <> struct RawSlot<uint16_t> {
    uint4 a, b;
    __device__ __forceinline__ void load(const uint16_t *x, const RotarySlot &at) {
        a = *reinterpret_cast<const uint4 *>(x + at.a);
        b = *reinterpret_cast<const uint4 *>(x + at.b);
    }
    __device__ __forceinline__ void get(float (&v)[16]) const {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) v[2 * i] = bf16x2_lo(w[i]), v[2 * i + 1] = bf16x2_hi(w[i]);
    }
};
template <> struct RawSlot<float> {
    float4 a[4];
    __device__ __forceinline__ void load(const float *x, const RotarySlot &at) {
        a[0] = reinterpret_cast<const float4 *>(x + at.a)[0];
        a[1] = reinterpret_cast<const float4 *>(x + at.a)[1];
        a[2] = reinterpret_cast<const float4 *>(x + at.b)[0];
        a[3] = reinterpret_cast<const float4 *>(x + at.b)[1];
    }
    __device__ __forceinline__ void get(float (&v)[16]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * i] = a[i].x, v[4 * i + 1] = a[i].y, v[4 * i + 2] = a[i].z, v[4 * i + 3] = a[i].w;
    }
};

// Bound by memory: every component is read once and written once.  One thread
// has one slot (16 components) of one token and walks over `chunk` heads, so
// that the 8 sines and cosines, which the heads share, are computed once for
// all of them (they cost about as much as turning 4 heads); it has UN heads'
// loads in flight.  The lanes of a warp lie along the components and then
// along the tokens: whole 128-byte lines whichever way the strides run.
// Measured: bf16 32 + 8 heads of 2 x 8192 tokens, d = 128, 58 us or 5.8 TB/s (64 registers, of which the compiler
// spills 64 bytes; 4 heads in flight with 80: 64 us; 16 or 20 heads a thread: 60); fp32 to bf16, 16 + 16 heads of 2 x 4097
// tokens, half of d turned, 34 us or 6.0 TB/s (2 heads in flight: 38).
template <typename TI, typename TO>
__global__ void __launch_bounds__(kRopeThreads, sizeof(TI) == 2 ? 4 : 2)
fa_rope_kernel(const __grid_constant__ RopeParams p) {
    __shared__ uint64_t step[FA_ROTARY_MAX_DIM / 2];
    if (threadIdx.x < (p.dim >> 1)) step[threadIdx.x] = p.step[threadIdx.x];
    __syncthreads();
    const int slots = p.d >> 4, per_block = kRopeThreads / slots;
    const int r = threadIdx.x / slots, slot = threadIdx.x - r * slots;
    const long long row = (long long)blockIdx.x * per_block + r;
    if (r >= per_block || row >= p.rows) return;
    const RotarySlot at = rotary_slot(slot, p.d, p.dim);
    if (!at.rotated && !p.copy_tail) return;
    const int b = (int)row / p.N, n = (int)row - b * p.N;
    float c[8], s[8];
    if (at.rotated) {
        const int pos = p.pos ? p.pos[b * p.pos_stride + n] : p.pos0 + n;
#pragma unroll
        for (int j = 0; j < 8; ++j) rotary_cs(step[rotary_pair(slot, j, p.dim, p.interleaved)], pos, p.amplitude, p.sign, c[j], s[j]);
    }
    constexpr int UN = sizeof(TI) == 2 ? 2 : 4;
    const int h0 = blockIdx.y * p.chunk, h1 = min(h0 + p.chunk, p.heads);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const RopeTensor &t = p.t[i];
        const int off = i ? p.heads0 : 0;  // head h of the call is head h - off of the tensor
        const int lo = max(h0, off) - off, hi = (i ? h1 : min(h1, p.heads0)) - off;
        if (lo >= hi) continue;
        const TI *x = static_cast<const TI *>(t.x) + b * t.xs[0] + lo * t.xs[1] + n * t.xs[2];
        TO *y = static_cast<TO *>(t.y) + b * t.ys[0] + lo * t.ys[1] + n * t.ys[2];
        for (int h = lo; h < hi; h += UN) {
            RawSlot<TI> raw[UN];
#pragma unroll
            for (int u = 0; u < UN; ++u)
                if (h + u < hi) raw[u].load(x + u * t.xs[1], at);
#pragma unroll
            for (int u = 0; u < UN; ++u)
                if (h + u < hi) {
                    float v[16];
                    raw[u].get(v);
                    if (at.rotated) rotary_turn_slot(v, c, s, p.interleaved);
                    store8(y + u * t.ys[1] + at.a, v);
                    store8(y + u * t.ys[1] + at.b, v + 8);
                }
            x += UN * t.xs[1];
            y += UN * t.ys[1];
        }
    }
}

// Any dim, alignment and strides: one thread has one pair (or one component
// past dim) of one token and head, element by element.  Not made for speed: a sine and cosine for every
// head and 2-byte accesses.  Measured: 16 + 16 heads of 2 x 4096 tokens in bf16, 20 of 80 components turned, 134 us (84 MB, 13 us at
// the copy rate), 24 of 96 156 us; 32 of 128, which the kernel above takes, 26 us.
template <typename TI, typename TO>
__global__ void __launch_bounds__(kRopeThreads) fa_rope_any_kernel(const __grid_constant__ RopeParams p) {
    const int items = (p.dim >> 1) + (p.copy_tail ? p.d - p.dim : 0);
    const long long total = (long long)p.rows * p.heads * items;
    for (long long k = (long long)blockIdx.x * kRopeThreads + threadIdx.x; k < total;
         k += (long long)gridDim.x * kRopeThreads) {
        const long long rh = k / items;
        const int item = (int)(k - rh * items);
        const int h = (int)(rh % p.heads);
        const int row = (int)(rh / p.heads), b = row / p.N, n = row - b * p.N;
        const TI *x = rope_src<TI>(p, h, b, n);
        TO *y = rope_dst<TO>(p, h, b, n);
        if (item < (p.dim >> 1)) {
            const int pos = p.pos ? p.pos[b * p.pos_stride + n] : p.pos0 + n;
            const int ia = p.interleaved ? 2 * item : item, ib = p.interleaved ? ia + 1 : ia + (p.dim >> 1);
            float c, s, u = load1(x + ia), w = load1(x + ib);
            rotary_cs(p.step[item], pos, p.amplitude, p.sign, c, s);
            rotary_turn(u, w, c, s);
            store1(y + ia, u);
            store1(y + ib, w);
        } else {
            const int e = p.dim + item - (p.dim >> 1);
            store1(y + e, load1(x + e));
        }
    }
}

}  // namespace fa

namespace {

int elem_bytes(int dtype) { return dtype == FA_T_F32 ? 4 : 2; }

// Strides of whole 16 bytes (of the dimensions that have more than one entry)
// from a 16-byte aligned base.
bool vectors(const void *base, const int64_t *stride, int B, int heads, int N, int bytes) {
    const int n[3] = {B, heads, N};
    if (!fa_detail::aligned(base, 16)) return false;
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && (stride[i] * bytes) % 16 != 0) return false;
    return true;
}

template <typename TI, typename TO>
void launch_rope(const fa::RopeParams &kp, bool vec, int num_sms, cudaStream_t s) {
    if (vec) {
        const int per_block = fa::kRopeThreads / (kp.d >> 4);
        const dim3 grid((unsigned)((kp.rows + per_block - 1) / per_block), (unsigned)((kp.heads + kp.chunk - 1) / kp.chunk));
        fa::fa_rope_kernel<TI, TO><<<grid, fa::kRopeThreads, 0, s>>>(kp);
    } else {
        const long long total = (long long)kp.rows * kp.heads * kp.d;
        long long blocks = (total + fa::kRopeThreads - 1) / fa::kRopeThreads;
        if (blocks > 16LL * num_sms) blocks = 16LL * num_sms;
        fa::fa_rope_any_kernel<TI, TO><<<(unsigned)blocks, fa::kRopeThreads, 0, s>>>(kp);
    }
}

}  // namespace

namespace fa_detail {

fa_status validate_rotary(const fa_rotary *r, int d) {
    if (!r || r->ready != 1) return FA_ERR_INVALID_ARGUMENT;
    if (r->dim < 2 || r->dim > FA_ROTARY_MAX_DIM || (r->dim & 1) || r->dim > d) return FA_ERR_INVALID_ARGUMENT;
    if (r->layout != FA_ROTARY_HALF && r->layout != FA_ROTARY_INTERLEAVED) return FA_ERR_INVALID_ARGUMENT;
    return FA_OK;
}

}  // namespace fa_detail

extern "C" {

fa_status fa_rotary_init(fa_rotary *r, const fa_rotary_spec *sp) {
    if (!r || !sp) return FA_ERR_INVALID_ARGUMENT;
    if (sp->dim < 2 || sp->dim > FA_ROTARY_MAX_DIM || (sp->dim & 1)) return FA_ERR_INVALID_ARGUMENT;
    if (sp->layout != FA_ROTARY_HALF && sp->layout != FA_ROTARY_INTERLEAVED) return FA_ERR_INVALID_ARGUMENT;
    // as the kernels hold it: what fp32 makes an infinity, or 0 of something else, is refused too
    const float amplitude = sp->amplitude == 0.0 ? 1.f : (float)sp->amplitude;
    if (!std::isfinite(amplitude) || amplitude <= 0.f) return FA_ERR_INVALID_ARGUMENT;
    const long double two_pi = 6.283185307179586476925286766559L;
    long double w[FA_ROTARY_MAX_DIM / 2];
    if (sp->angles) {
        for (int i = 0; i < sp->dim / 2; ++i) {
            if (!(std::fabs(sp->angles[i]) <= 1048576.0)) return FA_ERR_INVALID_ARGUMENT;
            w[i] = sp->angles[i];
        }
    } else {
        if (!std::isfinite(sp->base) || sp->base <= 0.0) return FA_ERR_INVALID_ARGUMENT;
        if (sp->scaling < FA_ROTARY_NONE || sp->scaling > FA_ROTARY_PARTS) return FA_ERR_INVALID_ARGUMENT;
        if (sp->scaling != FA_ROTARY_NONE && !(std::isfinite(sp->factor) && sp->factor > 0.0))
            return FA_ERR_INVALID_ARGUMENT;
        if (sp->scaling == FA_ROTARY_BASE && sp->dim == 2) return FA_ERR_INVALID_ARGUMENT;
        if (sp->scaling == FA_ROTARY_PARTS &&
            !(std::isfinite(sp->original_length) && sp->original_length > 0.0 && sp->low_turns >= 0.0 &&
              sp->high_turns > sp->low_turns && std::isfinite(sp->high_turns)))
            return FA_ERR_INVALID_ARGUMENT;
        long double base = sp->base;
        if (sp->scaling == FA_ROTARY_BASE)
            base *= std::pow((long double)sp->factor, (long double)sp->dim / (sp->dim - 2));
        for (int i = 0; i < sp->dim / 2; ++i) {
            long double a = std::pow(base, -2.0L * i / sp->dim);
            if (sp->scaling == FA_ROTARY_LINEAR) a /= sp->factor;
            if (sp->scaling == FA_ROTARY_PARTS) {
                const long double turns = sp->original_length * a / two_pi;
                long double keep = (turns - sp->low_turns) / ((long double)sp->high_turns - sp->low_turns);
                keep = keep < 0 ? 0 : (keep > 1 ? 1 : keep);
                a = keep * a + (1 - keep) * a / sp->factor;
            }
            if (!(std::fabs(a) <= 1048576.0L)) return FA_ERR_INVALID_ARGUMENT;  // base far below 1
            w[i] = a;
        }
    }
    std::memset(r, 0, sizeof *r);
    r->dim = sp->dim;
    r->layout = sp->layout;
    r->amplitude = amplitude;
    for (int i = 0; i < sp->dim / 2; ++i) {
        long double t = w[i] / two_pi;
        t -= std::floor(t);
        t = std::floor(t * 18446744073709551616.0L + 0.5L);
        r->step[i] = t >= 18446744073709551616.0L ? 0 : (uint64_t)t;
    }
    r->ready = 1;
    return FA_OK;
}

fa_status fa_rope(const fa_rope_params *p, void *stream) {
    if (!p || p->B < 0 || p->N < 0 || p->t[0].heads < 0 || p->t[1].heads < 0) return FA_ERR_INVALID_ARGUMENT;
    if ((p->x_dtype != FA_T_BF16 && p->x_dtype != FA_T_F32) || (p->y_dtype != FA_T_BF16 && p->y_dtype != FA_T_F32))
        return FA_ERR_INVALID_ARGUMENT;
    if (p->inverse != 0 && p->inverse != 1) return FA_ERR_INVALID_ARGUMENT;
    if (p->d < 2 || p->d > FA_ROPE_MAX_D) return FA_ERR_UNSUPPORTED;
    fa_status st = fa_detail::validate_rotary(p->rotary, p->d);
    if (st != FA_OK) return st;
    const long long rows = (long long)p->B * p->N, heads = (long long)p->t[0].heads + p->t[1].heads;
    if (rows == 0 || heads == 0) return FA_OK;
    // rows are counted in 32 bits, with those that a last block has no work for
    if (rows > 0x7fffffffLL - (fa::kRopeThreads - 1) || heads > 65535) return FA_ERR_INVALID_ARGUMENT;
    const int xb = elem_bytes(p->x_dtype), yb = elem_bytes(p->y_dtype);
    bool vec = p->d % 16 == 0 && p->rotary->dim % 16 == 0;
    int in_place = 0, present = 0;
    for (const fa_rope_tensor &t : p->t) {
        if (t.heads == 0) continue;
        if (!t.x || !t.y) return FA_ERR_INVALID_ARGUMENT;
        if (!fa_detail::aligned(t.x, xb) || !fa_detail::aligned(t.y, yb)) return FA_ERR_MISALIGNED;
        vec = vec && vectors(t.x, t.x_stride, p->B, t.heads, p->N, xb) &&
              vectors(t.y, t.y_stride, p->B, t.heads, p->N, yb);
        ++present;
        const int n[3] = {p->B, t.heads, p->N};
        for (int i = 0; i < 3; ++i)
            if (n[i] > 1 && t.y_stride[i] == 0) return FA_ERR_INVALID_ARGUMENT;  // several results for one place
        if (t.x == t.y) {
            if (p->x_dtype != p->y_dtype) return FA_ERR_INVALID_ARGUMENT;
            for (int i = 0; i < 3; ++i)
                if (n[i] > 1 && t.x_stride[i] != t.y_stride[i]) return FA_ERR_INVALID_ARGUMENT;
            ++in_place;
        }
    }
    if (!p->pos && (long long)p->pos0 + p->N - 1 > 0x7fffffffLL) return FA_ERR_INVALID_ARGUMENT;
    if (!fa_detail::aligned(p->pos, 4)) return FA_ERR_MISALIGNED;
    int dev = 0, num_sms = 0;
    if ((st = fa_detail::current_device(&dev, &num_sms)) != FA_OK) return st;

    fa::RopeParams kp;
    std::memset(&kp, 0, sizeof kp);
    for (int i = 0; i < 2; ++i) {
        kp.t[i].x = p->t[i].x;
        kp.t[i].y = p->t[i].y;
        for (int j = 0; j < 3; ++j) {
            kp.t[i].xs[j] = p->t[i].x_stride[j];
            kp.t[i].ys[j] = p->t[i].y_stride[j];
        }
    }
    kp.heads0 = p->t[0].heads;
    kp.heads = (int)heads;
    kp.N = p->N;
    kp.d = p->d;
    kp.dim = p->rotary->dim;
    kp.rows = (int)rows;
    kp.interleaved = p->rotary->layout == FA_ROTARY_INTERLEAVED;
    kp.pos = p->pos;
    kp.pos_stride = p->pos_stride;
    kp.pos0 = p->pos0;
    kp.amplitude = p->rotary->amplitude;
    kp.sign = p->inverse ? -1.f : 1.f;
    kp.copy_tail = in_place < present;
    std::memcpy(kp.step, p->rotary->step, sizeof(uint64_t) * (kp.dim / 2));
    // heads for each thread: 8, so that the sines are shared, as long as that
    // leaves every SM 1024 threads; else fewer
    kp.chunk = 8;
    while (kp.chunk > 1 && rows * (p->d / 16) * ((heads + kp.chunk - 1) / kp.chunk) < 1024LL * num_sms) kp.chunk >>= 1;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (p->x_dtype == FA_T_BF16)
        p->y_dtype == FA_T_BF16 ? launch_rope<uint16_t, uint16_t>(kp, vec, num_sms, s)
                                : launch_rope<uint16_t, float>(kp, vec, num_sms, s);
    else
        p->y_dtype == FA_T_BF16 ? launch_rope<float, uint16_t>(kp, vec, num_sms, s)
                                : launch_rope<float, float>(kp, vec, num_sms, s);
    return cudaPeekAtLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
