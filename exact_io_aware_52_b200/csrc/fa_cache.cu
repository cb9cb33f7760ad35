// fa_cache.cu -- the paged 8-bit key/value cache: argument checks and launches
// of fa_cache_append, fa_cache_gather and fa_cache_attn.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "fa.h"
#include "fa_cache_attn_kernel.cuh"
#include "fa_cache_kernels.cuh"
#include "fa_internal.h"

namespace {

using fa_detail::aligned;
using fa_detail::kMaxDevices;

constexpr long long kMaxInt = 0x7fffffffLL;

int log2_of(int x) {
    int r = 0;
    while ((1 << r) < x) ++r;
    return r;
}

fa_status validate_cache(const fa_cache *c) {
    if (c->B < 0 || c->H_kv < 0 || c->n_pages < 0 || c->max_pages < 0 || c->table_stride < 0)
        return FA_ERR_INVALID_ARGUMENT;
    if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) return FA_ERR_UNSUPPORTED;
    if (c->d != 64 && c->d != 128 && c->d != 256) return FA_ERR_UNSUPPORTED;
    if ((long long)c->max_pages * c->page > kMaxInt || (long long)c->B * c->H_kv > kMaxInt)
        return FA_ERR_INVALID_ARGUMENT;
    // (page, head, 16 tokens) units of the pool are counted in 32 bits
    if ((long long)c->n_pages * c->H_kv > kMaxInt / (c->page / 16)) return FA_ERR_INVALID_ARGUMENT;
    if (c->B == 0 || c->H_kv == 0) return FA_OK;
    if (c->n_pages > 0 && (!c->k || !c->v || !c->k_scale || !c->v_scale)) return FA_ERR_INVALID_ARGUMENT;
    if (c->max_pages > 0 && !c->table) return FA_ERR_INVALID_ARGUMENT;
    if (!aligned(c->k, 16) || !aligned(c->v, 16)) return FA_ERR_MISALIGNED;
    if (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) || !aligned(c->table, 4)) return FA_ERR_MISALIGNED;
    return FA_OK;
}

fa::CacheView view_of(const fa_cache &c) {
    fa::CacheView v;
    v.k = static_cast<uint8_t *>(c.k);
    v.v = static_cast<uint8_t *>(c.v);
    v.k_scale = c.k_scale;
    v.v_scale = c.v_scale;
    v.table = c.table;
    v.table_stride = c.table_stride;
    v.n_pages = c.n_pages;
    v.max_pages = c.max_pages;
    v.B = c.B;
    v.H_kv = c.H_kv;
    v.page = c.page;
    v.d = c.d;
    v.page_log2 = log2_of(c.page);
    return v;
}

// 16-byte aligned base and strides of whole 16 bytes, where there is more than one entry.
bool vectors(const void *base, const int64_t *stride, int B, int H, int N) {
    const int n[3] = {B, H, N};
    if (!aligned(base, 16)) return false;
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && stride[i] % 8 != 0) return false;
    return true;
}

template <bool VEC, bool TWO>
fa_status launch_append(const fa::AppendParams &kp, int tokens, unsigned grid, int threads, int dev, cudaStream_t s) {
    static std::atomic<bool> ready[kMaxDevices];
    auto kern = fa::fa_cache_append_kernel<VEC, TWO>;
    // the sines and cosines of a page's new tokens: 8 bytes for each pair
    const int smem = VEC ? tokens * (kp.dim / 2) * 8 : 0;
    if (smem > 46 * 1024 && !ready[dev].load(std::memory_order_acquire)) {  // (2 KB are the kernel's own)
        constexpr int most = 128 * (FA_ROTARY_MAX_DIM / 2) * 8;
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess)
            return FA_ERR_CUDA;
        ready[dev].store(true, std::memory_order_release);
    }
    kern<<<grid, threads, smem, s>>>(kp);
    return cudaPeekAtLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// ---------------------------------------------------------------- attention
constexpr int kMaxCluster = 8;
// SMs of the GPU that the choice below is made for.  It does not ask the device, so that the scratch a call
// needs follows from its sizes; on a smaller part of one the clusters take turns.
constexpr int kSMs = 148;

// CTAs (of `warps` warps) for each pair when clusters of them take the (sequence, head) pairs whole; 0: split the
// keys of all pairs instead.  One CTA up to two tiles for a warp, of the tokens that a sequence can hold; more of
// them for one tile each, as long as all run at once (a cluster lies on one GPC, so that clusters of 4
// and 8 are sure of 7/8 of the SMs only).  Splitting costs a second launch and the parts' way through memory,
// and wins where a warp has more tiles than below, or where there are more than two rounds of CTAs.
// Measured on B200, d = 128, split against clusters, us: 4 rows, 8 pairs of 512, 2048 and 8192 tokens 9.0 / 7.1,
// 10.6 / 8.0, 13.1 / 10.9; 256 pairs of 200 14.5 / 10.4; 8 rows, 64 pairs of 1000 12.4 / 9.8; 16 rows, 128 pairs of
// 300 and 600 22.1 / 9.4, 27.5 / 11.6; 3 pairs of 8000, 8 tiles for a warp, 14.3 / 17.9; 512 pairs of 56
// rows and 300 tokens (four blocks of rows each) 22.3 / 29.2 in more than two rounds.
int direct_cluster(const fa_cache &c, int chunks, int nt, int warps) {
    const long long units = (long long)c.B * c.H_kv * chunks;
    const long long tiles = ((long long)c.max_pages * c.page) / fa::cattn::kTile;
    int n = 1;
    if (tiles > 2 * warps)
        while (n < kMaxCluster && (long long)n * warps < tiles) n *= 2;
    while (n > 1 && units * n > (n == 2 ? kSMs : kSMs / 8 * 7)) n /= 2;
    const int most = units < 8 ? (nt == 0 ? 4 : 2) : (nt == 0 ? 6 : 8);  // few pairs leave SMs idle
    return units * n <= 2 * kSMs && tiles <= (long long)most * n * warps ? n : 0;
}

int direct_warps(int d, int nt) {
    namespace ca = fa::cattn;
    if (d == 64) return nt < 2 ? ca::kDirectWarps<64, 1> : ca::kDirectWarps<64, 2>;
    if (d == 128) return nt < 2 ? ca::kDirectWarps<128, 1> : ca::kDirectWarps<128, 2>;
    return ca::kDirectWarps<256, 1>;
}

struct AttnPlan {
    int nt, rows, chunks;
    int cluster;              // CTAs for each pair, or 0 and
    int workers;              // warps that split the keys, for each chunk
    size_t o_bytes, ml_bytes; // their scratch
};

// CTAs that one SM holds (the kernel's launch bounds).
int attn_resident(int d, int nt) {
    namespace ca = fa::cattn;
    if (d == 64) return nt < 2 ? ca::kResident<64, 1> : ca::kResident<64, 2>;
    if (d == 128) return nt < 2 ? ca::kResident<128, 1> : ca::kResident<128, 2>;
    return ca::kResident<256, 1>;
}

AttnPlan plan_attn(const fa_cache_attn_params *p, int resident) {
    namespace ca = fa::cattn;
    AttnPlan a;
    const fa_cache &c = p->cache;
    a.rows = p->H / c.H_kv * p->N;
    a.nt = a.rows <= 4 ? 0 : ((a.rows <= 8 || c.d == 256) ? 1 : 2);
    const int per = ca::rows_of(a.nt);
    a.chunks = (a.rows + per - 1) / per;
    a.cluster = direct_cluster(c, a.chunks, a.nt, direct_warps(c.d, a.nt));
    a.workers = 0;
    a.o_bytes = a.ml_bytes = 0;
    if (a.cluster) return a;
    long long w = resident / a.chunks;
    const long long tiles = (long long)c.B * c.H_kv * (((long long)c.max_pages * c.page) / ca::kTile);
    if (w > tiles) w = tiles;  // a worker takes one at least
    a.workers = w < 1 ? 1 : (int)w;
    const size_t slots = (size_t)a.chunks * a.workers * 2 * per;
    a.o_bytes = slots * c.d * sizeof(float);
    a.ml_bytes = slots * 2 * sizeof(float);
    return a;
}

bool attn_empty(const fa_cache_attn_params *p) {
    return p->cache.B == 0 || p->cache.H_kv == 0 || p->H == 0 || p->N == 0;
}

template <int D, int WPR>
fa_status launch_merge(const fa::cattn::Params &kp, int rows_per, cudaStream_t s) {
    constexpr int warps = fa::cattn::kMergeWarps<WPR>, per_cta = warps / WPR;
    const long long rows = (long long)kp.c.B * kp.c.H_kv * kp.rows;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((rows + per_cta - 1) / per_cta));
    cfg.blockDim = dim3(32 * warps);
    cfg.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fa::cattn::fa_cache_merge_kernel<D, WPR>, kp, rows_per) == cudaSuccess ? FA_OK
                                                                                                       : FA_ERR_CUDA;
}

template <int D, int NT, int WARPS, bool FINE>
fa_status set_attn_smem(int dev) {
    static std::atomic<bool> ready[kMaxDevices];
    if (ready[dev].load(std::memory_order_acquire)) return FA_OK;
    if (cudaFuncSetAttribute(fa::cattn::fa_cache_attn_kernel<D, NT, WARPS, FINE>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, fa::cattn::kSmemBytes<D, NT, WARPS>) != cudaSuccess)
        return FA_ERR_CUDA;
    ready[dev].store(true, std::memory_order_release);
    return FA_OK;
}

template <int D, int NT, bool FINE>
fa_status launch_attn(const fa::cattn::Params &kp, int dev, int sms, cudaStream_t s) {
    namespace ca = fa::cattn;
    constexpr int W = ca::kDirectWarps<D, NT>;
    if (const int n = kp.cluster) {
        const fa_status st = set_attn_smem<D, NT, W, FINE>(dev);
        if (st != FA_OK) return st;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(kp.c.B * kp.c.H_kv * kp.chunks * n));
        cfg.blockDim = dim3(32 * W);
        cfg.dynamicSmemBytes = ca::kSmemBytes<D, NT, W>;
        cfg.stream = s;
        cudaLaunchAttribute at;
        at.id = cudaLaunchAttributeClusterDimension;
        at.val.clusterDim.x = n;
        at.val.clusterDim.y = at.val.clusterDim.z = 1;
        cfg.attrs = &at;
        cfg.numAttrs = n > 1 ? 1 : 0;
        return cudaLaunchKernelEx(&cfg, ca::fa_cache_attn_kernel<D, NT, W, FINE>, kp) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
    }
    const fa_status st = set_attn_smem<D, NT, ca::kWarps, FINE>(dev);
    if (st != FA_OK) return st;
    // few workers are spread over the SMs, one warp in a CTA at work
    const int warps = kp.chunks * kp.workers, ctas = ca::kResident<D, NT> * sms;
    const int full = (warps + ca::kWarps - 1) / ca::kWarps;
    ca::fa_cache_attn_kernel<D, NT, ca::kWarps, FINE>
        <<<full > ctas ? full : (warps < ctas ? warps : ctas), 32 * ca::kWarps, ca::kSmemBytes<D, NT, ca::kWarps>, s>>>(kp);
    if (cudaPeekAtLastError() != cudaSuccess) return FA_ERR_CUDA;

    // The merge is launched while the first kernel runs and waits in it for its results.  A pair
    // has about workers / pairs parts: one warp for a row, or more where there are many.
    const long long pairs = (long long)kp.c.B * kp.c.H_kv;
    if (kp.workers <= 4 * pairs) return launch_merge<D, 1>(kp, ca::rows_of(NT), s);
    if (kp.workers <= 64 * pairs) return launch_merge<D, 8>(kp, ca::rows_of(NT), s);
    return launch_merge<D, 32>(kp, ca::rows_of(NT), s);
}

template <int D, bool FINE>
fa_status launch_attn_rows(const fa::cattn::Params &kp, int nt, int dev, int sms, cudaStream_t s) {
    if constexpr (D < 256) {
        if (nt == 2) return launch_attn<D, 2, FINE>(kp, dev, sms, s);
    }
    return launch_attn<D, 1, FINE>(kp, dev, sms, s);
}

template <int D>
fa_status launch_attn_d(const fa::cattn::Params &kp, int nt, int dev, int sms, cudaStream_t s) {
    if (nt == 0) return launch_attn<D, 0, true>(kp, dev, sms, s);
    return kp.o_bf16 ? launch_attn_rows<D, false>(kp, nt, dev, sms, s) : launch_attn_rows<D, true>(kp, nt, dev, sms, s);
}

}  // namespace

extern "C" {

fa_status fa_cache_append(const fa_cache_append_params *p, void *stream) {
    if (!p || p->N < 0) return FA_ERR_INVALID_ARGUMENT;
    fa_status st = validate_cache(&p->cache);
    if (st != FA_OK) return st;
    const fa_cache &c = p->cache;
    if (p->rotary && (st = fa_detail::validate_rotary(p->rotary, c.d)) != FA_OK) return st;
    if (c.B == 0 || c.H_kv == 0 || p->N == 0) return FA_OK;
    if (!p->k || !p->v || !p->start) return FA_ERR_INVALID_ARGUMENT;
    if (!aligned(p->k, 2) || !aligned(p->v, 2) || !aligned(p->start, 4) || !aligned(p->n_new, 4) ||
        !aligned(p->dev_status, 4))
        return FA_ERR_MISALIGNED;
    int dev = 0, sms = 0;
    if ((st = fa_detail::current_device(&dev, &sms)) != FA_OK) return st;

    fa::AppendParams kp;
    std::memset(&kp, 0, sizeof kp);
    kp.c = view_of(c);
    kp.x[0] = static_cast<const uint16_t *>(p->k);
    kp.x[1] = static_cast<const uint16_t *>(p->v);
    for (int i = 0; i < 3; ++i) {
        kp.xs[0][i] = p->k_stride[i];
        kp.xs[1][i] = p->v_stride[i];
    }
    kp.N = p->N;
    // N tokens that begin in the last slot of a page
    kp.pages = (int)(((long long)p->N - 1 + c.page - 1) / c.page) + 1;
    kp.start = p->start;
    kp.n_new = p->n_new;
    kp.status = p->dev_status;
    bool vec = vectors(p->k, p->k_stride, c.B, c.H_kv, p->N) && vectors(p->v, p->v_stride, c.B, c.H_kv, p->N);
    if (p->rotary) {
        kp.dim = p->rotary->dim;
        kp.interleaved = p->rotary->layout == FA_ROTARY_INTERLEAVED;
        kp.amplitude = p->rotary->amplitude;
        std::memcpy(kp.step, p->rotary->step, sizeof(uint64_t) * (kp.dim / 2));
        vec = vec && kp.dim % 16 == 0;
    }
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (vec && (long long)p->N * (c.d / 16) <= 32) {
        const long long blocks = ((long long)c.B * c.H_kv + fa::kFewWarps - 1) / fa::kFewWarps;
        fa::fa_cache_append_few_kernel<<<(unsigned)blocks, 32 * fa::kFewWarps, 0, s>>>(kp);
        return cudaPeekAtLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
    }
    // slots of 16 components of as many new tokens as a page can get: a power of two, at most 2048
    int tokens = 1;
    while (tokens < c.page && tokens < p->N) tokens *= 2;
    const int slots = tokens * (c.d / 16);
    const int threads = slots < 32 ? 32 : (slots < 1024 ? slots : 1024);
    // as many heads in a block, which share the sines, as leave every SM 2048 threads in all
    const long long touched = (long long)c.B * kp.pages;
    kp.group = c.H_kv;
    while (kp.group > 1 && touched * ((c.H_kv + kp.group - 1) / kp.group) * threads < 2048LL * sms)
        kp.group = (kp.group + 1) / 2;
    const long long blocks = touched * ((c.H_kv + kp.group - 1) / kp.group);
    if (blocks > kMaxInt) return FA_ERR_INVALID_ARGUMENT;
    const unsigned grid = (unsigned)blocks;
    if (slots > 1024)
        return vec ? launch_append<true, true>(kp, tokens, grid, threads, dev, s)
                   : launch_append<false, true>(kp, tokens, grid, threads, dev, s);
    return vec ? launch_append<true, false>(kp, tokens, grid, threads, dev, s)
               : launch_append<false, false>(kp, tokens, grid, threads, dev, s);
}

fa_status fa_cache_gather(const fa_cache_gather_params *p, void *stream) {
    if (!p || p->N_k < 0) return FA_ERR_INVALID_ARGUMENT;
    fa_status st = validate_cache(&p->cache);
    if (st != FA_OK) return st;
    const fa_cache &c = p->cache;
    if (c.B == 0 || c.H_kv == 0 || p->N_k == 0) return FA_OK;
    if (!p->k || !p->v || !p->k_len) return FA_ERR_INVALID_ARGUMENT;
    if (!aligned(p->k, 16) || !aligned(p->v, 16) || !aligned(p->k_len, 4) || !aligned(p->dev_status, 4))
        return FA_ERR_MISALIGNED;
    int dev = 0, sms = 0;
    if ((st = fa_detail::current_device(&dev, &sms)) != FA_OK) return st;
    fa::GatherParams kp;
    std::memset(&kp, 0, sizeof kp);
    kp.c = view_of(c);
    kp.k_len = p->k_len;
    kp.k = static_cast<uint16_t *>(p->k);
    kp.v = static_cast<uint16_t *>(p->v);
    kp.N_k = p->N_k;
    kp.status = p->dev_status;
    const int per_block = fa::kGatherThreads * fa::kGatherItems / (c.d / 8);
    kp.row_blocks = (int)(((long long)p->N_k + per_block - 1) / per_block);
    const long long blocks = (long long)c.B * c.H_kv * kp.row_blocks;
    if (blocks > kMaxInt) return FA_ERR_INVALID_ARGUMENT;
    fa::fa_cache_gather_kernel<<<(unsigned)blocks, fa::kGatherThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(kp);
    return cudaPeekAtLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_cache_attn_workspace_bytes(const fa_cache_attn_params *p) {
    if (!p || validate_cache(&p->cache) != FA_OK || p->H <= 0 || p->N <= 0 || p->cache.B == 0 || p->cache.H_kv == 0 ||
        p->H % p->cache.H_kv != 0 || (long long)p->H / p->cache.H_kv * p->N > kMaxInt)
        return 0;
    const AttnPlan a = plan_attn(p, fa::cattn::kMaxWorkers);
    return a.o_bytes + a.ml_bytes;
}

fa_status fa_cache_attn(const fa_cache_attn_params *p, void *stream) {
    if (!p || p->H < 0 || p->N < 0) return FA_ERR_INVALID_ARGUMENT;
    fa_status st = validate_cache(&p->cache);
    if (st != FA_OK) return st;
    const fa_cache &c = p->cache;
    if ((p->causal != 0 && p->causal != 1) || !std::isfinite(p->scale) || p->scale <= 0.f)
        return FA_ERR_INVALID_ARGUMENT;
    if (p->o_dtype != FA_O_F32 && p->o_dtype != FA_O_BF16) return FA_ERR_INVALID_ARGUMENT;
    if (p->test_drop_load < 0) return FA_ERR_INVALID_ARGUMENT;
    if (attn_empty(p)) return FA_OK;
    if (p->H % c.H_kv != 0 || (long long)c.B * p->H > kMaxInt / p->N) return FA_ERR_INVALID_ARGUMENT;
    // the kernels' line of (sequence, head) pairs is counted in 32 bits
    if ((long long)c.B * c.H_kv > kMaxInt / ((long long)c.max_pages * (c.page / fa::cattn::kTile) + fa::cattn::kPairCost))
        return FA_ERR_INVALID_ARGUMENT;
    if (!p->q || !p->o || !p->lse || !p->k_len) return FA_ERR_INVALID_ARGUMENT;
    if (!aligned(p->q, 16) || !aligned(p->o, 16) || !aligned(p->workspace, 16) || !aligned(p->lse, 4) ||
        !aligned(p->k_len, 4) || !aligned(p->dev_status, 4))
        return FA_ERR_MISALIGNED;
    const size_t scratch = fa_cache_attn_workspace_bytes(p);
    if (scratch && (!p->workspace || p->workspace_bytes < scratch)) return FA_ERR_INVALID_ARGUMENT;
    int dev = 0, sms = 0;
    if ((st = fa_detail::current_device(&dev, &sms)) != FA_OK) return st;

    AttnPlan a = plan_attn(p, fa::cattn::kMaxWorkers);
    const int resident = attn_resident(c.d, a.nt) * fa::cattn::kWarps * sms;  // warps
    if (resident < fa::cattn::kMaxWorkers) a = plan_attn(p, resident);
    fa::cattn::Params kp;
    std::memset(&kp, 0, sizeof kp);
    kp.c = view_of(c);
    kp.q = static_cast<const uint16_t *>(p->q);
    kp.o = p->o;
    kp.lse = p->lse;
    kp.k_len = p->k_len;
    kp.status = p->dev_status;
    kp.o_part = static_cast<float *>(p->workspace);
    kp.ml_part = reinterpret_cast<float2 *>(static_cast<char *>(p->workspace) + a.o_bytes);
    kp.N = p->N;
    kp.rows = a.rows;
    kp.chunks = a.chunks;
    kp.workers = a.workers;
    kp.cluster = a.cluster;
    kp.causal = p->causal;
    kp.o_bf16 = p->o_dtype == FA_O_BF16;
    kp.scale_log2 = (float)((double)p->scale * 1.4426950408889634074);
    kp.timeout_ns = (uint64_t)(p->timeout_ms ? p->timeout_ms : 2000u) * 1000000ull;
    kp.drop_load = p->test_drop_load;
    // without any page there is nothing to copy; the map only has to be a valid one
    const bool pages = c.n_pages > 0;
    const int line = c.d == 256 ? 256 : 128, lines = fa::cattn::kTile * c.d / line;
    const long long tiles = pages ? (long long)c.n_pages * c.H_kv * (c.page / fa::cattn::kTile) : 1;
    if ((st = fa_detail::encode_cache_map(&kp.tm_k, pages ? c.k : p->o, tiles, lines, line)) != FA_OK ||
        (st = fa_detail::encode_cache_map(&kp.tm_v, pages ? c.v : p->o, tiles, lines, line)) != FA_OK)
        return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return c.d == 64 ? launch_attn_d<64>(kp, a.nt, dev, sms, s)
                     : (c.d == 128 ? launch_attn_d<128>(kp, a.nt, dev, sms, s) : launch_attn_d<256>(kp, a.nt, dev, sms, s));
}

}  // extern "C"
