/*
 * fa.h -- C ABI of the B200 (sm_100a) exact attention forward pass.
 *
 * The operation (page "FlashAttention (ES)", section "El problema de la
 * atencion estandar", the Attention equation; masking from section "Fusion de
 * operaciones en un unico kernel de CUDA"):
 *
 *     O   = softmax(Q K^T * scale + mask) V
 *     lse = log( sum over allowed keys of exp(scale * q . k) )   (natural log)
 *
 * computed by one fused kernel launch that tiles Q, K and V through shared
 * memory (section "Tiling y procesamiento por bloques"), keeps a running row
 * maximum and running sum of exponentials (section "Calculo de Softmax en
 * linea") and writes only O and lse (section "Fusion de operaciones en un
 * unico kernel de CUDA"): no N x N buffer, no workspace of any kind.
 *
 * Layout (all tensors contiguous, row-major):
 *   q       : bf16  [B, H, N, d]      (one N x d matrix per (b, h))
 *   k, v    : bf16  [B, H_kv, N_k, d] (fa_fwd: H_kv = H and N_k = N; fa_fwd_ex
 *             may group heads -- query head h attends with key/value head
 *             h / (H / H_kv), the multi-query attention of section
 *             "FlashAttention-2 (2023)" -- and may give more keys than queries,
 *             the cached-keys setting of section "Soluciones especializadas":
 *             query i then sits at key position i + N_k - N)
 *   o       : fp32  [B, H, N, d]  (fa_fwd; fa_fwd_ex may select bf16)
 *   lse     : fp32  [B, H, N]
 *   k_len   : int32 [B]  (fa_fwd_ex only; key j of batch b is masked iff
 *             j >= k_len[b]; values are clamped to [0, N_k] on the device)
 * Mask: causal masks key j for query i when j > i + N_k - N (j > i when
 * N_k = N).  A row with no allowed key gets O = 0, lse = -inf.
 *
 * Further down: rotary positions (fa_rotary_init, fa_rope) and a paged key/value
 * cache in 8 bits (fa_cache_append, fa_cache_attn, fa_cache_gather), whose
 * layouts are given there.
 *
 * Ownership: the caller owns every buffer.  The library allocates, frees and
 * synchronises nothing (except fa_read_device_status and fa_fwd_host, which
 * say so), holds no state beyond a per-device cache of properties (and the two
 * copy streams of fa_fwd_host) and the driver's tensor-map entry point, and is
 * safe to call from several threads.
 *
 * Errors: argument errors are returned synchronously and launch nothing.
 * Device-side errors (a pipeline wait that exceeded its time limit) are
 * written to the optional device status word.  All calls are asynchronous on
 * `stream` (a cudaStream_t; NULL is the legacy default stream).
 */
#ifndef EXACT_IO_AWARE_52_FA_H
#define EXACT_IO_AWARE_52_FA_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define FA_EXPORT __attribute__((visibility("default")))
#else
#define FA_EXPORT
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FA_OK = 0,
    FA_ERR_INVALID_ARGUMENT = 1, /* NULL pointer, negative size, bad scale, bad dtype */
    FA_ERR_MISALIGNED = 2,       /* a pointer not 16-byte aligned (TMA requirement)   */
    FA_ERR_UNSUPPORTED = 3,      /* d not in {64, 128, 256}, or the device is not sm_100 */
    FA_ERR_CUDA = 4,             /* a CUDA runtime/driver call or the launch failed   */
    FA_ERR_DEVICE_TIMEOUT = 5,   /* (device status word) a pipeline wait timed out     */
    FA_ERR_WORKSPACE_LIMIT = 6,  /* fa_fwd_static_workspace: the splits need more than
                                    FA_STATIC_WORKSPACE_BYTES of scratch                */
    FA_ERR_SCHED_BUSY = 7,       /* (device status word) the launch's scheduler slot stayed
                                    in use by another in-flight launch for longer than the
                                    wait limit; the launch did no work                  */
    FA_ERR_BAD_PAGE = 8          /* (device status word) a page-table entry outside
                                    [0, n_pages), or a position outside the table       */
} fa_status;

typedef enum { FA_O_F32 = 0, FA_O_BF16 = 1 } fa_o_dtype;

/* Element type of q, k and v. */
typedef enum {
    FA_IN_BF16 = 0, /* bfloat16, the default                                        */
    FA_IN_E4M3 = 1  /* FP8 E4M3 (one byte; OCP "fn" variant: no infinities), d = 128 */
} fa_in_dtype;

/* Flags for fa_fwd_params.flags. */
enum {
    /* Rescale the running output whenever a row maximum grows, instead of
     * only when it grows by more than a factor 2^8 (bf16 inputs) or 2^1.75
     * (E4M3 inputs, whose weights must stay below E4M3's largest value), the
     * defaults.  Both are exact up to rounding; the default skips most
     * rescales, this one keeps the largest softmax weight of each row at
     * exactly 1 (E4M3: 2^7) before rounding. */
    FA_FLAG_EAGER_RESCALE = 1
};

/*
 * fa_fwd -- the attention forward pass, fp32 output, no key padding.
 *   q, k, v : device bf16 [B, H, N, d], 16-byte aligned
 *   o       : device fp32 [B, H, N, d], 16-byte aligned
 *   lse     : device fp32 [B, H, N]
 *   B, H, N : >= 0 (B*H*N == 0 is a no-op returning FA_OK)
 *   d       : 64, 128 or 256
 *   causal  : 0 or 1
 *   scale   : finite, > 0 (the definition's 1/sqrt(d_k))
 *   stream  : cudaStream_t
 * Equivalent to fa_fwd_ex with k_len = NULL, o_dtype = FA_O_F32, flags = 0,
 * no status word and the default time limit.
 */
FA_EXPORT fa_status fa_fwd(const void *q, const void *k, const void *v, float *o, float *lse,
                 int B, int H, int N, int d, int causal, float scale, void *stream);

typedef struct {
    const void *q, *k, *v;   /* device, in_dtype: q [B, H, N, d]; k, v [B, H_kv, N_k, d] */
    void *o;                 /* device [B, H, N, d], fp32 or bf16 per o_dtype         */
    float *lse;              /* device fp32 [B, H, N]                                 */
    const int32_t *k_len;    /* device int32 [B], or NULL (no key padding)           */
    int32_t *dev_status;     /* device int32 word or NULL; the kernel stores a
                                fa_status there on a device-side error (first error
                                wins); the caller zeroes it before the launch        */
    int B, H, N, d;
    int causal;
    float scale;
    int o_dtype;             /* fa_o_dtype                                            */
    int flags;               /* FA_FLAG_* bits, 0 by default                          */
    uint32_t timeout_ms;     /* per-wait time limit on the device; 0 = 2000 ms        */
    int H_kv;                /* key/value heads (k, v are [B, H_kv, N_k, d]); 0 means H;
                                must divide H (1 = multi-query attention)             */
    int N_k;                 /* keys; 0 means N (queries); query i sits at key
                                position i + N_k - N                                  */
    int num_splits;          /* 0 or 1: one pass over each row's keys.  S > 1: the key
                                range is cut into S contiguous parts processed in
                                parallel (more work units when B*H*ceil(N/256) is
                                below the SM count), their partial results written
                                to `workspace` and merged by a second kernel          */
    void *workspace;         /* device scratch, 16-byte aligned, at least
                                fa_fwd_workspace_bytes(p) bytes; unused when
                                num_splits <= 1.  Owned by the caller; the library
                                writes every byte it reads from it in the same call   */
    size_t workspace_bytes;  /* size of workspace                                     */
    int in_dtype;            /* fa_in_dtype of q, k, v                                */
    float descale_q, descale_k, descale_v;
                             /* E4M3 inputs: the values are q * descale_q, k * descale_k,
                                v * descale_v (per-tensor scales; 0 means 1).  Ignored
                                for bf16.  The products Q K^T and P V run on E4M3 with
                                fp32 accumulation; P is rounded to E4M3 before P V;
                                the softmax is fp32.  Finite and >= 0.                */
    int test_drop_load;      /* test only; 0 (off) in every normal call.  n > 0: the TMA
                                producer of the kernel's first CTA never issues its n-th
                                key-tile load (d = 256: its n-th K/V half-tile load), so
                                the pipeline wait for that tile runs out after timeout_ms
                                and the time-out path (status word, NaN rows, drain,
                                exit) runs with no copy in flight.  Must be >= 0.       */
} fa_fwd_params;

/*
 * fa_fwd_workspace_bytes -- device scratch bytes fa_fwd_ex needs for *p
 * (0 when p->num_splits <= 1): the partial outputs of the key splits, fp32
 * [S][B, H, N, d] and [S][B, H, N].  Host arithmetic only; 0 for a NULL p.
 */
FA_EXPORT size_t fa_fwd_workspace_bytes(const fa_fwd_params *p);

/*
 * fa_fwd_suggest_splits -- a key-split count for *p on the current device.
 * Returns 1 when the unsplit grid already gives every SM two work units or
 * the keys fit one 128-key tile; otherwise the count in [1, key tiles] that
 * minimises a cost model of whole waves of (query block, split) units over
 * the SMs plus the partials' HBM round trip.  Returns 0 on error (NULL, a
 * non-positive size, no CUDA device).
 */
FA_EXPORT int fa_fwd_suggest_splits(const fa_fwd_params *p);

/*
 * fa_fwd_ex -- the forward pass with key padding, output dtype and a status
 * word.  Causal problems hand their work units out through a per-launch
 * counter held by the library (64 slots per device, taken round-robin by
 * causal fa_fwd / fa_fwd_ex / fa_bwd launches).  Each launch's CTAs claim its
 * slot for their grid before taking a unit, so launches that meet on a slot
 * (more than 64 in flight at once on one device, or one CUDA graph replayed
 * on several streams) run one after the other instead of sharing a counter;
 * a launch whose wait for its slot outlasts timeout_ms does no work and
 * stores FA_ERR_SCHED_BUSY in *dev_status.
 *
 * On a device-side timeout the kernel stores FA_ERR_DEVICE_TIMEOUT in
 * *dev_status and stops: the CTA that timed out writes NaN to the rows of the
 * unit it was working on, but its remaining units are never written, and
 * with key splits the merge still runs over whatever partials the workspace
 * holds.  After FA_ERR_DEVICE_TIMEOUT the whole of o and lse is undefined;
 * the error is seen only through the status word, so pass one when the
 * result matters.
 *
 * The library caches device addresses (its scheduler words, and the scratch
 * array of fa_fwd_static_workspace) per device ordinal for the life of the
 * process.  Do not reset a device (cudaDeviceReset) between calls into this
 * library: the module is reloaded at a possibly different address and the
 * cached addresses would be stale.
 */
FA_EXPORT fa_status fa_fwd_ex(const fa_fwd_params *p, void *stream);

typedef struct {
    const void *q, *k, *v;   /* host, dev.in_dtype, shapes as in dev (pinned for async copies) */
    const int32_t *k_len;    /* host int32 [B] or NULL                                */
    void *o;                 /* host output, dtype per dev.o_dtype                    */
    float *lse;              /* host fp32 [B, H, N]                                   */
    fa_fwd_params dev;       /* device buffers of the same shapes (q, k, v, o, lse,
                                and k_len when k_len is not NULL) plus the options    */
} fa_fwd_host_params;

/*
 * fa_fwd_host -- end-to-end call on HOST buffers: copies q, k, v (and k_len)
 * host -> device into the caller's device buffers, runs fa_fwd_ex, copies o
 * and lse device -> host, and synchronises `stream` before returning.
 * A call whose copies total 64 MB or more, and that gives every SM at least
 * two work units per piece, is cut into up to 8 pieces: whole batch elements
 * (B > 1) or whole groups of query heads sharing a key/value head (B = 1).
 * Piece c's copies in run on a copy-in stream, its fa_fwd_ex on `stream` once
 * they have landed, and its copies out on a copy-out stream once the kernel is
 * done, so that copies in both directions and the kernels of different pieces
 * overlap (the two streams are created once per device and kept).  The
 * result equals the single call's bit for bit (each piece is a valid
 * fa_fwd_ex problem with the caller's options; a call that cannot be cut that
 * way runs whole).  Host buffers should be pinned for the copies to overlap.
 * Work queued earlier on `stream` completes before the first copy.  If
 * dev.dev_status is set, a device-side error found after the copies is
 * returned as its fa_status.
 */
FA_EXPORT fa_status fa_fwd_host(const fa_fwd_host_params *p, void *stream);

/*
 * fa_read_device_status -- synchronises `stream`, reads the device status
 * word and returns it as a fa_status (FA_ERR_CUDA if the read fails).
 */
FA_EXPORT fa_status fa_read_device_status(const int32_t *dev_status, void *stream);

/* Human-readable name of a status code (static string, never NULL). */
FA_EXPORT const char *fa_status_string(fa_status s);

/* Library version as an integer MAJOR*10000 + MINOR*100 + PATCH. */
FA_EXPORT int fa_version(void);

/*
 * Backward pass: the gradients of the forward's O with respect to q, k and v
 * for a given dO.  The pages report training speed-ups of the method (page
 * "FlashAttention (ES)", section "Resultados empiricos") but give no
 * backward algorithm; this is the derivative of the definition of section
 * "El problema de la atencion estandar", with P recomputed from q, k and the
 * forward's lse:
 *     dV = P^T dO,  dP = dO V^T,  dS = scale * P o (dP - D),  D_i = dO_i . O_i,
 *     dQ = dS K,    dK = dS^T Q
 * (o the elementwise product).  Masks, N_k, grouped heads and k_len are those
 * of the forward; dK and dV of a key/value head sum over its query heads.
 */
typedef struct {
    const void *q, *k, *v;   /* device bf16: q [B, H, N, d]; k, v [B, H_kv, N_k, d]    */
    const void *o;           /* device forward output [B, H, N, d], fp32 or bf16 (o_dtype) */
    const void *dout;        /* device bf16 [B, H, N, d]: gradient of the loss w.r.t. O  */
    const float *lse;        /* device fp32 [B, H, N] from the forward with the same inputs */
    float *dq;               /* device fp32 [B, H, N, d], overwritten                   */
    float *dk, *dv;          /* device fp32 [B, H_kv, N_k, d], overwritten              */
    const int32_t *k_len;    /* device int32 [B] or NULL, as in fa_fwd_params           */
    int32_t *dev_status;     /* device status word or NULL, as in fa_fwd_params         */
    int B, H, N, d;          /* d in {64, 128}                                          */
    int causal;
    float scale;
    int o_dtype;             /* fa_o_dtype of o                                         */
    uint32_t timeout_ms;     /* per-wait time limit on the device; 0 = 2000 ms          */
    int H_kv, N_k;           /* 0 means H and N                                         */
    void *workspace;         /* device scratch of at least fa_bwd_workspace_bytes(p),
                                16-byte aligned, owned by the caller                    */
    size_t workspace_bytes;
} fa_bwd_params;

/* Scratch bytes fa_bwd needs for *p: D, fp32 [B, H, N].  0 for a NULL p. */
FA_EXPORT size_t fa_bwd_workspace_bytes(const fa_bwd_params *p);

/*
 * fa_bwd -- two launches on `stream`: D and a zeroed dQ, then the gradients
 * (dQ accumulated in fp32 by TMA reduce-adds, one key tile per work unit).
 * All pointers except k_len and dev_status must be 16-byte aligned.  Errors
 * as for fa_fwd_ex (d not in {64, 128}: FA_ERR_UNSUPPORTED).  dq, dk and dv
 * are deterministic up to the order of the fp32 additions into dq.
 */
FA_EXPORT fa_status fa_bwd(const fa_bwd_params *p, void *stream);

/* Size of the library's fixed device scratch array (64 MiB), per device. */
#define FA_STATIC_WORKSPACE_BYTES (64u * 1024u * 1024u)

/*
 * fa_fwd_static_workspace -- fa_fwd_ex with the key-split scratch taken from
 * a fixed device array inside the library instead of p->workspace, so that
 * the call allocates no memory.  The pages have no counterpart: their
 * forward pass has no key splits and hence no scratch; this is an interface
 * convenience of this library.
 *
 * p is read as by fa_fwd_ex except that p->workspace and p->workspace_bytes
 * are ignored.  With p->num_splits > 1 the scratch is a file-scope device
 * array of FA_STATIC_WORKSPACE_BYTES; a problem whose splits need more
 * (fa_fwd_workspace_bytes(p) > FA_STATIC_WORKSPACE_BYTES) is rejected with
 * FA_ERR_WORKSPACE_LIMIT before anything is launched.  With num_splits <= 1
 * no scratch is used and the call is fa_fwd_ex.
 *
 * The array is one per device and every call on that device uses it:
 * calls whose executions overlap (on different streams, or from different
 * host threads) race on it and their results are undefined.  Serialise them,
 * e.g. on one stream.  Nothing in it has to start at zero.
 *
 * The first call with num_splits > 1 on a device looks the array's address
 * up (cudaGetSymbolAddress, with that device current) and caches it; make
 * that first call before any stream capture.  Errors: those of fa_fwd_ex,
 * FA_ERR_WORKSPACE_LIMIT, and FA_ERR_CUDA if the lookup fails.
 */
FA_EXPORT fa_status fa_fwd_static_workspace(const fa_fwd_params *p, void *stream);

/*
 * Rotary positions.  Component pair i of a head's first `dim` components is
 * turned by the angle position * w_i:
 *     (a, b) -> m * (a cos - b sin, b cos + a sin)
 * (m the amplitude), which makes q . k of two turned heads a function of the
 * distance of their positions.  The components from `dim` on pass unchanged.
 */
typedef enum {
    FA_ROTARY_HALF = 0,       /* pair i is (x[i], x[i + dim / 2])  */
    FA_ROTARY_INTERLEAVED = 1 /* pair i is (x[2 i], x[2 i + 1])    */
} fa_rotary_layout;

/* How w_i = base^(-2 i / dim) is changed for contexts longer than the original length. */
typedef enum {
    FA_ROTARY_NONE = 0,   /* w_i                                                        */
    FA_ROTARY_LINEAR = 1, /* w_i / factor (positions interpolated)                      */
    FA_ROTARY_BASE = 2,   /* base * factor^(dim / (dim - 2)) in place of base: the
                             slowest pair is divided by factor, the fastest kept        */
    FA_ROTARY_PARTS = 3   /* by turns_i = original_length * w_i / 2 pi: w_i / factor up
                             to low_turns, w_i from high_turns on, and linear in turns_i
                             between the two                                            */
} fa_rotary_scaling;

typedef struct {
    int dim;                 /* rotated leading components: even, 2 .. FA_ROTARY_MAX_DIM */
    int layout;              /* fa_rotary_layout                                        */
    double base;             /* > 0, finite (10000 is common)                           */
    int scaling;             /* fa_rotary_scaling                                       */
    double factor;           /* > 0, finite; unused by FA_ROTARY_NONE                   */
    double original_length;  /* FA_ROTARY_PARTS: > 0                                    */
    double low_turns, high_turns; /* FA_ROTARY_PARTS: 0 <= low < high                   */
    double amplitude;        /* m above; 0 means 1; else > 0 and finite as fp32          */
    const double *angles;    /* host, w_i in radians for each of the dim / 2 pairs, or
                                NULL.  If given, base and scaling are not used; finite,
                                |w_i| <= 2^20                                           */
} fa_rotary_spec;

#define FA_ROTARY_MAX_DIM 256

/* A rotation ready for use: a plain value that the caller keeps and may copy. */
typedef struct {
    int dim, layout;
    float amplitude;
    int ready;                              /* set by fa_rotary_init                    */
    uint64_t step[FA_ROTARY_MAX_DIM / 2];   /* w_i in units of 2^-64 turn: position * step
                                               modulo 2^64 is the angle without the whole
                                               turns, exact however far the position    */
} fa_rotary;

/* fa_rotary_init -- fills *r from *spec.  Host arithmetic only. */
FA_EXPORT fa_status fa_rotary_init(fa_rotary *r, const fa_rotary_spec *spec);

/* Element type of a plain tensor. */
typedef enum { FA_T_BF16 = 0, FA_T_F32 = 1 } fa_dtype;

typedef struct {
    const void *x;           /* device [B, heads, N, d] by strides, x_dtype             */
    void *y;                 /* device [B, heads, N, d] by strides, y_dtype; may be x
                                itself (same type and strides), else no overlap         */
    int heads;               /* >= 0; 0: the tensor is absent                           */
    int64_t x_stride[3];     /* elements from one batch element, head, token to the next
                                (components are contiguous); any order of dimensions    */
    int64_t y_stride[3];     /* not 0 in a dimension of several entries                 */
} fa_rope_tensor;

typedef struct {
    fa_rope_tensor t[2];     /* queries and keys, say; one launch turns both; 65535
                                heads at most together                                  */
    int B, N, d;             /* d: rotary dim .. FA_ROPE_MAX_D; B * N <= 2^31 - 256     */
    int x_dtype, y_dtype;    /* fa_dtype                                                */
    const int32_t *pos;      /* device int32 positions, pos[b * pos_stride + n], or NULL:
                                the position of token n is pos0 + n (below 2^31)        */
    int64_t pos_stride;      /* 0: one row of positions for the whole batch             */
    int32_t pos0;
    int inverse;             /* 1: turn by the negative angles (with the amplitude, the
                                transpose: what the gradient of the turned tensor needs)*/
    const fa_rotary *rotary; /* host                                                    */
} fa_rope_params;

#define FA_ROPE_MAX_D 1024

/*
 * fa_rope -- one launch.  The products are formed in fp32 from the inputs and
 * rounded once to y_dtype.  No alignment beyond the element type is needed;
 * 16-byte aligned tensors with strides of whole 16 bytes, and d and dim that
 * are multiples of 16, are read and written 16 bytes at a time.
 */
FA_EXPORT fa_status fa_rope(const fa_rope_params *p, void *stream);

/*
 * A paged key/value cache in 8 bits.  Token t of sequence b lies in slot
 * t % page of page table[b * table_stride + t / page]; a page has, for every
 * key/value head, `page` slots of d E4M3 codes, and one scale: the value is
 * code * scale.  The caller owns all of it and says which pages a sequence
 * has; several sequences may share pages that are only read.
 */
typedef struct {
    void *k, *v;               /* device E4M3 [n_pages, H_kv, page, d], 16-byte aligned  */
    float *k_scale, *v_scale;  /* device fp32 [n_pages, H_kv]                            */
    const int32_t *table;      /* device int32 [B, max_pages]; entries past a sequence's
                                  last page are not read                                 */
    int64_t table_stride;      /* elements from one row of the table to the next         */
    int n_pages, max_pages;
    int B, H_kv, page, d;      /* page in {16, 32, 64, 128}, d in {64, 128, 256}         */
} fa_cache;

typedef struct {
    fa_cache cache;
    const void *k, *v;         /* device bf16 [B, H_kv, N, d] by strides                 */
    int64_t k_stride[3], v_stride[3]; /* elements from one batch element, head, token to
                                  the next (components are contiguous)                   */
    int N;                     /* tokens given for each sequence                         */
    const int32_t *start;      /* device int32 [B]: position of the first new token, that
                                  is the tokens that the sequence holds already          */
    const int32_t *n_new;      /* device int32 [B] or NULL (N): of each sequence's N
                                  tokens the first n_new[b] are written (clamped to
                                  [0, N]), the others are not read                       */
    const fa_rotary *rotary;   /* host, or NULL; turns each key by its position on the way
                                  (dim <= d)                                             */
    int32_t *dev_status;       /* device status word or NULL, as in fa_fwd_params        */
} fa_cache_append_params;

/*
 * fa_cache_append -- writes new tokens into the cache; one launch.
 *
 * The scale of a page and head is a power of two, 2^e with the least
 * e >= -100 for which the largest finite magnitude of its values is at most
 * 448 * 2^e (E4M3's largest code).  A page that holds tokens from before
 * keeps the larger of its scale and that; if it grows, the codes of those
 * tokens (slots below the first new one) are rescaled, which for
 * power-of-two scales is exact but for codes that become subnormal.  A page
 * whose slot 0 is written has no scale from before.  Infinities and NaN
 * become the code NaN.  (Finite magnitudes from 1.9375 * 2^127 on are nearest to a code that stands for
 * 2^128, which fp32 and bf16 read as infinity.)  Slots behind the last new token are left as they are.
 *
 * A token whose position is negative or past the table, or whose page is
 * outside [0, n_pages), is not written and FA_ERR_BAD_PAGE is stored in
 * *dev_status.  No page may be written through two entries of the table in one call.
 */
FA_EXPORT fa_status fa_cache_append(const fa_cache_append_params *p, void *stream);

typedef struct {
    fa_cache cache;
    const int32_t *k_len;      /* device int32 [B]: tokens that each sequence holds,
                                  clamped to [0, max_pages * page]                       */
    void *k, *v;               /* device bf16 [B, H_kv, N_k, d], contiguous, 16-byte
                                  aligned                                                */
    int N_k;
    int32_t *dev_status;
} fa_cache_gather_params;

/*
 * fa_cache_gather -- the cache's first N_k tokens of every sequence as
 * contiguous keys and values, the form that fa_fwd_ex reads (with k_len);
 * zero behind a sequence's end.  Exact for the scales that fa_cache_append
 * writes; code * scale rounded once for any others.  The tokens of a page
 * outside [0, n_pages) read as zero and store FA_ERR_BAD_PAGE.
 */
FA_EXPORT fa_status fa_cache_gather(const fa_cache_gather_params *p, void *stream);

typedef struct {
    fa_cache cache;            /* scales: finite, >= 0, subnormal ones included.  The sums
                                  over the keys are fp32: values (code * scale) of more
                                  than 2^88 in magnitude may overflow them               */
    const void *q;             /* device bf16 [B, H, N, d], contiguous, 16-byte aligned  */
    void *o;                   /* device [B, H, N, d], fp32 or bf16 per o_dtype          */
    float *lse;                /* device fp32 [B, H, N]                                  */
    const int32_t *k_len;      /* device int32 [B]: tokens that each sequence holds, the
                                  N queries' own included; clamped to
                                  [0, max_pages * page]                                  */
    int32_t *dev_status;
    int H, N;                  /* query heads (a multiple of H_kv) and query tokens      */
    int causal;                /* 1: query i of sequence b sits at position
                                  k_len[b] - N + i and sees the keys up to itself        */
    float scale;               /* finite, > 0                                            */
    int o_dtype;               /* fa_o_dtype                                             */
    void *workspace;           /* device scratch, 16-byte aligned, at least
                                  fa_cache_attn_workspace_bytes(p) bytes; owned by the
                                  caller, nothing in it has to be set, and not shared by
                                  calls whose executions overlap                         */
    size_t workspace_bytes;
    uint32_t timeout_ms;       /* per-wait time limit on the device; 0 = 2000 ms.  After
                                  FA_ERR_DEVICE_TIMEOUT all of o and lse is undefined    */
    int test_drop_load;        /* test only, 0 in every normal call; n > 0: the first CTA's
                                  first warp never loads its n-th tile of keys and values,
                                  so that the wait for it runs out                       */
} fa_cache_attn_params;

/* Scratch bytes fa_cache_attn needs for *p; host arithmetic only; 0 for a NULL p, and where a few short
 * sequences (by what the table can hold) need none. */
FA_EXPORT size_t fa_cache_attn_workspace_bytes(const fa_cache_attn_params *p);

/*
 * fa_cache_attn -- attention of a few query tokens for each sequence over the
 * cache, O and lse as in fa_fwd.  Made for decoding: each key and value is read
 * once for the query heads that share it (for up to 16 rows of heads and
 * tokens; once more for each further 16, 8 for d = 256).  The keys are split evenly
 * over the whole GPU whatever the sequences' lengths, and the parts are merged by a
 * second launch; few sequences that can hold few tokens (by max_pages) are
 * taken whole by clusters, in one launch.  For the many tokens of a prompt,
 * fa_fwd_ex on the contiguous keys (fa_cache_gather) is the faster call.  Sums,
 * softmax statistics and products accumulate in fp32.  For the product with the codes a weight
 * (times its page's value scale) is rounded by at most 2^-20 of itself, for FA_O_BF16 and more than 4
 * rows of heads and tokens by at most 2^-11; besides that by at most 2^-32 of the row's largest.  A row with
 * no allowed key gets O = 0, lse = -inf.  The keys of a page outside [0, n_pages) are left out
 * and FA_ERR_BAD_PAGE is stored.  Results do not depend on timing.
 */
FA_EXPORT fa_status fa_cache_attn(const fa_cache_attn_params *p, void *stream);

/*
 * Test hooks (not for production use): the scheduler slot the next causal
 * launch from this process will take, and a synchronous read (get4) and/or
 * overwrite (set4) of a slot's four words on the current device ([0] next
 * unit, [1] CTAs done, [2..3] the 64-bit owner, little-endian; all zero when
 * the slot is free).  They let a test hold a slot the way an in-flight
 * launch would, without a second launch.  Errors: FA_ERR_INVALID_ARGUMENT
 * for a slot outside [0, 64), FA_ERR_UNSUPPORTED / FA_ERR_CUDA from the
 * device.
 */
FA_EXPORT int fa_testhook_sched_next_slot(void);
FA_EXPORT fa_status fa_testhook_sched_slot(int slot, const uint32_t *set4, uint32_t *get4);

#ifdef __cplusplus
}
#endif

#endif /* EXACT_IO_AWARE_52_FA_H */
