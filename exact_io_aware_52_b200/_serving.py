"""Rotary positions and the paged 8-bit key/value cache: the binding of
fa_rope, fa_cache_append, fa_cache_attn and fa_cache_gather (include/fa.h).

Argument checks and marshalling only.  Every call runs on the device of its
tensors, whichever device is current, on `stream` (default: that device's
current stream), and allocates its outputs with torch unless they are given.
A wrong dtype, shape, layout or device raises ValueError, a status that the
library returns raises FaError; neither launches anything.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _binding as fb

_LAYOUTS = {"half": fb.FA_ROTARY_HALF, "interleaved": fb.FA_ROTARY_INTERLEAVED}
_SCALINGS = {"none": fb.FA_ROTARY_NONE, "linear": fb.FA_ROTARY_LINEAR, "base": fb.FA_ROTARY_BASE,
             "parts": fb.FA_ROTARY_PARTS}
_DTYPES = {torch.bfloat16: fb.FA_T_BF16, torch.float32: fb.FA_T_F32}
_I3 = ctypes.c_int64 * 3


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _device_of(t, name):
    _need(t.is_cuda, f"{name} must be a CUDA tensor")
    return t.get_device()


def _ints(t, name, shape, dev):
    """The address of an int32 tensor of this shape on this device; None passes."""
    if t is None:
        return None
    _need(t.dtype == torch.int32 and tuple(t.shape) == shape and t.get_device() == dev and t.is_contiguous(),
          f"{name} must be a contiguous int32 tensor of shape {shape} on the same device")
    return t.data_ptr()


@contextlib.contextmanager
def _elsewhere(dev, stream):
    """The given device and stream as the current ones, so that tensors allocated
    meanwhile belong to that stream."""
    with torch.cuda.device(dev):
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream(dev)
        with torch.cuda.stream(stream):
            yield


def _run(dev, stream, call, *args):
    """call(*args) with `dev` and `stream` current."""
    if stream is None and dev == torch.cuda.current_device():
        return call(*args)
    with _elsewhere(dev, stream):
        return call(*args)


def _raw_stream(dev):
    return torch.cuda.current_stream(dev).cuda_stream


class Rotary:
    """A rotation by positions, ready for use (fa_rotary_init).

    dim: rotated leading components of each head (even, up to 256); layout:
    "half" pairs component i with i + dim / 2, "interleaved" 2 i with 2 i + 1.  Pair i
    turns by base^(-2 i / dim) radians for each position, changed for contexts longer
    than the original length by `scaling`: "linear" divides all by factor;
    "base" takes base * factor^(dim / (dim - 2)); "parts" divides what turns
    at most low_turns times within original_length, keeps what turns at least
    high_turns times, and goes linearly in between.  angles: radians per position for
    each pair, in place of all that.  amplitude multiplies the result.
    """

    def __init__(self, dim, layout="half", base=10000.0, scaling="none", factor=1.0, original_length=0.0,
                 low_turns=1.0, high_turns=32.0, amplitude=1.0, angles=None):
        _need(layout in _LAYOUTS, f"layout must be one of {sorted(_LAYOUTS)}")
        _need(scaling in _SCALINGS, f"scaling must be one of {sorted(_SCALINGS)}")
        _need(amplitude > 0.0, "amplitude must be positive")
        spec = fb.FaRotarySpec(dim=int(dim), layout=_LAYOUTS[layout], base=float(base), scaling=_SCALINGS[scaling],
                               factor=float(factor), original_length=float(original_length),
                               low_turns=float(low_turns), high_turns=float(high_turns), amplitude=float(amplitude))
        if angles is not None:
            own = [float(a) for a in angles]
            _need(len(own) == int(dim) // 2, "angles must have one entry for each of the dim / 2 pairs")
            spec.angles = (ctypes.c_double * len(own))(*own)
        self.struct = fb.FaRotary()
        fb._check(fb.load().fa_rotary_init(ctypes.byref(self.struct), ctypes.byref(spec)), "fa_rotary_init")
        self.dim = int(dim)
        self.layout = layout
        self._ref = ctypes.pointer(self.struct)


def _head_tensor(t, name):
    _need(t.dim() == 4, f"{name} must be [B, heads, N, d]")
    _need(t.shape[3] <= 1 or t.stride(3) == 1, f"{name}: the components of a head must be contiguous")


def rope(rotary, q, k=None, *, pos=None, pos0=0, inverse=False, out_dtype=None, out=None, stream=None):
    """fa_rope: the heads of q (and k, in the same launch) turned by their positions.

    q: [B, H, N, d], k: [B, H_kv, N, d], bf16 or fp32, any strides with contiguous
    components.  pos: int32 [B, N] or [N], or None: token n is at pos0 + n.
    inverse turns back by the same angles, which gives the gradient of q and k from
    that of the turned ones.  Returns the contiguous result in out_dtype (default: q's),
    or a pair with k.  out: a tensor (or a pair) to write instead, any strides; the inputs
    themselves turn in place.  They must not overlap the inputs otherwise.
    """
    dev = _device_of(q, "q")
    _need(isinstance(rotary, Rotary), "rotary must be a Rotary")
    _head_tensor(q, "q")
    B, H, N, d = q.shape
    if k is not None:
        _head_tensor(k, "k")
        _need(k.shape[0] == B and k.shape[2] == N and k.shape[3] == d and k.dtype == q.dtype and k.get_device() == dev,
              "k must be [B, H_kv, N, d] of q's dtype and on its device")
    if out is None:
        _need(q.dtype in _DTYPES and (out_dtype is None or out_dtype in _DTYPES), "dtypes must be bf16 or fp32")
        y_type = out_dtype or q.dtype
        outs = None
    else:
        outs = tuple(out) if k is not None else (out,)
        y_type = outs[0].dtype
        for x, y, name in zip((q, k), outs, ("out of q", "out of k")):
            _head_tensor(y, name)
            _need(y.shape == x.shape and y.get_device() == dev and y.dtype == y_type,
                  f"{name} must have its input's shape and device, and both the same dtype")
        _need(q.dtype in _DTYPES and y_type in _DTYPES and (out_dtype is None or out_dtype == y_type),
              "dtypes must be bf16 or fp32, and out of out_dtype")
    pos_stride = 0
    if pos is not None:
        _need(pos.dtype == torch.int32 and pos.get_device() == dev and pos.shape[-1:] == (N,) and
              (pos.dim() == 1 or (pos.dim() == 2 and pos.shape[0] == B)) and (N <= 1 or pos.stride(-1) == 1),
              "pos must be int32 [B, N] or [N] on the same device, contiguous along the tokens")
        pos_stride = pos.stride(0) if pos.dim() == 2 else 0
    return _run(dev, stream, _rope, rotary, q, k, outs, y_type, pos, pos_stride, int(pos0), int(bool(inverse)), dev)


def _rope(rotary, q, k, outs, y_type, pos, pos_stride, pos0, inverse, dev):
    B, H, N, d = q.shape
    if outs is None:
        outs = (torch.empty((B, H, N, d), dtype=y_type, device=q.device),)
        if k is not None:
            outs += (torch.empty(k.shape, dtype=y_type, device=q.device),)
    p = fb.FaRopeParams()
    for t, x, y in zip(p.t, (q, k), outs):
        t.x = x.data_ptr()
        t.y = y.data_ptr()
        t.heads = x.shape[1]
        t.x_stride[:] = x.stride()[:3]
        t.y_stride[:] = y.stride()[:3]
    p.B, p.N, p.d = B, N, d
    p.x_dtype, p.y_dtype = _DTYPES[q.dtype], _DTYPES[y_type]
    if pos is not None:
        p.pos = pos.data_ptr()
        p.pos_stride = pos_stride
    p.pos0 = pos0
    p.inverse = inverse
    p.rotary = rotary._ref
    fb._check(fb.load().fa_rope(p, _raw_stream(dev)), "fa_rope")
    return outs if k is not None else outs[0]


class PagedCache:
    """A paged key/value cache in 8 bits: the caller's tensors, checked once.

    k, v: float8_e4m3fn (or uint8) [n_pages, H_kv, page, d], contiguous; page 16, 32,
    64 or 128, d 64, 128 or 256.  k_scale, v_scale: fp32 [n_pages, H_kv].
    table: int32 [B, max_pages]: token t of sequence b lies in slot t % page
    of page table[b, t // page]; entries past a sequence's end are not read.  What the
    tensors hold may change between calls; their places may not.
    """

    def __init__(self, k, v, k_scale, v_scale, table):
        dev = _device_of(k, "k")
        _need(k.dim() == 4 and k.shape == v.shape, "k and v must be [n_pages, H_kv, page, d]")
        for t, name in ((k, "k"), (v, "v")):
            _need(t.dtype in (torch.float8_e4m3fn, torch.uint8) and t.is_contiguous() and t.get_device() == dev,
                  f"{name} must be a contiguous float8_e4m3fn (or uint8) tensor on the same device")
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            _need(t.dtype == torch.float32 and t.shape == k.shape[:2] and t.is_contiguous() and t.get_device() == dev,
                  f"{name} must be a contiguous fp32 [n_pages, H_kv] tensor on the same device")
        _need(table.dtype == torch.int32 and table.dim() == 2 and table.get_device() == dev and
              (table.shape[1] <= 1 or table.stride(1) == 1),
              "table must be int32 [B, max_pages] on the same device, contiguous along the pages")
        self.k, self.v, self.k_scale, self.v_scale, self.table = k, v, k_scale, v_scale, table
        self.device_index = dev
        self.n_pages, self.H_kv, self.page, self.d = k.shape
        self.B, self.max_pages = table.shape
        self.struct = fb.FaCache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), table.data_ptr(),
                                 table.stride(0), self.n_pages, self.max_pages, self.B, self.H_kv, self.page, self.d)
        _need(self.page in (16, 32, 64, 128) and self.d in (64, 128, 256),
              "page must be 16, 32, 64 or 128 and d 64, 128 or 256")
        self._workspace = {}  # (H, N) -> bytes


def cache_append(cache, k, v, start, *, n_new=None, rotary=None, dev_status=None, stream=None):
    """fa_cache_append: writes new keys and values behind what each sequence holds.

    k, v: bf16 [B, H_kv, N, d], any strides with contiguous components.  start:
    int32 [B], the tokens that each sequence holds already.  n_new: int32 [B], how many of
    its N tokens are written (default: all).  rotary turns the keys by their
    positions on the way.  dev_status: int32 status word for FA_ERR_BAD_PAGE.
    """
    dev = cache.device_index
    for t, name in ((k, "k"), (v, "v")):
        _head_tensor(t, name)
        _need(t.dtype == torch.bfloat16 and t.get_device() == dev, f"{name} must be bf16 on the cache's device")
    N = k.shape[2]
    _need(tuple(k.shape) == (cache.B, cache.H_kv, N, cache.d) and v.shape == k.shape,
          f"k and v must be [{cache.B}, {cache.H_kv}, N, {cache.d}]")
    _need(rotary is None or isinstance(rotary, Rotary), "rotary must be a Rotary")
    p = fb.FaCacheAppendParams(
        cache.struct, k.data_ptr(), v.data_ptr(), _I3(*k.stride()[:3]), _I3(*v.stride()[:3]), N,
        _ints(start, "start", (cache.B,), dev), _ints(n_new, "n_new", (cache.B,), dev),
        None if rotary is None else rotary._ref, _ints(dev_status, "dev_status", (1,), dev))
    _run(dev, stream, _append, p, dev)


def _append(p, dev):
    fb._check(fb.load().fa_cache_append(p, _raw_stream(dev)), "fa_cache_append")


def cache_gather(cache, k_len, N_k, *, out=None, dev_status=None, stream=None):
    """fa_cache_gather: the first N_k tokens of every sequence as contiguous bf16 keys
    and values [B, H_kv, N_k, d], zero from token k_len[b] (int32 [B]) on: what
    attention(..., k_len=k_len) reads.  out: a pair of such tensors to write."""
    dev = cache.device_index
    N_k = int(N_k)
    _need(N_k >= 0, "N_k must not be negative")
    shape = (cache.B, cache.H_kv, N_k, cache.d)
    if out is not None:
        for t in out:
            _need(t.dtype == torch.bfloat16 and tuple(t.shape) == shape and t.is_contiguous() and
                  t.get_device() == dev, f"out must be two contiguous bf16 tensors of shape {shape}")
    return _run(dev, stream, _gather, cache, _ints(k_len, "k_len", (cache.B,), dev), shape, out,
                _ints(dev_status, "dev_status", (1,), dev), dev)


def _gather(cache, k_len, shape, out, dev_status, dev):
    if out is None:
        out = tuple(torch.empty(shape, dtype=torch.bfloat16, device=cache.k.device) for _ in range(2))
    p = fb.FaCacheGatherParams(cache.struct, k_len, out[0].data_ptr(), out[1].data_ptr(), shape[2], dev_status)
    fb._check(fb.load().fa_cache_gather(p, _raw_stream(dev)), "fa_cache_gather")
    return tuple(out)


def cache_attention_workspace_bytes(cache, H, N):
    """Scratch bytes that cache_attention needs for H query heads and N query tokens."""
    size = cache._workspace.get((H, N))
    if size is None:
        p = fb.FaCacheAttnParams(cache=cache.struct, H=H, N=N)
        size = cache._workspace[(H, N)] = int(fb.load().fa_cache_attn_workspace_bytes(ctypes.byref(p)))
    return size


def cache_attention(cache, q, k_len, causal, scale, *, out_dtype=None, out=None, workspace=None, dev_status=None,
                    timeout_ms=0, stream=None, test_drop_load=0):
    """fa_cache_attn: attention of N query tokens for each sequence over the cache.

    q: bf16 [B, H, N, d], contiguous, H a multiple of the cache's heads.  k_len:
    int32 [B], the tokens that each sequence holds, the queries' own included.  causal:
    query i of sequence b sits at position k_len[b] - N + i.  Returns O in
    out_dtype (fp32 default) and lse (fp32 [B, H, N]), or writes the pair `out`.  workspace: a
    tensor of cache_attention_workspace_bytes bytes, not shared by calls that overlap
    (two captured graphs, say); allocated for the call by default.  dev_status: int32 status
    word for FA_ERR_BAD_PAGE and FA_ERR_DEVICE_TIMEOUT (a wait longer than timeout_ms, 0 = 2000).
    """
    dev = cache.device_index
    _need(q.dim() == 4 and q.dtype == torch.bfloat16 and q.is_contiguous() and q.get_device() == dev,
          "q must be a contiguous bf16 [B, H, N, d] tensor on the cache's device")
    B, H, N, d = q.shape
    _need(B == cache.B and d == cache.d, f"q must be [{cache.B}, H, N, {cache.d}]")
    _need(cache.H_kv == 0 or H % cache.H_kv == 0, "H must be a multiple of the cache's heads")
    o_type = out_dtype or torch.float32
    if out is not None:
        o, lse = out
        o_type = o.dtype
        _need(o.shape == q.shape and o.is_contiguous() and o.get_device() == dev and lse.dtype == torch.float32 and
              lse.shape == q.shape[:3] and lse.is_contiguous() and lse.get_device() == dev and
              (out_dtype is None or out_dtype == o_type),
              "out must be a contiguous O of q's shape and an fp32 lse [B, H, N] on the same device")
    _need(o_type in _DTYPES, "out_dtype must be bf16 or fp32")
    if workspace is not None:
        _need(workspace.is_contiguous() and workspace.get_device() == dev,
              "workspace must be contiguous and on the same device")
    return _run(dev, stream, _attention, cache, q, _ints(k_len, "k_len", (B,), dev), int(bool(causal)), float(scale),
                out, o_type, workspace, _ints(dev_status, "dev_status", (1,), dev), timeout_ms, test_drop_load, dev)


def _attention(cache, q, k_len, causal, scale, out, o_type, workspace, dev_status, timeout_ms, test_drop_load, dev):
    B, H, N, d = q.shape
    if out is None:
        out = (torch.empty((B, H, N, d), dtype=o_type, device=q.device),
               torch.empty((B, H, N), dtype=torch.float32, device=q.device))
    if workspace is None:
        workspace = torch.empty(cache_attention_workspace_bytes(cache, H, N), dtype=torch.uint8, device=q.device)
    p = fb.FaCacheAttnParams(cache.struct, q.data_ptr(), out[0].data_ptr(), out[1].data_ptr(), k_len, dev_status, H, N,
                             causal, scale, fb.FA_O_BF16 if o_type == torch.bfloat16 else fb.FA_O_F32,
                             workspace.data_ptr(),
                             workspace.numel() * workspace.element_size(), timeout_ms, test_drop_load)
    fb._check(fb.load().fa_cache_attn(p, _raw_stream(dev)), "fa_cache_attn")
    return tuple(out)
