"""Rotary positions and the paged 8-bit key/value cache: the binding of
fa_rope, fa_cache_append, fa_cache_attn and fa_cache_gather (include/fa.h).

Argument checks and marshalling only.  Every call runs on the device of its
tensors, whichever device is current, on `stream` (default: that device's
current stream), and allocates its outputs with torch unless they are given.
A wrong dtype, shape, layout or device raises ValueError, a status that the
library returns raises FaError; neither launches anything.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import _binding as fb

_LAYOUTS = {"half": fb.FA_ROTARY_HALF, "interleaved": fb.FA_ROTARY_INTERLEAVED}
_SCALINGS = {"none": fb.FA_ROTARY_NONE, "linear": fb.FA_ROTARY_LINEAR, "base": fb.FA_ROTARY_BASE,
             "parts": fb.FA_ROTARY_PARTS}
_DTYPES = {torch.bfloat16: fb.FA_T_BF16, torch.float32: fb.FA_T_F32}
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


def _internal(path, default):
    """A function of torch's internals that does a fraction of the public one's work on the host, if this
    torch has it."""
    at = torch._C
    for name in path.split("."):
        at = getattr(at, name, None)
        if at is None:
            return default
    return at


_raw_stream = _internal("_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = _internal("_cuda_getDevice", torch.cuda.current_device)
# (size, strides, dtype), on the current device
_empty_strided = _internal("_dynamo.guards._empty_strided_cuda",
                           lambda size, stride, dtype: torch.empty_strided(size, stride, dtype=dtype, device="cuda"))


def _empty(B, H, N, d, dtype):
    return _empty_strided((B, H, N, d), (H * N * d, N * d, d, 1), dtype)


# A decoding step makes several of these calls for kernels of a few microseconds, so the parameter
# structures are packed in one go (filling a ctypes.Structure takes several times as long).
_TENSOR = "PPi3q3q"
_ROPE = struct.Struct("@" + _TENSOR + _TENSOR + "iiiiiPqiiP")
_CACHE = struct.Struct("@PPPPPqiiiiii")
_APPEND = struct.Struct("@PP3q3qiPPPP")      # what follows the cache
_GATHER = struct.Struct("@PPPiP")
_ATTN = struct.Struct("@PPPPPiiifiPNIi")
for _s, _c, _rest in ((_ROPE, fb.FaRopeParams, 0), (_CACHE, fb.FaCache, 0), (_APPEND, fb.FaCacheAppendParams, _CACHE.size),
                      (_GATHER, fb.FaCacheGatherParams, _CACHE.size), (_ATTN, fb.FaCacheAttnParams, _CACHE.size)):
    assert _s.size + _rest == ctypes.sizeof(_c), _c.__name__
_calls = {}


def _call(name):
    """The library's function, taking a packed structure."""
    f = _calls.get(name)
    if f is None:
        f = fb.load()[name]
        f.restype = ctypes.c_int
        f.argtypes = [ctypes.c_char_p, ctypes.c_void_p]
        _calls[name] = f
    return f


def _refuse(what):
    raise ValueError(what)


def _pack(form, *values):
    try:
        return form.pack(*values)
    except (struct.error, OverflowError) as e:
        raise ValueError(f"an argument is not a number of its range: {e}") from None


def _ints(t, name, size, dev):
    """The address of an int32 tensor of this size on this device; 0 for None."""
    if t is None:
        return 0
    if t.dtype is not _I32 or t.dim() != 1 or t.shape[0] != size or t.get_device() != dev or not t.is_contiguous():
        _refuse(f"{name} must be a contiguous int32 tensor of {size} on the same device")
    return t.data_ptr()


def _heads(t, name, dev):
    if t.dim() != 4 or t.get_device() != dev or dev < 0:
        _refuse(f"{name} must be a CUDA tensor [B, heads, N, d], all on the same device")
    st = t.stride()
    if st[3] != 1 and t.shape[3] > 1:
        _refuse(f"{name}: the components of a head must be contiguous")
    return st


def _elsewhere(dev, stream):
    """The given device and stream as the current ones, so that tensors allocated
    meanwhile belong to that stream."""
    if stream is None:
        return torch.cuda.device(dev)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=dev) if stream else torch.cuda.default_stream(dev)
    if stream.device_index != dev:
        _refuse("stream belongs to another device than the tensors")
    return torch.cuda.stream(stream)


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
        if layout not in _LAYOUTS:
            _refuse(f"layout must be one of {sorted(_LAYOUTS)}")
        if scaling not in _SCALINGS:
            _refuse(f"scaling must be one of {sorted(_SCALINGS)}")
        if not amplitude > 0.0:
            _refuse("amplitude must be positive")
        spec = fb.FaRotarySpec(dim=int(dim), layout=_LAYOUTS[layout], base=float(base), scaling=_SCALINGS[scaling],
                               factor=float(factor), original_length=float(original_length),
                               low_turns=float(low_turns), high_turns=float(high_turns), amplitude=float(amplitude))
        if angles is not None:
            own = [float(a) for a in angles]
            if len(own) != int(dim) // 2:
                _refuse("angles must have one entry for each of the dim / 2 pairs")
            spec.angles = (ctypes.c_double * len(own))(*own)
        self.struct = fb.FaRotary()
        fb._check(fb.load().fa_rotary_init(ctypes.byref(self.struct), ctypes.byref(spec)), "fa_rotary_init")
        self.dim = int(dim)
        self.layout = layout
        self._address = ctypes.addressof(self.struct)

    def __getstate__(self):
        return {k: v for k, v in self.__dict__.items() if k != "_address"}

    def __setstate__(self, state):  # of a copy, which has a table of its own
        self.__dict__.update(state)
        self._address = ctypes.addressof(self.struct)


def rope(rotary, q, k=None, *, pos=None, pos0=0, inverse=False, out_dtype=None, out=None, stream=None):
    """fa_rope: the heads of q (and k, in the same launch) turned by their positions.

    q: [B, H, N, d], k: [B, H_kv, N, d], bf16 or fp32, any strides with contiguous
    components.  pos: int32 [B, N] or [N], or None: token n is at pos0 + n.
    inverse turns back by the same angles, which gives the gradient of q and k from
    that of the turned ones.  Returns the contiguous result in out_dtype (default: q's),
    or a pair with k.  out: a tensor (or a pair) to write instead, any strides; the inputs
    themselves turn in place.  They must not overlap the inputs otherwise.
    """
    dev = q.get_device()
    if not isinstance(rotary, Rotary):
        _refuse("rotary must be a Rotary")
    B, H, N, d = q.shape  # (ValueError for other numbers of dimensions)
    sq = q.stride()
    if dev < 0 or (sq[3] != 1 and d > 1):
        _refuse("q must be a CUDA tensor whose heads have contiguous components")
    x_dtype = q.dtype
    x_type = _DTYPES.get(x_dtype)
    if k is not None:
        Bk, Hk, Nk, dk = k.shape
        sk = k.stride()
        if Bk != B or Nk != N or dk != d or k.dtype is not x_dtype or k.get_device() != dev or (sk[3] != 1 and d > 1):
            _refuse("k must be [B, H_kv, N, d] of q's dtype, on its device, with contiguous components")
    if out is None:
        yq = yk = None
        y_dtype = x_dtype if out_dtype is None else out_dtype
    else:
        yq, yk = (out, None) if k is None else out
        y_dtype = yq.dtype
        for x, y in ((q, yq), (k, yk)):
            if x is not None:
                sy = _heads(y, "out", dev)
                if y.shape != x.shape or y.dtype is not y_dtype:
                    _refuse("out must have its input's shape, and both the same dtype")
                if 0 in sy and any(n > 1 and st == 0 for n, st in zip(y.shape, sy)):
                    _refuse("out must not be expanded")
        if out_dtype is not None and out_dtype is not y_dtype:
            _refuse("out must be of out_dtype")
    y_type = _DTYPES.get(y_dtype)
    if x_type is None or y_type is None:
        _refuse("dtypes must be bf16 or fp32")
    pos_at = pos_stride = 0
    if pos is not None:
        sp = pos.shape
        if (pos.dtype is not _I32 or pos.get_device() != dev or len(sp) not in (1, 2) or sp[-1] != N or
                (len(sp) == 2 and sp[0] != B) or (N > 1 and pos.stride(-1) != 1)):
            _refuse("pos must be int32 [B, N] or [N] on the same device, contiguous along the tokens")
        pos_at = pos.data_ptr()
        pos_stride = pos.stride(0) if len(sp) == 2 else 0
    if stream is not None or dev != _current_device():
        with _elsewhere(dev, stream):
            return rope(rotary, q, k, pos=pos, pos0=pos0, inverse=inverse, out_dtype=out_dtype, out=out)

    if yq is None:
        yq = _empty(B, H, N, d, y_dtype)
    syq = yq.stride()
    if k is None:
        p = _pack(_ROPE, q.data_ptr(), yq.data_ptr(), H, sq[0], sq[1], sq[2], syq[0], syq[1], syq[2],
                  0, 0, 0, 0, 0, 0, 0, 0, 0,
                  B, N, d, x_type, y_type, pos_at, pos_stride, pos0, 1 if inverse else 0, rotary._address)
    else:
        if yk is None:
            yk = _empty(B, Hk, N, d, y_dtype)
        syk = yk.stride()
        p = _pack(_ROPE, q.data_ptr(), yq.data_ptr(), H, sq[0], sq[1], sq[2], syq[0], syq[1], syq[2],
                  k.data_ptr(), yk.data_ptr(), Hk, sk[0], sk[1], sk[2], syk[0], syk[1], syk[2],
                  B, N, d, x_type, y_type, pos_at, pos_stride, pos0, 1 if inverse else 0, rotary._address)
    st = _call("fa_rope")(p, _raw_stream(dev))
    if st:
        raise fb.FaError(st, "fa_rope")
    return yq if k is None else (yq, yk)


class PagedCache:
    """A paged key/value cache in 8 bits: the caller's tensors, checked once.

    k, v: float8_e4m3fn (or uint8) [n_pages, H_kv, page, d], contiguous; page 16, 32,
    64 or 128, d 64, 128 or 256.  k_scale, v_scale: fp32 [n_pages, H_kv].
    table: int32 [B, max_pages]: token t of sequence b lies in slot t % page
    of page table[b, t // page]; entries past a sequence's end are not read.  What the
    tensors hold may change between calls; their places may not: for other tensors make
    another PagedCache (assigning to this one's is refused).  A deep copy has copies of the tensors.
    """

    def __init__(self, k, v, k_scale, v_scale, table):
        dev = k.get_device()
        if dev < 0 or k.dim() != 4 or k.shape != v.shape:
            _refuse("k and v must be CUDA tensors [n_pages, H_kv, page, d]")
        for t, name in ((k, "k"), (v, "v")):
            if t.dtype not in (torch.float8_e4m3fn, torch.uint8) or not t.is_contiguous() or t.get_device() != dev:
                _refuse(f"{name} must be a contiguous float8_e4m3fn (or uint8) tensor on the same device")
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t.dtype is not _F32 or t.shape != k.shape[:2] or not t.is_contiguous() or t.get_device() != dev:
                _refuse(f"{name} must be a contiguous fp32 [n_pages, H_kv] tensor on the same device")
        if (table.dtype is not _I32 or table.dim() != 2 or table.get_device() != dev or
                (table.shape[1] > 1 and table.stride(1) != 1)):
            _refuse("table must be int32 [B, max_pages] on the same device, contiguous along the pages")
        self.k, self.v, self.k_scale, self.v_scale, self.table = k, v, k_scale, v_scale, table
        self._workspace = {}  # (H, N) -> bytes
        self.device_index = dev
        self.n_pages, self.H_kv, self.page, self.d = k.shape
        self.B, self.max_pages = table.shape
        if self.page not in (16, 32, 64, 128) or self.d not in (64, 128, 256):
            _refuse("page must be 16, 32, 64 or 128 and d 64, 128 or 256")
        self._packed = _CACHE.pack(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                   table.data_ptr(), table.stride(0), self.n_pages, self.max_pages, self.B, self.H_kv,
                                   self.page, self.d)

    # What a call takes from the tensors it was made of, or follows from them.
    _FIXED = frozenset(("k", "v", "k_scale", "v_scale", "table", "device_index", "n_pages", "H_kv", "page", "d", "B",
                        "max_pages", "_workspace", "_packed"))

    def __setattr__(self, name, value):
        if name in self._FIXED and "_packed" in self.__dict__:
            raise AttributeError("a PagedCache is for the tensors that it was made of: make another one for others")
        super().__setattr__(name, value)

    def __getstate__(self):
        more = {name: value for name, value in self.__dict__.items() if name not in self._FIXED}
        return (self.k, self.v, self.k_scale, self.v_scale, self.table), more

    def __setstate__(self, state):  # of a copy: its addresses are its own tensors'
        tensors, more = state
        PagedCache.__init__(self, *tensors)
        self.__dict__.update(more)


def cache_append(cache, k, v, start, *, n_new=None, rotary=None, dev_status=None, stream=None):
    """fa_cache_append: writes new keys and values behind what each sequence holds.

    k, v: bf16 [B, H_kv, N, d], any strides with contiguous components.  start:
    int32 [B], the tokens that each sequence holds already.  n_new: int32 [B], how many of
    its N tokens are written (default: all).  rotary turns the keys by their
    positions on the way.  dev_status: int32 status word for FA_ERR_BAD_PAGE.  No page may be
    written through two entries of the table in one call.
    """
    dev = cache.device_index
    sk, sv = _heads(k, "k", dev), _heads(v, "v", dev)
    B, H, N, d = k.shape
    if B != cache.B or H != cache.H_kv or d != cache.d or v.shape != k.shape:
        _refuse(f"k and v must be [{cache.B}, {cache.H_kv}, N, {cache.d}]")
    if k.dtype is not _BF16 or v.dtype is not _BF16:
        _refuse("k and v must be bf16")
    if rotary is not None and not isinstance(rotary, Rotary):
        _refuse("rotary must be a Rotary")
    if start is None:
        _refuse("start must be given")
    p = cache._packed + _pack(
        _APPEND, k.data_ptr(), v.data_ptr(), sk[0], sk[1], sk[2], sv[0], sv[1], sv[2], N,
        _ints(start, "start", B, dev), _ints(n_new, "n_new", B, dev), 0 if rotary is None else rotary._address,
        _ints(dev_status, "dev_status", 1, dev))
    if stream is None and dev == _current_device():
        st = _call("fa_cache_append")(p, _raw_stream(dev))
    else:
        with _elsewhere(dev, stream):
            st = _call("fa_cache_append")(p, _raw_stream(dev))
    if st:
        raise fb.FaError(st, "fa_cache_append")


def cache_gather(cache, k_len, N_k, *, out=None, dev_status=None, stream=None):
    """fa_cache_gather: the first N_k tokens of every sequence as contiguous bf16 keys
    and values [B, H_kv, N_k, d], zero from token k_len[b] (int32 [B]) on: what
    attention(..., k_len=k_len) reads.  out: a pair of such tensors to write."""
    dev = cache.device_index
    N_k = int(N_k)
    if not 0 <= N_k < 1 << 31:
        _refuse("N_k must be in [0, 2^31)")
    shape = (cache.B, cache.H_kv, N_k, cache.d)
    if out is not None:
        for t in out:
            if t.dtype is not _BF16 or t.shape != shape or not t.is_contiguous() or t.get_device() != dev:
                _refuse(f"out must be two contiguous bf16 tensors of shape {shape}")
    if k_len is None:
        _refuse("k_len must be given")
    if stream is not None or dev != _current_device():
        with _elsewhere(dev, stream):
            return cache_gather(cache, k_len, N_k, out=out, dev_status=dev_status)
    if out is None:
        out = (_empty(*shape, _BF16), _empty(*shape, _BF16))
    k, v = out
    p = cache._packed + _pack(_GATHER, _ints(k_len, "k_len", cache.B, dev), k.data_ptr(), v.data_ptr(), N_k,
                                     _ints(dev_status, "dev_status", 1, dev))
    st = _call("fa_cache_gather")(p, _raw_stream(dev))
    if st:
        raise fb.FaError(st, "fa_cache_gather")
    return k, v


def cache_attention_workspace_bytes(cache, H, N):
    """Scratch bytes that cache_attention needs for H query heads and N query tokens."""
    size = cache._workspace.get((H, N))
    if size is None:
        f = fb.load()["fa_cache_attn_workspace_bytes"]
        f.restype = ctypes.c_size_t
        f.argtypes = [ctypes.c_char_p]
        size = cache._workspace[(H, N)] = f(cache._packed + _pack(_ATTN, 0, 0, 0, 0, 0, H, N, 0, 0.0, 0, 0, 0, 0, 0))
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
    if q.dim() != 4 or q.dtype is not _BF16 or not q.is_contiguous() or q.get_device() != dev:
        _refuse("q must be a contiguous bf16 [B, H, N, d] tensor on the cache's device")
    B, H, N, d = q.shape
    if B != cache.B or d != cache.d:
        _refuse(f"q must be [{cache.B}, H, N, {cache.d}]")
    if cache.H_kv and H % cache.H_kv:
        _refuse("H must be a multiple of the cache's heads")
    if out is None:
        o_dtype = _F32 if out_dtype is None else out_dtype
    else:
        o, lse = out
        o_dtype = o.dtype
        if (o.shape != q.shape or not o.is_contiguous() or o.get_device() != dev or lse.dtype is not _F32 or
                lse.shape != q.shape[:3] or not lse.is_contiguous() or lse.get_device() != dev or
                (out_dtype is not None and out_dtype is not o_dtype)):
            _refuse("out must be a contiguous O of q's shape and an fp32 lse [B, H, N] on the same device")
    if o_dtype is not _BF16 and o_dtype is not _F32:
        _refuse("out_dtype must be bf16 or fp32")
    if workspace is not None and (not workspace.is_contiguous() or workspace.get_device() != dev):
        _refuse("workspace must be contiguous and on the same device")
    if k_len is None:
        _refuse("k_len must be given")
    if stream is not None or dev != _current_device():
        with _elsewhere(dev, stream):
            return cache_attention(cache, q, k_len, causal, scale, out_dtype=out_dtype, out=out, workspace=workspace,
                                   dev_status=dev_status, timeout_ms=timeout_ms, test_drop_load=test_drop_load)
    if out is None:
        o = _empty(B, H, N, d, o_dtype)
        lse = _empty_strided((B, H, N), (H * N, N, 1), _F32)
    scratch = 0
    if workspace is None:
        size = cache_attention_workspace_bytes(cache, H, N)
        if size:
            workspace = _empty_strided((size,), (1,), torch.uint8)
            scratch = workspace.data_ptr()
    else:
        size = workspace.numel() * workspace.element_size()
        scratch = workspace.data_ptr()
    p = cache._packed + _pack(
        _ATTN, q.data_ptr(), o.data_ptr(), lse.data_ptr(), _ints(k_len, "k_len", B, dev), _ints(dev_status, "dev_status", 1, dev),
        H, N, 1 if causal else 0, scale, fb.FA_O_BF16 if o_dtype is _BF16 else fb.FA_O_F32, scratch, size,
        timeout_ms, test_drop_load)
    st = _call("fa_cache_attn")(p, _raw_stream(dev))
    if st:
        raise fb.FaError(st, "fa_cache_attn")
    return o, lse
