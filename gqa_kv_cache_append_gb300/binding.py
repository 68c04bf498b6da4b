"""Thin ctypes binding of libgqa.so (include/gqa.h), same names as the C ABI.

Argument marshalling only: tensors become device pointers, torch dtypes
become GQA_F32 / GQA_BF16, and the current torch CUDA stream is passed when
no stream is given.  Every step of the computation runs in the library's
CUDA kernels; there is no fallback.  Loading fails loudly when the library
has not been built (``python -m gqa_kv_cache_append_gb300.build``).
"""
from __future__ import annotations

import ctypes
import os

import torch

from .build import LIB

GQA_F32 = 0
GQA_BF16 = 1
GQA_F16 = 2

GQA_OK = 0
GQA_ERR_NULL = -1
GQA_ERR_SHAPE = -2
GQA_ERR_DTYPE = -3
GQA_ERR_ALIGN = -4
GQA_ERR_UNSUPPORTED = -5
GQA_ERR_CUDA = -6
GQA_ERR_DEVICE = -7
GQA_ERR_SCRATCH_LIMIT = -8

GQA_STEP_EARLY_STREAM = 1
GQA_STEP_CUDA_CORES = 2

GQA_DEV_BAD_SEQ_LEN = 1
GQA_DEV_WAIT_TIMEOUT = 2
GQA_DEV_INTERNAL = 4
GQA_DEV_BAD_BLOCK = 8
GQA_DEV_BAD_TOKENS = 16

GQA_ROPE_HALF = 0
GQA_ROPE_PAIRS = 1
GQA_ROPE_PLAIN = 0
GQA_ROPE_LINEAR = 1
GQA_ROPE_WAVELENGTH = 2
GQA_ROPE_YARN = 3

# every function the header declares, with its C signature
_VP, _I, _F, _LL = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_longlong
_D = ctypes.c_double
# q .. rope_scale, q_out, k_cache, v_cache of the rotate-and-append calls
_ROPE = [_VP, _VP, _VP, _LL, _LL, _LL, _VP, _VP, _VP, _VP, _F, _VP, _I, _I, _F, _VP, _VP, _VP]
SIGNATURES = {
    "gqa_kv_append": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I, _VP]),
    "gqa_decode_attn": (_I, [_VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _F, _VP, _I, _I, _VP]),
    "gqa_decode_attn_noalloc": (_I, [_VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _F, _VP, _I, _I,
                                     _VP]),
    "gqa_decode_step": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _F, _VP, _I,
                             _I, _I, _VP]),
    "gqa_kv_append_multi": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I, _I, _VP]),
    "gqa_decode_attn_multi": (_I, [_VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I, _F, _VP, _I, _I,
                                   _VP]),
    "gqa_decode_step_multi": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I, _F,
                                   _VP, _I, _I, _I, _VP]),
    "gqa_project_qkv": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I, _I,
                             _I, _VP]),
    "gqa_project_out": (_I, [_VP, _VP, _VP, _I, _I, _I, _I, _I, _I, _VP]),
    "gqa_decode_layer": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I,
                              _F, _VP, _I, _I, _I, _VP]),
    "gqa_kv_append_paged": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I, _I, _I,
                                 _I, _VP]),
    "gqa_decode_attn_paged": (_I, [_VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I, _F, _VP, _I,
                                   _I, _I, _I, _VP]),
    "gqa_decode_step_paged": (_I, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _I, _I, _I, _I, _I, _I,
                                   _F, _VP, _I, _I, _I, _I, _I, _VP]),
    "gqa_decode_plan": (_I, [_I, _I, _I, _I, _I, _I, _I, _I, _I, _I, ctypes.POINTER(_I),
                             ctypes.POINTER(_I), ctypes.POINTER(_I), ctypes.POINTER(_I),
                             ctypes.POINTER(_LL), ctypes.POINTER(_I)]),
    "gqa_rope_table": (_I, [_I, _D, _I, _D, _D, _D, _D, ctypes.POINTER(ctypes.c_uint64),
                            ctypes.POINTER(_F)]),
    "gqa_rope_append": (_I, _ROPE + [_I] * 8 + [_VP]),
    "gqa_rope_append_paged": (_I, _ROPE + [_VP] + [_I] * 10 + [_VP]),
    "gqa_rope_append_fp8_paged": (_I, _ROPE + [_VP, _VP, _VP] + [_I] * 10 + [_VP]),
    "gqa_kv_read_fp8_paged": (_I, [_VP] * 8 + [_I] * 9 + [_VP]),
    "gqa_chunk_attn": (_I, [_VP] * 5 + [_I] * 6 + [_F, _VP, _I, _I, _VP, _LL, _VP]),
    "gqa_chunk_attn_paged": (_I, [_VP] * 6 + [_I] * 6 + [_F, _VP] + [_I] * 4 + [_VP, _LL, _VP]),
    "gqa_chunk_attn_workspace": (_I, [_I] * 6 + [ctypes.POINTER(_LL)]),
    "gqa_decode_attn_fp8_paged": (_I, [_VP] * 7 + [_I] * 6 + [_F, _VP] + [_I] * 4 +
                                  [_VP, _LL, _VP]),
    "gqa_decode_attn_fp8_workspace": (_I, [_I] * 6 + [_LL, _I, ctypes.POINTER(_LL)]),
    "gqa_device_status": (_I, [_VP, ctypes.POINTER(ctypes.c_uint32)]),
    "gqa_selftest_wait_timeout": (_I, [_LL, _VP]),
    "gqa_status_string": (ctypes.c_char_p, [_I]),
    "gqa_version": (_I, []),
}


class GqaError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} returned {code} ({status_string(code)})")
        self.code = code


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB):
        raise ImportError(
            f"{LIB} is missing: build it with `python -m gqa_kv_cache_append_gb300.build` "
            "(or __graft_entry__.build()); there is no fallback implementation")
    lib = ctypes.CDLL(LIB)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


def status_string(code: int) -> str:
    return lib.gqa_status_string(int(code)).decode()


def _ptr(x, name: str = "tensor", nbytes: int = 0, index: bool = False) -> int:
    """Device address of a tensor argument (raw integers pass through
    unchecked).  The kernels read and write whole extents through it, so a
    host tensor, a strided view, a tensor smaller than the shapes passed
    (nbytes) or, for lengths and block tables (index), another type than
    int32 is refused here, before anything is launched."""
    if isinstance(x, torch.Tensor):
        if not x.is_contiguous():
            raise ValueError(f"{name}: must be contiguous")
        if index and x.dtype != torch.int32:
            raise ValueError(f"{name}: must be int32, got {x.dtype}")
        have = x.numel() * x.element_size()
        if have < nbytes:
            raise ValueError(f"{name}: holds {have} bytes, the shapes passed need {nbytes}")
        if not x.is_cuda:
            # reported by _call once every argument has been checked
            return _HostTensor(name, x.device)
        return x.data_ptr()
    return int(x) if x is not None else 0


class _HostTensor:
    """Stands for a tensor argument that is not on a CUDA device."""

    def __init__(self, name, device):
        self.name, self.device = name, device


def _call(fn_name: str, fn, *args) -> None:
    """Call a library entry point once no argument is a host tensor; raise
    GqaError on a non-zero return code."""
    for a in args:
        if isinstance(a, _HostTensor):
            raise ValueError(f"{a.name}: a CUDA tensor is required, got one on {a.device}")
    _check(fn_name, fn(*args))


def _elt(code: int) -> int:
    """Bytes per element of a dtype code (0 for an unknown code, which the
    library rejects)."""
    return {GQA_F32: 4, GQA_BF16: 2, GQA_F16: 2}.get(code, 0)


def _n(*dims) -> int:
    """Product of the dims, 0 when one is not positive (the library then
    reports the shape error)."""
    out = 1
    for d in dims:
        d = int(d)
        if d <= 0:
            return 0
        out *= d
    return out


def _dtype(x, dtype) -> int:
    if dtype is not None:
        return int(dtype)
    if isinstance(x, torch.Tensor):
        if x.dtype == torch.bfloat16:
            return GQA_BF16
        if x.dtype == torch.float32:
            return GQA_F32
        if x.dtype == torch.float16:
            return GQA_F16
        return -99  # the library rejects it with GQA_ERR_DTYPE
    raise ValueError("dtype must be given when passing raw pointers")


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(fn: str, code: int) -> None:
    if code != GQA_OK:
        raise GqaError(fn, code)


def gqa_kv_append(k_new, v_new, k_cache, v_cache, seq_lens, b, g, d_k, d_v,
                  cap=None, dtype=None, stream=None) -> None:
    """Write row seq_lens[i] - 1 of every (i, j) of the caches (in place)."""
    if cap is None:
        cap = k_cache.shape[2]
    dt = _dtype(k_cache, dtype)
    e = _elt(dt)
    _call("gqa_kv_append", lib.gqa_kv_append,
        _ptr(k_new, "k_new", _n(b, g, d_k) * e), _ptr(v_new, "v_new", _n(b, g, d_v) * e),
        _ptr(k_cache, "k_cache", _n(b, g, cap, d_k) * e),
        _ptr(v_cache, "v_cache", _n(b, g, cap, d_v) * e),
        _ptr(seq_lens, "seq_lens", _n(b) * 4, index=True),
        int(b), int(g), int(d_k), int(d_v), int(cap), dt, _stream(stream))


def gqa_decode_attn(q, k_cache, v_cache, seq_lens, b, h, g, d_k, d_v, scale,
                    out, cap=None, dtype=None, stream=None) -> None:
    """out[i, a, :] = softmax_p(scale * q[i, a] . K[i, a // (h/g), p]) V[...]."""
    if cap is None:
        cap = k_cache.shape[2]
    dt = _dtype(q, dtype)
    e = _elt(dt)
    _call("gqa_decode_attn", lib.gqa_decode_attn,
        _ptr(q, "q", _n(b, h, d_k) * e), _ptr(k_cache, "k_cache", _n(b, g, cap, d_k) * e),
        _ptr(v_cache, "v_cache", _n(b, g, cap, d_v) * e),
        _ptr(seq_lens, "seq_lens", _n(b) * 4, index=True), int(b), int(h),
        int(g), int(d_k), int(d_v), float(scale), _ptr(out, "out", _n(b, h, d_v) * e), int(cap),
        dt, _stream(stream))


def gqa_decode_step(q, k_new, v_new, k_cache, v_cache, seq_lens, b, h, g, d_k, d_v,
                    scale, out, cap=None, dtype=None, flags=0, stream=None) -> None:
    """Append k_new / v_new at row seq_lens[i] - 1 and attend, in one launch.
    flags=GQA_STEP_EARLY_STREAM: see include/gqa.h (the kernels still running
    ahead on the stream must not write seq_lens or this call's older rows)."""
    if cap is None:
        cap = k_cache.shape[2]
    dt = _dtype(q, dtype)
    e = _elt(dt)
    _call("gqa_decode_step", lib.gqa_decode_step,
        _ptr(q, "q", _n(b, h, d_k) * e), _ptr(k_new, "k_new", _n(b, g, d_k) * e),
        _ptr(v_new, "v_new", _n(b, g, d_v) * e), _ptr(k_cache, "k_cache", _n(b, g, cap, d_k) * e),
        _ptr(v_cache, "v_cache", _n(b, g, cap, d_v) * e),
        _ptr(seq_lens, "seq_lens", _n(b) * 4, index=True),
        int(b), int(h), int(g), int(d_k), int(d_v), float(scale),
        _ptr(out, "out", _n(b, h, d_v) * e), int(cap), dt, int(flags), _stream(stream))


def gqa_decode_attn_noalloc(q, k_cache, v_cache, seq_lens, b, h, g, d_k, d_v, scale,
                            out, cap=None, dtype=None, stream=None) -> None:
    """gqa_decode_attn for callers that cannot allocate device memory: the
    split partials live in the library's fixed 4 MiB device array instead of
    a cudaMalloc'd workspace.  Calls share that array, so calls that overlap
    on the GPU race; make the first call on a device before any stream
    capture (it looks up the array's device address)."""
    if cap is None:
        cap = k_cache.shape[2]
    dt = _dtype(q, dtype)
    e = _elt(dt)
    _call("gqa_decode_attn_noalloc", lib.gqa_decode_attn_noalloc,
        _ptr(q, "q", _n(b, h, d_k) * e), _ptr(k_cache, "k_cache", _n(b, g, cap, d_k) * e),
        _ptr(v_cache, "v_cache", _n(b, g, cap, d_v) * e),
        _ptr(seq_lens, "seq_lens", _n(b) * 4, index=True), int(b), int(h),
        int(g), int(d_k), int(d_v), float(scale), _ptr(out, "out", _n(b, h, d_v) * e), int(cap),
        dt, _stream(stream))


def gqa_kv_append_multi(k_new, v_new, k_cache, v_cache, seq_lens, b, n, g, d_k, d_v,
                        cap=None, dtype=None, stream=None) -> None:
    """Write rows seq_lens[i] - n .. seq_lens[i] - 1 of every (i, j) of the
    caches from k_new / v_new [b, n, g, d] (in place)."""
    if cap is None:
        cap = k_cache.shape[2]
    dt = _dtype(k_cache, dtype)
    e = _elt(dt)
    _call("gqa_kv_append_multi", lib.gqa_kv_append_multi,
        _ptr(k_new, "k_new", _n(b, n, g, d_k) * e), _ptr(v_new, "v_new", _n(b, n, g, d_v) * e),
        _ptr(k_cache, "k_cache", _n(b, g, cap, d_k) * e),
        _ptr(v_cache, "v_cache", _n(b, g, cap, d_v) * e),
        _ptr(seq_lens, "seq_lens", _n(b) * 4, index=True),
        int(b), int(n), int(g), int(d_k), int(d_v), int(cap), dt, _stream(stream))


def gqa_decode_attn_multi(q, k_cache, v_cache, seq_lens, b, n, h, g, d_k, d_v, scale,
                          out, cap=None, dtype=None, stream=None) -> None:
    """n queries per sequence (q, out [b, n, h, d]) with the causal mask:
    token s sees positions p <= seq_lens[i] - n + s."""
    if cap is None:
        cap = k_cache.shape[2]
    dt = _dtype(q, dtype)
    e = _elt(dt)
    _call("gqa_decode_attn_multi", lib.gqa_decode_attn_multi,
        _ptr(q, "q", _n(b, n, h, d_k) * e), _ptr(k_cache, "k_cache", _n(b, g, cap, d_k) * e),
        _ptr(v_cache, "v_cache", _n(b, g, cap, d_v) * e),
        _ptr(seq_lens, "seq_lens", _n(b) * 4, index=True), int(b), int(n), int(h),
        int(g), int(d_k), int(d_v), float(scale), _ptr(out, "out", _n(b, n, h, d_v) * e),
        int(cap), dt, _stream(stream))


def gqa_decode_step_multi(q, k_new, v_new, k_cache, v_cache, seq_lens, b, n, h, g, d_k,
                          d_v, scale, out, cap=None, dtype=None, flags=0,
                          stream=None) -> None:
    """Append the n new rows and attend causally, in one launch."""
    if cap is None:
        cap = k_cache.shape[2]
    dt = _dtype(q, dtype)
    e = _elt(dt)
    _call("gqa_decode_step_multi", lib.gqa_decode_step_multi,
        _ptr(q, "q", _n(b, n, h, d_k) * e), _ptr(k_new, "k_new", _n(b, n, g, d_k) * e),
        _ptr(v_new, "v_new", _n(b, n, g, d_v) * e),
        _ptr(k_cache, "k_cache", _n(b, g, cap, d_k) * e),
        _ptr(v_cache, "v_cache", _n(b, g, cap, d_v) * e),
        _ptr(seq_lens, "seq_lens", _n(b) * 4, index=True),
        int(b), int(n), int(h), int(g), int(d_k), int(d_v), float(scale),
        _ptr(out, "out", _n(b, n, h, d_v) * e), int(cap), dt, int(flags), _stream(stream))


def gqa_project_qkv(x, w_q, w_k, w_v, q, k_new, v_new, b, d_model, h, g, d_k, d_v,
                    dtype=None, flags=0, stream=None) -> None:
    """q / k_new / v_new = x . P_q / P_k / P_v ("bd,hdk->bhk" and its KV forms)."""
    dt = _dtype(x, dtype)
    e, D = _elt(dt), d_model
    _call("gqa_project_qkv", lib.gqa_project_qkv,
        _ptr(x, "x", _n(b, D) * e), _ptr(w_q, "w_q", _n(h, D, d_k) * e),
        _ptr(w_k, "w_k", _n(g, D, d_k) * e), _ptr(w_v, "w_v", _n(g, D, d_v) * e),
        _ptr(q, "q", _n(b, h, d_k) * e), _ptr(k_new, "k_new", _n(b, g, d_k) * e),
        _ptr(v_new, "v_new", _n(b, g, d_v) * e),
        int(b), int(d_model), int(h), int(g), int(d_k), int(d_v), dt, int(flags),
        _stream(stream))


def gqa_project_out(o, w_o, y, b, d_model, h, d_v, dtype=None, flags=0, stream=None) -> None:
    """y = "bhv,hdv->bd"(o, P_o)."""
    dt = _dtype(o, dtype)
    e, D = _elt(dt), d_model
    _call("gqa_project_out", lib.gqa_project_out,
        _ptr(o, "o", _n(b, h, d_v) * e), _ptr(w_o, "w_o", _n(h, D, d_v) * e),
        _ptr(y, "y", _n(b, D) * e), int(b), int(d_model), int(h), int(d_v), dt, int(flags),
        _stream(stream))


def gqa_decode_layer(x, w_q, w_k, w_v, w_o, k_cache, v_cache, seq_lens, b, d_model, h, g,
                     d_k, d_v, scale, y, cap=None, dtype=None, flags=0, stream=None) -> None:
    """The incremental layer: project x, append, attend, project the output."""
    if cap is None:
        cap = k_cache.shape[2]
    dt = _dtype(x, dtype)
    e, D = _elt(dt), d_model
    _call("gqa_decode_layer", lib.gqa_decode_layer,
        _ptr(x, "x", _n(b, D) * e), _ptr(w_q, "w_q", _n(h, D, d_k) * e),
        _ptr(w_k, "w_k", _n(g, D, d_k) * e), _ptr(w_v, "w_v", _n(g, D, d_v) * e),
        _ptr(w_o, "w_o", _n(h, D, d_v) * e), _ptr(k_cache, "k_cache", _n(b, g, cap, d_k) * e),
        _ptr(v_cache, "v_cache", _n(b, g, cap, d_v) * e),
        _ptr(seq_lens, "seq_lens", _n(b) * 4, index=True), int(b), int(d_model), int(h),
        int(g), int(d_k), int(d_v), float(scale), _ptr(y, "y", _n(b, D) * e), int(cap), dt,
        int(flags), _stream(stream))


def _paged_ptrs(k_pool, v_pool, block_table, b, g, d_k, d_v, e):
    """Checked pool and table pointers, and (block_size, max_blocks,
    num_blocks) read from the pool [num_blocks, g, block_size, d_k] and the
    table [b, max_blocks]."""
    nb, _, bs, _ = k_pool.shape
    mb = block_table.shape[1]
    return (_ptr(k_pool, "k_pool", _n(nb, g, bs, d_k) * e),
            _ptr(v_pool, "v_pool", _n(nb, g, bs, d_v) * e),
            _ptr(block_table, "block_table", _n(b, mb) * 4, index=True), int(bs), int(mb), int(nb))


def gqa_kv_append_paged(k_new, v_new, k_pool, v_pool, block_table, seq_lens, b, g, d_k, d_v,
                        n=1, dtype=None, stream=None) -> None:
    """Append n new rows per sequence into a paged cache (pools
    [num_blocks, g, block_size, d], block_table [b, max_blocks])."""
    dt = _dtype(k_pool, dtype)
    e = _elt(dt)
    kp, vp, tp, bs, mb, nb = _paged_ptrs(k_pool, v_pool, block_table, b, g, d_k, d_v, e)
    _call("gqa_kv_append_paged", lib.gqa_kv_append_paged,
        _ptr(k_new, "k_new", _n(b, n, g, d_k) * e), _ptr(v_new, "v_new", _n(b, n, g, d_v) * e),
        kp, vp, tp, _ptr(seq_lens, "seq_lens", _n(b) * 4, index=True),
        int(b), int(n), int(g), int(d_k), int(d_v), bs, mb, nb, dt, _stream(stream))


def gqa_decode_attn_paged(q, k_pool, v_pool, block_table, seq_lens, b, h, g, d_k, d_v, scale,
                          out, n=1, dtype=None, stream=None) -> None:
    """gqa_decode_attn (n = 1) or gqa_decode_attn_multi over a paged cache."""
    dt = _dtype(q, dtype)
    e = _elt(dt)
    kp, vp, tp, bs, mb, nb = _paged_ptrs(k_pool, v_pool, block_table, b, g, d_k, d_v, e)
    _call("gqa_decode_attn_paged", lib.gqa_decode_attn_paged,
        _ptr(q, "q", _n(b, n, h, d_k) * e), kp, vp, tp,
        _ptr(seq_lens, "seq_lens", _n(b) * 4, index=True), int(b), int(n),
        int(h), int(g), int(d_k), int(d_v), float(scale), _ptr(out, "out", _n(b, n, h, d_v) * e),
        bs, mb, nb, dt, _stream(stream))


def gqa_decode_step_paged(q, k_new, v_new, k_pool, v_pool, block_table, seq_lens, b, h, g, d_k,
                          d_v, scale, out, n=1, dtype=None, flags=0, stream=None) -> None:
    """Append and attend over a paged cache in one launch (n new tokens)."""
    dt = _dtype(q, dtype)
    e = _elt(dt)
    kp, vp, tp, bs, mb, nb = _paged_ptrs(k_pool, v_pool, block_table, b, g, d_k, d_v, e)
    _call("gqa_decode_step_paged", lib.gqa_decode_step_paged,
        _ptr(q, "q", _n(b, n, h, d_k) * e), _ptr(k_new, "k_new", _n(b, n, g, d_k) * e),
        _ptr(v_new, "v_new", _n(b, n, g, d_v) * e), kp, vp, tp,
        _ptr(seq_lens, "seq_lens", _n(b) * 4, index=True), int(b), int(n), int(h), int(g),
        int(d_k), int(d_v), float(scale), _ptr(out, "out", _n(b, n, h, d_v) * e), bs, mb, nb,
        dt, int(flags), _stream(stream))


_DTYPES = {"f32": GQA_F32, "bf16": GQA_BF16, "f16": GQA_F16}


def gqa_decode_plan(b, n, h, g, d_k, d_v, cap, dtype, num_sms=0, flags=0) -> dict:
    """How a decode call with these shapes runs (host only when num_sms > 0):
    kernels per call, decode CTAs, positions per tile, tensor-core kernel or
    not, split workspace bytes, CTAs per cluster (0: no clusters).  dtype:
    GQA_* code or "f32"/"bf16"/"f16"; flags: as for gqa_decode_step."""
    dt = _DTYPES[dtype] if isinstance(dtype, str) else int(dtype)
    k, c, t, tc, cl = (ctypes.c_int(0) for _ in range(5))
    ws = ctypes.c_longlong(0)
    _check("gqa_decode_plan", lib.gqa_decode_plan(
        int(b), int(n), int(h), int(g), int(d_k), int(d_v), int(cap), dt, int(flags),
        int(num_sms),
        ctypes.byref(k), ctypes.byref(c), ctypes.byref(t), ctypes.byref(tc), ctypes.byref(ws),
        ctypes.byref(cl)))
    return {"kernels": k.value, "ctas": c.value, "tile": t.value, "tensor_core": bool(tc.value),
            "workspace_bytes": ws.value, "cluster": cl.value}


# ---------------------------------------------------------------------------
# packed tokens, 8-bit cache
# ---------------------------------------------------------------------------
def _tensor(x, name, n, types, dev) -> int:
    """Device address of a tensor argument of at least n elements of one of
    `types` on device `dev` (the current one, whose stream the call runs on);
    like _ptr otherwise (raw integers pass through unchecked).  The common
    case takes few calls into torch: at single tokens they are most of a
    call's time."""
    if isinstance(x, torch.Tensor):
        if (x.dtype in types and x.get_device() == dev and x.is_contiguous()
                and x.numel() >= n):
            return x.data_ptr()
        if x.dtype not in types:
            raise ValueError(f"{name}: must be {_names(types)}, got {x.dtype}")
        if x.is_cuda and x.get_device() != dev:
            raise ValueError(f"{name}: on {x.device}, the current device is cuda:{dev}")
        return _ptr(x, name, n * x.element_size())
    return int(x) if x is not None else 0


def _tokens(x, name, total, heads, d, types, dev):
    """Pointer and token stride (elements) of a packed tensor [total, heads, d]
    whose heads are contiguous; consecutive tokens may lie further apart."""
    if not isinstance(x, torch.Tensor):
        return _ptr(x, name), heads * d
    if x.shape != (total, heads, d):
        raise ValueError(f"{name}: must be [{total}, {heads}, {d}], got {list(x.shape)}")
    s0, s1, s2 = x.stride()
    if total > 0 and (s2 != 1 and d > 1 or s1 != d and heads > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    if x.dtype not in types:
        raise ValueError(f"{name}: must be {_names(types)}, got {x.dtype}")
    at = x.get_device()
    if at != dev:
        if x.is_cuda:
            raise ValueError(f"{name}: on {x.device}, the current device is cuda:{dev}")
        return _HostTensor(name, x.device), heads * d
    return x.data_ptr(), s0 if total > 1 else heads * d


def _names(types) -> str:
    return " or ".join(map(str, types or (torch.float32, torch.bfloat16, torch.float16)))


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _here(x, stream):
    """(current device, stream handle) of a call whose first tensor is x; no
    device (-2, which no tensor is on) when that is a host tensor."""
    if isinstance(x, torch.Tensor) and not x.is_cuda:
        return -2, 0
    dev = torch.cuda.current_device()
    if stream is None and _raw_stream is not None:
        return dev, _raw_stream(dev)
    return dev, _stream(stream)


def _launch(fn_name, fn, *args) -> None:
    """_call without a look at every argument: a host tensor's stand-in is no
    pointer, so its conversion fails before the library is entered."""
    try:
        code = fn(*args)
    except ctypes.ArgumentError:
        for a in args:
            if isinstance(a, _HostTensor):
                raise ValueError(
                    f"{a.name}: a CUDA tensor is required, got one on {a.device}") from None
        raise
    if code != GQA_OK:
        raise GqaError(fn_name, code)


_TORCH = {GQA_F32: (torch.float32,), GQA_BF16: (torch.bfloat16,), GQA_F16: (torch.float16,)}
_I32 = (torch.int32,)
_I64 = (torch.int64,)
_F32 = (torch.float32,)
_U8 = (torch.uint8,)
_E4M3 = (torch.float8_e4m3fn, torch.uint8)


def gqa_rope_table(rot, theta=10000.0, scaling="none", factor=1.0, original_len=0.0, low=1.0,
                   high=32.0, device=None):
    """Position table of gqa_rope_append: (phase, rope_scale), phase an int64
    tensor [rot / 2] on `device` (the current CUDA device by default; made
    once, kept by the caller).  scaling: "none", "linear", "wavelength" or
    "yarn" (or a GQA_ROPE_* code), see include/gqa.h."""
    codes = {"none": GQA_ROPE_PLAIN, "linear": GQA_ROPE_LINEAR,
             "wavelength": GQA_ROPE_WAVELENGTH, "yarn": GQA_ROPE_YARN}
    if isinstance(scaling, str) and scaling not in codes:
        raise ValueError(f"scaling: one of {sorted(codes)}, got {scaling!r}")
    host = (ctypes.c_uint64 * max(1, int(rot) // 2))()
    scale = ctypes.c_float(0.0)
    _check("gqa_rope_table", lib.gqa_rope_table(
        int(rot), float(theta), codes[scaling] if isinstance(scaling, str) else int(scaling),
        float(factor), float(original_len), float(low), float(high), host, ctypes.byref(scale)))
    phase = torch.tensor([v - (1 << 64) if v >> 63 else v for v in host], dtype=torch.int64)
    return phase.to("cuda" if device is None else device), float(scale.value)


def _rope_args(q, k_new, v_new, cu_tokens, seq_lens, q_out, b, h, g, d_k, d_v, rope, rope_scale,
               layout, q_weight, k_weight, eps, total, dtype, dev):
    """(dtype code, total, the arguments from q to rope_scale, q_out)."""
    dt = _dtype(k_new, dtype)
    ty = _TORCH.get(dt, ())
    if total is None:
        total = k_new.shape[0]
    qp, qs = (0, 0) if q is None else _tokens(q, "q", total, h, d_k, ty, dev)
    kp, ks = _tokens(k_new, "k_new", total, g, d_k, ty, dev)
    vp, vs = _tokens(v_new, "v_new", total, g, d_v, ty, dev)
    rot = 0
    if isinstance(rope, torch.Tensor):
        rot = 2 * rope.numel()
    elif rope is not None:
        raise ValueError("rope: must be the tensor of gqa_rope_table")
    return dt, total, (
        qp, kp, vp, qs, ks, vs, _tensor(cu_tokens, "cu_tokens", b + 1, _I32, dev),
        _tensor(seq_lens, "seq_lens", b, _I32, dev),
        _tensor(q_weight, "q_weight", d_k, ty, dev), _tensor(k_weight, "k_weight", d_k, ty, dev),
        float(eps), _tensor(rope, "rope", 0, _I64, dev), rot, int(layout),
        float(rope_scale), _tensor(q_out, "q_out", total * h * d_k, ty, dev))


def gqa_rope_append(q, k_new, v_new, cu_tokens, seq_lens, q_out, k_cache, v_cache, b, h, g, d_k,
                    d_v, rope=None, rope_scale=1.0, layout=GQA_ROPE_HALF, q_weight=None,
                    k_weight=None, eps=1e-6, total=None, cap=None, dtype=None,
                    stream=None) -> None:
    """Per-head norm (with q_weight and k_weight), rotary positions (rope and
    rope_scale of gqa_rope_table) and append of packed tokens, in one launch.
    q, k_new, v_new [total, heads, d] may be slices of one projection's
    output (heads contiguous, tokens further apart); q_out may be q."""
    dev, st = _here(k_new, stream)
    dt, total, args = _rope_args(q, k_new, v_new, cu_tokens, seq_lens, q_out, b, h, g, d_k, d_v,
                                 rope, rope_scale, layout, q_weight, k_weight, eps, total, dtype,
                                 dev)
    if cap is None:
        cap = k_cache.shape[2]
    ty = _TORCH.get(dt, ())
    _launch("gqa_rope_append", lib.gqa_rope_append, *args,
            _tensor(k_cache, "k_cache", b * g * cap * d_k, ty, dev),
            _tensor(v_cache, "v_cache", b * g * cap * d_v, ty, dev),
            int(b), int(total), int(h), int(g), int(d_k), int(d_v), int(cap), dt, st)


def _pools(k_pool, v_pool, block_table, b, g, d_k, d_v, ty, dev):
    """_paged_ptrs with the checks of _tensor."""
    nb, _, bs, _ = k_pool.shape
    mb = block_table.shape[1]
    return (_tensor(k_pool, "k_pool", nb * g * bs * d_k, ty, dev),
            _tensor(v_pool, "v_pool", nb * g * bs * d_v, ty, dev),
            _tensor(block_table, "block_table", b * mb, _I32, dev), int(bs), int(mb), int(nb))


def gqa_rope_append_paged(q, k_new, v_new, cu_tokens, seq_lens, q_out, k_pool, v_pool,
                          block_table, b, h, g, d_k, d_v, rope=None, rope_scale=1.0,
                          layout=GQA_ROPE_HALF, q_weight=None, k_weight=None, eps=1e-6,
                          total=None, dtype=None, stream=None) -> None:
    """gqa_rope_append into a paged cache (pools [num_blocks, g, block_size,
    d], block_table [b, max_blocks])."""
    dev, st = _here(k_new, stream)
    dt, total, args = _rope_args(q, k_new, v_new, cu_tokens, seq_lens, q_out, b, h, g, d_k, d_v,
                                 rope, rope_scale, layout, q_weight, k_weight, eps, total, dtype,
                                 dev)
    kp, vp, tp, bs, mb, nb = _pools(k_pool, v_pool, block_table, b, g, d_k, d_v,
                                    _TORCH.get(dt, ()), dev)
    _launch("gqa_rope_append_paged", lib.gqa_rope_append_paged, *args, kp, vp, tp, int(b),
            int(total), int(h), int(g), int(d_k), int(d_v), bs, mb, nb, dt, st)


def _pools8(k_pool, v_pool, k_scale, v_scale, block_table, b, g, d_k, d_v, dev):
    """_pools of an 8-bit cache, with the pointers of its scales [num_blocks,
    g, block_size]."""
    kp, vp, tp, bs, mb, nb = _pools(k_pool, v_pool, block_table, b, g, d_k, d_v, _E4M3, dev)
    n = nb * g * bs
    return (kp, vp, _tensor(k_scale, "k_scale", n, _F32, dev),
            _tensor(v_scale, "v_scale", n, _F32, dev),
            tp, bs, mb, nb)


def gqa_rope_append_fp8_paged(q, k_new, v_new, cu_tokens, seq_lens, q_out, k_pool, v_pool,
                              k_scale, v_scale, block_table, b, h, g, d_k, d_v, rope=None,
                              rope_scale=1.0, layout=GQA_ROPE_HALF, q_weight=None, k_weight=None,
                              eps=1e-6, total=None, dtype=None, stream=None) -> None:
    """gqa_rope_append into an 8-bit paged cache: e4m3 pools (torch.float8_e4m3fn
    or uint8) and one fp32 scale per row.  q = q_out = None with rope = None
    is the plain quantising append."""
    dev, st = _here(k_new, stream)
    dt, total, args = _rope_args(q, k_new, v_new, cu_tokens, seq_lens, q_out, b, h, g, d_k, d_v,
                                 rope, rope_scale, layout, q_weight, k_weight, eps, total, dtype,
                                 dev)
    kp, vp, ks, vs, tp, bs, mb, nb = _pools8(k_pool, v_pool, k_scale, v_scale, block_table, b, g,
                                             d_k, d_v, dev)
    _launch("gqa_rope_append_fp8_paged", lib.gqa_rope_append_fp8_paged, *args, kp, vp, ks, vs, tp,
            int(b), int(total), int(h), int(g), int(d_k), int(d_v), bs, mb, nb, dt, st)


def gqa_kv_read_fp8_paged(k_pool, v_pool, k_scale, v_scale, block_table, seq_lens, k_cache,
                          v_cache, b, g, d_k, d_v, cap=None, dtype=None, stream=None) -> None:
    """Rows [0, seq_lens[i]) of an 8-bit paged cache as contiguous caches
    [b, g, cap, d] of the caches' type."""
    dev, st = _here(k_cache, stream)
    dt = _dtype(k_cache, dtype)
    ty = _TORCH.get(dt, ())
    if cap is None:
        cap = k_cache.shape[2]
    kp, vp, ks, vs, tp, bs, mb, nb = _pools8(k_pool, v_pool, k_scale, v_scale, block_table, b, g,
                                             d_k, d_v, dev)
    _launch("gqa_kv_read_fp8_paged", lib.gqa_kv_read_fp8_paged, kp, vp, ks, vs, tp,
            _tensor(seq_lens, "seq_lens", b, _I32, dev),
            _tensor(k_cache, "k_cache", b * g * cap * d_k, ty, dev),
            _tensor(v_cache, "v_cache", b * g * cap * d_v, ty, dev), int(b), int(g), int(d_k),
            int(d_v), bs, mb, nb, int(cap), dt, st)


def gqa_chunk_attn_workspace(total, h, g, d_k, d_v, num_sms=0) -> int:
    """Bytes of workspace of gqa_chunk_attn(_paged) for up to `total` packed
    rows (host only when num_sms > 0)."""
    n = ctypes.c_longlong(0)
    _check("gqa_chunk_attn_workspace", lib.gqa_chunk_attn_workspace(
        int(total), int(h), int(g), int(d_k), int(d_v), int(num_sms), ctypes.byref(n)))
    return int(n.value)


def _workspace(ws, stream, dev, like, size, *shape):
    """The workspace argument (tensor, bytes): the caller's, or a tensor made
    for this call on its stream (the allocator orders its next use behind
    the call)."""
    if ws is None and isinstance(like, torch.Tensor) and like.is_cuda:
        n = size(*shape)
        if stream is None:
            ws = torch.empty(n, dtype=torch.uint8, device=like.device)
        else:
            s = stream if isinstance(stream, torch.cuda.Stream) else (
                torch.cuda.ExternalStream(int(stream), device=like.device))
            with torch.cuda.stream(s):
                ws = torch.empty(n, dtype=torch.uint8, device=like.device)
    if isinstance(ws, torch.Tensor):
        return _tensor(ws, "workspace", 0, _U8, dev), ws.numel() * ws.element_size(), ws
    if ws is None:
        return 0, 0, None
    raise ValueError("workspace: must be a tensor")


def gqa_chunk_attn(q, k_cache, v_cache, cu_tokens, seq_lens, b, h, g, d_k, d_v, scale, out,
                   total=None, cap=None, dtype=None, workspace=None, stream=None) -> None:
    """Causal attention of packed chunks of new tokens (q [total, h, d_k], out
    [total, h, d_v]) over caches that already hold their rows.  workspace:
    a uint8 tensor of gqa_chunk_attn_workspace bytes to reuse between calls
    (by default one is made per call)."""
    dev, st = _here(q, stream)
    dt = _dtype(q, dtype)
    ty = _TORCH.get(dt, ())
    if total is None:
        total = q.shape[0]
    if cap is None:
        cap = k_cache.shape[2]
    wp, wn, _keep = _workspace(workspace, stream, dev, q, gqa_chunk_attn_workspace, total, h, g,
                               d_k, d_v)
    _launch("gqa_chunk_attn", lib.gqa_chunk_attn, _tensor(q, "q", total * h * d_k, ty, dev),
            _tensor(k_cache, "k_cache", b * g * cap * d_k, ty, dev),
            _tensor(v_cache, "v_cache", b * g * cap * d_v, ty, dev),
            _tensor(cu_tokens, "cu_tokens", b + 1, _I32, dev),
            _tensor(seq_lens, "seq_lens", b, _I32, dev), int(b), int(total), int(h), int(g),
            int(d_k), int(d_v), float(scale), _tensor(out, "out", total * h * d_v, ty, dev),
            int(cap), dt, wp, wn, st)


def gqa_chunk_attn_paged(q, k_pool, v_pool, block_table, cu_tokens, seq_lens, b, h, g, d_k, d_v,
                         scale, out, total=None, dtype=None, workspace=None,
                         stream=None) -> None:
    """gqa_chunk_attn over a paged cache."""
    dev, st = _here(q, stream)
    dt = _dtype(q, dtype)
    ty = _TORCH.get(dt, ())
    if total is None:
        total = q.shape[0]
    kp, vp, tp, bs, mb, nb = _pools(k_pool, v_pool, block_table, b, g, d_k, d_v, ty, dev)
    wp, wn, _keep = _workspace(workspace, stream, dev, q, gqa_chunk_attn_workspace, total, h, g,
                               d_k, d_v)
    _launch("gqa_chunk_attn_paged", lib.gqa_chunk_attn_paged,
            _tensor(q, "q", total * h * d_k, ty, dev), kp, vp, tp,
            _tensor(cu_tokens, "cu_tokens", b + 1, _I32, dev),
            _tensor(seq_lens, "seq_lens", b, _I32, dev), int(b), int(total), int(h), int(g),
            int(d_k), int(d_v), float(scale), _tensor(out, "out", total * h * d_v, ty, dev), bs,
            mb, nb, dt, wp, wn, st)


def gqa_decode_attn_fp8_workspace(b, n, h, g, d_k, d_v, cap, num_sms=0) -> int:
    """Bytes of workspace of gqa_decode_attn_fp8_paged, cap = max_blocks *
    block_size (host only when num_sms > 0)."""
    out = ctypes.c_longlong(0)
    _check("gqa_decode_attn_fp8_workspace", lib.gqa_decode_attn_fp8_workspace(
        int(b), int(n), int(h), int(g), int(d_k), int(d_v), int(cap), int(num_sms),
        ctypes.byref(out)))
    return int(out.value)


def gqa_decode_attn_fp8_paged(q, k_pool, v_pool, k_scale, v_scale, block_table, seq_lens, b, h,
                              g, d_k, d_v, scale, out, n=1, dtype=None, workspace=None,
                              stream=None) -> None:
    """gqa_decode_attn_paged over an 8-bit paged cache (e4m3 pools, one fp32
    scale per row).  workspace: a uint8 tensor of
    gqa_decode_attn_fp8_workspace bytes to reuse between calls (by default
    one is made per call)."""
    dev, st = _here(q, stream)
    dt = _dtype(q, dtype)
    ty = _TORCH.get(dt, ())
    kp, vp, ks, vs, tp, bs, mb, nb = _pools8(k_pool, v_pool, k_scale, v_scale, block_table, b, g,
                                             d_k, d_v, dev)
    wp, wn, _keep = _workspace(workspace, stream, dev, q, gqa_decode_attn_fp8_workspace, b, n, h,
                               g, d_k, d_v, bs * mb)
    _launch("gqa_decode_attn_fp8_paged", lib.gqa_decode_attn_fp8_paged,
            _tensor(q, "q", b * n * h * d_k, ty, dev), kp, vp, ks, vs, tp,
            _tensor(seq_lens, "seq_lens", b, _I32, dev), int(b), int(n), int(h), int(g),
            int(d_k), int(d_v), float(scale), _tensor(out, "out", b * n * h * d_v, ty, dev), bs,
            mb, nb, dt, wp, wn, st)


def gqa_device_status(stream=None) -> int:
    """Read and clear the device status word (synchronizes the stream)."""
    bits = ctypes.c_uint32(0)
    _check("gqa_device_status", lib.gqa_device_status(_stream(stream), ctypes.byref(bits)))
    return int(bits.value)


def gqa_selftest_wait_timeout(budget_cycles: int, stream=None) -> None:
    _check("gqa_selftest_wait_timeout",
           lib.gqa_selftest_wait_timeout(int(budget_cycles), _stream(stream)))


def gqa_version() -> int:
    return int(lib.gqa_version())


def decode_step(q, k_cache, v_cache, k_new, v_new, seq_lens, g, scale, out,
                stream=None, fused=False, flags=0) -> None:
    """One layer's decode step in the order of the decode notes: push the new
    K/V rows, then attend.  fused=False makes the two C-ABI calls
    (gqa_kv_append, gqa_decode_attn); fused=True makes one gqa_decode_step."""
    b, h, d = q.shape
    if fused:
        gqa_decode_step(q, k_new, v_new, k_cache, v_cache, seq_lens, b, h, g, d,
                        v_cache.shape[-1], scale, out, flags=flags, stream=stream)
        return
    gqa_kv_append(k_new, v_new, k_cache, v_cache, seq_lens, b, g, d, v_new.shape[-1],
                  stream=stream)
    gqa_decode_attn(q, k_cache, v_cache, seq_lens, b, h, g, d, v_cache.shape[-1],
                    scale, out, stream=stream)
