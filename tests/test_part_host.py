"""The calls over a window and over a shared prefix without a GPU: argument
checks of the C ABI (before any CUDA call) and of the binding, workspace
sizes."""
import ctypes

import pytest
import torch

# calls that pass every check with addresses that are not memory: with a GPU
# they would be launched
pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="addresses that no kernel may follow: without a GPU only")

A = 0x10000  # a 256-byte aligned address that is never dereferenced
BIG = 1 << 40
MAX = 0x7FFFFFFF
NULL, SHAPE, DTYPE, ALIGN, UNSUPPORTED, CUDA, SCRATCH = -1, -2, -3, -4, -5, -6, -8


def _b():
    from gqa_kv_cache_append_gb300 import build
    build.build()
    from gqa_kv_cache_append_gb300 import binding
    return binding


def chunk(op, paged, **kw):
    a = dict(q=A, k=A, v=A, table=A, cu=A, lens=A, b=2, total=40, h=8, g=2, dk=128, dv=128,
             scale=0.1, window=32, sinks=4, prefix=48, out=A, cap=64, bs=16, mb=4, nb=9, dtype=1,
             ws=A, wsb=BIG)
    assert not set(kw) - set(a)
    a.update(kw)
    lib = _b().lib
    part = [a["window"], a["sinks"]] if op == "window" else [a["prefix"]]
    head = [a[k] for k in ("q", "k", "v", "table", "cu", "lens") if paged or k != "table"]
    mid = [a[k] for k in ("b", "total", "h", "g", "dk", "dv", "scale")] + part + [a["out"]]
    size = [a["bs"], a["mb"], a["nb"]] if paged else [a["cap"]]
    fn = getattr(lib, f"gqa_chunk_attn_{op}" + ("_paged" if paged else ""))
    return fn(*head, *mid, *size, a["dtype"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("op", ["window", "prefix"])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(q=0), NULL), (dict(k=0), NULL), (dict(v=0), NULL), (dict(out=0), NULL),
    (dict(cu=0), NULL), (dict(lens=0), NULL), (dict(ws=0), NULL),
    (dict(dtype=5), DTYPE), (dict(dtype=0), UNSUPPORTED),
    (dict(b=0), SHAPE), (dict(total=-1), SHAPE), (dict(h=9), SHAPE), (dict(g=0), SHAPE),
    (dict(h=0), SHAPE), (dict(h=-8), SHAPE), (dict(dk=0), SHAPE), (dict(total=1 << 29), SHAPE),
    (dict(dk=96), UNSUPPORTED), (dict(dv=256), UNSUPPORTED), (dict(h=258, g=2), UNSUPPORTED),
    (dict(b=70000), UNSUPPORTED),
    (dict(q=A + 8), ALIGN), (dict(out=A + 8), ALIGN), (dict(k=A + 4), ALIGN),
    (dict(cu=A + 2), ALIGN), (dict(ws=A + 128), ALIGN),
    (dict(), CUDA), (dict(h=256, g=2), CUDA), (dict(total=0, q=0, out=0), CUDA),
])
def test_chunk_checks(op, paged, kw, code):
    assert chunk(op, paged, **kw) == code


@pytest.mark.parametrize("paged", [False, True])
def test_window_and_prefix_checks(paged):
    for kw, code in ((dict(window=0), SHAPE), (dict(window=-5), SHAPE), (dict(sinks=-1), SHAPE),
                     (dict(window=1, sinks=0), CUDA), (dict(window=MAX, sinks=MAX), CUDA)):
        assert chunk("window", paged, **kw) == code
    for kw, code in ((dict(prefix=-1), SHAPE), (dict(prefix=65), SHAPE), (dict(prefix=64), CUDA),
                     (dict(prefix=0), CUDA)):
        assert chunk("prefix", paged, **kw) == code


@pytest.mark.parametrize("op", ["window", "prefix"])
def test_form_specific_checks(op):
    assert chunk(op, False, cap=0) == SHAPE
    assert chunk(op, False, b=40000, g=8, cap=8000) == SHAPE
    assert chunk(op, True, bs=48) == UNSUPPORTED and chunk(op, True, table=0) == NULL
    assert chunk(op, True, bs=16, mb=(1 << 27) - 1, nb=9) == SHAPE  # positions past 2^31 - 256
    assert chunk(op, True, bs=1 << 10, mb=1 << 20, nb=9) == CUDA


def fp8(**kw):
    a = dict(q=A, k=A, v=A, ks=A, vs=A, table=A, lens=A, b=2, n=1, h=8, g=2, dk=128, dv=128,
             scale=0.1, window=20, sinks=4, out=A, bs=16, mb=4, nb=9, dtype=1, ws=A, wsb=BIG)
    assert not set(kw) - set(a)
    a.update(kw)
    return _b().lib.gqa_decode_attn_fp8_window_paged(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), NULL), (dict(k=0), NULL), (dict(ks=0), NULL), (dict(vs=0), NULL),
    (dict(table=0), NULL), (dict(lens=0), NULL), (dict(out=0), NULL), (dict(ws=0), NULL),
    (dict(dtype=9), DTYPE), (dict(dtype=0), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED),
    (dict(b=0), SHAPE), (dict(n=0), SHAPE), (dict(n=65), SHAPE), (dict(h=9), SHAPE),
    (dict(n=9), UNSUPPORTED), (dict(h=66), UNSUPPORTED), (dict(dk=192), UNSUPPORTED),
    (dict(b=70000), UNSUPPORTED), (dict(bs=20), UNSUPPORTED),
    (dict(ks=A + 4), ALIGN), (dict(vs=A + 8), ALIGN), (dict(q=A + 8), ALIGN),
    (dict(ws=A + 64), ALIGN),
    (dict(window=0), SHAPE), (dict(window=-1), SHAPE), (dict(sinks=-1), SHAPE),
    (dict(window=MAX, sinks=MAX), CUDA), (dict(), CUDA), (dict(n=8), CUDA),
])
def test_decode_fp8_window_checks(kw, code):
    assert fp8(**kw) == code


def test_prefix_workspace():
    B = _b()
    size = lambda b, t, h=64, g=8: B.gqa_chunk_attn_prefix_workspace(b, t, h, g, 128, 128,
                                                                     num_sms=152)
    plain = lambda t: B.gqa_chunk_attn_workspace(t, 64, 8, 128, 128, num_sms=152)
    # few tokens a sequence: both results of every row, fp32, on top
    rows = 2 * 64 * 64
    assert rows * 130 * 4 <= size(64, 64) - plain(64) <= rows * 130 * 4 + 64 * 8 * 16 + 4096
    # one sequence shares nothing
    assert size(1, 1000) == plain(1000)
    # what serves a total serves every smaller one
    for b in (2, 5, 64):
        last = 0
        for t in (0, 1, b, 2 * b, 15 * b, 16 * b - 1, 16 * b, 16 * b + 1, 100 * b):
            assert size(b, t) >= last
            last = size(b, t)
    for bad in (0, -1):
        with pytest.raises(B.GqaError) as e:
            size(bad, 10)
        assert e.value.code == SHAPE
    with pytest.raises(B.GqaError) as e:
        size(2, 10, h=258, g=2)
    assert e.value.code == UNSUPPORTED
    f, x = B.lib.gqa_chunk_attn_prefix_workspace, ctypes.c_longlong()
    assert f(2, 16, 64, 8, 128, 128, 152, None) == NULL
    assert f(2, 16, 64, 8, 128, 128, -1, ctypes.byref(x)) == SHAPE
    assert f(70000, 16, 64, 8, 128, 128, 152, ctypes.byref(x)) == UNSUPPORTED


def test_binding_refusals_without_a_gpu():
    B = _b()
    T, h, g, d = 4, 8, 2, 128
    bf = torch.bfloat16
    q, out = (torch.zeros(T, h, d, dtype=bf) for _ in range(2))
    k, v = (torch.zeros(2, g, 16, d, dtype=bf) for _ in range(2))
    cu, lens = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    table = torch.zeros(2, 4, dtype=torch.int32)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    dims = (2, h, g, d, d, 0.1)
    for fn, part in ((B.gqa_chunk_attn_window, 8), (B.gqa_chunk_attn_prefix, 8)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            fn(q, k, v, cu, lens, *dims, part, out, workspace=ws)
        with pytest.raises(ValueError, match="out: must be"):
            fn(q, k, v, cu, lens, *dims, part, out.float(), workspace=ws)
        with pytest.raises(ValueError, match="k_cache: holds"):
            fn(q, k[:1], v, cu, lens, *dims, part, out, workspace=ws)
        with pytest.raises(ValueError, match="seq_lens: must be torch.int32"):
            fn(q, k, v, cu, lens.long(), *dims, part, out, workspace=ws)
        with pytest.raises(ValueError, match="workspace: must be torch.uint8"):
            fn(q, k, v, cu, lens, *dims, part, out, workspace=ws.float())
    for fn in (B.gqa_chunk_attn_window_paged, B.gqa_chunk_attn_prefix_paged):
        with pytest.raises(ValueError, match="CUDA tensor"):
            fn(q, k, v, table, cu, lens, *dims, 8, out, workspace=ws)
        with pytest.raises(ValueError, match="block_table: holds"):
            fn(q, k, v, table[:1], cu, lens, *dims, 8, out, workspace=ws)
        with pytest.raises(ValueError, match="v_pool: must be contiguous"):
            fn(q, k, v.transpose(1, 2).contiguous().transpose(1, 2), table, cu, lens, *dims, 8,
               out, workspace=ws)
    k8, sc = torch.zeros(9, g, 16, d, dtype=torch.uint8), torch.zeros(9, g, 16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        B.gqa_decode_attn_fp8_window_paged(q[:2], k8, k8, sc, sc, table, lens, *dims, 8, out[:2],
                                           workspace=ws)
    with pytest.raises(ValueError, match="v_scale: holds"):
        B.gqa_decode_attn_fp8_window_paged(q[:2], k8, k8, sc, sc[:5], table, lens, *dims, 8,
                                           out[:2], workspace=ws)
