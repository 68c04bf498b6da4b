"""The calls on packed tokens and on the 8-bit cache without a GPU: argument
checks of the C ABI (before any CUDA call) and of the binding, the position
table against its formulas, workspace sizes."""
import ctypes
import math

import pytest
import torch

A = 0x10000  # a 256-byte aligned address that is never dereferenced
BIG = 1 << 40


def _b():
    from gqa_kv_cache_append_gb300 import build
    build.build()
    from gqa_kv_cache_append_gb300 import binding
    return binding


NULL, SHAPE, DTYPE, ALIGN, UNSUPPORTED, CUDA, SCRATCH = -1, -2, -3, -4, -5, -6, -8

ROPE = dict(q=A, k=A, v=A, qs=1024, ks=256, vs=256, cu=A, lens=A, qw=A, kw=A, eps=1e-6, phase=A,
            rot=128, layout=0, scale=1.0, qo=A, kc=A, vc=A)
DIMS = dict(b=2, total=4, h=8, g=2, dk=128, dv=128)
PAGED = dict(bs=16, mb=4, nb=9, dtype=1)


def rope(form, **kw):
    """One call of gqa_rope_append / _paged / _fp8_paged with changed arguments."""
    a = dict(ROPE, **DIMS, **PAGED, cap=64, ksc=A, vsc=A, table=A)
    assert not set(kw) - set(a)
    a.update(kw)
    head = [a[k] for k in ROPE]
    dims = [a[k] for k in DIMS]
    lib = _b().lib
    if form == "flat":
        return lib.gqa_rope_append(*head, *dims, a["cap"], a["dtype"], None)
    tail = [a["bs"], a["mb"], a["nb"], a["dtype"], None]
    if form == "paged":
        return lib.gqa_rope_append_paged(*head, a["table"], *dims, *tail)
    return lib.gqa_rope_append_fp8_paged(*head, a["ksc"], a["vsc"], a["table"], *dims, *tail)


@pytest.mark.parametrize("form", ["flat", "paged", "fp8"])
@pytest.mark.parametrize("kw,code", [
    (dict(k=0), NULL), (dict(v=0), NULL), (dict(cu=0), NULL), (dict(lens=0), NULL),
    (dict(kc=0), NULL), (dict(vc=0), NULL), (dict(q=0), NULL), (dict(qo=0), NULL),
    (dict(qw=0), NULL), (dict(kw=0), NULL),
    (dict(dtype=3), DTYPE), (dict(dtype=-1), DTYPE),
    (dict(b=0), SHAPE), (dict(total=-1), SHAPE), (dict(g=0), SHAPE), (dict(h=7), SHAPE),
    (dict(dk=0), SHAPE), (dict(dv=-8), SHAPE),
    (dict(qs=1016), SHAPE), (dict(ks=128), SHAPE), (dict(vs=0), SHAPE),
    (dict(rot=0), SHAPE), (dict(rot=144), SHAPE), (dict(total=1 << 30), SHAPE),
    (dict(rot=120), UNSUPPORTED), (dict(layout=2), UNSUPPORTED), (dict(layout=-1), UNSUPPORTED),
    (dict(dk=132), UNSUPPORTED), (dict(dv=264, vs=528), UNSUPPORTED),
    (dict(q=A + 8), ALIGN), (dict(k=A + 2), ALIGN), (dict(qo=A + 4), ALIGN),
    (dict(kc=A + 8), ALIGN), (dict(cu=A + 2), ALIGN), (dict(lens=A + 1), ALIGN),
    (dict(qw=A + 8), ALIGN), (dict(phase=A + 4), ALIGN), (dict(qs=1028), ALIGN),
])
def test_rope_append_checks(form, kw, code):
    assert rope(form, **kw) == code


@pytest.mark.parametrize("form", ["paged", "fp8"])
@pytest.mark.parametrize("kw,code", [
    (dict(table=0), NULL), (dict(table=A + 2), ALIGN), (dict(bs=24), UNSUPPORTED),
    (dict(bs=8), UNSUPPORTED), (dict(mb=0), SHAPE), (dict(nb=0), SHAPE),
    (dict(mb=1 << 28), SHAPE),
])
def test_rope_append_paged_checks(form, kw, code):
    assert rope(form, **kw) == code


def test_rope_append_form_specific_checks():
    assert rope("flat", cap=0) == SHAPE
    assert rope("flat", b=40000, g=8, h=8, cap=8000, ks=1024, vs=1024) == SHAPE
    assert rope("fp8", ksc=0) == NULL and rope("fp8", vsc=0) == NULL
    assert rope("fp8", ksc=A + 2) == ALIGN
    assert rope("fp8", dv=136, vs=272) == UNSUPPORTED  # rows of whole 16 bytes
    # without a table, rot and layout are not looked at
    assert rope("flat", phase=0, rot=-3, layout=9) == CUDA
    # no queries; no norm
    assert rope("flat", q=0, qo=0) == CUDA
    assert rope("flat", qw=0, kw=0) == CUDA
    for form in ("flat", "paged", "fp8"):
        assert rope(form) == CUDA  # (no device here)


def chunk(paged=False, **kw):
    a = dict(q=A, k=A, v=A, table=A, cu=A, lens=A, b=2, total=40, h=8, g=2, dk=128, dv=128,
             scale=0.1, out=A, cap=64, bs=16, mb=4, nb=9, dtype=1, ws=A, wsb=BIG)
    assert not set(kw) - set(a)
    a.update(kw)
    lib = _b().lib
    dims = [a[k] for k in ("b", "total", "h", "g", "dk", "dv")]
    if paged:
        return lib.gqa_chunk_attn_paged(a["q"], a["k"], a["v"], a["table"], a["cu"], a["lens"],
                                        *dims, a["scale"], a["out"], a["bs"], a["mb"], a["nb"],
                                        a["dtype"], a["ws"], a["wsb"], None)
    return lib.gqa_chunk_attn(a["q"], a["k"], a["v"], a["cu"], a["lens"], *dims, a["scale"],
                              a["out"], a["cap"], a["dtype"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(q=0), NULL), (dict(k=0), NULL), (dict(v=0), NULL), (dict(out=0), NULL),
    (dict(cu=0), NULL), (dict(lens=0), NULL), (dict(ws=0), NULL),
    (dict(dtype=5), DTYPE), (dict(dtype=0), UNSUPPORTED),
    (dict(b=0), SHAPE), (dict(total=-1), SHAPE), (dict(h=9), SHAPE), (dict(g=0), SHAPE),
    (dict(dk=0), SHAPE), (dict(total=1 << 29), SHAPE),
    (dict(dk=96), UNSUPPORTED), (dict(dv=256), UNSUPPORTED), (dict(h=258, g=2), UNSUPPORTED),
    (dict(b=70000), UNSUPPORTED),
    (dict(q=A + 8), ALIGN), (dict(out=A + 8), ALIGN), (dict(k=A + 4), ALIGN),
    (dict(cu=A + 2), ALIGN), (dict(ws=A + 128), ALIGN),
    (dict(), CUDA), (dict(h=256, g=2), CUDA), (dict(total=0, q=0, out=0), CUDA),
])
def test_chunk_attn_checks(paged, kw, code):
    assert chunk(paged, **kw) == code


def test_chunk_attn_form_specific_checks():
    assert chunk(cap=0) == SHAPE
    assert chunk(b=40000, g=8, cap=8000) == SHAPE
    assert chunk(True, bs=48) == UNSUPPORTED and chunk(True, table=0) == NULL


def fp8(**kw):
    a = dict(q=A, k=A, v=A, ks=A, vs=A, table=A, lens=A, b=2, n=1, h=8, g=2, dk=128, dv=128,
             scale=0.1, out=A, bs=16, mb=4, nb=9, dtype=1, ws=A, wsb=BIG)
    assert not set(kw) - set(a)
    a.update(kw)
    return _b().lib.gqa_decode_attn_fp8_paged(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), NULL), (dict(k=0), NULL), (dict(ks=0), NULL), (dict(vs=0), NULL),
    (dict(table=0), NULL), (dict(lens=0), NULL), (dict(out=0), NULL), (dict(ws=0), NULL),
    (dict(dtype=9), DTYPE), (dict(dtype=0), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED),
    (dict(b=0), SHAPE), (dict(n=0), SHAPE), (dict(n=65), SHAPE), (dict(h=9), SHAPE),
    (dict(n=9), UNSUPPORTED), (dict(h=66), UNSUPPORTED), (dict(dk=192), UNSUPPORTED),
    (dict(b=70000), UNSUPPORTED), (dict(bs=20), UNSUPPORTED),
    (dict(ks=A + 4), ALIGN), (dict(vs=A + 8), ALIGN), (dict(q=A + 8), ALIGN),
    (dict(ws=A + 64), ALIGN), (dict(), CUDA), (dict(n=8), CUDA),
])
def test_decode_attn_fp8_checks(kw, code):
    assert fp8(**kw) == code


def read(**kw):
    a = dict(k=A, v=A, ks=A, vs=A, table=A, lens=A, kc=A, vc=A, b=2, g=2, dk=128, dv=128, bs=16,
             mb=4, nb=9, cap=64, dtype=1)
    assert not set(kw) - set(a)
    a.update(kw)
    return _b().lib.gqa_kv_read_fp8_paged(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(k=0), NULL), (dict(ks=0), NULL), (dict(lens=0), NULL), (dict(vc=0), NULL),
    (dict(table=0), NULL), (dict(dtype=4), DTYPE), (dict(b=0), SHAPE), (dict(cap=0), SHAPE),
    (dict(g=0), SHAPE), (dict(dk=24), UNSUPPORTED), (dict(dv=272), UNSUPPORTED),
    (dict(bs=12), UNSUPPORTED), (dict(kc=A + 8), ALIGN), (dict(lens=A + 2), ALIGN), (dict(), CUDA),
])
def test_kv_read_fp8_checks(kw, code):
    assert read(**kw) == code


def test_workspace_sizes():
    B = _b()
    n = B.gqa_chunk_attn_workspace(4096, 64, 8, 128, 128, num_sms=152)
    # two pieces a CTA of 256 rows: output, maximum and sum in fp32
    rows = 2 * 152 * 256
    assert rows * 130 * 4 <= n <= rows * 130 * 4 + 152 * 64 + 4096
    # few tokens: one side's rows
    assert B.gqa_chunk_attn_workspace(16, 64, 8, 128, 128, num_sms=152) < 0.51 * n
    assert B.gqa_chunk_attn_workspace(17, 64, 8, 128, 128, num_sms=152) == n
    assert B.gqa_chunk_attn_workspace(0, 64, 8, 64, 64, num_sms=152) > 0
    with pytest.raises(B.GqaError) as e:
        B.gqa_chunk_attn_workspace(16, 64, 8, 96, 128, num_sms=152)
    assert e.value.code == UNSUPPORTED
    assert B.lib.gqa_chunk_attn_workspace(16, 64, 8, 128, 128, 152, None) == NULL
    x = ctypes.c_longlong()
    assert B.lib.gqa_chunk_attn_workspace(16, 64, 8, 128, 128, -1, ctypes.byref(x)) == SHAPE
    m = B.gqa_decode_attn_fp8_workspace(32, 1, 64, 8, 128, 128, 8192, num_sms=152)
    assert m >= (256 + 152) * 8 * 130 * 4
    assert B.lib.gqa_decode_attn_fp8_workspace(32, 1, 64, 8, 128, 128, 8192, 152, None) == NULL
    with pytest.raises(B.GqaError):
        B.gqa_decode_attn_fp8_workspace(32, 5, 64, 8, 128, 128, 8192, num_sms=152)


def table(B, rot, theta, scaling, **kw):
    phase, scale = B.gqa_rope_table(rot, theta, scaling, device="cpu", **kw)
    assert phase.dtype == torch.int64 and phase.shape == (rot // 2,)
    return [(int(v) % (1 << 64)) / 2.0 ** 64 * 2 * math.pi for v in phase], scale


@pytest.mark.parametrize("rot", [2, 16, 64, 128, 256])
@pytest.mark.parametrize("theta", [10000.0, 500000.0])
def test_rope_table_plain_and_linear(rot, theta):
    B = _b()
    f, s = table(B, rot, theta, "none")
    g, _ = table(B, rot, theta, "linear", factor=4.0)
    assert s == 1.0
    for m in range(rot // 2):
        want = theta ** (-2.0 * m / rot)
        assert abs(f[m] - want) <= 4e-16 * want + 2.0 ** -62
        assert abs(g[m] - want / 4) <= 4e-16 * want + 2.0 ** -62


def test_rope_table_wavelength():
    B = _b()
    f, s = table(B, 128, 500000.0, "wavelength", factor=8.0, original_len=8192.0, low=1.0,
                 high=4.0)
    assert s == 1.0
    kept = stretched = blended = 0
    for m in range(64):
        base = 500000.0 ** (-2.0 * m / 128)
        turns = 8192.0 * base / (2 * math.pi)
        if turns >= 4.0:
            want, kept = base, kept + 1
        elif turns <= 1.0:
            want, stretched = base / 8, stretched + 1
        else:
            x = (turns - 1.0) / 3.0
            want, blended = (1 - x) * base / 8 + x * base, blended + 1
        assert abs(f[m] - want) <= 1e-15 * want + 2.0 ** -62
    assert kept and stretched and blended


def test_rope_table_yarn():
    B = _b()
    f, s = table(B, 128, 10000.0, "yarn", factor=16.0, original_len=4096.0, low=1.0, high=32.0)
    assert abs(s - (0.1 * math.log(16.0) + 1.0)) < 1e-7
    assert table(B, 128, 10000.0, "yarn", factor=0.5, original_len=4096.0)[1] == 1.0
    base = [10000.0 ** (-2.0 * m / 128) for m in range(64)]
    r = [b / x for b, x in zip(base, f)]  # 1 (kept) up to 16 (stretched)
    assert abs(r[0] - 1) < 1e-12 and abs(r[-1] - 16) < 1e-9
    assert all(a <= b + 1e-9 for a, b in zip(r, r[1:]))
    at = lambda t: 128 * math.log(4096 / (2 * math.pi * t)) / (2 * math.log(10000.0))
    first, last = math.floor(at(32.0)), math.ceil(at(1.0))
    assert abs(r[first] - 1) < 1e-12 and r[first + 1] > 1 + 1e-6
    assert abs(r[last] - 16) < 1e-9 and r[last - 1] < 16 - 1e-6


def test_rope_table_refusals():
    B = _b()
    f = B.lib.gqa_rope_table
    ph = (ctypes.c_uint64 * 64)()
    sc = ctypes.c_float()
    ok = [128, 10000.0, 2, 8.0, 8192.0, 1.0, 4.0, ph, ctypes.byref(sc)]
    assert f(*ok) == 0
    for pos, val, code in ((0, 0, SHAPE), (0, 3, SHAPE), (1, 0.5, SHAPE),
                           (1, float("inf"), SHAPE), (1, float("nan"), SHAPE), (2, 4, UNSUPPORTED),
                           (2, -1, UNSUPPORTED), (3, 0.0, SHAPE), (3, float("nan"), SHAPE),
                           (4, 0.0, SHAPE), (5, 0.0, SHAPE), (6, 1.0, SHAPE), (7, None, NULL),
                           (8, None, NULL)):
        a = list(ok)
        a[pos] = val
        assert f(*a) == code, (pos, val)
    with pytest.raises(ValueError):
        B.gqa_rope_table(64, scaling="other", device="cpu")


def test_binding_refusals_without_a_gpu():
    """Host tensors, wrong types and shapes are refused before the library is
    entered."""
    B = _b()
    T, h, g, d = 4, 8, 2, 128
    bf = torch.bfloat16
    t = dict(q=torch.zeros(T, h, d, dtype=bf), k_new=torch.zeros(T, g, d, dtype=bf),
             v_new=torch.zeros(T, g, d, dtype=bf), cu_tokens=torch.zeros(3, dtype=torch.int32),
             seq_lens=torch.zeros(2, dtype=torch.int32), q_out=torch.zeros(T, h, d, dtype=bf),
             k_cache=torch.zeros(2, g, 16, d, dtype=bf), v_cache=torch.zeros(2, g, 16, d, dtype=bf))

    def call(**kw):
        a = dict(t, **kw)
        B.gqa_rope_append(*a.values(), 2, h, g, d, d)

    with pytest.raises(ValueError, match="CUDA tensor"):
        call()
    with pytest.raises(ValueError, match="k_new: must be"):
        call(k_new=torch.zeros(T, g, d, dtype=torch.float16).to(bf)[:, :, :64])
    with pytest.raises(ValueError, match="v_new: must be torch.bfloat16"):
        call(v_new=torch.zeros(T, g, d))
    with pytest.raises(ValueError, match="heads of a token"):
        call(q=torch.zeros(T, d, h, dtype=bf).transpose(1, 2))
    with pytest.raises(ValueError, match="cu_tokens: must be torch.int32"):
        call(cu_tokens=torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="seq_lens: holds"):
        call(seq_lens=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="k_cache: must be contiguous"):
        call(k_cache=torch.zeros(2, 16, g, d, dtype=bf).transpose(1, 2))
    with pytest.raises(ValueError, match="rope: must be the tensor"):
        B.gqa_rope_append(*t.values(), 2, h, g, d, d, rope=[1, 2])
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA tensor"):
        B.gqa_chunk_attn(t["q"], t["k_cache"], t["v_cache"], t["cu_tokens"], t["seq_lens"], 2, h,
                         g, d, d, 0.1, t["q_out"], workspace=ws)
    with pytest.raises(ValueError, match="workspace: must be torch.uint8"):
        B.gqa_chunk_attn(t["q"], t["k_cache"], t["v_cache"], t["cu_tokens"], t["seq_lens"], 2, h,
                         g, d, d, 0.1, t["q_out"], workspace=ws.float())
    with pytest.raises(ValueError, match="out: must be"):
        B.gqa_chunk_attn(t["q"], t["k_cache"], t["v_cache"], t["cu_tokens"], t["seq_lens"], 2, h,
                         g, d, d, 0.1, t["q_out"].float(), workspace=ws)
    k8 = torch.zeros(9, g, 16, d, dtype=torch.uint8)
    sc = torch.zeros(9, g, 16)
    tab = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="k_pool: must be torch.float8_e4m3fn or torch.uint8"):
        B.gqa_kv_read_fp8_paged(k8.to(bf), k8, sc, sc, tab, t["seq_lens"], t["k_cache"],
                                t["v_cache"], 2, g, d, d)
    with pytest.raises(ValueError, match="v_scale: holds"):
        B.gqa_kv_read_fp8_paged(k8, k8, sc, sc[:5], tab, t["seq_lens"], t["k_cache"],
                                t["v_cache"], 2, g, d, d)
    with pytest.raises(ValueError, match="CUDA tensor"):
        B.gqa_decode_attn_fp8_paged(t["q"][:2], k8, k8, sc, sc, tab, t["seq_lens"], 2, h, g, d, d,
                                    0.1, t["q_out"][:2], workspace=ws)
