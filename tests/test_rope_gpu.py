"""gqa_rope_append(_paged, _fp8_paged) and gqa_kv_read_fp8_paged against a
plain implementation in 64 bits.

Tolerances.  A rotated value is a cos t - c sin t (and its mate).  The angle
is off by at most half of 2^-32 turns and a rounding to fp32 of a number below
one half turn, pi 2^-25 together with it below 1.1e-7 rad; sine, cosine, the
factor and the two products round five times at 2^-23 or less (sincospi two
units): below (|a| + |c|) * factor * 1e-6.  The norm: mean of d <= 256 squares
(each product and sum 2^-24, at most 8 + 5 in a chain), reciprocal root 2^-22
and two products: below 2^-19 relative.  One rounding to the type at the end:
u = eps / 2 relative, and half of its smallest subnormal (fp16 2^-25).
e4m3 rows: the scale inherits the row's error (2^-19 and 2^-24 for the
division), a value is off by half a step, 2^-4 of itself, or 2^-10 scale
below the type's normal range.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}


def _b():
    from gqa_kv_cache_append_gb300 import binding
    return binding


def frequencies(rot, theta, scaling, factor, original_len, low, high):
    """f_m by the scalar formulas."""
    out = []
    two_pi = 2 * math.pi
    if scaling == "yarn":
        at = lambda t: rot * math.log(original_len / (t * two_pi)) / (2 * math.log(theta))
        first, last = max(math.floor(at(high)), 0), min(math.ceil(at(low)), rot - 1)
    for m in range(rot // 2):
        f = theta ** (-2.0 * m / rot)
        if scaling == "linear":
            f /= factor
        elif scaling == "wavelength":
            x = min(max((original_len * f / two_pi - low) / (high - low), 0.0), 1.0)
            f = (1 - x) * f / factor + x * f
        elif scaling == "yarn":
            x = min(max((m - first) / max(last - first, 1e-3), 0.0), 1.0)
            f = f * (1 - x) + f / factor * x
        out.append(f)
    return out


class Rope:
    def __init__(self, ns, ls, h=8, g=2, dk=128, dv=128, dtype="bf16", block=0, rot=None,
                 layout="half", norm=False, theta=10000.0, pad=0, seed=0, rope=True, fp8=False,
                 sliced=True, **scaling):
        B = _b()
        gen = torch.Generator("cpu").manual_seed(77 + seed)
        ty = TYPES[dtype]
        self.ns, self.ls, self.h, self.g, self.dk, self.dv = ns, ls, h, g, dk, dv
        self.b, self.t, self.dtype, self.block, self.fp8 = len(ns), sum(ns), dtype, block, fp8
        self.total = self.t + pad
        self.rot = rot or dk
        self.layout, self.theta = layout, theta
        self.cu = torch.from_numpy(np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)).cuda()
        self.lens = torch.tensor(ls, dtype=torch.int32).cuda()
        w = h * dk + g * (dk + dv)
        qkv = torch.randn((self.total, w), generator=gen).to(ty).cuda()
        self.q = qkv[:, :h * dk].unflatten(1, (h, dk))
        self.kn = qkv[:, h * dk:(h + g) * dk].unflatten(1, (g, dk))
        self.vn = qkv[:, (h + g) * dk:].unflatten(1, (g, dv))
        if not sliced:
            self.q, self.kn, self.vn = (x.contiguous() for x in (self.q, self.kn, self.vn))
        self.qout = torch.full((self.total, h, dk), 5.0, dtype=ty).cuda()
        cap = max(ls) + 3
        lead = (self.b, g, cap)
        if block:
            mb = -(-cap // block)
            nb = self.b * mb + 2
            self.table = torch.randperm(nb, generator=gen)[:self.b * mb].view(
                self.b, mb).to(torch.int32).cuda()
            lead = (nb, g, block)
        self.lead = lead
        cty = torch.uint8 if fp8 else ty
        self.k = torch.full((*lead, dk), 3, dtype=cty).cuda()
        self.v = torch.full((*lead, dv), 3, dtype=cty).cuda()
        self.ks = torch.full(lead, 2.0).cuda()
        self.vs = torch.full(lead, 2.0).cuda()
        self.kw = dict(eps=1e-6)
        if norm:
            self.kw.update(
                q_weight=(1 + 0.3 * torch.randn(dk, generator=gen)).to(ty).cuda(),
                k_weight=(1 + 0.3 * torch.randn(dk, generator=gen)).to(ty).cuda())
        self.f = None
        self.factor = 1.0
        if rope:
            s = dict(scaling="none", factor=1.0, original_len=0.0, low=1.0, high=32.0)
            s.update(scaling)
            phase, self.factor = B.gqa_rope_table(self.rot, theta=theta, **s)
            self.f = frequencies(self.rot, theta, **s)
            self.kw.update(rope=phase, rope_scale=self.factor,
                           layout=B.GQA_ROPE_HALF if layout == "half" else B.GQA_ROPE_PAIRS)

    def run(self, q=True, qout=None, **kw):
        B = _b()
        qo = self.qout if qout is None else qout
        a = (self.q if q else None, self.kn, self.vn, self.cu, self.lens, qo if q else None,
             self.k, self.v)
        dims = (self.b, self.h, self.g, self.dk, self.dv)
        if self.fp8:
            B.gqa_rope_append_fp8_paged(*a, self.ks, self.vs, self.table, *dims, **self.kw, **kw)
        elif self.block:
            B.gqa_rope_append_paged(*a, self.table, *dims, **self.kw, **kw)
        else:
            B.gqa_rope_append(*a, *dims, **self.kw, **kw)

    def turned(self, x, weight):
        """Norm and rotation in 64 bits: (value, error before the last
        rounding)."""
        x = x[:self.t].double()
        rel = 0.0
        if weight is not None:
            x = x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * weight.double()
            rel = 2.0 ** -19
        err = x.abs() * rel
        if self.f is None:
            return x, err
        pos = np.concatenate([np.arange(l - n, l) for n, l in zip(self.ns, self.ls)])
        ang = torch.tensor([[float(math.fmod(p * f, 2 * math.pi)) for f in self.f] for p in pos],
                           dtype=torch.float64).cuda()
        c, s = (ang.cos() * self.factor)[:, None], (ang.sin() * self.factor)[:, None]
        r = self.rot
        i0 = list(range(r // 2)) if self.layout == "half" else list(range(0, r, 2))
        i1 = list(range(r // 2, r)) if self.layout == "half" else list(range(1, r, 2))
        y, e = x.clone(), err.clone()
        y[..., i0] = x[..., i0] * c - x[..., i1] * s
        y[..., i1] = x[..., i1] * c + x[..., i0] * s
        mag = (x[..., i0].abs() + x[..., i1].abs()) * self.factor * (1e-6 + rel)
        e[..., i0] = mag
        e[..., i1] = mag
        return y, e

    def rows(self, pool):
        """The new rows [t, g, ...] of a cache or pool."""
        out = []
        for i, (n, l) in enumerate(zip(self.ns, self.ls)):
            for p in range(l - n, l):
                if self.block:
                    out.append(pool[int(self.table[i, p // self.block]), :, p % self.block])
                else:
                    out.append(pool[i, :, p])
        return torch.stack(out) if out else pool.new_zeros((0,))

    def untouched(self, pool, fill):
        """Every other row of a cache or pool still holds `fill`."""
        m = torch.zeros(self.lead, dtype=torch.bool, device="cuda")
        for i, (n, l) in enumerate(zip(self.ns, self.ls)):
            for p in range(l - n, l):
                if self.block:
                    m[int(self.table[i, p // self.block]), :, p % self.block] = True
                else:
                    m[i, :, p] = True
        return bool((pool[~m] == fill).all())

    def close(self, got, want, err):
        u = U[self.dtype]
        tol = err + u * (want.abs() + err) + (2.0 ** -25 if self.dtype == "f16" else 1e-30)
        d = (got.double() - want).abs()
        assert (d <= tol).all(), float((d - tol).max())

    def check(self, q=True):
        assert _b().gqa_device_status() == 0
        if q:
            self.close(self.qout[:self.t], *self.turned(self.q, self.kw.get("q_weight")))
        else:
            assert (self.qout == 5.0).all()
        assert (self.qout[self.t:] == 5.0).all()
        k, ek = self.turned(self.kn, self.kw.get("k_weight"))
        v, ev = self.vn[:self.t].double(), torch.zeros_like(self.vn[:self.t].double())
        if not self.fp8:
            self.close(self.rows(self.k), k, ek)
            assert torch.equal(self.rows(self.v), self.vn[:self.t])
            assert self.untouched(self.k, 3) and self.untouched(self.v, 3)
            return
        for pool, scale, x, e in ((self.k, self.ks, k, ek), (self.v, self.vs, v, ev)):
            sc = self.rows(scale).double()
            amax, emax = x.abs().amax(-1), e.amax(-1)
            assert ((sc - amax / 448).abs() <= (emax + 2.0 ** -23 * amax) / 448 + 1e-45).all()
            val = self.rows(pool).view(torch.float8_e4m3fn).double() * sc[..., None]
            tol = 2.0 ** -4 * (x.abs() + e) + 2.0 ** -10 * sc[..., None] + 1.1 * e + (
                2.0 ** -22 * x.abs())
            assert ((val - x).abs() <= tol).all()
            top = self.rows(pool).view(torch.float8_e4m3fn).double().abs().amax(-1)
            assert ((top == 448.0) | (amax == 0)).all()
            assert self.untouched(pool, 3) and self.untouched(scale, 2.0)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("block", [0, 16])
@pytest.mark.parametrize("norm", [False, True])
def test_types_layouts(dtype, layout, block, norm):
    r = Rope([3, 1, 40], [3, 70, 300], dtype=dtype, layout=layout, block=block, norm=norm, pad=2)
    r.run()
    r.check()


@pytest.mark.parametrize("dk,dv,rot", [(64, 64, 64), (64, 128, 16), (128, 64, 64), (96, 80, 48),
                                       (192, 128, 64), (256, 256, 256), (8, 16, None),
                                       (16, 8, 16), (112, 112, 112), (256, 64, 32)])
@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_head_dims(dk, dv, rot, layout, dtype):
    r = Rope([5, 2], [9, 33], h=6, g=3, dk=dk, dv=dv, rot=rot, layout=layout, norm=True,
             dtype=dtype, rope=rot is not None)
    r.run()
    r.check()


@pytest.mark.parametrize("scaling", [
    dict(), dict(scaling="linear", factor=4.0),
    dict(scaling="wavelength", factor=8.0, original_len=8192.0, low=1.0, high=4.0),
    dict(scaling="yarn", factor=16.0, original_len=4096.0, low=1.0, high=32.0)])
@pytest.mark.parametrize("theta", [10000.0, 500000.0])
def test_scalings_far_positions(scaling, theta):
    """Positions where a product in 32 bits has lost the angle."""
    r = Rope([3, 2], [(1 << 20) + 3, 100001], g=1, h=2, theta=theta, block=65536, **scaling)
    r.run()
    r.check()


def test_many_sequences_and_rows():
    rng = np.random.default_rng(1)
    ns = [int(x) for x in rng.integers(0, 4, 1500)]
    ls = [n + int(c) for n, c in zip(ns, rng.integers(0, 20, 1500))]
    r = Rope(ns, ls, h=2, g=1, dk=64, dv=64, block=16, pad=7, norm=True)
    r.run()
    r.check()


@pytest.mark.parametrize("h,g", [(64, 8), (28, 4), (8, 8), (71, 1), (1, 1)])
def test_heads(h, g):
    r = Rope([200, 1, 130], [200, 9, 131], h=h, g=g, norm=True, block=32)
    r.run()
    r.check()


def test_in_place_and_without_queries():
    r = Rope([20, 5], [20, 50], norm=True, sliced=False)
    before = r.q.clone()
    r.run(qout=r.q)
    r.qout[:] = r.q
    r.q = before
    r.check()
    r = Rope([20, 5], [20, 50], norm=True)
    r.run(q=False)
    r.check(q=False)


def test_plain_append_is_bit_exact():
    """Without table and weights the rows are copied."""
    r = Rope([20, 5], [20, 50], rope=False, block=16)
    r.run()
    r.check()
    assert torch.equal(r.rows(r.k), r.kn[:r.t]) and torch.equal(r.qout[:r.t], r.q[:r.t])


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dk,dv,block", [(128, 128, 16), (64, 128, 64), (256, 48, 16)])
@pytest.mark.parametrize("rope", [True, False])
def test_fp8_append(dtype, dk, dv, block, rope):
    r = Rope([30, 1, 7], [30, 65, 300], dk=dk, dv=dv, dtype=dtype, block=block, fp8=True,
             norm=rope, rope=rope, pad=3)
    r.kn[4] = 0  # a row of zeros has scale 0
    r.vn[4] = 0
    r.run(q=rope)
    r.check(q=rope)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dk,dv,block", [(128, 128, 16), (64, 128, 64), (256, 48, 256)])
def test_fp8_read(dtype, dk, dv, block):
    """scale * value rounded once: the same bits as the product in fp32
    rounded by torch; rows behind L_i stay."""
    B = _b()
    gen = torch.Generator("cpu").manual_seed(3)
    ls, g = [0, 1, 65, 300, 64], 3
    cap = 320
    mb = -(-cap // block)
    nb = 5 * mb
    table = torch.randperm(nb, generator=gen).view(5, mb).to(torch.int32)
    for i, l in enumerate(ls):
        table[i, -(-l // block):] = -1  # never read
    kp = torch.randn((nb, g, block, dk), generator=gen).mul(100).to(torch.float8_e4m3fn)
    vp = torch.randn((nb, g, block, dv), generator=gen).mul(100).to(torch.float8_e4m3fn)
    ks, vs = torch.rand((2, nb, g, block), generator=gen)
    ty = TYPES[dtype]
    kc = torch.full((5, g, cap, dk), 7.0, dtype=ty).cuda()
    vc = torch.full((5, g, cap, dv), 7.0, dtype=ty).cuda()
    B.gqa_kv_read_fp8_paged(kp.cuda(), vp.cuda(), ks.cuda(), vs.cuda(), table.cuda(),
                            torch.tensor(ls, dtype=torch.int32).cuda(), kc, vc, 5, g, dk, dv)
    assert B.gqa_device_status() == 0
    for pool, sc, got in ((kp, ks, kc.cpu()), (vp, vs, vc.cpu())):
        x = pool.float() * sc[..., None]
        for i, l in enumerate(ls):
            for p in range(l):
                want = x[table[i, p // block], :, p % block].to(ty)
                # (the few values past the type's range are NaN, and stay NaN)
                torch.testing.assert_close(got[i, :, p], want, rtol=0, atol=0, equal_nan=True)
            assert (got[i, :, l:] == 7.0).all()


def test_fp8_read_errors():
    B = _b()
    z = lambda *s, **k: torch.zeros(s, device="cuda", **k)
    kp = z(4, 1, 16, 64, dtype=torch.uint8)
    sc = z(4, 1, 16)
    table = torch.tensor([[0, 1], [2, 9]], dtype=torch.int32).cuda()
    kc, vc = z(2, 1, 32, 64), z(2, 1, 32, 64)
    for lens, bits in (([33, 4], B.GQA_DEV_BAD_SEQ_LEN), ([-1, 4], B.GQA_DEV_BAD_SEQ_LEN),
                       ([3, 20], B.GQA_DEV_BAD_BLOCK), ([32, 16], 0)):
        B.gqa_kv_read_fp8_paged(kp, kp, sc, sc, table,
                                torch.tensor(lens, dtype=torch.int32).cuda(), kc, vc, 2, 1, 64,
                                64)
        assert B.gqa_device_status() == bits


def test_bad_lengths_tokens_and_blocks():
    B = _b()
    r = Rope([4, 5, 6], [100, 60, 80], block=16)
    r.run()
    good = r.qout.clone()
    for lens, cu, block, bits in (
            ([100, 4, 80], None, None, B.GQA_DEV_BAD_SEQ_LEN),
            ([100, 5000, 80], None, None, B.GQA_DEV_BAD_SEQ_LEN),
            (None, [0, 4, 9, 16], None, B.GQA_DEV_BAD_TOKENS),
            (None, [0, 4, 2, 15], None, B.GQA_DEV_BAD_TOKENS),
            (None, None, -1, B.GQA_DEV_BAD_BLOCK), (None, None, 9999, B.GQA_DEV_BAD_BLOCK)):
        c = Rope([4, 5, 6], [100, 60, 80], block=16)
        if lens:
            c.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        if cu:
            c.cu.copy_(torch.tensor(cu, dtype=torch.int32))
        if block is not None:
            c.table[1, 3] = block
        c.run()
        assert B.gqa_device_status() & bits
        if cu == [0, 4, 2, 15]:
            continue  # rows 2 and 3 lie in two sequences' ranges
        assert torch.equal(c.qout[:4], good[:4])  # sequence 0 is not affected
        if lens:
            assert (c.qout[4:9] == 5.0).all() and torch.equal(c.qout[9:], good[9:])


def test_graph_and_stream():
    B = _b()
    r = Rope([3, 1, 40], [3, 70, 300], block=16, norm=True)
    r.run()
    st = torch.cuda.Stream()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=st):
        r.run()
    for x, f in ((r.qout, 5.0), (r.k, 3), (r.v, 3)):
        x.fill_(f)
    gr.replay()
    torch.cuda.synchronize()
    r.check()
    for x, f in ((r.qout, 5.0), (r.k, 3), (r.v, 3)):
        x.fill_(f)
    torch.cuda.synchronize()
    r.run(stream=st)
    st.synchronize()
    r.check()
    assert B.gqa_device_status() == 0
