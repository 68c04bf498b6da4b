"""Rows at the ends of what an 8-bit cache can hold: tiny ones (whose factor
448 / max|x| is past fp32), zeros, huge ones, infinities and NaN, written by
gqa_rope_append_fp8_paged, read back, and met by gqa_decode_attn_fp8_paged.

Tolerance: the scale is one fp32 division, exact against torch's.  A stored
value is off from x * 448 / max|x| by half a step of e4m3, 2^-4 of itself or
2^-10, behind three fp32 roundings (2^-24 each: the factor and two products),
which can also move a value across the middle between two steps."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _b():
    from gqa_kv_cache_append_gb300 import binding
    return binding


class Pool:
    """Sequences of whole prompts, quantised and stored."""

    def __init__(self, k, v, lens, block=16):
        self.g, self.d = k.shape[1:]
        self.lens_h, self.b, self.block = lens, len(lens), block
        mb = -(-max(lens) // block)
        self.table = torch.randperm(self.b * mb, device="cuda").view(-1, mb).to(torch.int32)
        shape = (self.b * mb, self.g, block, self.d)
        self.k8, self.v8 = (torch.full(shape, 0x55, dtype=torch.uint8, device="cuda")
                            for _ in range(2))
        self.ks, self.vs = (torch.full(shape[:3], 7.0, device="cuda") for _ in range(2))
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        cu = torch.tensor([sum(lens[:i]) for i in range(self.b + 1)], dtype=torch.int32,
                          device="cuda")
        B = _b()
        B.gqa_rope_append_fp8_paged(None, k, v, cu, self.lens, None, self.k8, self.v8, self.ks,
                                    self.vs, self.table, self.b, self.g, self.g, self.d, self.d)
        assert B.gqa_device_status() == 0

    def rows(self, pool, i=0):
        t = self.table[i].long()
        return pool[t].transpose(1, 2).flatten(0, 1)[:self.lens_h[i]]  # [L, g, ..]

    def read(self, dtype):
        B = _b()
        out = [torch.full((self.b, self.g, max(self.lens_h), self.d), 9.0, dtype=dtype,
                          device="cuda") for _ in range(2)]
        B.gqa_kv_read_fp8_paged(self.k8, self.v8, self.ks, self.vs, self.table, self.lens, *out,
                                self.b, self.g, self.d, self.d)
        assert B.gqa_device_status() == 0
        return out


def values(rows8):
    return rows8.view(torch.float8_e4m3fn)


@pytest.mark.parametrize("dtype,powers", [
    (torch.float32, [-147, -140, -127, -126, -118, -110, -101, -100, -99, -60, 0, 60, 118, 126]),
    (BF, [-131, -127, -126, -110, -101, -100, -99, 0, 126]),
    (torch.float16, [-22, -16, -14, 0, 14]),
])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_sizes(dtype, powers, d):
    gen = torch.Generator("cuda").manual_seed(d)
    n, g = len(powers) + 1, 3
    x = torch.rand((n, g, d), generator=gen, device="cuda", dtype=torch.float64) * 2 - 1
    p = torch.tensor(powers + [0], device="cuda", dtype=torch.float64)
    x = (x * torch.exp2(p)[:, None, None]).to(dtype)
    x[-1] = 0
    pool = Pool(x, x.flip(1), [n])
    for rows, scale, src in ((pool.rows(pool.k8), pool.rows(pool.ks), x),
                             (pool.rows(pool.v8), pool.rows(pool.vs), x.flip(1))):
        amax = src.float().abs().amax(-1)
        # (divided in 64 bits: torch multiplies fp32 by the rounded 1 / 448)
        assert torch.equal(scale, (amax.double() / 448).float())
        y = src.double() * (448 / amax.double())[..., None]
        y[-1] = 0
        got = values(rows).double()
        assert (got.abs().amax(-1)[:-1] == 448).all()
        tol = torch.maximum(2.0 ** -4 * y.abs(), torch.tensor(2.0 ** -10)) * (1 + 2.0 ** -18)
        bad = (got - y).abs() > tol
        assert not bad.any(), bad.nonzero()[0].tolist()
    back = pool.read(torch.float32)
    want = values(pool.rows(pool.k8)).float() * pool.rows(pool.ks)[..., None]
    assert torch.equal(back[0][0].transpose(0, 1), want)


@pytest.mark.parametrize("dtype", [torch.float32, BF, torch.float16])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_that_are_not_finite(dtype, d):
    gen = torch.Generator("cuda").manual_seed(d + 1)
    x = torch.randn((40, 2, d), generator=gen, device="cuda").to(dtype)
    clean = Pool(x, x, [40])
    y = x.clone()
    for row, value in ((3, math.inf), (17, -math.inf), (20, math.nan)):
        y[row, 1, row] = value
    y[31, 0] = math.nan
    pool = Pool(y, y, [40])
    for a, c, sa, sc in ((pool.k8, clean.k8, pool.ks, clean.ks),
                         (pool.v8, clean.v8, pool.vs, clean.vs)):
        got, ref = pool.rows(a), clean.rows(c)
        nan = torch.isnan(values(got).float())
        for row, head in ((3, 1), (17, 1), (20, 1), (31, 0)):
            assert nan[row, head].any()
            nan[row, head] = False
            got[row, head] = ref[row, head]
        assert not nan.any() and torch.equal(got, ref)  # the other rows as ever
    back = pool.read(BF)[0][0]
    assert torch.isnan(back[1, 3]).all() and torch.isnan(back[1, 17]).all()
    assert torch.isnan(back[1, 20, 20]) and torch.isnan(back[0, 31]).all()
    assert torch.isnan(back).sum() >= 3 * d + 1
    assert torch.isfinite(back[:, 4:17]).all() and torch.isfinite(back[:, 32:]).all()


# positions of one sequence whole on a CTA, and cut between many
@pytest.mark.parametrize("lens", [[300, 40], [30000, 700]])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("n", [1, 4])
def test_decode_over_them(lens, which, value, n):
    """Every new token that sees the row has no finite output of that KV head,
    the other heads and sequences keep their bits."""
    B = _b()
    gen = torch.Generator("cuda").manual_seed(n)
    g, r, d = 2, 4, 128
    x = torch.randn((sum(lens), g, d), generator=gen, device="cuda").to(BF)
    q = torch.randn((2, n, g * r, d), generator=gen, device="cuda").to(BF)

    def run(pool):
        out = torch.full_like(q, 5.0)
        B.gqa_decode_attn_fp8_paged(q, pool.k8, pool.v8, pool.ks, pool.vs, pool.table, pool.lens,
                                    2, g * r, g, d, d, 1 / math.sqrt(d), out, n=n)
        assert B.gqa_device_status() == 0
        return out

    torch.manual_seed(0)
    ref = run(Pool(x, x, lens))
    assert torch.isfinite(ref).all()
    for pos in (0, lens[0] // 2, lens[0] - n):
        y = x.clone()
        y[pos, 1, 33] = value
        torch.manual_seed(0)
        out = run(Pool(y if which == "k" else x, y if which == "v" else x, lens))
        bad = out[0, :, r:]
        if which == "v" and math.isnan(value):
            bad = bad[..., 33]
        assert torch.isnan(bad).all()
        out[0, :, r:] = ref[0, :, r:]
        assert torch.equal(out, ref)
