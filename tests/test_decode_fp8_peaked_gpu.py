"""gqa_decode_attn_fp8_paged where a few positions hold nearly all of the weight
and others of the output: a dominant first position whose V row is small, V
rows of very different sizes, both over long contexts.

Tolerance, elementwise, against 64 bits over the values the cache stands for
(u = 2^-8, A = sum_p w_p |v_p|; tiles of 256 positions, T_t the largest
w_p vscale_p of tile t, 8-bit values v8_p):
  output rounding                                           u |out|
  weights times V scales as two e4m3 pieces                 u A
  ... whose step is 2^-13 below 2^-6, with 256 for T_t: off by 2^-14 / 256
                                     2^-22 sum_t T_t sum_(p in t) |v8_p|
  logits: query pieces off by at most 2^-21 of the row's largest, d products
  accumulated in fp32 (2^-23 each), three factors (2^-23 each), exp2 (2^-22)
  and its argument, on weights and on their total (E = |scale| sum |q k| at
  its largest)
     2 (2^-21 |scale| max|q| sum|k| + (d + 8) 2^-23 E) A + 2^-16 A
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
U = 2.0 ** -8


def _b():
    from gqa_kv_cache_append_gb300 import binding
    return binding


class Peaked:
    """b sequences over the same blocks, each with queries of its own."""

    def __init__(self, b, length, h=16, g=8, d=128, n=1, share=0.99, sink=0.001, v_spread=0.0,
                 block=64, seed=0):
        gen = torch.Generator("cuda").manual_seed(900 + seed)
        self.b, self.L, self.h, self.g, self.d, self.n, self.block = b, length, h, g, d, n, block
        self.scale = 1 / math.sqrt(d)
        nb = -(-length // block)

        def rand(*shape):
            return torch.randn(shape, generator=gen, device="cuda")

        k = 0.5 * rand(g, nb * block, d)
        # V rows with a common direction, of different sizes where asked for
        v = rand(g, 1, d) + 0.5 * rand(g, nb * block, d)
        v = v * torch.exp(v_spread * rand(g, nb * block, 1))
        v[:, 0] *= sink
        base = rand(g, d)
        if share > 0:
            # the first position's key: the query's direction, so long that it
            # takes `share` of the weight
            x = (k[:, 1:length] @ base[:, :, None])[..., 0] * self.scale
            want = torch.logsumexp(x.double(), -1) + math.log(share / (1 - share))
            k[:, 0] = base * (want / (self.scale * (base.double() ** 2).sum(-1)))[:, None].float()
        r = h // g
        q = base[None, None, :, None] * torch.ones((b, n, g, r, d), device="cuda")
        self.q = (q + 0.02 * rand(b, n, g, r, d)).flatten(2, 3).to(BF).contiguous()
        self.pools = []
        for x in (k, v):
            sc = x.abs().amax(-1) / 448
            x8 = (x / torch.where(sc > 0, sc, 1.0)[..., None]).to(torch.float8_e4m3fn)
            x8 = x8.view(torch.uint8)
            self.pools.append((x8.view(g, nb, block, d).transpose(0, 1).contiguous(),
                               sc.view(g, nb, block).transpose(0, 1).contiguous()))
        self.table = torch.arange(nb, dtype=torch.int32, device="cuda").repeat(b, 1)
        self.lens = torch.full((b,), length, dtype=torch.int32, device="cuda")
        self.out = torch.full((b, n, h, d), 5.0, dtype=BF, device="cuda")

    def run(self):
        B = _b()
        (k8, ks), (v8, vs) = self.pools
        B.gqa_decode_attn_fp8_paged(self.q, k8, v8, ks, vs, self.table, self.lens, self.b, self.h,
                                    self.g, self.d, self.d, self.scale, self.out, n=self.n)
        assert B.gqa_device_status() == 0

    def check(self):
        L, g, d, r = self.L, self.g, self.d, self.h // self.g
        (k8, ks), (v8, vs) = [(x.transpose(0, 1).flatten(1, 2)[:, :L].view(
            torch.float8_e4m3fn).double(), s.transpose(0, 1).flatten(1, 2)[:, :L].double())
            for x, s in self.pools]
        k, v = k8 * ks[..., None], v8 * vs[..., None]
        pad = -L % 256
        v8t = torch.nn.functional.pad(v8.abs(), (0, 0, 0, pad)).view(g, -1, 256, d).sum(2)
        ksum = k.abs().sum(-1).amax(-1)[:, None, None]
        for i in {0, self.b // 2, self.b - 1}:
            for s in range(self.n):
                q = self.q[i, s].double().view(g, r, d)
                x = q @ k.transpose(1, 2) * self.scale
                see = L - self.n + s + 1
                x[..., see:] = -math.inf
                w = torch.softmax(x, -1)
                ref, A = w @ v, w @ v.abs()
                T = torch.nn.functional.pad(w * vs.abs()[:, None], (0, pad)).view(g, r, -1, 256).amax(-1)
                E = (q.abs() @ k.abs().transpose(1, 2) * self.scale).amax(-1, keepdim=True)
                Q = 2.0 ** -21 * self.scale * q.abs().amax(-1, keepdim=True) * ksum
                tol = (U * ref.abs() + U * A + 2.0 ** -22 * (T @ v8t) +
                       2 * (Q + (d + 8) * 2.0 ** -23 * E) * A + 2.0 ** -16 * A)
                err = (self.out[i, s].double().view(g, r, d) - ref).abs()
                assert (err <= tol).all(), (i, s, float((err / tol).max()),
                                            float((err.norm() / ref.norm())))


@pytest.mark.parametrize("share,sink", [(0.99, 0.03), (0.99, 0.001), (0.999, 0.0001)])
@pytest.mark.parametrize("length", [1000, 32768, 131072])
def test_dominant_first_position_whole_units(length, share, sink):
    c = Peaked(19, length, share=share, sink=sink)  # as many units as SMs
    c.run()
    c.check()


@pytest.mark.parametrize("share,sink", [(0.99, 0.001), (0.999, 0.0)])
@pytest.mark.parametrize("length", [32768, 131001])
@pytest.mark.parametrize("h,n", [(8, 1), (16, 3), (64, 4)])
def test_dominant_first_position_cut_units(length, share, sink, h, n):
    c = Peaked(1, length, h=h, n=n, share=share, sink=sink, seed=1)
    c.run()
    c.check()


@pytest.mark.parametrize("share", [0.0, 0.999999])
@pytest.mark.parametrize("v_spread", [2.0, 8.0])
@pytest.mark.parametrize("b,length", [(19, 2048), (1, 20001)])
def test_rows_of_very_different_sizes(b, length, v_spread, share):
    c = Peaked(b, length, share=share, sink=2.0 ** -30 if share else 1.0, v_spread=v_spread,
               seed=2)
    c.run()
    c.check()


@pytest.mark.parametrize("power", [-115, -40, 100])
def test_rows_all_small_or_large(power):
    c = Peaked(2, 700, sink=0.1, seed=3)
    c.pools[1][1].mul_(2.0 ** power)
    c.run()
    c.check()


@pytest.mark.parametrize("which", ["some", "all"])
@pytest.mark.parametrize("length", [700, 20001])
def test_negative_scales(which, length):
    """Rows are scale times value, whatever the scale's sign."""
    c = Peaked(2, length, share=0.0, sink=1.0, v_spread=2.0, seed=5)
    for _, sc in c.pools:
        flip = torch.rand(sc.shape, device="cuda") < 0.5 if which == "some" else sc > 0
        sc.copy_(torch.where(flip, -sc, sc))
    c.run()
    c.check()


def test_rows_of_zeros():
    c = Peaked(2, 700, sink=0.1, seed=4)
    for x in c.pools[1]:
        x.zero_()
    c.run()
    assert (c.out == 0).all()
