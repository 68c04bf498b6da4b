"""gqa_decode_attn_fp8_window_paged against a plain implementation in 64 bits over
the values the cache stands for.

Tolerance, elementwise (u = 2^-8, A = sum_p w_p |v_p|, M = largest |V| the row
sees, S = 1 / largest weight, E = |scale| sum |q k| at its largest):
  output rounding                                   u |out|
  weights times V scales as two e4m3 pieces: 2^-4 of the residual, itself
  2^-4 of the value                                 u A
  ... below the pieces' normal range 2^-14 of 256 parts of the tile's largest
  scale, for each of the positions seen, whose weights sum to at least 1 / S of
  the largest one's                                 2^-22 (positions) M / S
  query pieces: exact for a bf16 value down to 2^-13 of its row's largest,
  below that off by 2^-21 of the largest; logits accumulate d <= 128 products
  in fp32 (2^-23 each), three factors (2^-23 each), exp2 (2^-22) and its
  argument: a factor exp of the sum on weights and on their total
     2 (2^-21 |scale| max|q| sum|k| + (d + 8) 2^-23 E) A + 2^-16 A
"""
import math

import numpy as np
import pytest
import torch

from part_cases import binding

pytestmark = pytest.mark.gpu


class Case:
    """Rows that no new token sees hold NaN values and scales; entries of blocks
    of such rows are not in the pool."""

    def __init__(self, lens, h, g, window, sinks=0, dk=128, dv=128, n=1, block=16, seed=0,
                 scale=None, spread=0.5, extra=0):
        gen = torch.Generator("cpu").manual_seed(900 + seed)
        self.lens_h, self.b, self.h, self.g, self.n = list(lens), len(lens), h, g, n
        self.dk, self.dv, self.block, self.window, self.sinks = dk, dv, block, window, sinks
        self.scale = 1.0 / math.sqrt(dk) if scale is None else scale
        cap = max(max(lens), n) + extra
        self.mb = mb = -(-cap // block)
        kept = [sorted({int(p) // block for p in self.used(l)}) for l in lens]
        nb = sum(map(len, kept)) + 2
        perm = torch.randperm(nb, generator=gen).to(torch.int32)
        table = torch.full((self.b, mb), -3, dtype=torch.int32)  # unused: never read
        live = torch.zeros((nb, block), dtype=torch.bool)
        at = 0
        for i, l in enumerate(lens):
            for m in kept[i]:
                table[i, m] = perm[at]
                at += 1
            for p in self.used(l):
                live[int(table[i, int(p) // block]), int(p) % block] = True
        self.q = torch.randn((self.b, n, h, dk), generator=gen).to(torch.bfloat16).cuda()
        pools = []
        for d in (dk, dv):
            x = torch.randn((nb, g, block, d), generator=gen)
            # rows of different sizes, and zeros
            x *= torch.exp(spread * torch.randn((nb, g, block, 1), generator=gen))
            x[torch.rand((nb, g, block), generator=gen) < 0.02] = 0
            sc = x.abs().amax(-1) / 448
            q8 = (x / torch.where(sc > 0, sc, 1.0)[..., None]).to(torch.float8_e4m3fn)
            q8 = q8.view(torch.uint8)
            q8.transpose(1, 2)[~live] = 0x7F
            sc.transpose(1, 2)[~live] = float("nan")
            pools.append([q8.cuda(), sc.cuda()])
        (self.k8, self.ks), (self.v8, self.vs) = pools
        self.table = table.cuda()
        self.lens = torch.tensor(lens, dtype=torch.int32).cuda()
        self.out = torch.full((self.b, n, h, dv), 5.0, dtype=torch.bfloat16).cuda()

    def used(self, l):
        p = np.arange(max(l, 0))
        return p[(p < self.sinks) | (p > l - self.n - self.window)]

    def run(self, **kw):
        binding().gqa_decode_attn_fp8_window_paged(
            self.q, self.k8, self.v8, self.ks, self.vs, self.table, self.lens, self.b, self.h,
            self.g, self.dk, self.dv, self.scale, self.window, self.out, sinks=self.sinks,
            n=self.n, **kw)
        return self.out

    def rows(self, pool, sc, i, p):
        t = self.table[i].long()[p // self.block]
        x = pool[t, :, p % self.block].view(torch.float8_e4m3fn).double()
        return (x * sc[t, :, p % self.block].double()[..., None]).transpose(0, 1)

    def check(self, skip=()):
        u = 2.0 ** -8
        r = self.h // self.g
        for i, l in enumerate(self.lens_h):
            if i in skip:
                continue
            for s in range(self.n):
                pos = l - self.n + s
                p = torch.arange(pos + 1, device="cuda")
                p = p[(p > pos - self.window) | (p < self.sinks)]
                kk, vv = self.rows(self.k8, self.ks, i, p), self.rows(self.v8, self.vs, i, p)
                q = self.q[i, s].double().view(self.g, r, self.dk)
                x = q @ kk.transpose(1, 2) * self.scale
                w = torch.softmax(x, -1)
                ref, A = w @ vv, w @ vv.abs()
                M = vv.abs().amax((1, 2))[:, None, None]
                S = 1.0 / w.amax(-1, keepdim=True)
                E = (q.abs() @ kk.abs().transpose(1, 2) * abs(self.scale)).amax(-1, keepdim=True)
                Q = (2.0 ** -21 * abs(self.scale) * q.abs().amax(-1, keepdim=True) *
                     kk.abs().sum(-1).amax(-1)[:, None, None])
                tol = (u * ref.abs() + u * A + 2.0 ** -22 * len(p) * M / S +
                       2 * (Q + (self.dk + 8) * 2.0 ** -23 * E) * A + 2.0 ** -16 * A + 1e-30)
                got = self.out[i, s].double().view(self.g, r, self.dv)
                bad = ~((got - ref).abs() <= tol)
                assert not bad.any(), (i, s, bad.nonzero()[0].tolist(),
                                       float((got - ref).abs().max()), float(tol.max()))


@pytest.mark.parametrize("lens", [[1], [17], [256], [257], [513, 1, 300], [1000, 64, 5, 4000]])
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 1), (100, 0), (200, 64), (255, 70),
                                          (300, 300), (9999, 4)])
@pytest.mark.parametrize("block", [16, 64, 256])
def test_lengths_and_blocks(lens, window, sinks, block):
    c = Case(lens, 16, 2, window, sinks, block=block)
    c.run()
    assert binding().gqa_device_status() == 0
    c.check()


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
@pytest.mark.parametrize("h,g,n", [(8, 2, 1), (12, 1, 1), (28, 4, 2), (32, 1, 1), (8, 1, 4),
                                   (6, 2, 10), (1, 1, 32), (17, 1, 1)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (150, 7)])
def test_head_dims_and_rows(dk, dv, h, g, n, window, sinks):
    c = Case([n, 300 + n, 700, 33 + n], h, g, window, sinks, dk=dk, dv=dv, n=n, block=32)
    c.run()
    assert binding().gqa_device_status() == 0
    c.check()


@pytest.mark.parametrize("lens", [[20000], [9000, 14097, 12]])
@pytest.mark.parametrize("h,g,n", [(4, 1, 1), (32, 1, 1), (16, 2, 2)])
def test_split_units(lens, h, g, n):
    c = Case(lens, h, g, 8000, 100, n=n, block=64)
    c.run()
    assert binding().gqa_device_status() == 0
    c.check()


def test_many_units_a_cta():
    rng = np.random.default_rng(2)
    c = Case([int(x) for x in rng.integers(1, 1700, 90)], 16, 4, 333, 5, block=16, extra=3000)
    c.run()
    assert binding().gqa_device_status() == 0
    c.check()


@pytest.mark.parametrize("scale", [-0.1, 0.0, 1.0])
@pytest.mark.parametrize("spread", [0.0, 3.0])
def test_scales(scale, spread):
    c = Case([700, 20], 8, 1, 450, 3, scale=scale, spread=spread)
    c.run()
    assert binding().gqa_device_status() == 0
    c.check()


def test_largest_window_is_the_whole_cache():
    B = binding()
    c = Case([700, 20, 3000], 8, 2, 0x7FFFFFFF, 0x7FFFFFFF)
    got = c.run().clone()
    c.check()
    B.gqa_decode_attn_fp8_paged(c.q, c.k8, c.v8, c.ks, c.vs, c.table, c.lens, c.b, c.h, c.g, c.dk,
                                c.dv, c.scale, c.out)
    assert B.gqa_device_status() == 0
    assert torch.equal(got, c.out)


def test_bits_repeat_and_workspace_contents():
    B = binding()
    c = Case([5000, 70, 9000], 8, 1, 4000, 9, n=2)
    n = B.gqa_decode_attn_fp8_workspace(c.b, c.n, c.h, c.g, c.dk, c.dv, c.mb * c.block)
    outs = []
    for fill in (0, 255, 127):
        outs.append(c.run(workspace=torch.full((n,), fill, dtype=torch.uint8,
                                               device="cuda")).clone())
    c.check()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_bad_lengths_and_blocks():
    B = binding()
    c = Case([300, 400, 500], 8, 2, 150, 5)
    for bad in (0, -4, c.mb * c.block + 1):
        c.lens[1] = bad
        c.out.fill_(5.0)
        c.run()
        assert B.gqa_device_status() == B.GQA_DEV_BAD_SEQ_LEN
        assert (c.out[1] == 5.0).all()
        c.check(skip=(1,))
    c.lens[1] = 400
    for entry in (0, 15, 24):
        keep = int(c.table[1, entry])
        for bad in (-1, c.k8.shape[0]):
            c.table[1, entry] = bad
            c.run()
            assert B.gqa_device_status() == (B.GQA_DEV_BAD_BLOCK)
            c.check(skip=(1,))
        c.table[1, entry] = keep
    c.run()
    assert B.gqa_device_status() == 0
    c.check()


def test_two_graphs_on_streams_of_their_own():
    cs = [Case([3000, 4100], 8, 1, 2100, 4, seed=s) for s in (1, 2)]
    for c in cs:
        c.run()
    torch.cuda.synchronize()
    graphs, streams = [], [torch.cuda.Stream() for _ in cs]
    for c, st in zip(cs, streams):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            c.run()
        graphs.append(gr)
        c.out.fill_(5.0)
    torch.cuda.synchronize()
    for _ in range(5):
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    for c in cs:
        c.check()
    st = torch.cuda.Stream()
    cs[0].out.fill_(5.0)
    torch.cuda.synchronize()
    cs[0].run(stream=st)
    st.synchronize()
    cs[0].check()
