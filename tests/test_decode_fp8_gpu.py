"""gqa_decode_attn_fp8_paged against a plain implementation in 64 bits over the
values the cache stands for.

Tolerance, elementwise (u = 2^-8, A = sum_p w_p |v_p|, M = largest |V| the
row sees, S = 1 / largest weight, E = |scale| sum |q k| at its largest):
  output rounding                                   u |out|
  weights times V scales as two e4m3 pieces: 2^-4 of the residual, itself
  2^-4 of the value                                 u A
  ... below the pieces' normal range 2^-14 of 256 parts of the tile's largest
  scale, for each of L positions whose weights sum to at least 1 / S of the
  largest one's                                     2^-22 L M / S
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

pytestmark = pytest.mark.gpu


def _b():
    from gqa_kv_cache_append_gb300 import binding
    return binding


class Case:
    def __init__(self, lens, h, g, dk=128, dv=128, n=1, block=16, seed=0, scale=None, spread=0.5,
                 extra=0):
        gen = torch.Generator("cpu").manual_seed(500 + seed)
        self.lens_h, self.b, self.h, self.g, self.n = lens, len(lens), h, g, n
        self.dk, self.dv, self.block = dk, dv, block
        self.scale = 1.0 / math.sqrt(dk) if scale is None else scale
        cap = max(max(lens), n) + extra
        self.mb = mb = -(-cap // block)
        used = [-(-l // block) for l in lens]
        nb = sum(used) + 2
        perm = torch.randperm(nb, generator=gen).to(torch.int32)
        table = torch.full((self.b, mb), -3, dtype=torch.int32)  # unused: never read
        at = 0
        for i, u in enumerate(used):
            table[i, :u] = perm[at:at + u]
            at += u
        self.q = torch.randn((self.b, n, h, dk), generator=gen).to(torch.bfloat16).cuda()
        pools = []
        for d in (dk, dv):
            x = torch.randn((nb, g, block, d), generator=gen)
            # rows of different sizes, and zeros
            x *= torch.exp(spread * torch.randn((nb, g, block, 1), generator=gen))
            x[torch.rand((nb, g, block), generator=gen) < 0.02] = 0
            sc = x.abs().amax(-1) / 448
            q8 = (x / torch.where(sc > 0, sc, 1.0)[..., None]).to(torch.float8_e4m3fn)
            pools.append([q8.view(torch.uint8), sc])
        # rows past the lengths, and unused blocks: NaN values and scales
        live = torch.zeros((nb, block), dtype=torch.bool)
        for i, l in enumerate(lens):
            for m in range(used[i]):
                live[int(table[i, m]), :min(block, l - m * block)] = True
        for q8, sc in pools:
            q8.transpose(1, 2)[~live] = 0x7F
            sc.transpose(1, 2)[~live] = float("nan")
        (self.k8, self.ks), (self.v8, self.vs) = [[y.cuda() for y in x] for x in pools]
        self.table = table.cuda()
        self.lens = torch.tensor(lens, dtype=torch.int32).cuda()
        self.out = torch.full((self.b, n, h, dv), 5.0, dtype=torch.bfloat16).cuda()

    def run(self, **kw):
        _b().gqa_decode_attn_fp8_paged(self.q, self.k8, self.v8, self.ks, self.vs, self.table,
                                       self.lens, self.b, self.h, self.g, self.dk, self.dv,
                                       self.scale, self.out, n=self.n, **kw)
        return self.out

    def rows(self, pool, sc, i, l):
        t = self.table[i, :-(-l // self.block)].long()
        x = pool[t].view(torch.float8_e4m3fn).double() * sc[t].double()[..., None]
        return x.transpose(0, 1).flatten(1, 2)[:, :l]

    def check(self, skip=()):
        u = 2.0 ** -8
        r = self.h // self.g
        for i, l in enumerate(self.lens_h):
            if i in skip:
                continue
            k, v = self.rows(self.k8, self.ks, i, l), self.rows(self.v8, self.vs, i, l)
            for s in range(self.n):
                see = l - self.n + s + 1
                q = self.q[i, s].double().view(self.g, r, self.dk)
                kk, vv = k[:, :see], v[:, :see]
                x = q @ kk.transpose(1, 2) * self.scale
                w = torch.softmax(x, -1)
                ref, A = w @ vv, w @ vv.abs()
                M = vv.abs().amax((1, 2))[:, None, None]
                S = 1.0 / w.amax(-1, keepdim=True)
                E = (q.abs() @ kk.abs().transpose(1, 2) * abs(self.scale)).amax(-1, keepdim=True)
                Q = (2.0 ** -21 * abs(self.scale) * q.abs().amax(-1, keepdim=True) *
                     kk.abs().sum(-1).amax(-1)[:, None, None])
                tol = (u * ref.abs() + u * A + 2.0 ** -22 * see * M / S +
                       2 * (Q + (self.dk + 8) * 2.0 ** -23 * E) * A + 2.0 ** -16 * A + 1e-30)
                got = self.out[i, s].double().view(self.g, r, self.dv)
                bad = ~((got - ref).abs() <= tol)
                assert not bad.any(), (i, s, bad.nonzero()[0].tolist(),
                                       float((got - ref).abs().max()), float(tol.max()))


@pytest.mark.parametrize("lens", [[1], [2], [16], [17], [255], [256], [257], [513, 1, 300],
                                  [1000, 64, 5, 777]])
@pytest.mark.parametrize("block", [16, 64, 256, 1024])
def test_lengths_and_blocks(lens, block):
    c = Case(lens, 16, 2, block=block)
    c.run()
    assert _b().gqa_device_status() == 0
    c.check()


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
@pytest.mark.parametrize("h,g,n", [(8, 2, 1), (8, 1, 1), (12, 1, 1), (16, 1, 1), (28, 4, 2),
                                   (32, 1, 1), (8, 1, 4), (6, 2, 10), (1, 1, 32), (1, 1, 1),
                                   (17, 1, 1)])
def test_head_dims_and_rows(dk, dv, h, g, n):
    c = Case([n, 300 + n, 700, 33 + n], h, g, dk, dv, n=n, block=32)
    c.run()
    assert _b().gqa_device_status() == 0
    c.check()


@pytest.mark.parametrize("lens", [[20000], [9000, 4097, 12]])
@pytest.mark.parametrize("h,g,n", [(4, 1, 1), (32, 1, 1), (16, 2, 2)])
def test_split_units(lens, h, g, n):
    c = Case(lens, h, g, n=n, block=64)
    c.run()
    assert _b().gqa_device_status() == 0
    c.check()


def test_many_units_a_cta():
    rng = np.random.default_rng(2)
    c = Case([int(x) for x in rng.integers(1, 700, 90)], 16, 4, block=16, extra=3000)
    c.run()
    assert _b().gqa_device_status() == 0
    c.check()


@pytest.mark.parametrize("scale", [-0.1, 0.0, 1.0])
@pytest.mark.parametrize("spread", [0.0, 3.0])
def test_scales(scale, spread):
    c = Case([700, 20], 8, 1, scale=scale, spread=spread)
    c.run()
    assert _b().gqa_device_status() == 0
    c.check()


def test_zero_query_and_large_queries():
    c = Case([300, 40], 8, 2)
    c.q[0, 0, 0] = 0
    c.q[0, 0, 1] *= 2.0 ** 30
    c.q[0, 0, 2] *= 2.0 ** -100
    c.q[1, 0, 0, :100] *= 2.0 ** -20
    c.scale = 2.0 ** -31
    c.run()
    assert _b().gqa_device_status() == 0
    c.check()


def test_bits_repeat_and_workspace_contents():
    B = _b()
    c = Case([5000, 70, 9000], 8, 1, n=2)
    n = B.gqa_decode_attn_fp8_workspace(c.b, c.n, c.h, c.g, c.dk, c.dv, c.mb * c.block)
    outs = []
    for fill in (0, 255, 127):
        outs.append(c.run(workspace=torch.full((n,), fill, dtype=torch.uint8,
                                               device="cuda")).clone())
    c.check()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_bad_lengths_and_blocks():
    B = _b()
    c = Case([300, 400, 500], 8, 2)
    for bad in (0, -4, c.mb * c.block + 1):
        c.lens[1] = bad
        c.out.fill_(5.0)
        c.run()
        assert B.gqa_device_status() == B.GQA_DEV_BAD_SEQ_LEN
        assert (c.out[1] == 5.0).all()
        c.check(skip=(1,))
    c.lens[1] = 400
    keep = int(c.table[1, 3])
    for bad in (-1, c.k8.shape[0]):
        c.table[1, 3] = bad
        c.run()
        assert B.gqa_device_status() == B.GQA_DEV_BAD_BLOCK
        c.check(skip=(1,))
    c.table[1, 3] = keep
    c.run()
    assert B.gqa_device_status() == 0
    c.check()


def test_two_graphs_on_streams_of_their_own():
    cs = [Case([3000, 4100], 8, 1, seed=s) for s in (1, 2)]
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
