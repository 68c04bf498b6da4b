"""gqa_chunk_attn(_paged): causal attention of packed chunks over the cache,
against a plain implementation in 64 bits.

Tolerance, elementwise, with u = eps / 2 of the type (bf16 2^-8, fp16 2^-11)
and A = sum_p w_p |v_p| (the weighted mean of |V|, from the reference):
  rounding of the softmax weights for P.V    u A
  rounding of the output                     u |out|
  logits: fp32 accumulation of d <= 128 products, each step off by at most
  2^-23 of the running sum, itself at most E = |scale| sum |q k|: the exponent
  is off by at most d 2^-23 E, and a weight and the weights' sum by a factor
  exp of that each                           2 d 2^-23 E A
  exp2 (2^-22), its argument (2^-23 of at most 64 + E), row sums and rescales
  in fp32                                    2^-16 A
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def _b():
    from gqa_kv_cache_append_gb300 import binding
    return binding


class Case:
    """Packed chunks and a cache filled so that every row that must not count
    holds NaN."""

    def __init__(self, ns, ls, h, g, dk, dv, block=0, dtype="bf16", pad=0, scale=None, seed=0,
                 spread=1.0, slack=0):
        gen = torch.Generator("cpu").manual_seed(1234 + seed)
        ty = TYPES[dtype]
        self.ns, self.ls, self.h, self.g, self.dk, self.dv = ns, ls, h, g, dk, dv
        self.b, self.t, self.dtype, self.block = len(ns), sum(ns), dtype, block
        self.total = self.t + pad
        self.scale = 1.0 / math.sqrt(dk) if scale is None else scale
        cu = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
        self.cu = torch.from_numpy(cu).cuda()
        self.lens = torch.tensor(ls, dtype=torch.int32).cuda()
        r = lambda *s: torch.randn(s, generator=gen).to(ty)
        self.q = (spread * r(self.total, h, dk)).to(ty).cuda()
        if pad:
            self.q[self.t:] = float("nan")
        cap = max(max(ls), 1) + slack
        k = torch.full((self.b, g, cap, dk), float("nan"), dtype=ty)
        v = torch.full((self.b, g, cap, dv), float("nan"), dtype=ty)
        for i, l in enumerate(ls):
            k[i, :, :l] = r(g, l, dk)
            v[i, :, :l] = r(g, l, dv)
        self.k, self.v, self.cap = k.cuda(), v.cuda(), cap
        if block:
            mb = -(-cap // block)
            used = [-(-l // block) for l in ls]
            nb = sum(used) + 2
            perm = torch.randperm(nb, generator=gen).to(torch.int32)
            self.table = torch.full((self.b, mb), -7, dtype=torch.int32)  # unused: never read
            kp = torch.full((nb, g, block, dk), float("nan"), dtype=ty)
            vp = torch.full((nb, g, block, dv), float("nan"), dtype=ty)
            at = 0
            for i, l in enumerate(ls):
                for m in range(used[i]):
                    blk = int(perm[at])
                    at += 1
                    self.table[i, m] = blk
                    n = min(block, l - m * block)
                    kp[blk, :, :n] = k[i, :, m * block:m * block + n]
                    vp[blk, :, :n] = v[i, :, m * block:m * block + n]
            self.kp, self.vp, self.table = kp.cuda(), vp.cuda(), self.table.cuda()
        self.out = torch.full((self.total, h, dv), 5.0, dtype=ty).cuda()

    def run(self, **kw):
        B = _b()
        a = (self.b, self.h, self.g, self.dk, self.dv, self.scale)
        if self.block:
            B.gqa_chunk_attn_paged(self.q, self.kp, self.vp, self.table, self.cu, self.lens, *a,
                                   self.out, **kw)
        else:
            B.gqa_chunk_attn(self.q, self.k, self.v, self.cu, self.lens, *a, self.out, **kw)
        return self.out

    def reference(self):
        """out, A and the largest E per row, in 64 bits."""
        r = self.h // self.g
        out = torch.zeros(self.t, self.h, self.dv, dtype=torch.float64, device="cuda")
        A, E = torch.zeros_like(out), torch.zeros(self.t, self.h, 1, dtype=torch.float64,
                                                  device="cuda")
        at = 0
        for i, (n, l) in enumerate(zip(self.ns, self.ls)):
            for j in range(self.g if n else 0):
                k, v = self.k[i, j, :l].double(), self.v[i, j, :l].double()
                for a in range(r):
                    q = self.q[at:at + n, j * r + a].double()
                    for lo in range(0, n, 1024):
                        hi = min(n, lo + 1024)
                        s = q[lo:hi] @ k.T * self.scale
                        e = (q[lo:hi].abs() @ k.abs().T * abs(self.scale))
                        seen = (torch.arange(l, device="cuda")[None] <=
                                torch.arange(l - n + lo, l - n + hi, device="cuda")[:, None])
                        w = torch.softmax(s.masked_fill(~seen, -math.inf), -1)
                        out[at + lo:at + hi, j * r + a] = w @ v
                        A[at + lo:at + hi, j * r + a] = w @ v.abs()
                        E[at + lo:at + hi, j * r + a, 0] = (e * seen).amax(-1)
            at += n
        return out, A, E

    def check(self, status=0):
        B = _b()
        assert B.gqa_device_status() == status
        ref, A, E = self.reference()
        u = U[self.dtype]
        tol = u * A + u * ref.abs() + 2 * self.dk * 2.0 ** -23 * E * A + 2.0 ** -16 * A + 1e-7
        got = self.out[:self.t].double()
        err = (got - ref).abs()
        bad = ~(err <= tol)
        assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} off, first at "
                               f"{bad.nonzero()[0].tolist()}, worst {float(err.max())}")
        if self.total > self.t:
            assert (self.out[self.t:] == 5.0).all()  # rows behind the last sequence


LENGTHS = [
    ([1], [1]), ([1], [128]), ([1], [129]), ([5], [5]), ([127], [127]), ([128], [128]),
    ([129], [300]), ([33, 1, 64], [33, 500, 190]), ([300], [300]), ([2, 0, 3], [2, 70, 400]),
    ([1, 1, 1, 1], [1, 16, 17, 1000]), ([1000], [1500]), ([257, 3], [257, 2049]),
]


@pytest.mark.parametrize("ns,ls", LENGTHS)
def test_lengths_contiguous(ns, ls):
    c = Case(ns, ls, 16, 2, 128, 128, slack=3)
    c.run()
    c.check()


@pytest.mark.parametrize("ns,ls", LENGTHS)
@pytest.mark.parametrize("block", [16, 64, 256])
def test_lengths_paged(ns, ls, block):
    c = Case(ns, ls, 8, 2, 128, 128, block=block)
    c.run()
    c.check()


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("block", [0, 32])
def test_head_dims_and_types(dk, dv, dtype, block):
    c = Case([70, 1, 200], [333, 129, 200], 8, 2, dk, dv, block=block, dtype=dtype)
    c.run()
    c.check()


@pytest.mark.parametrize("h,g", [(1, 1), (8, 8), (3, 1), (7, 1), (28, 4), (16, 1), (71, 1),
                                 (128, 1), (64, 1)])
def test_head_groups(h, g):
    c = Case([37, 150, 1], [90, 150, 260], h, g, 128, 128, pad=4)
    c.run()
    c.check()


def test_many_sequences():
    rng = np.random.default_rng(5)
    ns = [int(x) for x in rng.integers(0, 40, 150)]
    ls = [int(n + c) for n, c in zip(ns, rng.integers(0, 300, 150))]
    c = Case(ns, ls, 4, 2, 64, 64, block=16, pad=9)
    c.run()
    c.check()


@pytest.mark.parametrize("block", [0, 16, 128])
def test_split_long_cache(block):
    """Few rows over a long cache: every unit is cut into many pieces."""
    c = Case([3, 9], [20000, 30001], 8, 1, 128, 128, block=block)
    c.run()
    c.check()


def test_large_prompt_many_units():
    """Runs of many units, whose ends snap to unit edges."""
    c = Case([2500, 1300], [2500, 1700], 16, 4, 128, 128, seed=3)
    c.run()
    c.check()


@pytest.mark.parametrize("scale", [-0.09, 0.0, 1.0, 4.0])
def test_scales(scale):
    """Negative, zero and large scales (large: one weight dominates, the
    running maximum is raised often)."""
    c = Case([40, 3], [400, 50], 8, 2, 64, 64, scale=scale, dtype="f16")
    c.run()
    c.check()


def test_growing_logits():
    """Keys whose logits grow along the cache raise the maximum in every tile."""
    c = Case([64], [1024], 2, 1, 64, 64)
    ramp = torch.linspace(0.2, 6.0, 1024, device="cuda")[None, None, :, None]
    c.q.abs_()
    c.k.copy_((c.k.float().abs() * ramp).to(c.k.dtype))
    c.run()
    c.check()


def test_workspace_contents_do_not_matter_and_bits_repeat():
    B = _b()
    c = Case([50, 3, 700], [5000, 3, 900], 16, 2, 128, 128, block=64)
    n = B.gqa_chunk_attn_workspace(c.total, c.h, c.g, c.dk, c.dv)
    outs = []
    for fill in (0, 255, 127):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        outs.append(c.run(workspace=ws).clone())
    c.check()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_empty_batch():
    c = Case([0, 0], [0, 40], 8, 2, 128, 128, pad=6)
    c.run()
    assert _b().gqa_device_status() == 0
    assert (c.out == 5.0).all()
    c = Case([0], [40], 8, 2, 128, 128)
    c.run()
    assert _b().gqa_device_status() == 0


def test_bad_lengths_tokens_and_blocks():
    B = _b()
    c = Case([4, 5, 6], [100, 60, 80], 8, 2, 128, 128, block=16)
    c.run()
    good = c.out.clone()
    c.lens[1] = 4  # below its new tokens
    c.out.fill_(5.0)
    c.run()
    assert B.gqa_device_status() == B.GQA_DEV_BAD_SEQ_LEN
    assert (c.out[4:9] == 5.0).all()
    assert torch.equal(c.out[:4], good[:4]) and torch.equal(c.out[9:], good[9:])
    c.lens[1] = c.table.shape[1] * 16 + 1  # beyond the table
    c.run()
    assert B.gqa_device_status() == B.GQA_DEV_BAD_SEQ_LEN
    c.lens[1] = 60
    for bad in (-1, 16):
        cu = c.cu.clone()
        c.cu[3] = bad if bad > 0 else -1
        c.out.fill_(5.0)
        c.run()
        assert B.gqa_device_status() & B.GQA_DEV_BAD_TOKENS
        assert torch.equal(c.out[:9], good[:9]) and (c.out[9:] == 5.0).all()
        c.cu.copy_(cu)
    for bad in (-1, c.kp.shape[0]):
        t = c.table.clone()
        c.table[1, 2] = bad
        c.run()
        assert B.gqa_device_status() == B.GQA_DEV_BAD_BLOCK
        assert torch.equal(c.out[:4], good[:4]) and torch.equal(c.out[9:], good[9:])
        c.table.copy_(t)
    c.run()
    c.check()


def test_two_graphs_on_streams_of_their_own():
    """Two captured calls replayed side by side, each with the workspace that
    the call makes under its capture."""
    cs = [Case([40, 3], [3000, 4100], 8, 1, 128, 128, seed=s) for s in (1, 2)]
    for c in cs:
        c.run()
    torch.cuda.synchronize()
    graphs, streams = [], [torch.cuda.Stream() for _ in cs]
    for c, st in zip(cs, streams):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            c.run()
        graphs.append(gr)
    for c in cs:
        c.out.fill_(5.0)
    torch.cuda.synchronize()
    for _ in range(5):
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    for c in cs:
        c.check()
    # other data through the same graph
    cs[0].q.copy_(torch.randn_like(cs[0].q.float()).to(cs[0].q.dtype))
    cs[0].lens[0] -= 130
    graphs[0].replay()
    torch.cuda.synchronize()
    cs[0].ls[0] -= 130
    cs[0].check()


def test_another_stream():
    c = Case([40, 3], [3000, 4100], 8, 1, 128, 128)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    c.run(stream=st)
    st.synchronize()
    c.check()
    c.out.fill_(5.0)
    torch.cuda.synchronize()
    c.run(stream=st.cuda_stream)
    st.synchronize()
    c.check()
