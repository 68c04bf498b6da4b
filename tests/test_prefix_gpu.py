"""gqa_chunk_attn_prefix(_paged): packed chunks of sequences with a common
prefix, against a plain implementation in 64 bits (tolerances: part_cases.py)."""
import math

import numpy as np
import pytest
import torch

from part_cases import Part, binding

pytestmark = pytest.mark.gpu

# new tokens, and positions between the prefix and them
SHAPES = [
    ([1], [0]), ([1, 1], [0, 5]), ([1] * 5, [0, 1, 63, 300, 1000]),
    ([0, 1, 1, 0, 2], [9, 0, 40, 3, 7]),
    ([3, 1, 4], [130, 20, 0]), ([200, 1, 3], [5, 0, 40]), ([300], [20]), ([70, 90], [0, 400]),
]


@pytest.mark.parametrize("prefix", [1, 64, 100, 128, 1000])
@pytest.mark.parametrize("block", [0, 16, 64, 256])
@pytest.mark.parametrize("ns,ctx", SHAPES)
def test_shapes(ns, ctx, prefix, block):
    c = Part(ns, [prefix + x + n for n, x in zip(ns, ctx)], 16, 2, prefix=prefix, block=block,
             slack=3)
    c.run()
    c.check()


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("block", [0, 32])
@pytest.mark.parametrize("ns", [[1, 4, 2], [70, 1, 200]])
def test_head_dims_and_types(dk, dv, dtype, block, ns):
    c = Part(ns, [333 + n + 50 * i for i, n in enumerate(ns)], 8, 2, dk, dv, prefix=333,
             block=block, dtype=dtype)
    c.run()
    c.check()


@pytest.mark.parametrize("h,g", [(1, 1), (8, 8), (3, 1), (7, 1), (28, 4), (16, 1), (71, 1),
                                 (128, 1), (64, 1)])
def test_head_groups(h, g):
    c = Part([2, 1, 1, 0, 1], [290, 278, 500, 277, 300], h, g, prefix=277, pad=4)
    c.run()
    c.check()


@pytest.mark.parametrize("block", [0, 16])
@pytest.mark.parametrize("prefix", [40, 900, 5000])
def test_many_sequences(block, prefix):
    """More tokens than a unit holds, units of the prefix and of the sequences
    cut and whole."""
    rng = np.random.default_rng(5)
    ns = [int(x) for x in rng.integers(0, 4, 150)]
    ls = [int(prefix + n + c) for n, c in zip(ns, rng.integers(0, 300, 150))]
    c = Part(ns, ls, 8, 2, 64, 64, prefix=prefix, block=block, pad=9)
    c.run()
    c.check()


@pytest.mark.parametrize("block", [0, 64])
def test_long_prefix_and_long_sequences(block):
    c = Part([1, 3, 1, 2], [30001, 20011, 29000, 22000], 8, 1, prefix=20000, block=block)
    c.run()
    c.check()


def test_same_as_the_causal_call():
    """Over caches that hold the prefix for every sequence, both forms of the
    work agree with gqa_chunk_attn to the rounding of the type."""
    B = binding()
    for ns in ([1, 2, 1, 3], [40, 60, 200, 1]):
        c = Part(ns, [500 + n + 30 * i for i, n in enumerate(ns)], 8, 2, prefix=500)
        c.k[1:, :, :500], c.v[1:, :, :500] = c.k[:1, :, :500], c.v[:1, :, :500]
        got = c.run().clone()
        c.check()
        B.gqa_chunk_attn(c.q, c.k, c.v, c.cu, c.lens, c.b, c.h, c.g, c.dk, c.dv, c.scale, c.out)
        c.check()
        assert (got.double() - c.out.double()).abs().max() < 2.0 ** -5


@pytest.mark.parametrize("block", [0, 16])
def test_prefix_of_zero_is_the_causal_form(block):
    c = Part([1, 5, 1], [300, 20, 1], 8, 2, prefix=0, block=block)
    c.run()
    c.check()


@pytest.mark.parametrize("scale", [-0.09, 0.0, 1.0, 4.0])
def test_scales(scale):
    c = Part([2, 3], [400, 470], 8, 2, 64, 64, prefix=333, scale=scale, dtype="f16")
    c.run()
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_one_side_holds_nearly_all_weight(dtype):
    """Weights of the prefix far above those of the sequence's own rows, and far
    below them."""
    for where in (3, 450):
        c = Part([1, 1, 1], [460, 500, 451], 4, 1, prefix=450, dtype=dtype)
        c.k[0 if where < 450 else slice(None), :, where] = c.q[0, 0] * 0.5
        c.run()
        c.check()


@pytest.mark.parametrize("which", ["k", "v"])
def test_nan(which):
    """A NaN in the prefix reaches every token, one in a sequence's own row that
    sequence alone."""
    c = Part([1, 2, 1], [400, 333, 500], 8, 2, prefix=300)
    good = c.run().clone()
    getattr(c, which)[2, 1, 499, 3] = math.nan
    c.run()
    assert torch.equal(c.out[:3], good[:3]) and torch.equal(c.out[3, :4], good[3, :4])
    bad = c.out[3, 4:] if which == "k" else c.out[3, 4:, 3]
    assert bad.isnan().all()
    c = Part([1, 2, 1], [400, 333, 500], 8, 2, prefix=300)
    getattr(c, which)[0, 1, 7, 3] = math.nan
    c.run()
    assert torch.equal(c.out[:, :4], good[:, :4])
    bad = c.out[:, 4:] if which == "k" else c.out[:, 4:, 3]
    assert bad.isnan().all()


def test_workspace_contents_do_not_matter_and_bits_repeat():
    B = binding()
    for ns, ctx in (([1] * 20, range(20)), ([100, 20, 9], [4, 900, 0])):
        c = Part(ns, [4000 + n + x for n, x in zip(ns, ctx)], 16, 2, prefix=4000, block=64)
        n = B.gqa_chunk_attn_prefix_workspace(c.b, c.total, c.h, c.g, c.dk, c.dv)
        outs = []
        for fill in (0, 255, 127):
            ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
            outs.append(c.run(workspace=ws).clone())
        c.check()
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_workspace_of_a_larger_total():
    """One workspace for every step of a batch, of few tokens and of many."""
    B = binding()
    n = B.gqa_chunk_attn_prefix_workspace(4, 500, 16, 2, 128, 128)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    for ns in ([1, 1, 1, 1], [0, 1, 0, 0], [16, 16, 16, 15], [16, 16, 16, 16], [100, 300, 1, 99]):
        c = Part(ns, [700 + x for x in ns], 16, 2, prefix=700)
        c.run(workspace=ws)
        c.check()


def test_empty_batch():
    c = Part([0, 0], [0, 640], 8, 2, prefix=600, pad=6)
    c.run()
    assert binding().gqa_device_status() == 0
    assert (c.out == 5.0).all()


def test_bad_lengths_tokens_and_blocks():
    B = binding()
    c = Part([1, 2, 3], [100, 160, 180], 8, 2, prefix=96, block=16)
    c.run()
    c.check()
    good = c.out.clone()
    for bad in (97, 1, c.table.shape[1] * 16 + 1):  # (97: its new tokens begin in the prefix)
        c.lens[1] = bad
        c.out.fill_(5.0)
        c.run()
        assert B.gqa_device_status() == B.GQA_DEV_BAD_SEQ_LEN
        assert (c.out[1:3] == 5.0).all()
        # (the rest with its units cut in other places)
        got, c.out = c.out, good
        assert (got[[0, 3, 4, 5]].double() - good[[0, 3, 4, 5]].double()).abs().max() < 2.0 ** -5
    c.out = good.clone()
    c.lens[1] = 160
    for bad in (-1, 16):
        cu = c.cu.clone()
        c.cu[3] = bad
        c.out.fill_(5.0)
        c.run()
        assert B.gqa_device_status() & B.GQA_DEV_BAD_TOKENS
        assert (c.out[3:] == 5.0).all()
        c.cu.copy_(cu)
    for row, entry, bad in ((0, 2, -1), (0, 0, c.kp.shape[0]), (1, 8, -1)):
        t = c.table.clone()
        c.table[row, entry] = bad
        c.run()
        assert B.gqa_device_status() == B.GQA_DEV_BAD_BLOCK
        c.table.copy_(t)
    c.run()
    c.check()


def test_graphs_streams_and_other_data():
    cs = [Part([1, 3, 1], [3000, 4100, 2600], 8, 1, prefix=2500, seed=s) for s in (1, 2)]
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
    c = cs[0]
    c.q.copy_(torch.randn_like(c.q.float()).to(c.q.dtype))
    c.lens[0] -= 130
    c.ls[0] -= 130
    graphs[0].replay()
    torch.cuda.synchronize()
    c.check()
    st = torch.cuda.Stream()
    for handle in (st, st.cuda_stream):
        c.out.fill_(5.0)
        torch.cuda.synchronize()
        c.run(stream=handle)
        st.synchronize()
        c.check()
