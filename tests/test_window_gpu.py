"""gqa_chunk_attn_window(_paged): packed chunks over their last positions and the
first ones, against a plain implementation in 64 bits (tolerances:
part_cases.py)."""
import math

import numpy as np
import pytest
import torch

from part_cases import Part, binding

pytestmark = pytest.mark.gpu

LENGTHS = [
    ([1], [1]), ([1], [300]), ([1], [1000]), ([5], [5]), ([129], [129]), ([300], [300]),
    ([33, 1, 64], [33, 500, 190]), ([2, 0, 3], [2, 70, 400]), ([1, 1, 1, 1], [1, 64, 129, 3000]),
    ([700], [1500]), ([257, 3], [257, 2049]),
]


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (100, 4), (128, 64), (200, 65),
                                          (65, 130), (1000, 3), (5000, 0), (5000, 5000)])
@pytest.mark.parametrize("ns,ls", LENGTHS)
def test_lengths_contiguous(ns, ls, window, sinks):
    c = Part(ns, ls, 16, 2, window=window, sinks=sinks, slack=3)
    c.run()
    c.check()


@pytest.mark.parametrize("window,sinks", [(1, 0), (17, 1), (100, 0), (128, 4), (300, 70),
                                          (5000, 16)])
@pytest.mark.parametrize("block", [16, 32, 64, 256])
@pytest.mark.parametrize("ns,ls", LENGTHS[2:])
def test_lengths_paged(ns, ls, window, sinks, block):
    c = Part(ns, ls, 8, 2, window=window, sinks=sinks, block=block)
    c.run()
    c.check()


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("block", [0, 32])
def test_head_dims_and_types(dk, dv, dtype, block):
    c = Part([70, 1, 200], [333, 1290, 200], 8, 2, dk, dv, window=90, sinks=5, block=block,
             dtype=dtype)
    c.run()
    c.check()


@pytest.mark.parametrize("h,g", [(1, 1), (8, 8), (3, 1), (7, 1), (28, 4), (16, 1), (71, 1),
                                 (128, 1), (64, 1)])
def test_head_groups(h, g):
    c = Part([37, 150, 1], [900, 150, 260], h, g, window=77, sinks=2, pad=4)
    c.run()
    c.check()


@pytest.mark.parametrize("block", [0, 16])
def test_many_sequences(block):
    rng = np.random.default_rng(5)
    ns = [int(x) for x in rng.integers(0, 40, 150)]
    ls = [int(n + c) for n, c in zip(ns, rng.integers(0, 600, 150))]
    c = Part(ns, ls, 4, 2, 64, 64, window=120, sinks=4, block=block, pad=9)
    c.run()
    c.check()


@pytest.mark.parametrize("block", [0, 16, 128])
@pytest.mark.parametrize("sinks", [0, 4, 200])
def test_long_windows_split(block, sinks):
    """Few rows over a long window: every unit is cut into many pieces."""
    c = Part([3, 9], [20000, 30001], 8, 1, window=15000, sinks=sinks, block=block)
    c.run()
    c.check()


@pytest.mark.parametrize("window,sinks", [(300, 4), (1024, 0), (2049, 100)])
def test_prompts_many_units(window, sinks):
    """Runs of many units, growing ones and full ones."""
    c = Part([2500, 1300], [2500, 1700], 16, 4, window=window, sinks=sinks, seed=3)
    c.run()
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_window_beyond_every_length_is_the_causal_form(dtype):
    c = Part([300, 1, 40], [300, 700, 500], 8, 2, window=1 << 30, sinks=0, dtype=dtype)
    c.run()
    c.check()
    c = Part([300, 1, 40], [300, 700, 500], 8, 2, window=0x7FFFFFFF, sinks=0x7FFFFFFF, block=16,
             dtype=dtype)
    c.run()
    c.check()


def test_window_of_one_is_v():
    """A token that sees itself alone: its V row, bit for bit."""
    c = Part([50, 1], [400, 33], 6, 2, window=1)
    c.run()
    assert binding().gqa_device_status() == 0
    want = torch.cat([c.v[0, :, 350:400].transpose(0, 1), c.v[1, :, 32:33].transpose(0, 1)])
    assert torch.equal(c.out, want.repeat_interleave(3, 1))


@pytest.mark.parametrize("scale", [-0.09, 0.0, 1.0, 4.0])
def test_scales(scale):
    c = Part([40, 3], [400, 500], 8, 2, 64, 64, window=130, sinks=7, scale=scale, dtype="f16")
    c.run()
    c.check()


def test_growing_logits():
    """Keys whose logits grow along the cache raise the maximum in every tile."""
    c = Part([64], [1024], 2, 1, 64, 64, window=700, sinks=100)
    ramp = torch.linspace(0.2, 6.0, 1024, device="cuda")[None, None, :, None]
    c.q.abs_()
    c.k.copy_((c.k.float().abs() * ramp).to(c.k.dtype))
    c.run()
    c.check()


def test_dominant_sink():
    """Sinks that take nearly all weight, and fp16 weights behind them."""
    for dtype in ("bf16", "f16"):
        c = Part([20, 1], [900, 2000], 4, 1, window=500, sinks=3, dtype=dtype)
        c.k[:, :, 0] = c.q[0, 0] * 0.3
        c.run()
        c.check()


@pytest.mark.parametrize("block", [0, 64])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_values_that_are_not_finite_next_to_the_window(block, value):
    """A single token's result does not depend on what lies before its window,
    between the sinks and it, or behind its length."""
    c = Part([1, 1], [777, 2000], 8, 2, window=200, sinks=5, block=block)
    c.run()
    c.check()
    good = c.out.clone()
    for x in (c.k, c.v):
        x[x.isnan()] = value
    if block:
        for x in (c.kp, c.vp):
            x[x.isnan()] = value
    c.run()
    assert torch.equal(c.out, good)


def test_nan_in_the_window_and_in_a_sink():
    good = Part([1, 1], [777, 2000], 8, 2, window=200, sinks=5).run().clone()
    for pos in (577, 4, 776):
        c = Part([1, 1], [777, 2000], 8, 2, window=200, sinks=5)
        c.v[0, 1, pos, 5] = math.nan
        c.run()
        assert c.out[0, 4:, 5].isnan().all()
        c.out[0, 4:, 5] = good[0, 4:, 5]
        assert torch.equal(c.out, good)


def test_workspace_contents_do_not_matter_and_bits_repeat():
    B = binding()
    c = Part([50, 3, 700], [5000, 3, 900], 16, 2, window=3000, sinks=4, block=64)
    n = B.gqa_chunk_attn_workspace(c.total, c.h, c.g, c.dk, c.dv)
    outs = []
    for fill in (0, 255, 127):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        outs.append(c.run(workspace=ws).clone())
    c.check()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_empty_batch():
    c = Part([0, 0], [0, 40], 8, 2, window=10, sinks=2, pad=6)
    c.run()
    assert binding().gqa_device_status() == 0
    assert (c.out == 5.0).all()
    c = Part([0], [40], 8, 2, window=10)
    c.run()
    assert binding().gqa_device_status() == 0


def test_bad_lengths_tokens_and_blocks():
    B = binding()
    c = Part([4, 5, 6], [100, 600, 800], 8, 2, window=70, sinks=3, block=16)
    c.run()
    c.check()
    good = c.out.clone()
    for bad in (4, -1, c.table.shape[1] * 16 + 1):
        c.lens[1] = bad
        c.out.fill_(5.0)
        c.run()
        assert B.gqa_device_status() == B.GQA_DEV_BAD_SEQ_LEN
        assert (c.out[4:9] == 5.0).all()
        assert torch.equal(c.out[:4], good[:4]) and torch.equal(c.out[9:], good[9:])
    c.lens[1] = 600
    for bad in (-1, 16):
        cu = c.cu.clone()
        c.cu[3] = bad
        c.out.fill_(5.0)
        c.run()
        assert B.gqa_device_status() & B.GQA_DEV_BAD_TOKENS
        assert torch.equal(c.out[:9], good[:9]) and (c.out[9:] == 5.0).all()
        c.cu.copy_(cu)
    for entry, bad in ((0, -1), (0, c.kp.shape[0]), (36, -1), (37, c.kp.shape[0])):
        t = c.table.clone()
        c.table[1, entry] = bad
        c.run()
        assert B.gqa_device_status() == B.GQA_DEV_BAD_BLOCK
        assert torch.equal(c.out[:4], good[:4]) and torch.equal(c.out[9:], good[9:])
        c.table.copy_(t)
    c.run()
    c.check()


def test_graphs_streams_and_other_data():
    """Two captured calls replayed side by side, then other data and lengths
    through the same graph; a stream given as object and as handle."""
    cs = [Part([40, 3], [3000, 4100], 8, 1, window=2500, sinks=4, seed=s) for s in (1, 2)]
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
    for x in (c.k, c.v):
        x.copy_(torch.randn_like(x.float()).to(x.dtype))
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


def test_outputs_aligned_to_16_bytes():
    c = Part([70, 3], [300, 400], 6, 2, 64, 64, window=100, sinks=1)
    c.run()
    c.check()
    n = c.out.numel()
    good, c.out = c.out, torch.zeros(n + 8, dtype=c.out.dtype, device="cuda")[8:].view(c.out.shape)
    assert c.out.data_ptr() % 32 == 16
    c.run()
    assert torch.equal(c.out, good)
