"""The chunk calls (causal, window, prefix) give the same bits on every call,
whatever ran on the GPU before them: lanes and rows without a query take what
shared and tensor memory held."""
import random

import pytest
import torch

from part_cases import Part, binding

pytestmark = pytest.mark.gpu


def _causal(c):
    """gqa_chunk_attn over the case's rows, its other rows set to zero."""
    B = binding()
    k, v = (x.nan_to_num(0.0) for x in (c.k, c.v))

    def run():
        B.gqa_chunk_attn(c.q, k, v, c.cu, c.lens, c.b, c.h, c.g, c.dk, c.dv, c.scale, c.out)
        return c.out
    return run


def _disturb(seed):
    """Calls with large logits and NaN, which leave other values behind."""
    for size in (1, 40, 300):
        c = Part([size], [size + 900], 16, 1, window=700, sinks=3, scale=8.0, seed=seed)
        c.q[::2] = float("nan")
        c.run()
    binding().gqa_device_status()


@pytest.mark.parametrize("kind", ["window", "prefix", "causal"])
@pytest.mark.parametrize("h,g", [(3, 1), (7, 1), (8, 1), (28, 4), (16, 2), (71, 1)])
@pytest.mark.parametrize("ns", [[1], [1, 1, 1], [5, 1, 40], [70, 3], [200, 1]])
def test_same_bits_after_other_calls(kind, h, g, ns):
    kw = dict(prefix=300) if kind == "prefix" else dict(window=200, sinks=2)
    c = Part(ns, [300 + n + 130 * i for i, n in enumerate(ns)], h, g, seed=len(ns), **kw)
    run = _causal(c) if kind == "causal" else c.run
    first = run().clone()
    for k in range(3):
        _disturb(k)
        c.out.fill_(5.0)
        assert torch.equal(run(), first)
    assert binding().gqa_device_status() == 0


def test_single_tokens_over_whole_tiles():
    """Many units of one token and of whole tiles, back to back in a graph."""
    B = binding()
    b, h, g, d = 64, 64, 8, 128
    for length in (100, 128, 1024, 4096):
        gen = torch.Generator("cuda").manual_seed(length)
        k, v = (torch.randn((b, g, length, d), generator=gen, device="cuda",
                            dtype=torch.bfloat16) for _ in range(2))
        q = torch.randn((b, h, d), generator=gen, device="cuda", dtype=torch.bfloat16)
        cu = torch.arange(b + 1, dtype=torch.int32, device="cuda")
        lens = torch.full((b,), length, dtype=torch.int32, device="cuda")
        outs = [torch.empty_like(q) for _ in range(2)]
        args = (q, k, v, cu, lens, b, h, g, d, d, 0.09)

        def run():
            B.gqa_chunk_attn(*args, outs[0])
            B.gqa_chunk_attn_window(*args, length, outs[1])
        run()
        assert B.gqa_device_status() == 0
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(6):
                run()
        for _ in range(5):
            graph.replay()
        assert B.gqa_device_status() == 0
        w = torch.softmax(q.double().view(b, g, -1, d) @ k.double().transpose(2, 3) * 0.09, -1)
        want, a = (w @ x for x in (v.double(), v.double().abs()))
        for out in outs:
            err = (out.double().view(want.shape) - want).abs()
            assert (err <= 2.0 ** -8 * (want.abs() + a) + 2.0 ** -15 * a).all()


def test_random_cases():
    rng = random.Random(11)
    for n in range(60):
        g, r, b = rng.choice([1, 2, 4]), rng.choice([1, 3, 4, 7, 8, 16]), rng.choice([1, 2, 5, 20])
        dk, dv = rng.choice([(64, 64), (128, 128), (64, 128), (128, 64)])
        ns = [rng.choice([0, 1, 1, 2, 9, rng.randint(1, 100), rng.randint(1, 400)])
              for _ in range(b)]
        if sum(ns) == 0:
            continue
        kw = dict(block=rng.choice([0, 0, 16, 64, 256]), dtype=rng.choice(["bf16", "f16"]))
        if rng.random() < 0.6:
            kw.update(window=rng.choice([1, 30, 100, 300, 1000]),
                      sinks=rng.choice([0, 1, 5, 64, 100]))
            ls = [x + rng.choice([0, rng.randint(0, 100), rng.randint(0, 1500)]) for x in ns]
        else:
            kw["prefix"] = rng.choice([1, 40, 64, 100, 500, 1500])
            ls = [kw["prefix"] + x + rng.choice([0, rng.randint(0, 300)]) for x in ns]
        c = Part(ns, ls, g * r, g, dk, dv, seed=n, **kw)
        first = c.run().clone()
        c.check()
        for _ in range(3):
            c.out.fill_(5.0)
            assert torch.equal(c.run(), first)
