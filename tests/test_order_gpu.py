"""Calls that follow one another on a stream without anything between them: each
is ordered behind all that came before it, also behind a decode call none of
whose units is cut (its combine launch then has nothing to do).  The bits of
a run of calls equal those of the same calls with a synchronisation after
each, in a stream and as one captured graph."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _b():
    from gqa_kv_cache_append_gb300 import binding
    return binding


def both_ways(calls, state, results):
    """Bits of `results` after the calls from the same `state`: serialised, in a
    row, and replayed as a graph."""
    B = _b()
    keep = [x.clone() for x in state]

    def restore():
        for x, k in zip(state, keep):
            x.copy_(k)
        torch.cuda.synchronize()

    def bits():
        torch.cuda.synchronize()
        return [x.clone() for x in results()]

    restore()
    for call in calls:
        call()
        torch.cuda.synchronize()
    want = bits()
    assert all(torch.isfinite(x).all() for x in want)
    for _ in range(5):
        restore()
        for call in calls:
            call()
        for a, w in zip(bits(), want):
            assert torch.equal(a, w)
    gr = torch.cuda.CUDAGraph()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):  # (the projections' workspace is per stream)
        for call in calls:
            call()
    torch.cuda.synchronize()
    with torch.cuda.graph(gr, stream=st):
        for call in calls:
            call()
    for _ in range(5):
        restore()
        gr.replay()
        for a, w in zip(bits(), want):
            assert torch.equal(a, w)
    assert B.gqa_device_status() == 0


@pytest.mark.parametrize("order", ["project_first", "append_first"])
@pytest.mark.parametrize("longest", [256, 700])
def test_eight_bit_decode_then_its_consumers(order, longest):
    """Decode, the projection that reads its output, the rotation that
    overwrites its queries and the rows it read, and the next decode on the
    same workspace."""
    B = _b()
    gen = torch.Generator("cuda").manual_seed(41)
    b, h, g, d, bs, D = 128, 64, 8, 128, 64, 512
    mb = -(-longest // bs)
    lens = torch.randint(200, longest + 1, (b,), generator=gen, device="cuda").to(torch.int32)
    table = torch.randperm(b * mb, generator=gen, device="cuda").view(b, mb).to(torch.int32)
    k8, v8 = (torch.randn((b * mb, g, bs, d), generator=gen, device="cuda").to(
        torch.float8_e4m3fn).view(torch.uint8) for _ in range(2))
    ks, vs = (torch.rand((b * mb, g, bs), generator=gen, device="cuda") for _ in range(2))
    q, q2 = (torch.randn((b, h, d), generator=gen, device="cuda").to(BF) for _ in range(2))
    kn, vn = (torch.randn((b, g, d), generator=gen, device="cuda").to(BF) for _ in range(2))
    w_o = (torch.randn((h, D, d), generator=gen, device="cuda") / math.sqrt(h * d)).to(BF)
    cu = torch.arange(b + 1, dtype=torch.int32, device="cuda")
    phase, rs = B.gqa_rope_table(d)
    ws = torch.empty(B.gqa_decode_attn_fp8_workspace(b, 1, h, g, d, d, mb * bs),
                     dtype=torch.uint8, device="cuda")
    outs, ys = ([torch.zeros((b, n, m) if m else (b, n), dtype=BF, device="cuda")
                 for _ in range(2)] for n, m in ((h, d), (D, 0)))

    def decode(out):
        B.gqa_decode_attn_fp8_paged(q, k8, v8, ks, vs, table, lens, b, h, g, d, d,
                                    1 / math.sqrt(d), out, workspace=ws)

    def project(k):
        B.gqa_project_out(outs[k], w_o, ys[k], b, D, h, d)

    def append():
        B.gqa_rope_append_fp8_paged(q2, kn, vn, cu, lens, q, k8, v8, ks, vs, table, b, h, g, d, d,
                                    rope=phase, rope_scale=rs)

    mid = [lambda: project(0), append]
    if order == "append_first":
        mid.reverse()
    calls = [lambda: decode(outs[0]), *mid, lambda: decode(outs[1]), lambda: project(1)]
    both_ways(calls, [q, k8, v8, ks, vs, *outs, *ys], lambda: [*outs, *ys])


def test_decode_of_short_sequences_in_a_large_cache():
    """The 16-bit decode's combine launch, where no unit is cut either."""
    B = _b()
    gen = torch.Generator("cuda").manual_seed(42)
    b, h, g, d, cap, D = 2, 16, 1, 128, 1 << 16, 512
    assert B.gqa_decode_plan(b, 1, h, g, d, d, cap, B.GQA_BF16, num_sms=152)["ctas"] > 2 * b * g
    k, v = (torch.randn((b, g, cap, d), generator=gen, device="cuda").to(BF) for _ in range(2))
    q, q2 = (torch.randn((b, h, d), generator=gen, device="cuda").to(BF) for _ in range(2))
    kn, vn = (torch.randn((b, g, d), generator=gen, device="cuda").to(BF) for _ in range(2))
    w_o = (torch.randn((h, D, d), generator=gen, device="cuda") / math.sqrt(h * d)).to(BF)
    lens = torch.tensor([60, 128], dtype=torch.int32, device="cuda")
    cu = torch.arange(b + 1, dtype=torch.int32, device="cuda")
    outs, ys = ([torch.zeros((b, n, m) if m else (b, n), dtype=BF, device="cuda")
                 for _ in range(2)] for n, m in ((h, d), (D, 0)))

    def decode(out):
        B.gqa_decode_attn(q, k, v, lens, b, h, g, d, d, 1 / math.sqrt(d), out)

    calls = [lambda: decode(outs[0]),
             lambda: B.gqa_rope_append(q2, kn, vn, cu, lens, q, k, v, b, h, g, d, d),
             lambda: B.gqa_project_out(outs[0], w_o, ys[0], b, D, h, d),
             lambda: decode(outs[1]),
             lambda: B.gqa_project_out(outs[1], w_o, ys[1], b, D, h, d)]
    both_ways(calls, [q, k, v, *outs, *ys], lambda: [*outs, *ys])
