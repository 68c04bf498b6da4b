"""gqa_chunk_attn where one early position holds nearly all of the weight and its
V row next to nothing, over long caches: the output is the small weights'.

Tolerance, elementwise, against 64 bits (u = 2^-8 for bf16, 2^-11 for fp16,
half a step; A = sum_p w_p |v_p|; W the row's largest weight):
  output rounding                                   u |out|
  weights rounded to the type                       u A
  ... for fp16 their step is 2^-24 below 2^-14, with at least 2^11 for the
  largest weight: off by 2^-25 / 2^11               2^-36 W sum_p |v_p|
  logits: d products accumulated in fp32 (2^-23 each), the factor, exp2 and its
  argument (2^-22 each), on weights and on their total, E = |scale| sum |q k|
  at its largest                                    2 (d + 8) 2^-23 E A + 2^-16 A
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def _b():
    from gqa_kv_cache_append_gb300 import binding
    return binding


def peaked(lens, ns, h, g, d, dtype, share, sink, seed):
    B = _b()
    gen = torch.Generator("cuda").manual_seed(300 + seed)
    b, cap, total, r = len(lens), max(lens), sum(ns), h // g
    scale = 1 / math.sqrt(d)

    def rand(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    base = rand(g, d)
    k = 0.3 * rand(b, g, cap, d)
    v = (rand(1, g, 1, d) + 0.5 * rand(b, g, cap, d)).to(dtype)
    v[:, :, 0] *= sink
    for i, l in enumerate(lens):
        x = (k[i, :, 1:l] @ base[:, :, None])[..., 0] * scale
        want = torch.logsumexp(x.double(), -1) + math.log(share / (1 - share))
        k[i, :, 0] = base * (want / (scale * (base.double() ** 2).sum(-1)))[:, None].float()
    k = k.to(dtype)
    q = (base.repeat_interleave(r, 0) + 0.02 * rand(total, h, d)).to(dtype)
    out = torch.full((total, h, d), 5.0, dtype=dtype, device="cuda")
    cu = torch.tensor([sum(ns[:i]) for i in range(b + 1)], dtype=torch.int32, device="cuda")
    le = torch.tensor(lens, dtype=torch.int32, device="cuda")
    B.gqa_chunk_attn(q, k, v, cu, le, b, h, g, d, d, scale, out)
    assert B.gqa_device_status() == 0
    u = 2.0 ** (-8 if dtype == torch.bfloat16 else -11)
    for i, (l, n) in enumerate(zip(lens, ns)):
        kk, vv = k[i].double(), v[i].double()
        for s in sorted({0, n // 2, n - 1}):
            see = l - n + s + 1
            row = sum(ns[:i]) + s
            qq = q[row].double().view(g, r, d)
            w = torch.softmax(qq @ kk[:, :see].transpose(1, 2) * scale, -1)
            ref, A = w @ vv[:, :see], w @ vv[:, :see].abs()
            E = (qq.abs() @ kk[:, :see].abs().transpose(1, 2) * scale).amax(-1, keepdim=True)
            tol = (u * ref.abs() + u * A + 2 * (d + 8) * 2.0 ** -23 * E * A + 2.0 ** -16 * A)
            if dtype == torch.float16:
                tol += 2.0 ** -36 * w.amax(-1, keepdim=True) * vv[:, :see].abs().sum(1)[:, None]
            err = (out[row].double().view(g, r, d) - ref).abs()
            assert (err <= tol).all(), (i, s, float((err / tol).max()),
                                        float(err.norm() / ref.norm()))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("share,sink", [(0.9, 0.01), (0.999, 0.0001)])
@pytest.mark.parametrize("lens,ns,h,g,d", [
    ([131072], [1], 8, 1, 64),            # one sequence cut between all CTAs
    ([131072], [300], 8, 2, 128),
    ([30000] * 40, [1] * 40, 16, 4, 64),  # a unit or two to a CTA
    ([5000, 30000, 200], [5000, 70, 200], 8, 2, 64),
])
def test_dominant_first_position(lens, ns, h, g, d, share, sink, dtype):
    peaked(lens, ns, h, g, d, dtype, share, sink, len(lens))


def test_fp16_weights_rise_slowly():
    """Logits that grow with the position: the maximum is raised in every tile,
    and P stays inside fp16's range between raises."""
    B = _b()
    gen = torch.Generator("cuda").manual_seed(310)
    for step in (0.5, 3.9, 4.1, 9.0, 40.0):  # base 2, a tile of 128 positions
        L, h, d = 4000, 4, 64
        q = torch.zeros((1, h, d), dtype=torch.float16, device="cuda")
        q[..., 0] = 1
        k = torch.zeros((1, 1, L, d), dtype=torch.float16, device="cuda")
        k[..., 0] = torch.arange(L, device="cuda").div(128, rounding_mode="floor") * step
        v = torch.randn((1, 1, L, d), generator=gen, device="cuda").to(torch.float16)
        out = torch.zeros_like(q)
        cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
        le = torch.tensor([L], dtype=torch.int32, device="cuda")
        B.gqa_chunk_attn(q, k, v, cu, le, 1, h, 1, d, d, math.log(2), out)
        assert B.gqa_device_status() == 0
        x = k[0, 0, :, 0].double() * math.log(2)
        w = torch.softmax(x, -1)
        ref, A = w @ v[0, 0].double(), w @ v[0, 0].double().abs()
        E = float(x.max())
        tol = 2.0 ** -11 * (ref.abs() + A) + 2 * (d + 8) * 2.0 ** -23 * E * A + 2.0 ** -16 * A
        assert ((out[0].double() - ref).abs() <= tol).all(), step
