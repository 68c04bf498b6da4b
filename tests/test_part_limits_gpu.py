"""The window and prefix calls with as many sequences as a call takes, 65,535, each
with one new token or none.  Tolerance: part_cases.py."""
import math

import pytest
import torch

from part_cases import binding

pytestmark = pytest.mark.gpu

B_MAX, D = 65535, 64


@pytest.mark.parametrize("form", ["window", "prefix", "prefix_shared"])
def test_most_sequences(form):
    B = binding()
    gen = torch.Generator("cuda").manual_seed(5)
    prefix = {"window": 0, "prefix": 3, "prefix_shared": 40}[form]
    cap = prefix + 9
    rand = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)
    k, v = rand(B_MAX, 1, cap, D), rand(B_MAX, 1, cap, D)
    n = (torch.rand(B_MAX, generator=gen, device="cuda") < 0.7).int()
    lens = (prefix + torch.randint(1, 9, (B_MAX,), generator=gen, device="cuda")).int()
    cu = torch.cat([torch.zeros(1, device="cuda"), n.cumsum(0)]).int()
    t = int(cu[-1])
    q, out = rand(t, 1, D), torch.full((t, 1, D), 5.0, dtype=torch.bfloat16, device="cuda")
    dims = (B_MAX, 1, 1, D, D, 1 / math.sqrt(D))
    p = torch.arange(cap, device="cuda")
    own = n.bool()
    last = lens[own, None] - 1
    seen = p <= last
    if form == "window":
        B.gqa_chunk_attn_window(q, k, v, cu, lens, *dims, 4, out, sinks=1)
        seen &= (p > last - 4) | (p < 1)
    else:
        ws = torch.empty(B.gqa_chunk_attn_prefix_workspace(B_MAX, t, 1, 1, D, D),
                         dtype=torch.uint8, device="cuda")
        B.gqa_chunk_attn_prefix(q, k, v, cu, lens, *dims, prefix, out, workspace=ws)
        assert int(ws[:32].view(torch.int32)[5]) == (t if form == "prefix_shared" else 0)
        k[1:, :, :prefix], v[1:, :, :prefix] = k[:1, :, :prefix].clone(), v[:1, :, :prefix].clone()
    assert B.gqa_device_status() == 0
    kk, vv, qq = k[own, 0].double(), v[own, 0].double(), q[:, 0].double()
    x = torch.einsum("td,tpd->tp", qq, kk) / math.sqrt(D)
    w = torch.softmax(x.masked_fill(~seen, -math.inf), -1)
    ref = torch.einsum("tp,tpd->td", w, vv)
    A = torch.einsum("tp,tpd->td", w, vv.abs())
    E = ((qq.abs()[:, None] * kk.abs()).sum(-1) / math.sqrt(D) * seen).amax(-1, keepdim=True)
    u = 2.0 ** -8
    tol = u * A + u * ref.abs() + 2 * D * 2.0 ** -23 * E * A + 2.0 ** -16 * A + 1e-7
    assert ((out[:, 0].double() - ref).abs() <= tol).all()
