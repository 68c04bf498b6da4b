"""gqa_chunk_attn with infinities and NaN in rows that tokens see: those tokens'
outputs are not finite whether or not a unit's positions are cut between CTAs,
and the other heads and sequences keep their bits."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def _b():
    from gqa_kv_cache_append_gb300 import binding
    return binding


class Chunk:
    def __init__(self, lens, ns, h=16, g=2, d=128, dtype=torch.bfloat16, seed=0):
        gen = torch.Generator("cuda").manual_seed(800 + seed)
        self.lens, self.ns, self.h, self.g, self.d = lens, ns, h, g, d
        b, cap = len(lens), max(lens)
        self.q = torch.randn((sum(ns), h, d), generator=gen, device="cuda").to(dtype)
        self.k, self.v = (torch.randn((b, g, cap, d), generator=gen, device="cuda").to(dtype)
                          for _ in range(2))
        self.cu = torch.tensor([sum(ns[:i]) for i in range(b + 1)], dtype=torch.int32,
                               device="cuda")
        self.le = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def run(self):
        B = _b()
        out = torch.full_like(self.q, 5.0)
        B.gqa_chunk_attn(self.q, self.k, self.v, self.cu, self.le, len(self.lens), self.h, self.g,
                         self.d, self.d, 1 / math.sqrt(self.d), out)
        assert B.gqa_device_status() == 0
        return out


@pytest.mark.parametrize("lens,ns", [
    ([200, 100], [1, 1]),         # whole units
    ([40000, 300], [1, 1]),       # a unit of twins cut between many CTAs
    ([40000, 300], [3, 300]),
    ([30000, 9000], [300, 100]),  # two-sided units cut
])
@pytest.mark.parametrize("where", [0.0, 0.37, 0.99])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_nan_in_a_row_that_every_token_sees(lens, ns, where, which, dtype):
    c = Chunk(lens, ns, dtype=dtype)
    ref = c.run()
    assert torch.isfinite(ref).all()
    pos = int(where * (lens[0] - ns[0]))
    getattr(c, which)[0, 1, pos, 5] = math.nan
    out = c.run()
    heads = slice(c.h // 2, c.h)  # of KV head 1
    bad = out[:ns[0], heads] if which == "k" else out[:ns[0], heads, 5]
    assert torch.isnan(bad).all()
    if which == "k":
        out[:ns[0], heads] = ref[:ns[0], heads]
    else:
        out[:ns[0], heads, 5] = ref[:ns[0], heads, 5]
    assert torch.equal(out, ref)


@pytest.mark.parametrize("lens,ns", [([200, 100], [1, 1]), ([40000, 300], [2, 300])])
def test_query(lens, ns):
    c = Chunk(lens, ns, seed=1)
    ref = c.run()
    for value in (math.inf, -math.inf, math.nan):
        q = c.q.clone()
        c.q[0, 3, 9] = value
        out = c.run()
        c.q = q
        assert torch.isnan(out[0, 3]).all()
        out[0, 3] = ref[0, 3]
        assert torch.equal(out, ref)


def test_infinite_key_elements():
    """A key element of minus infinity beside positive query elements takes no
    weight, wherever the position lies."""
    c = Chunk([40000], [2], seed=2)
    c.q[..., 7] = c.q[..., 7].abs() + 1
    for pos in (0, 17000, 39997):
        k = c.k.clone()
        c.k[0, :, pos, 7] = -math.inf
        out = c.run()
        c.k = k
        q = c.q.double().view(2, c.g, -1, c.d).transpose(0, 1)
        x = q @ c.k[0].double().transpose(1, 2)[:, None] / math.sqrt(c.d)
        x[..., pos] = -math.inf
        x[:, 0, :, -1] = -math.inf
        w = torch.softmax(x, -1)
        v = c.v[0].double()[:, None]
        ref, A = w @ v, w @ v.abs()
        got = out.double().view(2, c.g, -1, c.d).transpose(0, 1)
        assert ((got - ref).abs() <= 2.0 ** -8 * (ref.abs() + A) + 2.0 ** -8 * A).all()
