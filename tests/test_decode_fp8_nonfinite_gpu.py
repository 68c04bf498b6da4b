"""gqa_decode_attn_fp8_paged with infinities and NaN among its inputs: the query
rows that the formula gives no finite value for are NaN, the others are what
they are without them, bit for bit."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _b():
    from gqa_kv_cache_append_gb300 import binding
    return binding


class Decode:
    def __init__(self, lens, h=16, g=2, d=128, n=1, block=32, seed=0):
        gen = torch.Generator("cuda").manual_seed(700 + seed)
        self.b, self.h, self.g, self.d, self.n, self.block = len(lens), h, g, d, n, block
        mb = -(-max(lens) // block)
        nb = self.b * mb
        self.table = torch.randperm(nb, generator=gen, device="cuda").view(-1, mb).to(torch.int32)
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.q = torch.randn((self.b, n, h, d), generator=gen, device="cuda").to(BF)
        self.k8, self.v8 = (torch.randn((nb, g, block, d), generator=gen, device="cuda").to(
            torch.float8_e4m3fn).view(torch.uint8) for _ in range(2))
        self.ks, self.vs = (0.5 + torch.rand((nb, g, block), generator=gen, device="cuda")
                            for _ in range(2))

    def run(self):
        B = _b()
        out = torch.full_like(self.q, 5.0)
        B.gqa_decode_attn_fp8_paged(self.q, self.k8, self.v8, self.ks, self.vs, self.table,
                                    self.lens, self.b, self.h, self.g, self.d, self.d,
                                    1 / math.sqrt(self.d), out, n=self.n)
        assert B.gqa_device_status() == 0
        return out

    def at(self, i, pos):  # block and row of a position
        return int(self.table[i, pos // self.block]), pos % self.block


# lengths whose units are whole on a CTA, and cut between many
@pytest.mark.parametrize("lens", [[200, 31, 256], [40000, 300]])
@pytest.mark.parametrize("n", [1, 3])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_query(lens, n, value):
    c = Decode(lens, n=n)
    ref = c.run()
    assert torch.isfinite(ref).all()
    rows = [(0, 0, 3), (0, n - 1, 9), (1, n - 1, 0)]
    for i, s, a in rows:
        c.q[i, s, a, 77] = value
    out = c.run()
    for i, s, a in rows:
        assert torch.isnan(out[i, s, a]).all()
        ref[i, s, a] = out[i, s, a] = 0
    assert torch.equal(out, ref)
