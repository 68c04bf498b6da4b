"""The angles of gqa_rope_append by themselves: rows whose pairs are (1, 0) come
out as cosine and sine of the position's angles, from position 1 to the last
one below 2^31, however small the angle.

Tolerance: the angle over pi, exact to 2^-64 turns, is rounded to fp32 from two
halves, the upper one's rounding and the sum's (2^-24 of itself each),
sincospi is off by at most two units (2^-22), and the product with the factor
1 and the mate 0 adds nothing: 2^-23 |t| + 2^-22 |x|, with the table's own last
place, position * 2^-64 turns, beside it."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def _b():
    from gqa_kv_cache_append_gb300 import binding
    return binding


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("theta", [10000.0, 1e7])
def test_cosine_and_sine(layout, theta):
    B = _b()
    d, bs = 64, 65536
    pos = [1, 2, 3, 7, 100, 4095, 65537, 999983, (1 << 24) + 1, (1 << 30) + 12345,
           0x7FFFFF00 // bs * bs - 1]
    b, mb = len(pos), 0x7FFFFF00 // bs
    table = torch.arange(b, dtype=torch.int32, device="cuda")[:, None].repeat(1, mb)
    pools = [torch.zeros((b, 1, bs, d), device="cuda") for _ in range(2)]
    phase, factor = B.gqa_rope_table(d, theta)
    x = torch.zeros((b, 1, d), device="cuda")
    first = slice(0, d // 2) if layout == "half" else slice(0, d, 2)
    second = slice(d // 2, d) if layout == "half" else slice(1, d, 2)
    x[..., first] = 1
    lens = torch.tensor([p + 1 for p in pos], dtype=torch.int32, device="cuda")
    cu = torch.arange(b + 1, dtype=torch.int32, device="cuda")
    out = torch.zeros_like(x)
    B.gqa_rope_append_paged(x, x, x, cu, lens, out, *pools, table, b, 1, 1, d, d, rope=phase,
                            rope_scale=factor,
                            layout=B.GQA_ROPE_HALF if layout == "half" else B.GQA_ROPE_PAIRS)
    assert B.gqa_device_status() == 0
    for i, p in enumerate(pos):
        turns = [((int(f) * p + (1 << 63)) % (1 << 64)) - (1 << 63) for f in phase.tolist()]
        t = torch.tensor([v / 2.0 ** 64 * 2 * math.pi for v in turns], dtype=torch.float64,
                         device="cuda")
        key = pools[0][i, 0, p % bs].double()
        for got, want in ((out[i, 0, first].double(), t.cos()),
                          (out[i, 0, second].double(), t.sin()),
                          (key[first], t.cos()), (key[second], t.sin())):
            tol = 2.0 ** -23 * t.abs() + 2.0 ** -22 * want.abs() + p * 2.0 ** -64 * 2 * math.pi
            bad = (got - want).abs() > tol
            assert not bad.any(), (p, bad.nonzero().flatten().tolist(),
                                   float((got - want).abs().max()))
