"""gqa_rope_append with q_out = q, which the kernel then both reads and writes:
the bits of the call with an output of its own, for few tokens (rows dealt out
to many warps) and many (a warp to a token)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _b():
    from gqa_kv_cache_append_gb300 import binding
    return binding


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("total,h,d,rot", [(1, 64, 128, 128), (40, 64, 64, 32), (9, 33, 8, None),
                                           (6000, 16, 128, 64), (3000, 5, 256, 256)])
@pytest.mark.parametrize("norm", [False, True])
def test_same_bits(dtype, layout, total, h, d, rot, norm):
    B = _b()
    gen = torch.Generator("cuda").manual_seed(total)

    def rand(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(dtype)

    q, k, v = rand(total, h, d), rand(total, 1, d), rand(total, 1, d)
    cu = torch.tensor([0, total // 3, total], dtype=torch.int32, device="cuda")
    lens = torch.tensor([total, total + 5], dtype=torch.int32, device="cuda")
    kc, vc = (torch.zeros((2, 1, total + 8, d), dtype=dtype, device="cuda") for _ in range(2))
    kw = dict(layout=layout)
    if rot is not None:
        kw["rope"], kw["rope_scale"] = B.gqa_rope_table(rot)
    if norm:
        kw["q_weight"], kw["k_weight"] = rand(d), rand(d)
    out = torch.zeros_like(q)
    B.gqa_rope_append(q, k, v, cu, lens, out, kc, vc, 2, h, 1, d, d, **kw)
    for _ in range(3):
        own = q.clone()
        B.gqa_rope_append(own, k, v, cu, lens, own, kc, vc, 2, h, 1, d, d, **kw)
        assert torch.equal(own, out)
    assert B.gqa_device_status() == 0
