"""Windows, sinks and prefixes past 32 bits: the C ABI takes 32-bit integers, and
what a caller's number means must not change on the way there."""
import pytest
import torch

MAX, MIN = 0x7FFFFFFF, -0x80000000


@pytest.fixture()
def sent(monkeypatch):
    """The arguments that the binding would hand to the library."""
    from gqa_kv_cache_append_gb300 import build
    build.build()
    from gqa_kv_cache_append_gb300 import binding as B
    calls = []
    monkeypatch.setattr(B, "_launch", lambda name, fn, *a: calls.append(a))
    return B, calls


def tensors():
    bf = torch.bfloat16
    q, out = (torch.zeros(2, 8, 128, dtype=bf) for _ in range(2))
    k, v = (torch.zeros(2, 2, 16, 128, dtype=bf) for _ in range(2))
    cu, lens = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    return q, out, k, v, cu, lens, torch.zeros(2, 4, dtype=torch.int32)


NUMBERS = [(1, 1), (MAX, MAX), (MAX + 1, MAX), ((1 << 32) + 5, MAX), (1 << 40, MAX),
           ((1 << 63) - 1, MAX), (-1, -1), (MIN - 1, MIN), (-(1 << 32) + 7, MIN)]


@pytest.mark.parametrize("given,got", NUMBERS)
def test_window_and_sinks(sent, given, got):
    B, calls = sent
    q, out, k, v, cu, lens, table = tensors()
    dims, ws = (2, 8, 2, 128, 128, 0.1), torch.zeros(1 << 20, dtype=torch.uint8)
    for window, sinks in ((given, 3), (9, given)):
        B.gqa_chunk_attn_window(q, k, v, cu, lens, *dims, window, out, sinks=sinks, workspace=ws)
        B.gqa_chunk_attn_window_paged(q, k, v, table, cu, lens, *dims, window, out, sinks=sinks,
                                      workspace=ws)
        k8, sc = torch.zeros(9, 2, 16, 128, dtype=torch.uint8), torch.zeros(9, 2, 16)
        B.gqa_decode_attn_fp8_window_paged(q, k8, k8, sc, sc, table, lens, *dims, window, out,
                                           sinks=sinks, workspace=ws)
        want = (got, 3) if window == given and sinks == 3 else (9, got)
        for a in calls:
            at = a.index(0.1)  # (the scale stands before them)
            assert a[at + 1:at + 3] == want
        calls.clear()


@pytest.mark.parametrize("given,got", NUMBERS)
def test_prefix(sent, given, got):
    B, calls = sent
    q, out, k, v, cu, lens, table = tensors()
    dims, ws = (2, 8, 2, 128, 128, 0.1), torch.zeros(1 << 20, dtype=torch.uint8)
    B.gqa_chunk_attn_prefix(q, k, v, cu, lens, *dims, given, out, workspace=ws)
    B.gqa_chunk_attn_prefix_paged(q, k, v, table, cu, lens, *dims, given, out, workspace=ws)
    assert len(calls) == 2
    for a in calls:
        assert a[a.index(0.1) + 1] == got
