"""Attention behind a shared prefix where entries of cu_tokens, lengths or blocks are
unusable: the other sequences' rows are as ever (tolerance: part_cases.py)."""
import pytest
import torch

from part_cases import Part, binding

pytestmark = pytest.mark.gpu


# heads: with 96 units three sequences of a few tokens share a prefix of 2,500
HEADS = [(8, 2), (64, 32)]


def shared_rows(c):
    """Rows that the prefix's own units held in a call (0: the prefix was not shared),
    from the first CTA's record in the workspace."""
    n = binding().gqa_chunk_attn_prefix_workspace(c.b, c.total, c.h, c.g, c.dk, c.dv)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    c.run(workspace=ws)
    return int(ws[:32].view(torch.int32)[5])


@pytest.mark.parametrize("h,g", HEADS)
@pytest.mark.parametrize("block", [0, 16])
@pytest.mark.parametrize("prefix", [96, 2500])
@pytest.mark.parametrize("cu,rows,end", [
    ([0, 1, 3, 4, -1], [0, 1, 2, 3], 4),    # the last sequence's end
    ([0, 1, 3, 4, 16], [0, 1, 2, 3], 4),
    ([0, 1, 9, 4, 6], [0, 4, 5], 6),        # middle ones: two sequences are unusable
    ([0, -4, 3, 4, 6], [3, 4, 5], 6),
    ([7, 1, 3, 4, 6], [1, 2, 3, 4, 5], 6),  # the first one's start
])
def test_bad_tokens_take_their_own_sequences_alone(cu, rows, end, prefix, block, h, g):
    B = binding()
    c = Part([1, 2, 1, 2], [prefix + x for x in (4, 64, 84, 20)], h, g, 64, 64, prefix=prefix,
             block=block)
    c.cu.copy_(torch.tensor(cu, dtype=torch.int32))
    assert shared_rows(c) == (end if g == 32 and prefix == 2500 else 0)
    c.check(status=B.GQA_DEV_BAD_TOKENS, rows=rows)
    skipped = torch.ones(6, dtype=torch.bool)
    skipped[rows] = False
    assert (c.out[skipped.cuda()] == 5.0).all()


@pytest.mark.parametrize("h,g", HEADS)
@pytest.mark.parametrize("prefix", [96, 2500])
def test_a_bad_length_takes_its_own_sequence_alone(prefix, h, g):
    B = binding()
    c = Part([1, 2, 3], [prefix + 4, prefix + 64, prefix + 84], h, g, 64, 64, prefix=prefix,
             block=16)
    for bad in (prefix + 1, 1, c.table.shape[1] * 16 + 1):
        c.lens[1] = bad
        c.out.fill_(5.0)
        c.run()
        c.check(status=B.GQA_DEV_BAD_SEQ_LEN, rows=[0, 3, 4, 5])
        assert (c.out[1:3] == 5.0).all()


@pytest.mark.parametrize("h,g", HEADS)
@pytest.mark.parametrize("prefix", [96, 2500])
def test_a_bad_block_takes_its_own_sequence_alone(prefix, h, g):
    B = binding()
    c = Part([1, 2, 3], [prefix + 4, prefix + 64, prefix + 84], h, g, 64, 64, prefix=prefix,
             block=16)
    c.table[1, (prefix + 40) // 16] = -1
    c.run()
    c.check(status=B.GQA_DEV_BAD_BLOCK, rows=[0, 3, 4, 5])


@pytest.mark.parametrize("h,g", HEADS)
@pytest.mark.parametrize("block", [0, 64])
@pytest.mark.parametrize("prefix", [200, 2500])
@pytest.mark.parametrize("ns", [[1] * 6, [2, 0, 1, 3, 1], [9, 3, 17], [30, 20, 12]])
def test_room_for_more_rows_changes_nothing(ns, prefix, block, h, g):
    """Bits depend on the tokens that are there, not on `total` (a captured step
    has room for more rows)."""
    c = Part(ns, [prefix + 40 * i + n for i, n in enumerate(ns)], h, g, 64, 64, prefix=prefix,
             block=block, pad=64 * len(ns) + 1)
    shared = shared_rows(c)
    assert shared == (c.t if prefix == 2500 and (g == 32 or c.t == 62) else 0)
    c.check()
    padded = c.out.clone()
    for total in (c.t, c.t + 3, 2 * len(ns) + 1):
        if total < c.t:
            continue
        c.out.fill_(5.0)
        c.run(total=total)
        c.check()
        assert torch.equal(c.out, padded)


@pytest.mark.parametrize("h,g", HEADS)
@pytest.mark.parametrize("prefix", [200, 2500])
@pytest.mark.parametrize("ns", [[1, 1, 1], [20, 16, 25], [1], [33, 30]])
def test_room_for_more_sequences_changes_nothing(ns, prefix, h, g):
    """... nor on how many empty sequences a batch has."""
    more = ns + [0] * 61
    c = Part(more, [prefix + 70 * i + n for i, n in enumerate(ns)] + [0] * 61, h, g, 64, 64,
             prefix=prefix, block=16)
    shared = shared_rows(c)
    if prefix == 2500 and len(ns) > 1:
        assert shared == (c.t if g == 32 or c.t in (61, 63) else 0)
    else:
        assert shared == 0
    c.check()
    many = c.out.clone()
    c.out.fill_(5.0)
    c.b = len(ns)
    c.run()
    c.check()
    assert torch.equal(c.out, many)


# ---------------------------------------------------------------------------
# the shared form, at sizes at which it is taken
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("ns,ctx", [
    ([1, 1], [0, 5]), ([1] * 5, [0, 1, 63, 300, 1000]), ([0, 1, 1, 0, 2], [9, 0, 40, 3, 7]),
    ([3, 1, 4], [130, 20, 0]), ([70, 1, 3], [5, 0, 40]), ([30, 25], [0, 400]),
])
@pytest.mark.parametrize("prefix", [2000, 2049, 3100])
@pytest.mark.parametrize("block", [0, 16, 512])
def test_shared_shapes(ns, ctx, prefix, block):
    c = Part(ns, [prefix + x + n for n, x in zip(ns, ctx)], 64, 32, 64, 64, prefix=prefix,
             block=block, slack=3, pad=5)
    assert shared_rows(c) == c.t
    c.check()


@pytest.mark.parametrize("ns", [[12, 13, 12], [30, 1, 40], [31, 0, 32], [90, 1, 2]])
@pytest.mark.parametrize("prefix,block", [(1024, 0), (1025, 128), (2500, 1024)])
def test_shared_by_few_units(ns, prefix, block):
    c = Part(ns, [prefix + 70 * i + n for i, n in enumerate(ns)], 8, 2, prefix=prefix, block=block)
    assert shared_rows(c) == (c.t if ns != [31, 0, 32] else 63)
    c.check()


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (128, 64), (64, 128)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("block", [0, 32])
@pytest.mark.parametrize("ns", [[1, 4, 2], [20, 1, 30]])
def test_shared_head_dims_and_types(dk, dv, dtype, block, ns):
    c = Part(ns, [2333 + n + 50 * i for i, n in enumerate(ns)], 96, 24, dk, dv, prefix=2333,
             block=block, dtype=dtype)
    assert shared_rows(c) == c.t
    c.check()


@pytest.mark.parametrize("h,g", [(32, 32), (96, 32), (224, 32), (284, 4), (256, 16), (512, 8),
                                 (640, 5)])
def test_shared_head_groups(h, g):
    b = -(-64 // g)
    ns = [1] * b
    c = Part(ns, [3277 + 1 + 31 * i for i in range(b)], h, g, 64, 64, prefix=3277, pad=4)
    want = c.t if h // g < 128 else 0  # (a token's rows fill a side)
    assert shared_rows(c) == (want if 128 // (h // g) > 1 else 0)
    c.check()


def test_rows_ahead_of_the_first_sequence():
    """cu_tokens need not begin at zero."""
    c = Part([3, 1, 2], [2507, 2540, 2560], 64, 32, 64, 64, prefix=2500, block=16)
    c.cu[0] = 1  # sequence 0 has two new tokens then, at the same positions
    assert shared_rows(c) == 6
    c.check(rows=slice(1, 6))
    assert (c.out[0] == 5.0).all()


def test_one_graph_takes_both_forms():
    """A captured call whose tokens change between replays: not shared, shared, not
    shared."""
    c = Part([90, 100, 80], [2700, 2650, 2600], 64, 32, 64, 64, prefix=2500, block=32)
    n = binding().gqa_chunk_attn_prefix_workspace(c.b, c.total, c.h, c.g, c.dk, c.dv)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    c.run(workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(workspace=ws)
    many = c.ns
    for ns in (many, [1, 2, 1], many, [0, 4, 30], [1, 0, 0]):
        c.ns, c.t = list(ns), sum(ns)
        c.cu.copy_(torch.tensor([0, ns[0], ns[0] + ns[1], sum(ns)], dtype=torch.int32))
        c.out.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        assert int(ws[:32].view(torch.int32)[5]) == (sum(ns) if 1 < sum(ns) < 40 else 0)
        c.check()
