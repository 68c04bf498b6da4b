"""Attention behind a shared prefix where entries of cu_tokens, lengths or blocks are
unusable: the other sequences' rows are as ever (tolerance: part_cases.py)."""
import pytest
import torch

from part_cases import Part, binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("block", [0, 16])
@pytest.mark.parametrize("prefix", [96, 2500])
@pytest.mark.parametrize("cu,rows", [
    ([0, 1, 3, -1], slice(0, 3)),  # the last sequence's end
    ([0, 1, 3, 16], slice(0, 3)),
    ([0, 9, 3, 6], slice(3, 6)),   # a middle one: the first two sequences are unusable
    ([0, -4, 3, 6], slice(3, 6)),
    ([7, 1, 3, 6], slice(1, 6)),   # the first one's start
])
def test_bad_tokens_take_their_own_sequences_alone(cu, rows, prefix, block):
    B = binding()
    c = Part([1, 2, 3], [prefix + 4, prefix + 64, prefix + 84], 8, 2, prefix=prefix, block=block)
    c.cu.copy_(torch.tensor(cu, dtype=torch.int32))
    c.run()
    c.check(status=B.GQA_DEV_BAD_TOKENS, rows=rows)
    skipped = torch.ones(6, dtype=torch.bool)
    skipped[rows] = False
    assert (c.out[skipped.cuda()] == 5.0).all()


@pytest.mark.parametrize("prefix", [96, 2500])
def test_a_bad_length_takes_its_own_sequence_alone(prefix):
    B = binding()
    c = Part([1, 2, 3], [prefix + 4, prefix + 64, prefix + 84], 8, 2, prefix=prefix, block=16)
    for bad in (prefix + 1, 1, c.table.shape[1] * 16 + 1):
        c.lens[1] = bad
        c.out.fill_(5.0)
        c.run()
        c.check(status=B.GQA_DEV_BAD_SEQ_LEN, rows=[0, 3, 4, 5])
        assert (c.out[1:3] == 5.0).all()


@pytest.mark.parametrize("prefix", [96, 2500])
def test_a_bad_block_takes_its_own_sequence_alone(prefix):
    B = binding()
    c = Part([1, 2, 3], [prefix + 4, prefix + 64, prefix + 84], 8, 2, prefix=prefix, block=16)
    c.table[1, (prefix + 40) // 16] = -1
    c.run()
    c.check(status=B.GQA_DEV_BAD_BLOCK, rows=[0, 3, 4, 5])


@pytest.mark.parametrize("block", [0, 64])
@pytest.mark.parametrize("prefix", [200, 2500])
@pytest.mark.parametrize("ns", [[1] * 6, [2, 0, 1, 3, 1], [9, 3, 17]])
def test_room_for_more_rows_changes_nothing(ns, prefix, block):
    """Bits depend on the tokens that are there, not on `total` (a captured step
    has room for more rows)."""
    c = Part(ns, [prefix + 40 * i + n for i, n in enumerate(ns)], 8, 2, prefix=prefix, block=block,
             pad=32 * len(ns) + 1)
    c.run()
    c.check()
    padded = c.out.clone()
    for total in (c.t, c.t + 3, 2 * len(ns) + 1):
        if total < c.t:
            continue
        c.out.fill_(5.0)
        c.run(total=total)
        c.check()
        assert torch.equal(c.out, padded)


@pytest.mark.parametrize("prefix", [200, 2500])
@pytest.mark.parametrize("ns", [[1, 1, 1], [20, 40, 30], [1], [33, 40]])
def test_room_for_more_sequences_changes_nothing(ns, prefix):
    """... nor on how many empty sequences a batch has."""
    more = ns + [0] * 61
    c = Part(more, [prefix + 70 * i + n for i, n in enumerate(ns)] + [0] * 61, 8, 2, prefix=prefix,
             block=16)
    c.run()
    c.check()
    many = c.out.clone()
    c.out.fill_(5.0)
    c.b = len(ns)
    c.run(workspace=torch.empty(binding().gqa_chunk_attn_prefix_workspace(
        c.b, c.total, c.h, c.g, c.dk, c.dv), dtype=torch.uint8, device="cuda"))
    c.check()
    assert torch.equal(c.out, many)
