"""The calls of a serving loop together: a prompt in chunks (norm, rotation and
append, then attention over the cache), decode steps on the same cache with
the library's decode calls, and the same over the 8-bit cache, each against a
plain implementation in 64 bits of the whole layer; a step captured into a
graph and replayed while lengths move on; batches padded to a fixed size;
blocks shared between sequences.

Tolerance of an attention output: what its inputs' roundings to bf16 (q and k
after rotation, u = 2^-8 each) and to e4m3 (2^-4 of a value) do to a logit
is left out by computing the reference from the cached rows and rotated
queries themselves, which are compared on their own (tests of each call);
what remains is each attention's own bound (u of |out| and of the weighted
mean of |V| for the weights' rounding, 2^-12 for the rest at these sizes:
E = |scale| sum |q k| < 64 gives 2 * 136 * 2^-23 * 64 < 2^-8.9; with A below
4 here, 2^-6 covers it)."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


def _b():
    from gqa_kv_cache_append_gb300 import binding
    return binding


def attend(q, k, v, scale):
    """One query [h, d] over rows [g, L, d] in 64 bits: out, weighted mean |V|."""
    g = k.shape[0]
    q = q.double().view(g, -1, q.shape[-1])
    w = torch.softmax(q @ k.double().transpose(1, 2) * scale, -1)
    o, a = w @ v.double(), w @ v.double().abs()
    return o.flatten(0, 1), a.flatten(0, 1)


class Engine:
    """A layer's cache and weights, sequences of their own lengths."""

    def __init__(self, b=3, h=16, g=2, d=128, block=32, cap=512, seed=0):
        self.B = _b()
        gen = torch.Generator("cuda").manual_seed(seed)
        self.gen, self.b, self.h, self.g, self.d, self.block = gen, b, h, g, d, block
        mb = cap // block
        self.table = torch.randperm(b * mb + 1, generator=gen, device="cuda")[:b * mb].view(
            b, mb).to(torch.int32)
        bf = torch.bfloat16
        shape = (b * mb + 1, g, block, d)
        self.k, self.v = (torch.full(shape, float("nan"), dtype=bf, device="cuda")
                          for _ in range(2))
        self.k8, self.v8 = (torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda")
                            for _ in range(2))
        self.ks, self.vs = (torch.full(shape[:3], float("nan"), device="cuda") for _ in range(2))
        self.lens = torch.zeros(b, dtype=torch.int32, device="cuda")
        self.scale = 1 / math.sqrt(d)
        self.phase, self.rs = self.B.gqa_rope_table(d, 500000.0)
        self.w = [(1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(bf)
                  for _ in range(2)]

    def tokens(self, total):
        w = (self.h + 2 * self.g) * self.d
        qkv = torch.randn((total, w), generator=self.gen, device="cuda").to(torch.bfloat16)
        h, g, d = self.h, self.g, self.d
        return (qkv[:, :h * d].unflatten(1, (h, d)), qkv[:, h * d:(h + g) * d].unflatten(1, (g, d)),
                qkv[:, (h + g) * d:].unflatten(1, (g, d)))

    def append(self, q, k, v, cu, qo, fp8=False):
        a = (q, k, v, cu, self.lens, qo)
        rest = (self.table, self.b, self.h, self.g, self.d, self.d)
        kw = dict(rope=self.phase, rope_scale=self.rs, q_weight=self.w[0], k_weight=self.w[1])
        if fp8:
            self.B.gqa_rope_append_fp8_paged(*a, self.k8, self.v8, self.ks, self.vs, *rest, **kw)
        else:
            self.B.gqa_rope_append_paged(*a, self.k, self.v, *rest, **kw)

    def rows(self, pool, i, l, scale=None):
        t = self.table[i, :-(-l // self.block)].long()
        x = pool[t]
        if scale is not None:
            x = x.view(torch.float8_e4m3fn).double() * scale[t].double()[..., None]
        return x.transpose(0, 1).flatten(1, 2)[:, :l]

    def check(self, i, pos, q, out, fp8=False):
        if fp8:
            k, v = self.rows(self.k8, i, pos + 1, self.ks), self.rows(self.v8, i, pos + 1, self.vs)
        else:
            k, v = self.rows(self.k, i, pos + 1), self.rows(self.v, i, pos + 1)
        o, a = attend(q, k, v, self.scale)
        err = (out.double() - o).abs()
        assert (err <= U * o.abs() + U * a + 2.0 ** -6).all(), float(err.max())


def cu_of(ns):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)).cuda()


def test_prompt_in_chunks_then_decode():
    e = Engine()
    B = e.B
    done = [0, 0, 0]
    for ns in ([100, 1, 37], [150, 0, 64], [1, 20, 1]):
        for i, n in enumerate(ns):
            done[i] += n
        e.lens.copy_(torch.tensor(done, dtype=torch.int32))
        t = sum(ns)
        q, k, v = e.tokens(t + 5)  # (padded)
        cu = cu_of(ns)
        qo = torch.zeros((t + 5, e.h, e.d), dtype=torch.bfloat16, device="cuda")
        out = torch.full_like(qo, 9.0)
        e.append(q, k, v, cu, qo)
        B.gqa_chunk_attn_paged(qo, e.k, e.v, e.table, cu, e.lens, e.b, e.h, e.g, e.d, e.d,
                               e.scale, out)
        assert B.gqa_device_status() == 0
        assert (out[t:] == 9.0).all()
        at = 0
        for i, n in enumerate(ns):
            for s in sorted({0, n // 2, n - 1}) if n else []:
                e.check(i, done[i] - n + s, qo[at + s], out[at + s])
            at += n
    # decode steps with the decode kernel on the same cache, and the chunk
    # kernel beside it
    for _ in range(3):
        done = [x + 1 for x in done]
        e.lens += 1
        q, k, v = e.tokens(e.b)
        cu = cu_of([1] * e.b)
        qo = torch.zeros((e.b, e.h, e.d), dtype=torch.bfloat16, device="cuda")
        o1, o2 = torch.zeros_like(qo), torch.zeros_like(qo)
        e.append(q, k, v, cu, qo)
        B.gqa_decode_attn_paged(qo, e.k, e.v, e.table, e.lens, e.b, e.h, e.g, e.d, e.d, e.scale,
                                o1)
        B.gqa_chunk_attn_paged(qo, e.k, e.v, e.table, cu, e.lens, e.b, e.h, e.g, e.d, e.d,
                               e.scale, o2)
        assert B.gqa_device_status() == 0
        for i in range(e.b):
            e.check(i, done[i] - 1, qo[i], o1[i])
            e.check(i, done[i] - 1, qo[i], o2[i])


def test_eight_bit_cache_from_prompt_to_decode():
    e = Engine(seed=1)
    B = e.B
    ns = [200, 3, 65]
    e.lens.copy_(torch.tensor(ns, dtype=torch.int32))
    q, k, v = e.tokens(sum(ns))
    cu = cu_of(ns)
    qo = torch.zeros((sum(ns), e.h, e.d), dtype=torch.bfloat16, device="cuda")
    e.append(q, k, v, cu, qo, fp8=True)
    # the prompt attends over the rows read back
    kc, vc = (torch.zeros((e.b, e.g, 256, e.d), dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    B.gqa_kv_read_fp8_paged(e.k8, e.v8, e.ks, e.vs, e.table, e.lens, kc, vc, e.b, e.g, e.d, e.d)
    out = torch.zeros_like(qo)
    B.gqa_chunk_attn(qo, kc, vc, cu, e.lens, e.b, e.h, e.g, e.d, e.d, e.scale, out)
    assert B.gqa_device_status() == 0
    at = 0
    for i, n in enumerate(ns):
        o, a = attend(qo[at + n - 1], kc[i, :, :n], vc[i, :, :n], e.scale)
        assert ((out[at + n - 1].double() - o).abs() <= U * o.abs() + U * a + 2.0 ** -6).all()
        at += n
    for step in range(3):
        e.lens += 1
        q, k, v = e.tokens(e.b)
        qo = torch.zeros((e.b, e.h, e.d), dtype=torch.bfloat16, device="cuda")
        out = torch.zeros_like(qo)
        e.append(q, k, v, cu_of([1] * e.b), qo, fp8=True)
        B.gqa_decode_attn_fp8_paged(qo, e.k8, e.v8, e.ks, e.vs, e.table, e.lens, e.b, e.h, e.g,
                                    e.d, e.d, e.scale, out)
        assert B.gqa_device_status() == 0
        for i in range(e.b):
            e.check(i, ns[i] + step, qo[i], out[i], fp8=True)


def test_captured_step_while_lengths_move_on():
    """One graph of a whole step (append and attention, both caches), replayed
    with new tokens and lengths."""
    e = Engine(seed=2)
    B = e.B
    q, k, v = e.tokens(e.b)
    cu = cu_of([1] * e.b)
    qo = torch.zeros((e.b, e.h, e.d), dtype=torch.bfloat16, device="cuda")
    o16, o8 = torch.zeros_like(qo), torch.zeros_like(qo)

    def step():
        e.append(q, k, v, cu, qo)
        B.gqa_chunk_attn_paged(qo, e.k, e.v, e.table, cu, e.lens, e.b, e.h, e.g, e.d, e.d,
                               e.scale, o16)
        e.append(q, k, v, cu, qo, fp8=True)
        B.gqa_decode_attn_fp8_paged(qo, e.k8, e.v8, e.ks, e.vs, e.table, e.lens, e.b, e.h, e.g,
                                    e.d, e.d, e.scale, o8)

    e.lens.fill_(1)
    step()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        step()
    for n in range(1, 40):
        e.lens.fill_(n)
        for dst, src in zip((q, k, v), e.tokens(e.b)):
            dst.copy_(src)
        gr.replay()
    assert B.gqa_device_status() == 0
    for i in range(e.b):
        e.check(i, 38, qo[i], o16[i])
        e.check(i, 38, qo[i], o8[i], fp8=True)


def test_shared_blocks_and_repeated_calls():
    """Two sequences with a common prefix in the same blocks; the same call
    twice gives the same bits."""
    e = Engine(b=2, seed=3)
    B = e.B
    e.table[1, :2] = e.table[0, :2]
    e.lens.copy_(torch.tensor([64, 0], dtype=torch.int32))
    q, k, v = e.tokens(64)
    qo = torch.zeros((64, e.h, e.d), dtype=torch.bfloat16, device="cuda")
    e.append(q, k, v, cu_of([64, 0]), qo)
    e.append(q, k, v, cu_of([64, 0]), qo, fp8=True)
    ns = [5, 9]
    e.lens.copy_(torch.tensor([69, 73], dtype=torch.int32))
    q, k, v = e.tokens(14)
    qo = torch.zeros((14, e.h, e.d), dtype=torch.bfloat16, device="cuda")
    cu = cu_of(ns)
    outs = []
    for _ in range(2):
        e.append(q, k, v, cu, qo)
        out = torch.zeros_like(qo)
        B.gqa_chunk_attn_paged(qo, e.k, e.v, e.table, cu, e.lens, 2, e.h, e.g, e.d, e.d, e.scale,
                               out)
        outs.append(out)
    assert B.gqa_device_status() == 0
    assert torch.equal(outs[0], outs[1])
    for i, (at, n, l) in enumerate(((0, 5, 69), (5, 9, 73))):
        for s in range(n):
            e.check(i, l - n + s, qo[at + s], outs[0][at + s])
    # decode over the shared 8-bit blocks
    e.lens.fill_(64)
    q1 = qo[:2].clone()
    out = torch.zeros_like(q1)
    B.gqa_decode_attn_fp8_paged(q1, e.k8, e.v8, e.ks, e.vs, e.table, e.lens, 2, e.h, e.g, e.d,
                                e.d, e.scale, out)
    assert B.gqa_device_status() == 0
    for i in range(2):
        e.check(i, 63, q1[i], out[i], fp8=True)


def test_small_workspaces_and_other_devices_are_refused(monkeypatch):
    e = Engine(seed=4)
    B = e.B
    e.lens.fill_(3)
    q, k, v = e.tokens(6)
    cu = cu_of([2, 2, 2])
    qo = torch.zeros((6, e.h, e.d), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(qo)
    args = (qo, e.k, e.v, e.table, cu, e.lens, e.b, e.h, e.g, e.d, e.d, e.scale, out)
    n = B.gqa_chunk_attn_workspace(6, e.h, e.g, e.d, e.d)
    with pytest.raises(B.GqaError) as err:
        B.gqa_chunk_attn_paged(*args, workspace=torch.zeros(n - 1, dtype=torch.uint8,
                                                            device="cuda"))
    assert err.value.code == B.GQA_ERR_SCRATCH_LIMIT
    m = B.gqa_decode_attn_fp8_workspace(e.b, 1, e.h, e.g, e.d, e.d, 512)
    with pytest.raises(B.GqaError) as err:
        B.gqa_decode_attn_fp8_paged(qo[:3], e.k8, e.v8, e.ks, e.vs, e.table, e.lens, e.b, e.h,
                                    e.g, e.d, e.d, e.scale, out[:3],
                                    workspace=torch.zeros(m - 1, dtype=torch.uint8,
                                                          device="cuda"))
    assert err.value.code == B.GQA_ERR_SCRATCH_LIMIT
    # a current device that the tensors are not on
    monkeypatch.setattr(B.torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(B, "_raw_stream", lambda dev: 0)
    with pytest.raises(ValueError, match="the current device is cuda:1"):
        B.gqa_chunk_attn_paged(*args, workspace=torch.zeros(n, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="the current device is cuda:1"):
        e.append(q, k, v, cu, qo)


def test_unaligned_outputs():
    """16-byte aligned outputs that are not on a 32-byte sector."""
    e = Engine(seed=5)
    B = e.B
    ns = [40, 7, 130]
    e.lens.copy_(torch.tensor(ns, dtype=torch.int32))
    t = sum(ns)
    q, k, v = e.tokens(t)
    qo = torch.zeros((t, e.h, e.d), dtype=torch.bfloat16, device="cuda")
    e.append(q, k, v, cu_of(ns), qo)
    e.append(q, k, v, cu_of(ns), qo, fp8=True)
    outs = []
    for off in (0, 8):
        out = torch.zeros(t * e.h * e.d + 8, dtype=torch.bfloat16, device="cuda")[off:]
        out = out[:t * e.h * e.d].view(t, e.h, e.d)
        B.gqa_chunk_attn_paged(qo, e.k, e.v, e.table, cu_of(ns), e.lens, e.b, e.h, e.g, e.d, e.d,
                               e.scale, out)
        outs.append(out)
    assert torch.equal(outs[0], outs[1])
    backs = []
    for off in (0, 8):
        n = e.b * e.g * 160 * e.d
        kc, vc = (torch.zeros(n + 8, dtype=torch.bfloat16, device="cuda")[off:][:n].view(
            e.b, e.g, 160, e.d) for _ in range(2))
        B.gqa_kv_read_fp8_paged(e.k8, e.v8, e.ks, e.vs, e.table, e.lens, kc, vc, e.b, e.g, e.d,
                                e.d)
        backs.append((kc, vc))
    assert torch.equal(backs[0][0], backs[1][0]) and torch.equal(backs[0][1], backs[1][1])
    assert B.gqa_device_status() == 0


def test_legacy_default_stream():
    e = Engine(seed=6)
    B = e.B
    e.lens.fill_(50)
    q, k, v = e.tokens(150)
    cu = cu_of([50, 50, 50])
    qo = torch.zeros((150, e.h, e.d), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(qo)
    e.append(q, k, v, cu, qo)
    torch.cuda.synchronize()
    B.gqa_chunk_attn_paged(qo, e.k, e.v, e.table, cu, e.lens, e.b, e.h, e.g, e.d, e.d, e.scale,
                           out, stream=0)
    assert B.gqa_device_status(0) == 0
    for i in range(3):
        e.check(i, 49, qo[50 * i + 49], out[50 * i + 49])


def test_pools_past_32_bits():
    """Blocks that begin past 2^32 elements of their pool (2^33 bytes of the
    16-bit ones), beside blocks at its start."""
    e = Engine(seed=7)
    B, bf = e.B, torch.bfloat16
    nb = (1 << 32) // (e.g * e.block * e.d) + 100
    shape = (nb, e.g, e.block, e.d)
    e.k, e.v = (torch.empty(shape, dtype=bf, device="cuda") for _ in range(2))
    e.k8, e.v8 = (torch.empty(shape, dtype=torch.uint8, device="cuda") for _ in range(2))
    e.ks, e.vs = (torch.empty(shape[:3], device="cuda") for _ in range(2))
    e.table = torch.where(e.table % 3 == 0, e.table, nb - 1 - e.table).to(torch.int32)
    for pool, fill in ((e.k, float("nan")), (e.v, float("nan")), (e.k8, 0x7F), (e.v8, 0x7F),
                       (e.ks, float("nan")), (e.vs, float("nan"))):
        pool[:100] = fill
        pool[-100:] = fill
    ns = [500, 33, 270]
    e.lens.copy_(torch.tensor(ns, dtype=torch.int32))
    t = sum(ns)
    q, k, v = e.tokens(t)
    qo, out = (torch.zeros((t, e.h, e.d), dtype=bf, device="cuda") for _ in range(2))
    e.append(q, k, v, cu_of(ns), qo)
    e.append(q, k, v, cu_of(ns), qo, fp8=True)
    B.gqa_chunk_attn_paged(qo, e.k, e.v, e.table, cu_of(ns), e.lens, e.b, e.h, e.g, e.d, e.d,
                           e.scale, out)
    last = torch.stack([qo[sum(ns[:i + 1]) - 1] for i in range(3)])
    o8 = torch.zeros_like(last)
    B.gqa_decode_attn_fp8_paged(last, e.k8, e.v8, e.ks, e.vs, e.table, e.lens, e.b, e.h, e.g,
                                e.d, e.d, e.scale, o8)
    kc, vc = (torch.zeros((e.b, e.g, 512, e.d), dtype=bf, device="cuda") for _ in range(2))
    B.gqa_kv_read_fp8_paged(e.k8, e.v8, e.ks, e.vs, e.table, e.lens, kc, vc, e.b, e.g, e.d, e.d)
    assert B.gqa_device_status() == 0
    at = 0
    for i, n in enumerate(ns):
        assert torch.equal(e.rows(e.v, i, n).transpose(0, 1), v[at:at + n])
        for s in range(0, n, 61):
            e.check(i, s, qo[at + s], out[at + s])
        e.check(i, n - 1, qo[at + n - 1], out[at + n - 1])
        e.check(i, n - 1, last[i], o8[i], fp8=True)
        want = e.rows(e.v8, i, n, e.vs).float().to(bf)  # (the product in fp32, then bf16)
        assert torch.equal(vc[i, :, :n], want)
        at += n


def test_cache_past_32_bits():
    """A contiguous cache of more than 2^32 elements: a sequence of 33 million
    positions, whose heads each look for rows far apart, and one behind it."""
    B, bf = _b(), torch.bfloat16
    gen = torch.Generator("cuda").manual_seed(8)
    h, d, cap, ns = 8, 64, (1 << 25) + 40, [3, 5]
    ls = [cap, 200]
    k, v = (torch.randn((2, 1, cap, d), generator=gen, device="cuda", dtype=bf) for _ in range(2))
    cu, lens = cu_of(ns), torch.tensor(ls, dtype=torch.int32, device="cuda")
    q, kn, vn = (torch.randn((8, n, d), generator=gen, device="cuda", dtype=bf)
                 for n in (h, 1, 1))
    # (no outlier in length: |q| = 8: a query's logit with four times itself is 32)
    q = (q.float() * 8 / q.float().norm(dim=-1, keepdim=True)).to(bf)
    phase, factor = B.gqa_rope_table(d, 500000.0)
    qo, out = (torch.zeros_like(q) for _ in range(2))
    B.gqa_rope_append(q, kn, vn, cu, lens, qo, k, v, 2, h, 1, d, d, rope=phase,
                      rope_scale=factor)
    # the appended rows: the angle is the table's turns times the position
    for i, (at, n, l) in enumerate(((0, 3, ls[0]), (3, 5, ls[1]))):
        assert torch.equal(v[i, 0, l - n:l], vn[at:at + n, 0])
        for s in range(n):
            pos = l - n + s
            ang = torch.tensor([(int(f) % (1 << 64)) * pos % (1 << 64) / 2.0 ** 64 * 2 * math.pi
                                for f in phase.tolist()], dtype=torch.float64, device="cuda")
            x = kn[at + s, 0].double()
            a, c = x[:d // 2], x[d // 2:]
            want = torch.cat([a * ang.cos() - c * ang.sin(), c * ang.cos() + a * ang.sin()])
            err = 1e-6 * (a.abs() + c.abs()).repeat(2)
            got = k[i, 0, pos].double()
            assert ((got - want).abs() <= err + U * (want.abs() + err)).all()
    # a row for each head of the first sequence's last token, far apart
    for a in range(h):
        k[0, 0, a * (cap - 4) // (h - 1)] = 4 * qo[2, a]
    B.gqa_chunk_attn(qo, k, v, cu, lens, 2, h, 1, d, d, 0.125, out)
    assert B.gqa_device_status() == 0
    for at, i, pos in ((2, 0, cap - 1), (3, 1, 195), (7, 1, 199)):
        o, a = attend(qo[at], k[i, :, :pos + 1], v[i, :, :pos + 1], 0.125)
        err = (out[at].double() - o).abs()
        assert (err <= U * o.abs() + U * a + 2.0 ** -6).all(), float(err.max())
