"""The calls over a window and over a shared prefix as a serving loop uses them,
next to the rotation and append, and the caches they share: chunks, then single
tokens; blocks given back as the window moves on; a prefix written once."""
import math
import os
import subprocess
import sys

import pytest
import torch

from part_cases import binding

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U = 2.0 ** -8
H, G, D, BS = 16, 2, 128, 32


def attend(q, k, v, seen, scale):
    """64-bit attention of q [h, d] over k, v [g, l, d] at the positions seen, and
    the weighted mean of |v|."""
    k, v = k[:, seen].double(), v[:, seen].double()
    w = torch.softmax(q.double().view(k.shape[0], -1, D) @ k.transpose(1, 2) * scale, -1)
    return (w @ v).view(-1, D), (w @ v.abs()).view(-1, D)


def close(got, want, a, slack=1.0):
    # (rounding of weights and output, logits in fp32: part_cases.py; the 8-bit
    # cache's weights as two pieces are within the same rounding)
    return ((got.double() - want).abs() <= slack * (U * want.abs() + U * a) + 2.0 ** -9 * a).all()


class Engine:
    def __init__(self, b, blocks, seed=0, pool_blocks=None):
        self.gen = torch.Generator("cuda").manual_seed(70 + seed)
        self.b, self.scale = b, 1 / math.sqrt(D)
        bf = torch.bfloat16
        nb = pool_blocks or b * blocks
        self.k, self.v = (torch.full((nb, G, BS, D), float("nan"), dtype=bf, device="cuda")
                          for _ in range(2))
        self.k8, self.v8 = (torch.full((nb, G, BS, D), 0x7F, dtype=torch.uint8, device="cuda")
                            for _ in range(2))
        self.ks, self.vs = (torch.full((nb, G, BS), float("nan"), device="cuda") for _ in range(2))
        self.table = torch.randperm(b * blocks, generator=self.gen, device="cuda").view(
            b, blocks).to(torch.int32)
        self.lens = torch.zeros(b, dtype=torch.int32, device="cuda")
        self.phase, self.factor = binding().gqa_rope_table(D, 500000.0)
        # what the caches hold, by position: the reference's copy
        self.hist = [[torch.empty((G, 0, D), dtype=bf, device="cuda") for _ in range(2)]
                     for _ in range(b)]
        self.hist8 = [[torch.empty((G, 0, D), device="cuda") for _ in range(2)] for _ in range(b)]

    def append(self, ns):
        """New tokens of every sequence into both caches: (rotated queries, cu)."""
        B, t = binding(), sum(ns)
        q, k, v = (torch.randn((t, x, D), generator=self.gen, device="cuda").bfloat16()
                   for x in (H, G, G))
        cu = torch.tensor([sum(ns[:i]) for i in range(self.b + 1)], dtype=torch.int32,
                          device="cuda")
        self.lens += torch.tensor(ns, dtype=torch.int32, device="cuda")
        qo = torch.empty_like(q)
        rope = dict(rope=self.phase, rope_scale=self.factor)
        dims = (self.b, H, G, D, D)
        B.gqa_rope_append_paged(q, k, v, cu, self.lens, qo, self.k, self.v, self.table, *dims,
                                **rope)
        B.gqa_rope_append_fp8_paged(q, k, v, cu, self.lens, qo, self.k8, self.v8, self.ks, self.vs,
                                    self.table, *dims, **rope)
        lens = self.lens.tolist()
        for i, n in enumerate(ns):
            p = torch.arange(lens[i] - n, lens[i], device="cuda")
            t = self.table[i].long()[p // BS]
            for w, (pool, pool8, sc) in enumerate(((self.k, self.k8, self.ks),
                                                   (self.v, self.v8, self.vs))):
                rows = pool[t, :, p % BS].transpose(0, 1)
                self.hist[i][w] = torch.cat([self.hist[i][w], rows], 1)
                x = pool8[t, :, p % BS].view(torch.float8_e4m3fn).float()
                x = (x * sc[t, :, p % BS][..., None]).transpose(0, 1)
                self.hist8[i][w] = torch.cat([self.hist8[i][w], x], 1)
        return qo, cu

    def release(self, window, sinks):
        """Blocks that no later token sees: their rows overwritten, their entries
        pointing outside the pool."""
        for i, l in enumerate(self.lens.tolist()):
            for m in range(l // BS):
                if m * BS >= sinks and (m + 1) * BS <= l - window + 1 and self.table[i, m] >= 0:
                    blk = int(self.table[i, m])
                    for x in (self.k, self.v, self.ks, self.vs):
                        x[blk] = float("nan")
                    self.k8[blk] = self.v8[blk] = 0x7F
                    self.table[i, m] = -1

    def check(self, i, pos, q, out, window, sinks, fp8=False):
        k, v = (self.hist8 if fp8 else self.hist)[i]
        p = torch.arange(pos + 1, device="cuda")
        seen = (p > pos - window) | (p < sinks)
        want, a = attend(q, k[:, :pos + 1], v[:, :pos + 1], seen, self.scale)
        assert close(out, want, a, 1.5 if fp8 else 1.0), (i, pos, fp8)


def test_window_layer_chunks_then_tokens():
    B, window, sinks = binding(), 100, 5
    e = Engine(3, 40)
    dims = (3, H, G, D, D)
    for ns in ([300, 1, 64], [0, 200, 7], [33, 1, 1], *([[1, 1, 1]] * 6), [1, 0, 90], [1, 1, 1]):
        qo, cu = e.append(ns)
        out = torch.full_like(qo, 5.0)
        B.gqa_chunk_attn_window_paged(qo, e.k, e.v, e.table, cu, e.lens, *dims, e.scale, window,
                                      out, sinks=sinks)
        o8 = None
        if max(ns) == 1 and min(ns) == 1:  # a decode step, over the 8-bit cache too
            o8 = torch.full_like(qo, 5.0)
            B.gqa_decode_attn_fp8_window_paged(qo, e.k8, e.v8, e.ks, e.vs, e.table, e.lens, *dims,
                                               e.scale, window, o8, sinks=sinks)
        assert B.gqa_device_status() == 0
        at = 0
        for i, (n, l) in enumerate(zip(ns, e.lens.tolist())):
            for s in sorted({0, n // 3, n // 2, n - 1} if n else ()):
                e.check(i, l - n + s, qo[at + s], out[at + s], window, sinks)
                if o8 is not None:
                    e.check(i, l - n + s, qo[at + s], o8[at + s], window, sinks, fp8=True)
            at += n
        e.release(window, sinks)
    # lengths 341, 209, 169: blocks 1 .. 6, 1 .. 2 and 1 end at or before position
    # L - 99 (block 0 holds the sinks)
    assert e.lens.tolist() == [341, 209, 169] and (e.table == -1).sum() == 9


@pytest.mark.parametrize("prefix", [256, 300])
def test_prefix_written_once(prefix):
    """Sequence 0 brings the prompt; the others' tables begin with its blocks (a
    block that the prefix ends in is copied), then all continue."""
    B = binding()
    e = Engine(4, 24)
    dims = (4, H, G, D, D)
    everything = 1 << 30
    qo, cu = e.append([prefix, 0, 0, 0])
    out = torch.empty_like(qo)
    B.gqa_chunk_attn_paged(qo, e.k, e.v, e.table, cu, e.lens, *dims, e.scale, out)
    assert B.gqa_device_status() == 0
    whole, rest = prefix // BS, prefix % BS
    for i in range(1, 4):
        e.table[i, :whole] = -1  # (read through row 0)
        if rest:
            src, dst = int(e.table[0, whole]), int(e.table[i, whole])
            e.k[dst, :, :rest], e.v[dst, :, :rest] = e.k[src, :, :rest], e.v[src, :, :rest]
        e.hist[i] = [x.clone() for x in e.hist[0]]
        e.hist8[i] = [x.clone() for x in e.hist8[0]]
        e.lens[i] = prefix
    for ns in ([1, 1, 1, 1], [0, 3, 1, 2], [2, 100, 60, 1], [1, 1, 0, 1]):
        table = e.table.clone()
        qo, cu = e.append(ns)
        assert torch.equal(table, e.table)
        out = torch.full_like(qo, 5.0)
        B.gqa_chunk_attn_prefix_paged(qo, e.k, e.v, e.table, cu, e.lens, *dims, e.scale, prefix,
                                      out)
        assert B.gqa_device_status() == 0
        at = 0
        for i, (n, l) in enumerate(zip(ns, e.lens.tolist())):
            for s in sorted({0, n // 2, n - 1} if n else ()):
                e.check(i, l - n + s, qo[at + s], out[at + s], everything, 0)
            at += n


def test_pools_past_32_bits():
    """Blocks that begin past 2^32 elements of their pool beside blocks at its
    start."""
    B = binding()
    nb = (1 << 32) // (G * BS * D) + 100
    e = Engine(2, 24, seed=3, pool_blocks=100)
    bf = torch.bfloat16
    for name, dtype in (("k", bf), ("v", bf), ("k8", torch.uint8), ("v8", torch.uint8)):
        setattr(e, name, torch.empty((nb, G, BS, D), dtype=dtype, device="cuda"))
    e.ks, e.vs = (torch.empty((nb, G, BS), device="cuda") for _ in range(2))
    e.table = torch.where(e.table % 3 == 0, e.table, nb - 1 - e.table).to(torch.int32)
    dims = (2, H, G, D, D)
    for ns in ([500, 270], [1, 1]):
        qo, cu = e.append(ns)
        outs = [torch.full_like(qo, 5.0) for _ in range(3)]
        B.gqa_chunk_attn_window_paged(qo, e.k, e.v, e.table, cu, e.lens, *dims, e.scale, 150,
                                      outs[0], sinks=40)
        if ns[0] == 1:
            B.gqa_decode_attn_fp8_window_paged(qo, e.k8, e.v8, e.ks, e.vs, e.table, e.lens, *dims,
                                               e.scale, 150, outs[1], sinks=40)
            # (both see sequence 0's first 200 positions)
            B.gqa_chunk_attn_prefix_paged(qo, e.k, e.v, e.table, cu, e.lens, *dims, e.scale, 200,
                                          outs[2])
        assert B.gqa_device_status() == 0
        at = 0
        for i, (n, l) in enumerate(zip(ns, e.lens.tolist())):
            for s in (0, n // 2, n - 1):
                e.check(i, l - n + s, qo[at + s], outs[0][at + s], 150, 40)
            if n == 1:
                e.check(i, l - 1, qo[at], outs[1][at], 150, 40, fp8=True)
            at += n
    e.hist[1] = [torch.cat([x[:, :200], y[:, 200:]], 1) for x, y in zip(*e.hist)]
    for i, l in enumerate(e.lens.tolist()):
        e.check(i, l - 1, qo[i], outs[2][i], 1 << 30, 0)


FIRST = """
import sys, threading
sys.path.insert(0, "tests")
import torch
from part_cases import Part, binding
from test_decode_fp8_window_gpu import Case
B = binding()

def cases(seed):
    ns = [1, 3, 1]
    return [Part([40, 3], [300, 410], 8, 2, window=100, sinks=4, seed=seed),
            Part([40, 3], [300, 410], 8, 2, 64, 64, window=100, block=16, dtype="f16", seed=seed),
            Part(ns, [300 + n for n in ns], 8, 2, prefix=300, seed=seed),
            Part([100, 90], [400, 390], 8, 2, prefix=300, block=32, seed=seed),
            Case([300, 40], 8, 2, 90, 3, seed=seed)]
"""

CAPTURED = FIRST + """
cs = cases(1)
x = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda")
B.gqa_kv_append(x[0], x[0], x, x.clone(), torch.ones(1, dtype=torch.int32, device="cuda"), 1, 1,
                64, 64)  # (any call on the device comes before a capture)
torch.cuda.synchronize()
gr = torch.cuda.CUDAGraph()
with torch.cuda.graph(gr):
    for c in cs:
        c.run()
gr.replay()
torch.cuda.synchronize()
assert B.gqa_device_status() == 0
for c in cs:
    c.check()
"""

THREADS = FIRST + """
groups = [cases(s) for s in range(4)]
torch.cuda.synchronize()
errors, start = [], threading.Barrier(len(groups))

def work(cs):
    try:
        with torch.cuda.stream(torch.cuda.Stream()):
            start.wait()
            for _ in range(20):
                for c in cs:
                    c.run()
    except Exception as e:
        errors.append(e)

threads = [threading.Thread(target=work, args=(cs,)) for cs in groups]
for t in threads:
    t.start()
for t in threads:
    t.join()
assert not errors, errors
torch.cuda.synchronize()
assert B.gqa_device_status() == 0
for cs in groups:
    for c in cs:
        c.check()
"""


@pytest.mark.parametrize("code", [CAPTURED, THREADS], ids=["captured", "threads"])
def test_first_calls(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
