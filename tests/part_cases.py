"""Caches, calls and 64-bit references of the attention over a part of a cache
(window and sinks) and over a shared prefix.

Rows that no new token of their sequence sees hold NaN, and table entries of
blocks of such rows alone are not in the pool.

Tolerance, elementwise, with u = eps / 2 of the type (bf16 2^-8, fp16 2^-11)
and A = sum_p w_p |v_p| (from the reference):
  rounding of the softmax weights for P.V    u A
  rounding of the output                     u |out|
  logits: fp32 accumulation of d <= 128 products, each step off by at most
  2^-23 of the running sum, itself at most E = |scale| sum |q k|: the exponent
  is off by at most d 2^-23 E, and a weight and the weights' sum by a factor
  exp of that each                           2 d 2^-23 E A
  exp2 (2^-22), its argument (2^-23 of at most 64 + E), row sums, rescales and
  the factors of joined pieces in fp32       2^-16 A
"""
import math

import numpy as np
import torch

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def binding():
    from gqa_kv_cache_append_gb300 import binding as B
    return B


class Part:
    """Packed chunks over part of a cache: `window` and `sinks`, or `prefix`."""

    def __init__(self, ns, ls, h, g, dk=128, dv=128, window=None, sinks=0, prefix=None, block=0,
                 dtype="bf16", pad=0, scale=None, seed=0, slack=0, spread=1.0):
        gen = torch.Generator("cpu").manual_seed(4321 + seed)
        ty = TYPES[dtype]
        self.ns, self.ls, self.h, self.g, self.dk, self.dv = list(ns), list(ls), h, g, dk, dv
        self.window, self.sinks, self.prefix = window, sinks, prefix
        self.b, self.t, self.dtype, self.block = len(ns), sum(ns), dtype, block
        self.total = self.t + pad
        self.scale = 1.0 / math.sqrt(dk) if scale is None else scale
        self.cu = torch.from_numpy(np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)).cuda()
        self.lens = torch.tensor(ls, dtype=torch.int32).cuda()
        rand = lambda *s: torch.randn(s, generator=gen).to(ty)
        self.q = (spread * rand(self.total, h, dk)).to(ty).cuda()
        if pad:
            self.q[self.t:] = float("nan")
        cap = max(max(ls), prefix or 0, 1) + slack
        k, v = (torch.full((self.b, g, cap, d), float("nan"), dtype=ty) for d in (dk, dv))
        for i in range(self.b):
            live = torch.from_numpy(self.used(i))
            k[i, :, live] = rand(g, len(live), dk)
            v[i, :, live] = rand(g, len(live), dv)
        self.k, self.v, self.cap = k.cuda(), v.cuda(), cap
        if block:
            mb = -(-cap // block)
            kept = [sorted({int(p) // block for p in self.used(i)}) for i in range(self.b)]
            nb = sum(map(len, kept)) + 2
            perm = torch.randperm(nb, generator=gen).to(torch.int32)
            table = torch.full((self.b, mb), -7, dtype=torch.int32)  # unused: never read
            kp, vp = (torch.full((nb, g, block, d), float("nan"), dtype=ty) for d in (dk, dv))
            at = 0
            for i in range(self.b):
                for m in kept[i]:
                    blk = int(perm[at])
                    at += 1
                    table[i, m] = blk
                    n = min(block, cap - m * block)
                    kp[blk, :, :n] = k[i, :, m * block:m * block + n]
                    vp[blk, :, :n] = v[i, :, m * block:m * block + n]
            self.kp, self.vp, self.table = kp.cuda(), vp.cuda(), table.cuda()
        self.out = torch.full((self.total, h, dv), 5.0, dtype=ty).cuda()

    def used(self, i):
        """Positions of sequence i's own rows that are used."""
        n, l = self.ns[i], self.ls[i]
        p = np.arange(l)
        if self.prefix is not None:
            if i == 0:  # (the prefix; with n = 0 whatever the length)
                return np.arange(max(self.prefix, l if n else 0))
            return p[p >= self.prefix] if n else p[:0]
        if n == 0:
            return p[:0]
        return p[(p < self.sinks) | (p > l - n - self.window)]

    def run(self, **kw):
        B = binding()
        a = (self.b, self.h, self.g, self.dk, self.dv, self.scale)
        if self.prefix is not None:
            flat, paged, a = B.gqa_chunk_attn_prefix, B.gqa_chunk_attn_prefix_paged, a + (
                self.prefix, self.out)
        else:
            flat, paged, a = B.gqa_chunk_attn_window, B.gqa_chunk_attn_window_paged, a + (
                self.window, self.out)
            kw.setdefault("sinks", self.sinks)
        if self.block:
            paged(self.q, self.kp, self.vp, self.table, self.cu, self.lens, *a, **kw)
        else:
            flat(self.q, self.k, self.v, self.cu, self.lens, *a, **kw)
        return self.out

    def sees(self, p, pos):
        """[queries at pos, positions p]"""
        seen = p[None] <= pos[:, None]
        if self.prefix is None:
            seen &= (p[None] > pos[:, None] - self.window) | (p[None] < self.sinks)
        return seen

    def reference(self):
        """out, A and the largest E per row, in 64 bits."""
        r = self.h // self.g
        out = torch.zeros(self.t, self.h, self.dv, dtype=torch.float64, device="cuda")
        A, E = torch.zeros_like(out), torch.zeros(self.t, self.h, 1, dtype=torch.float64,
                                                  device="cuda")
        at = 0
        for i, (n, l) in enumerate(zip(self.ns, self.ls)):
            for lo in range(0, n, 512):
                hi = min(n, lo + 512)
                pos = torch.arange(l - n + lo, l - n + hi, device="cuda")
                if self.prefix is not None:
                    own = torch.arange(self.prefix, l - n + hi, device="cuda")
                    p = torch.cat([torch.arange(self.prefix, device="cuda"), own])
                    K, V = (torch.cat([x[0, :, :self.prefix], x[i][:, own]], 1).double()
                            for x in (self.k, self.v))
                else:
                    first = max(0, l - n + lo - self.window + 1)
                    p = torch.cat([torch.arange(min(self.sinks, first), device="cuda"),
                                   torch.arange(first, l - n + hi, device="cuda")])
                    K, V = self.k[i][:, p].double(), self.v[i][:, p].double()
                seen = self.sees(p, pos)
                for j in range(self.g):
                    for a in range(j * r, j * r + r):
                        q = self.q[at + lo:at + hi, a].double()
                        s = q @ K[j].T * self.scale
                        w = torch.softmax(s.masked_fill(~seen, -math.inf), -1)
                        out[at + lo:at + hi, a] = w @ V[j]
                        A[at + lo:at + hi, a] = w @ V[j].abs()
                        e = q.abs() @ K[j].abs().T * abs(self.scale)
                        E[at + lo:at + hi, a, 0] = (e * seen).amax(-1)
            at += n
        return out, A, E

    def check(self, status=0, rows=slice(None)):
        assert binding().gqa_device_status() == status
        ref, A, E = self.reference()
        u = U[self.dtype]
        tol = u * A + u * ref.abs() + 2 * self.dk * 2.0 ** -23 * E * A + 2.0 ** -16 * A + 1e-7
        err = (self.out[:self.t].double() - ref).abs()
        bad = ~(err <= tol)[rows]
        assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} off, first at "
                               f"{bad.nonzero()[0].tolist()}, worst {float(err[rows].max())}")
        if self.total > self.t:
            assert (self.out[self.t:] == 5.0).all()  # rows behind the last sequence
