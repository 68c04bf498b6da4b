"""Calls whose kernels this process has not run yet: inside a capture, once any
call has been made on the device, and from several threads at once."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SETUP = """
import math, threading
import torch
from gqa_kv_cache_append_gb300 import binding as B
gen = torch.Generator("cuda").manual_seed(0)
h, g, d, bs, lens = 16, 2, 128, 32, [300, 50, 700]
b, mb = len(lens), 22

class Case:
    def __init__(self, dtype):
        rand = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dtype)
        self.q, self.k, self.v = rand(sum(lens), h, d), rand(sum(lens), g, d), rand(sum(lens), g, d)
        self.cu = torch.tensor([0, 300, 350, 1050], dtype=torch.int32, device="cuda")
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.table = torch.randperm(b * mb, generator=gen, device="cuda").view(b, mb).to(torch.int32)
        self.k8, self.v8 = (torch.zeros((b * mb, g, bs, d), dtype=torch.uint8, device="cuda")
                            for _ in range(2))
        self.ks, self.vs = (torch.zeros((b * mb, g, bs), device="cuda") for _ in range(2))
        self.kc, self.vc = (torch.zeros((b, g, 704, d), dtype=dtype, device="cuda")
                            for _ in range(2))
        self.phase, self.f = B.gqa_rope_table(d)
        self.outs = [torch.zeros_like(self.q) for _ in range(2)] + [torch.zeros_like(self.q[:b])]
        self.fp8 = dtype == torch.bfloat16

    def run(self):
        qo, out, out8 = self.outs
        dims = (b, h, g, d, d)
        B.gqa_rope_append_fp8_paged(self.q, self.k, self.v, self.cu, self.lens, qo, self.k8,
                                    self.v8, self.ks, self.vs, self.table, *dims, rope=self.phase,
                                    rope_scale=self.f)
        B.gqa_kv_read_fp8_paged(self.k8, self.v8, self.ks, self.vs, self.table, self.lens, self.kc,
                                self.vc, b, g, d, d)
        B.gqa_chunk_attn(qo, self.kc, self.vc, self.cu, self.lens, *dims, 0.1, out)
        if self.fp8:
            B.gqa_decode_attn_fp8_paged(qo[:b], self.k8, self.v8, self.ks, self.vs, self.table,
                                        self.lens, *dims, 0.1, out8)
        return self.outs

def same(case, again):
    torch.cuda.synchronize()
    got = [x.clone() for x in case.outs]
    for x in case.outs:
        x.zero_()
    again()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got, case.outs))
    assert got[1].abs().sum() > 0 and B.gqa_device_status() == 0
"""

CAPTURED = SETUP + """
cases = [Case(torch.bfloat16), Case(torch.float16)]
B.gqa_kv_append(cases[0].k[:b], cases[0].v[:b], cases[0].kc, cases[0].vc, cases[0].lens, b, g, d, d)
torch.cuda.synchronize()
gr = torch.cuda.CUDAGraph()
with torch.cuda.graph(gr):
    for c in cases:
        c.run()
gr.replay()
for c in cases:
    same(c, c.run)
"""

THREADS = SETUP + """
cases = [Case(t) for t in (torch.bfloat16, torch.float16) * 4]
torch.cuda.synchronize()
errors = []
start = threading.Barrier(len(cases))

def work(c):
    try:
        with torch.cuda.stream(torch.cuda.Stream()):
            start.wait()
            for _ in range(20):
                c.run()
    except Exception as e:
        errors.append(e)

threads = [threading.Thread(target=work, args=(c,)) for c in cases]
for t in threads:
    t.start()
for t in threads:
    t.join()
assert not errors, errors
for c in cases:
    same(c, c.run)
"""


@pytest.mark.parametrize("code", [CAPTURED, THREADS], ids=["captured", "threads"])
def test_first_calls(code):
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
