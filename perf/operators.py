"""Cases, plain forms and calls of the serving operators beside the decode step.

Four operators over the same caches:

rope_append   per-head RMS norm of q and k, rotary positions and the append of
              k and v, for packed tokens of sequences of different lengths;
chunk_attn    causal attention of packed chunks of new tokens over the cache
              (a whole prompt is a chunk whose length is the sequence's);
fp8_cache     the append into an 8-bit cache (e4m3, one fp32 scale for each
              row of a KV head) and the read back into 16 bits;
fp8_decode    decode attention over the 8-bit cache.

A case names its sizes; the sequences' lengths follow from its ``mix`` number.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decode step's new tokens of 64 sequences, before the attention:
        # a call of a few microseconds that every layer makes
        dict(name="rope_decode_b64", op="rope_append", dtype="bf16", b=64, h=64, g=8, d_k=128,
             d_v=128, rot=128, layout="half", norm=True, scaling="none", theta=500000.0,
             n_lo=1, n_hi=1, ctx_lo=200, ctx_hi=4000, block=64, mix=1),
        # two prompts of 4096 tokens, contiguous caches, half of the head
        # rotated in interleaved pairs, no norm
        dict(name="rope_prompt_2x4096_f16", op="rope_append", dtype="f16", b=2, h=32, g=8,
             d_k=128, d_v=128, rot=64, layout="pairs", norm=False, scaling="none", theta=10000.0,
             n_lo=4096, n_hi=4096, ctx_lo=0, ctx_hi=0, block=0, mix=2),
        # ragged chunks far into long sequences, stretched positions
        dict(name="rope_ragged_long", op="rope_append", dtype="bf16", b=24, h=28, g=4, d_k=128,
             d_v=128, rot=128, layout="half", norm=True, scaling="wavelength", theta=500000.0,
             n_lo=17, n_hi=2000, ctx_lo=1000, ctx_hi=100000, block=16, mix=3),
        # four proposed tokens of each of 8 short sequences: latency counts
        dict(name="chunk_small_b8", op="chunk_attn", dtype="bf16", b=8, h=32, g=8, d_k=128,
             d_v=128, n_lo=4, n_hi=12, ctx_lo=100, ctx_hi=2000, block=16, mix=4),
        # a whole prompt of 8192 tokens
        dict(name="chunk_prompt_8192", op="chunk_attn", dtype="bf16", b=1, h=64, g=8, d_k=128,
             d_v=128, n_lo=8192, n_hi=8192, ctx_lo=0, ctx_hi=0, block=0, mix=5),
        # a serving engine's mixed batch: single tokens, chunks and prompts,
        # seven query heads to a KV head
        dict(name="chunk_mixed_b32", op="chunk_attn", dtype="bf16", b=32, h=28, g=4, d_k=128,
             d_v=128, n_lo=1, n_hi=1500, ctx_lo=1, ctx_hi=16000, block=64, mix=6),
        # packed short prompts of a small model, 64-wide heads, fp16
        dict(name="chunk_packed_d64_f16", op="chunk_attn", dtype="f16", b=48, h=8, g=1, d_k=64,
             d_v=64, n_lo=30, n_hi=1200, ctx_lo=0, ctx_hi=0, block=0, mix=7),
        # one decode step's write into the 8-bit cache and its read back for
        # an engine that continues on a 16-bit copy
        dict(name="fp8_write_read_b8", op="fp8_cache", dtype="bf16", b=8, h=32, g=8, d_k=128,
             d_v=128, rot=128, layout="half", norm=False, scaling="none", theta=10000.0,
             n_lo=1, n_hi=1, ctx_lo=500, ctx_hi=4000, block=16, mix=8),
        # chunks of prompts written and read back
        dict(name="fp8_write_read_prompt", op="fp8_cache", dtype="bf16", b=6, h=64, g=8, d_k=128,
             d_v=128, rot=128, layout="half", norm=True, scaling="yarn", theta=500000.0,
             n_lo=300, n_hi=2048, ctx_lo=100, ctx_hi=8000, block=64, mix=9),
        # two short sequences: latency counts
        dict(name="fp8_decode_small", op="fp8_decode", dtype="bf16", b=2, h=32, g=8, d_k=128,
             d_v=128, n=1, ctx_lo=300, ctx_hi=900, block=16, mix=10),
        # the batch of the benchmark's default workload on the 8-bit cache
        dict(name="fp8_decode_b32_8192", op="fp8_decode", dtype="bf16", b=32, h=64, g=8, d_k=128,
             d_v=128, n=1, ctx_lo=8191, ctx_hi=8191, block=64, mix=11),
        # ragged lengths up to 32768, two tokens a step
        dict(name="fp8_decode_ragged_n2", op="fp8_decode", dtype="bf16", b=24, h=28, g=4, d_k=128,
             d_v=128, n=2, ctx_lo=512, ctx_hi=32766, block=32, mix=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope_append", "chunk_attn", "chunk_attn", "fp8_cache", "fp8_decode"])
    g = rng.choice([1, 2, 4, 8])
    r = rng.choice([1, 2, 4, 7, 8] if op == "fp8_decode" else [1, 2, 3, 5, 7, 8, 16])
    while g * r > 64:
        r = rng.choice([1, 2, 4, 7, 8])
    types = ["bf16"] if op == "fp8_decode" else ["bf16", "bf16", "f16"]
    d_k, d_v = rng.choice([(128, 128), (128, 128), (64, 64), (128, 64)])
    case = dict(op=op, dtype=rng.choice(types), h=g * r, g=g, d_k=d_k, d_v=d_v,
                mix=rng.randrange(100, 1 << 30))
    if op in ("rope_append", "fp8_cache"):
        case["rot"] = rng.choice([d_k, d_k, d_k // 2, d_k // 4])
        case["layout"] = rng.choice(["half", "pairs"])
        case["norm"] = rng.random() < 0.5
        case["scaling"] = rng.choice(["none", "linear", "wavelength", "yarn"])
        case["theta"] = rng.choice([10000.0, 500000.0, 1000000.0])
    if op == "fp8_decode":
        case["n"] = rng.choice([1, 1, 2, 4])
        while case["n"] * r > 32:
            case["n"] //= 2
        rows = 32 * 8 * 8192
        case["ctx_hi"] = _log_int(rng, 200, 32000)
        case["ctx_lo"] = max(1, case["ctx_hi"] // rng.choice([1, 3, 20]))
        case["b"] = max(1, min(_log_int(rng, 1, 64), rows // (case["ctx_hi"] * g)))
        case["block"] = rng.choice([16, 32, 64, 128, 256])
        return case
    case["block"] = rng.choice([16, 32, 64, 128, 256] if op == "fp8_cache" else
                               [0, 16, 32, 64, 128, 256])
    if op == "chunk_attn":
        case["b"] = _log_int(rng, 1, 40)
        case["n_hi"] = _log_int(rng, 1, 8192 // case["b"])
        case["ctx_hi"] = rng.choice([0, _log_int(rng, 10, 20000)])
        # no more products than a prompt of 8192 tokens with 64 heads
        pairs = 64 * 8192 * 4096
        while case["b"] * case["n_hi"] * (case["ctx_hi"] + case["n_hi"]) * g * r > pairs:
            case["n_hi"] = max(1, case["n_hi"] // 2)
            case["ctx_hi"] //= 2
    else:
        tokens = 8192 if op == "rope_append" else 4096
        case["b"] = _log_int(rng, 1, 64)
        case["n_hi"] = _log_int(rng, 1, max(1, tokens // case["b"]))
        case["ctx_hi"] = rng.choice([0, _log_int(rng, 10, 32000)])
        rows = 6 * 8 * 8000
        while case["b"] * (case["n_hi"] + case["ctx_hi"]) * g > (rows if op == "fp8_cache" else
                                                                 8 * rows):
            case["ctx_hi"] //= 2
            case["b"] = max(1, case["b"] - 1)
    case["n_lo"] = max(1, case["n_hi"] // rng.choice([1, 4, 100]))
    case["ctx_lo"] = case["ctx_hi"] // rng.choice([1, 4, 100])
    if op == "rope_append" and case["block"] == 0 and case["ctx_hi"] > 4000:
        case["block"] = 16  # (contiguous caches of far positions would be mostly unused)
    return case


def _lens(case):
    """New tokens n_i and lengths L_i (after the append) of the case."""
    rng = random.Random(case["mix"])
    ns, ls = [], []
    for _ in range(case["b"]):
        n = case["n"] if "n" in case else _log_int(rng, case["n_lo"], case["n_hi"])
        ctx = _log_int(rng, case["ctx_lo"], case["ctx_hi"]) if case["ctx_lo"] > 0 else (
            rng.randint(0, case["ctx_hi"]))
        ns.append(n)
        ls.append(ctx + n)
    return ns, ls


def work(case):
    ns, ls = _lens(case)
    h, g, dk, dv = case["h"], case["g"], case["d_k"], case["d_v"]
    t = sum(ns)
    if case["op"] == "rope_append":
        # q, k, v read and written once
        return {"bytes": 2 * 2 * t * (h * dk + g * dk + g * dv), "flops": 6 * t * (h + g) * dk}
    if case["op"] == "fp8_cache":
        new = 2 * t * (2 * h * dk + g * (dk + dv)) + t * g * (dk + dv + 8)
        back = sum(ls) * g * (3 * (dk + dv) + 8)
        return {"bytes": new + back, "flops": 6 * t * (h + g) * dk + sum(ls) * g * (dk + dv)}
    pairs = sum(n * (l - n) + n * (n + 1) // 2 for n, l in zip(ns, ls))
    flops = 2 * (dk + dv) * h * pairs
    row = dk + dv + 8 if case["op"] == "fp8_decode" else 2 * (dk + dv)
    return {"bytes": 2 * t * h * (dk + dv) + sum(ls) * g * row, "flops": flops}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _rope_args(case):
    """Arguments of the position table for the case's scaling."""
    if case["scaling"] == "linear":
        return dict(scaling="linear", factor=4.0)
    if case["scaling"] == "wavelength":
        return dict(scaling="wavelength", factor=8.0, original_len=8192, low=1.0, high=4.0)
    if case["scaling"] == "yarn":
        return dict(scaling="yarn", factor=16.0, original_len=4096, low=1.0, high=32.0)
    return dict(scaling="none")


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(seed * 7919 + case["mix"])
    ty = _TYPES[case["dtype"]]
    b, h, g, dk, dv = (case[k] for k in ("b", "h", "g", "d_k", "d_v"))
    ns, ls = _lens(case)
    t = sum(ns)

    def normal(*shape, dtype=ty):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dtype)

    s = dict(case=case, ns=ns, ls=ls, scale=1.0 / math.sqrt(dk),
             seq_lens=torch.tensor(ls, dtype=torch.int32, device=dev))
    cu = [0]
    for n in ns:
        cu.append(cu[-1] + n)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    bs = case["block"]
    if bs:
        mb = -(-max(ls) // bs)
        used = [-(-l // bs) for l in ls]
        nb = sum(used) + 3
        perm = torch.randperm(nb, generator=gen, device=dev).to(torch.int32).tolist()
        rows, at = [], 0
        for u in used:
            rows.append(perm[at:at + u] + [0] * (mb - u))
            at += u
        s["table"] = torch.tensor(rows, dtype=torch.int32, device=dev)
        lead = (nb, g, bs)
    else:
        s["cap"] = max(ls)
        lead = (b, g, s["cap"])
    op = case["op"]
    if op in ("fp8_cache", "fp8_decode"):
        # rows as the append leaves them: the largest magnitude of a row at
        # the type's largest value, scales of rows of unit variance
        for name, d in (("k", dk), ("v", dv)):
            x = normal(*lead, d, dtype=torch.float32)
            sc = x.abs().amax(-1) / 448.0
            s[name + "_pool"] = (x / sc[..., None]).to(torch.float8_e4m3fn)
            s[name + "_scale"] = sc
            del x
    elif op == "chunk_attn":
        s["k"], s["v"] = normal(*lead, dk), normal(*lead, dv)
    else:
        s["k"] = torch.zeros((*lead, dk), dtype=ty, device=dev)
        s["v"] = torch.zeros((*lead, dv), dtype=ty, device=dev)
    if op == "chunk_attn":
        s["q"] = normal(t, h, dk)
        s["out"] = torch.empty((t, h, dv), dtype=ty, device=dev)
    elif op == "fp8_decode":
        s["q"] = normal(b, case["n"], h, dk)
        s["out"] = torch.empty((b, case["n"], h, dv), dtype=ty, device=dev)
    else:
        # the projection's output: q, k and v of a token side by side
        qkv = normal(t, h * dk + g * (dk + dv))
        s["q"] = qkv[:, :h * dk].unflatten(1, (h, dk))
        s["k_new"] = qkv[:, h * dk:(h + g) * dk].unflatten(1, (g, dk))
        s["v_new"] = qkv[:, (h + g) * dk:].unflatten(1, (g, dv))
        s["q_out"] = torch.empty((t, h, dk), dtype=ty, device=dev)
        if case["norm"]:
            s["q_weight"] = (1 + 0.2 * normal(dk, dtype=torch.float32)).to(ty)
            s["k_weight"] = (1 + 0.2 * normal(dk, dtype=torch.float32)).to(ty)
    if op == "fp8_cache":
        s["cap"] = max(ls)
        s["k_back"] = torch.zeros((b, g, s["cap"], dk), dtype=ty, device=dev)
        s["v_back"] = torch.zeros((b, g, s["cap"], dv), dtype=ty, device=dev)
    if own:
        from gqa_kv_cache_append_gb300 import binding as B
        s["B"] = B
        if "rot" in case:
            s["phase"], s["rope_scale"] = B.gqa_rope_table(case["rot"], theta=case["theta"],
                                                           device=dev, **_rope_args(case))
        if op == "chunk_attn":
            s["ws"] = torch.empty(B.gqa_chunk_attn_workspace(t, h, g, dk, dv), dtype=torch.uint8,
                                  device=dev)
        elif op == "fp8_decode":
            s["ws"] = torch.empty(
                B.gqa_decode_attn_fp8_workspace(b, case["n"], h, g, dk, dv,
                                                bs * s["table"].shape[1]),
                dtype=torch.uint8, device=dev)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    c, B = s["case"], s["B"]
    b, h, g, dk, dv = c["b"], c["h"], c["g"], c["d_k"], c["d_v"]
    if c["op"] == "chunk_attn":
        if c["block"]:
            B.gqa_chunk_attn_paged(s["q"], s["k"], s["v"], s["table"], s["cu"], s["seq_lens"], b,
                                   h, g, dk, dv, s["scale"], s["out"], workspace=s["ws"])
        else:
            B.gqa_chunk_attn(s["q"], s["k"], s["v"], s["cu"], s["seq_lens"], b, h, g, dk, dv,
                             s["scale"], s["out"], workspace=s["ws"])
        return s["out"]
    if c["op"] == "fp8_decode":
        B.gqa_decode_attn_fp8_paged(s["q"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"],
                                    s["table"], s["seq_lens"], b, h, g, dk, dv, s["scale"],
                                    s["out"], n=c["n"], workspace=s["ws"])
        return s["out"]
    rope = dict(rope=s["phase"], rope_scale=s["rope_scale"],
                layout=B.GQA_ROPE_HALF if c["layout"] == "half" else B.GQA_ROPE_PAIRS)
    if c["norm"]:
        rope.update(q_weight=s["q_weight"], k_weight=s["k_weight"], eps=1e-6)
    if c["op"] == "fp8_cache":
        B.gqa_rope_append_fp8_paged(s["q"], s["k_new"], s["v_new"], s["cu"], s["seq_lens"],
                                    s["q_out"], s["k_pool"], s["v_pool"], s["k_scale"],
                                    s["v_scale"], s["table"], b, h, g, dk, dv, **rope)
        B.gqa_kv_read_fp8_paged(s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["table"],
                                s["seq_lens"], s["k_back"], s["v_back"], b, g, dk, dv)
        return s["q_out"], s["k_back"], s["v_back"]
    if c["block"]:
        B.gqa_rope_append_paged(s["q"], s["k_new"], s["v_new"], s["cu"], s["seq_lens"],
                                s["q_out"], s["k"], s["v"], s["table"], b, h, g, dk, dv, **rope)
    else:
        B.gqa_rope_append(s["q"], s["k_new"], s["v_new"], s["cu"], s["seq_lens"], s["q_out"],
                          s["k"], s["v"], b, h, g, dk, dv, **rope)
    return s["q_out"], s["k"], s["v"]


def _frequencies(case, dev):
    """Angle per position of each pair of the rotated part (64 bits), and the
    factor on sine and cosine."""
    rot, theta = case["rot"], case["theta"]
    a = _rope_args(case)
    i = torch.arange(rot // 2, dtype=torch.float64, device=dev)
    f = theta ** (-2.0 * i / rot)
    if a["scaling"] == "linear":
        return f / a["factor"], 1.0
    if a["scaling"] == "wavelength":
        # pairs that turn less than `low` times over the original length are
        # stretched, those over `high` times kept, those between blended
        turns = a["original_len"] * f / (2 * math.pi)
        mix = ((turns - a["low"]) / (a["high"] - a["low"])).clamp(0.0, 1.0)
        return (1 - mix) * f / a["factor"] + mix * f, 1.0
    if a["scaling"] == "yarn":
        # a ramp over the pair index between the pairs of `high` and `low`
        # turns, and a factor on the logits' temperature
        def at(turns):
            return rot * math.log(a["original_len"] / (turns * 2 * math.pi)) / (
                2 * math.log(theta))
        lo, hi = max(math.floor(at(a["high"])), 0), min(math.ceil(at(a["low"])), rot - 1)
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
        return f * (1 - ramp) + f / a["factor"] * ramp, 0.1 * math.log(a["factor"]) + 1.0
    return f, 1.0


def _positions(s):
    ls, ns = s["ls"], s["ns"]
    dev = s["seq_lens"].device
    return torch.cat([torch.arange(l - n, l, device=dev) for n, l in zip(ns, ls)])


def _norm_rope(s, x, weight, cos, sin):
    """Norm and rotation of [T, heads, d] in 32 bits; cos, sin [T, 1, rot/2]."""
    c = s["case"]
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float()
    rot = c["rot"]
    if c["layout"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    ra, rb = a * cos - b * sin, b * cos + a * sin
    if c["layout"] == "half":
        y = torch.cat([ra, rb], -1)
    else:
        y = torch.stack([ra, rb], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _slots(s, i, lo, hi):
    """Block and row of positions lo .. hi - 1 of sequence i."""
    bs = s["case"]["block"]
    p = torch.arange(lo, hi, device=s["table"].device)
    return s["table"][i].long()[p // bs], p % bs


def _run_plain(s):
    c = s["case"]
    if c["op"] in ("chunk_attn", "fp8_decode"):
        return _plain_attention(s)
    f, factor = _frequencies(c, s["q"].device)
    angle = _positions(s).double()[:, None] * f
    cos = (angle.cos() * factor).float()[:, None]
    sin = (angle.sin() * factor).float()[:, None]
    q = _norm_rope(s, s["q"], s.get("q_weight"), cos, sin)
    k = _norm_rope(s, s["k_new"], s.get("k_weight"), cos, sin)
    s["q_out"].copy_(q)
    at = 0
    fp8 = c["op"] == "fp8_cache"
    for i, (n, l) in enumerate(zip(s["ns"], s["ls"])):
        for name, new in (("k", k), ("v", s["v_new"].float())):
            rows = new[at:at + n]  # [n, g, d]
            if fp8:
                scale = rows.abs().amax(-1) / 448.0
                blk, row = _slots(s, i, l - n, l)
                s[name + "_scale"][blk, :, row] = scale
                div = torch.where(scale > 0, scale, torch.ones_like(scale))
                q8 = (rows / div[..., None]).to(torch.float8_e4m3fn)
                s[name + "_pool"].view(torch.uint8)[blk, :, row] = q8.view(torch.uint8)
            elif c["block"]:
                blk, row = _slots(s, i, l - n, l)
                s[name][blk, :, row] = rows.to(s[name].dtype)
            else:
                s[name][i, :, l - n:l] = rows.transpose(0, 1).to(s[name].dtype)
        at += n
    if not fp8:
        return s["q_out"], s["k"], s["v"]
    for name in ("k", "v"):
        for i, l in enumerate(s["ls"]):
            s[name + "_back"][i, :, :l] = _rows8(s, name, i, l).to(s[name + "_back"].dtype)
    return s["q_out"], s["k_back"], s["v_back"]


def _rows8(s, name, i, l):
    """Rows 0 .. l - 1 of sequence i of an 8-bit pool, [g, l, d] in 32 bits."""
    nb = -(-l // s["case"]["block"])
    t = s["table"][i, :nb].long()
    x = s[name + "_pool"].view(torch.uint8)[t].view(torch.float8_e4m3fn).float()
    x = x * s[name + "_scale"][t][..., None]
    return x.transpose(0, 1).flatten(1, 2)[:, :l]


def _rows16(s, name, i, l):
    if s["case"]["block"]:
        nb = -(-l // s["case"]["block"])
        x = s[name][s["table"][i, :nb].long()].float()
        return x.transpose(0, 1).flatten(1, 2)[:, :l]
    return s[name][i, :, :l].float()


def _plain_attention(s):
    c = s["case"]
    h, g, dk, dv = c["h"], c["g"], c["d_k"], c["d_v"]
    r = h // g
    rows = _rows8 if c["op"] == "fp8_decode" else _rows16
    q = s["q"].reshape(-1, h, dk)
    out = s["out"].view(-1, h, dv)
    at = 0
    for i, (n, l) in enumerate(zip(s["ns"], s["ls"])):
        k, v = rows(s, "k", i, l), rows(s, "v", i, l)
        qi = q[at:at + n].float().reshape(n, g, r, dk).permute(1, 2, 0, 3)  # [g, r, n, d]
        step = max(1, (1 << 29) // (h * l))  # queries at a time: scores of 2 GiB
        for lo in range(0, n, step):
            hi = min(n, lo + step)
            x = torch.matmul(qi[:, :, lo:hi].reshape(g, -1, dk), k.transpose(1, 2)) * s["scale"]
            x = x.view(g, r, hi - lo, l)
            pos = torch.arange(l - n + lo, l - n + hi, device=q.device)
            seen = torch.arange(l, device=q.device)[None] <= pos[:, None]
            x = x.masked_fill_(~seen, -math.inf)
            x = (x - x.amax(-1, keepdim=True)).exp_()
            o = torch.matmul(x.view(g, -1, l), v) / x.sum(-1).view(g, -1, 1)
            out[at + lo:at + hi] = o.view(g, r, hi - lo, dv).permute(2, 0, 1, 3).flatten(
                1, 2).to(out.dtype)
        at += n
    return s["out"]


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("rope_append", "fp8_cache"):
        return _exact_rope(case, s)
    return _exact_attention(case, s)


def _exact_frequencies(case):
    rot, base, how = case["rot"], case["theta"], _rope_args(case)
    freqs, factor = [], 1.0
    if how["scaling"] == "yarn":
        factor = 1.0 + math.log(how["factor"]) / 10
        period = how["original_len"] / (2 * math.pi)
        # the pair index whose angle turns `high` (`low`) times
        first = max(0, math.floor(rot / 2 * math.log(period / how["high"], base)))
        last = min(rot - 1, math.ceil(rot / 2 * math.log(period / how["low"], base)))
    for i in range(rot // 2):
        f = math.exp(-2 * i / rot * math.log(base))
        if how["scaling"] == "linear":
            f = f / how["factor"]
        elif how["scaling"] == "wavelength":
            wave = 2 * math.pi / f
            if wave > how["original_len"] / how["low"]:
                f = f / how["factor"]
            elif wave >= how["original_len"] / how["high"]:
                m = (how["original_len"] / wave - how["low"]) / (how["high"] - how["low"])
                f = (1 - m) * f / how["factor"] + m * f
        elif how["scaling"] == "yarn":
            t = 0.0 if i <= first else 1.0 if i >= last else (i - first) / (last - first)
            f = f / how["factor"] * t + f * (1 - t)
        freqs.append(f)
    return freqs, factor


def _exact_rope(case, s):
    dev = s["q"].device
    d, rot, half = case["d_k"], case["rot"], case["rot"] // 2
    freq, factor = _exact_frequencies(case)
    freq = torch.tensor(freq, dtype=torch.float64, device=dev)
    pos = []
    for n, l in zip(s["ns"], s["ls"]):
        pos += range(l - n, l)
    # each pair as a complex number, turned by e^(i angle)
    angle = torch.tensor(pos, dtype=torch.float64, device=dev)[:, None] * freq
    turn = torch.polar(torch.full_like(angle, factor), angle)
    if case["layout"] == "half":
        first = list(range(half))
        second = list(range(half, rot))
    else:
        first = list(range(0, rot, 2))
        second = list(range(1, rot, 2))

    def rotate(x, w):
        y = x.double()
        if w is not None:
            y = y / (y.pow(2).sum(-1, keepdim=True) / d + 1e-6).sqrt() * w.double()
        z = torch.complex(y[..., first], y[..., second]) * turn[:, None]
        y = y.clone()
        y[..., first] = z.real
        y[..., second] = z.imag
        return y

    q = rotate(s["q"], s.get("q_weight"))
    new = {"k": rotate(s["k_new"], s.get("k_weight")), "v": s["v_new"].double()}
    if case["op"] == "rope_append":
        res = []
        for name in ("k", "v"):
            y = s[name].double()
            at = 0
            for i, (n, l) in enumerate(zip(s["ns"], s["ls"])):
                part = new[name][at:at + n]
                if case["block"]:
                    # one block of the table at a time
                    p = l - n
                    while p < l:
                        m = min(l - p, case["block"] - p % case["block"])
                        blk = int(s["table"][i, p // case["block"]])
                        r0 = p % case["block"]
                        y[blk, :, r0:r0 + m] = part[p - l + n:p - l + n + m].transpose(0, 1)
                        p += m
                else:
                    y[i, :, l - n:l] = part.transpose(0, 1)
                at += n
            res.append(y)
        return q, res[0], res[1]
    # the 8-bit cache: values of the rows that were there; the new rows'
    # have no value finer than the type's steps
    return q, None, None


def _exact_attention(case, s):
    g, r = case["g"], case["h"] // case["g"]
    dk, dv, bs = case["d_k"], case["d_v"], case["block"]
    pairs = sum(n * l for n, l in zip(s["ns"], s["ls"]))
    if pairs * case["h"] * (dk + dv) * 2 > 6e12:
        return None
    q = s["q"].reshape(-1, case["h"], dk)
    res = torch.empty((q.shape[0], case["h"], dv), dtype=torch.float64, device=q.device)
    at = 0
    for i, (n, l) in enumerate(zip(s["ns"], s["ls"])):
        for j in range(g):
            kv = []
            for name in ("k", "v"):
                if case["op"] == "fp8_decode":
                    ids = s["table"][i, :-(-l // bs)].long()
                    x = s[name + "_pool"][:, j].view(torch.uint8)[ids].view(torch.float8_e4m3fn)
                    x = x.double() * s[name + "_scale"][:, j][ids].double().unsqueeze(-1)
                    kv.append(x.flatten(0, 1)[:l])
                elif bs:
                    ids = s["table"][i, :-(-l // bs)].long()
                    kv.append(s[name][ids, j].double().flatten(0, 1)[:l])
                else:
                    kv.append(s[name][i, j, :l].double())
            step = max(1, (1 << 27) // l)
            for a in range(r):
                head = j * r + a
                for lo in range(0, n, step):
                    hi = min(n, lo + step)
                    x = q[at + lo:at + hi, head].double() @ kv[0].T * s["scale"]
                    # query row t sees l - n + lo + t + 1 positions
                    x = x + torch.full_like(x, -math.inf).triu(l - n + lo + 1)
                    res[at + lo:at + hi, head] = torch.softmax(x, -1) @ kv[1]
        at += n
    return res.view(s["out"].shape)
