"""Cases, plain forms and calls of attention over part of a cache and over a
prefix that a batch shares.

Three operators over the framework's caches:

window       causal attention of packed chunks of new tokens (prompts, chunks,
             single tokens) in which a token sees the last ``window`` positions
             up to its own and the first ``sinks`` ones;
fp8_window   the same for one or a few new tokens over the 8-bit paged cache;
prefix       causal attention of packed chunks whose sequences have their first
             ``prefix`` positions in common, held once (by sequence 0).

A case names its sizes; the sequences' lengths follow from its ``mix`` number.
Blocks of a paged cache that only hold positions outside the window are given
back, as an engine does: their table entries are -1.
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
        # a chat of four short sequences, one new token each, in a window
        # layer: latency counts
        dict(name="window_decode_small_b4", op="window", dtype="bf16", b=4, h=32, g=8, d_k=128,
             d_v=128, n_lo=1, n_hi=1, ctx_lo=200, ctx_hi=3000, window=512, sinks=4, block=16,
             mix=1),
        # a decode step of 64 long sequences, the window's blocks alone kept
        dict(name="window_decode_b64", op="window", dtype="bf16", b=64, h=64, g=8, d_k=128,
             d_v=128, n_lo=1, n_hi=1, ctx_lo=3000, ctx_hi=60000, window=4096, sinks=4, block=64,
             mix=2),
        # a whole prompt of 8192 tokens, contiguous cache
        dict(name="window_prompt_8192", op="window", dtype="bf16", b=1, h=64, g=8, d_k=128,
             d_v=128, n_lo=8192, n_hi=8192, ctx_lo=0, ctx_hi=0, window=2048, sinks=4, block=0,
             mix=3),
        # a serving engine's mixed batch: single tokens, chunks and prompts,
        # seven query heads to a KV head
        dict(name="window_mixed_b32", op="window", dtype="bf16", b=32, h=28, g=4, d_k=128,
             d_v=128, n_lo=1, n_hi=1500, ctx_lo=1, ctx_hi=16000, window=1000, sinks=16, block=32,
             mix=4),
        # packed documents of a small model, 64-wide heads, fp16, a short
        # window without sinks
        dict(name="window_packed_d64_f16", op="window", dtype="f16", b=20, h=8, g=1, d_k=64,
             d_v=64, n_lo=100, n_hi=3500, ctx_lo=0, ctx_hi=0, window=256, sinks=0, block=0,
             mix=5),
        # two sequences on the 8-bit cache: latency counts
        dict(name="fp8_window_small", op="fp8_window", dtype="bf16", b=2, h=32, g=8, d_k=128,
             d_v=128, n=1, ctx_lo=300, ctx_hi=2000, window=512, sinks=4, block=16, mix=6),
        # a decode step of 64 long sequences on the 8-bit cache
        dict(name="fp8_window_b64", op="fp8_window", dtype="bf16", b=64, h=64, g=8, d_k=128,
             d_v=128, n=1, ctx_lo=3000, ctx_hi=60000, window=4096, sinks=4, block=64, mix=7),
        # ragged lengths, two tokens a step, many sinks
        dict(name="fp8_window_ragged_n2", op="fp8_window", dtype="bf16", b=24, h=28, g=4, d_k=128,
             d_v=128, n=2, ctx_lo=512, ctx_hi=32766, window=2000, sinks=100, block=32, mix=8),
        # four answers being drawn from one short prompt: latency counts
        dict(name="prefix_small_b4", op="prefix", dtype="bf16", b=4, h=32, g=8, d_k=128, d_v=128,
             n_lo=1, n_hi=1, prefix=700, ctx_lo=5, ctx_hi=200, block=16, mix=9),
        # 64 conversations behind one long system prompt, a decode step
        dict(name="prefix_decode_b64", op="prefix", dtype="bf16", b=64, h=64, g=8, d_k=128,
             d_v=128, n_lo=1, n_hi=1, prefix=8192, ctx_lo=50, ctx_hi=2000, block=64, mix=10),
        # a search over continuations of a long document, four proposed tokens
        # each, contiguous caches, fp16, an odd prefix
        dict(name="prefix_spec_n4_f16", op="prefix", dtype="f16", b=16, h=28, g=4, d_k=128,
             d_v=128, n_lo=4, n_hi=4, prefix=20011, ctx_lo=10, ctx_hi=500, block=0, mix=11),
        # questions of a hundred to a few hundred tokens on the same document
        dict(name="prefix_chunks_b16", op="prefix", dtype="bf16", b=16, h=32, g=8, d_k=128,
             d_v=128, n_lo=50, n_hi=400, prefix=6000, ctx_lo=0, ctx_hi=0, block=32, mix=12),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["window", "window", "window", "fp8_window", "prefix", "prefix"])
    g = rng.choice([1, 2, 4, 8])
    r = rng.choice([1, 2, 4, 7, 8] if op == "fp8_window" else [1, 2, 3, 5, 7, 8, 16])
    while g * r > 64:
        r = rng.choice([1, 2, 4, 7, 8])
    types = ["bf16"] if op == "fp8_window" else ["bf16", "bf16", "f16"]
    d_k, d_v = rng.choice([(128, 128), (128, 128), (64, 64), (128, 64)])
    case = dict(op=op, dtype=rng.choice(types), h=g * r, g=g, d_k=d_k, d_v=d_v,
                mix=rng.randrange(100, 1 << 30))
    case["block"] = rng.choice([16, 32, 64, 128, 256] if op == "fp8_window" else
                               [0, 16, 32, 64, 128, 256])
    rows = 64 * 8 * 4096        # of the cache, as much as the largest listed decode step
    pairs = 64 * 8192 * 1900    # of a query row and a position
    if op == "prefix":
        case["b"] = _log_int(rng, 1, 128)
        case["prefix"] = _log_int(rng, 16, 32000)
        case["n_hi"] = rng.choice([1, 1, _log_int(rng, 1, max(1, 4096 // case["b"]))])
        case["ctx_hi"] = rng.choice([0, _log_int(rng, 10, 4000)])
    else:
        case["window"] = _log_int(rng, 16, 8192)
        case["sinks"] = rng.choice([0, 1, 4, _log_int(rng, 1, 300)])
        case["ctx_hi"] = _log_int(rng, 10, 60000)
        if op == "fp8_window":
            case["n"] = rng.choice([1, 1, 2, 4])
            while case["n"] * r > 32:
                case["n"] //= 2
            case["b"] = _log_int(rng, 1, 64)
        else:
            case["b"] = _log_int(rng, 1, 64)
            case["n_hi"] = rng.choice([1, _log_int(rng, 1, max(1, 8192 // case["b"]))])
            case["ctx_hi"] = rng.choice([0, case["ctx_hi"]])
            if case["block"] == 0 and case["ctx_hi"] > 4000:
                case["block"] = 16  # (contiguous caches of far positions are mostly unused)
    case["ctx_lo"] = case["ctx_hi"] // rng.choice([1, 3, 20])
    if op == "fp8_window":
        case["ctx_lo"] = max(1, case["ctx_lo"])
        n = case["n"]
    else:
        case["n_lo"] = max(1, case["n_hi"] // rng.choice([1, 4, 100]))
        n = case["n_hi"]
    # no more work than the largest listed cases
    while True:
        b, ctx = case["b"], case["ctx_hi"]
        if op == "prefix":
            seen, held = case["prefix"] + ctx + n, case["prefix"] + b * (ctx + n)
            if case["block"] == 0:
                held = b * (case["prefix"] + ctx + n)  # (reserved, if not read)
        else:
            seen = min(ctx + n, case["window"] + case["sinks"])
            held = b * min(ctx + n, n + case["window"] + case["sinks"])
            if case["block"] == 0:
                held = b * (ctx + n)
        if held * g <= rows and b * n * seen * g * r <= pairs:
            return case
        if op == "prefix" and case["prefix"] > 8000:
            case["prefix"] = case["prefix"] * 2 // 3
        elif "n_hi" in case and case["n_hi"] > 64:
            n = case["n_hi"] = case["n_hi"] * 2 // 3
            case["n_lo"] = min(case["n_lo"], n)
        else:
            case["b"] = max(1, b * 2 // 3)


def _lens(case):
    """New tokens n_i and lengths L_i (after the append, with the prefix)."""
    rng = random.Random(case["mix"])
    ns, ls = [], []
    for _ in range(case["b"]):
        n = case["n"] if "n" in case else _log_int(rng, case["n_lo"], case["n_hi"])
        ctx = _log_int(rng, case["ctx_lo"], case["ctx_hi"]) if case["ctx_lo"] > 0 else (
            rng.randint(0, case["ctx_hi"]))
        ns.append(n)
        ls.append(case.get("prefix", 0) + ctx + n)
    return ns, ls


def _seen(case, n, l):
    """First position of the window of the first of a sequence's n new tokens,
    and the sinks before it."""
    lo = max(0, l - n - case["window"] + 1)
    return lo, min(case["sinks"], lo)


def work(case):
    ns, ls = _lens(case)
    h, g, dk, dv = case["h"], case["g"], case["d_k"], case["d_v"]
    t, rows, pairs = sum(ns), case.get("prefix", 0), 0
    for n, l in zip(ns, ls):
        if case["op"] == "prefix":
            rows += l - case["prefix"]
            pairs += n * (l - n) + n * (n + 1) // 2
            continue
        lo, sinks = _seen(case, n, l)
        rows += l - lo + sinks
        w, s = case["window"], case["sinks"]
        for p in range(l - n, l):
            pairs += min(p + 1, w) + min(s, max(0, p + 1 - w))
    row = dk + dv + 8 if case["op"] == "fp8_window" else 2 * (dk + dv)
    return {"bytes": 2 * t * h * (dk + dv) + rows * g * row, "flops": 2 * (dk + dv) * h * pairs}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
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
        # the blocks that each sequence keeps, and the block of each
        mb, held, rows = -(-max(ls) // bs), 0, []
        for i, (n, l) in enumerate(zip(ns, ls)):
            used = -(-l // bs)
            row = [-1] * mb
            for m in range(used):
                if case["op"] == "prefix":
                    if i > 0 and (m + 1) * bs <= case["prefix"]:
                        row[m] = rows[0][m]
                        continue
                else:
                    lo, sinks = _seen(case, n, l)
                    if m * bs >= sinks and (m + 1) * bs <= lo:
                        continue
                row[m] = held
                held += 1
            rows.append(row)
        nb = held + 3
        perm = torch.randperm(nb, generator=gen, device=dev).to(torch.int32)
        table = torch.tensor(rows, dtype=torch.int32, device=dev)
        s["table"] = torch.where(table >= 0, perm[table.clamp(min=0).long()], table).contiguous()
        lead = (nb, g, bs)
    else:
        s["cap"] = max(ls)
        lead = (b, g, s["cap"])
    if case["op"] == "fp8_window":
        # rows as the append leaves them: the largest magnitude of a row at
        # the type's largest value, scales of rows of unit variance
        for name, d in (("k", dk), ("v", dv)):
            x = normal(*lead, d, dtype=torch.float32)
            sc = x.abs().amax(-1) / 448.0
            s[name + "_pool"] = (x / sc[..., None]).to(torch.float8_e4m3fn)
            s[name + "_scale"] = sc
            del x
        s["q"] = normal(b, case["n"], h, dk)
        s["out"] = torch.empty((b, case["n"], h, dv), dtype=ty, device=dev)
    else:
        s["k"], s["v"] = normal(*lead, dk), normal(*lead, dv)
        if case["op"] == "prefix" and bs and case["prefix"] % bs:
            # a block that the prefix ends in is each sequence's own copy
            m, rest = case["prefix"] // bs, case["prefix"] % bs
            at = s["table"][:, m].long()
            for x in (s["k"], s["v"]):
                x[at[1:], :, :rest] = x[at[:1], :, :rest]
        s["q"] = normal(t, h, dk)
        s["out"] = torch.empty((t, h, dv), dtype=ty, device=dev)
    if own:
        from gqa_kv_cache_append_gb300 import binding as B
        s["B"] = B
        if case["op"] == "fp8_window":
            n = B.gqa_decode_attn_fp8_workspace(b, case["n"], h, g, dk, dv,
                                                bs * s["table"].shape[1])
        elif case["op"] == "prefix":
            n = B.gqa_chunk_attn_prefix_workspace(b, t, h, g, dk, dv)
        else:
            n = B.gqa_chunk_attn_workspace(t, h, g, dk, dv)
        s["ws"] = torch.empty(n, dtype=torch.uint8, device=dev)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    c, B = s["case"], s["B"]
    a = (c["b"], c["h"], c["g"], c["d_k"], c["d_v"], s["scale"])
    if c["op"] == "fp8_window":
        B.gqa_decode_attn_fp8_window_paged(
            s["q"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["table"],
            s["seq_lens"], *a, c["window"], s["out"], sinks=c["sinks"], n=c["n"],
            workspace=s["ws"])
        return s["out"]
    if c["op"] == "window":
        a, kw = (*a, c["window"], s["out"]), dict(sinks=c["sinks"], workspace=s["ws"])
        call, paged = B.gqa_chunk_attn_window, B.gqa_chunk_attn_window_paged
    else:
        a, kw = (*a, c["prefix"], s["out"]), dict(workspace=s["ws"])
        call, paged = B.gqa_chunk_attn_prefix, B.gqa_chunk_attn_prefix_paged
    if c["block"]:
        paged(s["q"], s["k"], s["v"], s["table"], s["cu"], s["seq_lens"], *a, **kw)
    else:
        call(s["q"], s["k"], s["v"], s["cu"], s["seq_lens"], *a, **kw)
    return s["out"]


def _rows(s, name, i, p):
    """Rows at the positions p (a tensor) of sequence i, [g, len(p), d] in 32
    bits."""
    bs = s["case"]["block"]
    if not bs:
        return s[name][i][:, p].float()
    blk, row = s["table"][i].long()[p // bs], p % bs
    if s["case"]["op"] == "fp8_window":
        x = s[name + "_pool"].view(torch.uint8)[blk, :, row].view(torch.float8_e4m3fn).float()
        x = x * s[name + "_scale"][blk, :, row][..., None]
    else:
        x = s[name][blk, :, row].float()
    return x.transpose(0, 1)


def _attend(q, k, v, seen, scale):
    """Maximum, sum and unnormalised output of queries [g, m, d_k] over keys
    [g, l, d_k], seen [m, l]."""
    x = torch.matmul(q, k.transpose(1, 2)) * scale
    x = x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = (x - top).exp_()
    return top, x.sum(-1, keepdim=True), torch.matmul(x, v)


def _run_plain(s):
    return _plain_prefix(s) if s["case"]["op"] == "prefix" else _plain_window(s)


def _plain_window(s):
    c = s["case"]
    h, g, dk, dv, w = c["h"], c["g"], c["d_k"], c["d_v"], c["window"]
    r = h // g
    dev = s["q"].device
    q = s["q"].reshape(-1, h, dk)
    out = s["out"].view(-1, h, dv)
    at = 0
    for i, (n, l) in enumerate(zip(s["ns"], s["ls"])):
        step = max(64, w // 2)  # queries at a time, over the positions they see
        for t0 in range(0, n, step):
            t1 = min(n, t0 + step)
            first, last = l - n + t0, l - n + t1 - 1
            lo = max(0, first - w + 1)
            pos = torch.cat([torch.arange(min(c["sinks"], lo), device=dev),
                             torch.arange(lo, last + 1, device=dev)])
            mine = torch.arange(first, last + 1, device=dev)[:, None]
            seen = (pos <= mine) & ((pos > mine - w) | (pos < c["sinks"]))
            k, v = _rows(s, "k", i, pos), _rows(s, "v", i, pos)
            m = t1 - t0
            x = q[at + t0:at + t1].float().reshape(m, g, r, dk).permute(1, 2, 0, 3)
            _, total, o = _attend(x.reshape(g, r * m, dk), k, v, seen.repeat(r, 1), s["scale"])
            o = (o / total).view(g, r, m, dv).permute(2, 0, 1, 3).flatten(1, 2)
            out[at + t0:at + t1] = o.to(out.dtype)
        at += n
    return s["out"]


def _plain_prefix(s):
    c = s["case"]
    h, g, dk, dv, pre = c["h"], c["g"], c["d_k"], c["d_v"], c["prefix"]
    r = h // g
    dev = s["q"].device
    out, t = s["out"], s["q"].shape[0]
    x = s["q"].float().view(t, g, r, dk).permute(1, 0, 2, 3).reshape(g, t * r, dk)
    # the prefix for every query, then each sequence's own positions
    k, v = (_rows(s, name, 0, torch.arange(pre, device=dev)) for name in ("k", "v"))
    top, total, o = (torch.empty((g, t * r, d), device=dev) for d in (1, 1, dv))
    step = max(1, (1 << 28) // (g * pre))  # query rows at a time: scores of 1 GiB
    for m0 in range(0, t * r, step):
        m1 = min(t * r, m0 + step)
        every = torch.ones((1, 1), dtype=torch.bool, device=dev)
        top[:, m0:m1], total[:, m0:m1], o[:, m0:m1] = _attend(x[:, m0:m1], k, v, every, s["scale"])
    at = 0
    for i, (n, l) in enumerate(zip(s["ns"], s["ls"])):
        pos = torch.arange(pre, l, device=dev)
        k, v = _rows(s, "k", i, pos), _rows(s, "v", i, pos)
        mine = torch.arange(l - n, l, device=dev)[:, None]
        part = slice(at * r, (at + n) * r)
        top1, total1, o1 = _attend(x[:, part], k, v, (pos <= mine).repeat_interleave(r, 0),
                                   s["scale"])
        m = torch.maximum(top[:, part], top1)
        a, b = (top[:, part] - m).exp(), (top1 - m).exp()
        y = (o[:, part] * a + o1 * b) / (total[:, part] * a + total1 * b)
        out[at:at + n] = y.view(g, n, r, dv).permute(1, 0, 2, 3).reshape(n, h, dv).to(out.dtype)
        at += n
    return out


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    """A token and a KV head at a time where tokens are few, else blocks of 128
    tokens, over all positions that can be seen."""
    ns, ls = _lens(case)
    if work(case)["flops"] > 4e12:
        return None
    s = prepare(case, seed)
    g, r = case["g"], case["h"] // case["g"]
    bs, dev = case["block"], s["q"].device
    q = s["q"].reshape(-1, g, r, case["d_k"])
    res = torch.empty((q.shape[0], g, r, case["d_v"]), dtype=torch.float64, device=dev)

    def fetch(name, i, a, b):
        """Positions a .. b - 1 of sequence i, block after block: [b - a, g, d]."""
        if not bs:
            return s[name][i, :, a:b].double().transpose(0, 1)
        if b <= a:
            return torch.empty((0, g, case["d_" + name]), dtype=torch.float64, device=dev)
        ids = s["table"][i, a // bs:(b - 1) // bs + 1].long()
        if case["op"] == "fp8_window":
            x = s[name + "_pool"].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double()
            x = x * s[name + "_scale"][ids].double().unsqueeze(-1)
        else:
            x = s[name][ids].double()
        x = x.permute(0, 2, 1, 3).flatten(0, 1)
        return x[a % bs:a % bs + b - a]

    at = 0
    shared = None
    if case["op"] == "prefix":
        shared = [fetch(name, 0, 0, case["prefix"]) for name in ("k", "v")]
    for i, (n, l) in enumerate(zip(ns, ls)):
        for t0 in range(0, n, 128):
            t1 = min(n, t0 + 128)
            p0, p1 = l - n + t0, l - n + t1
            if shared is not None:
                first, head = case["prefix"], case["prefix"]
                k, v = (torch.cat([x, fetch(name, i, first, p1)]) for x, name in
                        zip(shared, ("k", "v")))
            else:
                first = max(0, p0 + 1 - case["window"])
                head = min(case["sinks"], first)
                k, v = (torch.cat([fetch(name, i, 0, head), fetch(name, i, first, p1)])
                        for name in ("k", "v"))
            where = list(range(head)) + list(range(first, p1))
            where = torch.tensor(where, device=dev)
            tok = torch.arange(p0, p1, device=dev).view(-1, 1)
            hidden = where > tok
            if shared is None:
                hidden |= (tok - where >= case["window"]) & (where >= case["sinks"])
            y = torch.einsum("tgrd,pgd->grtp", q[at + t0:at + t1].double(), k) * s["scale"]
            y = torch.softmax(y.masked_fill(hidden, -math.inf), -1)
            res[at + t0:at + t1] = torch.einsum("grtp,pgd->tgrd", y, v)
        at += n
    return res.view(s["out"].shape)
