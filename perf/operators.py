"""Cases of the paged-cache operators: position rotation with append, windowed
attention, and the 4-bit cache.

`run` computes an operator in its plain form (elementary torch operations in
fp32, rounded once at the end), or, where `own` is true, through the package's
entry points.  `exact` computes it from the definition in float64.

The operators, with head_dim 128, 64-token pages and kv head h // G of query
head h (G = hq / hkv):
  append   rotate q and the new keys by their positions, store keys and values
           in BF16 pages;
  append4  the same into 4-bit pages, and the stored tokens read back as values;
  window   attention over BF16 pages, the query at position p seeing the tokens
           t <= p with t < sinks or t > p - window (window < 0: every t <= p);
  attend4  the same attention over 4-bit pages.
"""
import math

import numpy as np
import torch

own = False

PAGE, D = 64, 128
BLOCK = 512   # query rows whose scores the plain form holds at a time


# ---- cases -------------------------------------------------------------------
def listed():
    return [
        # One request's new token in a long chat: a launch and its latency.
        dict(name="append-step-1", op="append", hq=32, hkv=8, n=1, lo=100000, hi=100000, qlo=1, qhi=1, rotary=128,
             interleaved=False),
        # Chunked prefill of a ragged batch, 32K tokens in all.
        dict(name="append-prefill-32k", op="append", hq=32, hkv=8, n=7, lo=0, hi=30001, qlo=601, qhi=8761, rotary=128,
             interleaved=False),
        # A decode step of a batch into the 4-bit cache.
        dict(name="append4-step-32", op="append4", hq=32, hkv=8, n=32, lo=16384, hi=65000, qlo=1, qhi=1, rotary=128,
             interleaved=False, group=128),
        # Prefill of one 16K prompt into the 4-bit cache, two groups per head, partial interleaved rotation.
        dict(name="append4-prefill-16k", op="append4", hq=32, hkv=8, n=1, lo=37, hi=37, qlo=16347, qhi=16347, rotary=64,
             interleaved=True, group=64),
        # One request decoding with a short window: the smallest attention call.
        dict(name="window-decode-1", op="window", hq=32, hkv=8, n=1, lo=30001, hi=30001, qlo=1, qhi=1, window=256,
             sinks=64, out="f32"),
        # A decode batch of long requests with an 8K window.
        dict(name="window-decode-32", op="window", hq=32, hkv=8, n=32, lo=16384, hi=65536, qlo=1, qhi=1, window=8192,
             sinks=64, out="f32"),
        # One 100K request without a window.
        dict(name="window-decode-100k", op="window", hq=32, hkv=8, n=1, lo=100000, hi=100000, qlo=1, qhi=1, window=-1,
             sinks=0, out="f32"),
        # Ragged chunked prefill, GQA 8, a 1K window behind four sinks.
        dict(name="window-prefill-ragged", op="window", hq=64, hkv=8, n=6, lo=900, hi=9001, qlo=77, qhi=2601,
             window=1024, sinks=4, out="bf16"),
        # One 16K prompt, a 4K window.
        dict(name="window-prefill-16k", op="window", hq=32, hkv=8, n=1, lo=16384, hi=16384, qlo=16384, qhi=16384,
             window=4096, sinks=64, out="bf16"),
        # 4-bit decode of one 30K request.
        dict(name="attend4-30k", op="attend4", hq=32, hkv=8, n=1, lo=30000, hi=30000, qlo=1, qhi=1, window=-1, sinks=0,
             group=128, out="f32"),
        # 4-bit decode of one 100K request, two groups per head, GQA 8.
        dict(name="attend4-100k", op="attend4", hq=64, hkv=8, n=1, lo=100000, hi=100000, qlo=1, qhi=1, window=-1,
             sinks=0, group=64, out="f32"),
        # 4-bit decode of a batch of 16K to 64K requests.
        dict(name="attend4-32", op="attend4", hq=32, hkv=8, n=32, lo=16384, hi=65536, qlo=1, qhi=1, window=-1, sinks=0,
             group=128, out="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append4", "window", "window", "attend4"])
    hkv = rng.choice([2, 4, 8])
    c = dict(op=op, hq=hkv * rng.choice([1, 2, 4, 8]), hkv=hkv, n=_log(rng, 1, 32))
    if op in ("append", "append4"):
        c["lo"] = _log(rng, 1, 60000) - 1
        c["hi"] = c["lo"] + _log(rng, 1, 30000)
        c["qhi"] = _log(rng, 1, (32768 if op == "append" else 16384) // c["n"])
        c["qlo"] = rng.randint(1, c["qhi"])
        c["rotary"] = rng.choice([32, 64, 128, 128])
        c["interleaved"] = rng.random() < 0.3
        if op == "append4":
            c["group"] = rng.choice([64, 128])
        return c
    c["window"] = rng.choice([-1, _log(rng, 16, 16384), _log(rng, 16, 16384)])
    c["sinks"] = rng.choice([0, 4, rng.randint(1, 200)])
    c["out"] = "f32"
    prefill = op == "window" and rng.random() < 0.5
    budget = 600000
    if prefill:
        c["n"] = min(c["n"], 8)
        c["qhi"] = _log(rng, 17, 4096)
        c["qlo"] = rng.randint(1, c["qhi"])
        c["out"] = rng.choice(["bf16", "bf16", "f32"])
        budget = 32768
    elif op == "attend4":
        c["group"] = rng.choice([64, 128])
        c["qlo"] = c["qhi"] = rng.choice([1, 1, 2])
    else:
        c["qlo"] = c["qhi"] = rng.choice([1, 1, 1, 2])
    c["hi"] = max(c["qhi"], _log(rng, 64, max(65, min(100000, budget // c["n"]))))
    c["lo"] = rng.randint(min(c["hi"], max(c["qhi"], c["hi"] // 8)), c["hi"])
    return c


def _spread(lo, hi, n, step):
    """n lengths from lo to hi, the ends among them, off the round numbers between."""
    return [min(hi, lo + (hi - lo) * i // max(1, n - 1) + (step * i % 61 if 0 < i < n - 1 else 0)) for i in range(n)]


def _lengths(c):
    """Per request: the tokens that the cache holds (before an append, at an attention) and the new or query tokens."""
    base = _spread(c["lo"], c["hi"], c["n"], 37)
    new = _spread(c["qlo"], c["qhi"], c["n"], 23)
    return base, new if c["op"] in ("append", "append4") else [min(a, b) for a, b in zip(base, new)]


def _record(group):
    """Bytes of one 4-bit (page, kv head) record: K codes, V codes, K then V {scale, zero} in fp16."""
    return 2 * PAGE * (D // 2) + 2 * PAGE * 4 * (D // group)


def _visible(c, total, m):
    """(query, token) pairs and distinct tokens that the last m positions of a request see."""
    w = c["window"] if c["window"] >= 0 else total
    p = np.arange(total - m, total, dtype=np.int64)
    lo = np.maximum(0, p - w + 1)
    s = np.minimum(c["sinks"], p + 1)
    pairs = np.where(s >= lo, p + 1, s + p + 1 - lo)
    first, sink = int(lo[0]), min(c["sinks"], total)
    return int(pairs.sum()), total if sink >= first else sink + total - first


def work(case):
    c = case
    base, new = _lengths(c)
    rows = sum(new)
    if c["op"] == "append":
        return {"bytes": 2 * rows * (2 * (c["hq"] + 2 * c["hkv"]) * D) + 4 * rows * c["rotary"],
                "flops": 3 * rows * (c["hq"] + c["hkv"]) * c["rotary"]}
    if c["op"] == "append4":
        token = _record(c["group"]) // PAGE * c["hkv"]
        return {"bytes": rows * (2 * (2 * c["hq"] + 2 * c["hkv"]) * D + 2 * token + 4 * 2 * c["hkv"] * D)
                + 4 * rows * c["rotary"],
                "flops": rows * (3 * (c["hq"] + c["hkv"]) * c["rotary"] + 2 * c["hkv"] * D * 8)}
    pairs, tokens = 0, 0
    for t, m in zip(base, new):
        a, b = _visible(c, t, m)
        pairs, tokens = pairs + a, tokens + b
    token = c["hkv"] * (4 * D if c["op"] == "window" else _record(c["group"]) // PAGE)
    size = 4 if c["out"] == "f32" else 2
    return {"bytes": tokens * token + rows * c["hq"] * (D * (2 + size) + 4), "flops": 4 * D * c["hq"] * pairs}


# ---- inputs ------------------------------------------------------------------
def _rope_table(length, rotary):
    """fp32 [length][rotary]: cosines, then sines, of position * 10000^(-2 i / rotary); angles in float64."""
    inv = 10000.0 ** (-2.0 * torch.arange(rotary // 2, dtype=torch.float64, device="cuda") / rotary)
    a = torch.arange(length, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    base, new = _lengths(c)
    append = c["op"] in ("append", "append4")
    ends = [a + b for a, b in zip(base, new)] if append else base
    need = [-(-t // PAGE) for t in ends]
    s = {"case": dict(c), "lens": base, "new": new}
    # an append writes the last pages alone; the pages before them need no memory of their own
    first = [a // PAGE if append else 0 for a in base]
    held = [b - a for a, b in zip(first, need)]
    pages = sum(held) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(c["n"], max(need), dtype=torch.int32, device="cuda")
    at = 0
    for i, (f, h) in enumerate(zip(first, held)):
        table[i, f:f + h] = order[at:at + h]
        at += h
    s["table"] = table
    s["error"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    rows = sum(new)
    row_req = np.repeat(np.arange(c["n"]), new)
    start = np.concatenate([[0], np.cumsum(new)[:-1]])
    off = np.arange(rows) - start[row_req]
    pos0 = np.array(base) if append else np.array(base) - np.array(new)
    s["row_req"] = torch.from_numpy(row_req).cuda()
    s["row_pos"] = torch.from_numpy(pos0[row_req] + off).cuda()
    # per-channel spread with a few large key channels, as trained keys have
    spread = torch.exp(0.3 * rand(c["hkv"], D))
    spread[:, 5] *= 8
    if append:
        # q, k and v are the parts of one projection's output, rows of (hq + 2 hkv) heads
        qkv = rand(rows, c["hq"] + 2 * c["hkv"], D)
        qkv[:, c["hq"]:c["hq"] + c["hkv"]] *= spread
        qkv = qkv.to(torch.bfloat16)
        s["q"], s["k"], s["v"] = qkv.split([c["hq"], c["hkv"], c["hkv"]], 1)
        s["rope"] = _rope_table(max(ends), c["rotary"])
        s["q_out"] = torch.empty(rows, c["hq"], D, dtype=torch.bfloat16, device="cuda")
        if c["op"] == "append":
            s["kv"] = torch.zeros(pages, c["hkv"], 2, PAGE, D, dtype=torch.bfloat16, device="cuda")
        else:
            s["kv"] = torch.zeros(pages, c["hkv"], _record(c["group"]), dtype=torch.uint8, device="cuda")
            s["k_out"] = torch.empty(rows, c["hkv"], D, device="cuda")
            s["v_out"] = torch.empty(rows, c["hkv"], D, device="cuda")
        return s
    s["q"] = (rand(rows, c["hq"], D) * 0.8).to(torch.bfloat16)
    if c["op"] == "window":
        kv = torch.empty(pages, c["hkv"], 2, PAGE, D, dtype=torch.bfloat16, device="cuda")
        kv.normal_(generator=g)
        kv[:, :, 0] *= spread[:, None].to(torch.bfloat16)
        s["kv"] = kv
    else:
        ng = D // c["group"]
        kv = torch.randint(0, 256, (pages, c["hkv"], _record(c["group"])), dtype=torch.uint8, generator=g, device="cuda")
        meta = kv[:, :, 2 * PAGE * D // 2:].view(torch.float16).view(pages, c["hkv"], 2, PAGE, ng, 2)
        scale = 0.35 * torch.exp(0.3 * rand(pages, c["hkv"], 2, PAGE, ng))
        meta[..., 0] = scale.half()
        meta[..., 1] = (scale * (-7.5 + 0.8 * rand(*scale.shape))).half()
        s["kv"] = kv
    s["out"] = torch.empty(rows, c["hq"], D, dtype=torch.float32 if c["out"] == "f32" else torch.bfloat16, device="cuda")
    s["lse"] = torch.empty(rows, c["hq"], device="cuda")
    s["workspace"] = None
    return s


# ---- one pass ----------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    if op == "append":
        return _plain_append(state)
    if op == "append4":
        return _plain_append4(state)
    return _plain_attention(state, _read16 if op == "window" else _read4)


def _own(s, op):
    from bit_rotated_kv_decode_gb300 import binding
    c = s["case"]
    if op == "append":
        binding.bf16_append(s["kv"], s["table"], s["lens"], s["k"], s["v"], s["rope"], q=s["q"], q_out=s["q_out"],
                            new_lens=s["new"], interleaved=c["interleaved"], error=s["error"])
        return {"kv": s["kv"], "q": s["q_out"]}
    if op == "append4":
        binding.int4_append(s["kv"], s["table"], s["lens"], s["k"], s["v"], s["rope"], q=s["q"], q_out=s["q_out"],
                            new_lens=s["new"], interleaved=c["interleaved"], group_size=c["group"], error=s["error"])
        binding.int4_read(s["kv"], s["table"], s["lens"], s["new"], s["k_out"], s["v_out"], group_size=c["group"],
                          error=s["error"])
        return {"k": s["k_out"], "v": s["v_out"], "q": s["q_out"]}
    if op == "window":
        s["workspace"] = binding.window_attention(
            s["kv"], s["table"], s["lens"], s["q"], s["out"], c["hkv"], c["window"], c["sinks"], q_lens=s["new"],
            lse=s["lse"], workspace=s["workspace"], error=s["error"])
    else:
        s["workspace"] = binding.int4_attention(
            s["kv"], s["table"], s["lens"], s["q"], s["out"], c["hkv"], c["window"], c["sinks"], q_lens=s["new"],
            group_size=c["group"], lse=s["lse"], workspace=s["workspace"], error=s["error"])
    return {"out": s["out"], "lse": s["lse"]}


def _rotate(x, table, pos, interleaved):
    """bf16 [rows][heads][128] rotated by the table's rows, fp32, every product and difference rounded by itself."""
    x = x.float()
    r = table.shape[1]
    cos, sin = table[pos].unsqueeze(1).split(r // 2, -1)
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., r:]], -1)


def _plain_append(s):
    c, pos = s["case"], s["row_pos"]
    page, row = s["table"][s["row_req"], pos // PAGE], pos % PAGE
    s["kv"][page, :, 0, row] = _rotate(s["k"], s["rope"], pos, c["interleaved"]).to(torch.bfloat16)
    s["kv"][page, :, 1, row] = s["v"]
    return {"kv": s["kv"], "q": _rotate(s["q"], s["rope"], pos, c["interleaved"]).to(torch.bfloat16)}


def _quantise(x, group):
    """Codes 0 .. 15 and fp16 {scale, zero} of each group of a bf16 tensor's last axis."""
    x = x.float().unflatten(-1, (-1, group))
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    # a tensor as the divisor: dividing by a Python number multiplies by its reciprocal, which rounds otherwise
    zero, scale = lo.half(), ((hi - lo) / torch.full_like(lo, 15.0)).half()
    code = torch.round((x - zero.float()) / scale.float()).clamp(0, 15)
    code = torch.where(scale == 0, torch.zeros_like(code), code)
    return code.flatten(-2).to(torch.uint8), torch.cat([scale, zero], -1)


def _store4(kv, page, row, which, x, group):
    code, meta = _quantise(x, group)
    half = kv[..., :2 * PAGE * D // 2].view(kv.shape[0], kv.shape[1], 2, PAGE, D // 2)
    tail = kv[..., 2 * PAGE * D // 2:].view(torch.float16).view(kv.shape[0], kv.shape[1], 2, PAGE, D // group, 2)
    half[page, :, which, row] = code[..., 0::2] | (code[..., 1::2] << 4)
    tail[page, :, which, row] = meta


def _plain_append4(s):
    c, pos = s["case"], s["row_pos"]
    page, row = s["table"][s["row_req"], pos // PAGE], pos % PAGE
    _store4(s["kv"], page, row, 0, _rotate(s["k"], s["rope"], pos, c["interleaved"]).to(torch.bfloat16), c["group"])
    _store4(s["kv"], page, row, 1, s["v"], c["group"])
    q = _rotate(s["q"], s["rope"], pos, c["interleaved"]).to(torch.bfloat16)
    return {"k": _read4(s["kv"], page, row, 0, c), "v": _read4(s["kv"], page, row, 1, c), "q": q}


def _read16(kv, page, row, which, c):
    return kv[page, :, which, row].float()


def _read4(kv, page, row, which, c):
    half = kv[..., :2 * PAGE * D // 2].view(kv.shape[0], kv.shape[1], 2, PAGE, D // 2)
    tail = kv[..., 2 * PAGE * D // 2:].view(torch.float16).view(kv.shape[0], kv.shape[1], 2, PAGE, D // c["group"], 2)
    b, meta = half[page, :, which, row], tail[page, :, which, row].float()
    code = torch.stack([b & 15, b >> 4], -1).flatten(-2).unflatten(-1, (-1, c["group"])).float()
    return (code * meta[..., :1] + meta[..., 1:]).flatten(-2)


def _attend(read, kv, table, total, q, c):
    """Attention of the last m positions of n requests: q [n][m][hq][128] -> fp32 out, log-sum-exp."""
    n, m, hq, _ = q.shape
    g = hq // c["hkv"]
    longest, w = int(max(total)), c["window"]
    total = torch.tensor(total, device="cuda")[:, None]
    if w < 0:
        t = torch.arange(longest, device="cuda").expand(n, -1)
        sink = torch.ones_like(t, dtype=torch.bool)
    else:
        s = torch.arange(min(c["sinks"], longest), device="cuda").expand(n, -1)
        recent = total - m - w + 1 + torch.arange(w + m - 1, device="cuda")
        t = torch.cat([s, recent], 1)
        sink = torch.cat([torch.ones_like(s, dtype=torch.bool), torch.zeros_like(recent, dtype=torch.bool)], 1)
    p = total - m + torch.arange(m, device="cuda")
    near = t[:, None] > p[:, :, None] - (w if w >= 0 else longest + 1)
    # a sink inside the window is taken once, from the sinks' part of the list
    see = (t[:, None] <= p[:, :, None]) & torch.where(sink[:, None], True, near & (t[:, None] >= c["sinks"]))
    at = t.clamp(0, longest - 1)
    page, row = table.gather(1, at // PAGE), at % PAGE
    k = read(kv, page, row, 0, c).permute(0, 2, 3, 1)                                    # [n][hkv][128][tokens]
    x = q.float().unflatten(2, (c["hkv"], g)).permute(0, 2, 1, 3, 4).flatten(2, 3) / math.sqrt(D)
    a = torch.matmul(x, k).unflatten(2, (m, g))
    a = a.masked_fill(~see[:, None, :, None], -math.inf)
    top = a.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    a = torch.exp(a - top)
    total = a.sum(-1, keepdim=True)
    v = read(kv, page, row, 1, c).transpose(1, 2)                                        # [n][hkv][tokens][128]
    o = torch.matmul(a.flatten(2, 3), v).unflatten(2, (m, g))
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4).flatten(2, 3)
    return o, (total.log() + top).squeeze(-1).permute(0, 2, 1, 3).flatten(2, 3)


def _plain_attention(s, read):
    c, lens, new = s["case"], s["lens"], s["new"]
    kind = torch.float32 if c["out"] == "f32" else torch.bfloat16
    if max(new) * c["hq"] <= 2 * BLOCK and min(new) == max(new):   # a decode batch, padded to its longest request
        o, l = _attend(read, s["kv"], s["table"], lens, s["q"].unflatten(0, (c["n"], -1)), c)
        return {"out": o.flatten(0, 1).to(kind), "lse": l.flatten(0, 1)}
    out, lse, row = [], [], 0
    for i, (t, m) in enumerate(zip(lens, new)):
        for b in range(0, m, BLOCK):                               # blocks of queries, so that the scores fit
            e = min(m, b + BLOCK)
            o, l = _attend(read, s["kv"], s["table"][i:i + 1], [t - m + e], s["q"][None, row + b:row + e], c)
            out.append(o[0])
            lse.append(l[0])
        row += m
    return {"out": torch.cat(out).to(kind), "lse": torch.cat(lse)}


# ---- the definition in float64 -----------------------------------------------
def _turn(x, s, c):
    """The definition of the rotation, as a product of complex numbers."""
    r = s["rope"].shape[1]
    f = s["rope"].double()[s["row_pos"]][:, None]
    unit = torch.complex(f[..., :r // 2].contiguous(), f[..., r // 2:].contiguous())
    y = x.double().clone()
    if c["interleaved"]:
        z = torch.complex(y[..., 0:r:2].contiguous(), y[..., 1:r:2].contiguous()) * unit
        y[..., 0:r:2], y[..., 1:r:2] = z.real, z.imag
    else:
        z = torch.complex(y[..., :r // 2].contiguous(), y[..., r // 2:r].contiguous()) * unit
        y[..., :r // 2], y[..., r // 2:r] = z.real, z.imag
    return y


def _turn_stored(x, s, c):
    """The rotated key that the 4-bit cache quantises.  The operator defines it bit for bit, since a code hangs on it:
    each product, then each sum, rounded to fp32, and the result to bf16.  The products are exact in float64."""
    r = s["rope"].shape[1]
    f = s["rope"].double()[s["row_pos"]][:, None]
    cos, sin = f[..., :r // 2], f[..., r // 2:]
    y = x.double().clone()
    i = torch.arange(0, r, 2, device="cuda") if c["interleaved"] else torch.arange(r // 2, device="cuda")
    j = i + 1 if c["interleaved"] else i + r // 2
    a, b = y[..., i], y[..., j]
    once = lambda v: v.float().double()  # noqa: E731
    y[..., i], y[..., j] = once(once(a * cos) - once(b * sin)), once(once(b * cos) + once(a * sin))
    return y.to(torch.bfloat16).double()


def _levels(x, group):
    """The values that the 4-bit cache holds of x (bf16 values in float64)."""
    shape = x.shape
    x = x.reshape(-1, group)
    z = x.min(1, keepdim=True).values.half().double()
    d = ((x.max(1, keepdim=True).values - x.min(1, keepdim=True).values) / 15).half().double()
    code = torch.clamp(torch.round((x - z) / torch.where(d == 0, 1.0, d)), 0, 15)
    return (z + torch.where(d == 0, 0.0, d * code)).reshape(shape)


def _held(s, c, i, total):
    """Keys and values [total][hkv][128] of request i, float64, page by page."""
    p = s["table"][i, :-(-total // PAGE)].long()
    x = s["kv"][p]
    if c["op"] == "window":
        x = x.double().permute(2, 0, 3, 1, 4).reshape(2, -1, c["hkv"], D)
        return x[0, :total], x[1, :total]
    b = x[:, :, :PAGE * D].reshape(len(p), c["hkv"], 2, PAGE, D // 2).int()
    m = x[:, :, PAGE * D:].contiguous().view(torch.float16).double().reshape(len(p), c["hkv"], 2, PAGE, -1, 2)
    y = torch.empty(len(p), c["hkv"], 2, PAGE, D, dtype=torch.float64, device="cuda")
    y[..., 0::2], y[..., 1::2] = (b % 16).double(), (b // 16).double()
    group = c["group"]
    for k in range(D // group):
        y[..., k * group:(k + 1) * group] *= m[..., k, 0, None]
        y[..., k * group:(k + 1) * group] += m[..., k, 1, None]
    y = y.permute(2, 0, 3, 1, 4).reshape(2, -1, c["hkv"], D)
    return y[0, :total], y[1, :total]


def exact(case, seed):
    c = case
    if work(c)["flops"] > 1.5e12:
        return None   # float64 products of this size take too long
    s = prepare(c, seed)
    if c["op"] in ("append", "append4"):
        q = _turn(s["q"], s, c)
        if c["op"] == "append4":
            return {"k": _levels(_turn_stored(s["k"], s, c), c["group"]), "v": _levels(s["v"].double(), c["group"]),
                    "q": q}
        k = _turn(s["k"], s, c)
        kv = s["kv"].double()
        slot = s["table"][s["row_req"], s["row_pos"] // PAGE].long() * PAGE + s["row_pos"] % PAGE
        flat = kv.permute(0, 3, 2, 1, 4).reshape(-1, 2, c["hkv"], D)
        flat[slot] = torch.stack([k, s["v"].double()], 1)
        return {"kv": flat.reshape(kv.shape[0], PAGE, 2, c["hkv"], D).permute(0, 3, 2, 1, 4).contiguous(), "q": q}
    g = c["hq"] // c["hkv"]
    outs, lses, row = [], [], 0
    for i, (t, m) in enumerate(zip(s["lens"], s["new"])):
        k, v = _held(s, c, i, t)
        for b in range(0, m, 256):
            e = min(m, b + 256)
            p = torch.arange(t - m + b, t - m + e, device="cuda")
            lo = 0 if c["window"] < 0 else max(0, t - m + b - c["window"] + 1)
            at = torch.arange(t - m + e, device="cuda")
            at = at[(at >= lo) | (at < c["sinks"])]
            gone = at[None] > p[:, None]
            if c["window"] >= 0:
                gone |= (at[None] <= p[:, None] - c["window"]) & (at[None] >= c["sinks"])
            o_heads, l_heads = [], []
            for h in range(c["hq"]):
                a = s["q"][row + b:row + e, h].double() @ k[at, h // g].T / math.sqrt(D)
                a[gone] = -math.inf
                l_heads.append(torch.logsumexp(a, 1))
                a = torch.nan_to_num(torch.softmax(a, 1))
                o_heads.append(a @ v[at, h // g])
            outs.append(torch.stack(o_heads, 1))
            lses.append(torch.stack(l_heads, 1))
        row += m
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
