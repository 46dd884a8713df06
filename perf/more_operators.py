"""Cases of the operators that a prompt meets around the 2-bit cache: attention
inside a packed batch of prompts, writing the cache in chunks, reading it back,
and attention of a chunk of new tokens over it.

`run` computes an operator in its plain form (elementary torch operations in
fp32, rounded once at the end; the rotation before the quantiser in float64,
since a code hangs on the side of a border that a value falls to), or, where
`own` is true, through the package's entry points.  `exact` computes it from
the definition in float64.

The cache of a request of T tokens, head_dim 128: the first 64 tokens in BF16,
the last up to 256 in BF16, and those between (the history) rotated by R_K, R_V
of their kv head, clipped to +-tau and held as 2-bit codes c with an fp16 scale s
and zero z for each group of 128 or 64 channels, x = z + s c.
  prompt  causal attention of packed sequences, queries, keys and values as one
          projection's output holds them; with its log-sum-exp;
  extend  a request's tokens written in chunks, and all of them read back;
  read    tokens of filled requests as values in their own basis;
  chunk   new tokens of each request attend to its cached tokens and, causally,
          to each other; the cache stays as it is.
"""
import math

import torch

own = False

D, SINK, RECENT = 128, 64, 256
SCORES = 1 << 28   # scores that the plain form holds at a time


# ---- cases -------------------------------------------------------------------
def listed():
    return [
        # Three short prompts that arrive together: a launch and its latency.
        dict(name="prompt-short", op="prompt", hq=32, hkv=8, n=3, lo=1, hi=90, out="bf16"),
        # A ragged batch of prompts, eight query heads a kv head.
        dict(name="prompt-ragged", op="prompt", hq=64, hkv=8, n=7, lo=33, hi=4001, out="bf16"),
        # One 16K prompt.
        dict(name="prompt-16k", op="prompt", hq=32, hkv=8, n=1, lo=16384, hi=16384, out="bf16"),
        # Prompts for an evaluation that keeps fp32 outputs.
        dict(name="prompt-f32", op="prompt", hq=32, hkv=8, n=2, lo=700, hi=1901, out="f32"),
        # A short prompt in two pieces.
        dict(name="extend-400", op="extend", hkv=8, n=1, lo=400, hi=400, chunk=200, group=128),
        # A batch of prompts, two groups a head, 1024 tokens of each at a time.
        dict(name="extend-batch", op="extend", hkv=8, n=6, lo=300, hi=6001, chunk=1024, group=64),
        # A 32K prompt, 8192 tokens at a time.
        dict(name="extend-32k", op="extend", hkv=8, n=1, lo=32768, hi=32768, chunk=8192, group=128),
        # A whole 30K request for a move to BF16 pages.
        dict(name="read-30k", op="read", hkv=8, n=1, lo=30001, hi=30001, count=30001, group=128, out="bf16"),
        # A piece of each request of a batch, in fp32, to look at.
        dict(name="read-pieces", op="read", hkv=8, n=16, lo=500, hi=8000, count=333, group=64, out="f32"),
        # Five drafted tokens of one long request.
        dict(name="chunk-draft-100k", op="chunk", hq=32, hkv=8, n=1, lo=100000, hi=100000, qlo=5, qhi=5, group=128),
        # A ragged batch that continues, among it a request that has nothing cached yet; eight query heads a kv head.
        dict(name="chunk-ragged", op="chunk", hq=64, hkv=8, n=5, lo=0, hi=20001, qlo=3, qhi=1501, group=64),
        # The next 2048 tokens of a prompt of which 60K are cached.
        dict(name="chunk-2k-60k", op="chunk", hq=32, hkv=8, n=1, lo=60000, hi=60000, qlo=2048, qhi=2048, group=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "extend", "read", "chunk", "chunk", "chunk"])
    hkv = rng.choice([2, 4, 8])
    c = dict(op=op, hkv=hkv)
    if op in ("prompt", "chunk"):
        c["hq"] = hkv * rng.choice([1, 2, 4, 8])
    if op != "prompt":
        c["group"] = rng.choice([64, 128])
    if op in ("prompt", "read"):
        c["out"] = rng.choice(["bf16", "bf16", "f32"])
    if op == "prompt":
        c["n"] = _log(rng, 1, 24)
        c["hi"] = _log(rng, 4, 16384 // c["n"] if c["out"] == "bf16" else 4096 // c["n"])
        c["lo"] = rng.randint(1, c["hi"])
    elif op == "extend":
        c["n"] = _log(rng, 1, 8)
        c["hi"] = _log(rng, 50, 32768 // c["n"])
        c["lo"] = rng.randint(1, c["hi"])
        c["chunk"] = rng.randint(max(1, c["hi"] // 8), c["hi"])
    elif op == "read":
        c["n"] = _log(rng, 1, 24)
        c["hi"] = _log(rng, 70, 30001 // c["n"])
        c["lo"] = rng.randint(max(1, c["hi"] // 4), c["hi"])
        c["count"] = _log(rng, 1, c["hi"])
    else:
        c["n"] = _log(rng, 1, 32)
        c["qhi"] = _log(rng, 1, 2048 // c["n"])
        c["qlo"] = rng.randint(1, c["qhi"])
        c["hi"] = _log(rng, 64, min(100000, 600000 // c["n"]))
        # as many scores as the largest listed case has, at most
        c["hi"] = max(64, min(c["hi"], 2048 * 60000 * 32 // (c["n"] * c["qhi"] * c["hq"])))
        c["lo"] = rng.choice([0, rng.randint(0, c["hi"]), rng.randint(c["hi"] // 2, c["hi"])])
    return c


def _spread(lo, hi, n, step):
    """n lengths from lo to hi, the ends among them, off the round numbers between."""
    return [min(hi, lo + (hi - lo) * i // max(1, n - 1) + (step * i % 61 if 0 < i < n - 1 else 0)) for i in range(n)]


def _lengths(c):
    """Per request: its tokens (of a prompt, in the cache) and its rows (new tokens, or those read)."""
    base = _spread(c["lo"], c["hi"], c["n"], 37)
    if c["op"] == "chunk":
        return base, _spread(c["qlo"], c["qhi"], c["n"], 23)
    return base, [min(c["count"], t) for t in base] if c["op"] == "read" else base


def _split(t):
    """Tokens of a request of t that the sink holds, and the first that the recent window holds (t >= it >= sink)."""
    return min(t, SINK), max(min(t, SINK), t - RECENT)


def _record(group):
    """Bytes of the keys or values of a history token of one kv head."""
    return D // 4 + 4 * (D // group)


def _first(c, base, rows):
    """The first token that is read of each request: pieces from different places."""
    return [(t - m) * (i + 1) // (len(base) + 1) if t > m else 0 for i, (t, m) in enumerate(zip(base, rows))]


def work(case):
    c = case
    base, new = _lengths(c)
    rows, hkv = sum(new), c["hkv"]
    if c["op"] == "prompt":
        pairs = sum(t * (t + 1) // 2 for t in base)
        return {"bytes": rows * (D * (2 * c["hq"] + 4 * hkv + (4 if c["out"] == "f32" else 2) * c["hq"]) + 4 * c["hq"]),
                "flops": 4 * D * c["hq"] * pairs}
    token = 2 * hkv * _record(c["group"])
    turn = 2 * 2 * D * D * hkv   # rotation of a token's keys and values
    if c["op"] == "extend":
        hist = sum(max(0, b - a) for a, b in map(_split, base))
        held = hist * token + (rows - hist) * 4 * D * hkv
        return {"bytes": rows * 4 * D * hkv + 2 * held + rows * 8 * D * hkv, "flops": 2 * hist * turn}
    if c["op"] == "read":
        hist = 0
        for t, m, f in zip(base, new, _first(c, base, new)):
            a, b = _split(t)
            hist += max(0, min(b, f + m) - max(a, f))
        size = 4 if c["out"] == "f32" else 2
        return {"bytes": hist * token + (rows - hist) * 4 * D * hkv + rows * 2 * size * D * hkv, "flops": hist * turn}
    hist = sum(b - a for a, b in map(_split, base))
    pairs = sum(m * t + m * (m + 1) // 2 for t, m in zip(base, new))
    return {"bytes": hist * token + (sum(base) - hist + rows) * 4 * D * hkv + rows * c["hq"] * D * 4,
            "flops": 4 * D * c["hq"] * pairs + 4 * D * D * c["hq"] * rows}


# ---- inputs ------------------------------------------------------------------
def _rand(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 29)
    return lambda *shape: torch.randn(*shape, generator=g, device="cuda")


def _tokens(rand, rows, hkv, spread):
    """bf16 keys or values [rows][hkv][128]: a spread over the channels with a few large ones, as trained ones have."""
    return (rand(rows, hkv, D) * spread).to(torch.bfloat16)


def _inputs(c, seed):
    """What every form of an operator works on, from the seed alone."""
    rand = _rand(c, seed)
    base, new = _lengths(c)
    hkv, s = c["hkv"], {"lens": base, "new": new}
    k_spread = torch.exp(0.3 * rand(hkv, D))
    k_spread[:, 5] *= 8
    v_spread = torch.exp(0.3 * rand(hkv, D))
    if c["op"] == "prompt":
        qkv = rand(sum(base), c["hq"] + 2 * hkv, D)   # one projection's output
        qkv[:, c["hq"]:c["hq"] + hkv] *= k_spread
        s["q"], s["k"], s["v"] = qkv.to(torch.bfloat16).split([c["hq"], hkv, hkv], 1)
        return s
    s["rot_k"], s["rot_v"] = (torch.linalg.qr(rand(hkv, D, D).double())[0].float() for _ in range(2))
    s["k"], s["v"] = _tokens(rand, sum(base), hkv, k_spread), _tokens(rand, sum(base), hkv, v_spread)
    # thresholds as a calibration finds them: the 0.9 quantile of |x R| over a sample
    s["tau_k"], s["tau_v"] = (
        torch.einsum("thi,hij->thj", _tokens(rand, 512, hkv, w).float(), r).abs().permute(1, 0, 2).reshape(hkv, -1)
        .kthvalue(int(0.9 * 512 * D), 1).values for w, r in ((k_spread, s["rot_k"]), (v_spread, s["rot_v"])))
    if c["op"] == "chunk":
        qkv = rand(sum(new), c["hq"] + 2 * hkv, D)
        qkv[:, c["hq"]:c["hq"] + hkv] *= k_spread
        qkv[:, c["hq"] + hkv:] *= v_spread
        s["q"], s["k_new"], s["v_new"] = qkv.to(torch.bfloat16).split([c["hq"], hkv, hkv], 1)
    return s


def prepare(case, seed):
    c = case
    s = _inputs(c, seed)
    s["case"] = dict(c)
    rows, base, new, hkv = sum(s["new"]), s["lens"], s["new"], c["hkv"]
    kind = torch.float32 if c.get("out") == "f32" else torch.bfloat16
    s["workspace"] = None
    if c["op"] in ("prompt", "chunk"):
        s["out"] = torch.empty(rows, c["hq"], D, dtype=kind, device="cuda")
    if c["op"] == "prompt":
        s["lse"] = torch.empty(rows, c["hq"], device="cuda")
        return s
    starts = [sum(base[:i]) for i in range(c["n"])]
    if c["op"] == "extend":
        kind = torch.float32
        # the chunks as they come in: each request's next tokens, one request after another
        s["steps"] = []
        for at in range(0, max(base), c["chunk"]):
            some = [(i, min(c["chunk"], t - at)) for i, t in enumerate(base) if t > at]
            rows_of = torch.cat([torch.arange(starts[i] + at, starts[i] + at + m) for i, m in some]).cuda()
            s["steps"].append(([i for i, _ in some], [m for _, m in some], s["k"][rows_of], s["v"][rows_of]))
        place = torch.cat([torch.arange(t) for t in base])
        low = torch.repeat_interleave(torch.tensor([_split(t)[0] for t in base]), torch.tensor(base))
        high = torch.repeat_interleave(torch.tensor([_split(t)[1] for t in base]), torch.tensor(base))
        s["history"] = torch.nonzero((place >= low) & (place < high))[:, 0].cuda()
    if c["op"] in ("extend", "read"):
        s["k_out"], s["v_out"] = (torch.empty(rows, hkv, D, dtype=kind, device="cuda") for _ in range(2))
    if c["op"] == "read":
        s["first"] = _first(c, base, new)
    # The cache as a program has it before the call: the package's handle, filled by its prefill, for the package's calls,
    # and the same codes, scales and zeros as plain tensors for the plain form.
    if own:
        _cache(s, c, base, starts)
    elif c["op"] != "extend":
        _held(s, c, base, starts)
    if c["op"] != "extend":
        del s["k"], s["v"]
    return s


def _cache(s, c, base, starts):
    from bit_rotated_kv_decode_gb300 import binding
    pages = [-(-max(0, t - SINK) // 64) + 1 for t in base]
    cfg = binding.make_config(1, c.get("hq", c["hkv"]), c["hkv"], c["n"], max(pages), sum(pages), page_perm_seed=11,
                              group_size=c["group"])
    s["cache"] = binding.OscarCache(cfg, s["rot_k"][None].contiguous(), s["rot_v"][None].contiguous(),
                                    s["tau_k"].cpu().numpy(), s["tau_v"].cpu().numpy())
    if c["op"] == "extend":
        return
    s["reqs"] = [s["cache"].open() for _ in base]
    for r, a, t in zip(s["reqs"], starts, base):
        if t:
            s["cache"].prefill(r, 0, s["k"][a:a + t], s["v"][a:a + t])


def _held(s, c, base, starts):
    """The requests' caches, padded to the longest: codes [n][hkv][history][32 bytes], {scale, zero}, and BF16 tokens."""
    split = [_split(t) for t in base]
    most = max(1, max(b - a for a, b in split))
    for name in ("k", "v"):
        x = s[name]
        codes = torch.zeros(c["n"], c["hkv"], most, D // 4, dtype=torch.uint8, device="cuda")
        meta = torch.zeros(c["n"], c["hkv"], most, D // c["group"], 2, dtype=torch.float16, device="cuda")
        near = torch.zeros(c["n"], SINK + RECENT, c["hkv"], D, dtype=torch.bfloat16, device="cuda")
        for i, (at, t, (a, b)) in enumerate(zip(starts, base, split)):
            near[i, :a] = x[at:at + a]
            near[i, a:a + t - b] = x[at + b:at + t]
            for h in range(a, b, 8192):
                e = min(b, h + 8192)
                q, m = _quantise(_turn64(x[at + h:at + e], s["rot_" + name]), s["tau_" + name], c["group"])
                q = q.unflatten(-1, (-1, 4)) << torch.tensor([0, 2, 4, 6], dtype=torch.uint8, device="cuda")
                codes[i, :, h - a:e - a] = q.sum(-1, dtype=torch.uint8).transpose(0, 1)
                meta[i, :, h - a:e - a] = m.transpose(0, 1)
        s["codes_" + name], s["meta_" + name], s["near_" + name] = codes, meta, near


# ---- one pass ----------------------------------------------------------------
def run(state):
    if own:
        return _own(state)
    return {"prompt": _plain_prompt, "extend": _plain_extend, "read": _plain_read, "chunk": _plain_chunk}[
        state["case"]["op"]](state)


def _own(s):
    op = s["case"]["op"]
    if op == "prompt":
        from bit_rotated_kv_decode_gb300 import binding
        s["workspace"] = binding.prompt_attention(s["q"], s["k"], s["v"], s["out"], s["lens"], lse=s["lse"],
                                                  workspace=s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    cache = s["cache"]
    if op == "chunk":
        s["workspace"] = cache.chunk_attention(0, s["reqs"], s["q"], s["k_new"], s["v_new"], s["out"],
                                               new_lens=s["new"], workspace=s["workspace"])
        return {"out": s["out"]}
    if op == "read":
        cache.read(0, s["reqs"], s["first"], s["new"], s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    reqs = [cache.open() for _ in s["lens"]]
    for who, lens, k, v in s["steps"]:
        cache.extend(0, [reqs[i] for i in who], k, v, new_lens=lens)
    cache.read(0, reqs, [0] * len(reqs), s["lens"], s["k_out"], s["v_out"])
    for r in reqs:
        cache.close(r)
    return {"k": s["k_out"], "v": s["v_out"]}


def _turn64(x, rot):
    """fp32 of x R, the sum in float64: bf16 [rows][hkv][128] and fp32 [hkv][128][128]."""
    return torch.matmul(x.transpose(0, 1).double(), rot.double()).transpose(0, 1).float()


def _quantise(x, tau, group):
    """Codes 0 .. 3 and fp16 {scale, zero} of each group of fp32 [rows][hkv][128]."""
    tau = tau[:, None]
    x = (torch.maximum(torch.minimum(x, tau), -tau) + 0.0).unflatten(-1, (-1, group))
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    # a tensor as the divisor: dividing by a Python number multiplies by its reciprocal, which rounds otherwise
    zero, scale = lo.half(), ((hi - lo) / torch.full_like(lo, 3.0)).half()
    code = torch.round((x - zero.float()) / scale.float()).clamp(0, 3)
    code = torch.where(scale == 0, torch.zeros_like(code), code)
    return code.flatten(-2).to(torch.uint8), torch.cat([scale, zero], -1)


def _values(code, meta):
    """z + s c of codes [...][128] with {scale, zero} [...][groups][2], fp32."""
    x = code.unflatten(-1, (meta.shape[-2], -1)).float()
    return (x * meta[..., :1].float() + meta[..., 1:].float()).flatten(-2)


def _unpack(b):
    return ((b[..., None] >> torch.tensor([0, 2, 4, 6], dtype=torch.uint8, device=b.device)) & 3).flatten(-2)


def _plain_extend(s):
    c, at = s["case"], s["history"]
    out = {}
    for name in ("k", "v"):
        x = s[name].float()
        code, meta = _quantise(_turn64(s[name][at], s["rot_" + name]), s["tau_" + name], c["group"])
        x[at] = torch.matmul(_values(code, meta).transpose(0, 1), s["rot_" + name].mT).transpose(0, 1)
        out[name] = x
    return out


def _plain_read(s):
    c = s["case"]
    kind = torch.float32 if c["out"] == "f32" else torch.bfloat16
    out = {}
    for name in ("k", "v"):
        rows = []
        for i, (t, m, f) in enumerate(zip(s["lens"], s["new"], s["first"])):
            a, b = _split(t)
            p, q = max(a, min(f, b)), max(a, min(f + m, b))
            x = _values(_unpack(s["codes_" + name][i, :, p - a:q - a]), s["meta_" + name][i, :, p - a:q - a])
            x = torch.matmul(x, s["rot_" + name].mT).transpose(0, 1)
            near = s["near_" + name][i].float()
            rows += [near[min(f, a):min(f + m, a)], x, near[max(f, b) - b + a:max(f + m, b) - b + a]]
        out[name] = torch.cat(rows).to(kind)
    return out


def _softmax(a, see):
    """exp(a - top) where seen, the sum and the top of each row; a is overwritten."""
    a.masked_fill_(~see, -math.inf)
    top = a.amax(-1, keepdim=True)
    a.sub_(top).exp_()
    return a, a.sum(-1, keepdim=True), top


def _plain_prompt(s):
    c = s["case"]
    g, kind = c["hq"] // c["hkv"], torch.float32 if c["out"] == "f32" else torch.bfloat16
    outs, lses, row = [], [], 0
    for t in s["lens"]:
        k, v = s["k"][row:row + t].float().permute(1, 2, 0), s["v"][row:row + t].float().transpose(0, 1)
        step = max(1, min(t, SCORES // (c["hq"] * t)))
        for b in range(0, t, step):                        # blocks of queries, so that the scores fit
            e = min(t, b + step)
            q = s["q"][row + b:row + e].float().unflatten(1, (c["hkv"], g)).permute(1, 2, 0, 3).flatten(1, 2)
            a = torch.matmul(q / math.sqrt(D), k[..., :e]).unflatten(1, (g, e - b))
            see = torch.arange(e, device="cuda") <= torch.arange(b, e, device="cuda")[:, None]
            a, total, top = _softmax(a, see)
            o = torch.matmul(a.flatten(1, 2), v[:, :e]).unflatten(1, (g, e - b)) / total
            outs.append(o.permute(2, 0, 1, 3).flatten(1, 2))
            lses.append((total.log() + top).squeeze(-1).permute(2, 0, 1).flatten(1, 2))
        row += t
    return {"out": torch.cat(outs).to(kind), "lse": torch.cat(lses)}


def _history(s, pick, most):
    """Values of the first `most` history tokens of the requests `pick`, in the rotated basis."""
    return [_values(_unpack(s["codes_" + w][pick, :, :most]), s["meta_" + w][pick, :, :most]) for w in "kv"]


def _chunk_rows(s, c, pick, far, q, k_new, v_new, before):
    """Queries q [n][m][hq][128] of the requests `pick`, at the new tokens before, before + 1, ...: fp32 out.  far: their
    _history(); k_new and v_new [n][before + m][hkv][128]."""
    n, m, g = q.shape[0], q.shape[1], c["hq"] // c["hkv"]
    far_k, far_v = far
    most = far_k.shape[2]
    split = torch.tensor([_split(t) for t in s["lens"][pick]], device="cuda")
    total = torch.tensor(s["lens"][pick], device="cuda")
    x = q.float().unflatten(2, (c["hkv"], g)) / math.sqrt(D)
    x_rot = torch.einsum("nmhgi,hij->nhgmj", x, s["rot_k"]).flatten(2, 3)
    x = x.permute(0, 2, 3, 1, 4).flatten(2, 3)
    near_k, near_v = (torch.cat([s["near_" + w][pick], y], 1).float().transpose(1, 2)
                      for w, y in (("k", k_new), ("v", v_new)))
    a = torch.cat([torch.matmul(x_rot, far_k.mT), torch.matmul(x, near_k.mT)], -1).unflatten(2, (g, m))
    held = torch.cat([torch.arange(most, device="cuda") < (split[:, 1] - split[:, 0])[:, None],
                      torch.arange(SINK + RECENT, device="cuda") < (total - split[:, 1] + split[:, 0])[:, None]], 1)
    causal = torch.arange(before + m, device="cuda") <= torch.arange(before, before + m, device="cuda")[:, None]
    see = torch.cat([held[:, None].expand(-1, m, -1), causal.expand(n, -1, -1)], 2)
    a, l, _ = _softmax(a, see[:, None, None])
    a = a.flatten(2, 3)
    o = torch.matmul(torch.matmul(a[..., :most], far_v), s["rot_v"].mT) + torch.matmul(a[..., most:], near_v)
    return (o.unflatten(2, (g, m)) / l).permute(0, 3, 1, 2, 4).flatten(2, 3)


def _plain_chunk(s):
    c, new = s["case"], s["new"]
    if min(new) == max(new) and c["n"] * new[0] * c["hq"] * max(s["lens"]) <= SCORES:   # a batch of few tokens
        rows = [s[w].unflatten(0, (c["n"], -1)) for w in ("q", "k_new", "v_new")]
        pick = slice(0, c["n"])
        far = _history(s, pick, s["codes_k"].shape[2])
        return {"out": _chunk_rows(s, c, pick, far, *rows, 0).flatten(0, 1).to(torch.bfloat16)}
    out, row = [], 0
    for i, (t, m) in enumerate(zip(s["lens"], new)):
        step = max(1, min(m, SCORES // (c["hq"] * (t + m))))
        pick, (low, high) = slice(i, i + 1), _split(t)
        far = _history(s, pick, high - low)
        for b in range(0, m, step):                        # blocks of queries, so that the scores fit
            e = min(m, b + step)
            q, k, v = s["q"][None, row + b:row + e], s["k_new"][None, row:row + e], s["v_new"][None, row:row + e]
            out.append(_chunk_rows(s, c, pick, far, q, k, v, b)[0])
        row += m
    return {"out": torch.cat(out).to(torch.bfloat16)}


# ---- the definition in float64 -----------------------------------------------
def _stored(x, rot, tau, group):
    """What the cache holds of bf16 history tokens [rows][hkv][128], as float64 values in their own basis, a head at a
    time.  The operator defines the codes bit for bit, in fp32 steps on the fp32 rounding of x R."""
    y = torch.empty(x.shape, dtype=torch.float64, device="cuda")
    for h in range(x.shape[1]):
        r, lim = rot[h].double(), float(tau[h])
        w = (x[:, h].double() @ r).to(torch.float32).clamp(-lim, lim).reshape(-1, group)
        low, high = w.min(1, keepdim=True).values, w.max(1, keepdim=True).values
        z = low.to(torch.float16).float()
        d = torch.true_divide(high - low, torch.tensor(3.0, device="cuda").expand_as(low).contiguous()).half().float()
        n = torch.where(d > 0, torch.round(torch.true_divide(w - z, torch.where(d > 0, d, 1.0))), 0.0).clamp(0, 3)
        y[:, h] = (z.double() + d.double() * n.double()).reshape(-1, D) @ r.T
    return y


def _all_tokens(s, c, name, at, t):
    """Keys or values [t][hkv][128] of a request, float64, as its cache holds them."""
    y = s[name][at:at + t].double()
    if t > SINK + RECENT:
        for b in range(SINK, t - RECENT, 16384):
            e = min(t - RECENT, b + 16384)
            y[b:e] = _stored(s[name][at + b:at + e], s["rot_" + name], s["tau_" + name], c["group"])
    return y


def exact(case, seed):
    c = case
    if work(c)["flops"] > 4e12:
        return None   # float64 products of this size take too long
    s = _inputs(c, seed)
    base, new = s["lens"], s["new"]
    outs, lses, ks, vs, at, row = [], [], [], [], 0, 0
    for i, (t, m) in enumerate(zip(base, new)):
        if c["op"] == "prompt":
            k, v, before = s["k"][at:at + t].double(), s["v"][at:at + t].double(), 0
        else:
            k, v, before = _all_tokens(s, c, "k", at, t), _all_tokens(s, c, "v", at, t), t
        at += t
        if c["op"] in ("extend", "read"):
            f = 0 if c["op"] == "extend" else _first(c, base, new)[i]
            ks.append(k[f:f + m])
            vs.append(v[f:f + m])
            continue
        if c["op"] == "chunk":
            k = torch.cat([k, s["k_new"][row:row + m].double()])
            v = torch.cat([v, s["v_new"][row:row + m].double()])
        for b in range(0, m, 256):
            e = min(m, b + 256)
            last = before + e
            gone = torch.ones(e - b, last, dtype=torch.bool, device="cuda").triu(before + b + 1)
            o_heads, l_heads = [], []
            for h in range(c["hq"]):
                j = h * c["hkv"] // c["hq"]
                x = (s["q"][row + b:row + e, h].double() @ k[:last, j].T) * D ** -0.5
                x[gone] = -math.inf
                l_heads.append(x.logsumexp(1))
                o_heads.append(x.softmax(1) @ v[:last, j])
            outs.append(torch.stack(o_heads, 1))
            lses.append(torch.stack(l_heads, 1))
        row += m
    if c["op"] in ("extend", "read"):
        return {"k": torch.cat(ks), "v": torch.cat(vs)}
    return {"out": torch.cat(outs), "lse": torch.cat(lses)} if c["op"] == "prompt" else {"out": torch.cat(outs)}
