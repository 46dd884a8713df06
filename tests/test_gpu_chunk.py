"""Prompt attention, and the chunk calls on the three-segment cache -- extend, read, chunk
attention -- against float64.

Caches start as 0xFF bytes (NaN values, scales and zeros), so that anything read that was
not written shows; page orders are shuffled.

Tolerances, derived before the first run.  u = 2^-24.  A rounding is off by at most half a
step: bf16 2^-8, fp16 2^-11 of the value.
  logit    a product of 128 terms on the matrix unit: 8 steps, each off by at most 36 u of the
           sum of magnitudes: 288 u; against history 2^-11 more for q R_K and for the values;
  weight   the logit's error, 2^-21 for ex2, and 2^-8 where it enters the product with V as bf16
           (2^-11 as fp16, 2^-24 as three parts); normalising doubles it;
  values   against history 2^-11 for the value, 2^-11 for R_V, 2^-11 for the row that is rotated
           back, relative to the magnitudes that the rotation sums;
  sums     288 u per 128 keys that the accumulator takes, counted as 64 steps: 2^-16;
  output   2^-8 of itself as bf16.
All relative to sum p |v|.  Beside that the error over the whole output, whose roundings are
independent: 2^-8 / sqrt(3) for a bf16 output and as much for bf16 weights, 3.2e-3 together; 4e-3 is taken.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module")
def b():
    from bit_rotated_kv_decode_gb300 import binding, build
    build.build()
    binding.load()
    return binding


def rand(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *shape: torch.randn(*shape, generator=g, device="cuda")


def attend(q, k, v, see, scale=None):
    """float64 softmax attention of q [m][hq][128] over k, v [t][hkv][128] where see [m][t]: out, lse, sum p |v|, and per
    query and head the largest sum of magnitudes of a logit."""
    m, hq, _ = q.shape
    g = hq // k.shape[1]
    scale = scale or 1 / math.sqrt(D)
    q, k, v = q.double(), k.double().repeat_interleave(g, 1), v.double().repeat_interleave(g, 1)
    a = torch.einsum("mhd,thd->mht", q, k) * scale
    a = a.masked_fill(~see[:, None], -math.inf)
    lse = torch.logsumexp(a, -1)
    p = torch.nan_to_num(torch.softmax(a, -1))
    mag = torch.einsum("mhd,thd->mht", q.abs(), k.abs()).masked_fill(~see[:, None], 0).amax(-1) * scale
    return torch.einsum("mht,thd->mhd", p, v), lse, torch.einsum("mht,thd->mhd", p, v.abs()), mag


def off_by(got, want):
    return float((got.double() - want).norm() / want.norm())


# ---- prompt attention -----------------------------------------------------------
def check_prompt(b, lens, hq, hkv, out_type, window=-1, sinks=0, seed=0, scale=0.0, poison=False):
    rnd = rand(seed)
    rows = sum(lens)
    qkv = rnd(rows, hq + 2 * hkv, D)
    qkv[:, hq:hq + hkv, 5] *= 6
    q, k, v = qkv.bfloat16().split([hq, hkv, hkv], 1)
    out = torch.full((rows, hq, D), float("nan"), device="cuda", dtype=out_type)
    lse = torch.full((rows, hq), float("nan"), device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = b.prompt_workspace(lens, hq, hkv)
    ws.fill_(0xFF)
    assert b.prompt_attention(q, k, v, out, lens, window, sinks, scale, lse=lse, workspace=ws, error=err) is ws
    assert int(err) == 0
    at = 0
    for t in filter(None, lens):
        p = torch.arange(t, device="cuda")
        see = p[None] <= p[:, None]
        if window >= 0:
            see &= (p[None] > p[:, None] - window) | (p[None] < sinks)
        want, l, pv, mag = attend(q[at:at + t], k[at:at + t], v[at:at + t], see, scale)
        got, gl = out[at:at + t].double(), lse[at:at + t].double()
        f32 = out_type == torch.float32
        logit = 288 * 2 ** -24 * mag[..., None] * 1.5
        tol = (2 * logit + 2 * 2 ** -21 + (2 ** -24 if f32 else 2 ** -8) + (2 ** -18 if f32 else 2 ** -16)) * pv + (0 if f32 else 2 ** -8) * want.abs()
        none = ~see.any(1)
        assert bool((got[none] == 0).all()) and bool((gl[none] == -math.inf).all())
        assert bool(((got - want).abs() <= tol + 1e-30).all()), float(((got - want).abs() / (tol + 1e-30)).max())
        assert bool(((gl - l).abs()[~none] <= logit[..., 0][~none] + 2 ** -20 * (1 + l[~none].abs())).all())
        at += t
    if rows and window < 0:
        want = torch.cat([attend(q[s:s + t], k[s:s + t], v[s:s + t], torch.ones(t, t, device="cuda").tril().bool(), scale)[0]
                          for s, t in zip(np.cumsum([0] + lens[:-1]).tolist(), lens) if t])
        assert off_by(out, want) < (4e-6 if out_type == torch.float32 else 4e-3)


@pytest.mark.parametrize("hq,hkv", [(4, 4), (4, 2), (8, 2), (16, 2)])
@pytest.mark.parametrize("out_type", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens", [[1], [0, 5, 0, 64, 1], [63, 65, 127, 129], [700], [257, 1, 0, 511]])
def test_prompt(b, lens, hq, hkv, out_type):
    check_prompt(b, lens, hq, hkv, out_type, seed=len(lens) + hq)


@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 3), (1, 0), (64, 0), (100, 70), (2 ** 31 - 1, 5)])
@pytest.mark.parametrize("out_type", [torch.bfloat16, torch.float32])
def test_prompt_window(b, window, sinks, out_type):
    check_prompt(b, [300, 1, 450], 8, 2, out_type, window, sinks, seed=3)


def test_prompt_many_sequences_and_scale(b):
    check_prompt(b, [(7 * i) % 23 for i in range(256)], 4, 2, torch.bfloat16, seed=4, scale=0.2)
    check_prompt(b, [1900], 2, 2, torch.bfloat16, seed=5)      # few blocks: key tiles split
    check_prompt(b, [1900], 2, 2, torch.float32, seed=5)


def test_prompt_sequences_do_not_mix(b):
    """NaN in one sequence stays there: in its keys, values and queries; another's rows are what they were alone."""
    rnd = rand(6)
    lens, hq, hkv = [100, 33, 200], 8, 2
    q, k, v = rnd(333, hq, D).bfloat16(), rnd(333, hkv, D).bfloat16(), rnd(333, hkv, D).bfloat16()
    out = torch.empty(333, hq, D, device="cuda", dtype=torch.bfloat16)
    b.prompt_attention(q, k, v, out, lens)
    clean = out.clone()
    for x in (q, k, v):
        x[100:133] = float("nan")
    b.prompt_attention(q, k, v, out, lens)
    assert torch.equal(out[:100], clean[:100]) and torch.equal(out[133:], clean[133:])
    assert bool(out[100:133].isnan().all())


def test_prompt_matches_window_attention_over_pages(b):
    rnd = rand(7)
    lens, hq, hkv = [130, 700, 64], 8, 2
    rows = sum(lens)
    q, k, v = rnd(rows, hq, D).bfloat16(), rnd(rows, hkv, D).bfloat16(), rnd(rows, hkv, D).bfloat16()
    pages = sum(-(-t // 64) for t in lens)
    kv = torch.zeros(pages, hkv, 2, 64, D, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(3, 11, dtype=torch.int32, device="cuda")
    at = 0
    for i, t in enumerate(lens):
        n = -(-t // 64)
        table[i, :n] = torch.arange(at, at + n)
        at += n
    b.bf16_append(kv, table, [0, 0, 0], k, v, new_lens=lens)
    one, two = torch.empty_like(q), torch.empty_like(q)
    b.window_attention(kv, table, lens, q, one, hkv, 100, 5, q_lens=lens)
    b.prompt_attention(q, k, v, two, lens, 100, 5)
    assert torch.equal(one, two)


def test_prompt_refusals(b):
    q, k = torch.zeros(9, 4, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(9, 2, D, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    ok = dict(q=q, k=k, v=k, out=out, lens=[4, 5])
    b.prompt_attention(**ok)
    for change in (dict(lens=[4, 4]), dict(lens=[]), dict(lens=[10, -1]), dict(q=q.float()), dict(k=k[:8]), dict(v=k[:, :1]),
                   dict(out=out.half()), dict(out=out[:, :2]), dict(q=q.cpu()), dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)),
                   dict(lse=torch.zeros(9, 3, device="cuda")), dict(error=torch.zeros(0, dtype=torch.int32, device="cuda")),
                   dict(sinks=-1), dict(scale=float("nan")), dict(q=torch.zeros(9, 6, D, dtype=torch.bfloat16, device="cuda"),
                                                                   out=torch.zeros(9, 6, D, dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(b.OscarError):
            b.prompt_attention(**{**ok, **change})
    small = b.new_workspace(256)
    big = b.prompt_attention(q[:, :2].contiguous().repeat(300, 1, 1), k.repeat(300, 1, 1), k.repeat(300, 1, 1),
                             torch.zeros(2700, 2, D, dtype=torch.bfloat16, device="cuda"), [2700], workspace=small)
    assert big.numel() > small.numel()


# ---- the three-segment cache ------------------------------------------------------
class Held:
    """A cache of one layer or more, its rotations and thresholds, and the tokens that were written to it."""

    def __init__(self, b, hq=8, hkv=2, requests=4, tokens=3000, group=128, seed=0, quantile=0.9, layers=1, pages=None):
        rnd = self.rnd = rand(seed)
        self.b, self.hq, self.hkv, self.group = b, hq, hkv, group
        self.rot = [torch.linalg.qr(rnd(layers, hkv, D, D).double())[0].float().contiguous() for _ in range(2)]
        self.spread = [torch.exp(0.3 * rnd(hkv, D)) for _ in range(2)]
        self.spread[0][:, 5] *= 8
        tau = []
        for w, r in zip(self.spread, self.rot):
            x = torch.einsum("thi,lhij->lhtj", (rnd(256, hkv, D) * w).bfloat16().float(), r).abs().flatten(2)
            tau.append(x.kthvalue(max(1, int(quantile * x.shape[-1])), -1).values.cpu().numpy())
        table = tokens // 64 + 1
        cfg = b.make_config(layers, hq, hkv, requests, table, pages or requests * table, page_perm_seed=seed + 7, group_size=group)
        self.cache = b.OscarCache(cfg, *self.rot, *tau)
        for layer in range(layers):
            self.cache.int2_pool(layer).fill_(255)
            self.cache.bf16_pool(layer).fill_(-1)

    def tokens(self, n):
        return [(self.rnd(n, self.hkv, D) * w).bfloat16() for w in self.spread]

    def stored(self, req, layer=0):
        """Keys and values [T][hkv][128] float64 from the cache's own bytes, and of history the magnitudes that undoing the
        rotation sums."""
        T, he = self.cache.length(req, layer)
        hist, near = self.cache.pages(req)
        pool, bf = self.cache.int2_pool(layer), self.cache.bf16_pool(layer).view(torch.bfloat16)
        ng = D // self.group
        vals, mags = [], []
        p = torch.arange(T, device="cuda")
        slot = torch.where(p < 64, p, (p - 64) % 256 + 64)
        page = torch.tensor(near, device="cuda")[slot // 64]
        rec = pool[torch.tensor(hist, device="cuda")] if hist else None
        for which in range(2):
            x = bf[page, :, which, slot % 64].double()
            mag = x.abs()
            if he > 64 and T > 64:
                code = rec[:, :, 2048 * which:2048 * (which + 1)].reshape(len(hist), self.hkv, 64, 32, 1)
                code = (code >> torch.tensor([0, 2, 4, 6], dtype=torch.uint8, device="cuda") & 3).reshape(len(hist), self.hkv, 64, ng, -1)
                meta = rec[:, :, 4096 + 256 * ng * which:4096 + 256 * ng * (which + 1)].contiguous().view(torch.float16)
                meta = meta.reshape(len(hist), self.hkv, 64, ng, 2).double()
                y = (meta[..., 1:] + meta[..., :1] * code.double()).reshape(len(hist), self.hkv, 64, D)
                y = y.transpose(1, 2).reshape(-1, self.hkv, D)[:he - 64]
                r = self.rot[which][layer].double()
                x[64:he] = torch.einsum("thj,hij->thi", y, r)
                mag[64:he] = torch.einsum("thj,hij->thi", y.abs(), r.abs())
            vals.append(x)
            mags.append(mag)
        return vals, mags, (min(T, 64), max(min(T, 64), he if T > 64 else 0))


def same_caches(one, two, reqs, layer=0):
    """The bytes of every token that a request of both caches holds."""
    for r in reqs:
        assert one.cache.length(r, layer) == two.cache.length(r, layer)
        (ka, _, _), (kb, _, _) = one.stored(r, layer), two.stored(r, layer)
        for x, y in zip(ka, kb):
            assert torch.equal(x, y)
        T, he = one.cache.length(r, layer)
        ng = D // one.group
        pa, pb = one.cache.pages(r)[0], two.cache.pages(r)[0]
        a, c = one.cache.int2_pool(layer), two.cache.int2_pool(layer)
        for i, (x, y) in enumerate(zip(pa, pb)):
            rows = min(64, he - 64 - 64 * i)
            if rows > 0:
                for at, w in ((0, 32), (2048, 32), (4096, 4 * ng), (4096 + 256 * ng, 4 * ng)):
                    assert torch.equal(a[x, :, at:at + rows * w], c[y, :, at:at + rows * w]), (r, i, at)


@pytest.mark.parametrize("group", [128, 64])
@pytest.mark.parametrize("quantile", [0.9, 0.97, 1.0])
def test_extend_writes_what_appends_write(b, group, quantile):
    one, two = (Held(b, group=group, quantile=quantile, seed=1, tokens=800) for _ in range(2))
    reqs = [one.cache.open() for _ in range(3)]
    assert reqs == [two.cache.open() for _ in range(3)]
    g = np.random.default_rng(group)
    for step in range(9):
        lens = [int(x) for x in g.choice([0, 1, 5, 63, 64, 130], 3)]
        if step == 4:
            one.cache.demote(0, reqs[:2])
            two.cache.demote(0, reqs[:2])
        k, v = one.tokens(sum(lens))
        one.cache.extend(0, reqs, k, v, new_lens=lens)
        at = [sum(lens[:i]) for i in range(3)]
        for j in range(max(lens)):
            some = [i for i in range(3) if j < lens[i]]
            rows = torch.tensor([at[i] + j for i in some], device="cuda")
            two.cache.append(0, [reqs[i] for i in some], k[rows].contiguous(), v[rows].contiguous())
    one.cache.check()
    two.cache.check()
    same_caches(one, two, reqs)


@pytest.mark.parametrize("scale", [1e-4, 1.0, 3000.0])
def test_extend_writes_what_prefill_writes(b, scale):
    """Values of any size, equal tokens and zeros, from parts of one projection's output, and after a fork."""
    one, two = (Held(b, seed=2, tokens=2000, quantile=0.95) for _ in range(2))
    tau = np.full((1, 2), 2.5 * scale, np.float32)
    for h in (one, two):
        cfg = b.make_config(1, 8, 2, 4, 40, 120, page_perm_seed=3)
        h.cache = b.OscarCache(cfg, *h.rot, tau, tau)
        h.cache.int2_pool(0).fill_(255)
    k, v = one.tokens(1500)
    k, v = (k * scale).bfloat16(), (v * scale).bfloat16()
    k[400:410] = 0
    v[500:520] = v[499]
    qkv = torch.cat([k, k, v], 1)
    r, s = one.cache.open(), two.cache.open()
    for at, m in ((0, 1), (1, 700), (701, 799)):
        one.cache.extend(0, [r], qkv[at:at + m, :2], qkv[at:at + m, 4:], new_lens=[m])
    two.cache.prefill(s, 0, k, v)
    same_caches(one, two, [r])
    f, e = one.cache.fork(r, 64 + 64 * 5), two.cache.fork(s, 64 + 64 * 5)
    assert f == e
    for at, m in ((0, 300), (300, 400)):
        one.cache.extend(0, [f], k[at:at + m], v[at:at + m], new_lens=[m])
    two.cache.prefill(e, 0, k[:700].contiguous(), v[:700].contiguous())
    one.cache.check()
    same_caches(one, two, [r, f])


def test_extend_leaves_other_layers_and_requests(b):
    h = Held(b, layers=2, seed=3, tokens=900)
    r = [h.cache.open() for _ in range(2)]
    k, v = h.tokens(700)
    for layer in (0, 1):
        h.cache.extend(layer, r, torch.cat([k, k]), torch.cat([v, v]), new_lens=[700, 700])
    before = h.stored(r[0], 1), h.stored(r[1], 0)
    h.cache.extend(0, [r[0]], *h.tokens(150), new_lens=[150])
    for (x, _, _), (y, _, _) in zip(before, (h.stored(r[0], 1), h.stored(r[1], 0))):
        assert all(torch.equal(i, j) for i, j in zip(x, y))
    assert h.cache.length(r[0], 1) == (700, 444)


@pytest.mark.parametrize("group", [128, 64])
@pytest.mark.parametrize("out_type", [torch.bfloat16, torch.float32])
def test_read(b, group, out_type):
    h = Held(b, group=group, seed=4, tokens=1500)
    reqs = [h.cache.open() for _ in range(4)]
    lens = [1200, 64, 5, 385]
    h.cache.extend(0, reqs, *h.tokens(sum(lens)), new_lens=lens)
    # whole requests, pieces around every border, one token, none, the same request twice
    which = [0, 1, 2, 3, 0, 0, 0, 0, 0, 3]
    start = [0, 0, 0, 0, 60, 63, 940, 944, 100, 385]
    count = [1200, 64, 5, 385, 10, 1, 8, 256, 200, 0]
    rows = sum(count)
    k, v = (torch.full((rows, h.hkv, D), float("nan"), device="cuda", dtype=out_type) for _ in range(2))
    h.cache.read(0, [reqs[i] for i in which], start, count, k, v)
    h.cache.check()
    for got, n in ((k, 0), (v, 1)):
        at = 0
        for i, s, m in zip(which, start, count):
            vals, mags, (a, c) = h.stored(reqs[i])
            want, mag = vals[n][s:s + m], mags[n][s:s + m]
            x = got[at:at + m].double()
            p = torch.arange(s, s + m, device="cuda")
            near = (p < a) | (p >= c)
            assert torch.equal(x[near], want[near])
            far = ~near
            # fp32: c' R on the matrix unit in eight steps of three parts, and a product's rounding; bf16: the
            # value and R in fp16
            tol = 400 * 2 ** -24 * 2 * mag if out_type == torch.float32 else (2 * 2 ** -11 + 2 ** -13) * mag + 2 ** -8 * want.abs()
            assert bool(((x - want).abs()[far] <= tol[far]).all())
            if far.any():
                assert off_by(x[far], want[far]) < (1e-6 if out_type == torch.float32 else 3e-3)
            at += m


def check_chunk(h, reqs, lens, layer=0, workspace=None, stream=None, strided=True):
    """One call against float64; the cache's bytes stay."""
    rows = sum(lens)
    k, v = h.tokens(rows)
    q = (h.rnd(rows, h.hq, D) * 1.3).bfloat16()
    if strided:
        q, k, v = torch.cat([q, k, v], 1).split([h.hq, h.hkv, h.hkv], 1)
    out = torch.full((rows, h.hq, D), float("nan"), device="cuda", dtype=torch.bfloat16)
    before = h.cache.mem.clone() if h.cache.mem.numel() < 1 << 28 else None
    ws = h.cache.chunk_attention(layer, reqs, q, k, v, out, new_lens=lens, workspace=workspace)
    h.cache.check()
    if before is not None:
        assert torch.equal(before, h.cache.mem)
    at, wants = 0, []
    for r, m in zip(reqs, lens):
        if m == 0:
            continue
        (kc, vc), (km, vm), (a, c) = h.stored(r, layer)
        t = kc.shape[0]
        p = torch.arange(t + m, device="cuda")
        see = p[None] <= torch.arange(t, t + m, device="cuda")[:, None]
        keys, values = torch.cat([kc, k[at:at + m].double()]), torch.cat([vc, v[at:at + m].double()])
        want, _, pv, mag = attend(q[at:at + m], keys, values, see)
        far = (p >= a) & (p < c)
        if far.any():   # the history's magnitudes are those in the rotated basis
            qm = torch.einsum("mhgi,hij->mhgj", q[at:at + m].double().unflatten(1, (h.hkv, -1)).abs(), h.rot[0][layer].double().abs())
            hm = torch.einsum("mhgi,thi->mhgt", qm, torch.einsum("thi,hij->thj", km[a:c].abs(), h.rot[0][layer].double().abs())).amax(-1)
            mag = torch.maximum(mag, hm.flatten(1) / math.sqrt(D) / 16)
            pv = torch.maximum(pv, attend(q[at:at + m], keys, torch.cat([vm, v[at:at + m].double()]), see)[2])
        got = out[at:at + m].double()
        logit = (288 * 2 ** -24 + (2 * 2 ** -11 if far.any() else 0)) * mag[..., None]
        tol = (2 * logit + 2 ** -20 + 2 ** -8 + (3 * 2 ** -11 if far.any() else 0) + 2 ** -16) * pv + 2 ** -8 * want.abs()
        assert bool(((got - want).abs() <= tol).all()), float(((got - want).abs() / tol).max())
        wants.append(want)
        at += m
    if rows:
        assert off_by(out, torch.cat(wants)) < 4e-3, off_by(out, torch.cat(wants))
    return ws


@pytest.mark.parametrize("t", [0, 1, 63, 64, 65, 320, 321, 383, 384, 385, 449, 1000])
@pytest.mark.parametrize("m", [1, 7, 65, 300])
def test_chunk_lengths(b, t, m):
    h = Held(b, seed=t + m, requests=1, tokens=1100)
    r = h.cache.open()
    if t:
        h.cache.extend(0, [r], *h.tokens(t), new_lens=[t])
    check_chunk(h, [r], [m])


@pytest.mark.parametrize("group", [128, 64])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (8, 2), (16, 2)])
def test_chunk_ragged(b, hq, hkv, group):
    h = Held(b, hq=hq, hkv=hkv, group=group, seed=hq, requests=7, tokens=2600)
    reqs = [h.cache.open() for _ in range(7)]
    held = [0, 2500, 40, 700, 1311, 320, 385]
    h.cache.extend(0, reqs, *h.tokens(sum(held)), new_lens=held)
    ws = check_chunk(h, reqs, [5, 1, 300, 33, 0, 2, 129])
    ws.fill_(0xFF)                                                  # no contents are needed
    check_chunk(h, reqs[1:], [17, 1, 130, 16, 65, 3], workspace=ws)
    check_chunk(h, [reqs[1]] * 3 + [reqs[4]], [4, 1, 4, 200])       # several drafts of one request
    check_chunk(h, reqs, [1] * 7, workspace=ws, strided=False)


def test_chunk_many_requests(b):
    h = Held(b, hq=4, hkv=2, seed=11, requests=256, tokens=500)
    reqs = [h.cache.open() for _ in range(256)]
    held = [(37 * i) % 450 for i in range(256)]
    h.cache.extend(0, reqs, *h.tokens(sum(held)), new_lens=held)
    check_chunk(h, reqs, [1 + (i % 3) for i in range(256)])


def test_chunk_window_of_any_fill(b):
    """The recent window emptied, half full and wrapped round the ring."""
    h = Held(b, seed=12, requests=3, tokens=900)
    r = h.cache.open()
    h.cache.extend(0, [r], *h.tokens(700), new_lens=[700])
    f = h.cache.fork(r, 64 + 64 * 5)
    check_chunk(h, [r, f], [40, 40])
    h.cache.extend(0, [f], *h.tokens(100), new_lens=[100])
    for _ in range(100):
        h.cache.demote(0, [r])
    check_chunk(h, [r, f], [9, 150])
    h.cache.extend(0, [r], *h.tokens(77), new_lens=[77])
    check_chunk(h, [f, r], [1, 70])


def test_chunk_peaks_and_growing_maxima(b):
    """Logits that grow from tile to tile and reach thousands; a weight of almost one; thresholds up to fp16's end."""
    h = Held(b, hq=4, hkv=2, seed=13, requests=1, tokens=1500)
    tau = np.full((1, 2), 65504, np.float32)
    h.cache = b.OscarCache(b.make_config(1, 4, 2, 1, 30, 30), *h.rot, tau, tau)
    r = h.cache.open()
    k, v = h.tokens(1400)
    k = (k.float() * torch.linspace(0.1, 20, 1400, device="cuda")[:, None, None]).bfloat16()
    v = (v.float() * 300).bfloat16()
    h.cache.extend(0, [r], k, v, new_lens=[1400])
    kq, vq = h.tokens(40)
    q = (h.rnd(40, 4, D)).bfloat16()
    out = torch.empty(40, 4, D, device="cuda", dtype=torch.bfloat16)
    h.cache.chunk_attention(0, [r], q, kq, vq, out, new_lens=[40])
    (kc, vc), _, _ = h.stored(r)
    p = torch.arange(1440, device="cuda")
    see = p[None] <= torch.arange(1400, 1440, device="cuda")[:, None]
    want = attend(q, torch.cat([kc, kq.double()]), torch.cat([vc, vq.double()]), see)[0]
    # logits of up to some hundred with an error of 2^-11 of their terms: weights off by a tenth at most
    assert bool(out.isfinite().all()) and off_by(out, want) < 0.1
    q[3] = float("nan")
    clean = out.clone()
    h.cache.chunk_attention(0, [r], q, kq, vq, out, new_lens=[40])
    assert bool(out[3].isnan().all())
    assert torch.equal(out[:3], clean[:3]) and torch.equal(out[4:], clean[4:])


def test_prompt_in_chunks_is_the_prompt(b):
    """Chunk by chunk, attention then extend, as a program feeds a prompt: the first two chunks see BF16 tokens only,
    so that they are prompt_attention's rows; then read gives what decode attends to."""
    h = Held(b, seed=14, requests=1, tokens=1200)
    r = h.cache.open()
    k, v = h.tokens(1000)
    q = h.rnd(1000, 8, D).bfloat16()
    out, whole = torch.empty_like(q), torch.empty_like(q)
    b.prompt_attention(q, k, v, whole, [1000])
    at = 0
    for m in (150, 170, 1, 300, 379):
        h.cache.chunk_attention(0, [r], q[at:at + m], k[at:at + m], v[at:at + m], out[at:at + m], new_lens=[m])
        h.cache.extend(0, [r], k[at:at + m], v[at:at + m], new_lens=[m])
        at += m
    h.cache.check()
    assert off_by(out[:320], whole[:320].double()) < 4e-3
    ko, vo = (torch.empty(1000, 2, D, device="cuda") for _ in range(2))
    h.cache.read(0, [r], [0], [1000], ko, vo)
    q1 = h.rnd(1, 8, D).bfloat16()
    dec = torch.empty(1, 8, D, device="cuda")
    h.cache.decode(0, [r], q1, dec, b.new_workspace(h.cache.workspace_bytes([r])))
    want = attend(q1, ko, vo, torch.ones(1, 1000, dtype=torch.bool, device="cuda"))[0]
    assert off_by(dec, want) < 5e-3


def test_pools_beyond_4_gib(b):
    pages = 130000                                          # x 8 heads x 4608 bytes = 4.8 GB
    h = Held(b, hq=8, hkv=8, seed=15, requests=2, tokens=2000, pages=pages)
    r = [h.cache.open() for _ in range(2)]
    h.cache.extend(0, r, *h.tokens(2600), new_lens=[1500, 1100])
    assert max(h.cache.pages(r[0])[0]) * 8 * 4608 > 1 << 32
    check_chunk(h, r, [20, 140])
    k, v = (torch.empty(2600, 8, D, device="cuda") for _ in range(2))
    h.cache.read(0, r, [0, 0], [1500, 1100], k, v)
    want = torch.cat([h.stored(x)[0][0] for x in r])
    assert off_by(k, want) < 1e-6


def test_captured_calls_replay(b):
    """Two chunk calls and a prompt call that share a workspace, captured on a stream of their own, replayed on new
    contents; two replays give the same bits."""
    h = Held(b, seed=16, requests=2, tokens=900)
    r = [h.cache.open() for _ in range(2)]
    h.cache.extend(0, r, *h.tokens(1500), new_lens=[800, 700])
    q, (k, v) = h.rnd(50, 8, D).bfloat16(), h.tokens(50)
    outs = [torch.empty_like(q) for _ in range(3)]
    ws = h.cache.chunk_workspace([45, 5])
    pw = b.prompt_workspace([30, 20], 8, 2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def calls():
        h.cache.chunk_attention(0, r, q, k, v, outs[0], new_lens=[45, 5], workspace=ws)
        h.cache.chunk_attention(0, r[::-1], q, k, v, outs[1], new_lens=[5, 45], workspace=ws)
        b.prompt_attention(q, k, v, outs[2], [30, 20], workspace=pw)

    with torch.cuda.stream(side):
        calls()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        calls()
    q.copy_(h.rnd(50, 8, D))
    k.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    got = [o.clone() for o in outs]
    for o in outs:
        o.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, outs))
    calls()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, outs))


def test_work_before_in_the_stream_is_seen(b):
    """q, k and v, and the cache's tokens, written by the launches right before, on another stream than the default."""
    h = Held(b, seed=17, requests=1, tokens=3000)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for n in range(6):
            r = h.cache.open()
            kc, vc = h.tokens(900 + 131 * n)
            h.cache.extend(0, [r], kc, vc, new_lens=[len(kc)])
            k, v = h.tokens(30)
            q = h.rnd(30, 8, D).bfloat16()
            out = torch.empty_like(q)
            h.cache.chunk_attention(0, [r], q, k, v, out, new_lens=[30])
            ko, vo = (torch.empty(len(kc), 2, D, device="cuda") for _ in range(2))
            h.cache.read(0, [r], [0], [len(kc)], ko, vo)
            (ks, vs), _, _ = h.stored(r)
            p = torch.arange(len(kc) + 30, device="cuda")
            see = p[None] <= torch.arange(len(kc), len(kc) + 30, device="cuda")[:, None]
            want = attend(q, torch.cat([ks, k.double()]), torch.cat([vs, v.double()]), see)[0]
            assert off_by(out, want) < 4e-3 and off_by(ko, ks) < 1e-6 and off_by(vo, vs) < 1e-6
            h.cache.close(r)


def test_bad_page_ids_are_reported(b):
    h = Held(b, seed=18, requests=1, tokens=900)
    r = h.cache.open()
    h.cache.extend(0, [r], *h.tokens(700), new_lens=[700])
    table = h.cache.device_page_table()
    good = table[r, 2].clone()
    q, (k, v) = h.rnd(3, 8, D).bfloat16(), h.tokens(3)
    out = torch.empty_like(q)
    ko, vo = (torch.empty(700, 2, D, device="cuda") for _ in range(2))
    for bad in (-1, 10 ** 9):
        for call in (lambda: h.cache.chunk_attention(0, [r], q, k, v, out, new_lens=[3]),
                     lambda: h.cache.read(0, [r], [0], [700], ko, vo)):
            table[r, 2] = bad
            call()
            with pytest.raises(b.OscarError, match="DEVICE_CHECK"):
                h.cache.check()
            table[r, 2] = good
            call()
            h.cache.check()
    at = (700 - 320) // 64
    good = table[r, at].clone()
    table[r, at] = 10 ** 9
    h.cache.extend(0, [r], *h.tokens(1), new_lens=[1])
    with pytest.raises(b.OscarError, match="DEVICE_CHECK"):
        h.cache.check()
    table[r, at] = good


def test_chunk_call_refusals(b):
    h = Held(b, seed=19, requests=2, tokens=900)
    r = [h.cache.open() for _ in range(2)]
    h.cache.extend(0, r, *h.tokens(500), new_lens=[400, 100])
    q, (k, v) = h.rnd(6, 8, D).bfloat16(), h.tokens(6)
    out = torch.empty_like(q)
    ok = dict(layer=0, reqs=r, q=q, k=k, v=v, out=out, new_lens=[2, 4])
    ws = h.cache.chunk_attention(**ok)
    for change in (dict(layer=1), dict(reqs=[r[0], 7]), dict(new_lens=[2, 3]), dict(new_lens=[6]), dict(q=q.float()),
                   dict(q=q[:, :4]), dict(k=k[:5]), dict(v=v.cpu()), dict(out=out.float()), dict(out=out.transpose(0, 1)),
                   dict(workspace=ws.float()), dict(workspace=ws[1:])):
        with pytest.raises(b.OscarError):
            h.cache.chunk_attention(**{**ok, **change})
    small = b.new_workspace(512)
    assert h.cache.chunk_attention(**{**ok, "workspace": small}).numel() > 512
    for change in (dict(k=k.float()), dict(k=k[:5]), dict(reqs=[r[0], r[0]]), dict(new_lens=[7, -1]), dict(layer=-1)):
        with pytest.raises(b.OscarError):
            h.cache.extend(**{**dict(layer=0, reqs=r, k=k, v=v, new_lens=[2, 4]), **change})
    ko = torch.empty(6, 2, D, device="cuda")
    for change in (dict(starts=[399, 0]), dict(k_out=ko.half(), v_out=ko.half()), dict(v_out=ko.bfloat16()), dict(counts=[2, 5]),
                   dict(k_out=ko[:5], v_out=ko[:5])):
        with pytest.raises(b.OscarError):
            h.cache.read(**{**dict(layer=0, reqs=r, starts=[3, 0], counts=[2, 4], k_out=ko, v_out=ko), **change})
    assert h.cache.length(r[0], 0) == (400, 144) and h.cache.length(r[1], 0) == (100, 64)
    # nothing to do
    none = torch.empty(0, 8, D, device="cuda", dtype=torch.bfloat16)
    h.cache.chunk_attention(0, r, none, none[:, :2], none[:, :2], none, new_lens=[0, 0])
    h.cache.extend(0, r, none[:, :2], none[:, :2], new_lens=[0, 0])
    h.cache.read(0, r, [0, 0], [0, 0], none[:, :2].contiguous(), none[:, :2].contiguous())
    h.cache.check()
    assert h.cache.length(r[0], 0) == (400, 144)


def test_calls_without_the_extension_are_the_same(b, monkeypatch):
    h = Held(b, seed=20, requests=2, tokens=900)
    q, (k, v) = h.rnd(9, 8, D).bfloat16(), h.tokens(9)
    kc, vc = h.tokens(600)
    got = []
    for fast in (True, False):
        if not fast:
            monkeypatch.setattr(b, "_calls", b._NotBuilt)
        r = h.cache.open()
        h.cache.extend(0, [r], kc, vc, new_lens=[600])
        out, ko, vo = torch.empty_like(q), torch.empty(600, 2, D, device="cuda"), torch.empty(600, 2, D, device="cuda")
        h.cache.chunk_attention(0, [r], q, k, v, out, new_lens=[9])
        h.cache.read(0, [r], [0], [600], ko, vo)
        two = torch.empty_like(q)
        b.prompt_attention(q, k, v, two, [4, 5])
        got.append((out, ko, vo, two))
        h.cache.close(r)
    assert all(torch.equal(x, y) for x, y in zip(*got))


@pytest.mark.parametrize("group", [128, 64])
def test_thresholds_far_above_the_values(b, group):
    """Thresholds that clip nothing, whatever the values' size: what is lost is relative to the values, not to them."""
    h = Held(b, group=group, seed=21, requests=2, tokens=1600)
    for size in (2.0 ** -9, 1.0, 2.0 ** 9):
        tau = np.full((1, 2), 65504, np.float32)
        h.cache = b.OscarCache(b.make_config(1, 8, 2, 2, 30, 60, group_size=group), *h.rot, tau, tau)
        r = [h.cache.open() for _ in range(2)]
        k, v = h.tokens(1500)
        v = (v * size).bfloat16()
        h.cache.extend(0, r, k, v, new_lens=[1300, 200])
        for lens in ([5], [200]):
            m = lens[0]
            kn, vn = h.tokens(m)
            q, vn = (h.rnd(m, 8, D) / 4).bfloat16(), (vn * size).bfloat16()
            out = torch.empty_like(q)
            h.cache.chunk_attention(0, r[:1], q, kn, vn, out, new_lens=lens)
            (kc, vc), _, _ = h.stored(r[0])
            p = torch.arange(1300 + m, device="cuda")
            see = p[None] <= torch.arange(1300, 1300 + m, device="cuda")[:, None]
            want = attend(q, torch.cat([kc, kn.double()]), torch.cat([vc, vn.double()]), see)[0]
            assert off_by(out, want) < 4e-3, (size, m, off_by(out, want))
        ko, vo = (torch.empty(1300, 2, D, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        h.cache.read(0, r[:1], [0], [1300], ko, vo)
        assert off_by(ko, kc) < 3e-3 and off_by(vo, vc) < 3e-3, (size, off_by(ko, kc), off_by(vo, vc))
        h.cache.check()


@pytest.mark.parametrize("group", [128, 64])
def test_values_of_many_sizes(b, group):
    """Values whose size changes along the request by up to 2^12, and with it their weight in the sum."""
    h = Held(b, group=group, seed=22, requests=1, tokens=1600)
    tau = np.full((1, 2), 65504, np.float32)
    h.cache = b.OscarCache(b.make_config(1, 8, 2, 1, 30, 30, group_size=group), *h.rot, tau, tau)
    r = h.cache.open()
    k, v = h.tokens(1500)
    v = (v * torch.exp2(torch.randint(-12, 1, (47,), device="cuda").repeat_interleave(32)[:1500].float())[:, None, None]).bfloat16()
    h.cache.extend(0, [r], k, v, new_lens=[1500])
    for m in (3, 150):
        kn, vn = h.tokens(m)
        q, vn = (h.rnd(m, 8, D) / 4).bfloat16(), (vn / 4096).bfloat16()
        out = torch.empty_like(q)
        h.cache.chunk_attention(0, [r], q, kn, vn, out, new_lens=[m])
        (kc, vc), _, _ = h.stored(r)
        p = torch.arange(1500 + m, device="cuda")
        see = p[None] <= torch.arange(1500, 1500 + m, device="cuda")[:, None]
        want = attend(q, torch.cat([kc, kn.double()]), torch.cat([vc, vn.double()]), see)[0]
        assert off_by(out, want) < 4e-3
    h.cache.check()


def test_values_that_are_not_finite(b):
    """Infinities and NaN among the new tokens: what appends write; another request's rows do not see them."""
    one, two = (Held(b, seed=23, tokens=900) for _ in range(2))
    r = [one.cache.open() for _ in range(2)]
    assert r == [two.cache.open() for _ in range(2)]
    k, v = one.tokens(1000)
    k[100, 0, 3], k[130, 1, 7], v[90, 0, 0], v[140] = math.inf, -math.inf, math.nan, -math.inf
    one.cache.extend(0, r, k, v, new_lens=[600, 400])
    for i in range(600):
        some = r if i < 400 else r[:1]
        rows = [i, 600 + i][:len(some)]
        two.cache.append(0, some, k[rows].contiguous(), v[rows].contiguous())
    one.cache.check()
    for x in r:
        pa, pb = one.cache.pages(x)[0], two.cache.pages(x)[0]
        he = one.cache.length(x, 0)[1] - 64
        for i, (p, q) in enumerate(zip(pa, pb)):
            rows = min(64, he - 64 * i)
            for at, w in ((0, 32), (2048, 32), (4096, 4), (4352, 4)):
                a, c = one.cache.int2_pool(0)[p, :, at:at + rows * w], two.cache.int2_pool(0)[q, :, at:at + rows * w]
                assert torch.equal(a, c), (x, i, at, (a != c).nonzero()[:8].tolist())
    kn, vn = one.tokens(90)
    q = one.rnd(90, 8, D).bfloat16()
    out = torch.empty_like(q)
    one.cache.chunk_attention(0, r, q, kn, vn, out, new_lens=[30, 60])
    clean = out.clone()
    kn[30:], vn[30:], q[30:] = math.nan, math.nan, math.nan
    one.cache.chunk_attention(0, r, q, kn, vn, out, new_lens=[30, 60])
    assert torch.equal(out[:30].view(torch.int16), clean[:30].view(torch.int16))


@pytest.mark.parametrize("group", [128, 64])
@pytest.mark.parametrize("m", [8, 9, 16, 17, 32, 33])
def test_chunk_rows_at_the_borders_of_the_forms(b, m, group):
    """64 and 72 rows a kv head (8 to a token), 128 and 136, 256 and 264."""
    h = Held(b, hq=16, hkv=2, group=group, seed=24 + m, requests=2, tokens=3500)
    r = [h.cache.open() for _ in range(2)]
    h.cache.extend(0, r, *h.tokens(3300 + 500), new_lens=[3300, 500])
    check_chunk(h, r, [m, m])
    check_chunk(h, r[:1], [m])


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 1), (96, 96), (160, 160)])
def test_chunk_any_number_of_heads(b, hq, hkv):
    h = Held(b, hq=hq, hkv=hkv, seed=hq, requests=2, tokens=800)
    r = [h.cache.open() for _ in range(2)]
    h.cache.extend(0, r, *h.tokens(1000), new_lens=[650, 350])
    check_chunk(h, r, [3, 1])
    check_chunk(h, r, [200, 2])
    k, v = (torch.empty(1000, hkv, D, device="cuda") for _ in range(2))
    h.cache.read(0, r, [0, 0], [650, 350], k, v)
    want = torch.cat([h.stored(x)[0][1] for x in r])
    assert off_by(v, want) < 1e-6


def test_chunk_queries_of_any_size(b):
    """Zeros (the mean of all values), tiny and huge queries beside ordinary ones, each its own scale."""
    h = Held(b, seed=30, requests=1, tokens=1200)
    r = h.cache.open()
    h.cache.extend(0, [r], *h.tokens(1111), new_lens=[1111])
    (kc, vc), _, _ = h.stored(r)
    for m in (4, 80):
        kn, vn = h.tokens(m)
        q = h.rnd(m, 8, D).bfloat16()
        q[0] = 0
        q[1] *= 2.0 ** -60
        q[2] = (q[2].float() * 2.0 ** -130).bfloat16()
        q[3, ::2] *= 2.0 ** 40
        out = torch.empty_like(q)
        h.cache.chunk_attention(0, [r], q, kn, vn, out, new_lens=[m])
        p = torch.arange(1111 + m, device="cuda")
        see = p[None] <= torch.arange(1111, 1111 + m, device="cuda")[:, None]
        want = attend(q, torch.cat([kc, kn.double()]), torch.cat([vc, vn.double()]), see)[0]
        for i in range(m):
            # logits of 2^40: one weight is 1, and which one it is fp32 decides where two are 2^-11 apart
            if i != 3:
                assert off_by(out[i], want[i]) < 2e-2, (m, i, off_by(out[i], want[i]))
        assert bool(out.isfinite().all())
        seen = torch.cat([vc, vn.double()]).abs().amax(0)
        assert bool((out[3].double().abs() <= 1.01 * seen.repeat_interleave(4, 0).view(8, D)).all())
    h.cache.check()


@pytest.mark.parametrize("out_type", [torch.bfloat16, torch.float32])
def test_prompt_queries_of_any_size(b, out_type):
    """Logits far beyond fp32's whole numbers: one key has the weight, and rows beside them are what they were."""
    rnd = rand(31)
    q, k, v = rnd(150, 8, D).bfloat16(), rnd(150, 2, D).bfloat16(), rnd(150, 2, D).bfloat16()
    out = torch.empty(150, 8, D, device="cuda", dtype=out_type)
    b.prompt_attention(q, k, v, out, [150])
    clean = out.clone()
    huge = q.clone()
    huge[40], huge[90] = huge[40] * 2.0 ** 40, huge[90] * 2.0 ** 90
    b.prompt_attention(huge, k, v, out, [150])
    rest = [i for i in range(150) if i not in (40, 90)]
    assert torch.equal(out[rest], clean[rest])
    see = torch.ones(150, 150, device="cuda").tril().bool()
    want = attend(huge, k, v, see)[0]
    # the two largest logits of a row are 2^-24 of them apart nowhere here
    assert off_by(out[[40, 90]], want[[40, 90]]) < (1e-6 if out_type == torch.float32 else 3e-3)


def unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def unclipped(b, h, tokens, threshold=65504):
    """One request of thresholds that clip nothing."""
    tau = np.full((1, h.hkv), threshold, np.float32)
    h.cache = b.OscarCache(b.make_config(1, h.hq, h.hkv, 1, tokens // 64 + 1, tokens // 64 + 1, group_size=h.group), *h.rot, tau, tau)
    h.cache.int2_pool(0).fill_(255)
    return h.cache.open()


@pytest.mark.parametrize("group", [128, 64])
@pytest.mark.parametrize("threshold", [65504, 160])
@pytest.mark.parametrize("m", [5, 30, 200])
def test_chunk_large_logits_keep_their_order(b, m, threshold, group):
    """The best key is a history token among long ones; a token of a tile of short ones, or one of the recent window or
    of the chunk, lies closer to the query's direction.  With queries of 2^10 to 2^100 the best key has all the weight: its
    logit is ahead by 2^-5 of the longest key's length times the query's or more, where the roundings of q R_K and of the
    keys are 2^-11 each.  Each row against float64, and ordinary rows beside them have the bits that they had."""
    h = Held(b, group=group, seed=40 + m, requests=1, tokens=1400)
    t, he = 1111, 855
    r = unclipped(b, h, t, threshold)
    length = torch.full((t,), 32.0, device="cuda")
    tile = (torch.arange(t, device="cuda") - 64) // 128
    length[(tile % 2 == 0) & (torch.arange(t, device="cuda") >= 64) & (torch.arange(t, device="cuda") < he)] = 256
    k = (unit(h.rnd(t, 2, D)) * length[:, None, None]).bfloat16()
    h.cache.extend(0, [r], k, h.tokens(t)[1], new_lens=[t])
    assert h.cache.length(r, 0) == (t, he)
    (kc, vc), (_, vm), _ = h.stored(r)
    kn, vn = (unit(h.rnd(m, 2, D)) * 32).bfloat16(), h.tokens(m)[1]
    keys, values, mags = (torch.cat(x) for x in ((kc, kn.double()), (vc, vn.double()), (vm, vn.double().abs())))
    p = torch.arange(t + m, device="cuda")
    see = p[None] <= torch.arange(t, t + m, device="cuda")[:, None]
    # per row and head: its best key, and one that lies closer to it
    rng = np.random.default_rng(m + group)
    short = [x for x in range(64, he) if (x - 64) // 128 % 2]
    long = [x for x in range(64, he) if (x - 64) // 128 % 2 == 0]
    best = torch.tensor(rng.choice(long, (m, 8)), device="cuda")
    far = torch.tensor(rng.choice(short, (m, 8)), device="cuda")
    near = torch.tensor([[int(rng.integers(he, t + i + 1)) for _ in range(8)] for i in range(m)], device="cuda")
    head = torch.arange(8, device="cuda") // 4
    other = torch.where(head == (torch.arange(m, device="cuda") // 2 % 2)[:, None], far, near)
    to = unit(keys)
    w, d = to[best, head], to[other, head]
    q = ((0.55 * w + 0.82 * unit(d - (d * w).sum(-1, keepdim=True) * w)) * 11).bfloat16()
    plain = (h.rnd(m, 8, D) / 16).bfloat16()   # ordinary rows: weights of many keys
    ordinary = torch.arange(m, device="cuda") % 4 == 1
    q[ordinary] = plain[ordinary]

    def run(q):
        out = torch.full((m, 8, D), float("nan"), device="cuda", dtype=torch.bfloat16)
        h.cache.chunk_attention(0, [r], q, kn, vn, out, new_lens=[m])
        h.cache.check()
        return out

    clean = run(plain)
    logit = torch.einsum("mhd,thd->mht", q.double(), keys.repeat_interleave(4, 1)).masked_fill(~see[:, None], -math.inf)
    top = logit.topk(2, -1)
    ahead = (top.values[..., 0] - top.values[..., 1]) / (q.double().norm(dim=-1) * keys.norm(dim=-1).max())
    big = ~ordinary
    assert torch.equal(top.indices[big][..., 0], best[big]) and float(ahead[big].min()) > 2 ** -5
    closer = torch.einsum("mhd,mhd->mh", q.double(), d) > torch.einsum("mhd,mhd->mh", q.double(), w)
    assert bool(closer[big].all())
    for e in (10, 13, 16, 20, 40, 100):
        x = torch.where(ordinary[:, None, None], q.float(), q.float() * 2.0 ** e).bfloat16()
        out = run(x)
        want, mag = attend(x, keys, values, see)[0], attend(x, keys, mags, see)[0]
        # one value: it, R_V, its weight and the sum that is rotated back in fp16; 2^-15 of its tile's largest, some 4
        # deviations, by the 11 that |R_V| sums, where mag is some 8 deviations: below 2^-12; and the result in bf16
        tol = (4 * 2 ** -11 + 2 ** -12) * mag + 2 ** -8 * want.abs()
        bad = ((out.double() - want).abs() > tol).flatten(1).any(-1) & big
        wrong = int(bad.sum())
        assert wrong == 0, (e, wrong, int(big.sum()))
        assert off_by(out[big], want[big]) < 4e-3
        assert torch.equal(out[ordinary].view(torch.int16), clean[ordinary].view(torch.int16)), e


@pytest.mark.parametrize("group", [128, 64])
@pytest.mark.parametrize("m", [5, 200])
def test_small_values_beside_large_ones(b, m, group):
    """Rows whose weight lies on one history token whose value is 2^-6 to 2^-12 of its tile's largest: fp16's 2^-11 of the
    value, and 2^-15 of that largest."""
    h = Held(b, group=group, seed=50 + m, requests=1, tokens=1400)
    t, he = 1111, 855
    r = unclipped(b, h, t)
    k, v = (unit(h.rnd(t, 2, D)) * 11).bfloat16(), h.rnd(t, 2, D)
    small = torch.arange(t, device="cuda") % 3 == 0
    v = torch.where(small[:, None, None], v * torch.exp2(-6.0 - 2 * (torch.arange(t, device="cuda") // 3 % 4))[:, None, None], v).bfloat16()
    h.cache.extend(0, [r], k, v, new_lens=[t])
    assert h.cache.length(r, 0) == (t, he)
    (kc, vc), (_, vm), _ = h.stored(r)
    kn, vn = (unit(h.rnd(m, 2, D)) * 11).bfloat16(), h.rnd(m, 2, D).bfloat16()
    best = torch.tensor(np.random.default_rng(m + group).choice([x for x in range(64, he) if x % 3 == 0], (m, 8)), device="cuda")
    head = torch.arange(8, device="cuda") // 4
    # (logits of 15 the best key's length, others' at most half of that: weights below 2^-30)
    q = (unit(kc[best, head]) * 11 * 16).bfloat16()
    out = torch.full((m, 8, D), float("nan"), device="cuda", dtype=torch.bfloat16)
    h.cache.chunk_attention(0, [r], q, kn, vn, out, new_lens=[m])
    h.cache.check()
    p = torch.arange(t + m, device="cuda")
    see = p[None] <= torch.arange(t, t + m, device="cuda")[:, None]
    keys, values = torch.cat([kc, kn.double()]), torch.cat([vc, vn.double()])
    logit = torch.einsum("mhd,thd->mht", q.double(), keys.repeat_interleave(4, 1)).masked_fill(~see[:, None], -math.inf)
    top = logit.topk(2, -1)
    assert torch.equal(top.indices[..., 0], best) and float((top.values[..., 0] - top.values[..., 1]).min()) / math.sqrt(D) > 30
    want = attend(q, keys, values, see)[0]
    # the largest rotated value of each tile, and what rotating it back sums of 2^-15 of it
    rot = h.rot[1][0].double()
    y = torch.einsum("thi,hij->thj", vc[64:he], rot).abs().amax(-1)
    most = torch.stack([y[64 * (2 * i):64 * (2 * i + 2)].amax(0) for i in range((he - 64 + 127) // 128)])   # [tiles][hkv]
    reach = rot.abs().sum(-1)                                                                               # [hkv][128]
    tile = (best - 64) // 128
    tol = (4 * 2 ** -11) * vm[best, head] + 2 ** -8 * want.abs() + 2 ** -15 * most[tile, head][..., None] * reach[head]
    assert bool(((out.double() - want).abs() <= tol).all()), float(((out.double() - want).abs() / tol).max())
