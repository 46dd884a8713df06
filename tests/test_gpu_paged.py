"""Paged-cache operators against the float64 oracle: append with position rotation
(bit for bit), the 4-bit cache, attention with a sliding window and sinks.

Pools start as NaN bit patterns (BF16) or 0xFF bytes (4 bits: NaN scales), pages
are shuffled, and the table entries of pages that no query sees are -1, so any
read of what a call must not see shows as a NaN or in the error word.

Tolerances of the attention, per output value, relative to sum p |v| (a weight's
relative error multiplies p |v|; normalising doubles it).  A 4-bit value s c + z is
summed in two parts, about the middle of its codes; without that care s c = x - z is at
most |x| + |z|, so |x| + 2 |z| stands for |x|:
  logit   each of 128 products is exact, their sum takes 8 steps of a fp32 matrix
          accumulator, at most 2^-22 of the running magnitude each (truncated, and
          aligned to the largest product): 8 2^-22 max |q| |k| scale; in 4 bits three
          more roundings (scale, product, sum), counted by doubling;
  weight  ex2 2^-22, and p's parts: three bf16 parts leave 2^-24, two fp16 parts
          2^-21; one bf16 part (long bf16 outputs) leaves 2^-8;
  sums    one rounding of 2^-22 per 16 tokens of a warp's share, 64 to fold.
A bf16 output adds 2^-8 of itself.
"""
import math

import numpy as np
import pytest

from oracle import paged

torch = pytest.importorskip("torch")
PAGE, D = 64, 128


@pytest.fixture(scope="module")
def b():
    from bit_rotated_kv_decode_gb300 import binding, build
    build.build()
    binding.load()
    return binding


class Pool:
    """A BF16 (group 0) or 4-bit pool with known keys and values, host and device."""

    def __init__(self, b, lens, hkv, group=0, seed=0, visible=None, spare=3):
        g = np.random.default_rng(seed)
        self.lens, self.hkv, self.group = lens, hkv, group
        need = [-(-t // PAGE) for t in lens]
        self.pages = sum(need) + spare
        order = g.permutation(self.pages)
        self.table = np.full((len(lens), max(1, max(need))), -1, np.int32)
        at = 0
        for i, m in enumerate(need):
            self.table[i, :m] = order[at:at + m]
            at += m
        if group == 0:
            self.host = np.full((self.pages, hkv, 2, PAGE, D), 0x7FFF, np.uint16)
        else:
            self.host = np.full((self.pages, hkv, paged.record_bytes(group)), 0xFF, np.uint8)
        self.k, self.v, self.kmag, self.vmag = [], [], [], []
        for i, t in enumerate(lens):
            k = g.standard_normal((t, hkv, D)).astype(np.float32)
            k[:, :, 5] *= 6
            v = (g.standard_normal((t, hkv, D)) * np.exp(0.5 * g.standard_normal((t, hkv, 1)))).astype(np.float32)
            kb, vb = paged.bf16_bits(k), paged.bf16_bits(v)
            if group == 0:
                kf, vf = paged.bf16_values(kb).astype(np.float64), paged.bf16_values(vb).astype(np.float64)
                for t0 in range(0, t, PAGE):
                    page, m = self.table[i, t0 // PAGE], min(PAGE, t - t0)
                    self.host[page, :, 0, :m] = kb[t0:t0 + m].transpose(1, 0, 2)
                    self.host[page, :, 1, :m] = vb[t0:t0 + m].transpose(1, 0, 2)
            else:
                (kc, km), (vc, vm) = paged.quantise4(kb, group), paged.quantise4(vb, group)
                kf, vf = paged.dequantise4(kc, km), paged.dequantise4(vc, vm)
                kz, vz = (np.repeat(np.abs(m[..., 1].astype(np.float64)), group, -1) for m in (km, vm))
                for tok in range(t):
                    for h in range(hkv):
                        rec = self.host[self.table[i, tok // PAGE], h]
                        paged.put4(rec, 0, tok % PAGE, kc[tok, h], km[tok, h])
                        paged.put4(rec, 1, tok % PAGE, vc[tok, h], vm[tok, h])
            self.k.append(kf)
            self.v.append(vf)
            self.kmag.append(np.abs(kf) + (2 * kz if group else 0))
            self.vmag.append(np.abs(vf) + (2 * vz if group else 0))

    def hide(self, q_lens, window, sinks):
        """Poison what no query of a request sees: -1 for whole pages, NaN for tokens (as a fresh pool holds)."""
        table = self.table.copy()
        for i, (t, m) in enumerate(zip(self.lens, q_lens)):
            vis = np.zeros(t, bool)
            for p in range(t - m, t):
                vis[paged.seen(p, window, sinks)] = True
            for page in range(-(-t // PAGE)):
                rows = vis[page * PAGE:(page + 1) * PAGE]
                if not rows.any():
                    table[i, page] = -1
                    continue
                if self.group == 0:
                    for r in np.nonzero(~rows)[0]:
                        self.host[self.table[i, page], :, :, r] = 0x7FC0
                else:
                    ng = D // self.group
                    for r in np.nonzero(~rows)[0]:
                        at = PAGE * D + r * 4 * ng
                        for which in range(2):
                            o = at + which * PAGE * 4 * ng
                            self.host[self.table[i, page], :, o:o + 4 * ng] = 0xFF
        self.table = table

    def device(self):
        kv = torch.from_numpy(self.host.view(np.int16) if self.group == 0 else self.host).cuda()
        return kv.view(torch.bfloat16) if self.group == 0 else kv, torch.from_numpy(self.table).cuda()


def bf16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).cuda()


def tolerance(out, mag, logit, tokens, four, one_part, out_bf16):
    weight = 2.0 ** -22 + (2.0 ** -8 if one_part else 2.0 ** -21 if four else 2.0 ** -24)
    rel = 2 * ((2 if four else 1) * 8 * 2.0 ** -22 * logit + weight) + 2.0 ** -22 * (tokens / 16 + 64)
    return rel * mag + (2.0 ** -8 * np.abs(out) if out_bf16 else 0)


def check_attention(pool, q, q_lens, window, sinks, got, lse, scale=0.0, one_part=lambda m: False):
    scale = scale if scale > 0 else 1 / math.sqrt(D)
    out_bf16 = got.dtype == torch.bfloat16
    got, lse = got.double().cpu().numpy(), lse.double().cpu().numpy()
    qf = paged.bf16_values(q).astype(np.float64)
    g = q.shape[1] // pool.hkv
    row = 0
    for i, (t, m) in enumerate(zip(pool.lens, q_lens)):
        for p in range(t - m, t):
            for h in range(q.shape[1]):
                out, ls, mag, logit = paged.attend(qf[row, h], pool.k[i][:, h // g], pool.v[i][:, h // g], p, window,
                                                   sinks, scale, pool.kmag[i][:, h // g], pool.vmag[i][:, h // g])
                n = len(paged.seen(p, window, sinks))
                tol = tolerance(out, mag, logit, n, pool.group, one_part(m), out_bf16)
                bad = ~(np.abs(got[row, h] - out) <= tol)
                assert not bad.any(), (i, p, h, np.abs(got[row, h] - out)[bad].max(), tol[bad].min())
                if ls == -np.inf:
                    assert lse[row, h] == -np.inf
                else:
                    assert abs(lse[row, h] - ls) <= 2 * 8 * 2.0 ** -22 * logit + 2.0 ** -20 + 2.0 ** -22 * (n / 16 + 64)
            row += 1


def run_attention(b, pool, q_lens, hq, window, sinks, out_dtype=torch.float32, seed=1, scale=0.0, workspace=None,
                  one_part=lambda m: False):
    rows = sum(q_lens)
    q = paged.bf16_bits(np.random.default_rng(seed).standard_normal((rows, hq, D)).astype(np.float32))
    pool.hide(q_lens, window, sinks)
    kv, table = pool.device()
    out = torch.full((rows + 1, hq, D), 7.0, dtype=out_dtype, device="cuda")
    lse = torch.full((rows + 1, hq), 7.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = dict(q_lens=q_lens, lse=lse[:rows], error=err, scale=scale, workspace=workspace)
    if pool.group:
        ws = b.int4_attention(kv, table, pool.lens, bf16(q), out[:rows], pool.hkv, window, sinks,
                              group_size=pool.group, **args)
    else:
        ws = b.window_attention(kv, table, pool.lens, bf16(q), out[:rows], pool.hkv, window, sinks, **args)
    torch.cuda.synchronize()
    assert err.item() == 0
    assert (out[rows] == 7).all() and (lse[rows] == 7).all()          # rows behind the last are left as they were
    assert int(ws[:65536].view(torch.int32).abs().sum()) == 0         # the merge counters are back at zero
    check_attention(pool, q, q_lens, window, sinks, out[:rows], lse[:rows], scale, one_part)
    return ws


# ---- decode: every group size, ragged lengths, windows, sinks ------------------
DECODE = [
    # lens, window, sinks
    ([1], -1, 0),
    ([1, 63, 64, 65, 16, 17], -1, 0),
    ([1000, 37, 4133], -1, 0),
    ([1000, 5, 4133, 320], 256, 64),
    ([777, 130, 129, 2500], 100, 4),
    ([500, 3], 1, 0),
    ([300, 64, 65], 0, 64),
    ([300, 1], 0, 0),
    ([200, 90], 50, 1000),
    ([2000], 333, 70),
]


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv", [(8, 2), (2, 2), (2, 1), (16, 2)])
@pytest.mark.parametrize("lens,window,sinks", DECODE)
def test_window_decode(b, hq, hkv, lens, window, sinks):
    run_attention(b, Pool(b, lens, hkv, seed=len(lens) + hq), [1] * len(lens), hq, window, sinks)


@pytest.mark.gpu
@pytest.mark.parametrize("group", [128, 64])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (1, 1), (4, 2), (8, 1)])
@pytest.mark.parametrize("lens,window,sinks", [c for c in DECODE if sum(c[0]) < 4500])
def test_int4_decode(b, group, hq, hkv, lens, window, sinks):
    run_attention(b, Pool(b, lens, hkv, group, seed=len(lens) + hq), [1] * len(lens), hq, window, sinks)


@pytest.mark.gpu
@pytest.mark.parametrize("group", [0, 128, 64])
@pytest.mark.parametrize("hq,hkv,q_lens", [(4, 1, [4, 2, 0, 1]), (8, 1, [2, 1, 0, 2]), (2, 2, [16, 7, 0, 3]),
                                           (4, 2, [3, 8, 0, 5])])
def test_a_few_query_tokens(b, group, hq, hkv, q_lens):
    lens = [300, 70, 0, 129]
    run_attention(b, Pool(b, lens, hkv, group, seed=hq), q_lens, hq, -1, 0)
    run_attention(b, Pool(b, lens, hkv, group, seed=hq), q_lens, hq, 40, 5, torch.bfloat16, scale=0.2)


@pytest.mark.gpu
@pytest.mark.parametrize("group", [0, 128])
def test_many_short_requests_and_a_long_one(b, group):
    # more segments than CTAs, then one segment over many CTAs, on one workspace
    lens = [1 + (37 * i) % 200 for i in range(90)]
    ws = run_attention(b, Pool(b, lens, 2, group, seed=5), [1] * 90, 4, -1, 0)
    lens = [9001 if group == 0 else 5001]
    run_attention(b, Pool(b, lens, 1, group, seed=6), [1], 4, -1, 0, workspace=ws)
    run_attention(b, Pool(b, [150] * 70, 2, group, seed=7), [1] * 70, 4, 64, 3, workspace=ws)


@pytest.mark.gpu
@pytest.mark.parametrize("hq", [8, 16, 32])
def test_long_shares(b, hq):
    """More segments than CTAs, each with more tokens than a CTA sums up at once (up to 8 rows); the requests share
    their pages.  A warp's sums are over 4096 tokens at most, or over an eighth of the segment (16 rows)."""
    n, hkv, top = 84, 2, 40000
    m = 2 if hq == 32 else 1                                  # 4, 8 and 16 rows
    hq = 16 if hq == 32 else hq
    pool = Pool(b, [top], hkv, seed=13)
    lens = [top - 61 * i for i in range(n)]
    kv, table = pool.device()
    bits = paged.bf16_bits(np.random.default_rng(13).standard_normal((n * m, hq, D)).astype(np.float32))
    out, lse = torch.empty(n * m, hq, D, device="cuda"), torch.empty(n * m, hq, device="cuda")
    b.window_attention(kv, table.expand(n, -1).contiguous(), lens, bf16(bits), out, hkv, q_lens=[m] * n, lse=lse)
    qf, out, lse = paged.bf16_values(bits).astype(np.float64), out.double().cpu().numpy(), lse.double().cpu().numpy()
    for i in (0, 1, 40, 83):
        for h in (0, hq - 1):
            row, kh = i * m + m - 1, h // (hq // hkv)
            want, ls, mag, logit = paged.attend(qf[row, h], pool.k[0][:, kh], pool.v[0][:, kh], lens[i] - 1, -1, 0,
                                                1 / math.sqrt(D), pool.kmag[0][:, kh], pool.vmag[0][:, kh])
            tol = tolerance(want, mag, logit, 4096 if m == 1 else top / 8, 0, False, False)
            assert (np.abs(out[row, h] - want) <= tol).all()
            assert abs(lse[row, h] - ls) <= 2 * 8 * 2.0 ** -22 * logit + 2.0 ** -20 + 2.0 ** -22 * (4096 / 16 + 64)


@pytest.mark.gpu
@pytest.mark.parametrize("group", [0, 128, 64])
def test_extreme_queries_and_scales(b, group):
    """A zero query under a tiny scale (equal weights), large and small queries in one batch."""
    hq, hkv, lens = 4, 1, [100, 70, 90]
    pool = Pool(b, lens, hkv, group, seed=8)
    x = np.random.default_rng(8).standard_normal((3, hq, D)).astype(np.float32)
    x[0] = 0
    x[1] *= 2.0 ** -40
    x[2] *= 8
    q = paged.bf16_bits(x)
    pool.hide([1] * 3, 50, 3)
    kv, table = pool.device()
    for scale in (1e-30, 0.0):
        out, lse = torch.empty(3, hq, D, device="cuda"), torch.empty(3, hq, device="cuda")
        args = (kv, table, lens, bf16(q), out, hkv, 50, 3)
        if group:
            b.int4_attention(*args, group_size=group, lse=lse, scale=scale)
        else:
            b.window_attention(*args, lse=lse, scale=scale)
        check_attention(pool, q, [1] * 3, 50, 3, out, lse, scale)


@pytest.mark.gpu
@pytest.mark.parametrize("group,m,t,out_dtype", [(0, 1, 300, "f32"), (0, 4, 3000, "f32"), (0, 100, 300, "f32"),
                                                 (0, 100, 300, "bf16"), (0, 70, 2500, "f32"), (0, 70, 2500, "bf16"),
                                                 (128, 1, 300, "f32"), (64, 4, 3000, "f32")])
def test_rows_that_are_not_finite_keep_to_themselves(b, group, m, t, out_dtype):
    """A NaN and an infinite query row: every other row has the bits that it has without them."""
    hq, hkv, window = 8, 2, 90 if t == 300 else -1
    pool = Pool(b, [t], hkv, group, seed=10)
    pool.hide([m], window, 3)
    kv, table = pool.device()
    q = torch.randn(m, hq, D, device="cuda", generator=torch.Generator("cuda").manual_seed(4)).to(torch.bfloat16)
    bad = q.clone()
    bad[m // 2, 1, 5] = float("nan")
    bad[m - 1, 6, 70] = float("inf")
    outs = []
    for x in (q, bad):
        out = torch.empty(m, hq, D, dtype=torch.float32 if out_dtype == "f32" else torch.bfloat16, device="cuda")
        lse = torch.empty(m, hq, device="cuda")
        args = (kv, table, [t], x, out, hkv, window, 3)
        if group:
            b.int4_attention(*args, q_lens=[m], group_size=group, lse=lse)
        else:
            b.window_attention(*args, q_lens=[m], lse=lse)
        outs.append((out, lse))
    (o0, l0), (o1, l1) = outs
    same = torch.ones(m, hq, dtype=torch.bool, device="cuda")
    same[m // 2, 1] = same[m - 1, 6] = False
    assert torch.equal(o0[same], o1[same]) and torch.equal(l0[same], l1[same])
    assert o1[m // 2, 1].isnan().all()


@pytest.mark.gpu
def test_two_threads_on_streams_of_their_own(b):
    """Calls from two threads at once, each with its stream, workspace and outputs."""
    import threading
    hq, hkv, lens = 8, 2, [2000, 300, 900]
    pool = Pool(b, lens, hkv, seed=11)
    pool.hide([1] * 3, 700, 5)
    kv, table = pool.device()
    bits = paged.bf16_bits(np.random.default_rng(11).standard_normal((3, hq, D)).astype(np.float32))
    q, got, wrong = bf16(bits), {}, []
    torch.cuda.synchronize()

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                out, lse, ws = torch.empty(3, hq, D, device="cuda"), torch.empty(3, hq, device="cuda"), None
                for k in range(50):
                    ws = b.window_attention(kv, table, lens, q, out, hkv, 700, 5, lse=lse, workspace=ws)
                    if k % 7 == i:
                        try:
                            b.window_attention(kv, table, lens, q, out, hkv, 700, -1 - i, workspace=ws)
                        except b.OscarError as e:
                            assert "sinks" in str(e)
                torch.cuda.current_stream().synchronize()
                got[i] = (out, lse)
        except Exception as e:   # to the test's thread
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not wrong, wrong
    for out, lse in got.values():
        check_attention(pool, bits, [1] * 3, 700, 5, out, lse)


# ---- prefill --------------------------------------------------------------------
PREFILL = [
    # lens, q_lens, window, sinks
    ([100], [100], -1, 0),
    ([513], [513], -1, 0),
    ([40, 300, 1, 257], [40, 300, 1, 130], -1, 0),
    ([700, 65, 333], [90, 65, 1], 128, 64),
    ([600], [600], 100, 4),
    ([600], [300], 1, 0),
    ([300, 200], [33, 150], 0, 70),
    ([300], [40], 0, 0),
    ([900], [200], 130, 200),
    # few rows on many keys: the keys are split
    ([2500, 40], [20, 40], -1, 0),
    ([2500], [70], 1500, 10),
    ([1300, 1100], [40, 18], 0, 3),
]


@pytest.mark.gpu
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_more_items_than_ctas(b, out):
    """Prefill of more items than the GPU has SMs (bf16: of one and of two tiles), then a small one, on one workspace."""
    lens = [70 + 13 * i % 90 for i in range(100)]
    kind = dict(out_dtype=torch.float32 if out == "f32" else torch.bfloat16, one_part=lambda m: out == "bf16")
    ws = run_attention(b, Pool(b, lens, 2, seed=3), lens, 4, 60, 3, **kind)
    run_attention(b, Pool(b, [300], 1, seed=4), [300], 4, -1, 0, workspace=ws, **kind)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv", [(4, 1), (2, 2), (8, 1), (2, 1)])
@pytest.mark.parametrize("lens,q_lens,window,sinks", PREFILL)
def test_window_prefill(b, hq, hkv, lens, q_lens, window, sinks):
    run_attention(b, Pool(b, lens, hkv, seed=len(lens) + hq), q_lens, hq, window, sinks)
    run_attention(b, Pool(b, lens, hkv, seed=len(lens) + hq), q_lens, hq, window, sinks, torch.bfloat16, scale=0.13,
                  one_part=lambda m: True)


# ---- append ----------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("group", [0, 128, 64])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (1, 1), (5, 3), (32, 8)])
@pytest.mark.parametrize("dim,interleaved", [(128, False), (128, True), (32, False), (96, False), (48, True), (0, False)])
def test_append_matches_the_oracle_bit_for_bit(b, group, hq, hkv, dim, interleaved):
    lens, new = [0, 63, 200, 5], [70, 1, 0, 129]
    rows, n = sum(new), len(lens)
    g = np.random.default_rng(hq * 7 + dim)
    x = g.standard_normal((rows, hq + 2 * hkv, D)).astype(np.float32)
    x[3] = 0.25                                   # a constant token: scale 0
    x[4, :, 7] = 300000.0                         # beyond fp16
    x[5, hq + hkv:, 3] = np.nan                   # (values are stored as they are, or saturated)
    x[6, hq + hkv:, 9] = -np.inf
    bits = paged.bf16_bits(x)
    qkv = bf16(bits)
    q, k, v = qkv.split([hq, hkv, hkv], 1)        # strided views of one tensor
    need = [-(-(a + m) // PAGE) for a, m in zip(lens, new)]
    pages = sum(need) + 2
    order = g.permutation(pages)
    table = np.full((n, max(need)), -1, np.int32)
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = order[at:at + m]
        at += m
    length = max(a + m for a, m in zip(lens, new))
    pos = np.concatenate([np.arange(a, a + m) for a, m in zip(lens, new)])
    req = np.repeat(np.arange(n), new)
    rope = b.rope_table(length, dim) if dim else None
    qb, kb, vb = bits[:, :hq], bits[:, hq:hq + hkv], bits[:, hq + hkv:]
    if dim:
        t = rope.cpu().numpy()
        qb, kb = paged.rotate(qb, t, pos, interleaved), paged.rotate(kb, t, pos, interleaved)
    if group == 0:
        host = g.integers(0, 65536, (pages, hkv, 2, PAGE, D)).astype(np.uint16)
        kv = bf16(host)
    else:
        host = g.integers(0, 256, (pages, hkv, paged.record_bytes(group))).astype(np.uint8)
        kv = torch.from_numpy(host.copy()).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = torch.empty(rows, hq, D, dtype=torch.bfloat16, device="cuda")
    args = dict(q=q, q_out=q_out, new_lens=new, interleaved=interleaved, error=err)
    dt = torch.from_numpy(table).cuda()
    if group == 0:
        b.bf16_append(kv, dt, lens, k, v, rope, **args)
    else:
        b.int4_append(kv, dt, lens, k, v, rope, group_size=group, **args)
    for r in range(rows):
        page, slot = table[req[r], pos[r] // PAGE], pos[r] % PAGE
        if group == 0:
            host[page, :, 0, slot], host[page, :, 1, slot] = kb[r], vb[r]
        else:
            (kc, km), (vc, vm) = paged.quantise4(kb[r], group), paged.quantise4(vb[r], group)
            for h in range(hkv):
                paged.put4(host[page, h], 0, slot, kc[h], km[h])
                paged.put4(host[page, h], 1, slot, vc[h], vm[h])
    assert err.item() == 0
    assert np.array_equal(q_out.view(torch.int16).cpu().numpy().view(np.uint16), qb)
    got = kv.view(torch.int16).cpu().numpy().view(np.uint16) if group == 0 else kv.cpu().numpy()
    assert np.array_equal(got, host)              # the other tokens' bytes among them
    if group:
        starts, counts = [3, 60, 0, 100], [60, 4, 0, 34]
        m = sum(counts)
        for kind in (torch.float32, torch.bfloat16):
            ko, vo = (torch.empty(m, hkv, D, dtype=kind, device="cuda") for _ in range(2))
            b.int4_read(kv, dt, starts, counts, ko, vo, group_size=group, error=err)
            at = 0
            for i, (a, c) in enumerate(zip(starts, counts)):
                for tok in range(a, a + c):
                    new_row = tok - lens[i]
                    if 0 <= new_row < new[i]:
                        r = sum(new[:i]) + new_row
                        for want, out in ((kb[r], ko), (vb[r], vo)):
                            w = paged.dequantise4(*paged.quantise4(want, group)).astype(np.float32)
                            w = paged.bf16_values(paged.bf16_bits(w)) if kind == torch.bfloat16 else w
                            assert np.array_equal(out[at].float().cpu().numpy(), w)
                    at += 1
        assert err.item() == 0


# ---- together ---------------------------------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("group", [0, 64])
def test_prefill_then_decode_steps(b, group):
    """A prompt appended and attended, then decode steps, as a serving loop makes them, on a stream of its own and the
    steps captured into a graph each; the outputs against the oracle on the oracle's own cache."""
    hq, hkv, steps = 8, 2, 3
    prompt = [70, 200]
    total = [t + steps for t in prompt]
    g = np.random.default_rng(11)
    table = g.permutation(2 * 5).reshape(2, 5).astype(np.int32)
    dt = torch.from_numpy(table).cuda()
    rope = b.rope_table(max(total))
    host = rope.cpu().numpy()
    kv = b.int4_pool(10, hkv, group) if group else torch.full((10, hkv, 2, PAGE, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    held = Pool(b, total, hkv, group)
    append = (lambda *a, **k: b.int4_append(*a, group_size=group, **k)) if group else b.bf16_append
    attend = (lambda *a, **k: b.int4_attention(*a, group_size=group, **k)) if group else b.window_attention
    stream = torch.cuda.Stream()
    lens = [0, 0]
    ws = b.attention_workspace(2, hq, hkv, prompt)
    torch.cuda.synchronize()
    for step in range(steps + 1):
        new = prompt if step == 0 else [1, 1]
        rows = sum(new)
        bits = paged.bf16_bits(g.standard_normal((rows, hq + 2 * hkv, D)).astype(np.float32))
        pos = np.concatenate([np.arange(a, a + m) for a, m in zip(lens, new)])
        qr = paged.rotate(bits[:, :hq], host, pos, False)
        kr = paged.rotate(bits[:, hq:hq + hkv], host, pos, False)
        vr = bits[:, hq + hkv:]
        row = 0
        for i, m in enumerate(new):
            for j in range(m):
                for dst, mag, x in ((held.k, held.kmag, kr[row]), (held.v, held.vmag, vr[row])):
                    if group:
                        code, meta = paged.quantise4(x, group)
                        y = paged.dequantise4(code, meta)
                        z = np.repeat(np.abs(meta[..., 1].astype(np.float64)), group, -1)
                    else:
                        y, z = paged.bf16_values(x).astype(np.float64), 0
                    dst[i][lens[i] + j], mag[i][lens[i] + j] = y, np.abs(y) + 2 * z
                row += 1
        q, k, v = bf16(bits).split([hq, hkv, hkv], 1)
        q_out = torch.empty(rows, hq, D, dtype=torch.bfloat16, device="cuda")
        now = [a + m for a, m in zip(lens, new)]
        q_lens = [min(m, 2) for m in new] if group else new
        last = np.concatenate([np.arange(sum(new[:i + 1]) - ql, sum(new[:i + 1])) for i, ql in enumerate(q_lens)])
        out = torch.empty(len(last), hq, D, device="cuda")
        lse = torch.empty(len(last), hq, device="cuda")
        torch.cuda.synchronize()

        def go():
            append(kv, dt, lens, k, v, rope, q=q, q_out=q_out, new_lens=new)
            attend(kv, dt, now, q_out[torch.from_numpy(last).cuda()] if step == 0 else q_out, out, hkv, 100, 8,
                   q_lens=q_lens, lse=lse, workspace=ws)

        with torch.cuda.stream(stream):
            if step == 0:
                go()
            else:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=stream):
                    go()
                graph.replay()
                graph.replay()
        torch.cuda.synchronize()
        held.lens = now
        sub = Pool.__new__(Pool)
        sub.lens, sub.hkv, sub.group = now, hkv, group
        sub.k = [x[:t] for x, t in zip(held.k, now)]
        sub.v = [x[:t] for x, t in zip(held.v, now)]
        sub.kmag = [x[:t] for x, t in zip(held.kmag, now)]
        sub.vmag = [x[:t] for x, t in zip(held.vmag, now)]
        check_attention(sub, qr[last], q_lens, 100, 8, out, lse)
        lens = now


# ---- far addresses, shared pages, replays ------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("group", [0, 128])
def test_pages_beyond_4_gib(b, group):
    """Pages at the end of a pool of more than 2^32 bytes, for every operator."""
    hq, hkv, t = 4, 2, 150
    per = hkv * (2 * PAGE * D * 2 if group == 0 else 8704)
    pages = (1 << 32) // per + 40
    kv = (torch.empty(pages, hkv, 2, PAGE, D, dtype=torch.bfloat16, device="cuda") if group == 0
          else torch.empty(pages, hkv, 8704, dtype=torch.uint8, device="cuda"))
    table = torch.tensor([[pages - 1, pages - 7, pages - 3]], dtype=torch.int32, device="cuda")
    g = np.random.default_rng(2)
    bits = paged.bf16_bits(g.standard_normal((t, hq + 2 * hkv, D)).astype(np.float32))
    q, k, v = bf16(bits).split([hq, hkv, hkv], 1)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    held = Pool.__new__(Pool)
    held.lens, held.hkv, held.group = [t], hkv, group
    if group == 0:
        b.bf16_append(kv, table, [0], k, v, new_lens=[t], error=err)
        held.k, held.v = ([paged.bf16_values(x).astype(np.float64)] for x in (bits[:, hq:hq + hkv], bits[:, hq + hkv:]))
        held.kmag, held.vmag = [np.abs(held.k[0])], [np.abs(held.v[0])]
        q_lens = [40]
        call = b.window_attention
    else:
        b.int4_append(kv, table, [0], k, v, new_lens=[t], error=err)
        both = [paged.quantise4(x, group) for x in (bits[:, hq:hq + hkv], bits[:, hq + hkv:])]
        held.k, held.v = ([paged.dequantise4(*x)] for x in both)
        held.kmag, held.vmag = ([np.abs(y[0]) + 2 * np.repeat(np.abs(x[1][..., 1].astype(np.float64)), group, -1)]
                                for x, y in zip(both, (held.k, held.v)))
        ko, vo = torch.empty(t, hkv, D, device="cuda"), torch.empty(t, hkv, D, device="cuda")
        b.int4_read(kv, table, [0], [t], ko, vo, error=err)
        assert np.array_equal(ko.cpu().numpy(), held.k[0].astype(np.float32))
        assert np.array_equal(vo.cpu().numpy(), held.v[0].astype(np.float32))
        q_lens = [4]
        call = b.int4_attention
    for m in ([1], q_lens):
        qq = bits[t - m[0]:, :hq]
        out, lse = torch.empty(m[0], hq, D, device="cuda"), torch.empty(m[0], hq, device="cuda")
        call(kv, table, [t], bf16(qq), out, hkv, 100, 3, q_lens=m, lse=lse, error=err)
        check_attention(held, qq, m, 100, 3, out, lse)
    assert err.item() == 0


@pytest.mark.gpu
def test_graphs_that_share_a_workspace_and_new_lengths(b):
    """Two graphs of different batches on one workspace, replayed in turn, with new contents of the same tensors; a
    split prefill and a decode among them; requests that share their prefix's pages."""
    hq, hkv = 8, 2
    pool = Pool(b, [700, 700, 130], hkv, seed=9)
    pool.table[1, :8] = pool.table[0, :8]                       # a shared prefix of 512 tokens
    pool.k[1][:512], pool.v[1][:512] = pool.k[0][:512], pool.v[0][:512]
    pool.kmag[1][:512], pool.vmag[1][:512] = pool.kmag[0][:512], pool.vmag[0][:512]
    kv, table = pool.device()
    ws = b.attention_workspace(3, hq, hkv, [1, 40, 1])
    stream = torch.cuda.Stream()
    sets = []
    for q_lens in ([1, 1, 1], [1, 40, 0]):
        rows = sum(q_lens)
        q = torch.zeros(rows, hq, D, dtype=torch.bfloat16, device="cuda")
        out, lse = torch.empty(rows, hq, D, device="cuda"), torch.empty(rows, hq, device="cuda")
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            b.window_attention(kv, table, pool.lens, q, out, hkv, 300, 4, q_lens=q_lens, lse=lse, workspace=ws)
        sets.append((q_lens, q, out, lse, graph))
    for turn in range(3):
        for q_lens, q, out, lse, graph in sets:
            bits = paged.bf16_bits(np.random.default_rng(turn).standard_normal(tuple(q.shape)).astype(np.float32))
            q.copy_(bf16(bits))
            graph.replay()
            torch.cuda.synchronize()
            check_attention(pool, bits, q_lens, 300, 4, out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("group", [128, 64])
def test_codes_of_exact_ties(b, group):
    """Half of the quotients lie exactly between two codes, for scales from fp16's least to 2^12; and a read into
    outputs that are aligned to 16 bytes only."""
    g = np.random.default_rng(12)
    rows, hkv = 64, 2
    k = g.integers(0, 31, (rows, hkv, D)).astype(np.float64)
    k[..., ::64], k[..., 1::64] = 0, 30
    scale = np.array([m * 2.0 ** e for m in (1, 3, 5, 7) for e in (-24, -20, -15, -9, -4, 0, 3, 10)])
    first = g.choice([0.0, -8.0, -15.0, 3.0], rows)            # the group's least value, in scales
    x = ((k / 2 + first[:, None, None]) * np.resize(scale, rows)[:, None, None]).astype(np.float32)
    bits = paged.bf16_bits(x)
    kv, table = b.int4_pool(1, hkv, group), torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    b.int4_append(kv, table, [0], bf16(bits), bf16(bits[::-1]), new_lens=[rows], group_size=group)
    host = np.zeros((hkv, paged.record_bytes(group)), np.uint8)
    levels = []
    for which, values in enumerate((bits, bits[::-1])):
        code, meta = paged.quantise4(values, group)
        levels.append(paged.dequantise4(code, meta).astype(np.float32))
        for r in range(rows):
            for h in range(hkv):
                paged.put4(host[h], which, r, code[r, h], meta[r, h])
    assert np.array_equal(kv[0].cpu().numpy(), host)
    out = torch.full((2, rows * hkv * D + 8), 7.0, device="cuda")
    ko, vo = (o[4:-4].view(rows, hkv, D) for o in out)         # 16 bytes off a 32-byte boundary
    b.int4_read(kv, table, [0], [rows], ko, vo, group_size=group)
    assert np.array_equal(ko.cpu().numpy(), levels[0]) and np.array_equal(vo.cpu().numpy(), levels[1])
    assert (out[:, :4] == 7).all() and (out[:, -4:] == 7).all()


# ---- the two ways through the binding -----------------------------------------------
@pytest.mark.gpu
@pytest.mark.parametrize("group", [0, 128])
def test_both_ways_through_the_binding_agree(b, group):
    """Calls marshalled in C (lists, the current stream, a workspace) and in Python (other sequences, a stream given):
    the same results; and the first kind is taken where it should be."""
    n, hq, hkv = 3, 8, 2
    kv = b.int4_pool(6, hkv) if group else torch.zeros(6, hkv, 2, PAGE, D, dtype=torch.bfloat16, device="cuda")
    kv2 = kv.clone()
    table = torch.tensor([[5, 0], [1, 2], [3, 4]], dtype=torch.int32, device="cuda")
    qkv = torch.randn(n, hq + 2 * hkv, D, device="cuda").to(torch.bfloat16)
    q, k, v = qkv.split([hq, hkv, hkv], 1)
    rope = b.rope_table(128)
    s = torch.cuda.current_stream()
    lens, new = [0, 70, 64], [1, 1, 1]
    extra = dict(group_size=group) if group else {}
    append, attend = (b.int4_append, b.int4_attention) if group else (b.bf16_append, b.window_attention)
    ws = b.attention_workspace(n, hq, hkv)
    qa, qb = torch.empty_like(q), torch.empty_like(q)
    oa, ob = torch.empty(n, hq, D, device="cuda"), torch.empty(n, hq, D, device="cuda")
    taken = b.calls().append(group, kv, table, lens, k, v, rope, q, qa, new, False, None, None)
    assert taken == 0
    append(kv2, table, np.array(lens), k, v, rope, q=q, q_out=qb, stream=s, **extra)
    assert torch.equal(qa, qb) and torch.equal(kv, kv2)
    now = [1, 71, 65]
    assert b.calls().attend(group, kv, table, now, qa, oa, hkv, 50, 2, None, 0.0, None, ws, None, None) == 0
    attend(kv2, table, np.array(now), qb, ob, hkv, 50, 2, workspace=ws, stream=s, **extra)
    assert torch.equal(oa, ob)
    # what the C side does not take
    for bad in (np.array(now), [1, 71], [1, 71, -1], [1, 71, 2.0], None, [1, 71, 2 ** 40]):
        assert b.calls().attend(group, kv, table, bad, qa, oa, hkv, 50, 2, None, 0.0, None, ws, None, None) is None
    assert b.calls().attend(group, kv, table, now, qa, oa, hkv, 50, 2, None, 0.0, None, None, None, None) is None
    assert b.calls().attend("x", kv, table, now, qa, oa, hkv, 50, 2, None, 0.0, None, ws, None, None) is None
    assert b.calls().attend(group, kv, table, now, qa.float(), oa, hkv, 50, 2, None, 0.0, None, ws, None, None) is None
    assert b.calls().attend(group, kv, table.cpu(), now, qa, oa, hkv, 50, 2, None, 0.0, None, ws, None, None) is None
    with pytest.raises(b.OscarError):
        attend(kv, table, [1, 71, 200], qa, oa, hkv, 50, 2, workspace=ws, **extra)
    small = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")
    grown = attend(kv, table, now, qa, ob, hkv, 50, 2, workspace=small, **extra)
    assert grown.numel() > small.numel() and torch.equal(oa, ob)


# ---- errors -------------------------------------------------------------------------
@pytest.mark.gpu
def test_bad_pages_set_the_error_word(b):
    kv = torch.ones(3, 2, 2, PAGE, D, dtype=torch.bfloat16, device="cuda")
    table = torch.tensor([[1, 99], [-5, 0]], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    x = torch.zeros(2, 2, D, dtype=torch.bfloat16, device="cuda")
    b.bf16_append(kv, table, [64, 3], x, x, error=err)
    assert err.item() == 1 and (kv == 1).all()                 # both stores are dropped
    err.zero_()
    q = torch.ones(2, 4, D, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(2, 4, D, device="cuda")
    b.window_attention(kv, table, [100, 4], q, out, 2, error=err)
    assert err.item() == 1 and (out == 1).all()                # a bad page reads as page 0
    err.zero_()
    kv4 = b.int4_pool(3, 2)
    b.int4_append(kv4, table, [64, 3], x, x, error=err)
    assert err.item() == 1 and (kv4 == 0).all()
    err.zero_()
    b.int4_attention(kv4, table, [100, 4], q, out, 2, error=err)
    assert err.item() == 1 and (out == 0).all()
    ko, vo = torch.ones(2, 2, 2, D, device="cuda")
    err.zero_()
    b.int4_read(kv4, table, [64, 0], [1, 1], ko, vo, error=err)
    assert err.item() == 1 and (ko == 0).all() and (vo == 0).all()
    b.window_attention(kv, table, [10, 4], q[:1], out[:1], 2, q_lens=[1, 0])   # no error word: nothing to tell
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_binding_refusals(b):
    kv = torch.zeros(4, 2, 2, PAGE, D, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    q = torch.zeros(2, 4, D, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(2, 4, D, device="cuda")
    k = torch.zeros(2, 2, D, dtype=torch.bfloat16, device="cuda")
    good = (kv, table, [5, 9], q, out, 2)
    b.window_attention(*good)
    for change in [dict(kv=kv.float()), dict(kv=kv[:, :1]), dict(table=table.long()), dict(table=table.cpu()),
                   dict(lens=[5, 129]), dict(lens=[5, 0]), dict(lens=[5]), dict(q=q[:1]), dict(q=q.float()),
                   dict(q=q.transpose(0, 1)), dict(out=out.half()), dict(out=out[:, :2]), dict(hkv=1), dict(hkv=4)]:
        args = dict(zip(("kv", "table", "lens", "q", "out", "hkv"), good))
        args.update(change)
        with pytest.raises(b.OscarError):
            b.window_attention(*args.values())
    for more in [dict(q_lens=[1, 2]), dict(q_lens=[3, -1]), dict(sinks=-1), dict(scale=float("nan")),
                 dict(lse=torch.zeros(2, 2, device="cuda")), dict(error=torch.zeros(1, device="cuda")),
                 dict(workspace=torch.zeros(1 << 20, device="cuda", dtype=torch.uint8)[1:])]:
        with pytest.raises(b.OscarError):
            b.window_attention(*good, **more)
    rope = b.rope_table(9)
    with pytest.raises(b.OscarError):
        b.bf16_append(kv, table, [5, 9], k, k, rope)             # position 9 is beyond the table
    for more in [dict(q=q), dict(q_out=q), dict(new_lens=[1, 2]), dict(new_lens=[3, -1]), dict(rope=rope[:, :24])]:
        with pytest.raises(b.OscarError):
            b.bf16_append(kv, table, [5, 6], k, k, **more)
    kv4 = b.int4_pool(4, 2)
    with pytest.raises(b.OscarError):
        b.int4_attention(kv4, table, [5, 9], q, out, 2, group_size=64)
    with pytest.raises(b.OscarError):
        b.int4_attention(kv4, table, [20, 20], torch.cat([q] * 9), torch.cat([out] * 9), 2, q_lens=[9, 9])
    with pytest.raises(b.OscarError):
        b.int4_append(kv4, table, [5, 9], k, k, group_size=32)


@pytest.mark.gpu
@pytest.mark.parametrize("group", [0, 128])
def test_ints_beyond_32_bits(b, group):
    """A window beyond 32 bits is no bound, whichever way the call takes; other such ints are refused and write nothing."""
    hq, hkv, lens = 4, 1, [100, 70]
    pool = Pool(b, lens, hkv, group, seed=14)
    kv, table = pool.device()
    q = torch.randn(2, hq, D, device="cuda").to(torch.bfloat16)
    append, attend = (b.int4_append, b.int4_attention) if group else (b.bf16_append, b.window_attention)
    want, got = torch.empty(2, hq, D, device="cuda"), torch.empty(2, hq, D, device="cuda")
    ws = attend(kv, table, lens, q, want, hkv)
    for window in (1 << 40, 2 ** 31, 2 ** 32 + 1, -2 ** 40):
        for seq, stream in ((lens, None), (np.array(lens), torch.cuda.current_stream())):
            got.fill_(7)
            attend(kv, table, seq, q, got, hkv, window, workspace=ws, stream=stream)
            assert torch.equal(got, want)
    got.fill_(7)
    before = kv.clone()
    k = torch.ones(2, hkv, D, dtype=torch.bfloat16, device="cuda")
    for far in (2 ** 32 + 3, 2 ** 40 + 64):
        for change in (dict(lens=[far, 70]), dict(sinks=far), dict(q_lens=[1, far])):
            with pytest.raises(b.OscarError, match="32 bits"):
                attend(kv, table, change.pop("lens", lens), q, got, hkv, workspace=ws, **change)
        for change in (dict(lens=[5, far]), dict(new_lens=[far, 1])):
            with pytest.raises(b.OscarError, match="32 bits"):
                append(kv, table, change.pop("lens", [5, 9]), k, k, **change)
    assert (got == 7).all() and torch.equal(kv.view(torch.uint8), before.view(torch.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("group,m", [(0, 1), (0, 20), (128, 1), (64, 2)])
def test_layers_that_share_their_buffers(b, group, m):
    """Append, then attention, over 30 layers without a wait of the host: one q_out, one page table and one workspace,
    the table changed by a kernel before each layer.  Every layer has the bits that it has by itself."""
    hq, hkv, lens, layers = 8, 2, [300, 1000], 30
    n, new = len(lens), [m] * len(lens)
    need = [-(-(t + m) // PAGE) for t in lens]
    pages = sum(need) + 2
    gen = torch.Generator("cuda").manual_seed(15 + group)
    append, attend = (b.int4_append, b.int4_attention) if group else (b.bf16_append, b.window_attention)
    extra = dict(group_size=group) if group else {}
    tables = torch.full((layers, n, max(need)), -1, dtype=torch.int32, device="cuda")
    kvs, qkvs = [], []
    for layer in range(layers):
        order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        tables[layer, 0, :need[0]], tables[layer, 1, :need[1]] = order[:need[0]], order[need[0]:need[0] + need[1]]
        kv = b.int4_pool(pages, hkv, group) if group else torch.zeros(pages, hkv, 2, PAGE, D, dtype=torch.bfloat16,
                                                                      device="cuda")
        old = torch.randn(sum(lens), 2 * hkv, D, device="cuda", generator=gen).to(torch.bfloat16)
        append(kv, tables[layer], [0, 0], old[:, :hkv], old[:, hkv:], new_lens=lens, **extra)
        kvs.append(kv)
        qkvs.append(torch.randn(n * m, hq + 2 * hkv, D, device="cuda", generator=gen).to(torch.bfloat16))
    rope = b.rope_table(max(lens) + m)
    now = [t + m for t in lens]
    ws = b.attention_workspace(n, hq, hkv, new)

    def layer_of(layer, kv, table, q_out, out, lse, workspace):
        q, k, v = qkvs[layer].split([hq, hkv, hkv], 1)
        append(kv, table, lens, k, v, rope, q=q, q_out=q_out, new_lens=new, **extra)
        attend(kv, table, now, q_out, out, hkv, 400, 5, q_lens=new, lse=lse, workspace=workspace, **extra)

    want = torch.empty(layers, n * m, hq, D, device="cuda"), torch.empty(layers, n * m, hq, device="cuda")
    for layer in range(layers):
        torch.cuda.synchronize()
        layer_of(layer, kvs[layer].clone(), tables[layer].clone(), torch.empty(n * m, hq, D, dtype=torch.bfloat16,
                 device="cuda"), want[0][layer], want[1][layer], torch.zeros_like(ws))
        torch.cuda.synchronize()
    table, q_out = torch.empty_like(tables[0]), torch.empty(n * m, hq, D, dtype=torch.bfloat16, device="cuda")
    got = torch.empty_like(want[0]), torch.empty_like(want[1])
    for turn in range(3):
        for x in got:
            x.fill_(7)
        for layer in range(layers):
            torch.add(tables[layer], 0, out=table)
            layer_of(layer, kvs[layer], table, q_out, got[0][layer], got[1][layer], ws)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("group,power", [(group, power) for group in (0, 128, 64) for power in (90, 115, 118, -60, -100)]
                         + [(group, power) for group in (128, 64) for power in (111, 113, 122, 124)])
def test_queries_of_any_size(b, group, power):
    """Queries times 2^power under a scale divided by it: every product is the same but for its exponent, so the outputs
    have the same bits.  (With BF16 pages q . k itself has to be finite in fp32; in 4 bits it carries its exponent
    apart.)"""
    hq, hkv, lens = 8, 2, [100, 700, 64]
    pool = Pool(b, lens, hkv, group, seed=16)
    pool.hide([1] * 3, 300, 3)
    kv, table = pool.device()
    x = np.clip(np.random.default_rng(16).standard_normal((3, hq, D)), -4, 4).astype(np.float32)
    call = b.int4_attention if group else b.window_attention
    extra = dict(group_size=group) if group else {}
    got = []
    for p in (0, power):
        y = np.ldexp(paged.bf16_values(paged.bf16_bits(x)), p)
        assert np.isfinite(y).all() and (power > 0 or np.abs(y[y != 0]).min() > 2.0 ** -126)
        largest = max((np.abs(y[i].astype(np.float64)).max(0) * np.abs(pool.k[i]).max((0, 1))).sum() for i in range(3))
        assert group or largest < np.finfo(np.float32).max      # (no partial sum of any q . k is larger)
        out, lse = torch.empty(3, hq, D, device="cuda"), torch.empty(3, hq, device="cuda")
        call(kv, table, lens, bf16(paged.bf16_bits(y)), out, hkv, 300, 3, scale=math.ldexp(0.0625, -p), lse=lse, **extra)
        got.append((out, lse))
    # scale x log2(e), which the kernels take, is 1.44 2^(-4 - power): exact for power <= 122.  Below 2^-126 it is
    # subnormal, in steps of 2^-149: at power 124 within 2^-150 / (1.44 2^-128) < 2^-22 of itself, which the logits'
    # tolerance holds eight times.
    if power <= 122:
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    for out, lse in got:
        check_attention(pool, paged.bf16_bits(x), [1] * 3, 300, 3, out, lse, 0.0625)


# ---- one key at a time ----------------------------------------------------------------
PEAKED = [
    # len, query tokens, window, sinks
    (700, 700, -1, 0),
    (700, 500, 130, 70),
    (600, 600, 64, 3),
    (523, 301, 200, 0),
    (2500, 70, -1, 0),        # few rows on many keys: split
    (1500, 130, 65, 129),
]


@pytest.mark.gpu
@pytest.mark.parametrize("out_type", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv", [(4, 1), (2, 2), (8, 1), (8, 2)])
@pytest.mark.parametrize("t,m,window,sinks", PEAKED)
def test_prefill_of_rows_that_look_at_one_key(b, out_type, hq, hkv, t, m, window, sinks):
    """Every query is a multiple of one key that it sees, which holds all but 1e-9 of its weight; the keys are taken in
    turn, those at the window's, the sinks' and the causal edge more often.  A value row that is dropped, doubled or
    taken from another place in either form's product moves an output by its whole size."""
    g, rng = hq // hkv, np.random.default_rng(17)
    k = np.clip(rng.standard_normal((t, hkv, D)), -3, 3).astype(np.float32)
    v = rng.standard_normal((t, hkv, D)).astype(np.float32)
    kb, vb = paged.bf16_bits(k), paged.bf16_bits(v)
    kf, vf = paged.bf16_values(kb).astype(np.float64), paged.bf16_values(vb).astype(np.float64)
    pages = -(-t // PAGE)
    table = rng.permutation(pages + 2)[:pages].astype(np.int32)[None]
    host = np.full((pages + 2, hkv, 2, PAGE, D), 0x7FC0, np.uint16)
    for t0 in range(0, t, PAGE):
        n = min(PAGE, t - t0)
        host[table[0, t0 // PAGE], :, 0, :n] = kb[t0:t0 + n].transpose(1, 0, 2)
        host[table[0, t0 // PAGE], :, 1, :n] = vb[t0:t0 + n].transpose(1, 0, 2)
    q, aim = np.zeros((m, hq, D), np.float32), np.zeros((m, hq), int)
    see = np.zeros((m, t), bool)
    for r in range(m):
        s = paged.seen(t - m + r, window, sinks)
        see[r, s] = True
        edge = [s[0], s[-1], s[np.searchsorted(s, sinks) % len(s)], s[len(s) // 2]]
        for h in range(hq):
            aim[r, h] = edge[(r // 3) % 4] if (r + h) % 3 == 0 else s[(5 * r + 31 * h) % len(s)]
            q[r, h] = 4 * kf[aim[r, h], h // g] / np.linalg.norm(kf[aim[r, h], h // g]) * math.sqrt(D)
    qb = paged.bf16_bits(q)
    out = torch.empty(m, hq, D, device="cuda", dtype=torch.bfloat16 if out_type == "bf16" else torch.float32)
    lse = torch.empty(m, hq, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    b.window_attention(bf16(host), torch.from_numpy(table).cuda(), [t], bf16(qb), out, hkv, window, sinks, q_lens=[m],
                       lse=lse, error=err)
    got, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert err.item() == 0
    qf = paged.bf16_values(qb).astype(np.float64)
    for h in range(hq):
        x = np.where(see, qf[:, h] @ kf[:, h // g].T / math.sqrt(D), -np.inf)
        top = x.max(1, keepdims=True)
        p = np.exp(x - top)
        total = p.sum(1, keepdims=True)
        assert (p[np.arange(m), aim[:, h]] > (1 - 1e-9) * total[:, 0]).all()
        want, mag = (p / total) @ vf[:, h // g], (p / total) @ np.abs(vf[:, h // g])
        logit = (np.where(see, np.abs(qf[:, h]) @ np.abs(kf[:, h // g]).T, 0).max(1) / math.sqrt(D))[:, None]
        tol = tolerance(want, mag, logit, see.sum(1)[:, None], 0, out_type == "bf16" and m * g > 16, out_type == "bf16")
        assert (np.abs(got[:, h] - want) <= tol).all(), h
        n = see.sum(1)
        assert (np.abs(lse[:, h] - (top + np.log(total))[:, 0])
                <= 2 * 8 * 2.0 ** -22 * logit[:, 0] + 2.0 ** -20 + 2.0 ** -22 * (n / 16 + 64)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv", [(4, 1), (2, 2), (8, 1)])
@pytest.mark.parametrize("lens,q_lens,window,sinks", [([700, 65, 333], [90, 2, 1], 128, 64), ([900, 300, 257], [1, 40, 2], -1, 0)])
def test_short_requests_beside_a_prompt(b, hq, hkv, lens, q_lens, window, sinks):
    """bf16 outputs: weights of one bf16 part only where a request has more than 16 rows a kv head."""
    run_attention(b, Pool(b, lens, hkv, seed=18), q_lens, hq, window, sinks, torch.bfloat16,
                  one_part=lambda m: m * (hq // hkv) > 16)


@pytest.mark.gpu
@pytest.mark.parametrize("group", [128, 64])
@pytest.mark.parametrize("hq", [8, 16, 32])
def test_long_shares_in_4_bits(b, group, hq):
    """As test_long_shares: 625 pages a segment, so that a warp (of 8 at least) sums up to 79 of them at once."""
    n, hkv, top = 84, 2, 40000
    m = 2 if hq == 32 else 1                                  # 4, 8 and 16 rows
    hq = 16 if hq == 32 else hq
    pool = Pool(b, [top], hkv, group, seed=13)
    lens = [top - 61 * i for i in range(n)]
    kv, table = pool.device()
    bits = paged.bf16_bits(np.random.default_rng(13).standard_normal((n * m, hq, D)).astype(np.float32))
    out, lse = torch.empty(n * m, hq, D, device="cuda"), torch.empty(n * m, hq, device="cuda")
    b.int4_attention(kv, table.expand(n, -1).contiguous(), lens, bf16(bits), out, hkv, q_lens=[m] * n, group_size=group,
                     lse=lse)
    qf, out, lse = paged.bf16_values(bits).astype(np.float64), out.double().cpu().numpy(), lse.double().cpu().numpy()
    for i in (0, 1, 40, 83):
        for h in (0, hq - 1):
            row, kh = i * m + m - 1, h // (hq // hkv)
            want, ls, mag, logit = paged.attend(qf[row, h], pool.k[0][:, kh], pool.v[0][:, kh], lens[i] - 1, -1, 0,
                                                1 / math.sqrt(D), pool.kmag[0][:, kh], pool.vmag[0][:, kh])
            tol = tolerance(want, mag, logit, 79 * PAGE, group, False, False)
            assert (np.abs(out[row, h] - want) <= tol).all()
            assert abs(lse[row, h] - ls) <= 2 * 8 * 2.0 ** -22 * logit + 2.0 ** -20 + 2.0 ** -22 * (79 * 4 + 64)


@pytest.mark.gpu
def test_an_empty_error_tensor_is_refused_whichever_way_the_call_takes(b):
    kv = torch.zeros(2, 1, 2, PAGE, D, dtype=torch.bfloat16, device="cuda")
    table, none = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
    q, out = torch.zeros(1, 2, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 2, D, device="cuda")
    ws = b.window_attention(kv, table, [5], q, out, 1)
    assert b.calls().attend(0, kv, table, [5], q, out, 1, -1, 0, None, 0.0, None, ws, none, None) is None
    assert b.calls().append(0, kv, table, [5], q[:, :1], q[:, :1], None, None, None, None, False, none, None) is None
    with pytest.raises(b.OscarError, match="error"):
        b.window_attention(kv, table, [5], q, out, 1, workspace=ws, error=none)
