"""Host logic of prompt attention and the chunk calls (no GPU): refusals, which come before any
change and any CUDA call, and the state that extend leaves, against appends."""
import ctypes

import numpy as np
import pytest


@pytest.fixture(scope="module")
def b():
    from bit_rotated_kv_decode_gb300 import binding, build
    build.build()
    binding.load()
    return binding


def ints(*v):
    return (ctypes.c_int32 * len(v))(*v)


A = 0x10000   # an aligned address that no refused call reaches

PROMPT = dict(lens=ints(3, 64), n=2, hq=8, hkv=2, window=-1, sinks=0, scale=0.0, q=A, qs=1024, k=A, ks=256, v=A, vs=256,
              out=A, kind=0, lse=None, error=None, ws=A, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("change", [
    dict(n=0), dict(n=257), dict(lens=None), dict(lens=ints(-1, 4)), dict(lens=ints(2 ** 25, 2 ** 25)),
    dict(lens=ints(2 ** 31 - 1, 1)), dict(hq=6), dict(hq=0), dict(hkv=0), dict(hq=32), dict(q=None), dict(k=None),
    dict(v=None), dict(out=None), dict(ws=None), dict(q=A + 8), dict(k=A + 2), dict(v=A + 4), dict(out=A + 8),
    dict(lse=A + 2), dict(error=A + 1), dict(ws=A + 128), dict(qs=1000), dict(qs=1028), dict(ks=248), dict(ks=260),
    dict(vs=128), dict(vs=1 << 40), dict(kind=2), dict(sinks=-1), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(scale=3.4e38), dict(ws_bytes=0), dict(ws_bytes=255)])
def test_prompt_refusals(b, change):
    lib = b.load()
    assert lib.oscar_prompt_attention(*{**PROMPT, **change}.values()) == b.OSCAR_ERR_INVALID_ARG
    assert lib.oscar_paged_last_error() != b""


def test_prompt_of_nothing_is_a_no_op(b):
    assert b.load().oscar_prompt_attention(*{**PROMPT, "lens": ints(0, 0)}.values()) == b.OSCAR_OK


def test_prompt_workspace(b):
    lib = b.load()
    for n, lens, hq, hkv in ((0, ints(1), 8, 2), (1, None, 8, 2), (257, ints(*[1] * 257), 8, 2), (1, ints(-1), 8, 2),
                             (1, ints(5), 6, 2), (1, ints(5), 8, 0)):
        assert lib.oscar_prompt_workspace_bytes(n, lens, hq, hkv) == 0
    assert lib.oscar_prompt_workspace_bytes(1, ints(0), 8, 2) >= 256
    # a call with this much is not refused for its workspace
    for lens in ((1,), (700,), (4000, 3, 0)):
        need = lib.oscar_prompt_workspace_bytes(len(lens), ints(*lens), 8, 2)
        for kind in (0, 1):
            v = {**PROMPT, "lens": ints(*lens), "n": len(lens), "kind": kind, "ws_bytes": need, "sinks": -1}
            lib.oscar_prompt_attention(*v.values())
            assert b"sinks" in lib.oscar_paged_last_error()


def dry(b, layers=2, hq=8, hkv=2, requests=4, table=16, pages=40, seed=0, group=128):
    cfg = b.make_config(layers, hq, hkv, requests, table, pages, 0, 0.0, seed, group_size=group)
    tau = np.ones((layers, hkv), np.float32)
    return b.OscarCache(cfg, tau_k=tau, tau_v=tau, dry_run=True)


def state(c, reqs, layers=2):
    return [[c.length(r, layer) for layer in range(layers)] + [c.pages(r)] for r in reqs], c.free_pages()


@pytest.mark.parametrize("seed", range(4))
def test_extend_leaves_the_state_of_as_many_appends(b, seed):
    """One request at a time, so that pages are taken in the same order."""
    g = np.random.default_rng(seed)
    one, many = dry(b, seed=seed), dry(b, seed=seed)
    reqs = [one.open() for _ in range(3)]
    assert reqs == [many.open() for _ in range(3)]
    for _ in range(60):
        r, layer, m = int(g.choice(reqs)), int(g.integers(0, 2)), int(g.choice([0, 1, 2, 63, 64, 65, 200, 257]))
        if one.length(r, layer)[0] + m > 900:
            continue
        if g.random() < 0.2 and one.length(r, layer)[1] < one.length(r, layer)[0]:
            one.demote(layer, [r])
            many.demote(layer, [r])
        one.extend(layer, [r], None, None, new_lens=[m])
        for _ in range(m):
            many.append(layer, [r], None, None)
        assert state(one, reqs) == state(many, reqs)


def test_extend_of_a_batch_and_a_fork(b):
    c = dry(b)
    r = [c.open() for _ in range(2)]
    c.extend(0, r, None, None, new_lens=[700, 5])
    c.extend(1, [r[0]], None, None, new_lens=[700])
    assert c.length(r[0], 0) == (700, 444) and c.length(r[1], 0) == (5, 64) and c.length(r[1], 1) == (0, 64)
    c.extend(0, r, None, None)
    assert c.length(r[0], 0) == (701, 445) and c.length(r[1], 0) == (6, 64)
    f = c.fork(r[0], 64 + 5 * 64)
    c.extend(0, [f], None, None, new_lens=[100])          # the window of a fork is empty
    assert c.length(f, 0) == (484, 384)
    c.extend(0, [f], None, None, new_lens=[300])
    assert c.length(f, 0) == (784, 528)


def test_extend_refusals_change_nothing(b):
    c = dry(b, table=6, pages=7)
    r = [c.open() for _ in range(3)]
    c.extend(0, r[:2], None, None, new_lens=[500, 400])
    before = state(c, r)
    P, lib, ok = dict(layer=0, n=2, reqs=ints(r[0], r[1]), lens=ints(1, 1), k=None, ks=256, v=None, vs=256), c.lib, 0
    for change, status in ((dict(layer=2), 1), (dict(layer=-1), 1), (dict(n=0), 1), (dict(n=257), 1), (dict(reqs=None), 1),
                           (dict(reqs=ints(r[0], r[0])), 1), (dict(reqs=ints(r[0], 3)), 1), (dict(reqs=ints(-1, 0)), 1),
                           (dict(lens=ints(-1, 1)), 1), (dict(lens=ints(1, 2 ** 30)), 1), (dict(ks=128), 1),
                           (dict(ks=260), 1), (dict(vs=255), 1), (dict(lens=ints(400, 1)), 1),       # beyond the page table
                           (dict(lens=ints(70, 200)), 2),                                        # out of pages
                           (dict(lens=ints(2 ** 25 - 600, 2 ** 25 - 600)), 1)):
        assert lib.oscar_extend(c.h, *{**P, **change}.values(), None) == status, change
        assert lib.oscar_last_error(c.h) != b""
        assert state(c, r) == before
        ok += 1
    assert ok == 16 and lib.oscar_extend(None, *P.values(), None) == 1
    assert lib.oscar_extend(c.h, *{**P, "lens": ints(0, 0)}.values(), None) == b.OSCAR_ERR_DRY_RUN
    assert state(c, r) == before


def test_read_and_chunk_refusals(b):
    c = dry(b)
    r = [c.open() for _ in range(2)]
    c.extend(0, r, None, None, new_lens=[500, 3])
    before = state(c, r)
    R, lib = dict(layer=0, n=2, reqs=ints(*r), starts=ints(0, 0), counts=ints(500, 3), k=None, v=None, kind=0), c.lib
    assert lib.oscar_read(c.h, *R.values(), None) == b.OSCAR_ERR_DRY_RUN
    assert lib.oscar_read(c.h, *{**R, "reqs": ints(r[0], r[0]), "counts": ints(5, 7)}.values(), None) == b.OSCAR_ERR_DRY_RUN
    for change in (dict(layer=2), dict(n=0), dict(n=257), dict(reqs=None), dict(reqs=ints(0, 3)), dict(starts=None),
                   dict(counts=None), dict(starts=ints(-1, 0)), dict(counts=ints(-1, 0)), dict(counts=ints(501, 3)),
                   dict(starts=ints(1, 0)), dict(counts=ints(2 ** 31 - 1, 3)), dict(kind=2), dict(layer=1)):
        assert lib.oscar_read(c.h, *{**R, **change}.values(), None) == b.OSCAR_ERR_INVALID_ARG, change
    C = dict(layer=0, n=2, reqs=ints(*r), lens=ints(4, 1), q=None, qs=1024, k=None, ks=256, v=None, vs=256, out=None, ws=None,
             ws_bytes=0)
    assert lib.oscar_chunk_attention(c.h, *C.values(), None) == b.OSCAR_ERR_DRY_RUN
    assert lib.oscar_chunk_attention(c.h, *{**C, "reqs": ints(r[0], r[0])}.values(), None) == b.OSCAR_ERR_DRY_RUN
    for change in (dict(layer=-1), dict(n=0), dict(n=257), dict(reqs=None), dict(reqs=ints(0, 2)), dict(lens=ints(-1, 1)),
                   dict(lens=ints(2 ** 30, 1)), dict(lens=ints(2 ** 24, 2 ** 24)), dict(qs=1016), dict(qs=1028),
                   dict(ks=128), dict(vs=264 - 4)):
        assert lib.oscar_chunk_attention(c.h, *{**C, **change}.values(), None) == b.OSCAR_ERR_INVALID_ARG, change
    assert state(c, r) == before


def test_chunk_workspace(b):
    c, need = dry(b, requests=260, pages=300), ctypes.c_size_t()
    size = lambda *lens: (c.lib.oscar_chunk_workspace_bytes(c.h, len(lens), ints(*lens), ctypes.byref(need)),  # noqa: E731
                          need.value)
    for bad in ((), [1] * 257, (-1,), (2 ** 25,)):
        assert size(*bad)[0] == b.OSCAR_ERR_INVALID_ARG
    assert c.lib.oscar_chunk_workspace_bytes(c.h, 1, ints(1), None) == b.OSCAR_ERR_INVALID_ARG
    assert c.lib.oscar_chunk_workspace_bytes(c.h, 3, None, ctypes.byref(need)) == 0 and need.value == size(1, 1, 1)[1]
    # it grows with the tokens, and does not depend on what the requests hold
    sizes = [size(m)[1] for m in (1, 16, 33, 300, 4000)]
    assert sizes == sorted(sizes)
    r = c.open()
    c.extend(0, [r], None, None, new_lens=[700])
    assert [size(m)[1] for m in (1, 16, 33, 300, 4000)] == sizes


def test_lists_of_the_wrong_length_are_refused(b):
    c = dry(b)
    r = c.open()
    for call in (lambda: c.extend(0, [r], None, None, new_lens=[1, 2]), lambda: c.extend(0, [], None, None),
                 lambda: c.read(0, [r], [0, 0], [1], None, None), lambda: c.read(0, [r], [0], [], None, None),
                 lambda: c.chunk_attention(0, [r], None, None, None, None, new_lens=[1, 1]),
                 lambda: c.extend(2 ** 32, [r], None, None), lambda: c.extend(0, [r], None, None, new_lens=[2 ** 32]),
                 lambda: c.chunk_attention(0, [r], None, None, None, None, new_lens=[-1])):
        with pytest.raises(b.OscarError):
            call()
    assert c.length(r, 0) == (0, 64)
