"""Argument checks of the paged-cache operators (no GPU: every refusal comes before
any CUDA call) and pins of their oracle."""
import ctypes

import numpy as np
import pytest

from oracle import paged


@pytest.fixture(scope="module")
def b():
    from bit_rotated_kv_decode_gb300 import binding, build
    build.build()
    binding.load()
    return binding


def ints(*v):
    return (ctypes.c_int32 * len(v))(*v)


A = 0x10000   # an aligned address that no refused call reaches

APPEND = dict(kv=A, pages=8, table=A, max_pages=4, lens=ints(3, 64), new=ints(1, 2), n=2, hq=8, hkv=2, rope=None, q=A,
              qs=1536, k=A, ks=1536, v=A, vs=1536, q_out=A, error=None, stream=None)


@pytest.mark.parametrize("change", [
    dict(kv=None), dict(kv=A + 8), dict(pages=0), dict(table=None), dict(max_pages=0), dict(lens=None),
    dict(lens=ints(-1, 0)), dict(lens=ints(3, 255)), dict(new=ints(1, -1)), dict(n=0), dict(n=257), dict(hkv=0),
    dict(hq=0), dict(q=A + 2), dict(q_out=None), dict(q=None), dict(k=None), dict(k=A + 4), dict(v=None),
    dict(ks=255), dict(ks=260), dict(vs=128), dict(qs=1000), dict(qs=1028), dict(rope=(A, 65, 128)),
    dict(rope=(A, 66, 8)), dict(rope=(A, 66, 136)), dict(rope=(A, 66, 40)), dict(rope=(None, 66, 128)),
    dict(rope=(A + 4, 66, 128)), dict(group=32), dict(group=0)])
def test_append_refusals(b, change):
    args = {**APPEND, **change}
    group = args.pop("group", None)
    if args["rope"] is not None:
        args["rope"] = ctypes.byref(b.oscar_rope(*args["rope"], 0))
    v = list(args.values())
    lib = b.load()
    if group is None:
        assert lib.oscar_bf16_append(*v) == b.OSCAR_ERR_INVALID_ARG
        assert lib.oscar_paged_last_error() != b""
    v.insert(9, 128 if group is None else group)
    assert lib.oscar_int4_append(*v) == b.OSCAR_ERR_INVALID_ARG


def test_append_of_nothing_is_a_no_op(b):
    v = list({**APPEND, "new": ints(0, 0)}.values())
    assert b.load().oscar_bf16_append(*v) == b.OSCAR_OK


ATTEND = dict(kv=A, pages=8, table=A, max_pages=4, lens=ints(3, 64), q_lens=ints(1, 2), n=2, hq=8, hkv=2, window=5,
              sinks=1, scale=0.0, q=A, qs=1024, out=A, kind=0, lse=None, error=None, ws=A, ws_bytes=1 << 40,
              stream=None)


@pytest.mark.parametrize("change", [
    dict(kv=None), dict(kv=A + 2), dict(pages=0), dict(table=None), dict(max_pages=0), dict(lens=None),
    dict(lens=ints(0, 5)), dict(lens=ints(3, 257)), dict(q_lens=ints(-1, 1)), dict(n=0), dict(n=257), dict(hkv=3),
    dict(hq=6), dict(hq=32), dict(sinks=-1), dict(scale=float("inf")), dict(scale=3e38), dict(q=None), dict(q=A + 2), dict(qs=1000),
    dict(qs=1028), dict(out=None), dict(out=A + 4), dict(kind=2), dict(ws=None), dict(ws=A + 16), dict(ws_bytes=100),
    dict(group=96)])
def test_attention_refusals(b, change):
    args = {**ATTEND, **change}
    group = args.pop("group", None)
    v = list(args.values())
    lib = b.load()
    if group is None:
        assert lib.oscar_window_attention(*v) == b.OSCAR_ERR_INVALID_ARG
    v.insert(9, 128 if group is None else group)
    assert lib.oscar_int4_attention(*v) == b.OSCAR_ERR_INVALID_ARG


def test_attention_bounds_the_visible_tokens(b):
    """Kv heads x visible 16-token units (4 bits: pages) of the decoded requests are below 2^31; a window counts."""
    lib = b.load()
    big = {**ATTEND, "hq": 1024, "hkv": 1024, "qs": 1024 * 128, "pages": 1024, "n": 16, "max_pages": 1 << 24,
           "lens": ints(*[1 << 25] * 16), "q_lens": ints(40, *[1] * 15), "window": -1}
    assert lib.oscar_window_attention(*big.values()) == b.OSCAR_ERR_INVALID_ARG
    assert b"visible tokens" in lib.oscar_paged_last_error()
    v = list({**big, "q_lens": None, "lens": ints(*[1 << 28] * 16)}.values())
    v.insert(9, 128)
    assert lib.oscar_int4_attention(*v) == b.OSCAR_ERR_INVALID_ARG
    assert b"visible tokens" in lib.oscar_paged_last_error()


def test_int4_attention_takes_a_few_query_tokens(b):
    v = list({**ATTEND, "q_lens": ints(1, 5)}.values())
    v.insert(9, 128)
    assert b.load().oscar_int4_attention(*v) == b.OSCAR_ERR_INVALID_ARG
    assert b"query tokens" in b.load().oscar_paged_last_error()


@pytest.mark.parametrize("change", [dict(kv=None), dict(starts=None), dict(counts=None), dict(starts=ints(-1, 0)),
                                    dict(counts=ints(1, 256)), dict(k=None), dict(v=A + 4), dict(kind=3), dict(group=1)])
def test_read_refusals(b, change):
    args = dict(kv=A, pages=8, table=A, max_pages=4, starts=ints(0, 3), counts=ints(4, 5), n=2, hkv=2, group=64, k=A,
                v=A, kind=1, error=None, stream=None)
    args.update(change)
    assert b.load().oscar_int4_read(*args.values()) == b.OSCAR_ERR_INVALID_ARG


def test_int4_pool(b):
    assert b.int4_pool(3, 2, device="cpu").shape == (3, 2, 8704) and b.int4_pool(1, 1, 64, "cpu").shape == (1, 1, 9216)
    with pytest.raises(b.OscarError):
        b.int4_pool(3, 2, 32, "cpu")


def test_workspace_size(b):
    lib = b.load()
    size = lib.oscar_attention_workspace_bytes
    assert size(0, None, 8, 2) == 0 and size(257, None, 8, 2) == 0 and size(1, None, 6, 2) == 0
    assert size(1, None, 24, 8) == 0 and size(256, None, 1024, 512) == 0 and size(1, ints(-1), 8, 2) == 0
    assert size(4, None, 8, 2) >= 65536 + 8 * 4 * 132 * 4
    assert size(1, ints(0), 8, 2) > 0


# ---- the oracle ------------------------------------------------------------------
def test_rotation_keeps_lengths_and_turns_by_the_angle():
    g = np.random.default_rng(0)
    bits = paged.bf16_bits(g.standard_normal((4, 2, 128)).astype(np.float32))
    angle = np.arange(4)[:, None] * np.ones(32)
    table = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    for inter in (False, True):
        y = paged.bf16_values(paged.rotate(bits, table, np.arange(4), inter)).astype(np.float64)
        x = paged.bf16_values(bits).astype(np.float64)
        i = np.arange(0, 64, 2) if inter else np.arange(32)
        j = i + 1 if inter else i + 32
        z = (x[..., i] + 1j * x[..., j]) * np.exp(1j * np.arange(4))[:, None, None]
        assert np.abs(y[..., i] - z.real).max() < 2 ** -7 * 4 and np.abs(y[..., j] - z.imag).max() < 2 ** -7 * 4
        assert np.array_equal(y[..., 64:], x[..., 64:]) and np.array_equal(y[0], x[0])


@pytest.mark.parametrize("group", [128, 64])
def test_quantise4_takes_the_nearest_level(group):
    g = np.random.default_rng(1)
    bits = paged.bf16_bits(g.standard_normal((50, 128)).astype(np.float32))
    code, meta = paged.quantise4(bits, group)
    x = paged.bf16_values(bits).astype(np.float64).reshape(50, -1, group)
    s, z = meta[..., :1].astype(np.float64), meta[..., 1:].astype(np.float64)
    levels = np.arange(16) * s[..., None] + z[..., None]
    best = np.abs(x[..., None] - levels).min(-1)
    mine = np.abs(x - paged.dequantise4(code, meta).reshape(x.shape))
    assert (mine <= best + 1e-6).all()
    const, m = paged.quantise4(paged.bf16_bits(np.full((1, 128), 0.5, np.float32)), group)
    assert (const == 0).all() and (m[..., 0] == 0).all() and (m[..., 1] == 0.5).all()


def test_record_holds_what_was_put():
    rec = np.zeros(paged.record_bytes(64), np.uint8)
    code = np.arange(128, dtype=np.uint8) % 16
    meta = np.array([[1, 2], [3, 4]], np.float16)
    paged.put4(rec, 1, 9, code, meta)
    assert np.array_equal(rec[4096 + 9 * 64:4096 + 10 * 64] & 15, code[0::2])
    assert np.array_equal(rec[8192 + 512 + 72:8192 + 512 + 80].view(np.float16), [1, 2, 3, 4])
    assert rec.astype(bool).sum() <= 64 + 8


def test_window_and_sinks():
    assert list(paged.seen(5, -1, 0)) == [0, 1, 2, 3, 4, 5]
    assert list(paged.seen(5, 2, 1)) == [0, 4, 5]
    assert list(paged.seen(5, 0, 2)) == [0, 1] and list(paged.seen(5, 0, 0)) == []
    assert list(paged.seen(1, 9, 4)) == [0, 1]


def test_rope_table_keeps_far_angles(b):
    t = b.rope_table(100001, 64, device="cpu").numpy()
    inv = np.longdouble(10000) ** (-2 * np.arange(32, dtype=np.longdouble) / 64)
    a = np.longdouble(100000) * inv
    assert np.abs(t[100000, :32] - np.cos(a)).max() < 2 ** -23 and np.abs(t[100000, 32:] - np.sin(a)).max() < 2 ** -23


def test_marshalling_extension_takes_nothing_before_its_setup(b):
    import importlib.machinery
    import importlib.util
    from bit_rotated_kv_decode_gb300 import build
    loader = importlib.machinery.ExtensionFileLoader("_oscar_calls", build.CALLS)
    mod = importlib.util.module_from_spec(importlib.util.spec_from_loader("_oscar_calls", loader))
    loader.exec_module(mod)
    assert mod.attend(*[None] * 15) is None and mod.append(*[None] * 13) is None and mod.read(*[None] * 9) is None
    assert mod.attend() is None and mod.append(1) is None and mod.read("x", *[1] * 8) is None
    with pytest.raises(TypeError):
        mod.setup(1, 2, 3)


# ---- ints beyond 32 bits, through the public calls --------------------------------
def tensors():
    import torch
    return dict(kv=torch.zeros(4, 2, 2, 64, 128, dtype=torch.bfloat16), table=torch.zeros(2, 2, dtype=torch.int32),
                q=torch.zeros(2, 4, 128, dtype=torch.bfloat16), out=torch.zeros(2, 4, 128),
                k=torch.zeros(2, 2, 128, dtype=torch.bfloat16), ws=torch.zeros(1 << 20, dtype=torch.uint8))


@pytest.fixture
def on_cpu(b, monkeypatch):
    """The Python path on CPU tensors, up to the C call."""
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(b, "_context", lambda stream: (torch, -1, None))
    return b


BEYOND = [2 ** 31, 2 ** 32 + 3, 2 ** 40 + 64]


@pytest.mark.parametrize("far", BEYOND)
@pytest.mark.parametrize("four", [False, True])
def test_lengths_beyond_32_bits_are_refused(on_cpu, far, four):
    b, t = on_cpu, tensors()
    kv = b.int4_pool(4, 2, device="cpu") if four else t["kv"]
    append = b.int4_append if four else b.bf16_append
    attend = b.int4_attention if four else b.window_attention
    for lens in ([far, 5], (5, far), np.array([5, far])):
        with pytest.raises(b.OscarError, match="32 bits"):
            append(kv, t["table"], lens, t["k"], t["k"])
        with pytest.raises(b.OscarError, match="32 bits"):
            attend(kv, t["table"], lens, t["q"], t["out"], 2, workspace=t["ws"])
        with pytest.raises(b.OscarError, match="32 bits"):
            b.int4_read(kv, t["table"], lens, [1, 1], t["k"].float(), t["k"].float())
    with pytest.raises(b.OscarError, match="32 bits"):
        append(kv, t["table"], [5, 9], t["k"], t["k"], new_lens=[far, 1])
    with pytest.raises(b.OscarError, match="32 bits"):
        attend(kv, t["table"], [5, 9], t["q"], t["out"], 2, q_lens=[1, far], workspace=t["ws"])
    with pytest.raises(b.OscarError, match="32 bits"):
        b.int4_read(kv, t["table"], [0, 0], [far, 1], t["k"].float(), t["k"].float())


@pytest.mark.parametrize("four", [False, True])
def test_sinks_and_heads_beyond_32_bits_are_refused(on_cpu, four):
    b, t = on_cpu, tensors()
    kv = b.int4_pool(4, 2, device="cpu") if four else t["kv"]
    attend = b.int4_attention if four else b.window_attention
    for far in BEYOND + [-far for far in BEYOND[1:]]:
        with pytest.raises(b.OscarError, match="32 bits"):
            attend(kv, t["table"], [5, 9], t["q"], t["out"], 2, 4, far, workspace=t["ws"])
        with pytest.raises(b.OscarError, match="32 bits"):
            attend(kv, t["table"], [5, 9], t["q"], t["out"], far, workspace=t["ws"])
        for args in ((far, 4, 2), (2, far, 2), (2, 4, far)):
            with pytest.raises(b.OscarError, match="32 bits"):
                b.attention_workspace(*args)
        with pytest.raises(b.OscarError, match="32 bits"):
            b.attention_workspace(2, 4, 2, q_lens=[1, abs(far)])
    for odd in (1.5, "4", None):
        with pytest.raises(b.OscarError, match="int"):
            attend(kv, t["table"], [5, 9], t["q"], t["out"], 2, odd, workspace=t["ws"])


@pytest.mark.parametrize("window,passed", [(2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, -1), (1 << 40, -1), (2 ** 32 + 5, -1),
                                           (-2 ** 31, -2 ** 31), (-2 ** 40, -1), (np.int64(2 ** 33), -1), (7, 7)])
def test_a_window_beyond_32_bits_is_no_bound(on_cpu, window, passed):
    """A window of so many tokens holds every cache, as a negative one does."""
    b, t, got = on_cpu, tensors(), []
    b._attention(lambda *a: got.append(a[9]) or 0, (), t["kv"], t["table"], [5, 9], t["q"], t["out"], 2, window, 0,
                 None, 0.0, None, t["ws"], None, None)
    assert got == [passed]


def test_kernels_that_overlap_the_grid_before_use_no_noncoherent_loads():
    """They start while the grid before may still write their inputs; ld.global.nc is for memory that nobody writes in
    a kernel's life."""
    import os
    import re
    from bit_rotated_kv_decode_gb300 import build
    seen = 0
    for name in sorted(os.listdir(build.CSRC)):
        text = open(os.path.join(build.CSRC, name)).read()
        if not name.startswith("paged") or not name.endswith((".cu", ".cuh")):
            continue
        code = re.sub(r"//[^\n]*", "", text)
        assert "__ldg" not in code and "global.nc" not in code and "__restrict__" not in code, name
        seen += "launch_dependent(" in code
    assert seen >= 4


@pytest.mark.parametrize("start,count", [(2 ** 31 - 5, 10), (2 ** 31 - 1, 1), (2 ** 30, 1), (2 ** 30 - 5, 6),
                                         (0, 2 ** 30 + 1)])
def test_positions_end_at_2_to_the_30(b, start, count):
    """Positions are ints in the kernels, and 2^30 tokens are what an attention takes; a table wide enough for more
    does not let them through."""
    lib, wide = b.load(), dict(max_pages=1 << 26, lens=ints(start, 0))
    for group in (None, 128, 64):
        v = list({**APPEND, **wide, "new": ints(count, 1)}.values())
        if group:
            v.insert(9, group)
        fn = lib.oscar_int4_append if group else lib.oscar_bf16_append
        assert fn(*v) == b.OSCAR_ERR_INVALID_ARG and b"2^30" in lib.oscar_paged_last_error()
    read = dict(kv=A, pages=8, table=A, max_pages=1 << 26, starts=ints(start, 0), counts=ints(count, 1), n=2, hkv=2,
                group=64, k=A, v=A, kind=1, error=None, stream=None)
    assert lib.oscar_int4_read(*read.values()) == b.OSCAR_ERR_INVALID_ARG
    assert b"2^30" in lib.oscar_paged_last_error()


@pytest.mark.parametrize("short", [1, 5, 11, 63])
def test_visible_units_leave_room_for_a_warps_step(b, short):
    """A warp steps through the units by the warps of its CTA, so the last ones must not come within a step of 2^31."""
    lens = [1 << 30] * 31 + [(1 << 30) - 16 * short]            # 2^31 - short units of 16 tokens
    v = {**ATTEND, "hq": 1, "hkv": 1, "qs": 128, "n": 32, "max_pages": 1 << 24, "lens": ints(*lens), "q_lens": None,
         "window": -1}
    assert b.load().oscar_window_attention(*v.values()) == b.OSCAR_ERR_INVALID_ARG
    assert b"visible tokens" in b.load().oscar_paged_last_error()


# ---- the build ---------------------------------------------------------------------
@pytest.fixture
def small_build(monkeypatch, tmp_path):
    """A build of the host file alone, in a folder of its own."""
    from bit_rotated_kv_decode_gb300 import build
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "obj"))
    monkeypatch.setattr(build, "LIBDIR", str(tmp_path / "lib"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib" / "lib.so"))
    monkeypatch.setattr(build, "SOURCES", ["host.cpp"])
    return build, tmp_path


def test_the_library_builds_without_torch(small_build, monkeypatch, capfd):
    import importlib.util
    build, tmp = small_build
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert build.build() == str(tmp / "lib" / "lib.so")
    assert [p.name for p in (tmp / "lib").iterdir()] == ["lib.so"]
    assert "torch" in capfd.readouterr().err


def test_the_library_is_there_though_the_extension_does_not_compile(small_build, monkeypatch):
    build, tmp = small_build
    monkeypatch.setattr(build, "_extension", lambda nvcc: (["false"], None))
    with pytest.raises(RuntimeError, match="build failed"):
        build.build()
    assert (tmp / "lib" / "lib.so").exists()


def test_another_torch_or_interpreter_takes_another_extension(monkeypatch):
    """It reads tensors by torch's own layout: one built for another version must not be loaded."""
    import importlib.metadata
    import sysconfig
    from bit_rotated_kv_decode_gb300 import build
    paths = {build.calls_path()}
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "9.9.9+x")
    paths.add(build.calls_path())
    config = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-399" if name == "SOABI" else config(name))
    paths.add(build.calls_path())
    assert len(paths) == 3 and all(p.startswith(build.LIBDIR) and p.endswith(".so") for p in paths)


def test_calls_are_marshalled_in_python_without_the_extension(on_cpu, monkeypatch):
    b, t, got = on_cpu, tensors(), []
    monkeypatch.setattr(b, "_calls", None)
    monkeypatch.setattr(b, "calls_path", lambda: "/nonexistent/_oscar_calls.so")
    with pytest.raises(RuntimeError, match="missing"):
        b.calls()
    with pytest.warns(RuntimeWarning, match="not built"):
        b._attention(lambda *a: got.append(a) or 0, (), t["kv"], t["table"], [5, 9], t["q"], t["out"], 2, 7, 0, None,
                     0.0, None, t["ws"], None, None)
    b._append(lambda *a: got.append(a) or 0, (), t["kv"], t["table"], [5, 9], t["k"], t["k"], None, None, None, None,
              False, None, None)
    assert len(got) == 2
    with pytest.raises(b.OscarError):
        b.int4_read(b.int4_pool(4, 2, device="cpu"), t["table"], [0, 0], [1], t["k"], t["k"])


def test_the_build_checks_the_registers_that_the_prefill_counts_on():
    from bit_rotated_kv_decode_gb300 import build
    def log(*kernels):
        return "".join(f"ptxas info    : Compiling entry function '{name}' for 'sm_103a'\nptxas info    : Function "
                       f"properties for {name}\n    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads\n"
                       f"ptxas info    : Used {regs} registers, used 2 barriers\n" for name, regs in kernels)
    name, fold = "_ZN5oscar20paged_prefill_kernelILb%dELb%dEEEv", "_ZN5oscar25paged_prefill_fold_kernelEv"
    four = [(name % (i, j), 168) for i in range(2) for j in range(2)]
    source = open(build.os.path.join(build.CSRC, "paged_prefill.cu")).read()
    assert "PF_REGS = 168," in source and build.REGISTERS["paged_prefill.cu"][2] == 168
    build.check_registers("paged_prefill.cu", log(*four, (fold, 40)))
    build.check_registers("paged_append.cu", log((fold, 40)))
    for bad in (four[:3], four[:3] + [(four[3][0], 160)], []):
        with pytest.raises(RuntimeError, match="168 registers"):
            build.check_registers("paged_prefill.cu", log(*bad, (fold, 40)))


def test_the_build_rejects_an_object_of_other_registers(small_build, monkeypatch):
    build, tmp = small_build
    monkeypatch.setattr(build, "_extension", lambda nvcc: (None, "left out"))
    monkeypatch.setattr(build, "check_registers", lambda src, out: (_ for _ in ()).throw(RuntimeError("registers")))
    for _ in range(2):                                  # no object is left that a second build would take
        with pytest.raises(RuntimeError, match="registers"):
            build.build()
        assert not (tmp / "lib" / "lib.so").exists()


@pytest.mark.parametrize("off", [1, 2, 3])
def test_error_and_lse_are_4_byte_aligned(b, off):
    """The kernels add to the error word and store the log-sum-exps as 32-bit values."""
    lib = b.load()
    for name, args, at in (("append", APPEND, 9), ("attention", ATTEND, 9)):
        for change in [dict(error=A + off)] + ([dict(lse=A + off)] if name == "attention" else []):
            v = list({**args, **change}.values())
            one = lib.oscar_bf16_append if name == "append" else lib.oscar_window_attention
            four = lib.oscar_int4_append if name == "append" else lib.oscar_int4_attention
            assert one(*v) == b.OSCAR_ERR_INVALID_ARG and b"misaligned" in lib.oscar_paged_last_error()
            v.insert(at, 128)
            assert four(*v) == b.OSCAR_ERR_INVALID_ARG and b"misaligned" in lib.oscar_paged_last_error()
    read = dict(kv=A, pages=8, table=A, max_pages=4, starts=ints(0, 3), counts=ints(4, 5), n=2, hkv=2, group=64, k=A,
                v=A, kind=1, error=A + off, stream=None)
    assert lib.oscar_int4_read(*read.values()) == b.OSCAR_ERR_INVALID_ARG


def test_an_empty_error_tensor_is_refused(on_cpu):
    """It has no word to tell a bad page in: taken as none, the error would be lost."""
    import torch
    b, t, none = on_cpu, tensors(), torch.zeros(0, dtype=torch.int32)
    with pytest.raises(b.OscarError, match="error"):
        b.window_attention(t["kv"], t["table"], [5, 9], t["q"], t["out"], 2, workspace=t["ws"], error=none)
    with pytest.raises(b.OscarError, match="error"):
        b.bf16_append(t["kv"], t["table"], [5, 9], t["k"], t["k"], error=none)
    with pytest.raises(b.OscarError, match="error"):
        b.int4_read(b.int4_pool(4, 2, device="cpu"), t["table"], [0, 0], [1, 1], t["k"].float(), t["k"].float(), error=none)
