"""Argument checks of the paged serving operators, before anything reaches a GPU:
fake (never dereferenced) pointers through the C ABI, host tensors through the
binding, and the rope table's angles against their formulas in 64 bits."""
import ctypes
import math
import subprocess
import sys
import sysconfig

import numpy as np
import pytest
import torch

import mla_latent_kv_nope_b200 as mla
from mla_latent_kv_nope_b200 import binding as bd
from mla_latent_kv_nope_b200 import build as bld

OK, INVALID, UNSUP, ALIGN, WS, CUDA = 0, 1, 2, 3, 4, 5
P = ctypes.c_void_p
GOOD, ODD = P(0x10000), P(0x10002)


@pytest.fixture(scope="module", autouse=True)
def lib():
    bld.build()
    return bd.load_library()


def dims(**kw):
    base = dict(B=4, H=16, d_c=512, d_r=64, d_nope=128, d_v=128, cache_capacity=256,
                dtype=bd.MLA_BF16)
    base.update(kw)
    return ctypes.byref(bd.CDims(**base))


@pytest.mark.parametrize("d", [2, 64, 128, 256])
@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("ntk", 8.0),
                                            ("yarn", 32.0)])
def test_rope_table(d, scaling, factor):
    if d == 2 and scaling == "ntk":
        with pytest.raises(mla.MLAError):
            mla.rope_table(d, scaling=scaling, factor=factor)
        return
    t = mla.rope_table(d, scaling=scaling, factor=factor, layout="interleaved")
    assert (t.d_r, t.layout) == (d, 1)
    k, base = np.arange(d // 2), 10000.0
    if scaling == "ntk":
        base *= factor ** (d / (d - 2))
    f = base ** (-2 * k / d)
    if scaling == "linear":
        f = f / factor
    if scaling == "yarn":
        at = lambda n: d * math.log(4096 / (2 * math.pi * n)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(32)), 0), min(math.ceil(at(1)), d - 1)
        g = np.clip((k - lo) / max(hi - lo, 1e-3), 0, 1)
        f = f * (1 - g) + g * f / factor
    got = np.array([v / 2.0 ** 64 for v in t.turn[:d // 2]]) * 2 * math.pi
    assert np.all(np.abs(got - f) <= 8 * 2.0 ** -52 * f + 2.0 ** -60)
    assert not any(t.turn[d // 2:])
    amp = 0.1 * math.log(factor) + 1 if scaling == "yarn" else 1.0
    assert abs(t.amplitude - amp) <= 2.0 ** -23 * amp
    assert abs(mla.rope_table(d, attention_factor=1.25).amplitude - 1.25) == 0


@pytest.mark.parametrize("kw", [
    dict(d_r=0), dict(d_r=3), dict(d_r=258), dict(base=1.0), dict(base=float("nan")),
    dict(base=float("inf")), dict(scaling="linear", factor=0.5),
    dict(scaling="yarn", factor=float("nan")), dict(scaling="yarn", factor=2.0, original_len=0.0),
    dict(scaling="yarn", factor=2.0, beta_fast=1.0), dict(scaling="yarn", factor=2.0, beta_slow=0.0),
    dict(attention_factor=float("inf"))])
def test_rope_table_refusals(kw):
    with pytest.raises(mla.MLAError) as e:
        mla.rope_table(**{"d_r": 64, **kw})
    assert e.value.status == INVALID
    with pytest.raises(ValueError, match="layout"):
        mla.rope_table(64, layout="thirds")
    with pytest.raises(ValueError, match="scaling"):
        mla.rope_table(64, scaling="cubic")


def test_rope_refusals(lib):
    t = mla.rope_table(64)

    def call(dtype=bd.MLA_BF16, table=t, n=4, H=2, x=GOOD, xt=128, xh=64, pos=GOOD, y=GOOD, yt=128,
             yh=64):
        return lib.mla_rope(dtype, ctypes.addressof(table) if table else None, n, H, x, xt, xh, pos,
                            y, yt, yh, 0, None)
    assert call(n=0) == OK
    for kw in (dict(dtype=9), dict(table=None), dict(n=-1), dict(H=0), dict(x=None), dict(y=None),
               dict(pos=None), dict(yt=63), dict(yh=0), dict(yh=63)):
        assert call(**kw) == INVALID, kw
    assert call(n=1 << 31) == UNSUP and call(H=65536) == UNSUP
    assert call(x=P(0x10001)) == ALIGN and call(pos=ODD) == ALIGN
    assert call(dtype=bd.MLA_F32, y=ODD) == ALIGN
    bad = mla.rope_table(64)
    bad.d_r = 300
    assert call(table=bad) == INVALID


def test_plan_refusals(lib):
    assert lib.mla_plan_pages_workspace_bytes() >= 4

    def plan(B=2, seq=GOOD, new=GOOD, tab=GOOD, blocks=4, free=GOOD, cap=9, cnt=GOOD, pages=9, T=8,
             qs=GOOD, pos=GOOD, slots=GOOD, req=None, so=GOOD, co=GOOD, ws=GOOD, wsb=256):
        return lib.mla_plan_pages(B, seq, new, tab, blocks, free, cap, cnt, pages, T, qs, pos, slots,
                                  req, so, co, ws, wsb, None)
    for kw in (dict(B=0), dict(blocks=0), dict(cap=-1), dict(pages=0), dict(T=-1), dict(seq=None),
               dict(new=None), dict(tab=None), dict(free=None), dict(cnt=None), dict(qs=None),
               dict(pos=None), dict(slots=None), dict(so=None), dict(co=None)):
        assert plan(**kw) == INVALID, kw
    for kw in (dict(B=65536), dict(pages=1 << 25), dict(blocks=1 << 25), dict(T=(1 << 30) + 1)):
        assert plan(**kw) == UNSUP, kw
    assert plan(slots=P(0x10004)) == ALIGN and plan(pos=ODD) == ALIGN and plan(req=ODD) == ALIGN
    assert plan(ws=None) == WS and plan(wsb=4) == WS

    def release(B=2, seq=GOOD, rel=GOOD, tab=GOOD, blocks=4, free=GOOD, cap=9, cnt=GOOD, pages=9):
        return lib.mla_release_pages(B, seq, rel, tab, blocks, free, cap, cnt, pages, None)
    for kw in (dict(B=0), dict(seq=None), dict(rel=None), dict(tab=None), dict(free=None),
               dict(cnt=None), dict(pages=0), dict(blocks=-1)):
        assert release(**kw) == INVALID, kw
    assert release(B=65536) == UNSUP and release(rel=ODD) == ALIGN


def test_write_refusals(lib):
    t, t32 = mla.rope_table(64), mla.rope_table(32)
    tp = ctypes.addressof

    def write(d=dims(), T=3, x=GOOD, st=576, g=None, eps=1e-6, tab=tp(t), pos=GOOD, slots=GOOD,
              pool=GOOD, pages=4):
        return lib.mla_cache_write_paged(d, T, x, st, g, eps, tab, pos, slots, pool, pages, None)

    def write8(d=dims(), T=3, x=GOOD, st=576, g=None, eps=1e-6, tab=tp(t), qs=GOOD, seq=GOOD,
               table=GOOD, blocks=4, pool=GOOD, sc=GOOD, pages=4):
        return lib.mla_cache_write_fp8_paged(d, T, x, st, g, eps, tab, qs, seq, table, blocks, pool,
                                             sc, pages, None)
    for f in (write, write8):
        assert f(T=0) == OK
        for kw in (dict(d=None), dict(T=-1), dict(x=None), dict(st=575), dict(eps=-1.0),
                   dict(eps=float("nan")), dict(tab=tp(t32)), dict(pool=None), dict(pages=0)):
            assert f(**kw) == INVALID, kw
        assert f(pages=1 << 25) == UNSUP
        for kw in (dict(x=P(0x10008)), dict(st=580), dict(g=P(0x10004)), dict(pool=ODD)):
            assert f(**kw) == ALIGN, kw
    assert write(slots=None) == INVALID and write(pos=None) == INVALID
    assert write(slots=P(0x10004)) == ALIGN
    # fp32 rows of 34 values are no multiple of 16 bytes.
    assert write(d=dims(dtype=bd.MLA_F32, d_c=32, d_r=2), st=36,
                 tab=tp(mla.rope_table(2))) == UNSUP
    assert write8(d=dims(d_c=256)) == INVALID or write8(d=dims(d_c=256), st=576) == UNSUP
    assert write8(d=dims(dtype=bd.MLA_F32)) == UNSUP and write8(d=dims(d_r=32), tab=tp(t32)) == UNSUP
    assert write8(d=dims(cache_capacity=257)) == INVALID       # more than 4 pages hold
    for kw in (dict(qs=None), dict(seq=None), dict(table=None), dict(sc=None), dict(blocks=0)):
        assert write8(**kw) == INVALID, kw
    assert write8(qs=ODD) == ALIGN and write8(table=ODD) == ALIGN


def test_decode_refusals(lib):
    used = ctypes.c_int(-1)
    need = lib.mla_decode_workspace_bytes(dims(), 4)

    def call(d=dims(), q=GOOD, pool=GOOD, sc=GOOD, pages=4, table=GOOD, blocks=4, seq=GOOD, scale=0.1,
             W=4, ws=GOOD, wsb=need):
        return lib.mla_decode_fp8_paged(d, q, pool, sc, pages, table, blocks, seq, scale, W, ws, wsb,
                                        ctypes.byref(used), None)
    for kw in (dict(d=None), dict(q=None), dict(pool=None), dict(sc=None), dict(pages=0),
               dict(table=None), dict(blocks=0), dict(seq=None), dict(scale=-0.5),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(W=-1), dict(W=1025),
               dict(d=dims(cache_capacity=257))):
        assert call(**kw) == INVALID, kw
    for kw in (dict(d=dims(d_c=256)), dict(d=dims(d_r=32)), dict(d=dims(dtype=bd.MLA_F32)),
               dict(pages=1 << 25)):
        assert call(**kw) == UNSUP, kw
    for kw in (dict(q=ODD), dict(pool=P(0x10008)), dict(sc=P(0x10004)), dict(seq=ODD), dict(ws=ODD)):
        assert call(**kw) == ALIGN, kw
    assert call(ws=None) == WS and call(wsb=need - 1) == WS
    assert used.value == -1


D = mla.Dims(2, 4, 512, 64, 128, 128, 128, "bf16")
bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
i4 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
i8 = lambda *s: torch.zeros(*s, dtype=torch.int64)  # noqa: E731
HOST = {
    "rope": lambda: mla.rope(mla.RopeTable(d_r=64), bf(3, 4, 64), i4(3)),
    "plan_pages": lambda: mla.plan_pages(i4(2), i4(2), i4(2, 2), i4(4), i4(1), 4, i4(3), i4(5), i8(5),
                                         i4(2), i4(1), i4(64)),
    "release_pages": lambda: mla.release_pages(i4(2), i4(2), i4(2, 2), i4(4), i4(1), 4),
    "cache_write_paged": lambda: mla.cache_write_paged(D, bf(3, 576), None, i4(3), i8(3),
                                                       bf(2, 64, 576)),
    "cache_write_fp8_paged": lambda: mla.cache_write_fp8_paged(
        D, bf(3, 576), None, i4(3), i4(2), i4(2, 2), torch.zeros(4, 64, 640, dtype=torch.uint8),
        torch.zeros(4)),
    "decode_fp8_paged": lambda: mla.decode_fp8_paged(
        D, bf(2, 4, 576), torch.zeros(4, 64, 640, dtype=torch.uint8), torch.zeros(4), i4(2, 2), i4(2),
        0.1, torch.zeros(64)),
}


@pytest.mark.parametrize("name", sorted(HOST))
def test_host_tensors_are_refused(name, monkeypatch):
    def no_lib(*a, **k):
        raise AssertionError("the library was reached with host tensors")
    monkeypatch.setattr(bd, "load_library", no_lib)
    with pytest.raises(ValueError, match="CUDA"):
        HOST[name]()


@pytest.mark.parametrize("T,H,yt,yh,ok", [
    (4, 2, 128, 64, True), (4, 2, 64, 256, True), (4, 2, 64, 64, False), (4, 2, 192, 128, True),
    (4, 2, 96, 64, False), (4, 2, 64, 192, False), (1, 2, 0, 64, True), (4, 1, 64, 0, True),
    (4, 1, 63, 0, False), (4, 2, -128, 64, True), (4, 2, -64, 64, False),
    (2, 2, 1 << 62, 1 << 61, True), (3, 3, 1 << 62, 1 << 62, False)])
def test_rope_refuses_rows_of_y_that_overlap(lib, T, H, yt, yh, ok):
    """Rows that would be written twice; calls that pass reach the launch, which fails
    without a GPU (the addresses are never used)."""
    if ok and torch.cuda.is_available():
        pytest.skip("a valid call with addresses that do not exist: only without a GPU")
    tab = mla.rope_table(64)
    got = lib.mla_rope(bd.MLA_F32, ctypes.byref(tab), T, H, GOOD, 64, 64, GOOD, GOOD, yt, yh, 0, None)
    assert got == (CUDA if ok else INVALID)


def test_paged_cache_counts_rows(monkeypatch):
    """A step planned for a number of rows is written with that many."""
    calls = []
    monkeypatch.setattr(bd, "plan_pages", lambda *a, **kw: calls.append(a[7].shape[0]))
    monkeypatch.setattr(bd, "cache_write_paged", lambda d, x, g, pos, slots, *a: calls.append(
        (x.shape[0], pos.shape[0], slots.shape[0])))
    cache = mla.PagedCache(mla.Dims(2, 16, 512, 64, 128, 128, 128, "bf16"), 4, 16, device="cpu")
    new = torch.ones(2, dtype=torch.int32)
    cache.plan(new, tokens=2)
    cache.write(torch.zeros(2, 576))
    for n in (1, 3):
        with pytest.raises(ValueError, match="planned for 2"):
            cache.write(torch.zeros(n, 576))
    cache.plan(new)
    cache.write(torch.zeros(3, 576))
    assert calls == [2, (2, 2, 2), 16, (3, 3, 3)]
    for n in (-1, 17):
        with pytest.raises(ValueError, match="tokens"):
            cache.plan(new, tokens=n)


def test_paged_cache_write_after_a_failed_plan(monkeypatch):
    """A step that was refused is not written, whatever its size: the last step's places and
    lengths are still there."""
    calls = []

    def plan_pages(*a, **kw):
        if a[7].shape[0] == 5:
            raise mla.MLAError("mla_plan_pages", 1, "invalid argument")
    monkeypatch.setattr(bd, "plan_pages", plan_pages)
    for name in ("cache_write_paged", "cache_write_fp8_paged"):
        monkeypatch.setattr(bd, name, lambda d, x, *a: calls.append(x.shape[0]))
    new = torch.ones(2, dtype=torch.int32)
    for fp8 in (False, True):
        cache = mla.PagedCache(mla.Dims(2, 16, 512, 64, 128, 128, 128, "bf16"), 4, 16, fp8=fp8,
                               device="cpu")
        with pytest.raises(ValueError, match="no step"):
            cache.write(torch.zeros(2, 576))
        cache.plan(new, tokens=2)
        with pytest.raises(ValueError, match="tokens"):
            cache.plan(new, tokens=17)
        for n in (2, 17):
            with pytest.raises(ValueError, match="no step"):
                cache.write(torch.zeros(n, 576))
        with pytest.raises(mla.MLAError):
            cache.plan(new, tokens=5)
        with pytest.raises(ValueError, match="no step"):
            cache.write(torch.zeros(5, 576))
        cache.plan(new, tokens=2)
        cache.write(torch.zeros(2, 576))
    assert calls == [2, 2]


def test_write_step_refusals(lib):
    """mla_cache_write_paged_step: mla_cache_write_paged's checks, and those of `planned`."""
    def write(T=3, slots=GOOD, planned=GOOD, x=GOOD, eps=1e-6):
        return lib.mla_cache_write_paged_step(dims(), T, x, 576, None, eps, None, None, slots, planned,
                                              GOOD, 4, None)
    assert write(T=0, planned=None) == OK
    for kw in (dict(T=0), dict(T=-1), dict(slots=None), dict(x=None), dict(eps=-1.0)):
        assert write(**kw) == INVALID, kw
    for kw in (dict(planned=ODD), dict(x=P(0x10008)), dict(slots=P(0x10004))):
        assert write(**kw) == ALIGN, kw


def test_paged_cache_states_the_step_to_the_device(monkeypatch):
    """Without a stated size the write of 16-bit pages gets the step's tokens from the plan."""
    calls = []
    monkeypatch.setattr(bd, "plan_pages", lambda *a, **kw: None)
    monkeypatch.setattr(bd, "cache_write_paged",
                        lambda d, x, g, pos, slots, pool, tab, eps, stream=None, planned=None:
                        calls.append(planned))
    cache = mla.PagedCache(mla.Dims(2, 16, 512, 64, 128, 128, 128, "bf16"), 4, 16, device="cpu")
    new = torch.ones(2, dtype=torch.int32)
    cache.plan(new)
    with pytest.raises(ValueError, match="tokens=0"):
        cache.write(torch.zeros(0, 576))
    cache.write(torch.zeros(3, 576))
    cache.plan(new, tokens=2)
    cache.write(torch.zeros(2, 576))
    assert calls[0].shape == (1,) and calls[0].data_ptr() == cache.query_start[2:].data_ptr()
    assert calls[1:] == [None]


def test_missing_calls_module_fails_every_time(tmp_path, monkeypatch):
    """The library is not loaded without the module of the short operators' calls, at the
    second attempt as little as at the first."""
    monkeypatch.setattr(bd, "_lib", None)
    monkeypatch.setattr(bd, "_calls", None)
    monkeypatch.setattr(bd, "_HERE", str(tmp_path))
    for _ in range(2):
        with pytest.raises(RuntimeError, match="missing"):
            bd.load_library(bld.LIB_PATH)
        assert bd._lib is None and bd._calls is None


def test_calls_module_of_another_torch_is_not_loaded(monkeypatch):
    """The module reads torch's structures: one that was built against another torch (or
    Python) is as good as missing."""
    monkeypatch.setattr(bd, "_lib", None)
    monkeypatch.setattr(bd, "_calls", None)
    assert bd.load_library() is not None
    for where, name, value in ((torch, "__version__", "0.0.0"),
                               (sysconfig, "get_config_var", lambda k: ".cpython-20.so")):
        with monkeypatch.context() as m:
            m.setattr(where, name, value)
            m.setattr(bd, "_lib", None)
            m.setattr(bd, "_calls", None)
            with pytest.raises(RuntimeError, match="missing"):
                bd.load_library()


def test_library_builds_without_torch(tmp_path):
    """The C ABI's library needs no torch; the calls module is for Python and is left out."""
    code = f"""
import importlib.util, sys
sys.modules["torch"] = None
spec = importlib.util.spec_from_file_location("build_alone", {bld.__file__!r})
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
b.HERE = {str(tmp_path)!r}
b.up_to_date = lambda: True
print(b.build() == b.LIB_PATH)
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.stdout.strip() == "True", r.stderr
    assert not list(tmp_path.iterdir())


def test_plan_capped_refusals(lib):
    """mla_plan_pages_capped: mla_plan_pages' checks, and a capacity within its blocks."""
    def plan(capacity=200, blocks=4, B=2, slots=GOOD, ws=GOOD):
        return lib.mla_plan_pages_capped(B, GOOD, GOOD, GOOD, blocks, capacity, GOOD, 9, GOOD, 9, 8,
                                         GOOD, GOOD, slots, None, GOOD, GOOD, ws, 256, None)
    for kw in (dict(capacity=0), dict(capacity=-1), dict(capacity=257), dict(capacity=1 << 40),
               dict(B=0), dict(blocks=0)):
        assert plan(**kw) == INVALID, kw
    assert plan(slots=P(0x10004)) == ALIGN and plan(ws=None) == WS and plan(B=65536) == UNSUP
