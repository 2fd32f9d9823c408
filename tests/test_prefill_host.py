"""Prefill attention and cache reads without a GPU: the plain implementations against differences of
their own kind, and every host-side refusal (none reaches a launch)."""
import ctypes
import math
import os
import sys

import pytest
import torch

from tests import prefill_reference as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20  # a 16-byte aligned stand-in address, never dereferenced


@pytest.fixture(scope="module")
def kvd():
    sys.path.insert(0, ROOT)
    import __graft_entry__ as g
    g._builder().build()
    import kv_cache_decode_split_gb300 as m
    return m


def test_reference_is_the_decode_of_every_prefix():
    g = torch.Generator().manual_seed(0)
    n, L, Hq, Hkv, D, W, ns = 7, 20, 4, 2, 8, 5, 2
    q, k, v = torch.randn(n, Hq, D, generator=g), torch.randn(L, Hkv, D, generator=g), torch.randn(L, Hkv, D, generator=g)
    sink = torch.randn(Hq, generator=g)
    for window, n_sink, s in ((0, 0, None), (W, ns, None), (W, 0, sink)):
        out, lse, tol, _ = R.attention(q, k, v, 0.3, window, n_sink, s, torch.float32)
        for i in range(n):
            p = L - n + i
            t = [t for t in range(p + 1) if not window or t > p - window or t < n_sink]
            for h in range(Hq):
                x = [0.3 * float(q[i, h].double() @ k[j, h // 2].double()) for j in t]
                total = sum(math.exp(y) for y in x) + (math.exp(float(s[h])) if s is not None else 0)
                want = sum(math.exp(y) / total * v[j, h // 2].double() for y, j in zip(x, t))
                assert torch.allclose(out[i, h], want, atol=1e-12) and abs(float(lse[i, h]) - math.log(total)) < 1e-12
    assert (tol > 0).all()


def test_held_positions_and_slots():
    for window, ns in ((0, 0), (5, 2), (1, 0), (3, 7)):
        for L in range(0, 30):
            held = R.held_positions(L, window, ns)
            assert held == sorted(set(held)) and len(held) == (min(L, window + ns) if window else L)
            assert sorted(R.slot_of(t, window, ns) for t in held) == list(range(len(held)))


def _packed(m, **kw):
    a = dict(q=A, k=2 * A, v=3 * A, cq=A, ck=A, out=64 * A, lse=128 * A, B=2, T=50, Tk=60, Hq=8, Hkv=2, D=64,
             qs=512, ks=128, vs=128, scale=0.125, dtype=1, window=0, sink=0, sl=None, ws=A, wsb=1 << 40, err=None)
    a.update(kw)
    vp = lambda x: None if x is None else ctypes.c_void_p(x)  # noqa: E731
    return m.lib.attn_prefill_gqa(*(vp(a[n]) for n in ("q", "k", "v", "cq", "ck", "out", "lse")), a["B"], a["T"],
                                  a["Tk"], a["Hq"], a["Hkv"], a["D"], a["qs"], a["ks"], a["vs"], a["scale"],
                                  a["dtype"], a["window"], a["sink"], vp(a["sl"]), vp(a["ws"]), a["wsb"],
                                  vp(a["err"]), None)


COMMON = [(dict(q=None), -1), (dict(out=None), -1), (dict(B=0), -1), (dict(T=-1), -1), (dict(Hq=7), -1),
          (dict(Hkv=0), -1), (dict(D=96), -2), (dict(dtype=2), -2), (dict(Hq=258, qs=258 * 64), -2),
          (dict(window=-1), -1), (dict(sink=-1), -1), (dict(sink=3), -1), (dict(scale=math.nan), -1),
          (dict(scale=math.inf), -1), (dict(q=A + 8), -1), (dict(out=64 * A + 8), -1), (dict(qs=504), -1),
          (dict(qs=516), -1), (dict(ws=None), -1), (dict(ws=A + 8), -1), (dict(wsb=16), -5),
          (dict(lse=128 * A + 2), -1), (dict(sl=A + 1), -1), (dict(err=A + 2), -1), (dict(out=A), -1),
          (dict(lse=A + 16), -1), (dict(lse=64 * A + 16), -1)]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(k=None), -1), (dict(v=None), -1), (dict(cq=None), -1), (dict(ck=None), -1), (dict(Tk=-1), -1),
    (dict(ks=120), -1), (dict(vs=132), -1), (dict(k=2 * A + 8), -1), (dict(out=2 * A + 256), -1),
    (dict(lse=3 * A + 256), -1), (dict(cq=A + 2), -1), (dict(ck=A + 1), -1)])
def test_packed_refusals(kvd, kw, status):
    assert _packed(kvd, **kw) == status


def _paged(m, **kw):
    a = dict(q=A, k=2 * A, v=16 * A, bt=A, lens=A, cq=A, out=64 * A, lse=128 * A, B=2, T=50, Hq=8, Hkv=2, D=64,
             qs=512, P=64, mp=4, np=8, scale=0.125, dtype=1, window=0, sink=0, sl=None, ws=A, wsb=1 << 40, err=None)
    a.update(kw)
    vp = lambda x: None if x is None else ctypes.c_void_p(x)  # noqa: E731
    return m.lib.attn_prefill_gqa_paged(*(vp(a[n]) for n in ("q", "k", "v", "bt", "lens", "cq", "out", "lse")),
                                        a["B"], a["T"], a["Hq"], a["Hkv"], a["D"], a["qs"], a["P"], a["mp"],
                                        a["np"], a["scale"], a["dtype"], a["window"], a["sink"], vp(a["sl"]),
                                        vp(a["ws"]), a["wsb"], vp(a["err"]), None)


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(k=None), -1), (dict(v=None), -1), (dict(bt=None), -1), (dict(lens=None), -1), (dict(cq=None), -1),
    (dict(P=48), -2), (dict(P=8), -2), (dict(P=512), -2), (dict(mp=0), -1), (dict(np=0), -1),
    (dict(np=1 << 26), -2), (dict(mp=1 << 24), -2), (dict(v=2 * A + 8), -1), (dict(out=2 * A + 256), -1),
    (dict(lse=16 * A + 256), -1), (dict(bt=A + 2), -1), (dict(lens=A + 2), -1)])
def test_paged_refusals(kvd, kw, status):
    assert _paged(kvd, **kw) == status


def test_nothing_to_do(kvd):
    assert _packed(kvd, T=0, q=None, out=None) == 0
    assert _paged(kvd, T=0, q=None, out=None) == 0
    assert _read(kvd, T=0) == 0


def _read(m, q4=False, **kw):
    a = dict(k=A, v=2 * A, bt=A, lens=A, cu=A, ko=64 * A, vo=128 * A, B=2, T=50, Hkv=2, D=64, ks=128, vs=128,
             P=64, mp=4, np=8, dtype=1, window=0, sink=0, err=None)
    a.update(kw)
    vp = lambda x: None if x is None else ctypes.c_void_p(x)  # noqa: E731
    f = m.lib.kvd_cache_read_q4 if q4 else m.lib.kvd_cache_read
    return f(*(vp(a[n]) for n in ("k", "v", "bt", "lens", "cu", "ko", "vo")), a["B"], a["T"], a["Hkv"], a["D"],
             a["ks"], a["vs"], a["P"], a["mp"], a["np"], a["dtype"], a["window"], a["sink"], vp(a["err"]), None)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(k=None), -1), (dict(v=None), -1), (dict(bt=None), -1), (dict(lens=None), -1), (dict(cu=None), -1),
    (dict(ko=None), -1), (dict(vo=None), -1), (dict(B=0), -1), (dict(T=-1), -1), (dict(Hkv=0), -1),
    (dict(D=80), -2), (dict(dtype=3), -2), (dict(P=24), -2), (dict(mp=0), -1), (dict(np=0), -1),
    (dict(window=-1), -1), (dict(sink=1), -1), (dict(window=250, sink=7), -1), (dict(ks=64), -1),
    (dict(vs=129), -1), (dict(ko=64 * A + 4), -1), (dict(k=A + 8), -1), (dict(ko=A), -1), (dict(vo=2 * A), -1),
    (dict(vo=64 * A + 128), -1), (dict(vo=64 * A + 512), -1), (dict(err=A + 1), -1), (dict(lens=A + 2), -1)])
def test_read_refusals(kvd, q4, kw, status):
    assert _read(kvd, q4, **kw) == status


def test_workspace_size(kvd):
    assert kvd.kvd_workspace_size("prefill", 1, 32, 8, 128) > 0
    for Hq, Hkv, D in ((30, 8, 128), (32, 8, 96), (258, 2, 64), (8, 0, 64)):
        assert kvd.kvd_workspace_size("prefill", 1, Hq, Hkv, D) == 0


def test_host_tensors_are_refused(kvd):
    z = torch.zeros
    i = torch.int32
    for call in (lambda: kvd.attn_prefill_gqa(z(3, 8, 64), z(3, 2, 64), z(3, 2, 64), z(2, dtype=i)),
                 lambda: kvd.attn_prefill_gqa_paged(z(3, 8, 64), z(1, 2, 16, 64), z(1, 2, 16, 64), z(1, 1, dtype=i),
                                                    z(1, dtype=i), z(2, dtype=i)),
                 lambda: kvd.cache_read(z(1, 2, 16, 64), z(1, 2, 16, 64), z(1, 1, dtype=i), z(1, dtype=i),
                                        z(2, dtype=i), z(3, 2, 64), z(3, 2, 64)),
                 lambda: kvd.cache_read_q4(z(1, 2, 576), z(1, 2, 576), z(1, 1, dtype=i), z(1, dtype=i),
                                           z(2, dtype=i), z(3, 2, 64), z(3, 2, 64))):
        with pytest.raises(TypeError, match="CUDA tensor"):
            call()


def test_the_option_that_lets_a_wait_run_out_has_a_range(kvd):
    try:
        for n in range(7):
            kvd.kvd_set_option("wait_timeout_test", n)
        for n in (-1, 7):
            with pytest.raises(kvd.KvdError):
                kvd.kvd_set_option("wait_timeout_test", n)
    finally:
        kvd.kvd_set_option("wait_timeout_test", 0)
