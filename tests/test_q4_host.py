"""The rotated append, the 4-bit rows and the attention over them without a GPU: the reference's own
layout, and every host-side refusal (none reaches a launch)."""
import ctypes
import os
import re
import shutil
import subprocess
import sys

import numpy as np
import pytest
import torch

from tests import q4_reference as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def kvd():
    sys.path.insert(0, ROOT)
    import __graft_entry__ as g
    g._builder().build()
    import kv_cache_decode_split_gb300 as m
    return m


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("is_k", [True, False])
def test_layout_holds_every_code_once(D, is_k):
    word, bit = R._address(D, is_k)
    assert len({(w, b) for w, b in zip(word.ravel(), bit.ravel())}) == 16 * D
    assert word.max() == 2 * D - 1
    # every word belongs to one token
    owner = {}
    for r in range(16):
        for w in word[r]:
            assert owner.setdefault(w, r) == r
    rng = np.random.default_rng(D)
    code = rng.integers(0, 16, (3, 2, 32, D)).astype(np.uint8)
    s, b = rng.random((2, 3, 2, 32, D // 64)).astype(np.float16)
    got = R.unpack(R.pack(code, s, b, is_k), D, is_k)
    assert all(np.array_equal(x, y) for x, y in zip(got, (code, s, b)))


def test_reference_quantiser_is_within_half_a_step():
    # |x - value| <= s / 2, what f16 rounding of b and s moves (2^-11 of b, 15 * 2^-11 of s) and
    # the float32 steps
    x = np.random.default_rng(0).standard_normal((100, 128)).astype(np.float32) * 3
    code, s, b = R.quantise(x)
    err = np.abs(R.value(code, s, b).astype(np.float64) - x).reshape(100, 2, 64).max(-1)
    s, b = s.astype(np.float64), np.abs(b.astype(np.float64))
    assert (err <= s * (0.5 + 16 * 2.0 ** -11) + b * 2.0 ** -11 + 1e-6).all()


def test_page_bytes(kvd):
    assert kvd.q4_page_bytes(16, 128) == 1152 and kvd.q4_page_bytes(64, 64) == 2304
    assert kvd.lib.kvd_q4_page_bytes(48, 128) == 0 and kvd.lib.kvd_q4_page_bytes(64, 96) == 0
    assert R.block_bytes(128) == 1152 and R.block_bytes(64) == 576
    with pytest.raises(kvd.KvdError):
        kvd.q4_page_bytes(8, 64)
    assert kvd.q4_pool(3, 2, 16, 64, device="cpu").shape == (3, 2, 576)


BASE = 1 << 24


def _append(lib, q4=False, **kw):
    a = dict(q=1, k=2, v=3, cs=4, cu=5, bt=6, sl=7, qo=8, kp=9, vp=10, ko=11, vo=12, B=2, T=6,
             Hq=8, Hkv=2, D=64, qs=512, ks=128, vs=128, rot=64, inter=0, mp=100, P=16, max_pages=4,
             num_pages=8, dt=1, W=0, ns=0, err=13)
    at = {n: (BASE * a[n] if a[n] else None) for n in
          ("q", "k", "v", "cs", "cu", "bt", "sl", "qo", "kp", "vp", "ko", "vo", "err")}
    for n, v in kw.items():
        (at if n in at else a)[n] = v
    p = lambda n: None if at[n] is None else ctypes.c_void_p(at[n])
    outs = ["qo", "kp", "vp"] + (["ko", "vo"] if q4 else [])
    f = lib.kvd_rope_append_q4 if q4 else lib.kvd_rope_append
    return f(*[p(n) for n in ["q", "k", "v", "cs", "cu", "bt", "sl"] + outs], a["B"], a["T"],
             a["Hq"], a["Hkv"], a["D"], a["qs"], a["ks"], a["vs"], a["rot"], a["inter"], a["mp"],
             a["P"], a["max_pages"], a["num_pages"], a["dt"], a["W"], a["ns"], p("err"), None)


@pytest.mark.parametrize("q4", [False, True])
def test_append_refusals(kvd, q4):
    call = lambda **kw: _append(kvd.lib, q4, **kw)
    for n in ("k", "v", "cs", "bt", "sl", "kp", "vp"):
        assert call(**{n: None}) == -1, n
        assert call(**{n: BASE + 2}) == -1, n              # misaligned
    assert call(q=None) == -1 and call(qo=None) == -1      # q and q_out go together
    assert call(cu=None) == -1                             # T != B without offsets
    assert call(B=0) == -1 and call(T=-1) == -1 and call(Hkv=0) == -1 and call(Hq=0) == -1
    assert call(mp=0) == -1 and call(num_pages=0) == -1 and call(max_pages=0) == -1
    assert call(D=96) == -2 and call(P=48) == -2 and call(P=512) == -2 and call(P=8) == -2
    assert call(dt=7) == -2
    assert call(rot=0) == -2 and call(rot=72) == -2 and call(rot=80) == -2 and call(rot=24) == -2
    assert call(W=-1) == -1 and call(ns=4) == -1           # sinks only of a rolling cache
    assert call(W=62, ns=3) == -1                          # ring larger than its table
    assert call(ks=64) == -1 and call(qs=500) == -1        # tokens overlap
    assert call(ks=132) == -1 and call(vs=130) == -1       # not 16 bytes apart
    assert call(err=BASE + 1) == -1 and call(cu=BASE + 2) == -1
    # outputs on inputs: only q_out == q, dense
    assert call(qo=BASE, qs=640) == -1
    assert call(qo=BASE + 16) == -1
    assert call(qo=2 * BASE) == -1
    if q4:
        assert call(ko=2 * BASE) == -1 and call(vo=BASE + 64) == -1
    # nothing to do is no error, and nothing is launched
    assert call(T=0, k=None, v=None, cs=None) == 0


def _attn(lib, **kw):
    a = dict(q=1, kp=2, vp=3, bt=4, sl=5, out=6, lse=7, sink=None, ws=8, err=9, B=2, Hq=8, Hkv=2,
             D=64, P=16, max_pages=4, num_pages=8, scale=0.125, dt=1, W=0, ns=0, ring=0,
             ws_bytes=1 << 34)
    at = {n: (BASE * a[n] if a[n] else None) for n in
          ("q", "kp", "vp", "bt", "sl", "out", "lse", "sink", "ws", "err")}
    for n, v in kw.items():
        (at if n in at else a)[n] = v
    p = lambda n: None if at[n] is None else ctypes.c_void_p(at[n])
    return lib.attn_decode_gqa_q4(p("q"), p("kp"), p("vp"), p("bt"), p("sl"), p("out"), p("lse"),
                                  a["B"], a["Hq"], a["Hkv"], a["D"], a["P"], a["max_pages"],
                                  a["num_pages"], a["scale"], a["dt"], a["W"], a["ns"], a["ring"],
                                  p("sink"), p("ws"), a["ws_bytes"], p("err"), None)


def test_attention_refusals(kvd):
    call = lambda **kw: _attn(kvd.lib, **kw)
    for n in ("q", "kp", "vp", "bt", "sl", "out", "ws"):
        assert call(**{n: None}) == -1, n
        assert call(**{n: BASE + 2}) == -1, n
    for n in ("lse", "sink", "err"):
        assert call(**{n: BASE + 2}) == -1, n
    assert call(B=0) == -1 and call(Hq=7) == -1 and call(max_pages=0) == -1
    assert call(scale=float("inf")) == -1
    assert call(D=96) == -2 and call(P=24) == -2 and call(dt=2) == -2 and call(Hq=512) == -2
    assert call(W=-1) == -1 and call(W=4, ns=-1) == -1
    assert call(ns=4) == -1 and call(ring=1) == -1         # without a window
    assert call(W=61, ns=4, ring=1) == -1                  # ring larger than its table
    assert call(ws_bytes=64) == -5
    # more tiles than a 32-bit count of them holds: refused, and no workspace is asked for
    big = dict(B=65536, Hq=8, Hkv=8, P=256, max_pages=1 << 15)
    assert call(**big) == -2 and kvd.kvd_workspace_size("gqa_q4", 65536, 8, 8, 64, 1 << 23) == 0
    assert kvd.kvd_workspace_size("gqa_q4", 2, 8, 2, 64, 64) > 0
    assert kvd.kvd_workspace_size("gqa_q4", 2, 8, 3, 64, 64) == 0
    assert kvd.kvd_workspace_size("gqa_q4", 2, 8, 2, 96, 64) == 0


def test_host_tensors_are_refused(kvd):
    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(TypeError, match="CUDA tensor"):
        kvd.rope_append(z(2, 8, 64), z(2, 2, 64), z(2, 2, 64), z(9, 64), z(4, 2, 16, 64),
                        z(4, 2, 16, 64), i(2, 2), i(2))
    pool = kvd.q4_pool(4, 2, 16, 64, device="cpu")
    with pytest.raises(TypeError, match="CUDA tensor"):
        kvd.rope_append_q4(None, z(2, 2, 64), z(2, 2, 64), z(9, 64), pool, pool, i(2, 2), i(2))
    with pytest.raises(TypeError, match="CUDA tensor"):
        kvd.attn_decode_gqa_q4(z(2, 8, 64), pool, pool, i(2, 2), i(2))


def _elsewhere(tmp_path, code, *without):
    """Run code where the package is a copy without some of its files: (exit code, output)."""
    src = os.path.join(ROOT, "kv_cache_decode_split_gb300")
    dst = tmp_path / "kv_cache_decode_split_gb300"
    dst.mkdir(exist_ok=True)
    for n in os.listdir(src):
        if n.endswith((".py", ".so")) and n not in without:
            shutil.copy(os.path.join(src, n), dst / n)
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True)
    return r.returncode, r.stdout + r.stderr


CALLS_ALL = """
import torch
{first}
import kv_cache_decode_split_gb300 as kvd
z, i = torch.zeros, lambda *s: torch.zeros(*s, dtype=torch.int32)
def says(f, *a):
    try:
        f(*a)
    except Exception as e:
        print(f.__name__, type(e).__name__, e)
says(kvd.attn_decode_gqa_paged, z(1, 8, 64), z(1, 2, 16, 64), z(1, 2, 16, 64), i(1, 1), i(1))
says(kvd.rope_append, None, z(2, 2, 64), z(2, 2, 64), z(9, 64), z(4, 2, 16, 64), z(4, 2, 16, 64), i(2, 2), i(2))
says(kvd.rope_append_q4, None, z(2, 2, 64), z(2, 2, 64), z(9, 64), z(4), z(4), i(2, 2), i(2))
says(kvd.attn_decode_gqa_q4, z(2, 8, 64), z(4), z(4), i(2, 2), i(2))
print(kvd.kvd_workspace_size("gqa_q4", 2, 8, 2, 64, 64) > 0)
"""
OWN = ("rope_append", "rope_append_q4", "attn_decode_gqa_q4")


def test_without_the_compiled_module_the_other_calls_work(kvd, tmp_path):
    rc, out = _elsewhere(tmp_path, CALLS_ALL.format(first=""), "_binding.so")
    assert rc == 0, out
    assert "attn_decode_gqa_paged TypeError q must be a CUDA tensor" in out and "True" in out
    for n in OWN:
        assert f"{n} ImportError _binding.so is missing" in out


def test_a_module_built_for_another_pytorch_is_refused(kvd, tmp_path):
    # its symbols may all be there, and tensors be laid out another way
    assert kvd._binding.built_for == torch.__version__
    rc, out = _elsewhere(tmp_path, CALLS_ALL.format(first="torch.__version__ = '2.0.0'"))
    assert rc == 0, out
    assert "attn_decode_gqa_paged TypeError q must be a CUDA tensor" in out and "True" in out
    for n in OWN:
        assert f"{n} ImportError _binding.so is missing or not built for this PyTorch" in out


def test_the_library_is_built_where_the_module_cannot_be(monkeypatch, tmp_path):
    import __graft_entry__ as g
    b = g._builder()
    for n in ("LIB", "BINDING", "BUILT_FOR"):
        monkeypatch.setattr(b, n, str(tmp_path / n))
    monkeypatch.setattr(b, "BUILD", str(tmp_path))
    (tmp_path / "BINDING").write_text("a module of an earlier library")

    def compiles(src, obj, verbose):
        if src.endswith(".cpp"):
            raise RuntimeError("no headers here")
        return src, ""

    def links(cmd, **kw):
        open(cmd[cmd.index("-o") + 1], "w").write("linked")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(b, "_compile", compiles)
    monkeypatch.setattr(b.subprocess, "run", links)
    with pytest.raises(RuntimeError, match="no headers here"):
        b.build()
    assert (tmp_path / "LIB").read_text() == "linked"
    assert not (tmp_path / "BINDING").exists() and not (tmp_path / "BUILT_FOR").exists()


@pytest.mark.skipif(shutil.which("nm") is None, reason="reads the library's symbol names")
def test_the_append_holds_only_kernels_that_a_call_launches(kvd):
    names = subprocess.run(["nm", "-C", os.path.join(ROOT, "kv_cache_decode_split_gb300", "libkvdecode.so")],
                           capture_output=True, text=True, check=True).stdout
    got = set(re.findall(r"rope_append_kernel<(\w+), (\d+), (\w+), (\d+), (\d+)>", names))
    # few rows; many of bfloat16, many of float32
    forms = [(t, "1", "1") for t in ("float", "__nv_bfloat16")] + [("__nv_bfloat16", "2", "4"), ("float", "1", "3")]
    want = {(t, d, q4, r, c) for t, r, c in forms for d in ("64", "128") for q4 in ("true", "false")}
    assert got == want


def test_no_unit_has_more_tiles_than_the_plan_counts(kvd, tmp_path):
    # the count that the plan chooses a form by, compiled on its own, against every length's tiles
    import __graft_entry__ as g
    b = g._builder()
    src = tmp_path / "tiles.cpp"
    src.write_text("""#include <cstdio>
        #include "kvd_host.h"
        int main() {
            long long n, w, s; int r;
            while (std::scanf("%lld %lld %lld %d", &n, &w, &s, &r) == 4)
                std::printf("%d\\n", kvd::q4_unit_tiles(n, w, s, r != 0));
        }""")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(b.nvcc()))), "include")
    subprocess.run(["g++", "-std=c++17", "-I", b.CSRC, "-I", b.INCLUDE, "-isystem", cuda, str(src), "-o",
                    str(tmp_path / "tiles")], check=True)
    cases = [(n, w, s, r) for n in (16, 64, 100, 192, 640) for w in (0, 1, 2, 63, 64, 65, 66, 130, 700)
             for s in (0, 1, 4, 64, 65, 90) for r in (0, 1)
             if not (w == 0 and (s or r)) and not (r and w + s > n)]
    said = subprocess.run([str(tmp_path / "tiles")], input="\n".join(" ".join(map(str, c)) for c in cases), text=True,
                          capture_output=True, check=True).stdout.split()
    count = lambda lo, hi: 0 if hi <= lo else (hi - 1) // 64 - lo // 64 + 1
    for (n, w, s, r), most in zip(cases, map(int, said)):
        tiles = []
        for L in range(n + 1):
            lo = max(0, L - w) if w else 0
            one = r or w == 0 or min(s, L) >= lo
            tiles.append(count(0, min(L, w + s) if r else L) if one else count(0, min(s, L)) + count(lo, L))
        assert max(tiles) <= most <= max(tiles) + 1, (n, w, s, r)


def test_a_module_without_a_version_is_refused(kvd, tmp_path):
    # one that an earlier build left
    (tmp_path / "kv_cache_decode_split_gb300").mkdir()
    (tmp_path / "kv_cache_decode_split_gb300" / "_binding.py").write_text("set_error = print\n")
    rc, out = _elsewhere(tmp_path, CALLS_ALL.format(first=""), "_binding.so")
    assert rc == 0, out
    for n in OWN:
        assert f"{n} ImportError _binding.so is missing or not built for this PyTorch" in out
