"""GPU: attention over the 4-bit cache against the float64 definition on the same stored values
(tests/q4_reference.py, which derives each output's bound), and the whole decode chain: rotated
append into 4 bits, then attention."""
import math

import numpy as np
import pytest
import torch

from tests import q4_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def kvd():
    import kv_cache_decode_split_gb300 as m
    return m


class Case:
    def __init__(self, lens, Hq, Hkv, D, P, dtype=BF, window=0, n_sink=0, ring=False, learned=False,
                 seed=0, scale=None, vscale=1.0, qscale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.D, self.P, self.dtype = list(lens), D, P, dtype
        self.window, self.n_sink, self.ring = window, n_sink, ring
        self.scale = 1 / math.sqrt(D) if scale is None else scale
        cap = window + n_sink
        self.bt, self.pages = R.make_table([cap] * len(lens) if ring else lens, P, g)
        self.kp = R.make_pool(self.pages, Hkv, P, D, True, seed + 1)
        self.vp = R.make_pool(self.pages, Hkv, P, D, False, seed + 2, vscale)
        self.q = (torch.randn(len(lens), Hq, D, generator=g) * qscale).to(dtype)
        self.sink = torch.randn(Hq, generator=g) * 2 if learned else None

    def gpu(self):
        return dict(q=self.q.to(DEV), k_pool=torch.from_numpy(self.kp).to(DEV),
                    v_pool=torch.from_numpy(self.vp).to(DEV), block_table=self.bt.to(DEV),
                    seq_lens=torch.tensor(self.lens, dtype=I32, device=DEV), window=self.window,
                    n_sink_tokens=self.n_sink, ring=self.ring, scale=self.scale,
                    sink_logit=None if self.sink is None else self.sink.to(DEV))

    def check(self, out, lse, exclude=()):
        ref, rl, tol, tol_l = R.attention(
            self.q.float().numpy(), self.kp, self.vp, self.bt.numpy(), self.lens, self.D, self.P,
            self.scale, self.window, self.n_sink, self.ring,
            None if self.sink is None else self.sink.numpy(), self.dtype)
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        # one rounding to the output's type
        tol = tol + np.abs(ref) * float(torch.finfo(self.dtype).eps) / 2 + 1e-30
        d = np.abs(out - ref)
        assert (d <= tol).all(), f"out: {np.max(d / tol):.3g} of the bound at {np.unravel_index(np.argmax(d / tol), d.shape)}"
        none = np.isneginf(rl)
        assert np.array_equal(np.isneginf(lse), none)
        dl = np.abs(np.where(none, 0, lse) - np.where(none, 0, rl))
        assert (dl <= tol_l).all(), f"lse: {np.max(dl - tol_l):.3g} past its bound"


def run(kvd, c, **kw):
    a = c.gpu()
    a.update(kw)
    lse = torch.full(c.q.shape[:2], 55.0, device=DEV)
    err = torch.zeros(1, dtype=I32, device=DEV)
    out = kvd.attn_decode_gqa_q4(**a, lse_out=lse, err=err)
    torch.cuda.synchronize()
    return out, lse, int(err.item())


def check(kvd, c):
    out, lse, err = run(kvd, c)
    assert err == 0
    c.check(out, lse)


LENS = [0, 1, 15, 16, 17, 31, 32, 33, 64, 100, 255, 513]


@pytest.mark.parametrize("D,P", [(64, 16), (64, 64), (128, 16), (128, 32), (128, 256)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_lengths(kvd, dtype, D, P):
    check(kvd, Case(LENS, 8, 2, D, P, dtype, seed=D + P))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (14, 2), (9, 1), (16, 1), (24, 1), (40, 2), (128, 1)])
@pytest.mark.parametrize("D,dtype", [(64, F32), (128, BF), (64, BF), (128, F32)])
def test_head_groups(kvd, Hq, Hkv, D, dtype):
    check(kvd, Case([3, 77, 200], Hq, Hkv, D, 32, dtype, seed=Hq))


@pytest.mark.parametrize("window,n_sink,learned", [(1, 0, False), (17, 3, True), (100, 4, False),
                                                    (64, 40, True), (5000, 4, True), (32, 0, True)])
@pytest.mark.parametrize("ring", [False, True])
def test_windows_and_rings(kvd, window, n_sink, learned, ring):
    cap = window + n_sink
    lens = [0, 1, n_sink + 1, max(1, cap - 1), cap, cap + 1, 2 * cap + 35]
    check(kvd, Case(lens, 8, 2, 64, 16, window=window, n_sink=n_sink, ring=ring, learned=learned,
                    seed=window))
    check(kvd, Case(lens[-3:], 4, 4, 128, 64, F32 if ring else BF, window=window, n_sink=n_sink,
                    ring=ring, learned=learned, seed=window))


def test_ring_lengths_are_unbounded(kvd):
    check(kvd, Case([2 ** 31 - 1, 10 ** 6, 3], 4, 1, 64, 16, window=40, n_sink=4, ring=True))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_long_sequences_are_cut_and_joined(kvd, dtype):
    check(kvd, Case([20011, 1, 9000], 4, 2, 128, 64, dtype, learned=True, seed=9))


def test_large_scores_and_uneven_values(kvd):
    # sharp weights, negative scale, values of very different sizes from token to token
    check(kvd, Case([700, 33], 8, 2, 128, 16, qscale=20.0, seed=11))
    check(kvd, Case([700, 33], 8, 2, 64, 16, scale=-0.5, seed=12))
    c = Case([900], 4, 1, 128, 64, seed=13)
    code, s, b = R.unpack(c.vp, 128, False)
    f = (10.0 ** np.random.default_rng(0).uniform(-4, 3, s.shape[:3]))[..., None]
    c.vp = R.pack(code, (s * f).astype(np.float16), (b * f).astype(np.float16), False)
    check(kvd, c)


def test_unused_slots_may_hold_anything(kvd):
    # bytes 0xFF (NaN scales) behind each sequence's end and in unused pages
    for P in (16, 64):
        c = Case([1, 17, 40, 100], 8, 2, 128, P, seed=21)
        for pool, is_k in ((c.kp, True), (c.vp, False)):
            code, s, b = R.unpack(pool, 128, is_k)
            used = np.zeros(s.shape[:1] + (P,), bool)
            for i, L in enumerate(c.lens):
                for t in range(L):
                    used[c.bt[i, t // P], t % P] = True
            free = ~used[:, None, :, None]
            pool[:] = R.pack(np.where(free, 15, code).astype(np.uint8),
                             np.where(free, np.float16(np.nan), s), np.where(free, np.float16(np.nan), b), is_k)
        check(kvd, c)


def test_nan_rows_reach_their_heads_only(kvd):
    c = Case([50, 50], 4, 2, 64, 16, seed=22)
    code, s, b = R.unpack(c.kp, 64, True)
    b = b.copy()
    b[int(c.bt[1, 1]), 1, 3] = np.nan     # sequence 1, token 19, KV head 1
    c.kp = R.pack(code, s, b, True)
    out, lse, err = run(kvd, c)
    bad = torch.isnan(out).all(-1)
    assert err == 0 and bad.tolist() == [[False] * 4, [False, False, True, True]]


def test_repeated_calls_and_any_workspace_are_bit_equal(kvd):
    big, small = Case([3000, 70, 1], 16, 2, 128, 16, seed=31), Case([5, 900], 8, 8, 64, 64, seed=32)
    n = max(kvd.kvd_workspace_size("gqa_q4", 3, 16, 2, 128, big.bt.shape[1] * 16),
            kvd.kvd_workspace_size("gqa_q4", 2, 8, 8, 64, small.bt.shape[1] * 64))
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
    first = {}
    for c in (big, small, big, small):
        out, lse, err = run(kvd, c, workspace=ws)
        assert err == 0
        if id(c) in first:
            assert torch.equal(out, first[id(c)][0]) and torch.equal(lse, first[id(c)][1])
        else:
            c.check(out, lse)
            first[id(c)] = (out, lse)
    out, _, _ = run(kvd, big, workspace=kvd.Workspace(DEV))
    assert torch.equal(out, first[id(big)][0])


def test_bad_lengths_and_pages_are_flagged(kvd):
    c = Case([40, 60], 4, 2, 64, 16, seed=41)
    bt = c.bt.clone()
    bt[1, 2] = c.pages + 7
    out, lse, err = run(kvd, c, block_table=bt.to(DEV))
    assert err == -6 and torch.isfinite(out).all()
    good, _, _ = run(kvd, c)
    assert torch.equal(out[0], good[0])
    for lens in ([40, -1], [40, c.bt.shape[1] * 16 + 1]):
        bt = c.bt.clone()
        bt[bt < 0] = 0
        out, _, err = run(kvd, c, seq_lens=torch.tensor(lens, dtype=I32, device=DEV),
                          block_table=bt.to(DEV))
        assert err == -6 and torch.isfinite(out).all() and torch.equal(out[0], good[0])


def test_refusals_of_the_binding(kvd):
    a = Case([40, 60], 4, 2, 64, 16).gpu()
    for name, bad, what in (("q", a["q"].transpose(0, 1), ValueError), ("q", a["q"].half(), TypeError),
                            ("k_pool", a["k_pool"][..., :-4].contiguous(), ValueError),
                            ("v_pool", a["v_pool"][:2], ValueError),
                            ("block_table", a["block_table"].long(), TypeError),
                            ("seq_lens", a["seq_lens"][:1], ValueError),
                            ("sink_logit", torch.zeros(3, device=DEV), ValueError)):
        with pytest.raises(what):
            kvd.attn_decode_gqa_q4(**{**a, name: bad})
    with pytest.raises(kvd.KvdError) as e:
        kvd.attn_decode_gqa_q4(**a, workspace=torch.zeros(64, dtype=torch.uint8, device=DEV))
    assert e.value.status == -5
    with pytest.raises(kvd.KvdError):
        kvd.attn_decode_gqa_q4(**{**a, "ring": True})


def test_offsets_past_32_bits(kvd):
    # pages in the last of more than 4 GiB of each pool
    P, D, Hkv = 64, 128, 8
    page = kvd.q4_page_bytes(P, D) * Hkv
    pages = (5 << 30) // page
    c = Case([100, 200], 16, Hkv, D, P, seed=51)
    a = c.gpu()
    for n in ("k_pool", "v_pool"):
        big = torch.empty(pages, Hkv, page // Hkv, dtype=torch.uint8, device=DEV)
        big[pages - c.pages:] = a[n]
        a[n] = big
    a["block_table"] = torch.where(a["block_table"] >= 0, a["block_table"] + pages - c.pages, -1).to(I32)
    lse = torch.empty(2, 16, device=DEV)
    out = kvd.attn_decode_gqa_q4(**a, lse_out=lse)
    c.check(out, lse)


def test_two_streams_and_two_graphs_at_once(kvd):
    # without a workspace of the caller's, calls that run at the same time share nothing
    cases = [Case([6000, 3000], 8, 2, 128, 64, seed=61), Case([5000, 100, 900], 8, 2, 128, 64, seed=62)]
    args = [c.gpu() for c in cases]
    want = [kvd.attn_decode_gqa_q4(**a) for a in args]
    streams, graphs, outs = [torch.cuda.Stream() for _ in cases], [], []
    torch.cuda.synchronize()
    for a, s in zip(args, streams):
        outs.append([kvd.attn_decode_gqa_q4(**a, stream=s) for _ in range(20)])
    torch.cuda.synchronize()
    for got, w in zip(outs, want):
        assert all(torch.equal(x, w) for x in got)
    outs = []
    for a in args:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(kvd.attn_decode_gqa_q4(**a))
        graphs.append(g)
    for _ in range(10):
        for x in outs:
            x.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, w) for x, w in zip(outs, want))


@pytest.mark.parametrize("D,dtype,window,n_sink,ring", [(128, BF, 0, 0, False), (64, F32, 24, 2, True),
                                                        (64, BF, 40, 4, False)])
def test_decode_chain(kvd, D, dtype, window, n_sink, ring):
    """A prompt, then single tokens: rotated append into 4 bits and attention, captured as one graph
    whose inputs change; each step against the definition over the values handed back."""
    B, Hq, Hkv, P, prompt, steps = 3, 8, 2, 16, [50, 7, 1], 40
    g = torch.Generator().manual_seed(71)
    lens = torch.tensor(prompt, dtype=I32)
    cap = window + n_sink
    bt, pages = R.make_table([cap if ring else n + steps for n in prompt], P, g)
    kp, vp = kvd.q4_pool(pages, Hkv, P, D), kvd.q4_pool(pages, Hkv, P, D)
    table = R.table(max(prompt) + steps, D).to(DEV)
    bt_d, sl = bt.to(DEV), lens.to(DEV)
    err = torch.zeros(1, dtype=I32, device=DEV)
    W = dict(window=window if ring else 0, n_sink=n_sink if ring else 0)
    T = sum(prompt)
    mk = lambda n, h: torch.randn(n, h, D, generator=g).to(dtype).to(DEV)
    cu = torch.tensor(np.cumsum([0] + prompt), dtype=I32, device=DEV)
    ko, vo = torch.empty(T, Hkv, D, dtype=dtype, device=DEV), torch.empty(T, Hkv, D, dtype=dtype, device=DEV)
    kvd.rope_append_q4(mk(T, Hq), mk(T, Hkv), mk(T, Hkv), table, kp, vp, bt_d, sl, cu_seqlens=cu,
                       k_out=ko, v_out=vo, err=err, **W)
    q, k, v = mk(B, Hq), mk(B, Hkv), mk(B, Hkv)
    k1, v1 = torch.empty_like(k), torch.empty_like(v)
    lse = torch.empty(B, Hq, device=DEV)
    q_rot, out = torch.empty_like(q), torch.empty_like(q)

    def step():
        sl.add_(1)
        kvd.rope_append_q4(q, k, v, table, kp, vp, bt_d, sl, q_out=q_rot, k_out=k1, v_out=v1, err=err, **W)
        kvd.attn_decode_gqa_q4(q_rot, kp, vp, bt_d, sl, window=window, n_sink_tokens=n_sink, ring=ring,
                               out=out, lse_out=lse, err=err)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for i in range(steps):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=g).to(dtype))
        graph.replay()
        lens += 1
        torch.cuda.synchronize()
        if i not in (0, 1, 17, steps - 1):
            continue
        # what was handed back is what the cache holds
        for b in range(B):
            r = R.slot_of(int(lens[b]) - 1, W["window"], W["n_sink"])
            pg, at = int(bt[b, r // P]), r % P
            held = R.value(*(a[:, at] for a in R.unpack(kp[pg].cpu().numpy(), D, True)))
            assert torch.equal(torch.from_numpy(held).to(dtype), k1[b].cpu())
        c = Case.__new__(Case)
        c.q, c.kp, c.vp, c.bt, c.lens = q_rot.cpu(), kp.cpu().numpy(), vp.cpu().numpy(), bt, lens.tolist()
        c.D, c.P, c.dtype, c.scale, c.sink = D, P, dtype, 1 / math.sqrt(D), None
        c.window, c.n_sink, c.ring = window, n_sink, ring
        c.check(out, lse)
    assert int(err.item()) == 0


def wide(c, pages=16384):
    """The same call with a block table for far more tokens, as a server's is."""
    c.bt = torch.cat([c.bt, torch.full((len(c.lens), pages - c.bt.shape[1]), -1, dtype=I32)], 1)
    return c


HEADS = [(8, 2, 128, BF), (10, 2, 128, BF), (32, 2, 128, BF), (32, 2, 128, F32), (8, 2, 64, BF),
         (32, 2, 64, F32), (3, 3, 64, F32)]


@pytest.mark.parametrize("Hq,Hkv,D,dtype", HEADS)
@pytest.mark.parametrize("lens", [[0, 1, 64, 65, 700, 2500], [2000], [130] * 17, [1500, 0] * 20,
                                  [900, 33, 0, 64, 1] * 20])
def test_tables_for_short_and_for_long_sequences(kvd, Hq, Hkv, D, dtype, lens):
    # the table's width decides how the work is divided, never the answer
    c = Case(lens, Hq, Hkv, D, 32, dtype, learned=True, seed=len(lens))
    check(kvd, c)
    check(kvd, wide(c))


@pytest.mark.parametrize("Hq,Hkv,D,dtype", HEADS)
def test_sequences_that_fill_every_warp(kvd, Hq, Hkv, D, dtype):
    # long ones, cut into many pieces; then more sequences than warps
    check(kvd, Case([45000, 21000, 0, 64 * 250, 1000], Hq, Hkv, D, 64, dtype, learned=True, seed=81))
    lens = np.random.default_rng(82).integers(0, 500, 310).tolist()
    check(kvd, Case(lens, Hq, Hkv, D, 16, dtype, seed=82))


def test_windows_in_wide_tables(kvd):
    for window, n_sink in ((200, 4), (64, 64), (3000, 0)):
        check(kvd, wide(Case([5000, 70, 0, 3000, 201], 8, 2, 128, 16, window=window, n_sink=n_sink,
                             seed=window)))


def test_no_sequence_has_tokens(kvd):
    for learned in (False, True):
        c = Case([0, 0, 0], 8, 2, 128, 64, learned=learned, seed=91)
        check(kvd, c)
        check(kvd, wide(c))


def test_outputs_are_complete_for_the_next_work_of_the_stream(kvd):
    # sequences that one warp has whole, and cut ones; copied by the stream at once, no host wait
    for lens in ([60] * 300, [60] * 299 + [30000]):
        c = wide(Case(lens, 4, 4, 64, 16, seed=95), 4096)
        a = c.gpu()
        want = kvd.attn_decode_gqa_q4(**a)
        out = torch.empty_like(want)
        torch.cuda.synchronize()
        copies = []
        for _ in range(30):
            out.zero_()
            kvd.attn_decode_gqa_q4(**a, out=out)
            copies.append(out.clone())
        torch.cuda.synchronize()
        assert all(torch.equal(x, want) for x in copies)


@pytest.mark.parametrize("Hq,Hkv,D,dtype", HEADS)
def test_fewer_tiles_than_warps(kvd, Hq, Hkv, D, dtype):
    for lens in ([30000], [9000, 0, 20000], [65]):
        check(kvd, wide(Case(lens, Hq, Hkv, D, 64, dtype, learned=True, seed=len(lens))))


def test_workspace_shared_with_another_operation_on_its_own_stream(kvd):
    # the shared buffer is filled with zeros for the other operation: on the call's stream
    c = Case([30000, 700], 8, 2, 128, 64, seed=97)
    a = c.gpu()
    want = kvd.attn_decode_gqa_q4(**a)
    q, pool = a["q"], torch.zeros(8, 2, 64, 128, dtype=BF, device=DEV)
    bt, sl = torch.zeros(2, 4, dtype=I32, device=DEV), torch.full((2,), 200, dtype=I32, device=DEV)
    other = kvd.attn_decode_gqa_paged(q, pool, pool, bt, sl)
    ws, s = kvd.Workspace(DEV), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    with torch.cuda.stream(s):
        for _ in range(20):
            got.append((kvd.attn_decode_gqa_q4(**a, workspace=ws, stream=s), want))
            got.append((kvd.attn_decode_gqa_paged(q, pool, pool, bt, sl, workspace=ws), other))
    for _ in range(20):
        got.append((kvd.attn_decode_gqa_q4(**a, workspace=ws, stream=s), want))
    torch.cuda.synchronize()
    assert all(torch.equal(x, w) for x, w in got)


@pytest.mark.parametrize("Hq,Hkv,D,dtype", HEADS + [(32, 2, 64, BF)])
@pytest.mark.parametrize("lens,in_wide,tiles", [
    ([1500, 0, 65, 900] * 10, False, [1, 2]), ([300, 0, 130, 64, 6000], False, [1]),
    ([45000, 21000, 0, 1000, 30], True, [1, 2]), ([60] * 300 + [3000, 0], True, [1]),
    (np.random.default_rng(83).integers(0, 900, 600).tolist(), True, [1, 2])])
def test_a_wait_that_runs_out_leaves_nan(kvd, Hq, Hkv, D, dtype, lens, in_wide, tiles):
    """Every warp's wait for its first or second tile runs out: each output is the right one or NaN, never what an
    earlier call left in the workspace, and the call says so. The next call is right again."""
    c = Case(lens, Hq, Hkv, D, 32, dtype, seed=len(lens))
    if in_wide:
        wide(c, 4096)
    ref, rl, tol, tol_l = R.attention(c.q.float().numpy(), c.kp, c.vp, c.bt.numpy(), c.lens, D, 32, c.scale, dtype=dtype)
    tol = tol + np.abs(ref) * float(torch.finfo(dtype).eps) / 2 + 1e-30
    some = np.broadcast_to((np.array(lens) > 0)[:, None], rl.shape)
    a = c.gpu()
    ws = torch.zeros(kvd.kvd_workspace_size("gqa_q4", len(lens), Hq, Hkv, D, c.bt.shape[1] * 32), dtype=torch.uint8,
                     device=DEV)
    for n in tiles:
        run(kvd, c, workspace=ws, q=(a["q"] * -2).contiguous())
        kvd.kvd_set_option("wait_timeout_test", n)
        try:
            out, lse, err = run(kvd, c, workspace=ws, out=torch.full_like(a["q"], 55.0))
        finally:
            kvd.kvd_set_option("wait_timeout_test", 0)
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        bad = np.isnan(out).any(-1)
        assert err == (-4 if bad.any() else 0) and not (bad & ~some).any()
        # (600 sequences of 7 tiles and 2 or 3 KV heads are 3 tiles and more for each of at most 2432 warps;
        # elsewhere no warp may have a second)
        assert bad.any() or (n > 1 and len(lens) < 600)
        assert n > 1 or (bad == some).all()
        assert np.array_equal(np.isnan(out).all(-1), bad) and np.array_equal(np.isnan(lse), bad)
        good = ~bad
        assert (np.abs(out - ref)[good] <= tol[good]).all()
        both = good & some
        assert (np.abs(lse[both] - rl[both]) <= tol_l[both]).all() and np.isneginf(lse[~some]).all()
        check(kvd, c)


# bfloat16 heads of 64, more than 8 to a KV head: blocks of 16 heads, 11 warps a CTA
WIDE_GROUPS = [(32, 2, 64, BF), (24, 2, 64, BF), (20, 1, 64, BF), (9, 1, 64, BF)]


@pytest.mark.parametrize("Hq,Hkv,D,dtype", WIDE_GROUPS)
@pytest.mark.parametrize("lens", [[0, 1, 64, 65, 700, 2500], [2000], [130] * 17, [1500, 0] * 40,
                                  [900, 33, 0, 64, 1] * 24, [1100, 5, 0, 64, 65, 640] * 16])
def test_wide_groups_in_narrow_and_wide_tables(kvd, Hq, Hkv, D, dtype, lens):
    c = Case(lens, Hq, Hkv, D, 32, dtype, learned=True, seed=len(lens))
    check(kvd, c)
    check(kvd, wide(c))


@pytest.mark.parametrize("Hq,Hkv,D,dtype", WIDE_GROUPS)
def test_wide_groups_that_fill_every_warp(kvd, Hq, Hkv, D, dtype):
    check(kvd, Case([45000, 21000, 0, 64 * 250, 1000], Hq, Hkv, D, 64, dtype, learned=True, seed=81))
    lens = np.random.default_rng(82).integers(0, 500, 310).tolist()
    check(kvd, Case(lens, Hq, Hkv, D, 16, dtype, seed=82))
    for lens in ([30000], [9000, 0, 20000], [65]):
        check(kvd, wide(Case(lens, Hq, Hkv, D, 64, dtype, learned=True, seed=len(lens))))
    for window, n_sink in ((200, 4), (3000, 0)):
        check(kvd, wide(Case([5000, 70, 0, 3000, 201], Hq, Hkv, D, 16, dtype, window=window, n_sink=n_sink,
                             seed=window)))


@pytest.mark.parametrize("Hq,D,dtype", [(3, 64, BF), (3, 128, F32), (12, 64, BF)])
def test_thousands_of_sequences(kvd, Hq, D, dtype):
    c = Case(np.random.default_rng(84).integers(0, 40, 5000).tolist(), Hq, 1, D, 16, dtype, learned=True, seed=85)
    check(kvd, c)
    check(kvd, wide(c, 512))


@pytest.mark.parametrize("Hq", [4, 8])
@pytest.mark.parametrize("dtype,ratio", [(BF, 2.0 ** 20), (F32, 2.0 ** 12)])
def test_groups_of_very_different_sizes(kvd, Hq, dtype, ratio):
    # the two groups of 64 channels share a softmax reference; one's scales are far above the other's
    for qscale in (1.0, 4.0):
        c = Case([3000, 41], Hq, 1, 128, 64, dtype, qscale=qscale, seed=86)
        code, s, b = R.unpack(c.vp, 128, False)
        f = np.array([ratio ** 0.5, ratio ** -0.5])
        c.vp = R.pack(code, (s * f).astype(np.float16), (b * f).astype(np.float16), False)
        check(kvd, c)


def repeated(kvd, c, log_tokens):
    """The call of a one-sequence case whose table repeats the sequence's pages up to 2^log_tokens tokens (each
    counts as often, so the output is the sequence's): relative error of the output in the 2-norm."""
    a = c.gpu()
    times = (1 << log_tokens) // c.lens[0]
    err = torch.zeros(1, dtype=I32, device=DEV)
    lse = torch.empty(c.q.shape[:2], device=DEV)
    a["block_table"] = c.bt.repeat(1, times).to(DEV)
    a["seq_lens"] = torch.tensor([times * c.lens[0]], dtype=I32, device=DEV)
    out = kvd.attn_decode_gqa_q4(**a, lse_out=lse, err=err)
    ref, rl, _, tol_l = R.attention(c.q.float().numpy(), c.kp, c.vp, c.bt.numpy(), c.lens, c.D, c.P, c.scale, dtype=c.dtype)
    assert int(err) == 0
    # the logarithm's own rounding, and the sum's: n / 64 additions in a lane's share of a warp's part
    assert (np.abs(lse.double().cpu().numpy() - rl - math.log(times)) <= tol_l + 2.0 ** -18).all()
    return np.linalg.norm(out.double().cpu().numpy() - ref) / np.linalg.norm(ref)


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (16, 2, 128), (16, 2, 64), (32, 2, 64)])
def test_float32_sums_do_not_drift(kvd, Hq, Hkv, D):
    # Scores below 8 are held to half a step of 2^-22, by at most 8 roundings, and each moves its token's
    # weight alone; everything added up behind them is rounded, so its errors cancel: 2^-19 in all
    for log_tokens in (18, 22):
        assert repeated(kvd, Case([8192], Hq, Hkv, D, 256, F32, seed=7), log_tokens) <= 2.0 ** -19


@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (16, 2, 128), (32, 2, 128), (16, 2, 64), (32, 2, 64)])
def test_bfloat16_sums_do_not_drift(kvd, Hq, Hkv, D):
    # An output's rounding is spread over half a step, 2^-8 of a value between 1 and 2: 2^-8 / sqrt(3) at
    # most in the 2-norm. The weights' (half a step of 2^-11, spread, of at most 15 + 15 steps of a code
    # whose own spread is 4.6) add 2^-12 / sqrt(3) * 30 / 4.6 = 2^-10.1 of the same: 2^-8.6 together.
    for log_tokens in (18, 24):
        assert repeated(kvd, Case([8192], Hq, Hkv, D, 256, BF, seed=7), log_tokens) <= 2.0 ** -8.6


@pytest.mark.parametrize("learned", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (14, 2, 128), (32, 2, 128), (10, 2, 64), (24, 2, 64)])
def test_many_tokens_of_a_warp_in_many_sequences(kvd, Hq, Hkv, D, learned):
    # sums put by across the ends of pieces, with references that rise and units that one warp has whole:
    # a table repeats the pages, so every length's output is a weighted one of the same tokens
    c = Case([4096], Hq, Hkv, D, 256, BF, qscale=3.0, learned=learned, seed=87)
    a, times = c.gpu(), [900, 1, 0, 333, 40, 700, 2, 500]
    width = max(times)
    for n in ("q",):
        a[n] = a[n].repeat(len(times), 1, 1)
    a["block_table"] = c.bt.repeat(len(times), width).to(DEV)
    a["seq_lens"] = torch.tensor([t * 4096 for t in times], dtype=I32, device=DEV)
    lse = torch.empty(len(times), Hq, device=DEV)
    err = torch.zeros(1, dtype=I32, device=DEV)
    out = kvd.attn_decode_gqa_q4(**a, lse_out=lse, err=err).double().cpu().numpy()
    assert int(err) == 0
    sink = None if c.sink is None else c.sink.numpy().astype(np.float64)
    # without the sink; its share then follows from the number of repetitions
    ref, rl, tol, tol_l = R.attention(c.q.float().numpy(), c.kp, c.vp, c.bt.numpy(), c.lens, D, 256, c.scale)
    for i, t in enumerate(times):
        if t == 0:
            assert (out[i] == 0).all()
            continue
        total = rl[0] + math.log(t)
        if sink is not None:
            total = np.logaddexp(total, sink)
        share = np.exp(rl[0] + math.log(t) - total)
        want = ref[0] * share[:, None]
        lim = tol[0] + np.abs(want) * (2.0 ** -8 + tol_l[0][:, None]) + 1e-30
        assert (np.abs(out[i] - want) <= lim).all(), i
        assert (np.abs(lse[i].double().cpu().numpy() - total) <= tol_l[0] + 2.0 ** -18).all()
