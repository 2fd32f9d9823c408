"""GPU: causal attention of many new tokens of each sequence, packed and over a paged cache, against the
float64 definition (tests/prefill_reference.py, which derives each output's bound)."""
import math

import pytest
import torch

from tests import prefill_reference as R
from tests import q4_reference as Q

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
NAN = float("nan")


@pytest.fixture(scope="module")
def kvd():
    import kv_cache_decode_split_gb300 as m
    return m


def cu(n):
    return torch.tensor([0] + list(torch.tensor(list(n)).cumsum(0)), dtype=I32, device=DEV)


class Case:
    """new[b] new tokens of sequence b, lens[b] keys with them."""

    def __init__(self, new, lens, Hq, Hkv, D, dtype=BF, window=0, n_sink=0, learned=False, seed=0,
                 scale=None, qscale=1.0, pad=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
        self.new, self.lens, self.Hkv, self.D, self.dtype, self.pad = list(new), list(lens), Hkv, D, dtype, pad
        self.window, self.n_sink = window, n_sink
        self.scale = 1 / math.sqrt(D) if scale is None else scale
        self.q = (rnd(sum(new) + pad, Hq, D) * qscale).to(dtype)
        self.k = [(rnd(n, Hkv, D) + 0.5 * rnd(Hkv, D)).to(dtype) for n in lens]
        self.v = [rnd(n, Hkv, D).to(dtype) for n in lens]
        self.sink = rnd(Hq) * 2 if learned else None
        self.g = g

    def more(self):
        return dict(window=self.window, n_sink_tokens=self.n_sink, sink_logit=self.sink, scale=self.scale)

    def packed(self, kvd, **kw):
        k = torch.cat(self.k + [torch.full((3, self.Hkv, self.D), NAN, dtype=self.dtype, device=DEV)])
        v = torch.cat(self.v + [torch.full((3, self.Hkv, self.D), NAN, dtype=self.dtype, device=DEV)])
        return self.call(kvd.attn_prefill_gqa, (self.q, k, v, cu(self.new), cu(self.lens)), **kw)

    def pools(self, P):
        """Pages of the caches; whatever is not a token's row is NaN."""
        bt, pages = Q.make_table([max(1, n) for n in self.lens], P, torch.Generator().manual_seed(P))
        pools = []
        for rows in (self.k, self.v):
            pool = torch.full((pages, self.Hkv, P, self.D), NAN, dtype=self.dtype, device=DEV)
            for b, x in enumerate(rows):
                for i in range(0, x.shape[0], P):
                    y = x[i:i + P]
                    pool[int(bt[b, i // P]), :, :y.shape[0]] = y.transpose(0, 1)
            pools.append(pool)
        return pools + [bt.to(DEV), torch.tensor(self.lens, dtype=I32, device=DEV)]

    def paged(self, kvd, P, **kw):
        return self.call(kvd.attn_prefill_gqa_paged, (self.q, *self.pools(P), cu(self.new)), **kw)

    def call(self, f, args, **kw):
        out, lse = torch.full_like(self.q, 77.0), torch.full(self.q.shape[:2], 55.0, device=DEV)
        err = torch.zeros(1, dtype=I32, device=DEV)
        f(*args, **{**self.more(), **dict(out=out, lse_out=lse, err=err), **kw})
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        return out, lse

    def check(self, out, lse, what=""):
        at = 0
        for b, n in enumerate(self.new):
            r = R.attention(self.q[at:at + n], self.k[b], self.v[b], self.scale, self.window, self.n_sink,
                            self.sink, self.dtype)
            R.compare(out[at:at + n], lse[at:at + n], *r, what=f"{what} sequence {b}")
            at += n
        assert (out[at:] == 77.0).all() and (lse[at:] == 55.0).all(), "padding rows were written"


def check(kvd, c, P=64):
    c.check(*c.packed(kvd), "packed")
    c.check(*c.paged(kvd, P), "paged")


@pytest.mark.parametrize("D,P", [(64, 16), (128, 64), (128, 256), (64, 128), (128, 32)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_prompts_of_many_lengths(kvd, dtype, D, P):
    n = [1, 2, 0, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300]
    check(kvd, Case(n, n, 8, 2, D, dtype, seed=D + P, pad=5), P)


@pytest.mark.parametrize("D,P", [(64, 64), (128, 16), (128, 128)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_chunks_behind_prefixes(kvd, dtype, D, P):
    new = [1, 5, 17, 64, 130, 3, 1, 0, 200]
    lens = [1, 700, 17, 65, 500, 128, 129, 40, 1000]
    check(kvd, Case(new, lens, 8, 2, D, dtype, seed=D, pad=1), P)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (14, 2), (9, 1), (16, 1), (24, 1), (40, 2), (65, 1), (128, 1)])
@pytest.mark.parametrize("D,dtype", [(64, F32), (128, BF), (64, BF), (128, F32)])
def test_head_groups(kvd, Hq, Hkv, D, dtype):
    check(kvd, Case([3, 50, 1], [3, 77, 200], Hq, Hkv, D, dtype, seed=Hq), 32)


@pytest.mark.parametrize("window,n_sink,learned", [(1, 0, False), (17, 3, True), (100, 4, False),
                                                    (128, 128, False), (64, 140, True), (5000, 4, True),
                                                    (32, 0, True), (200, 300, False)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_windows_and_sinks(kvd, dtype, window, n_sink, learned):
    new, lens = [1, 90, 400, 33], [600, 90, 700, 513]
    check(kvd, Case(new, lens, 8, 2, 64, dtype, window, n_sink, learned, seed=window))
    check(kvd, Case(new, lens, 4, 4, 128, dtype, window, n_sink, learned, seed=window), 16)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_that_see_nothing(kvd, dtype):
    # more new tokens than keys: the leading ones see nothing
    for learned in (False, True):
        c = Case([5, 200, 3, 140], [3, 90, 0, 1], 8, 2, 64, dtype, learned=learned, seed=3)
        out, lse = c.packed(kvd)
        c.check(out, lse)
        assert (out[:2] == 0).all()
    c = Case([700], [10], 8, 2, 128, dtype, seed=5)  # a call whose work list new tokens fill
    c.check(*c.packed(kvd))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_keys_fewer_than_new_tokens_are_recorded_in_a_cache(kvd, dtype):
    c = Case([5, 20], [3, 40], 8, 2, 128, dtype, seed=4)
    out, lse = torch.empty_like(c.q), torch.empty(c.q.shape[:2], device=DEV)
    err = torch.zeros(1, dtype=I32, device=DEV)
    kvd.attn_prefill_gqa_paged(c.q, *c.pools(16), cu(c.new), out=out, lse_out=lse, err=err, **c.more())
    assert int(err.item()) == -6
    c.check(out, lse)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window", [0, 100])
def test_values_that_are_not_finite_reach_their_rows_alone(kvd, dtype, window):
    c = Case([150, 300, 60], [150, 420, 60], 4, 2, 128, dtype, window=window, n_sink=2 if window else 0, seed=5)
    c.v[0][100, 0, 3] = math.inf
    c.v[1][250, 1, :] = NAN
    c.v[1][300, 0, 64] = -math.inf
    c.v[1][1, 0, 5] = -math.inf
    c.v[2][59, :, 0] = NAN  # the last token: seen by itself alone
    check(kvd, c)
    c = Case([300], [300], 2, 1, 64, dtype, window=window, n_sink=2 if window else 0, seed=6)
    c.v[0][130, 0, 3] = math.inf
    c.v[0][131, 0, 3] = -math.inf  # both: NaN
    check(kvd, c, 16)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_keys_that_are_not_finite_reach_their_rows_alone(kvd, dtype):
    c = Case([200, 40], [200, 300], 4, 2, 64, dtype, seed=7)
    c.k[0][150, 0, 5] = NAN
    c.k[1][290, 1, 0] = NAN
    out, lse = c.packed(kvd)
    for name, o, l in (("packed", out, lse), ("paged", *c.paged(kvd, 32))):
        o, l = o.float(), l
        assert torch.isnan(o[150:200, :2]).all() and torch.isnan(o[200 + 30:, 2:]).all(), name
        c2 = Case([200, 40], [200, 300], 4, 2, 64, dtype, seed=7)
        ref, _ = c2.packed(kvd)
        assert torch.equal(o[:150], ref[:150].float()) and torch.equal(o[:, 2:][:200], ref[:, 2:][:200].float())
        assert torch.equal(o[200:, :2], ref[200:, :2].float()) and torch.equal(o[200:230], ref[200:230].float())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_large_scores(kvd, dtype):
    # sharp weights, maxima that grow along the keys, a negative scale
    c = Case([300, 40], [300, 900], 8, 2, 128, dtype, qscale=20.0, seed=11)
    for k in c.k:
        k *= torch.linspace(0.01, 3.0, k.shape[0], device=DEV).to(dtype)[:, None, None]
    check(kvd, c, 16)
    check(kvd, Case([300], [400], 8, 2, 64, dtype, scale=-0.5, seed=12))
    check(kvd, Case([300], [400], 8, 2, 64, dtype, scale=0.0, seed=12))


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 32, 8), (64, 28, 4)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_long_sequences_are_cut_and_joined(kvd, dtype, D, Hq, Hkv):
    # few rows over long caches, whole prompts, and both in one call
    check(kvd, Case([4, 1, 7], [9001, 5000, 130], Hq, Hkv, D, dtype, seed=9))
    check(kvd, Case([1700, 3, 900], [1700, 2500, 2111], Hq, Hkv, D, dtype, learned=True, seed=10), 256)
    check(kvd, Case([700, 3], [6000, 2500], Hq, Hkv, D, dtype, window=1000, n_sink=5, seed=10), 32)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_slices_of_a_projection(kvd, dtype):
    Hq, Hkv, D, n = 8, 2, 64, [70, 3, 200]
    T = sum(n)
    g = torch.Generator(device=DEV).manual_seed(1)
    qkv = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device=DEV).to(dtype)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    out = kvd.attn_prefill_gqa(q, k, v, cu(n))
    want = kvd.attn_prefill_gqa(q.contiguous(), k.contiguous(), v.contiguous(), cu(n), cu(n))
    assert torch.equal(out, want)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_token_of_each_sequence_is_the_decode(kvd, dtype):
    lens = [1, 64, 700, 129, 5000]
    c = Case([1] * 5, lens, 32, 8, 128, dtype, seed=2)
    kp, vp, bt, sl = c.pools(64)
    lse = torch.empty(5, 32, device=DEV)
    out = kvd.attn_prefill_gqa_paged(c.q, kp, vp, bt, sl, lse_out=lse, **c.more())
    c.check(out, lse)
    other = kvd.attn_decode_gqa_paged(c.q, kp.nan_to_num(), vp.nan_to_num(), bt.clamp_min(0), sl, scale=c.scale)
    tol = 2.0 ** -6 if dtype == BF else 1e-5  # two kernels, each within its own bound
    assert (out.float() - other.float()).abs().max() <= tol


def test_streams_graphs_and_shared_workspaces(kvd):
    cs = [Case([300, 5], [300, 3000], 8, 2, 128, BF, seed=20), Case([64, 64], [900, 70], 8, 2, 128, BF, seed=21)]
    want = [c.paged(kvd, 64) for c in cs]
    args = [(c.q, *c.pools(64), cu(c.new)) for c in cs]
    outs = [torch.zeros_like(c.q) for c in cs]
    # two streams at once, each call with memory of its own
    ss = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        for a, o, s in zip(args, outs, ss):
            kvd.attn_prefill_gqa_paged(*a, out=o, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w[0])
    # one workspace, two captured graphs replayed in turn; replayed on other inputs
    ws = torch.full((kvd.kvd_workspace_size("prefill", 2, 8, 2, 128),), 255, dtype=torch.uint8, device=DEV)
    graphs = []
    for a, o in zip(args, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kvd.attn_prefill_gqa_paged(*a, out=o, workspace=ws)
        graphs.append(g)
    for o in outs:
        o.zero_()
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w[0])
    q = args[0][0].clone()
    args[0][0].copy_(q.flip(0))
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], kvd.attn_prefill_gqa_paged(*args[0]))
    # a Workspace object
    assert torch.equal(kvd.attn_prefill_gqa_paged(*args[1], workspace=kvd.Workspace()), want[1][0])


def test_results_do_not_depend_on_timing(kvd):
    c = Case([900, 3, 40], [3000, 7000, 40], 8, 2, 128, BF, seed=22)
    a = (c.q, *c.pools(64), cu(c.new))
    first = kvd.attn_prefill_gqa_paged(*a)
    for _ in range(20):
        assert torch.equal(kvd.attn_prefill_gqa_paged(*a), first)


def test_bad_offsets_lengths_and_pages_are_recorded(kvd):
    c = Case([20, 30], [20, 30], 8, 2, 64, BF, seed=23)
    k, v = torch.cat(c.k), torch.cat(c.v)

    def run(cq, ck):
        out = torch.full_like(c.q, 77.0)
        err = torch.zeros(1, dtype=I32, device=DEV)
        kvd.attn_prefill_gqa(c.q, k, v, torch.tensor(cq, dtype=I32, device=DEV),
                             torch.tensor(ck, dtype=I32, device=DEV), out=out, err=err)
        return out, int(err.item())

    good, e = run([0, 20, 50], [0, 20, 50])
    assert e == 0
    out, e = run([0, 20, 51], [0, 20, 50])
    assert e == -6 and torch.equal(out[:20], good[:20]) and (out[20:] == 77).all()
    out, e = run([0, 20, 10], [0, 20, 50])
    assert e == -6 and torch.equal(out[:20], good[:20]) and (out[20:] == 77).all()
    out, e = run([0, 20, 50], [0, 20, 60])
    assert e == -6 and torch.equal(out[:20], good[:20]) and (out[20:] == 77).all()
    out, e = run([0, 20, 50], [0, -1, 50])
    assert e == -6
    kp, vp, bt, sl = c.pools(16)
    kp, vp = kp.nan_to_num(), vp.nan_to_num()
    for table, lens in ((bt.clone(), sl.clone()), (bt.clone(), sl.clone())):
        err = torch.zeros(1, dtype=I32, device=DEV)
        kvd.attn_prefill_gqa_paged(c.q, kp, vp, table, lens, cu(c.new), err=err)
        assert int(err.item()) == 0
    for page in (-1, kp.shape[0], 2 ** 30):
        table = bt.clone()
        table[1, 0] = page
        err = torch.zeros(1, dtype=I32, device=DEV)
        out = kvd.attn_prefill_gqa_paged(c.q, kp, vp, table, sl, cu(c.new), err=err)
        assert int(err.item()) == -6 and torch.isfinite(out.float()).all()
    for length in (-1, 16 * bt.shape[1] + 1, 2 ** 31 - 1):
        lens = sl.clone()
        lens[1] = length
        err = torch.zeros(1, dtype=I32, device=DEV)
        out = kvd.attn_prefill_gqa_paged(c.q, kp, vp, bt.clamp_min(0), lens, cu(c.new), err=err)
        assert int(err.item()) == -6 and torch.isfinite(out.float()).all()


def test_offsets_past_32_bits(kvd):
    # pools of more than 2^31 elements each, a few long sequences at their end
    Hkv, D, P = 8, 128, 256
    pages = 8300
    assert pages * Hkv * P * D > 2 ** 31
    kp = torch.zeros(pages, Hkv, P, D, dtype=BF, device=DEV)
    vp = torch.zeros(pages, Hkv, P, D, dtype=BF, device=DEV)
    c = Case([9, 300], [1000, 513], 8, 8, D, BF, seed=24)
    bt = torch.tensor([[pages - 1, pages - 3, pages - 2, 0], [pages - 5, 1, pages - 4, -1]], dtype=I32, device=DEV)
    for pool, rows in ((kp, c.k), (vp, c.v)):
        for b, x in enumerate(rows):
            for i in range(0, x.shape[0], P):
                y = x[i:i + P]
                pool[int(bt[b, i // P]), :, :y.shape[0]] = y.transpose(0, 1)
    sl = torch.tensor(c.lens, dtype=I32, device=DEV)
    c.check(*c.call(kvd.attn_prefill_gqa_paged, (c.q, kp, vp, bt, sl, cu(c.new))))
    del kp, vp
    # packed rows whose tokens lie far apart
    wide = 1 << 22
    buf = torch.zeros(813, wide, dtype=BF, device=DEV)
    k, v = (buf.as_strided((813, Hkv, D), (wide, D, 1), wide - (i + 1) * Hkv * D) for i in (0, 1))
    c = Case([9, 300], [500, 313], 8, 8, D, BF, seed=25)
    k.copy_(torch.cat(c.k))
    v.copy_(torch.cat(c.v))
    c.check(*c.call(kvd.attn_prefill_gqa, (c.q, k, v, cu(c.new), cu(c.lens))))


def test_many_short_sequences(kvd):
    g = torch.Generator().manual_seed(0)
    new = torch.randint(0, 4, (700,), generator=g).tolist()
    lens = [n + int(torch.randint(0, 90, (1,), generator=g)) for n in new]
    c = Case(new, lens, 4, 2, 64, BF, seed=26)
    c.check(*c.packed(kvd))
    c.check(*c.paged(kvd, 16))


def test_append_then_attend_and_read_back(kvd):
    """The operators as they are used together: prompts appended to a 4-bit cache, later chunks appended,
    everything read back, and the chunks' attention over it; the same over a plain cache; and chunks
    behind a rolling cache."""
    Hq, Hkv, D, P = 8, 2, 128, 16
    g = torch.Generator(device=DEV).manual_seed(30)
    old, new = [100, 33, 0], [40, 5, 70]
    full = [a + b for a, b in zip(old, new)]
    table = Q.table(256, D).to(DEV)
    bt, pages = Q.make_table(full, P, torch.Generator().manual_seed(1))
    bt = bt.to(DEV)
    rnd = lambda n, h: torch.randn(n, h, D, generator=g, device=DEV).to(BF)  # noqa: E731
    qs, ks, vs = ([rnd(sum(n), h) for n in (old, new)] for h in (Hq, Hkv, Hkv))
    sl = [torch.tensor(x, dtype=I32, device=DEV) for x in (old, full)]
    for q4 in (True, False):
        append = kvd.rope_append_q4 if q4 else kvd.rope_append
        kp, vp = ((kvd.q4_pool(pages, Hkv, P, D) for _ in range(2)) if q4 else
                  (torch.full((pages, Hkv, P, D), NAN, dtype=BF, device=DEV) for _ in range(2)))
        append(qs[0], ks[0], vs[0], table, kp, vp, bt, sl[0], cu(old))
        q = append(qs[1], ks[1], vs[1], table, kp, vp, bt, sl[1], cu(new))
        k, v = (torch.empty(sum(full), Hkv, D, dtype=BF, device=DEV) for _ in range(2))
        (kvd.cache_read_q4 if q4 else kvd.cache_read)(kp, vp, bt, sl[1], cu(full), k, v)
        c = Case(new, full, Hq, Hkv, D, BF)
        c.q, c.k, c.v = q, list(k.split(full)), list(v.split(full))
        c.check(*c.call(kvd.attn_prefill_gqa, (q, k, v, cu(new), cu(full))))
        if not q4:
            c.check(*c.call(kvd.attn_prefill_gqa_paged, (q, kp, vp, bt, sl[1], cu(new))))
    # a rolling cache of 20 + 3: what it holds, then the chunk's own rows behind it
    W, ns = 20, 3
    bt, pages = Q.make_table([W + ns] * 3, P, torch.Generator().manual_seed(2))
    bt = bt.to(DEV)
    kp, vp = (torch.zeros(pages, Hkv, P, D, dtype=BF, device=DEV) for _ in range(2))
    kvd.rope_append(None, ks[0], vs[0], table, kp, vp, bt, sl[0], cu(old), window=W, n_sink=ns)
    held = [len(R.held_positions(n, W, ns)) for n in old]
    rows = [h + n for h, n in zip(held, new)]
    k, v = (torch.zeros(sum(rows), Hkv, D, dtype=BF, device=DEV) for _ in range(2))
    kvd.cache_read(kp, vp, bt, sl[0], cu(rows), k, v, window=W, n_sink=ns)
    at = cu(rows)[:-1].long()
    where = torch.cat([at[b] + held[b] + torch.arange(n, device=DEV) for b, n in enumerate(new)])
    k[where], v[where] = ks[1], vs[1]
    c = Case(new, rows, Hq, Hkv, D, BF, window=W, n_sink=ns)
    c.q, c.k, c.v = qs[1], list(k.split(rows)), list(v.split(rows))
    c.check(*c.call(kvd.attn_prefill_gqa, (qs[1], k, v, cu(new), cu(rows))))


def test_float32_values_beyond_bfloat16_count_as_infinite(kvd):
    """3.4e38 is a float32 number that rounds to a bfloat16 infinity: infinite for the rows that see it,
    nothing for the others, also those of the same tile."""
    c = Case([150, 40], [150, 300], 4, 2, 64, F32, seed=30)
    ref, _ = c.packed(kvd)
    c.v[0][100, 0, 3], c.v[0][90, 1, 5], c.v[1][270, 0, 60] = 3.4e38, 3.38e38, -3.4e38
    for out in (c.packed(kvd)[0], c.paged(kvd, 16)[0]):
        assert (out[100:150, :2, 3] == math.inf).all() and (out[150 + 10:, :2, 60] == -math.inf).all()
        same = torch.ones_like(ref, dtype=torch.bool)
        same[100:150, :2, 3] = same[160:, :2, 60] = same[90:150, 2:, 5] = False
        assert torch.equal(out[same], ref[same])
        assert torch.isfinite(out[90:150, 2:, 5]).all()  # 3.38e38 is a number like others


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 4), (128, 32, 8)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_outputs_that_begin_at_16_bytes(kvd, dtype, D, Hq, Hkv):
    c = Case([1, 130, 5], [900, 130, 260], Hq, Hkv, D, dtype, seed=31)
    step = 16 // c.q.element_size()
    room = torch.full((c.q.numel() + 2 * step,), 77.0, dtype=dtype, device=DEV)
    out = room[step:-step].view(c.q.shape)
    assert out.data_ptr() % 32 == 16
    for f in (lambda **kw: c.packed(kvd, **kw), lambda **kw: c.paged(kvd, 64, **kw)):
        want, _ = f()
        f(out=out)
        assert torch.equal(out, want)
        assert (room[:step] == 77).all() and (room[-step:] == 77).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_replayed_graph_follows_its_lengths(kvd, dtype):
    """Captured with short caches (no unit would be cut), replayed with long ones, other offsets and
    empty sequences, and back."""
    c = Case([5, 0, 40], [4000, 300, 2500], 8, 2, 128, dtype, seed=40)
    kp, vp, bt, _ = c.pools(64)
    sl, at = torch.zeros(3, dtype=I32, device=DEV), torch.zeros(4, dtype=I32, device=DEV)
    err = torch.zeros(1, dtype=I32, device=DEV)
    ws = torch.empty(kvd.kvd_workspace_size("prefill", 3, 8, 2, 128), dtype=torch.uint8, device=DEV)
    out, lse = torch.empty_like(c.q), torch.empty(45, 8, device=DEV)

    def call(**kw):
        kvd.attn_prefill_gqa_paged(c.q, kp, vp, bt, sl, at, out=out, lse_out=lse, workspace=ws, err=err, **kw)

    def lengths(new, lens):
        sl.copy_(torch.tensor(lens, dtype=I32))
        at.copy_(cu(new))

    short, long_, other = ([5, 0, 40], [9, 0, 41]), ([5, 0, 40], [4000, 300, 2500]), ([1, 44, 0], [1, 290, 7])
    lengths(*short)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for new, lens in (short, long_, other, short, long_):
        lengths(new, lens)
        out.fill_(77)
        graph.replay()
        got, got_lse = out.clone(), lse.clone()
        out.fill_(77)
        call()
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        assert torch.equal(got, out) and torch.equal(got_lse, lse)
        cut = Case.__new__(Case)
        cut.__dict__.update(c.__dict__)
        cut.new, cut.lens = new, lens
        cut.k, cut.v = [k[:n] for k, n in zip(c.k, lens)], [v[:n] for v, n in zip(c.v, lens)]
        cut.check(got, got_lse, f"{lens}")


@pytest.mark.parametrize("scale", [-0.125, 0.0, 3.0])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_scales(kvd, dtype, scale):
    check(kvd, Case([1, 70, 200], [300, 70, 333], 6, 2, 64, dtype, scale=scale, window=90, n_sink=3, seed=41), 32)


def fastest(f, n=6):
    """Milliseconds of the quickest of n calls behind a first one."""
    best = math.inf
    for i in range(n + 1):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        f()
        b.record()
        b.synchronize()
        if i:
            best = min(best, a.elapsed_time(b))
    return best


def strew(c, share, seed):
    """Infinities and NaN in a share of the values."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    for v in c.v:
        r = torch.rand(v.shape, generator=g, device=DEV)
        kind = torch.randint(0, 3, v.shape, generator=g, device=DEV)
        bad = torch.tensor([math.inf, -math.inf, NAN], device=DEV)[kind].to(v.dtype)
        v.copy_(torch.where(r < share, bad, v))


# dtypes of the tests of values that are not finite
NOT_FINITE = [F32, BF]


@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 128), (2, 2, 64), (14, 2, 64), (65, 1, 128)])
@pytest.mark.parametrize("window,n_sink", [(0, 0), (1, 0), (70, 3), (200, 100), (64, 140)])
@pytest.mark.parametrize("dtype", NOT_FINITE)
def test_many_values_that_are_not_finite(kvd, dtype, window, n_sink, Hq, Hkv, D):
    for share in (0.001, 0.5) if Hq < 10 else (0.002,):
        c = Case([150, 200, 5, 1], [150, 420, 300, 200], Hq, Hkv, D, dtype, window=window, n_sink=n_sink, seed=50)
        strew(c, share, 51)
        check(kvd, c, 32)


@pytest.mark.parametrize("dtype", NOT_FINITE)
def test_values_that_are_not_finite_in_cut_units(kvd, dtype):
    c = Case([4, 1, 300], [3001, 1500, 2111], 8, 2, 128, dtype, seed=52)
    strew(c, 0.0005, 53)
    check(kvd, c, 64)


@pytest.mark.parametrize("new,n", [(8192, 8192), (1, 65536), (200, 65536)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", NOT_FINITE)
def test_a_value_that_is_not_finite_costs_little(kvd, dtype, D, new, n):
    """Near the start of a long sequence: no wait may run out for it, its rows alone change, in its column
    alone, and the call takes about the time that it takes without."""
    Hq, Hkv = 4, 2
    c = Case([new, 40], [n, 300], Hq, Hkv, D, dtype, seed=54)
    cq, ck = cu(c.new), cu(c.lens)
    k, v = torch.cat(c.k), torch.cat(c.v)
    out, err = torch.empty_like(c.q), torch.zeros(1, dtype=I32, device=DEV)

    def call():
        kvd.attn_prefill_gqa(c.q, k, v, cq, ck, out=out, err=err)

    clean = fastest(call)
    ref = out.clone()
    v[1, 0, 5], v[n // 2, 1, D - 1] = -math.inf, NAN
    first = n - new  # position of the first row
    want = ref.clone()
    want[max(0, 1 - first):new, :Hq // Hkv, 5] = -math.inf
    want[max(0, n // 2 - first):new, Hq // Hkv:, D - 1] = NAN
    time = fastest(call)
    assert int(err.item()) == 0
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert torch.equal(out.nan_to_num(7.0), want.nan_to_num(7.0))
    assert time <= 1.5 * clean + 0.005, f"{time:.3f} ms, {clean:.3f} without"
    # all of them
    v[:n] = NAN
    call()
    assert torch.isnan(out[:new]).all() and torch.equal(out[new:], ref[new:]) and int(err.item()) == 0


@pytest.mark.parametrize("rise", [7.5, 8.5, 60.0])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_large_values_stay_numbers(kvd, dtype, rise):
    """A score that lies 2^rise above all before it, and large values there: with a row's weights at most 1
    the sums are the values themselves. Masked by a window, at the end of a unit, and in cut units."""
    for new, L in ((300, 300), (3, 4000)):
        for D in (64, 128):
            c = Case([new], [L], 4, 2, D, dtype, scale=1.0, seed=60)
            c.q.zero_()
            c.q[:, :, 0] = 1
            c.k[0][:, :, 0] = 0
            c.k[0][L - 2, :, 0] = rise * math.log(2)
            c.v[0][L - 2] = (c.v[0][L - 2] / c.v[0][L - 2].abs().amax() * 2.0 ** 127).to(dtype)
            check(kvd, c)


def repeated(q, k, v, L, scale, window=0, n_sink=0, sink=None, tiles=512):
    """prefill_reference.attention of one sequence whose L keys are those of k and v [U, Hkv, D] over and over:
    position t has key t % U. float64 outputs, lse and their bounds, for sums of which a tensor core cuts those of
    `tiles` tiles of 128 keys, 16 keys at a time (2^-23 of what has been added up), and the rest is rounded."""
    n, Hq, D = q.shape
    U, Hkv = k.shape[:2]
    pos = L - n + torch.arange(n, device=DEV)[:, None]
    at = torch.arange(U, device=DEV)[None, :]
    count = lambda x: (x - at + U - 1).clamp_min(0) // U  # noqa: E731 (of at's positions below x)
    low = (pos - window + 1).clamp_min(0) if window else torch.zeros_like(pos)
    times = (count(pos + 1) - count(low) + count(low.clamp_max(n_sink))).to(torch.float64)
    out = torch.empty(n, Hq, D, dtype=torch.float64, device=DEV)
    lse, tol, tol_l = torch.empty(n, Hq, dtype=torch.float64, device=DEV), torch.empty_like(out), None
    tol_l = torch.empty_like(lse)
    adds = tiles * 8 + L / (128 * tiles) * 8 + 64
    for h in range(Hq):
        x, y, z = q[:, h].double(), k[:, h // (Hq // Hkv)].double(), v[:, h // (Hq // Hkv)].double()
        s = scale * (x @ y.T) + times.log()
        A = abs(scale) * (x.abs() @ y.abs().T).amax(1)
        lse[:, h] = s.logsumexp(1) if sink is None else torch.logaddexp(s.logsumexp(1), sink[h].double())
        w = (s - lse[:, h, None]).exp()
        out[:, h] = w @ z
        ds = (D + 8) * 2.0 ** -23 * A
        wr = 2.0 ** -8 if scale else 0.0  # (equal weights are powers of two)
        tol[:, h] = (w @ z.abs()) * (2 * (ds + 2.0 ** -21) + wr + adds * 2.0 ** -23)[:, None]
        tol_l[:, h] = ds + 2.0 ** -21 + (adds / 4) * 2.0 ** -24 + 2.0 ** -22 * lse[:, h].abs()
    return out, lse, tol + 2.0 ** -8 * out.abs(), tol_l


def long_call(kvd, new, lens, Hq, Hkv, D, U=1024, P=256, seed=70, zero=False, **kw):
    """Sequences of lens[b] keys out of the same U / P pages."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF)  # noqa: E731
    q, kp, vp = rnd(sum(new), Hq, D), rnd(U // P, Hkv, P, D), rnd(U // P, Hkv, P, D) * 0.5 + 1
    scale = 0.0 if zero else 1 / math.sqrt(D)
    bt = (torch.arange(-(-max(lens) // P), device=DEV) % (U // P)).to(I32).repeat(len(lens), 1)
    out, lse = torch.full_like(q, 77.0), torch.full((sum(new), Hq), 55.0, device=DEV)
    err = torch.zeros(1, dtype=I32, device=DEV)
    kvd.attn_prefill_gqa_paged(q, kp, vp, bt, torch.tensor(lens, dtype=I32, device=DEV), cu(new), scale=scale,
                               out=out, lse_out=lse, err=err, **kw)
    assert int(err.item()) == 0
    k, v = (x.transpose(1, 2).reshape(U, Hkv, D) for x in (kp, vp))
    at = 0
    for b, n in enumerate(new):
        if n == 0 or (b > 3 and b < len(new) - 3 and b % 16):  # (a sample of many alike)
            at += n
            continue
        r = repeated(q[at:at + n], k, v, lens[b], scale, kw.get("window", 0), kw.get("n_sink_tokens", 0),
                     kw.get("sink_logit"))
        R.compare(out[at:at + n], lse[at:at + n], *r, what=f"sequence {b}")
        at += n


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("zero", [False, True])
def test_bfloat16_sums_do_not_drift(kvd, D, zero):
    # one token of 152 heads: as many units as CTAs, of 4 million keys each (before: lse 7e-4 off, equal
    # weights' means 1.2e-2)
    long_call(kvd, [1], [2 ** 22], 152, 152, D, zero=zero)


@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 64), (4, 1, 128), (7, 1, 64)])
@pytest.mark.parametrize("learned", [False, True])
def test_long_pieces_go_in_parts(kvd, Hq, Hkv, D, learned):
    # units of one and of two query tiles, whole and cut, of one part and of several
    sink = torch.randn(Hq, device=DEV) * 2 + 9 if learned else None
    long_call(kvd, [3, 0, 300, 1, 70], [65536, 65537, 200001, 131072, 66000], Hq, Hkv, D, sink_logit=sink)
    long_call(kvd, [1, 5] * 100, [65536 + 77 * i for i in range(200)], Hq, Hkv, D, sink_logit=sink)
    long_call(kvd, [300] * 40 + [40] * 50, [140000 - 50 * i for i in range(90)], Hq, Hkv, D, sink_logit=sink)
    long_call(kvd, [200, 1] * 60, [150000] * 120, Hq, Hkv, D, window=100000, n_sink_tokens=300, sink_logit=sink)


@pytest.mark.parametrize("Hq,new", [(4, 1), (4, 40), (1, 200)])
def test_values_that_are_not_finite_in_parts(kvd, Hq, new):
    # 160 units of several parts; the odd values lie in the last page of each sequence, which is seen by some rows
    g = torch.Generator(device=DEV).manual_seed(75)
    D, P, n, B = 64, 64, 1100, 160
    kp, vp = (torch.randn(6, 1, P, D, generator=g, device=DEV).to(BF) for _ in range(2))
    q = torch.randn(B * new, Hq, D, generator=g, device=DEV).to(BF)
    bt = (torch.arange(n, device=DEV) % 5).to(I32).repeat(B, 1)
    bt[:, -1] = 5
    lens = torch.tensor([n * P - b % P for b in range(B)], dtype=I32, device=DEV)
    err = torch.zeros(1, dtype=I32, device=DEV)

    def call():
        return kvd.attn_prefill_gqa_paged(q, kp, vp, bt, lens, cu([new] * B), err=err)

    want = call()
    for slot, col, x in ((0, 5, math.inf), (30, 63, -math.inf), (40, 0, NAN)):
        vp[5, 0, slot, col] = x
        pos = (lens[:, None] - new + torch.arange(new, device=DEV)[None]).flatten()
        want[pos >= (n - 1) * P + slot, :, col] = x
    got = call()
    assert int(err.item()) == 0
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(7.0, 8.0, 9.0), want.nan_to_num(7.0, 8.0, 9.0))


@pytest.mark.parametrize("new,lens", [([40, 1, 3], [40, 900, 70]), ([700, 5], [700, 5000]), ([3], [9000])])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("role", [1, 2, 3, 4, 5, 6])
def test_a_wait_that_runs_out_is_recorded(kvd, role, dtype, new, lens):
    """One role's warps first wait for what does not come: all roles give up, within their limits, copies and
    products that are under way are waited for, the call says so, and the next one is right again, with the
    same workspace. (float32 has no sixth role.)"""
    c = Case(new, lens, 8, 2, 128, dtype, seed=80)
    args = (c.q, *c.pools(64), cu(c.new))
    ws = torch.full((kvd.kvd_workspace_size("prefill", len(new), 8, 2, 128),), 255, dtype=torch.uint8, device=DEV)
    out, err = torch.empty_like(c.q), torch.zeros(1, dtype=I32, device=DEV)

    def call():
        kvd.attn_prefill_gqa_paged(*args, out=out, workspace=ws, err=err, **c.more())

    kvd.kvd_set_option("wait_timeout_test", role)
    try:
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        call()
        b.record()
        b.synchronize()
        time = a.elapsed_time(b)
    finally:
        kvd.kvd_set_option("wait_timeout_test", 0)
    assert int(err.item()) == (0 if dtype == F32 and role == 6 else -4)
    assert time < 100  # ms; the limit of a wait is about 2
    for _ in range(2):
        c.check(*c.call(kvd.attn_prefill_gqa_paged, args, workspace=ws))
    # a packed call takes the option too
    kvd.kvd_set_option("wait_timeout_test", role)
    try:
        err.zero_()
        kvd.attn_prefill_gqa(c.q, torch.cat(c.k), torch.cat(c.v), cu(c.new), cu(c.lens), workspace=ws, err=err)
        assert int(err.item()) == (0 if dtype == F32 and role == 6 else -4)
    finally:
        kvd.kvd_set_option("wait_timeout_test", 0)
    c.check(*c.packed(kvd, workspace=ws))


@pytest.mark.parametrize("new", [1, 3, 300])
def test_the_longest_window_sinks_and_table(kvd, new):
    # a unit's length in the work list is above 2^31 (held in an int, the call would have written nothing)
    long_call(kvd, [new], [2 ** 30 - 256], 1, 1, 64, window=2 ** 30, n_sink_tokens=2 ** 30)
    long_call(kvd, [new], [2 ** 30 - 256], 1, 1, 64, window=2 ** 31 - 1, n_sink_tokens=2 ** 31 - 1)


@pytest.mark.parametrize("P", [16, 64, 128, 256])
@pytest.mark.parametrize("window,n_sink", [(1, 0), (100, 4), (300, 0), (700, 33), (130, 260)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_pages_behind_the_window_may_be_gone(kvd, dtype, window, n_sink, P):
    for Hq, Hkv, D in ((8, 2, 64), (2, 2, 128)):
        new, lens = [1, 300, 40, 9], [1500, 1700, 900, 2311]
        c = Case(new, lens, Hq, Hkv, D, dtype, window=window, n_sink=n_sink, seed=90)
        kp, vp, bt, sl = c.pools(P)
        for b, (n, L) in enumerate(zip(new, lens)):
            seen = set(range(max(0, L - n - window + 1) // P, (L - 1) // P + 1)) | set(range(-(-min(n_sink, L) // P)))
            gone = [i for i in range(bt.shape[1]) if i not in seen]
            bt[b, torch.tensor(gone, device=DEV)] = -1
        assert (bt[1] < 0).any()
        c.check(*c.call(kvd.attn_prefill_gqa_paged, (c.q, kp, vp, bt, sl, cu(new))))


def test_where_float32_values_begin_to_count_as_infinite(kvd):
    # the neighbours of the first number that rounds to a bfloat16 infinity, as the only value of their column
    # that is not small
    below, first = (torch.tensor(x, dtype=I32).view(F32).item() for x in (0x7f7f7fff, 0x7f7f8000))
    for sign in (1, -1):
        c = Case([70, 5], [70, 300], 4, 2, 64, F32, seed=91)
        c.v[0][40, 0, 3], c.v[0][40, 1, 4] = sign * below, sign * first
        c.v[1][296, 0, 7], c.v[1][296, 1, 8] = sign * below, sign * first
        ref = Case([70, 5], [70, 300], 4, 2, 64, F32, seed=91)
        for r, x in zip(ref.v, c.v):
            r.copy_(x)
        ref.v[0][40, 1, 4] = ref.v[1][296, 1, 8] = sign * math.inf
        for out, lse in (c.packed(kvd), c.paged(kvd, 16)):
            ref.check(out, lse)


@pytest.mark.parametrize("exponent", [-100, -110, -118, -123])
def test_small_float32_values(kvd, exponent):
    # operands keep the bits down to 2^-133: half of the last, and as much for what is added up
    c = Case([70, 5], [70, 300], 4, 2, 64, F32, seed=92)
    for v in c.v:
        v *= 2.0 ** exponent
    out, lse = c.packed(kvd)
    at = 0
    for b, n in enumerate(c.new):
        ref, rl, tol, tol_l = R.attention(c.q[at:at + n], c.k[b], c.v[b], c.scale, dtype=F32)
        assert ((out[at:at + n].double() - ref).abs() <= tol + 2.0 ** -133).all()
        at += n


@pytest.mark.parametrize("learned", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_empty_sequences_of_one_token_each(kvd, dtype, learned):
    # without offsets a length of 0 is no error, as for the 4-bit decode
    lens = [0, 5, 0, 300, 64, 0]
    c = Case([1] * 6, lens, 8, 2, 64, dtype, learned=learned, seed=93)
    kp, vp, bt, sl = c.pools(16)
    c.check(*c.call(kvd.attn_prefill_gqa_paged, (c.q, kp, vp, bt, sl)))
    err = torch.zeros(1, dtype=I32, device=DEV)
    sl[2] = -1
    kvd.attn_prefill_gqa_paged(c.q, kp, vp, bt, sl, err=err)
    assert int(err.item()) == -6
