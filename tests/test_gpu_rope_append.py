"""GPU: new tokens rotated into a paged or rolling cache, in their own type or in 4 bits, against the
plain implementation in tests/q4_reference.py. The rotation's float32 steps are part of its
definition, so results are equal bit for bit (after one rounding to bf16); that the reference's
rotation is the formula's is checked against float64 (test_rotation_is_the_formulas)."""
import numpy as np
import pytest
import torch

from tests import q4_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


@pytest.fixture(scope="module")
def kvd():
    import kv_cache_decode_split_gb300 as m
    return m


class Case:
    """Inputs of one append, and what has to come of it."""

    def __init__(self, new, old, Hq, Hkv, D, P, dtype, rot, inter=False, window=0, n_sink=0, pad=0,
                 strided=True, seed=0, q4=False, cu=True):
        g = torch.Generator().manual_seed(seed)
        self.new, self.lens = list(new), [n + o for n, o in zip(new, old)]
        self.cu = [0] + np.cumsum(self.new).tolist()
        self.T = self.cu[-1] + pad
        self.Hq, self.Hkv, self.D, self.P, self.dtype = Hq, Hkv, D, P, dtype
        self.inter, self.window, self.n_sink, self.q4, self.use_cu = inter, window, n_sink, q4, cu
        cap = window + n_sink
        self.bt, self.pages = R.make_table([cap] * len(new) if window else self.lens, P, g)
        self.table = R.table(max(self.lens) + 1, rot)
        qkv = torch.randn(self.T, Hq + 2 * Hkv, D, generator=g).to(dtype)
        self.q, self.k, self.v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        if not strided:
            self.q, self.k, self.v = (x.contiguous() for x in (self.q, self.k, self.v))
        if q4:
            self.kp = torch.from_numpy(R.make_pool(self.pages, Hkv, P, D, True, seed + 1))
            self.vp = torch.from_numpy(R.make_pool(self.pages, Hkv, P, D, False, seed + 2))
        else:
            self.kp = torch.randn(self.pages, Hkv, P, D, generator=g).to(dtype)
            self.vp = torch.randn(self.pages, Hkv, P, D, generator=g).to(dtype)

    def gpu(self):
        base = self.q._base if self.q._base is not None else None
        if base is not None:
            d = base.to(DEV)
            q, k, v = d.split([self.Hq, self.Hkv, self.Hkv], 1)
        else:
            q, k, v = (x.to(DEV) for x in (self.q, self.k, self.v))
        cu = torch.tensor(self.cu, dtype=I32, device=DEV) if self.use_cu else None
        return dict(q=q, k_new=k, v_new=v, cos_sin=self.table.to(DEV), k_pool=self.kp.to(DEV),
                    v_pool=self.vp.to(DEV), block_table=self.bt.to(DEV),
                    seq_lens=torch.tensor(self.lens, dtype=I32, device=DEV), cu_seqlens=cu,
                    window=self.window, n_sink=self.n_sink, interleaved=self.inter)

    def want(self):
        """(q_out of the used rows, k and v of them in float32, k_pool, v_pool)."""
        n = self.cu[-1]
        pos = np.array([L - m + i for m, L in zip(self.new, self.lens) for i in range(m)], int)
        tab = self.table.numpy()
        qr = R.rotate(self.q[:n].float().numpy(), pos, tab, self.inter)
        kr = R.rotate(self.k[:n].float().numpy(), pos, tab, self.inter)
        vr = self.v[:n].float().numpy()
        kp, vp = self.kp.clone(), self.vp.clone()
        if self.q4:
            codes = [[a.copy() for a in R.unpack(x.numpy(), self.D, is_k)]
                     for x, is_k in ((kp, True), (vp, False))]
            rows = [R.quantise(kr), R.quantise(vr)]
        i = 0
        for b, m in enumerate(self.new):
            for t in range(self.lens[b] - m, self.lens[b]):  # in order: the last writer stays
                r = R.slot_of(t, self.window, self.n_sink)
                pg, at = int(self.bt[b, r // self.P]), r % self.P
                if self.q4:
                    for held, row in zip(codes, rows):
                        for a, x in zip(held, row):
                            a[pg, :, at] = x[i]
                else:
                    kp[pg, :, at] = torch.from_numpy(kr[i]).to(self.dtype)
                    vp[pg, :, at] = self.v[i]
                i += 1
        q = torch.from_numpy(qr).to(self.dtype)
        if self.q4:
            kp, vp = (torch.from_numpy(R.pack(*held, is_k)) for held, is_k in
                      zip(codes, (True, False)))
            kr, vr = R.value(*rows[0]), R.value(*rows[1])
        return q, torch.from_numpy(kr).to(self.dtype), torch.from_numpy(vr).to(self.dtype), kp, vp


def same(a, b):
    """Equal bit for bit, NaN with NaN."""
    a, b = a.cpu(), b.cpu()
    return a.shape == b.shape and torch.equal(torch.nan_to_num(a.float(), 7e7), torch.nan_to_num(b.float(), 7e7))


def run(kvd, c, **kw):
    a = c.gpu()
    a.update(kw)
    err = torch.zeros(1, dtype=I32, device=DEV)
    out = dict(q_out=torch.full((c.T, c.Hq, c.D), 77.0, dtype=c.dtype, device=DEV))
    if c.q4:
        out["k_out"] = torch.full((c.T, c.Hkv, c.D), 77.0, dtype=c.dtype, device=DEV)
        out["v_out"] = torch.full((c.T, c.Hkv, c.D), 77.0, dtype=c.dtype, device=DEV)
        kvd.rope_append_q4(**a, **out, err=err)
    else:
        kvd.rope_append(**a, **out, err=err)
    torch.cuda.synchronize()
    return out, a["k_pool"], a["v_pool"], int(err.item())


def same_pool(a, b, D, is_k):
    """Equal 4-bit pools: codes, scales and minima, but for groups that read back as NaN (b is
    NaN), whose other bits the definition leaves open."""
    a, b = (R.unpack(x.cpu().numpy(), D, is_k) for x in (a, b))
    nan = np.isnan(b[2])
    wide = np.repeat(nan, 64, -1)
    return (np.array_equal(np.isnan(a[2]), nan) and np.array_equal(a[0][~wide], b[0][~wide]) and
            np.array_equal(a[1][~nan], b[1][~nan]) and np.array_equal(a[2][~nan], b[2][~nan]))


def check(kvd, c):
    q, k, v, kp, vp = c.want()
    out, gk, gv, err = run(kvd, c)
    n = c.cu[-1]
    assert err == 0
    assert same(out["q_out"][:n], q)
    # the other rows of the pools are as they were
    if c.q4:
        assert same_pool(gk, kp, c.D, True) and same_pool(gv, vp, c.D, False)
    else:
        assert torch.equal(gk.cpu(), kp) and torch.equal(gv.cpu(), vp)
    if c.q4:
        assert same(out["k_out"][:n], k) and same(out["v_out"][:n], v)
    for x in out.values():
        assert (x[n:] == 77.0).all()  # rows behind the last sequence


def test_rotation_is_the_formulas():
    # float64 formula: two products of at most |x| |c| each rounded, and their difference:
    # three half steps of 2^-24 of |x| + |x'|
    rng = np.random.default_rng(1)
    x, pos, tab = rng.standard_normal((50, 3, 64)), np.arange(50) * 7, R.table(350, 48).numpy()
    for inter in (False, True):
        y = R.rotate(x.astype(np.float32), pos, tab, inter)
        X = x.astype(np.float32).astype(np.float64)
        for i in range(24):
            a, b = (2 * i, 2 * i + 1) if inter else (i, i + 24)
            c, s = tab[pos, i, None].astype(np.float64), tab[pos, 24 + i, None].astype(np.float64)
            lim = 3 * 2.0 ** -24 * (np.abs(X[..., a]) + np.abs(X[..., b]))
            assert (np.abs(y[..., a] - (X[..., a] * c - X[..., b] * s)) <= lim).all()
            assert (np.abs(y[..., b] - (X[..., b] * c + X[..., a] * s)) <= lim).all()
        assert np.array_equal(y[..., 48:], x.astype(np.float32)[..., 48:])


SHAPES = [  # new, old, Hq, Hkv, D, P, dtype, rot, interleaved, pad
    ([1, 1, 1], [0, 63, 64], 8, 2, 128, 64, BF, 128, False, 0),
    ([5, 0, 33, 1], [0, 7, 100, 15], 8, 8, 128, 16, BF, 64, False, 3),
    ([17, 2], [3, 250], 5, 1, 64, 256, BF, 64, True, 1),
    ([0, 0, 9, 0], [4, 1, 0, 2], 12, 4, 64, 32, F32, 48, False, 0),
    ([70, 1], [1, 1], 3, 3, 128, 32, F32, 112, True, 5),
    ([130], [1000], 6, 2, 64, 64, BF, 16, False, 0),
]


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("new,old,Hq,Hkv,D,P,dtype,rot,inter,pad", SHAPES)
def test_append(kvd, q4, new, old, Hq, Hkv, D, P, dtype, rot, inter, pad):
    check(kvd, Case(new, old, Hq, Hkv, D, P, dtype, rot, inter, pad=pad, q4=q4, seed=D + P))


@pytest.mark.parametrize("q4", [False, True])
def test_one_token_each_without_offsets(kvd, q4):
    check(kvd, Case([1] * 37, range(37), 8, 2, 64, 16, BF, 64, q4=q4, cu=False, strided=False))


@pytest.mark.parametrize("q4", [False, True])
def test_many_sequences(kvd, q4):
    # more offsets than one warp reads at once, most sequences without a token
    new = [(i * 7) % 3 if i % 5 == 0 else 0 for i in range(1500)]
    check(kvd, Case(new, [1] * 1500, 2, 1, 64, 16, BF, 64, q4=q4, seed=5))


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("window,n_sink", [(16, 0), (37, 4)])
def test_rolling(kvd, q4, window, n_sink):
    # a call whose later tokens replace its earlier ones, before, at and after the first wrap
    cap = window + n_sink
    c = Case([1, cap, cap + 1, 3 * cap + 2, 5], [0, 0, 0, 2, 9 * cap], 4, 2, 64, 16, BF, 64,
             window=window, n_sink=n_sink, q4=q4, seed=window)
    check(kvd, c)


@pytest.mark.parametrize("q4", [False, True])
def test_keys_and_values_only_and_in_place(kvd, q4):
    c = Case([4, 6], [0, 9], 8, 2, 128, 16, BF, 128, q4=q4, strided=False)
    q, _, _, kp, vp = c.want()
    f = kvd.rope_append_q4 if q4 else kvd.rope_append
    a = c.gpu()
    a["q"] = None
    assert f(**a) is None
    assert torch.equal(a["k_pool"].cpu(), kp) and torch.equal(a["v_pool"].cpu(), vp)
    a = c.gpu()
    assert f(**a, q_out=a["q"]) is a["q"]
    assert same(a["q"], q)


@pytest.mark.parametrize("q4", [False, True])
def test_nothing_to_append(kvd, q4):
    c = Case([0, 0], [5, 6], 4, 2, 64, 16, BF, 64, q4=q4)
    out, kp, vp, err = run(kvd, c)
    assert err == 0 and torch.equal(kp.cpu(), c.kp) and torch.equal(vp.cpu(), c.vp)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_q4_odd_values(kvd, dtype):
    # groups of one value, of zeros, tiny, beyond float16, with NaN or infinities
    c = Case([8], [3], 2, 2, 128, 16, dtype, 16, q4=True, strided=False)
    for x in (c.k, c.v):
        x[0] = 1.5
        x[1] = 0
        x[2] *= 1e-7
        x[3] *= 3e5
        x[4, 0, 70] = float("nan")
        x[5, 1, 3] = float("inf")
        x[6, :, 64:] = -float("inf")
        x[7, 0, 64:] = 1e-38
    check(kvd, c)


def test_append_refuses_and_flags(kvd):
    c = Case([2, 3], [10, 20], 4, 2, 64, 16, BF, 64, seed=3)
    q, _, _, kp, vp = c.want()
    out, gk, gv, err = run(kvd, c, block_table=torch.tensor([[c.pages, 0], [0, -1]], dtype=I32, device=DEV))
    assert err == -6 and same(out["q_out"], q)          # queries do not need the page
    assert torch.equal(gk.cpu(), c.kp) and torch.equal(gv.cpu(), c.vp)
    for lens in ([1, 23], [2 * 16 + 1, 23], [-5, 23]):   # shorter than its new tokens, past the table
        a_lens = torch.tensor(lens, dtype=I32, device=DEV)
        out, gk, gv, err = run(kvd, c, seq_lens=a_lens)
        assert err == -6 and (out["q_out"][:2] == 77.0).all() and same(out["q_out"][2:], q[2:])
    out, gk, gv, err = run(kvd, c, cos_sin=c.table[:21].contiguous().to(DEV))  # positions to 20
    assert err == -6 and same(out["q_out"][:3], q[:3]) and (out["q_out"][3:] == 77.0).all()
    # offsets that do not ascend stay inside every buffer
    _, _, _, err = run(kvd, c, cu_seqlens=torch.tensor([0, 9, 5], dtype=I32, device=DEV))
    assert err in (0, -6)
    a = c.gpu()
    for name, bad, what in (("k_new", a["k_new"].transpose(1, 2), ValueError),
                            ("k_new", a["k_new"][..., ::2], ValueError),
                            ("v_new", a["v_new"].float(), TypeError),
                            ("q", a["q"][:3], ValueError),
                            ("v_pool", a["v_pool"][:1], ValueError),
                            ("seq_lens", a["seq_lens"].long(), TypeError),
                            ("cu_seqlens", None, ValueError),
                            ("cos_sin", a["cos_sin"].half(), TypeError)):
        with pytest.raises(what):
            kvd.rope_append(**{**a, name: bad})
    with pytest.raises(kvd.KvdError):
        kvd.rope_append(**{**a, "cos_sin": a["cos_sin"][:, :24].contiguous()})


@pytest.mark.parametrize("q4", [False, True])
def test_captured_and_on_another_stream(kvd, q4):
    c = Case([3, 1], [5, 0], 4, 2, 64, 16, BF, 64, q4=q4)
    f = kvd.rope_append_q4 if q4 else kvd.rope_append
    q, _, _, kp, vp = c.want()
    a = c.gpu()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = f(**a, stream=s)
    s.synchronize()
    assert same(got, q) and torch.equal(a["k_pool"].cpu(), kp)
    a = c.gpu()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = f(**a)
    # new contents of the same tensors: every replay reads them
    a["k_pool"].copy_(c.kp.to(DEV))
    graph.replay()
    torch.cuda.synchronize()
    assert same(got, q) and torch.equal(a["k_pool"].cpu(), kp) and torch.equal(a["v_pool"].cpu(), vp)


FEW = [(1, 1, 128, BF), (15, 2, 128, BF), (2, 1, 64, BF), (3, 3, 64, BF), (4, 4, 64, BF), (6, 2, 64, F32), (4, 1, 128, F32)]


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,dtype", FEW)
def test_many_tokens_of_few_heads(kvd, q4, Hq, Hkv, D, dtype):
    # a warp has rows of several tokens: of one sequence, of neighbours, of none
    new, old = [1, 0, 701, 1, 1, 1, 333, 2, 0, 450, 5], [0, 3, 7, 90, 0, 31, 0, 5, 1, 64, 0]
    check(kvd, Case(new, old, Hq, Hkv, D, 32, dtype, 48, q4=q4, pad=7, inter=Hq == 2, seed=Hq))
    check(kvd, Case(new, old, Hq, Hkv, D, 16, dtype, 64, q4=q4, window=60, n_sink=4, seed=Hq))
    check(kvd, Case([1] * 1200, [i % 70 for i in range(1200)], Hq, Hkv, D, 16, dtype, 16, q4=q4, cu=False,
                    seed=Hq))


@pytest.mark.parametrize("q4", [False, True])
def test_bad_sequences_among_few_heads(kvd, q4):
    c = Case([3, 700, 2, 500, 1], [1, 5, 0, 9, 40], 2, 1, 128, 16, BF, 64, q4=q4, seed=8)
    q, k, _, _, _ = c.want()
    for b, lens in ((1, 699), (3, 508 + 1000), (2, -1)):
        bad = list(c.lens)
        bad[b] = lens
        out, _, _, err = run(kvd, c, seq_lens=torch.tensor(bad, dtype=I32, device=DEV))
        assert err == -6
        rows = torch.ones(c.T, dtype=torch.bool)
        rows[c.cu[b]:c.cu[b + 1]] = False
        assert same(out["q_out"][rows], q[rows]) and (out["q_out"][~rows] == 77.0).all()
        if q4:
            assert same(out["k_out"][rows], k[rows]) and (out["k_out"][~rows] == 77.0).all()
    # keys and values only
    a = c.gpu()
    a["q"] = None
    (kvd.rope_append_q4 if q4 else kvd.rope_append)(**a)
    assert torch.equal(a["k_pool"].cpu(), c.want()[3])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_q4_values_past_float16_on_one_side(kvd, dtype, D):
    # groups that lie next to the largest float16 (its steps are 32 there) and partly past it: the
    # definition clamps every value before it takes the minimum off
    c = Case([300, 41], [0, 3], 5, 3, D, 16, dtype, 16, q4=True, strided=False, seed=D)
    g = torch.Generator().manual_seed(D + 1)
    for x in (c.k, c.v):
        low = 64900 + 700 * torch.rand(*x.shape[:2], 1, generator=g)
        y = low + 400 * torch.rand(x.shape, generator=g)
        y[1::3] *= -1
        y[5, :, 1:], y[5, :, 0] = 65490.0, 70000.0
        y[6, :, 1:], y[6, :, 0] = 65072.0, 3e38
        x[2:] = y[2:].to(dtype)
    check(kvd, c)


# many tokens of more heads than the several-token form takes; heads that leave partial steps
LARGE = [(9, 3, 128, BF), (25, 5, 64, BF), (40, 8, 128, BF), (34, 17, 128, BF), (36, 35, 64, BF), (9, 3, 128, F32),
         (25, 5, 64, F32), (34, 17, 64, F32), (20, 20, 128, F32)]


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,dtype", LARGE)
def test_many_tokens_of_many_heads(kvd, q4, Hq, Hkv, D, dtype):
    cut = 3 if Hkv > 8 else 1
    new, old = [1, 0, 701 // cut, 1, 333 // cut, 2, 0, 450 // cut, 5], [0, 3, 7, 90, 31, 0, 5, 1, 64]
    check(kvd, Case(new, old, Hq, Hkv, D, 32, dtype, 48, q4=q4, pad=7, inter=Hq % 2 == 1, seed=Hq))
    check(kvd, Case(new, old, Hq, Hkv, D, 16, dtype, D, q4=q4, window=60, n_sink=4, seed=Hq))
    n = 1200 // cut
    check(kvd, Case([1] * n, [i % 70 for i in range(n)], Hq, Hkv, D, 16, dtype, 16, q4=q4, cu=False,
                    strided=False, seed=Hq))


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,dtype", [(9, 3, 128, BF), (25, 5, 64, F32)])
def test_bad_sequences_among_many_heads(kvd, q4, Hq, Hkv, D, dtype):
    c = Case([3, 700, 2, 500, 1], [1, 5, 0, 9, 40], Hq, Hkv, D, 16, dtype, 64, q4=q4, seed=8)
    q, k, _, _, _ = c.want()
    for b, lens in ((1, 699), (3, 508 + 1000), (2, -1)):
        bad = list(c.lens)
        bad[b] = lens
        out, _, _, err = run(kvd, c, seq_lens=torch.tensor(bad, dtype=I32, device=DEV))
        assert err == -6
        rows = torch.ones(c.T, dtype=torch.bool)
        rows[c.cu[b]:c.cu[b + 1]] = False
        assert same(out["q_out"][rows], q[rows]) and (out["q_out"][~rows] == 77.0).all()
        if q4:
            assert same(out["k_out"][rows], k[rows]) and (out["k_out"][~rows] == 77.0).all()
    # keys and values only
    a = c.gpu()
    a["q"] = None
    (kvd.rope_append_q4 if q4 else kvd.rope_append)(**a)
    assert torch.equal(a["k_pool"].cpu(), c.want()[3])


@pytest.mark.parametrize("q4", [False, True])
def test_offsets_past_32_bits(kvd, q4):
    # pages in the last of more than 4 GiB of each pool
    c = Case([3, 40], [5, 60], 4, 8, 128, 64, BF, 128, q4=q4, seed=3)
    _, _, _, kp, vp = c.want()
    a = c.gpu()
    pages = (5 << 30) // (a["k_pool"][0].numel() * a["k_pool"].element_size())
    first = pages - c.pages
    for n in ("k_pool", "v_pool"):
        big = torch.empty((pages,) + a[n].shape[1:], dtype=a[n].dtype, device=DEV)
        big[first:] = a[n]
        a[n] = big
    a["block_table"] = torch.where(a["block_table"] >= 0, a["block_table"] + first, -1).to(I32)
    (kvd.rope_append_q4 if q4 else kvd.rope_append)(**a)
    if q4:
        assert same_pool(a["k_pool"][first:], kp, 128, True) and same_pool(a["v_pool"][first:], vp, 128, False)
    else:
        assert torch.equal(a["k_pool"][first:].cpu(), kp) and torch.equal(a["v_pool"][first:].cpu(), vp)
