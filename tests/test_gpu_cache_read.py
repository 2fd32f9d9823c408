"""GPU: reading a paged, rolling or 4-bit cache back as packed rows, against the definition; exact."""
import pytest
import torch

from tests import prefill_reference as R
from tests import q4_reference as Q

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def kvd():
    import kv_cache_decode_split_gb300 as m
    return m


def cu(n):
    return torch.tensor([0] + list(torch.tensor(list(n)).cumsum(0)), dtype=I32, device=DEV)


class Case:
    def __init__(self, lens, Hkv, D, P, dtype, q4, window=0, n_sink=0, seed=0, spare=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.Hkv, self.D, self.P, self.dtype, self.q4 = list(lens), Hkv, D, P, dtype, q4
        self.window, self.n_sink = window, n_sink
        cap = window + n_sink
        self.bt, self.pages = Q.make_table([cap if window else n for n in lens], P, g)
        if q4:
            raw = [Q.make_pool(self.pages, Hkv, P, D, i == 0, seed + i) for i in range(2)]
            self.pools = [torch.from_numpy(x).to(DEV) for x in raw]
            self.values = [R.q4_values(x, D, i == 0).to(dtype) for i, x in enumerate(raw)]
        else:
            self.values = [torch.randn(self.pages, Hkv, P, D, generator=g).to(dtype) for _ in range(2)]
            self.pools = [x.to(DEV) for x in self.values]
        self.held = [len(R.held_positions(n, window, n_sink)) for n in lens]
        self.rows = [n + spare for n in self.held]

    def outs(self, wide=False):
        T = sum(self.rows) + 3
        if not wide:
            return [torch.full((T, self.Hkv, self.D), 9.0, dtype=self.dtype, device=DEV) for _ in range(2)]
        buf = torch.full((T, 2 * self.Hkv + 1, self.D), 9.0, dtype=self.dtype, device=DEV)
        return [buf[:, :self.Hkv], buf[:, self.Hkv:2 * self.Hkv]]

    def run(self, kvd, outs, **kw):
        err = torch.zeros(1, dtype=I32, device=DEV)
        f = kvd.cache_read_q4 if self.q4 else kvd.cache_read
        a = dict(block_table=self.bt.to(DEV), seq_lens=torch.tensor(self.lens, dtype=I32, device=DEV),
                 cu_seqlens=cu(self.rows), window=self.window, n_sink=self.n_sink, err=err)
        a.update(kw)
        f(self.pools[0], self.pools[1], k_out=outs[0], v_out=outs[1], **a)
        torch.cuda.synchronize()
        return int(err.item())

    def check(self, outs, skip=()):
        for values, out in zip(self.values, outs):
            want = R.read(values, self.bt, self.lens, self.P, self.window, self.n_sink)
            at = 0
            for b, (w, n) in enumerate(zip(want, self.rows)):
                got = out[at:at + n].cpu()
                if b in skip:
                    assert (got == 9.0).all(), f"sequence {b} was written"
                else:
                    assert torch.equal(got[:len(w)], w), f"sequence {b}"
                    assert (got[len(w):] == 9.0).all(), f"rows behind sequence {b}"
                at += n
            assert (out[at:] == 9.0).all()


LENS = [1, 0, 15, 16, 17, 31, 33, 64, 100, 257, 500]


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("D,P", [(64, 16), (64, 64), (128, 16), (128, 32), (128, 256)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_lengths(kvd, dtype, D, P, q4):
    for Hkv, wide, spare in ((1, False, 0), (3, True, 2), (8, False, 5)):
        c = Case(LENS, Hkv, D, P, dtype, q4, seed=D + P, spare=spare)
        outs = c.outs(wide)
        assert c.run(kvd, outs) == 0
        c.check(outs)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("window,n_sink", [(1, 0), (16, 0), (17, 3), (100, 4), (40, 40), (5, 33)])
def test_rolling(kvd, window, n_sink, q4):
    cap = window + n_sink
    lens = [0, 1, n_sink, max(1, cap - 1), cap, cap + 1, 2 * cap + 35, 3 * window + n_sink, 2 ** 31 - 1]
    for D, dtype in ((64, F32), (128, BF)):
        c = Case(lens, 2, D, 16, dtype, q4, window, n_sink, seed=window)
        outs = c.outs()
        c2 = [n for n in lens]
        c.lens = [min(n, 10 ** 6 + (n - 10 ** 6) % window) if n > 10 ** 6 else n for n in c2]  # the same slots
        want = c.lens
        c.lens = c2
        assert c.run(kvd, outs) == 0
        c.lens = want
        c.check(outs)


@pytest.mark.parametrize("q4", [False, True])
def test_what_is_bad_is_recorded_and_not_written(kvd, q4):
    c = Case([40, 70, 9], 2, 64, 16, BF, q4, seed=3)
    bt = c.bt.to(DEV)
    for page in (-1, c.pages, 2 ** 30):
        table = bt.clone()
        table[0, 1] = page
        outs = c.outs()
        assert c.run(kvd, outs, block_table=table) == -6
        assert all((o[16:32] == 9.0).all() for o in outs)
        for o in outs:
            o[16:32] = 0
        for o, v in zip(outs, c.values):
            o[16:32] = R.read(v, c.bt, c.lens, 16)[0][16:32].to(DEV)
        c.check(outs)
    for length in (-1, 16 * bt.shape[1] + 1, 71, 2 ** 31 - 1):  # 71: more than its rows
        outs = c.outs()
        lens = torch.tensor([40, length, 9], dtype=I32, device=DEV)
        assert c.run(kvd, outs, seq_lens=lens, block_table=bt.clamp_min(0)) == -6
        c.check(outs, skip=(1,))
    outs = c.outs()
    assert c.run(kvd, outs, cu_seqlens=torch.tensor([0, 40, 110, 200], dtype=I32, device=DEV)) == -6
    c.check(outs, skip=(2,))
    outs = c.outs()
    assert c.run(kvd, outs, cu_seqlens=torch.tensor([0, 40, 30, 119], dtype=I32, device=DEV)) == -6


@pytest.mark.parametrize("q4", [False, True])
def test_many_sequences_streams_and_graphs(kvd, q4):
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 60, (1100,), generator=g).tolist()
    c = Case(lens, 2, 64, 16, BF, q4, seed=6)
    outs = c.outs()
    assert c.run(kvd, outs) == 0
    c.check(outs)
    outs = c.outs()
    assert c.run(kvd, outs, stream=torch.cuda.Stream()) == 0
    c.check(outs)
    outs = c.outs()
    a = (c.bt.to(DEV), torch.tensor(lens, dtype=I32, device=DEV), cu(c.rows))
    f = kvd.cache_read_q4 if q4 else kvd.cache_read
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f(*c.pools, *a, *outs)
    for o in outs:
        o.fill_(9.0)
    graph.replay()
    torch.cuda.synchronize()
    c.check(outs)


def test_the_values_that_an_append_handed_back(kvd):
    Hkv, D, P, n = 4, 128, 64, [100, 1, 333]
    g = torch.Generator(device=DEV).manual_seed(8)
    k, v = (torch.randn(sum(n), Hkv, D, generator=g, device=DEV).to(BF) for _ in range(2))
    k[5, 1, 3], v[7, 0, 70] = float("nan"), float("inf")  # their groups read back as NaN
    bt, pages = Q.make_table(n, P, torch.Generator().manual_seed(1))
    kp, vp = (kvd.q4_pool(pages, Hkv, P, D) for _ in range(2))
    ko, vo, kr, vr = (torch.empty_like(k) for _ in range(4))
    a = (bt.to(DEV), torch.tensor(n, dtype=I32, device=DEV), cu(n))
    kvd.rope_append_q4(None, k, v, Q.table(400, D).to(DEV), kp, vp, a[0], a[1], a[2], k_out=ko, v_out=vo)
    kvd.cache_read_q4(kp, vp, *a, kr, vr)
    for x, y in ((ko, kr), (vo, vr)):
        assert torch.equal(torch.isnan(x), torch.isnan(y))
        assert torch.equal(x.nan_to_num(5.0), y.nan_to_num(5.0))


@pytest.mark.parametrize("q4", [False, True])
def test_sequences_in_front_of_a_bad_offset_are_written(kvd, q4):
    lens = [40, 70, 9, 100, 33, 1, 16, 200]
    c = Case(lens, 2, 64, 16, BF, q4, seed=7)
    good = cu(c.rows)
    for at in range(2, len(lens) + 1):  # offset `at` ends sequence at - 1
        for bad in (-5, -2 ** 31, 0, 17, int(good[at - 1]) - 1, sum(lens) + 4, 2 ** 31 - 1):
            offsets = good.clone()
            offsets[at] = bad
            outs = c.outs()
            assert c.run(kvd, outs, cu_seqlens=offsets) == -6
            for values, out in zip(c.values, outs):
                want = R.read(values, c.bt, lens, 16)
                for b in range(at - 1):
                    assert torch.equal(out[int(good[b]):int(good[b + 1])].cpu(), want[b]), (at, bad, b)
                assert (out[sum(lens):] == 9.0).all()


@pytest.mark.parametrize("q4", [False, True])
def test_a_first_offset_other_than_0_is_bad(kvd, q4):
    c = Case([9, 30], 2, 64, 16, BF, q4, seed=8, spare=20)
    for first in (1, 5, 16):
        outs = c.outs()
        offsets = cu(c.rows)
        offsets[0] = first
        assert c.run(kvd, outs, cu_seqlens=offsets) == -6
        assert all((o[:29] == 9.0).all() for o in outs)
