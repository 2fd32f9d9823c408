"""Plain float64 implementations of the prefill attention and of the cache reads, for the tests, with
the bound that each output of a float32-accumulating kernel has to keep.

Bounds, for a row with visible keys t, weights w_t = exp(s_t - lse) and m keys:
  scores   s = scale q.k. Products of inputs are exact or rounded once (2^-24), D of them are added in
           float32, each addition off by at most one unit of its result (2^-23; a tensor core cuts where
           a scalar rounds), then one multiplication by scale (and log2 e) and one subtraction of a
           maximum of the row, |maximum| <= A, each rounded:
               ds = (D + 8) 2^-23 A,  A = max over t of scale sum_d |q_d k_td|
  weights  the exponential is off by 2^-21 relative at most (its argument's rounding is in ds); an error
           ds of a score is one of ds of its weight. In bfloat16 kernels a weight is rounded to bfloat16
           before it multiplies a value: 2^-8 (half a step).
  sums     at most m additions and as many rescalings, each off by 2^-23 of what has been added up.
  out      V = sum_t w_t |v_t|:  |out - ref| <= V (2 (ds + 2^-21) + wr + (2 m + 64) 2^-23) + half |ref|
           where wr is 2^-8 or, float32, 2^-22 (products of split operands), and half is half a step of
           the output's type
  lse      |lse - ref| <= ds + 2^-21 + (m + 64) 2^-23 + 2^-22 |ref|
Not a proof for m of many thousands at the level of single units, where it is generous.
"""
import math

import torch

from tests import q4_reference as Q

F64 = torch.float64


def attention(q, k, v, scale, window=0, n_sink=0, sink=None, dtype=torch.bfloat16):
    """One sequence: q [n, Hq, D], k, v [L, Hkv, D] (any type) -> out, lse, bounds of both, float64."""
    n, Hq, D = q.shape
    L, Hkv = k.shape[0], k.shape[1]
    dev = q.device
    out = torch.zeros(n, Hq, D, dtype=F64, device=dev)
    lse = torch.full((n, Hq), -math.inf, dtype=F64, device=dev)
    tol, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    t = torch.arange(L, device=dev)[None, :]
    pos = (L - n + torch.arange(n, device=dev))[:, None]
    seen = t <= pos
    if window:
        seen = seen & ((t > pos - window) | (t < n_sink))
    some = seen.any(1) if L else torch.zeros(n, dtype=torch.bool, device=dev)
    m = seen.sum(1).to(F64)
    wr = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -22
    for h in range(Hq):
        g = h // (Hq // Hkv)
        x, y, z = q[:, h].to(F64), k[:, g].to(F64), v[:, g].to(F64)
        s = (x @ y.T) * scale
        big = abs(scale) * (x.abs() @ y.abs().T)
        s = torch.where(seen, s, -math.inf)
        A = torch.where(seen, big, 0.0).amax(1) if L else torch.zeros(n, dtype=F64, device=dev)
        top = s.amax(1) if L else torch.full((n,), -math.inf, dtype=F64, device=dev)
        if sink is not None:
            top = torch.maximum(top, sink[h].to(F64))
        safe = torch.where(torch.isinf(top), 0.0, top)
        w = torch.exp(s - safe[:, None])
        total = w.sum(1)
        if sink is not None:
            total = total + torch.exp(sink[h].to(F64) - safe)
        lse[:, h] = safe + total.log()
        w = w / torch.where(total > 0, total, 1.0)[:, None]
        # a value that a row does not see is not used at all
        bad = ~torch.isfinite(z)
        o = w @ torch.where(bad, 0.0, z)
        V = w @ torch.where(bad, 0.0, z).abs()
        if bad.any():
            for i in torch.nonzero(bad.any(1)).flatten().tolist():
                o = o + torch.where(seen[:, i: i + 1] & bad[i][None], z[i][None], 0.0)
        out[:, h] = o
        ds = (D + 8) * 2.0 ** -23 * A
        tol[:, h] = V * (2 * (ds + 2.0 ** -21) + wr + (2 * m + 64) * 2.0 ** -23)[:, None]
        tol_l[:, h] = ds + 2.0 ** -21 + (m + 64) * 2.0 ** -23 + 2.0 ** -22 * lse[:, h].abs()
        if sink is None:
            assert torch.equal(torch.isneginf(lse[:, h]), ~some)
    half = torch.finfo(dtype).eps / 2
    return out, lse, tol + half * out.abs(), tol_l


def compare(got, lse, ref, ref_lse, tol, tol_l, what=""):
    """Non-finite reference values have to be met as they are, the others within their bounds."""
    got, lse = got.to(F64), lse.to(F64)
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN in other places"
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), f"{what}: infinities"
    d = torch.where(fin, (got - ref).abs(), 0.0)
    over = d > torch.where(fin, tol, 0.0) + 1e-30
    assert not over.any(), \
        f"{what}: out {float((d / (tol + 1e-30)).max()):.3g} of its bound, {int(over.sum())} values"
    fin = torch.isfinite(ref_lse)
    assert torch.equal(lse[~fin], ref_lse[~fin]), f"{what}: lse of rows that see nothing"
    d = torch.where(fin, (lse - ref_lse).abs(), 0.0)
    assert (d <= torch.where(fin, tol_l, 0.0)).all(), \
        f"{what}: lse {float((d / (tol_l + 1e-30)).max()):.3g} of its bound"


def held_positions(L, window, n_sink):
    """Positions that a cache holds of L tokens, in order."""
    if window == 0:
        return list(range(L))
    return [t for t in range(min(L, n_sink))] + list(range(max(n_sink, L - window), L))


def slot_of(t, window, n_sink):
    return t if window == 0 or t < n_sink else n_sink + (t - n_sink) % window


def read(pool, bt, lens, P, window=0, n_sink=0):
    """pool [pages, Hkv, P, D] -> each sequence's held rows [n, Hkv, D]."""
    rows = []
    for b, L in enumerate(lens):
        at = [slot_of(t, window, n_sink) for t in held_positions(L, window, n_sink)]
        rows.append(torch.stack([pool[int(bt[b, s // P]), :, s % P] for s in at]) if at
                    else pool.new_zeros(0, pool.shape[1], pool.shape[3]))
    return rows


def q4_values(pool, D, is_k):
    """The float32 values [pages, Hkv, P, D] of a 4-bit pool (numpy bytes)."""
    return torch.from_numpy(Q.value(*Q.unpack(pool, D, is_k)))
