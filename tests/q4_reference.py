"""Plain implementations of the rotated append, the 4-bit rows and the attention over them, for the
tests: NumPy, written from the definitions. Rotation and codes step through float32 as defined (the
definition rounds each product and sum, so the codes are exact); attention is in float64."""
import numpy as np
import torch

F = np.float32


def rotate(x, pos, table, interleaved):
    """x [T, H, D] (any float), pos [T], table [positions, rot] -> float32 [T, H, D]."""
    x = np.asarray(x, F).copy()
    rot = table.shape[1]
    c, s = table[pos, None, : rot // 2].astype(F), table[pos, None, rot // 2:].astype(F)
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    u, v = x[..., a].copy(), x[..., b].copy()
    x[..., a] = u * c - v * s
    x[..., b] = v * c + u * s
    return x


def quantise(x):
    """x [..., D] float32 -> codes [..., D] uint8, scale and minimum [..., D / 64] float16."""
    with np.errstate(all="ignore"):
        g = np.asarray(x, F).reshape(*x.shape[:-1], -1, 64)
        bad = ~np.isfinite(g).all(-1)
        g = np.clip(g, F(-65504), F(65504))
        lo, hi = g.min(-1), g.max(-1)
        b, s = lo.astype(np.float16), ((hi - lo) * F(1 / 15)).astype(np.float16)
        inv = F(1) / s.astype(F)
        code = np.clip(np.rint((g - b.astype(F)[..., None]) * inv[..., None]), 0, 15)
        code = np.where(bad[..., None] | (s == 0)[..., None], 0, code).astype(np.uint8)
        b = np.where(bad, np.float16(np.nan), b)
    return code.reshape(x.shape), s, b


def value(code, s, b):
    """What codes stand for: float32."""
    g = code.reshape(*code.shape[:-1], -1, 64).astype(np.float64)
    v = g * s.astype(np.float64)[..., None] + b.astype(np.float64)[..., None]
    return v.reshape(code.shape).astype(F)


def _address(D, is_k):
    """For a 16-token block: the word and first bit of every (token, channel)."""
    r, c = np.meshgrid(np.arange(16), np.arange(D), indexing="ij")
    if is_k:
        w, t, n = c // 32, c // 8 % 4, c % 8
        return (r * 4 + t) * (D // 32) + w, (4 * n + 3) % 32
    f, t, o, w, j, g = r // 8, r // 2 % 4, r % 2, c // 64, c // 8 % 8, c % 8
    word = (((f * 8 + g) * 4 + t) * 2 + o) * 2 + w if D == 128 else ((g * 4 + t) * 2 + f) * 2 + o
    return word, 4 * j


def block_bytes(D):
    return 8 * D + D


def pack(code, s, b, is_k):
    """codes [..., P, D] and scales -> page bytes [..., page_bytes]."""
    *lead, P, D = code.shape
    word, bit = _address(D, is_k)
    c = code.reshape(-1, P // 16, 16, D).astype(np.uint64)
    out = np.zeros((c.shape[0], P // 16, block_bytes(D)), np.uint8)
    v = c << bit.astype(np.uint64)
    v = (v | (v >> np.uint64(32))) & np.uint64(0xFFFFFFFF)
    words = np.zeros((c.shape[0], P // 16, 2 * D), np.uint64)
    np.bitwise_or.at(words, (slice(None), slice(None), word.reshape(-1)),
                     v.reshape(c.shape[0], P // 16, -1))
    out[..., : 8 * D] = words.astype("<u4").view(np.uint8)
    par = np.stack([s, b], -1).reshape(c.shape[0], P // 16, -1).astype("<f2")
    out[..., 8 * D:] = par.view(np.uint8)
    return out.reshape(*lead, -1)


def unpack(pages, D, is_k):
    """page bytes [..., page_bytes] -> codes [..., P, D], scale, minimum [..., P, D / 64]."""
    lead = pages.shape[:-1]
    blk = np.ascontiguousarray(pages).reshape(-1, pages.shape[-1] // block_bytes(D), block_bytes(D))
    word, bit = _address(D, is_k)
    words = np.ascontiguousarray(blk[..., : 8 * D]).view("<u4").astype(np.uint64)
    w = words[..., word.reshape(-1)].reshape(*blk.shape[:2], 16, D)
    w = w | (w << np.uint64(32))  # the word as a ring
    code = ((w >> bit.astype(np.uint64)) & np.uint64(15)).astype(np.uint8)
    par = np.ascontiguousarray(blk[..., 8 * D:]).view("<f2").reshape(*blk.shape[:2], 16, D // 64, 2)
    P = blk.shape[1] * 16
    return (code.reshape(*lead, P, D), par[..., 0].reshape(*lead, P, -1),
            par[..., 1].reshape(*lead, P, -1))


def slot_of(t, window, n_sink):
    return t if window == 0 or t < n_sink else n_sink + (t - n_sink) % window


def visible(L, window, n_sink, ring):
    """Visible slots of a sequence of length L."""
    if window == 0:
        return np.arange(L)
    if ring:
        return np.arange(min(L, window + n_sink))
    t = np.arange(L)
    return t[(t >= L - window) | (t < n_sink)]


def attention(q, k_pool, v_pool, bt, lens, D, P, scale, window=0, n_sink=0, ring=False, sink=None,
              dtype=torch.bfloat16):
    """float64 (out, lse) and the error bound of each output, from packed pools (uint8 numpy).

    The bound counts, per weight: the score's float32 sums (each of the D products and of the
    scale and minimum terms, |q| (47 s + |b|) at most, rounded or cut by 2^-23 in each of about
    32 steps), 2^-21 for the exponential; the weight's rounding to float16 before it multiplies
    the codes (half a step, 2^-11, of p s code, code <= 15; with float32 queries two float16
    numbers, 2^-22, of codes held as c - 8 plus 8); and 2^-23 for each of the steps in which 16
    tokens are added to an output, each at most p (94 s + |b|) since codes are held with an
    offset of up to 79, plus the joining of partial sums."""
    weight = 2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -22
    q = np.asarray(q, np.float64)
    B, Hq, _ = q.shape
    Hkv = k_pool.shape[1]
    out, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    tol, tol_lse = np.zeros((B, Hq, D)), np.zeros((B, Hq))
    for b in range(B):
        t = visible(int(lens[b]), window, n_sink, ring)
        if len(t) == 0:
            if sink is not None:
                lse[b] = sink
                tol_lse[b] = 2.0 ** -20 * (1 + np.abs(sink))
            continue
        pages, at = bt[b, t // P], t % P
        used, inv = np.unique(pages, return_inverse=True)
        kc, ks, kb = (a[inv, :, at] for a in unpack(k_pool[used], D, True))
        vc, vs, vb = (a[inv, :, at] for a in unpack(v_pool[used], D, False))
        k = value(kc, ks, kb).astype(np.float64)  # [n, Hkv, D]
        v = value(vc, vs, vb).astype(np.float64)
        wide = 94 * vs.astype(np.float64) + np.abs(vb.astype(np.float64))
        kwide = 47 * ks.astype(np.float64) + np.abs(kb.astype(np.float64))
        for h in range(Hq):
            g = h // (Hq // Hkv)
            x = scale * (k[:, g] @ q[b, h])
            aq = np.abs(q[b, h]).reshape(-1, 64).sum(-1)
            ex = abs(scale) * (kwide[:, g] @ aq) * 32 * 2.0 ** -23 + np.abs(x) * 2.0 ** -22
            top = x.max() if sink is None else max(x.max(), sink[h])
            p = np.exp(x - top)
            den = p.sum() + (0 if sink is None else np.exp(sink[h] - top))
            out[b, h] = p @ v[:, g] / den
            lse[b, h] = top + np.log(den)
            rel = ex + 2.0 ** -21 + (len(t) / 16 + 64) * 2.0 ** -23
            e = (p * rel) @ wide[:, g] + (p * weight) @ (15 * vs[:, g].astype(np.float64))
            e = np.repeat(e, 64) / den
            drift = (p * (ex + 2.0 ** -21 + (len(t) / 8 + 64) * 2.0 ** -24)).sum() / den
            tol[b, h] = e + np.abs(out[b, h]) * drift
            tol_lse[b, h] = drift + np.abs(lse[b, h]) * 2.0 ** -22 + 2.0 ** -20
    return out, lse, tol, tol_lse


def table(positions, rot, base=10000.0):
    """Cosines and sines of every position, float32 [positions, rot]."""
    inv = base ** (-np.arange(rot // 2) / (rot // 2))
    a = np.arange(positions)[:, None] * inv[None]
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], 1).astype(F))


def make_table(lens, P, gen, spare=2, fill=-1):
    """Shuffled pages for the given numbers of slots: (block table, pages)."""
    need = [-(-int(n) // P) for n in lens]
    pages = sum(need) + spare
    perm = torch.randperm(pages, generator=gen).tolist()
    bt = torch.full((len(need), max(1, max(need))), fill, dtype=torch.int32)
    for b, n in enumerate(need):
        bt[b, :n] = torch.tensor(perm[:n], dtype=torch.int32)
        perm = perm[n:]
    return bt, pages


def make_pool(pages, H, P, D, is_k, seed, scale=1.0):
    """A packed pool of normals (keys with a mean for each channel): uint8 numpy."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((pages, H, P, D)).astype(F) * F(scale)
    if is_k:
        x += rng.standard_normal((H, 1, D)).astype(F)
    return pack(*quantise(x), is_k)
