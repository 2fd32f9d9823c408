"""Cases, plain forms and exact values of the operators around a rotated, paged and 4-bit KV cache:

  rope_append         new tokens' keys and values, rotated by position, into a paged or rolling cache
  rope_append_q4      the same into a cache held in 4 bits
  attn_decode_gqa_q4  single-token attention over the 4-bit cache

`own = False` computes an operator with elementary torch operations in float32; `own = True` calls the
library. The layout of the 4-bit pool (uint8 [num_pages, Hkv, page_bytes]) is, for D channels:
a page is page_size / 16 blocks of 16 tokens; a block is 16 * D / 2 bytes of codes, then 16 * D / 64
pairs (scale, minimum) in float16, [token][group of 64 channels][scale, minimum]. Codes are 32-bit words:
  K  word [token r][t < 4][w < D / 32]: code n < 8 is channel 32 w + 8 t + n, at bits 4 n + 3 (mod 32)
  V  token r = 8 f + 2 t + o, g < 8; word [f][g][t][o][w < 2] for D = 128 and [g][t][f][o] (w = 0) for
     D = 64: code j < 8 is channel 64 w + 8 j + g, at bits 4 j
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 32 sequences, Llama-3-8B heads: latency of a few hundred kilobytes
        dict(name="append decode bf16", op="append", dtype="bf16", B=32, Hq=32, Hkv=8, D=128, P=64, old_lo=4095,
             old_hi=8191, new_lo=1, new_hi=1, rot=128, inter=False, window=0, sink=0),
        # a ragged batch of prompts and prompt chunks, the same heads: bandwidth
        dict(name="append prompt bf16", op="append", dtype="bf16", B=9, Hq=32, Hkv=8, D=128, P=64, old_lo=0,
             old_hi=1001, new_lo=61, new_hi=3581, rot=128, inter=False, window=0, sink=0),
        # chunks into a rolling cache with sinks, part of the channels rotated in adjacent pairs, float32
        dict(name="append ring f32", op="append", dtype="f32", B=6, Hq=16, Hkv=4, D=64, P=16, old_lo=0,
             old_hi=777, new_lo=1, new_hi=700, rot=32, inter=True, window=512, sink=4),
        # one decode step into the 4-bit cache
        dict(name="append q4 decode bf16", op="append_q4", dtype="bf16", B=32, Hq=32, Hkv=8, D=128, P=64,
             old_lo=4095, old_hi=8191, new_lo=1, new_hi=1, rot=128, inter=False, window=0, sink=0),
        # prompts into the 4-bit cache, the stored values handed back for the prompt's own attention
        dict(name="append q4 prompt bf16", op="append_q4", dtype="bf16", B=9, Hq=32, Hkv=8, D=128, P=64, old_lo=0,
             old_hi=1001, new_lo=61, new_hi=3581, rot=128, inter=False, window=0, sink=0),
        # 64-wide heads, few tokens a sequence and sequences without any (speculative tokens), float32
        dict(name="append q4 few f32", op="append_q4", dtype="f32", B=64, Hq=16, Hkv=4, D=64, P=16, old_lo=1,
             old_hi=3001, new_lo=0, new_hi=9, rot=64, inter=False, window=0, sink=0),
        # one user, a short context: latency
        dict(name="attn q4 one short", op="attn_q4", dtype="bf16", B=1, Hq=32, Hkv=8, D=128, P=64, len_lo=513,
             len_hi=513, window=0, sink=0, ring=False, learned=False),
        # the ordinary batch: 32 sequences of 4096 to 8192 tokens, Llama-3-8B heads
        dict(name="attn q4 batch 32", op="attn_q4", dtype="bf16", B=32, Hq=32, Hkv=8, D=128, P=64, len_lo=4096,
             len_hi=8192, window=0, sink=0, ring=False, learned=False),
        # two very long sequences of an odd length, large pages: few rows, the long axis split
        dict(name="attn q4 long", op="attn_q4", dtype="bf16", B=2, Hq=32, Hkv=8, D=128, P=256, len_lo=131071,
             len_hi=131071, window=0, sink=0, ring=False, learned=False),
        # sliding window with sink tokens and a learned sink logit, 64-wide heads
        dict(name="attn q4 window", op="attn_q4", dtype="bf16", B=8, Hq=64, Hkv=8, D=64, P=64, len_lo=300,
             len_hi=32768, window=4096, sink=4, ring=False, learned=True),
        # many sequences, 16 query heads to a KV head, small pages
        dict(name="attn q4 group 16", op="attn_q4", dtype="bf16", B=96, Hq=32, Hkv=2, D=128, P=16, len_lo=97,
             len_hi=5003, window=0, sink=0, ring=False, learned=False),
        # float32 queries over a rolling cache
        dict(name="attn q4 ring f32", op="attn_q4", dtype="f32", B=5, Hq=16, Hkv=4, D=64, P=16, len_lo=9,
             len_hi=4000, window=1024, sink=4, ring=True, learned=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append_q4", "attn_q4"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 5, 8])
    G = rng.choice([1, 2, 3, 4, 7, 8] if op != "attn_q4" else [1, 2, 4, 5, 8, 8, 12, 16])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), Hq=Hkv * G, Hkv=Hkv, D=D, P=rng.choice([16, 32, 64, 128, 256]))
    if op == "attn_q4":
        # at most ~24000 visible tokens x 8 heads of 128 (the listed batch holds ~196000 x 8)
        c["B"] = _log(rng, 1, 48)
        c["len_hi"] = _log(rng, 17, 24000 // c["B"] * 4)
        c["len_lo"] = max(1, c["len_hi"] * rng.randint(1, 10) // 10)
        windowed = rng.random() < 0.4
        c["window"] = _log(rng, 15, 3000) if windowed else 0
        c["sink"] = rng.choice([0, 1, 4, 33]) if windowed else 0
        c["ring"] = windowed and rng.random() < 0.5
        c["learned"] = rng.random() < 0.3
        return c
    c["B"] = _log(rng, 1, 40)
    # at most what the listed prompts move
    most = 380e6 / ((2 * c["Hq"] + 4 * Hkv) * D * _SIZE[c["dtype"]])
    c["new_hi"] = _log(rng, 1, max(2, int(min(12000, most) / c["B"])))
    c["new_lo"] = min(c["new_hi"], rng.choice([0, 1, c["new_hi"]]))
    if c["new_hi"] * c["B"] < 8:  # at least a few tokens
        c["new_lo"] = c["new_hi"]
    c["old_lo"] = 0
    c["old_hi"] = _log(rng, 1, 4000)
    c["rot"] = rng.choice([D, D, D // 2, D - 16])
    c["inter"] = rng.random() < 0.3
    windowed = rng.random() < 0.25
    c["window"] = _log(rng, 16, 2000) if windowed else 0
    c["sink"] = rng.choice([0, 4]) if windowed else 0
    return c


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, the same ones for a case whatever the seed."""
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _lengths(case):
    """(new tokens, lengths after the call) of an append case; (0s, lengths) of an attention case."""
    B = case["B"]
    if case["op"] == "attn_q4":
        return [0] * B, _spread(case["len_lo"], case["len_hi"], B)
    new = _spread(case["new_lo"], case["new_hi"], B)
    old = _spread(case["old_lo"], case["old_hi"], B)[::-1]
    # a sequence in the cache has a token
    return new, [max(1, n + o) for n, o in zip(new, old)]


def _visible(case):
    _, lens = _lengths(case)
    if case["window"] == 0:
        return lens
    return [min(n, case["window"] + case["sink"]) for n in lens]


def _row_q4(D):
    return D // 2 + 4 * (D // 64)


def work(case):
    new, lens = _lengths(case)
    e, D, Hq, Hkv = _SIZE[case["dtype"]], case["D"], case["Hq"], case["Hkv"]
    if case["op"] == "attn_q4":
        vis = sum(_visible(case))
        return {"bytes": vis * Hkv * 2 * _row_q4(D) + 2 * case["B"] * Hq * D * e, "flops": 4 * vis * Hq * D}
    T = sum(new)
    table = 4 * case["rot"] * len({p for n, L in zip(new, lens) for p in range(L - n, L)})
    kept = sum(min(n, L if case["window"] == 0 else case["window"] + case["sink"]) for n, L in zip(new, lens))
    if case["op"] == "append":
        moved = T * (2 * Hq + 2 * Hkv) * D * e + kept * 2 * Hkv * D * e
    else:  # q read and written, k and v read and given back as values, the cache written
        moved = T * (2 * Hq + 4 * Hkv) * D * e + kept * 2 * Hkv * _row_q4(D)
    return {"bytes": moved + table, "flops": 3 * T * (Hq + Hkv) * case["rot"]}


# ------------------------------------------------------------------------------------ inputs
def _normal(gen, *shape, scale=1.0):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).mul_(scale)


def _table(lens, P, gen):
    """Shuffled pages of a pool with a few spare ones: (block table, pages)."""
    need = [-(-n // P) for n in lens]
    pages, most = sum(need) + 3, max(need)
    perm = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    start = torch.tensor(np.cumsum([0] + need[:-1]), device="cuda")
    at = start[:, None] + torch.arange(most, device="cuda")[None, :]
    held = torch.arange(most, device="cuda")[None, :] < torch.tensor(need, device="cuda")[:, None]
    return torch.where(held, perm[at.clamp_max(pages - 1)], -1).to(torch.int32).contiguous(), pages


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    rng = np.random.default_rng(int(seed))
    new, lens = _lengths(case)
    order = rng.permutation(case["B"])
    new, lens = [new[i] for i in order], [lens[i] for i in order]
    dt, D, Hq, Hkv, P = _DT[case["dtype"]], case["D"], case["Hq"], case["Hkv"], case["P"]
    cap = case["window"] + case["sink"]
    rolling = case["window"] > 0 and case.get("ring", True)
    slots = [cap] * case["B"] if rolling else lens
    bt, pages = _table(slots, P, gen)
    s = dict(case=case, bt=bt, sl=torch.tensor(lens, dtype=torch.int32, device="cuda"), pages=pages,
             err=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if case["op"] == "attn_q4":
        s["q"] = _normal(gen, case["B"], Hq, D).to(dt)
        # keys of uneven channels around a mean of their own, values around zero, as a model's
        s["k_pool"] = _filled_pool(gen, pages, Hkv, P, D, True)
        s["v_pool"] = _filled_pool(gen, pages, Hkv, P, D, False)
        s["sink_logit"] = _normal(gen, Hq) if case["learned"] else None
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(case["B"], Hq, device="cuda")
        if own:
            import kv_cache_decode_split_gb300 as kvd
            s["ws"] = torch.empty(kvd.kvd_workspace_size("gqa_q4", case["B"], Hq, Hkv, D, bt.shape[1] * P),
                                  dtype=torch.uint8, device="cuda")
        return s
    T = sum(new)
    # one projection's output holds q, k and v of a token side by side
    qkv = _normal(gen, T, (Hq + 2 * Hkv), D).to(dt)
    s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    s["cu"] = torch.tensor(np.cumsum([0] + new), dtype=torch.int32, device="cuda")
    half = case["rot"] // 2
    inv = 500000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    ang = torch.arange(max(lens), device="cuda", dtype=torch.float64)[:, None] * inv[None, :]
    s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
    s["q_out"] = torch.empty(T, Hq, D, dtype=dt, device="cuda")
    if case["op"] == "append":
        s["k_pool"] = _normal(gen, pages, Hkv, P, D).to(dt)
        s["v_pool"] = _normal(gen, pages, Hkv, P, D).to(dt)
    else:
        s["k_pool"] = torch.zeros(pages, Hkv, P * _row_q4(D), dtype=torch.uint8, device="cuda")
        s["v_pool"] = torch.zeros_like(s["k_pool"])
        s["k_out"] = torch.empty(T, Hkv, D, dtype=dt, device="cuda")
        s["v_out"] = torch.empty(T, Hkv, D, dtype=dt, device="cuda")
    if new == [1] * case["B"]:
        s["cu"] = None  # one token a sequence needs no offsets
    return s


def _filled_pool(gen, pages, Hkv, P, D, is_k):
    x = _normal(gen, pages, Hkv, P, D)
    if is_k:
        x.mul_(0.3 + 1.5 * torch.rand(Hkv, 1, D, generator=gen, device="cuda")).add_(_normal(gen, Hkv, 1, D))
    code, s, b = _quantise(x)
    return _pack(code, s, b, is_k)


# -------------------------------------------------------------------------- 4-bit rows, plain
def _quantise(x):
    """x [..., D] float32 -> codes [..., D] int32, scale and minimum [..., D / 64] float16."""
    g = x.unflatten(-1, (-1, 64))
    bad = ~torch.isfinite(g).all(-1, keepdim=True)
    g = g.clamp(-65504.0, 65504.0)
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    b, s = lo.half(), ((hi - lo) * (1.0 / 15.0)).half()
    inv = 1.0 / s.float()
    code = ((g - b.float()) * inv).round().clamp(0, 15)
    code = torch.where(bad | (s == 0), 0.0, code).to(torch.int32)
    b = torch.where(bad, float("nan"), b.float()).half()
    return code.flatten(-2), s.squeeze(-1), b.squeeze(-1)


def _value(code, s, b):
    """The values that codes [..., D] with scales and minima [..., D / 64] stand for, float32."""
    return (code.unflatten(-1, (-1, 64)).float() * s.float()[..., None] + b.float()[..., None]).flatten(-2)


def _pack(code, s, b, is_k):
    """codes [pages, Hkv, P, D] and scales -> the pool's bytes [pages, Hkv, page_bytes]."""
    n, h, P, D = code.shape
    c = code.view(n, h, P // 16, 16, D)
    at = torch.arange(8, device=code.device) * 4
    if is_k:
        c = c.view(n, h, P // 16, 16, D // 32, 4, 8).transpose(4, 5)  # [r][t][w][n]
        at = (at + 3) % 32
    else:
        c = c.view(n, h, P // 16, 2, 4, 2, D // 64, 8, 8)  # [f][t][o][w][j][g]
        c = c.permute(0, 1, 2, 3, 8, 4, 5, 6, 7) if D == 128 else c.permute(0, 1, 2, 8, 4, 3, 5, 6, 7)
    at = at.to(torch.int64)
    wide = c.to(torch.int64) << at
    word = (wide & 0xFFFFFFFF) | (wide >> 32)  # a code past bit 31 goes on at bit 0
    word = word.sum(-1)
    word = torch.where(word >= 2 ** 31, word - 2 ** 32, word).to(torch.int32).contiguous()
    codes = word.view(torch.uint8).reshape(n, h, P // 16, 16 * D // 2)
    par = torch.stack([s, b], -1).contiguous().view(torch.uint8).reshape(n, h, P // 16, 16 * 4 * (D // 64))
    return torch.cat([codes, par], -1).reshape(n, h, -1).contiguous()


def _unpack(blk, D, is_k):
    """Blocks [..., block_bytes] -> values [..., 16, D] float32."""
    cb = 16 * D // 2
    word = blk[..., :cb].contiguous().view(torch.int32)
    par = blk[..., cb:].contiguous().view(torch.float16).unflatten(-1, (16, D // 64, 2))
    lead, at = word.shape[:-1], torch.arange(8, device=blk.device, dtype=torch.int32) * 4
    if is_k:
        w = word.view(*lead, 16, 4, D // 32, 1)
        w = ((w >> 3) & 0x1FFFFFFF) | (w << 29)  # bits back in their natural places
        code = ((w >> at) & 15).transpose(-2, -3).reshape(*lead, 16, D)
    elif D == 128:
        code = ((word.view(*lead, 2, 8, 4, 2, 2, 1) >> at) & 15)  # [f][g][t][o][w][j]
        k = code.dim()
        code = code.permute(*range(k - 6), k - 6, k - 4, k - 3, k - 2, k - 1, k - 5).reshape(*lead, 16, D)
    else:
        code = ((word.view(*lead, 8, 4, 2, 2, 1) >> at) & 15)  # [g][t][f][o][j]
        k = code.dim()
        code = code.permute(*range(k - 5), k - 3, k - 4, k - 2, k - 1, k - 5).reshape(*lead, 16, D)
    return _value(code, par[..., 0], par[..., 1])


# ------------------------------------------------------------------------------- plain forms
def _positions(s):
    """Sequence and position of every new token."""
    T = s["q"].shape[0]
    if s["cu"] is None:
        seq = torch.arange(T, device="cuda")
        return seq, s["sl"].long() - 1
    i = torch.arange(T, device="cuda")
    seq = torch.searchsorted(s["cu"][1:].contiguous(), i, right=True)
    return seq, s["sl"].long()[seq] - s["cu"].long()[seq + 1] + i


def _rotate(x, cs, inter):
    R = cs.shape[-1]
    c, sn = cs[:, None, : R // 2], cs[:, None, R // 2:]
    x = x.float()
    if inter:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
    else:
        a, b = x[..., : R // 2], x[..., R // 2: R]
        y = torch.cat([a * c - b * sn, b * c + a * sn], -1)
    return torch.cat([y, x[..., R:]], -1)


def _plain_append(s):
    c = s["case"]
    dt = s["q"].dtype
    seq, pos = _positions(s)
    cs = s["cos_sin"][pos]
    q = _rotate(s["q"], cs, c["inter"]).to(dt)
    k, v = _rotate(s["k"], cs, c["inter"]), s["v"].float()
    if c["op"] == "append_q4":
        # the cache's bytes follow from codes and scales; the values they stand for are returned
        return {"q": q, "k": _value(*_quantise(k)).to(dt), "v": _value(*_quantise(v)).to(dt)}
    P, W, n_sink = c["P"], c["window"], c["sink"]
    kept, slot = torch.ones_like(pos, dtype=torch.bool), pos
    if W:
        kept = (pos < n_sink) | (pos >= s["sl"].long()[seq] - W)
        slot = torch.where(pos < n_sink, pos, n_sink + (pos - n_sink) % W)
    page = s["bt"].long()[seq, slot // P]
    at = (page[kept], slot[kept] % P)
    s["k_pool"].transpose(1, 2)[at] = k[kept].to(dt)
    s["v_pool"].transpose(1, 2)[at] = v[kept].to(dt)
    return {"q": q, "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _blocks_seen(s):
    """Logical blocks of 16 slots that hold every visible one: [n] or [B, n]."""
    c, most = s["case"], s["bt"].shape[1] * (s["case"]["P"] // 16)
    if c["window"] == 0 or c["ring"]:
        return torch.arange(most, device="cuda")[None, :].expand(c["B"], -1)
    n_sink = -(-c["sink"] // 16)
    first = ((s["sl"].long() - c["window"]).clamp_min(0) // 16).clamp_min(n_sink)
    window = first[:, None] + torch.arange(c["window"] // 16 + 2, device="cuda")
    return torch.cat([torch.arange(n_sink, device="cuda")[None, :].expand(c["B"], -1), window], 1)


def _plain_attn(s):
    c = s["case"]
    B, Hq, Hkv, D, P = c["B"], c["Hq"], c["Hkv"], c["D"], c["P"]
    per = P // 16
    blk = _blocks_seen(s)
    slot = (blk[..., None] * 16 + torch.arange(16, device="cuda")).flatten(1)
    L = s["sl"].long()[:, None]
    seen = slot < L
    if c["window"] and c["ring"]:
        seen = slot < L.clamp_max(c["window"] + c["sink"])
    elif c["window"]:
        seen = seen & ((slot >= L - c["window"]) | (slot < c["sink"]))
    page = torch.gather(s["bt"].long(), 1, (blk // per).clamp_max(s["bt"].shape[1] - 1)).clamp_min(0)
    rows = page * per + blk % per

    def values(pool, is_k):
        blocks = pool.view(-1, Hkv, per, pool.shape[2] // per).transpose(1, 2).flatten(0, 1)
        x = _unpack(blocks[rows], D, is_k)  # [B, blocks, Hkv, 16, D]
        return x.transpose(1, 2).flatten(2, 3)

    q = s["q"].float().view(B, Hkv, Hq // Hkv, D)
    x = torch.matmul(q, values(s["k_pool"], True).transpose(2, 3)) * (1.0 / math.sqrt(D))
    x = x.masked_fill(~seen[:, None, None, :], float("-inf"))
    top = x.amax(-1, keepdim=True)
    if s["sink_logit"] is not None:
        sink = s["sink_logit"].view(1, Hkv, -1, 1)
        top = torch.maximum(top, sink)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    if s["sink_logit"] is not None:
        total = total + torch.exp(sink - top)
    v = values(s["v_pool"], False).masked_fill(~seen[:, None, :, None], 0.0)
    out = torch.matmul(p, v) / total
    return {"out": out.reshape(B, Hq, D).to(s["q"].dtype), "lse": (top + total.log()).reshape(B, Hq)}


def run(state):
    c = state["case"]
    if not own:
        return _plain_attn(state) if c["op"] == "attn_q4" else _plain_append(state)
    import kv_cache_decode_split_gb300 as kvd
    s = state
    if c["op"] == "attn_q4":
        kvd.attn_decode_gqa_q4(s["q"], s["k_pool"], s["v_pool"], s["bt"], s["sl"], window=c["window"],
                               n_sink_tokens=c["sink"], ring=c["ring"], sink_logit=s["sink_logit"], out=s["out"],
                               lse_out=s["lse"], workspace=s["ws"], err=s["err"])
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "append":
        kvd.rope_append(s["q"], s["k"], s["v"], s["cos_sin"], s["k_pool"], s["v_pool"], s["bt"], s["sl"],
                        cu_seqlens=s["cu"], window=c["window"], n_sink=c["sink"], interleaved=c["inter"],
                        q_out=s["q_out"], err=s["err"])
        return {"q": s["q_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    kvd.rope_append_q4(s["q"], s["k"], s["v"], s["cos_sin"], s["k_pool"], s["v_pool"], s["bt"], s["sl"],
                       cu_seqlens=s["cu"], window=c["window"], n_sink=c["sink"], interleaved=c["inter"],
                       q_out=s["q_out"], k_out=s["k_out"], v_out=s["v_out"], err=s["err"])
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}


# ------------------------------------------------------------------------------------- exact
def _f32(x):
    """The float32 value next to x, as float64 (one rounding of the definition)."""
    return x.float().double()


def _exact_rotated(x, pos, cs, inter, step=lambda v: v):
    """x [T, H, D] rotated, channel by channel of the definition, float64; `step` rounds what it rounds."""
    R = cs.shape[1]
    x, y = x.double(), x.double().clone()
    for i in range(R // 2):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + R // 2)
        c, s = cs[pos, i].double()[:, None], cs[pos, R // 2 + i].double()[:, None]
        y[..., a] = step(step(x[..., a] * c) - step(x[..., b] * s))
        y[..., b] = step(step(x[..., a] * s) + step(x[..., b] * c))
    return y


def _exact_stored(x):
    """The 4-bit values of x [T, H, D], group by group. The definition's float32 roundings decide which code a
    value next to a border takes, so they are made here, each from the float64 result (one rounding each)."""
    y = torch.empty_like(x)
    for g in range(x.shape[2] // 64):
        part = x[..., 64 * g: 64 * g + 64].clamp(-65504.0, 65504.0)
        low = part.min(-1, keepdim=True).values
        base = low.half().double()
        wide = _f32(part.max(-1, keepdim=True).values - low)
        step = _f32(wide * _f32(torch.tensor(1.0 / 15.0, dtype=torch.float64))).half().double()
        code = _f32(_f32(part - base) * _f32(1.0 / step)).round().clamp(0, 15)
        y[..., 64 * g: 64 * g + 64] = base + torch.where(step > 0, code, torch.zeros_like(part)) * step
    return y


def _exact_cache(pool, pages, P, D, slots, is_k):
    """Values [Hkv, n, D] in float64 of the given slots of one sequence, each code found by its address."""
    size = 8 * D + 4 * (D // 4)
    page = pages[slots // P].long()
    r, base = slots % 16, (slots % P // 16) * size
    ch = torch.arange(D, device="cuda")[None, :]
    rr = r[:, None]
    if is_k:
        w, t, n = ch // 32, ch // 8 % 4, ch % 8
        word, bit = (rr * 4 + t) * (D // 32) + w, (4 * n + 3) % 32
    else:
        f, t, o, w, j, g = rr // 8, rr // 2 % 4, rr % 2, ch // 64, ch // 8 % 8, ch % 8
        word = (((f * 8 + g) * 4 + t) * 2 + o) * 2 + w if D == 128 else ((g * 4 + t) * 2 + f) * 2 + o
        bit = (4 * j).expand(slots.numel(), -1)
    bit = bit.expand(slots.numel(), -1)

    def byte(at):
        return torch.stack([pool[page[:, None], h, at].long() for h in range(pool.shape[1])])

    lo = base[:, None] + 4 * word
    first = byte(lo + bit // 8)
    second = byte(lo + (bit // 8 + 1) % 4)  # the rest of a code that a byte's end cuts
    code = (((second << 8) | first) >> (bit % 8)) & 15
    at = base[:, None] + 8 * D + (rr * (D // 64) + ch // 64) * 4

    def half(at):
        return ((byte(at + 1) << 8) | byte(at)).to(torch.int16).view(torch.float16).double()

    return half(at) * code.double() + half(at + 2)


def exact(case, seed):
    s = prepare(case, seed)
    dt = torch.float64
    if case["op"] != "attn_q4":
        new = [1] * case["B"] if s["cu"] is None else s["cu"].diff().tolist()
        lens = s["sl"].tolist()
        pos = torch.tensor([p for n, L in zip(new, lens) for p in range(L - n, L)], device="cuda", dtype=torch.long)
        q = _exact_rotated(s["q"], pos, s["cos_sin"], case["inter"])
        if case["op"] == "append_q4":
            k = _exact_rotated(s["k"], pos, s["cos_sin"], case["inter"], _f32)
            return {"q": q, "k": _exact_stored(k), "v": _exact_stored(s["v"].double())}
        k = _exact_rotated(s["k"], pos, s["cos_sin"], case["inter"])
        kp, vp, i = s["k_pool"].to(dt), s["v_pool"].to(dt), 0
        for b, (n, L) in enumerate(zip(new, lens)):
            t = torch.arange(L - n, L, device="cuda")
            row = i + torch.arange(n, device="cuda")
            i += n
            slot = t
            if case["window"]:  # the last writer of a slot wins
                W, ns = case["window"], case["sink"]
                last = (t < ns) | (t + W >= L)
                t, row = t[last], row[last]
                slot = torch.where(t < ns, t, ns + torch.remainder(t - ns, W))
            for h in range(case["Hkv"]):
                where = (s["bt"][b, slot // case["P"]].long(), torch.full_like(slot, h), slot % case["P"])
                kp[where], vp[where] = k[row, h], s["v"][row, h].to(dt)
        return {"q": q, "k_pool": kp, "v_pool": vp}
    outs, lses = [], []
    H, G, cap = case["Hkv"], case["Hq"] // case["Hkv"], case["window"] + case["sink"]
    for b, L in enumerate(s["sl"].tolist()):
        slots = torch.arange(L, device="cuda")
        if case["window"] and case["ring"]:
            slots = slots[: min(L, cap)]
        elif case["window"]:
            slots = slots[(slots >= L - case["window"]) | (slots < case["sink"])]
        parts = slots.split(16384)
        q = s["q"][b].to(dt).view(H, G, -1)
        keys = (_exact_cache(s["k_pool"], s["bt"][b], case["P"], case["D"], part, True) for part in parts)
        score = torch.cat([torch.bmm(q, k.transpose(1, 2)) for k in keys], 2) / math.sqrt(case["D"])
        top = score.max(2, keepdim=True).values
        sink = None if s["sink_logit"] is None else s["sink_logit"].to(dt).view(H, G, 1)
        if sink is not None:
            top = torch.maximum(top, sink)
        p = torch.exp(score - top)
        total = p.sum(2, keepdim=True) + (0 if sink is None else torch.exp(sink - top))
        out, done = 0, 0
        for part in parts:
            v = _exact_cache(s["v_pool"], s["bt"][b], case["P"], case["D"], part, False)
            out = out + torch.bmm(p[..., done: done + part.numel()], v)
            done += part.numel()
        outs.append((out / total).flatten(0, 1))
        lses.append((top + total.log()).flatten())
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}
