"""Cases, plain forms and exact values of attention over many new tokens of a sequence, and of reading
a cache back:

  attn_prefill_gqa        causal attention of whole prompts, packed one behind the other (or of their
                          ends, after a prefix that is in the keys and values already)
  attn_prefill_gqa_paged  causal attention of chunks of new tokens over their paged cache
  cache_read, cache_read_q4   the tokens that a paged, rolling or 4-bit cache holds, as packed rows

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
        # one user's short prompt, Llama-3-8B heads: latency
        dict(name="prompt one short", op="packed", dtype="bf16", B=1, Hq=32, Hkv=8, D=128, new_lo=513, new_hi=513,
             old_lo=0, old_hi=0, window=0, sink=0, learned=False),
        # a ragged batch of prompts, the same heads, values as a slice of the projection's output
        dict(name="prompt ragged batch", op="packed", dtype="bf16", B=9, Hq=32, Hkv=8, D=128, new_lo=61, new_hi=3581,
             old_lo=0, old_hi=0, window=0, sink=0, learned=False),
        # one long prompt of an odd length: the tensor cores' rate
        dict(name="prompt long", op="packed", dtype="bf16", B=1, Hq=32, Hkv=8, D=128, new_lo=16385, new_hi=16385,
             old_lo=0, old_hi=0, window=0, sink=0, learned=False),
        # float32, 64-wide heads, sliding window with sink tokens and a learned sink, after prefixes read back
        dict(name="prompt window f32", op="packed", dtype="f32", B=5, Hq=16, Hkv=4, D=64, new_lo=33, new_hi=1500,
             old_lo=0, old_hi=700, window=512, sink=4, learned=True),
        # one user's draft tokens, a short context: latency
        dict(name="chunk one draft", op="paged", dtype="bf16", B=1, Hq=32, Hkv=8, D=128, P=64, new_lo=5, new_hi=5,
             old_lo=1024, old_hi=1024, window=0, sink=0, learned=False),
        # drafts of a batch of 32 sequences to be verified, Llama-3-8B heads: the cache's bytes
        dict(name="chunk drafts", op="paged", dtype="bf16", B=32, Hq=32, Hkv=8, D=128, P=64, new_lo=1, new_hi=8,
             old_lo=4096, old_hi=8184, window=0, sink=0, learned=False),
        # a 2048-token chunk of each of two long prompts, large pages
        dict(name="chunk long prompt", op="paged", dtype="bf16", B=2, Hq=32, Hkv=8, D=128, P=256, new_lo=2048,
             new_hi=2048, old_lo=25600, old_hi=27953, window=0, sink=0, learned=False),
        # sliding window with sink tokens and a learned sink logit, 64-wide heads, small pages
        dict(name="chunk window", op="paged", dtype="bf16", B=8, Hq=64, Hkv=8, D=64, P=16, new_lo=200, new_hi=1000,
             old_lo=100, old_hi=8001, window=4096, sink=4, learned=True),
        # float32, seven query heads to a KV head, ragged chunks
        dict(name="chunk f32", op="paged", dtype="f32", B=6, Hq=14, Hkv=2, D=128, P=32, new_lo=1, new_hi=301,
             old_lo=400, old_hi=5003, window=0, sink=0, learned=False),
        # a ragged batch of contexts out of the 4-bit cache, for the attention of their next chunks
        dict(name="read 4 bits", op="read_q4", dtype="bf16", B=9, Hq=32, Hkv=8, D=128, P=64, new_lo=0, new_hi=0,
             old_lo=1001, old_hi=8191, window=0, sink=0, learned=False),
        # what rolling caches with sinks hold, float32
        dict(name="read rolling f32", op="read", dtype="f32", B=6, Hq=16, Hkv=4, D=64, P=16, new_lo=0, new_hi=0,
             old_lo=100, old_hi=3001, window=512, sink=4, learned=False),
        # a few short contexts out of a paged cache: latency
        dict(name="read few", op="read", dtype="bf16", B=4, Hq=32, Hkv=8, D=128, P=64, new_lo=0, new_hi=0, old_lo=33,
             old_hi=700, window=0, sink=0, learned=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["packed", "packed", "paged", "paged", "read", "read_q4"])
    Hkv = rng.choice([1, 2, 4, 5, 8])
    G = rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 12, 16])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), Hq=Hkv * G, Hkv=Hkv, D=rng.choice([64, 128]),
             P=rng.choice([16, 32, 64, 128, 256]))
    windowed = rng.random() < 0.35
    if op in ("read", "read_q4"):
        c["B"] = _log(rng, 1, 48)
        c["new_lo"] = c["new_hi"] = 0
        c["old_hi"] = _log(rng, 1, max(2, 60000 // c["B"]))
        c["old_lo"] = max(1, c["old_hi"] * rng.randint(0, 10) // 10)
        c["learned"] = False
    else:
        c["B"] = _log(rng, 1, 32)
        # chunks of one token to whole prompts; at most a quarter of the listed long prompt's pairs
        most = 2.0e9 / (c["B"] * c["Hq"])
        kind = rng.choice(["drafts", "chunks", "prompts"])
        if kind == "drafts":
            c["new_hi"] = _log(rng, 1, 16)
        else:
            c["new_hi"] = _log(rng, 1, max(2, min(8000, math.sqrt(most) / 1.5)))
        c["new_lo"] = rng.choice([1, max(1, c["new_hi"] // 2), c["new_hi"]])
        room = int(min(30000, most / c["new_hi"], 1.2e6 / c["B"])) - c["new_hi"]
        c["old_hi"] = 0 if kind == "prompts" or room < 2 else _log(rng, 1, room)
        c["old_lo"] = c["old_hi"] * rng.randint(0, 10) // 10
        c["learned"] = rng.random() < 0.3
    c["window"] = _log(rng, 15, 3000) if windowed else 0
    c["sink"] = rng.choice([0, 1, 4, 33]) if windowed else 0
    return c


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, the same ones for a case whatever the seed."""
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _lengths(case):
    """(new tokens, lengths with them) of every sequence."""
    new = _spread(case["new_lo"], case["new_hi"], case["B"])
    old = _spread(case["old_lo"], case["old_hi"], case["B"])[::-1]
    return new, [n + o for n, o in zip(new, old)]


def _held(case, L):
    """Tokens of a sequence of length L that its cache holds."""
    return L if case["window"] == 0 else min(L, case["window"] + case["sink"])


def _row_bytes(case):
    """Bytes of a key (or value) row of one head in the cache."""
    D = case["D"]
    return D // 2 + 4 * (D // 64) if case["op"] == "read_q4" else D * _SIZE[case["dtype"]]


def work(case):
    new, lens = _lengths(case)
    e, D, Hq, Hkv, W, ns = _SIZE[case["dtype"]], case["D"], case["Hq"], case["Hkv"], case["window"], case["sink"]
    if case["op"] in ("read", "read_q4"):
        rows = sum(_held(case, L) for L in lens) * 2 * Hkv
        return {"bytes": rows * (_row_bytes(case) + D * e), "flops": 2 * rows * D if case["op"] == "read_q4" else 0}
    pairs, keys = 0, 0
    for n, L in zip(new, lens):
        p = np.arange(L - n, L, dtype=np.int64)
        seen = p + 1
        if W:
            first = np.maximum(0, p - W + 1)
            seen = p + 1 - first + np.minimum(ns, first)
            low = int(first.min())
            keys += L - low + min(ns, low)
        else:
            keys += L
        pairs += int(seen.sum())
    T = sum(new)
    return {"bytes": keys * 2 * Hkv * D * e + T * Hq * (2 * D * e + 4), "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------------------------ inputs
def _normal(gen, *shape, scale=1.0):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).mul_(scale)


def _keys(gen, *shape):
    """Keys of uneven channels around a mean of their own, as a model's; the last dims are (heads, ..., D)."""
    D = shape[-1]
    return _normal(gen, *shape).mul_(0.3 + 1.2 * torch.rand(D, generator=gen, device="cuda")).add_(_normal(gen, D, scale=0.5))


def _table(slots, P, gen):
    """Shuffled pages of a pool with a few spare ones: (block table, pages)."""
    need = [-(-n // P) for n in slots]
    pages, most = sum(need) + 3, max(need)
    perm = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    start = torch.tensor(np.cumsum([0] + need[:-1]), device="cuda")
    at = start[:, None] + torch.arange(most, device="cuda")[None, :]
    held = torch.arange(most, device="cuda")[None, :] < torch.tensor(need, device="cuda")[:, None]
    return torch.where(held, perm[at.clamp_max(pages - 1)], -1).to(torch.int32).contiguous(), pages


def _cu(n):
    return torch.tensor(np.cumsum([0] + list(n)), dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    rng = np.random.default_rng(int(seed))
    new, lens = _lengths(case)
    order = rng.permutation(case["B"])
    new, lens = [new[i] for i in order], [lens[i] for i in order]
    dt, D, Hq, Hkv = _DT[case["dtype"]], case["D"], case["Hq"], case["Hkv"]
    s = dict(case=case, sl=torch.tensor(lens, dtype=torch.int32, device="cuda"),
             err=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if case["op"] in ("read", "read_q4"):
        held = [_held(case, L) for L in lens]
        rolling = case["window"] > 0
        s["bt"], pages = _table([case["window"] + case["sink"]] * case["B"] if rolling else lens, case["P"], gen)
        s["cu"], T = _cu(held), sum(held)
        if case["op"] == "read":
            s["k_pool"] = _keys(gen, pages, Hkv, case["P"], D).to(dt)
            s["v_pool"] = _normal(gen, pages, Hkv, case["P"], D).to(dt)
        else:
            s["k_pool"] = _filled_pool(gen, pages, Hkv, case["P"], D, True)
            s["v_pool"] = _filled_pool(gen, pages, Hkv, case["P"], D, False)
        s["k_out"] = torch.empty(T, Hkv, D, dtype=dt, device="cuda")
        s["v_out"] = torch.empty(T, Hkv, D, dtype=dt, device="cuda")
        return s
    T = sum(new)
    s["cu"] = _cu(new)
    s["q"] = _normal(gen, T, Hq, D).to(dt)
    s["sink_logit"] = _normal(gen, Hq) if case["learned"] else None
    s["out"] = torch.empty(T, Hq, D, dtype=dt, device="cuda")
    s["lse"] = torch.empty(T, Hq, device="cuda")
    if case["op"] == "packed":
        Tk = sum(lens)
        s["cu_k"] = _cu(lens)
        s["k"] = _keys(gen, Tk, Hkv, D).to(dt)
        # without a prefix the values are a slice of the projection that gave q, k and v
        wide = Hq + 2 * Hkv if case["old_hi"] == 0 else Hkv
        s["v"] = _normal(gen, Tk, wide, D).to(dt)[:, wide - Hkv:]
        return s
    s["bt"], pages = _table(lens, case["P"], gen)
    s["k_pool"] = _keys(gen, pages, Hkv, case["P"], D).to(dt)
    s["v_pool"] = _normal(gen, pages, Hkv, case["P"], D).to(dt)
    return s


def _filled_pool(gen, pages, Hkv, P, D, is_k):
    x = _keys(gen, pages, Hkv, P, D) if is_k else _normal(gen, pages, Hkv, P, D)
    return _pack(*_quantise(x), is_k)


# -------------------------------------------------------------------------- 4-bit rows, plain
def _quantise(x):
    """x [..., D] float32 -> codes [..., D] int32, scale and minimum [..., D / 64] float16."""
    g = x.unflatten(-1, (-1, 64))
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    b, s = lo.half(), ((hi - lo) * (1.0 / 15.0)).half()
    code = ((g - b.float()) * (1.0 / s.float())).round().clamp(0, 15)
    return code.to(torch.int32).flatten(-2), s.squeeze(-1), b.squeeze(-1)


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
    wide = c.to(torch.int64) << at.to(torch.int64)
    word = ((wide & 0xFFFFFFFF) | (wide >> 32)).sum(-1)  # a code past bit 31 goes on at bit 0
    word = torch.where(word >= 2 ** 31, word - 2 ** 32, word).to(torch.int32).contiguous()
    codes = word.view(torch.uint8).reshape(n, h, P // 16, 16 * D // 2)
    par = torch.stack([s, b], -1).contiguous().view(torch.uint8).reshape(n, h, P // 16, 16 * 4 * (D // 64))
    return torch.cat([codes, par], -1).reshape(n, h, -1).contiguous()


def _unpack(blk, D, is_k):
    """Blocks [..., block_bytes] -> values [..., 16, D] float32."""
    cb = 16 * D // 2
    word = blk[..., :cb].contiguous().view(torch.int32)
    par = blk[..., cb:].contiguous().view(torch.float16).unflatten(-1, (16, D // 64, 2)).float()
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
    return (code.unflatten(-1, (-1, 64)).float() * par[..., :1] + par[..., 1:]).flatten(-2)


# ------------------------------------------------------------------------------- plain forms
def _padded_rows(cu, most):
    """Row of token i of sequence b in the packed rows, and whether there is one: [B, most]."""
    i = torch.arange(most, device="cuda")[None, :]
    at = cu.long()[:-1, None] + i
    return at, i < cu.diff().long()[:, None]


def _plain_attention(s):
    c = s["case"]
    B, Hq, Hkv, D, W, ns = c["B"], c["Hq"], c["Hkv"], c["D"], c["window"], c["sink"]
    new, lens = _lengths(c)
    nq, nk = max(new), max(lens)
    q_at, q_in = _padded_rows(s["cu"], nq)
    t = torch.arange(nk, device="cuda")
    kv_in = t[None, :] < s["sl"].long()[:, None]
    if c["op"] == "packed":
        at = _padded_rows(s["cu_k"], nk)[0].clamp_max(s["k"].shape[0] - 1)
        k, v = s["k"][at], s["v"][at]  # [B, nk, Hkv, D]
    else:
        page = s["bt"].long()[:, t // c["P"]].clamp_min(0)
        k, v = s["k_pool"].transpose(1, 2)[page, t % c["P"]], s["v_pool"].transpose(1, 2)[page, t % c["P"]]
    k = k.permute(0, 2, 3, 1).float()
    v = v.transpose(1, 2).float().masked_fill(~kv_in[:, None, :, None], 0.0)
    q = s["q"][q_at.clamp_max(s["q"].shape[0] - 1)].float()  # [B, nq, Hq, D]
    q = q.view(B, nq, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    x = torch.matmul(q, k).mul_(1.0 / math.sqrt(D)).view(B, Hq, nq, nk)
    pos = (s["sl"].long() - s["cu"].long().diff())[:, None, None] + torch.arange(nq, device="cuda")[None, :, None]
    seen = t <= pos
    if W:
        seen &= (t > pos - W) | (t < ns)
    x.masked_fill_(~seen[:, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    if s["sink_logit"] is not None:
        sink = s["sink_logit"].view(1, Hq, 1, 1)
        top = torch.maximum(top, sink)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    if s["sink_logit"] is not None:
        total = total + torch.exp(sink - top)
    out = torch.matmul(p.view(B, Hkv, -1, nk), v).view(B, Hq, nq, D) / total
    lse = (top + total.log()).squeeze(-1)
    # the tokens of all sequences one behind the other again
    return {"out": out.transpose(1, 2)[q_in].to(s["q"].dtype), "lse": lse.transpose(1, 2)[q_in]}


def _plain_read(s):
    c = s["case"]
    P, W, ns = c["P"], c["window"], c["sink"]
    most = max(_held(c, L) for L in _lengths(c)[1])
    _, inside = _padded_rows(s["cu"], most)
    L = s["sl"].long()[:, None]
    t = torch.arange(most, device="cuda")[None, :].expand(c["B"], -1)
    if W:  # the sinks, then the newest tokens, each in its slot
        t = torch.where(t < ns, t, t + (L - (W + ns)).clamp_min(0))
        t = torch.where(t < ns, t, ns + (t - ns) % W)
    b, slot = torch.arange(c["B"], device="cuda")[:, None].expand(-1, most)[inside], t[inside]
    page = s["bt"].long()[b, slot // P]

    def rows(pool, is_k):
        if c["op"] == "read":
            return pool.transpose(1, 2)[page, slot % P]
        per = P // 16
        blocks = pool.view(-1, c["Hkv"], per, pool.shape[2] // per).transpose(1, 2)
        x = _unpack(blocks, c["D"], is_k)  # [pages, blocks, Hkv, 16, D]
        return x.transpose(2, 3)[page, slot % P // 16, slot % 16].to(s["k_out"].dtype)

    return {"k": rows(s["k_pool"], True), "v": rows(s["v_pool"], False)}


def run(state):
    s, c = state, state["case"]
    if not own:
        return _plain_read(s) if c["op"] in ("read", "read_q4") else _plain_attention(s)
    import kv_cache_decode_split_gb300 as kvd
    if c["op"] in ("read", "read_q4"):
        read = kvd.cache_read if c["op"] == "read" else kvd.cache_read_q4
        read(s["k_pool"], s["v_pool"], s["bt"], s["sl"], s["cu"], s["k_out"], s["v_out"], window=c["window"],
             n_sink=c["sink"], err=s["err"])
        return {"k": s["k_out"], "v": s["v_out"]}
    more = dict(window=c["window"], n_sink_tokens=c["sink"], sink_logit=s["sink_logit"], out=s["out"],
                lse_out=s["lse"], err=s["err"])
    if c["op"] == "packed":
        kvd.attn_prefill_gqa(s["q"], s["k"], s["v"], s["cu"], s["cu_k"], **more)
    else:
        kvd.attn_prefill_gqa_paged(s["q"], s["k_pool"], s["v_pool"], s["bt"], s["sl"], s["cu"], **more)
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------------------------- exact
def _exact_q4(pool, pages, P, D, slots, is_k):
    """Values [n, Hkv, D] in float64 of the given slots of one sequence, each code found by its address."""
    size = 8 * D + 4 * (D // 4)
    page = pages[slots // P].long()
    rr, base = (slots % 16)[:, None], (slots % P // 16) * size
    ch = torch.arange(D, device="cuda")[None, :]
    if is_k:
        w, t, n = ch // 32, ch // 8 % 4, ch % 8
        word, bit = (rr * 4 + t) * (D // 32) + w, (4 * n + 3) % 32
    else:
        f, t, o, w, j, g = rr // 8, rr // 2 % 4, rr % 2, ch // 64, ch // 8 % 8, ch % 8
        word = (((f * 8 + g) * 4 + t) * 2 + o) * 2 + w if D == 128 else ((g * 4 + t) * 2 + f) * 2 + o
        bit = 4 * j
    bit = bit.expand(slots.numel(), -1)

    def byte(at):
        return torch.stack([pool[page[:, None], h, at].long() for h in range(pool.shape[1])], 1)

    lo, bit = base[:, None] + 4 * word, bit[:, None]
    first, second = byte(lo + bit[:, 0] // 8), byte(lo + (bit[:, 0] // 8 + 1) % 4)
    code = (((second << 8) | first) >> (bit % 8)) & 15
    at = base[:, None] + 8 * D + (rr * (D // 64) + ch // 64) * 4

    def half(at):
        return ((byte(at + 1) << 8) | byte(at)).to(torch.int16).view(torch.float16).double()

    return half(at) * code.double() + half(at + 2)


def exact(case, seed):
    s = prepare(case, seed)
    P, W, ns, H = case.get("P"), case["window"], case["sink"], case["Hkv"]
    lens = s["sl"].tolist()
    if case["op"] in ("read", "read_q4"):
        ks, vs = [], []
        for b, L in enumerate(lens):
            t = torch.arange(L, device="cuda")
            if W:
                t = t[(t < ns) | (t >= L - W)]
                t = torch.where(t < ns, t, ns + torch.remainder(t - ns, W))
            for pool, to, is_k in ((s["k_pool"], ks, True), (s["v_pool"], vs, False)):
                if case["op"] == "read":
                    to.append(pool[s["bt"][b, t // P].long(), :, t % P].double())
                else:
                    to.append(torch.cat([_exact_q4(pool, s["bt"][b], P, case["D"], x, is_k) for x in t.split(4096)]))
        return {"k": torch.cat(ks), "v": torch.cat(vs)}
    new, scale = s["cu"].diff().tolist(), 1.0 / math.sqrt(case["D"])
    G, row, key_row = case["Hq"] // H, 0, 0
    outs, lses = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda"), torch.empty(s["lse"].shape, dtype=torch.float64, device="cuda")
    for b, (n, L) in enumerate(zip(new, lens)):
        t = torch.arange(L, device="cuda")
        if case["op"] == "packed":
            k, v = s["k"][key_row: key_row + L], s["v"][key_row: key_row + L]
        else:
            at = (s["bt"][b, t // P].long(), slice(None), t % P)
            k, v = s["k_pool"][at], s["v_pool"][at]
        k, v = k.transpose(0, 1).double(), v.transpose(0, 1).double()  # [H, L, D]
        for i in range(0, n, 1024):  # some queries at a time, with the keys up to the last of them
            m = min(1024, n - i)
            end = L - n + i + m
            p = torch.arange(end - m, end, device="cuda")[:, None]
            hidden = t[None, :end] > p
            if W:
                hidden |= (t[None, :end] <= p - W) & (t[None, :end] >= ns)
            for h in range(H):
                for g in range(h * G, h * G + G):
                    x = (s["q"][row + i: row + i + m, g].double() @ k[h, :end].T) * scale
                    x[hidden] = -math.inf
                    if s["sink_logit"] is not None:
                        x = torch.cat([x, s["sink_logit"][g].double().expand(m, 1)], 1)
                    z = torch.logsumexp(x, 1)
                    lses[row + i: row + i + m, g] = z
                    outs[row + i: row + i + m, g] = torch.exp(x[:, :end] - z[:, None]) @ v[h, :end]
        row, key_row = row + n, key_row + L
    return {"out": outs, "lse": lses}
