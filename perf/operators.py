"""The generation operators over an 8-bit key/value cache, as cases to be timed and compared.

  append   new keys and values are quantised into a cache of 8-bit codes with one power-of-two
           scale for each block of tokens of each head
  decode   the attention of a few new queries against that cache, which can also add every cached
           position's attention weight to a running total
  weights  the same totals for a prompt: column sums of its attention matrix, from the forward's
           log-sum-exp
  evict    the positions with the least total are dropped and the rest moved into another cache

With ``own`` true ``run`` calls the package's entry points, otherwise plain torch operations.
"""
import math

import torch

own = False

D = 64                                   # head size of every bf16 kernel of the package
QMAX = {"e4m3": 448.0, "int8": 127.0}
CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
FLOAT = {"bf16": torch.bfloat16, "f32": torch.float32}
LOW, HIGH = -40, 40                      # exponents that a scale may take


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one generation step of 64 sequences of the big model (16 heads): every head of every
        # sequence gets one new token, most of them into a block that is begun already
        dict(name="append step", op="append", B=64, H=16, N=1, Lmax=4096, block=64, dtype="bf16",
             code="e4m3", start="any"),
        # the big model's prompts, 8 sequences of 4096 tokens, into empty caches
        dict(name="append prompt", op="append", B=8, H=16, N=4096, Lmax=4608, block=64,
             dtype="bf16", code="int8", start="empty"),
        # a padded batch of short continuations in fp32, small blocks, odd sizes
        dict(name="append ragged", op="append", B=5, H=3, N=77, Lmax=777, block=16, dtype="f32",
             code="e4m3", start="any"),
        # one token of one sequence of the base model (8 heads), a short cache: latency
        dict(name="decode one", op="decode", B=1, H=8, Hkv=8, Nq=1, Lmax=64, block=64,
             dtype="bf16", code="e4m3", causal=True, add=False, lens="37"),
        # the generation step of the benchmark: 64 sequences, 16 heads, 4096 positions
        dict(name="decode step", op="decode", B=64, H=16, Hkv=16, Nq=1, Lmax=4096, block=64,
             dtype="bf16", code="int8", causal=True, add=True, lens="full"),
        # grouped heads, four new tokens at once (a draft being verified), ragged long caches
        dict(name="decode grouped", op="decode", B=8, H=32, Hkv=8, Nq=4, Lmax=16384, block=32,
             dtype="bf16", code="e4m3", causal=True, add=True, lens="any"),
        # one sequence with a very long cache, fp32 queries
        dict(name="decode long", op="decode", B=1, H=8, Hkv=8, Nq=1, Lmax=131072, block=128,
             dtype="f32", code="e4m3", causal=False, add=False, lens="full"),
        # the base model's decoder batch: 32 prompts of 256 tokens
        dict(name="weights base", op="weights", B=32, H=8, Hkv=8, N=256, dtype="bf16",
             mask="causal", lens="full"),
        # the big model's prompts
        dict(name="weights big", op="weights", B=8, H=16, Hkv=16, N=4096, dtype="bf16",
             mask="none", lens="full"),
        # padded prompts with grouped heads in fp32
        dict(name="weights ragged", op="weights", B=3, H=6, Hkv=2, N=333, dtype="f32",
             mask="key_padding", lens="any"),
        # prompts of 4096 tokens cut to 1024 after they were read
        dict(name="evict prompt", op="evict", B=64, H=16, Lmax=4096, Lout=1280, keep=1024,
             recent=128, block=64, code="e4m3", lens="full"),
        # one very long sequence cut to an odd number of positions
        dict(name="evict long", op="evict", B=1, H=8, Lmax=131072, Lout=8192, keep=8001,
             recent=33, block=128, code="int8", lens="full"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["append", "decode", "weights", "evict"])
    B, H = _log(rng, 1, 64), rng.choice([1, 2, 3, 5, 8, 16])
    block, code = rng.choice([16, 32, 64, 128]), rng.choice(["e4m3", "int8"])
    dtype, lens = rng.choice(["bf16", "f32"]), rng.choice(["any", "full"])
    if op == "append":
        N = _log(rng, 1, 4096)
        B = min(B, max(1, 32768 // N))
        return dict(op=op, B=B, H=H, N=N, Lmax=N + _log(rng, 1, 4096), block=block, dtype=dtype,
                    code=code, start=rng.choice(["any", "empty"]))
    if op == "decode":
        Lmax = _log(rng, 16, 131072)
        B = max(1, min(B, 2097152 // (Lmax * H)))
        return dict(op=op, B=B, H=H * rng.choice([1, 1, 2, 4, 8]), Hkv=H,
                    Nq=min(Lmax, rng.choice([1, 1, 1, 2, 4, 7, 16])), Lmax=Lmax, block=block,
                    dtype=dtype, code=code, causal=rng.random() < 0.7, add=rng.random() < 0.5,
                    lens=lens)
    if op == "weights":
        N = _log(rng, 1, 4096) if dtype == "bf16" else _log(rng, 1, 1024)
        G = rng.choice([1, 1, 2, 4])
        B = max(1, min(B, 536870912 // (N * N * H * G), 131072 // (N * H)))
        return dict(op=op, B=B, H=H * G, Hkv=H, N=N, dtype=dtype,
                    mask=rng.choice(["none", "causal", "key_padding"]), lens=lens)
    Lmax = _log(rng, 16, 131072)
    B = max(1, min(B, 4194304 // (Lmax * H)))
    keep = _log(rng, 1, min(Lmax, 16384))
    return dict(op=op, B=B, H=H, Lmax=Lmax, Lout=keep + rng.randrange(0, 300), keep=keep,
                recent=rng.choice([0, 1, keep // 8, keep]), block=block, code=code, lens=lens)


# ------------------------------------------------------------------ inputs
def _lens(g, c, cap):
    """int32 [B] valid lengths: all of `cap`, a given number, or anything from 0 to `cap`."""
    if c["lens"] == "full":
        return torch.full((c["B"],), cap, dtype=torch.int32, device="cuda")
    if c["lens"] != "any":
        return torch.full((c["B"],), int(c["lens"]), dtype=torch.int32, device="cuda")
    return torch.randint(0, cap + 1, (c["B"],), generator=g, device="cuda").to(torch.int32)


def _scale_for(amax, code):
    """The least power of two s with amax <= QMAX s, its exponent kept within LOW..HIGH."""
    m, e = torch.frexp(amax.float())
    qm, qe = math.frexp(QMAX[code])
    e = torch.where(m <= qm, e - qe, e - qe + 1).clamp(LOW, HIGH)
    return torch.ldexp(torch.ones_like(m), e)


def _encode(x, code):
    """The nearest 8-bit codes (ties to even) of x, saturating; a NaN stays NaN, or 0 in int8."""
    x = x.clamp(-QMAX[code], QMAX[code])
    if code == "e4m3":
        return x.to(torch.float8_e4m3fn)
    return x.nan_to_num(nan=0.0).round().to(torch.int8)


def _filled(g, c, H, L):
    """Codes and scales of a cache of L tokens: normal values, each head at its own size and a
    few tokens far larger than the rest, as keys and values have them."""
    B, bs = c["B"], c["block"]
    x = torch.randn(B, H, L, D, generator=g, device="cuda")
    x *= torch.exp2(torch.randn(1, H, 1, 1, generator=g, device="cuda"))
    x *= 1 + 5 * (torch.rand(B, H, L, 1, generator=g, device="cuda") < 0.01)
    pad = -L % bs
    xp = torch.nn.functional.pad(x, (0, 0, 0, pad)).view(B, H, -1, bs, D)
    s = _scale_for(xp.abs().amax((3, 4)), c["code"])
    codes = _encode(xp / s[..., None, None], c["code"]).reshape(B, H, L + pad, D)
    return codes.view(torch.uint8)[:, :, :L].contiguous().view(CODE[c["code"]]), s


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, dtype="f32"):
        return torch.randn(*shape, generator=g, device="cuda").to(FLOAT[dtype])

    s = {"case": c}
    if c["op"] == "append":
        B, H, N, Lmax = c["B"], c["H"], c["N"], c["Lmax"]
        s["k_cache"], s["k_scale"] = _filled(g, c, H, Lmax)
        s["v_cache"], s["v_scale"] = _filled(g, c, H, Lmax)
        s["weights"] = torch.rand(B, H, Lmax, generator=g, device="cuda")
        s["k"] = randn(B, H, N, D, dtype=c["dtype"]) * 3
        s["v"] = randn(B, H, N, D, dtype=c["dtype"])
        s["len"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        s["new_len"] = None
        if c["start"] == "any":
            s["len"] = _lens(g, dict(c, lens="any"), Lmax - N)
            if N > 1:
                s["new_len"] = _lens(g, dict(c, lens="any"), N)
    elif c["op"] == "decode":
        B, Hkv, Lmax = c["B"], c["Hkv"], c["Lmax"]
        s["k_cache"], s["k_scale"] = _filled(g, c, Hkv, Lmax)
        s["v_cache"], s["v_scale"] = _filled(g, c, Hkv, Lmax)
        s["weights"] = torch.rand(B, Hkv, Lmax, generator=g, device="cuda") if c["add"] else None
        s["q"] = randn(B, c["H"], c["Nq"], D, dtype=c["dtype"])
        s["len"] = _lens(g, c, Lmax)
    elif c["op"] == "weights":
        B, H, Hkv, N = c["B"], c["H"], c["Hkv"], c["N"]
        s["q"] = randn(B, H, N, D, dtype=c["dtype"])
        s["k"] = randn(B, Hkv, N, D, dtype=c["dtype"])
        s["key_len"] = s["query_len"] = None
        if c["mask"] == "key_padding":
            s["key_len"] = s["query_len"] = _lens(g, c, N)
        s["weights"] = torch.zeros(B, Hkv, N, device="cuda")  # the prompt is what comes first
        lse = torch.empty(B, H, N, device="cuda")
        for b in range(B):  # what the attention forward of the prompt has left
            one = slice(b, b + 1)
            lse[one] = torch.logsumexp(_scores(s["q"][one], s["k"][one], c["mask"],
                                               None if s["key_len"] is None
                                               else s["key_len"][one]), -1)
        s["lse"] = torch.where(lse == -math.inf, math.inf, lse)
    else:
        B, H, Lmax, Lout = c["B"], c["H"], c["Lmax"], c["Lout"]
        s["k_cache"], s["k_scale"] = _filled(g, c, H, Lmax)
        s["v_cache"], s["v_scale"] = _filled(g, c, H, Lmax)
        # totals of attention weight: a few positions hold most of it, many hold next to none
        s["weights"] = torch.exp(2 * torch.randn(B, H, Lmax, generator=g, device="cuda"))
        s["weights"] *= torch.rand(B, H, Lmax, generator=g, device="cuda") < 0.9
        s["len"] = _lens(g, c, Lmax)
        nb = -(-Lout // c["block"])
        for n in ("k", "v"):
            s[n + "_out"] = torch.zeros(B, H, Lout, D, dtype=torch.int8,
                                        device="cuda").view(CODE[c["code"]])
            s[n + "_scale_out"] = torch.ones(B, H, nb, device="cuda")
        s["weights_out"] = torch.zeros(B, H, Lout, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms
def _per_token(scale, block, L):
    return scale.repeat_interleave(block, 2)[:, :, :L]


def _append_one(x, cache, scale, s):
    c = s["case"]
    B, H, N, Lmax, bs = c["B"], c["H"], c["N"], c["Lmax"], c["block"]
    length = s["len"].long()
    n = torch.full_like(length, N) if s["new_len"] is None else s["new_len"].long()
    first = length // bs
    W = -(-N // bs) + 1                                   # blocks that N tokens can touch
    pos = first[:, None] * bs + torch.arange(W * bs, device="cuda")          # [B, W bs]
    i = pos - length[:, None]
    new = (i >= 0) & (i < n[:, None]) & (pos < Lmax)
    old = pos < length[:, None]
    at = pos.clamp(max=Lmax - 1)[:, None, :, None].expand(B, H, -1, D)
    take = i.clamp(0, N - 1)[:, None, :, None].expand(B, H, -1, D)
    fresh = torch.where(new[:, None, :, None], x.gather(2, take).float(), 0.0)
    codes = cache.view(torch.uint8).gather(2, at).view(cache.dtype).float()
    blocks = (first[:, None] + torch.arange(W, device="cuda")).clamp(max=scale.shape[2] - 1)
    blocks = blocks[:, None].expand(B, H, W)
    was = scale.gather(2, blocks)
    amax = torch.where(fresh.isfinite(), fresh.abs(), 0.0).view(B, H, W, bs * D).amax(3)
    now = _scale_for(amax, c["code"])
    begun = old.view(B, 1, W, bs).any(3)
    now = torch.where(begun, torch.maximum(was, now), now)
    each = now.repeat_interleave(bs, 2)[..., None]
    ratio = (was / now).repeat_interleave(bs, 2)[..., None]
    codes = torch.where(new[:, None, :, None], fresh / each, codes * ratio)
    touched = new.view(B, W, bs).any(2)                   # blocks that get a new token
    write = (new | old) & touched.repeat_interleave(bs, 1)
    b, p = write.nonzero(as_tuple=True)
    cache.view(torch.uint8)[b, :, pos[b, p]] = _encode(codes, c["code"]).view(torch.uint8)[b, :, p]
    b, p = touched.nonzero(as_tuple=True)
    scale[b, :, first[b] + p] = now[b, :, p]
    b, p = new.nonzero(as_tuple=True)
    s["weights"][b, :, pos[b, p]] = 0.0


def _scores(q, k, mask, key_len):
    """[B, H, Nq, Nk] scaled scores in 32 bits, -inf where a key is excluded."""
    B, H, Nq, _ = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    x = (q.float().reshape(B, Hkv, -1, D) @ k.float().transpose(2, 3)).view(B, H, Nq, Nk) / 8.0
    j = torch.arange(Nk, device=q.device)
    if mask == "causal":
        x = x.masked_fill_(j > torch.arange(Nq, device=q.device)[:, None], -math.inf)
    elif mask == "key_padding":
        x = x.masked_fill_(j >= key_len[:, None, None, None], -math.inf)
    return x


def _run_append(s):
    if own:
        import transformer_head_scaled_04_gb300 as mha

        mha.kv_append_q8(mha.KvCacheQ8(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                       s["weights"], s["case"]["block"]),
                         s["k"], s["v"], s["len"], s["new_len"])
    else:
        _append_one(s["k"], s["k_cache"], s["k_scale"], s)
        _append_one(s["v"], s["v_cache"], s["v_scale"], s)
    return {n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale", "weights")}


def _run_decode(s):
    c = s["case"]
    if own:
        import transformer_head_scaled_04_gb300 as mha

        out = mha.sdpa_decode_q8(s["q"], mha.KvCacheQ8(s["k_cache"], s["v_cache"], s["k_scale"],
                                                       s["v_scale"], s["weights"], c["block"]),
                                 s["len"], causal=c["causal"], add_weights=c["add"])
        return {"out": out, "weights": s["weights"]}
    B, H, Hkv, Nq, Lmax = c["B"], c["H"], c["Hkv"], c["Nq"], c["Lmax"]
    k = s["k_cache"].float() * _per_token(s["k_scale"], c["block"], Lmax)[..., None]
    v = s["v_cache"].float() * _per_token(s["v_scale"], c["block"], Lmax)[..., None]
    x = (s["q"].float().view(B, Hkv, -1, D) @ k.transpose(2, 3)).view(B, Hkv, -1, Nq, Lmax) / 8.0
    j = torch.arange(Lmax, device="cuda")
    last = s["len"][:, None].expand(B, Nq) - 1            # the last key that a query may see
    if c["causal"]:
        last = last - (Nq - 1) + torch.arange(Nq, device="cuda")
    x = x.masked_fill(j > last[:, None, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-37)
    out = (p.view(B, Hkv, -1, Lmax) @ v).view(B, H, Nq, D).to(s["q"].dtype)
    if c["add"]:
        s["weights"] += p.sum((2, 3))
    return {"out": out, "weights": s["weights"]}


def _run_weights(s):
    c = s["case"]
    if own:
        import transformer_head_scaled_04_gb300 as mha

        return mha.sdpa_key_weights(s["q"], s["k"], s["lse"], c["mask"], s["key_len"],
                                    s["query_len"], weights=s["weights"])
    B, Hkv, N = c["B"], c["Hkv"], c["N"]
    p = torch.exp(_scores(s["q"], s["k"], c["mask"], s["key_len"]) - s["lse"][..., None])
    if s["query_len"] is not None:
        i = torch.arange(N, device="cuda")
        p = p.masked_fill((i >= s["query_len"][:, None])[:, None, :, None], 0.0)
    s["weights"] += p.view(B, Hkv, -1, N).sum(2)
    return s["weights"]


def _run_evict(s):
    c = s["case"]
    B, H, Lmax, Lout, keep, bs = (c[n] for n in ("B", "H", "Lmax", "Lout", "keep", "block"))
    if own:
        import transformer_head_scaled_04_gb300 as mha

        length, kept = mha.kv_evict_q8(
            mha.KvCacheQ8(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["weights"], bs),
            mha.KvCacheQ8(s["k_out"], s["v_out"], s["k_scale_out"], s["v_scale_out"],
                          s["weights_out"], bs),
            s["len"], keep, c["recent"])
    else:
        j = torch.arange(Lmax, device="cuda")
        n = s["len"].long()[:, None, None]
        rank = torch.where(j < n - min(c["recent"], keep), 1, 0) + 2 * (j >= n)
        rank = rank.expand(B, H, Lmax)                    # the newest, the others, no token
        w = s["weights"].masked_fill(s["weights"].isnan(), -math.inf)
        order = w.argsort(dim=-1, descending=True, stable=True)
        order = order.gather(2, rank.gather(2, order).argsort(dim=-1, stable=True))[..., :keep]
        length = s["len"].clamp(max=keep)
        real = torch.arange(keep, device="cuda") < length[:, None, None]
        at = torch.where(real, order, Lmax).sort(-1).values
        kept = torch.where(real, at, -1).to(torch.int32)
        at = at.clamp(max=Lmax - 1)
        pad = -keep % bs
        for x in ("k", "v"):
            was = s[x + "_scale"].gather(2, at // bs)
            most = torch.nn.functional.pad(torch.where(real, was, 0.0), (0, pad))
            most = most.view(B, H, -1, bs).amax(3)
            now = most.repeat_interleave(bs, 2)[..., :keep]
            code = s[x + "_cache"].view(torch.uint8).gather(
                2, at[..., None].expand(-1, -1, -1, D)).view(CODE[c["code"]])
            code = _encode(code.float() * (was / now)[..., None], c["code"]).view(torch.uint8)
            to = s[x + "_out"].view(torch.uint8)[:, :, :keep]
            to.copy_(torch.where(real[..., None], code, to))
            to = s[x + "_scale_out"][..., :most.shape[2]]
            to.copy_(torch.where(most > 0, most, to))
        to = s["weights_out"][..., :keep]
        to.copy_(torch.where(real, s["weights"].gather(2, at), to))
    return {"k": s["k_out"], "v": s["v_out"], "k_scale": s["k_scale_out"],
            "v_scale": s["v_scale_out"], "weights": s["weights_out"], "kept": kept, "len": length}


def run(state):
    return {"append": _run_append, "decode": _run_decode, "weights": _run_weights,
            "evict": _run_evict}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "append":
        tokens = c["B"] * c["H"] * c["N"]                 # new K and V read, their codes written
        size = 2 if c["dtype"] == "bf16" else 4
        if c["start"] == "any" and c["N"] > 1:
            tokens /= 2                                   # lengths are even over 0..N
        return {"bytes": 2 * tokens * D * (size + 1) + 4 * tokens, "flops": 4 * tokens * D}
    if c["op"] == "decode":
        L = {"full": c["Lmax"], "any": c["Lmax"] / 2}.get(c["lens"]) or int(c["lens"])
        keys = c["B"] * c["Hkv"] * L                      # codes, scales, totals; q and out
        size = 2 if c["dtype"] == "bf16" else 4
        rows = c["B"] * c["H"] * c["Nq"]
        return {"bytes": keys * (2 * D + 8 / c["block"] + (8 if c["add"] else 0))
                + 2 * rows * D * size, "flops": 4 * D * L * rows}
    if c["op"] == "weights":
        size, N = 2 if c["dtype"] == "bf16" else 4, c["N"]
        pairs = c["B"] * c["H"] * N * N
        if c["mask"] == "causal":
            pairs /= 2
        elif c["mask"] == "key_padding" and c["lens"] == "any":
            pairs /= 3                                    # the mean of n^2, n even over 0..N
        return {"bytes": c["B"] * N * (c["H"] * (D * size + 4) + c["Hkv"] * (D * size + 8)),
                "flops": 2 * D * pairs}
    L = c["Lmax"] if c["lens"] == "full" else c["Lmax"] / 2
    kept = min(L, c["keep"])                              # totals read; what is kept moved
    heads = c["B"] * c["H"]
    return {"bytes": heads * (4 * L + kept * (4 * D + 8 + 16 / c["block"])), "flops": heads * L}


# ------------------------------------------------------------------ 64 bits
def _exact_append(s):
    """Token by token over the touched blocks of each sequence, in 64 bits on the host."""
    c = s["case"]
    bs, qmax = c["block"], QMAX[c["code"]]
    out = {}
    for n in ("k", "v"):
        cache, scale = s[n + "_cache"].view(torch.uint8).clone(), s[n + "_scale"].double()
        for b in range(c["B"]):
            L = int(s["len"][b])
            new = c["N"] if s["new_len"] is None else int(s["new_len"][b])
            end = min(L + new, c["Lmax"])
            x = s[n][b].double()
            for blk in range(L // bs, -(-end // bs) if end > L else 0):
                lo, hi = max(blk * bs, L), min((blk + 1) * bs, end)
                amax = x[:, lo - L:hi - L].abs().amax((1, 2))
                sc = torch.full_like(amax, 2.0 ** LOW)
                for e in range(LOW, HIGH):
                    sc = torch.where(amax > qmax * 2.0 ** e, 2.0 ** (e + 1), sc)
                if lo > blk * bs:
                    sc = torch.maximum(sc, scale[b, :, blk])
                    old = cache[b, :, blk * bs:lo].view(CODE[c["code"]]).double()
                    old = old * (scale[b, :, blk] / sc)[:, None, None]
                    cache[b, :, blk * bs:lo] = _nearest(old, c["code"])
                cache[b, :, lo:hi] = _nearest(x[:, lo - L:hi - L] / sc[:, None, None], c["code"])
                scale[b, :, blk] = sc
            out["weights"] = s["weights"] if n == "k" else out["weights"]
            out["weights"][b, :, L:end] = 0.0
        out[n + "_cache"] = cache.view(CODE[c["code"]]).double()
        out[n + "_scale"] = scale
    out["weights"] = out["weights"].double()
    return out


def _nearest(x, code):
    """Codes nearest to x by the step at each value's size, ties to even, from 64 bits."""
    if code == "int8":
        return torch.round(x).to(torch.int8).view(torch.uint8)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).float().to(torch.float8_e4m3fn).view(torch.uint8)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "append":
        if c["B"] * (c["N"] / c["block"] + 1) > 2500:
            return None
        return _exact_append(s)
    if c["op"] == "decode":
        G, Nq = c["H"] // c["Hkv"], c["Nq"]
        out = torch.zeros(c["B"], c["H"], Nq, D, dtype=torch.float64, device="cuda")
        total = s["weights"].double() if c["add"] else None
        for b in range(c["B"]):
            L = int(s["len"][b])
            t = torch.arange(L, device="cuda") // c["block"]
            for h in range(c["Hkv"]):
                k = s["k_cache"][b, h, :L].double() * s["k_scale"][b, h, t].double()[:, None]
                v = s["v_cache"][b, h, :L].double() * s["v_scale"][b, h, t].double()[:, None]
                for i in range(Nq):
                    n = L - (Nq - 1 - i if c["causal"] else 0)
                    if n < 1:
                        continue
                    q = s["q"][b, h * G:(h + 1) * G, i].double()
                    p = torch.softmax(q @ k[:n].T * 0.125, -1)
                    out[b, h * G:(h + 1) * G, i] = p @ v[:n]
                    if c["add"]:
                        total[b, h, :n] += p.sum(0)
        return {"out": out, "weights": total}
    if c["op"] == "weights":
        G, N, total = c["H"] // c["Hkv"], c["N"], s["weights"].double()
        for b in range(c["B"]):
            nk = N if s["key_len"] is None else int(s["key_len"][b])
            nq = N if s["query_len"] is None else int(s["query_len"][b])
            for h in range(c["H"]):
                x = s["k"][b, h // G, :nk].double() @ s["q"][b, h, :nq].double().T * 0.125
                p = torch.exp(x - s["lse"][b, h, :nq].double())      # [keys, queries]
                total[b, h // G, :nk] += (p.triu() if c["mask"] == "causal" else p).sum(1)
        return total
    if c["B"] * c["H"] * (c["keep"] / c["block"] + 1) > 1500:
        return None
    return _exact_evict(s)


def _exact_evict(s):
    """Head by head and block by block, in 64 bits."""
    c = s["case"]
    bs, keep = c["block"], c["keep"]
    out = {n: s[n + "_out"].double() for n in ("k", "v", "k_scale", "v_scale", "weights")}
    for b in range(c["B"]):
        L = int(s["len"][b])
        newest = range(max(L - min(c["recent"], keep), 0), L)
        for h in range(c["H"]):
            w = s["weights"][b, h, :L].double().tolist()
            rest = sorted(range(newest.start), key=lambda j: (-w[j], j))
            at = sorted(rest[:min(keep, L) - len(newest)]) + list(newest)
            for lo in range(0, len(at), bs):
                src = torch.tensor(at[lo:lo + bs], device="cuda")
                to = slice(lo, lo + len(src))
                for n in ("k", "v"):
                    sc = s[n + "_scale"][b, h, src // bs].double()
                    x = s[n + "_cache"][b, h].view(torch.uint8)[src].view(CODE[c["code"]]).double()
                    code = _nearest(x * (sc / sc.max())[:, None], c["code"])
                    out[n][b, h, to] = code.view(CODE[c["code"]]).double()
                    out[n + "_scale"][b, h, lo // bs] = sc.max()
                out["weights"][b, h, to] = s["weights"][b, h, src].double()
    return {**out, "kept": None, "len": None}
