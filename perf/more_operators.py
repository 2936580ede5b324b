"""Attention with a learned relative position bias, as cases to be timed and compared.

  forward   O = softmax(scale Q K^T + bias, masked) V and its row log-sum-exp; the bias of query i
            and key j is one learned number per head and bucket of the distance j - i
  backward  dQ, dK, dV and the gradient of the bias table
  decode    a few new queries against a key/value cache, with the same bias

With ``own`` true ``run`` calls the package's entry points, otherwise plain torch operations.
"""
import math

import torch

own = False

FLOAT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def _case(name, op, B, H, N, mask, dtype, lens="full", D=64, buckets=32, reach=128, both=True,
          table="f32", scale="head", Nq=0):
    """N: the positions of a sequence (of the cache, for decode); mask: for decode whether the new
    queries are causal among themselves; both: keys on either side have buckets of their own;
    scale: 1/sqrt(D) ("head") or 1 ("one", as the bias's first users have it)."""
    return dict(name=name, op=op, B=B, H=H, N=N, Nq=Nq or N, mask=mask, dtype=dtype, lens=lens, D=D,
                buckets=buckets, reach=reach, both=both, table=table, scale=scale)


def listed():
    return [
        # one short sentence through the base model's encoder (8 heads): latency
        _case("forward sentence", "forward", 1, 8, 37, "none", "bf16", scale="one"),
        # the base model's decoder batch: 32 targets of 256 tokens
        _case("forward base", "forward", 32, 8, 256, "causal", "bf16", both=False),
        # the big model's heads, 8 sequences of 4096 tokens
        _case("forward big", "forward", 8, 16, 4096, "none", "bf16"),
        # a padded batch in fp32, an odd length
        _case("forward padded", "forward", 8, 8, 1001, "key_padding", "f32", lens="any",
              table="bf16"),
        # training on the base model's decoder batch
        _case("backward base", "backward", 32, 8, 256, "causal", "bf16", both=False),
        # training on the big model's heads
        _case("backward big", "backward", 8, 16, 4096, "none", "bf16", table="bf16"),
        # a small ragged batch, many buckets that reach far
        _case("backward padded", "backward", 5, 3, 777, "key_padding", "bf16", lens="any",
              buckets=64, reach=500),
        # training in fp32
        _case("backward float", "backward", 4, 8, 500, "causal", "f32", both=False),
        # one new token of one sequence, a short cache: latency
        _case("decode one", "decode", 1, 8, 64, "causal", "bf16", lens="37", both=False,
              scale="one", Nq=1),
        # the generation step of the benchmark: 64 sequences, 16 heads, 4096 positions
        _case("decode step", "decode", 64, 16, 4096, "causal", "bf16", both=False, Nq=1),
        # four new tokens at once (a draft being verified), ragged long caches
        _case("decode draft", "decode", 8, 16, 16384, "causal", "bf16", lens="any", both=False,
              reach=1000, table="bf16", Nq=4),
        # one sequence with a very long cache in fp32
        _case("decode long", "decode", 1, 8, 131072, "causal", "f32", both=False, Nq=1),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["forward", "backward", "decode"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    B, H = _log(rng, 1, 64), rng.choice([1, 2, 3, 5, 8, 16])
    buckets = rng.choice([8, 16, 32, 32, 64, 128])
    c = dict(op=op, H=H, dtype=dtype, lens=rng.choice(["any", "full"]),
             D=64 if dtype == "bf16" else rng.choice([64, 64, 32, 40, 17, 128]), buckets=buckets,
             reach=rng.choice([buckets + 1, 128, 128, 300, 1000, 4096]), both=rng.random() < 0.5,
             table=rng.choice(["f32", "bf16"]), scale=rng.choice(["head", "one"]))
    if op == "decode":
        N = _log(rng, 16, 131072)
        Nq = rng.choice([1, 1, 1, 2, 4, 7, 16])
        room = (4194304 if dtype == "bf16" else 1048576) // (1 if Nq == 1 else 2)
        B = max(1, min(B, room // (N * H)))
        H = max(1, min(H, room // (N * B)))
        return dict(c, B=B, H=H, N=N, Nq=Nq, mask=rng.choice(["causal", "causal", "none"]))
    N = _log(rng, 16 if op == "backward" else 1, 4096 if dtype == "bf16" else 1024)
    pairs = 2147483648 if dtype == "bf16" else 8000000 if op == "backward" else 64000000
    if c["D"] == 128:
        pairs //= 2
    H = max(1, min(H, pairs // (N * N)))
    B = max(1, min(B, pairs // (N * N * H), 131072 // (N * H)))
    mask = rng.choice(["none", "causal", "key_padding"])
    return dict(c, B=B, H=H, N=N, Nq=N, mask=mask,
                lens=c["lens"] if mask == "key_padding" else "full")


# ------------------------------------------------------------------ inputs
def _lens(g, c):
    """int32 [B] valid lengths: all of N, a given number, or anything from 0 to N."""
    B, N = c["B"], c["N"]
    if c["lens"] == "any":
        n = torch.randint(0, N + 1, (B,), generator=g, device="cuda").to(torch.int32)
        if c["op"] == "backward":  # one key alone has no gradient but its rounding
            n = torch.where((n > 0) & (n < 8), min(8, N), n).to(torch.int32)
        return n
    n = N if c["lens"] == "full" else int(c["lens"])
    return torch.full((B,), n, dtype=torch.int32, device="cuda")


def _scale(c):
    return c["D"] ** -0.5 if c["scale"] == "head" else 1.0


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, H, N, Nq, D = c["B"], c["H"], c["N"], c["Nq"], c["D"]

    def randn(*shape, size=1.0, dtype=c["dtype"]):
        return (torch.randn(*shape, generator=g, device="cuda") * size).to(FLOAT[dtype])

    # queries of a model without the factor 1/sqrt(D) are that much smaller
    s = {"case": c, "q": randn(B, H, Nq, D, size=1.0 if c["scale"] == "head" else D ** -0.5),
         "k": randn(B, H, N, D), "v": randn(B, H, N, D),
         "table": randn(c["buckets"], H, size=1.5, dtype=c["table"]), "len": None}
    if c["op"] == "decode" or c["mask"] == "key_padding":
        s["len"] = _lens(g, c)
    if c["op"] == "backward":  # what the forward has left
        s["do"] = randn(B, H, N, D)
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(B, H, N, device="cuda")
        step = max(1, 268435456 // (H * N * N))
        for b in range(0, B, step):
            at = slice(b, b + step)
            s["o"][at], s["lse"][at] = _forward(s["q"][at], s["k"][at], s["v"][at], s["table"],
                                                None if s["len"] is None else s["len"][at], c)
    return s


# ------------------------------------------------------------------ plain forms
def _bucket(d, c):
    """The bucket of each distance d = (key's position) - (query's position)."""
    per = c["buckets"] // 2 if c["both"] else c["buckets"]
    exact = per // 2
    n = d.abs() if c["both"] else (-d).clamp(min=0)
    # a distance on the border of two buckets belongs to the farther one
    far = torch.log(n.clamp(min=1).double() / exact) * ((per - exact) / math.log(c["reach"] / exact))
    far = (exact + torch.floor(far + 1e-9).long()).clamp(max=per - 1)
    u = torch.where(n < exact, n, far)
    return u + per * (d > 0) if c["both"] else u


def _scores(q, k, table, length, c, first=0):
    """[B, H, Nq, Nk] scores in 32 bits, -inf where a key is excluded; query r of sequence b is at
    position first[b] + r."""
    Nq, Nk = q.shape[2], k.shape[2]
    x = (q.float() @ k.float().transpose(2, 3)).mul_(_scale(c))
    j = torch.arange(Nk, device=q.device)
    i = torch.arange(Nq, device=q.device)[:, None]
    if c["op"] == "decode":
        i = i + first[:, None, None]                                   # [B, Nq, 1]
        x += table.float()[_bucket(j - i, c)].permute(0, 3, 1, 2)
        out = j >= length[:, None, None]
        if c["mask"] == "causal":
            out = out | (j > i)
        return x.masked_fill_(out[:, None], -math.inf)
    x += table.float()[_bucket(j - i, c)].permute(2, 0, 1)
    if c["mask"] == "causal":
        x.masked_fill_(j > i, -math.inf)
    elif c["mask"] == "key_padding":
        x.masked_fill_(j >= length[:, None, None, None], -math.inf)
    return x


def _forward(q, k, v, table, length, c, first=0):
    x = _scores(q, k, table, length, c, first)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p @ v.float()) / torch.where(total == 0, 1.0, total)
    lse = torch.where(total == 0, math.inf, top + torch.log(total))
    return out.to(q.dtype), lse[..., 0]


def _backward(s):
    c = s["case"]
    q, k, v, g = (s[n].float() for n in ("q", "k", "v", "do"))
    p = _scores(s["q"], s["k"], s["table"], s["len"], c).sub_(s["lse"][..., None]).exp_()
    dv = p.transpose(2, 3) @ g
    ds = (g @ v.transpose(2, 3)).sub_((g * s["o"].float()).sum(-1, keepdim=True)).mul_(p)
    del p
    dq = (ds @ k) * _scale(c)
    dk = (ds.transpose(2, 3) @ q) * _scale(c)
    # the sums over the diagonals j - i, then over the distances of each bucket
    H, N = c["H"], c["N"]
    d = ds.sum(0).flip(1)
    del ds
    d = torch.nn.functional.pad(d, (0, N)).view(H, -1)[:, :N * (2 * N - 1)].view(H, N, 2 * N - 1)
    d = d.sum(1, dtype=torch.float64)
    u = _bucket(torch.arange(1 - N, N, device=d.device), c)
    one = (u[:, None] == torch.arange(c["buckets"], device=d.device)).double()
    out = s["q"].dtype
    return {"dq": dq.to(out), "dk": dk.to(out), "dv": dv.to(out),
            "dtable": (d @ one).t().to(s["table"].dtype)}


# ------------------------------------------------------------------ one pass
def run(state):
    s = state
    c = s["case"]
    if own:
        import transformer_head_scaled_04_gb300 as mha

        how = dict(scale=_scale(c), max_distance=c["reach"], bidirectional=c["both"])
        if c["op"] == "forward":
            out, lse = mha.sdpa_rel_with_lse(s["q"], s["k"], s["v"], s["table"], c["mask"], s["len"],
                                             **how)
            return {"out": out, "lse": lse}
        if c["op"] == "backward":
            got = mha.sdpa_rel_backward(s["q"], s["k"], s["v"], s["table"], s["o"], s["do"],
                                        s["lse"], c["mask"], s["len"], **how)
            return dict(zip(("dq", "dk", "dv", "dtable"), got))
        return {"out": mha.sdpa_rel_decode(s["q"], s["k"], s["v"], s["table"], s["len"],
                                           causal=c["mask"] == "causal", **how)}
    if c["op"] == "forward":
        out, lse = _forward(s["q"], s["k"], s["v"], s["table"], s["len"], c)
        return {"out": out, "lse": lse}
    if c["op"] == "backward":
        return _backward(s)
    return {"out": _forward(s["q"], s["k"], s["v"], s["table"], s["len"], c,
                            s["len"].long() - c["Nq"])[0]}


def work(case):
    c = case
    B, H, N, Nq, D = c["B"], c["H"], c["N"], c["Nq"], c["D"]
    size = 2 if c["dtype"] == "bf16" else 4
    part = 0.5 if c["lens"] == "any" else 1.0 if c["lens"] == "full" else int(c["lens"]) / N
    if c["op"] == "decode":
        return {"bytes": B * H * D * size * (2 * N * part + 2 * Nq), "flops": 4 * D * B * H * Nq * N * part}
    pairs = B * H * N * N * part * (0.5 if c["mask"] == "causal" else 1.0)
    row = B * H * N * D * size
    if c["op"] == "forward":
        return {"bytes": (2 + 2 * part) * row, "flops": 4 * D * pairs}
    return {"bytes": (4 + 4 * part) * row, "flops": 10 * D * pairs}


# ------------------------------------------------------------------ the definition in 64 bits
def _edges(c):
    """For each bucket the interval of distances [low, high] that it holds (an empty one has low >
    high), from whole numbers alone: n belongs to bucket e + t or a later one when
    (n / e)^(per - e) >= (reach / e)^t."""
    per = c["buckets"] // 2 if c["both"] else c["buckets"]
    e, far = per // 2, 1 << 40
    first = list(range(e))
    for t in range(per - e):
        low, high = e, c["reach"]
        while low < high:
            n = (low + high) // 2
            if n ** (per - e) >= e ** (per - e - t) * c["reach"] ** t:
                high = n
            else:
                low = n + 1
        first.append(low)
    sides = [(first[u], first[u + 1] - 1 if u + 1 < per else far) for u in range(per)]
    if not c["both"]:
        return [(-b, -a if a else far) for a, b in sides]
    return [(-b, -a) for a, b in sides] + [(max(a, 1), b) for a, b in sides]


def exact(case, seed):
    c, s = case, prepare(case, seed)
    B, H, N, Nq = c["B"], c["H"], c["N"], c["Nq"]
    if B * H * N * Nq > 4e9:
        return None
    edges = _edges(c)
    table = s["table"].double()
    w = _scale(c)
    j = torch.arange(N, device="cuda")
    same, got = None, []
    total = torch.zeros(c["buckets"], H, dtype=torch.float64, device="cuda")
    for b in range(B):
        q, k, v = (s[n][b].double() for n in ("q", "k", "v"))
        length = N if s["len"] is None else int(s["len"][b])
        i = torch.arange(Nq, device="cuda")[:, None] + (length - Nq if c["op"] == "decode" else 0)
        if same is None or c["op"] == "decode":
            d = j - i
            low = torch.tensor([a for a, _ in edges], device="cuda")
            order = torch.argsort(low, stable=True)
            held = torch.tensor([a <= z for a, z in edges], device="cuda")
            order = order[held[order]]
            same = order[torch.searchsorted(low[order], d, right=True) - 1]
        x = torch.einsum("hid,hjd->hij", q, k) * w + table.t()[:, same]
        seen = (j < length).expand(Nq, N)
        if c["mask"] == "causal":
            seen = seen & (j <= i)
        x = torch.where(seen, x, -math.inf)
        if c["op"] == "backward":
            g, o, lse = s["do"][b].double(), s["o"][b].double(), s["lse"][b].double()
            p = torch.exp(x - lse[:, :, None])
            ds = p * (torch.einsum("hid,hjd->hij", g, v) - (g * o).sum(2)[:, :, None])
            got.append((torch.einsum("hij,hjd->hid", ds, k) * w,
                        torch.einsum("hij,hid->hjd", ds, q) * w,
                        torch.einsum("hij,hid->hjd", p, g)))
            flat = torch.stack([ds.diagonal(int(t), 1, 2).sum(-1) for t in range(1 - N, N)])
            total.index_add_(0, order[torch.searchsorted(low[order], torch.arange(
                1 - N, N, device="cuda"), right=True) - 1], flat)
        else:
            lse = torch.logsumexp(x, 2)
            p = torch.exp(x - torch.where(lse == -math.inf, 0.0, lse)[:, :, None])
            got.append((torch.einsum("hij,hjd->hid", p, v),
                        torch.where(lse == -math.inf, math.inf, lse)))
    if c["op"] == "backward":
        dq, dk, dv = (torch.stack(x) for x in zip(*got))
        return {"dq": dq, "dk": dk, "dv": dv, "dtable": total}
    out, lse = (torch.stack(x) for x in zip(*got))
    return {"out": out, "lse": lse} if c["op"] == "forward" else {"out": out}
