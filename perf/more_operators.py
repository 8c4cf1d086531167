"""What a batch of many requests needs beside the projections and the paged cache: the attention of prompts' rows over the cache
(scores capped by a tanh, a bias that grows with distance, prefix masks, windows), the same scores for one new token per sequence,
and the requests' low-rank adapters on a projection.

Sizes: the attention shape of this repository's benchmark (28 query and 4 key/value heads of 128 over P = 4 shards: 7 and 1 per
shard, d = 3584, prompts of 16384 rows), and generic ones around it.  A case's rows, lengths, prefixes and adapters per row follow
from the case alone; the seed gives the values, the order of the sequences and the pages they live in.
"""
import math

import torch

own = False

BF, F32 = torch.bfloat16, torch.float32


# ------------------------------------------------------------------ cases

def _prompt(name, **k):
    c = dict(op="prompt", P=1, M=1, B=1, Hq=8, Hkv=1, D=128, dtype="bf16", kv="same", cached=0, prefix=0, page=16, window=0, cap=0.0,
             slopes=False, pad=0)
    c.update(k)
    return dict(c, name=name) if name else c


def _decode(name, **k):
    c = dict(op="decode", P=1, B=1, Hq=8, Hkv=1, D=128, dtype="bf16", kv="same", shortest=1, longest=1, page=16, window=0, cap=0.0,
             slopes=False)
    c.update(k)
    return dict(c, name=name) if name else c


def _lora(name, **k):
    c = dict(op="lora", P=1, M=1, K=4096, N=4096, R=16, adapters=1, rowwise=False, dtype="bf16", pad=0)
    c.update(k)
    return dict(c, name=name) if name else c


def listed():
    return [
        # eight conversations, five proposed tokens each to be checked at once: latency
        _prompt("prompt_few", P=4, M=40, B=8, Hq=7, cached=3000, cap=50.0),
        # the benchmark's prompt, one sequence, capped scores
        _prompt("prompt_long", P=4, M=16384, Hq=7, page=64, cap=50.0),
        # pieces of nine prompts behind what is cached of them, a bias by distance, two padding rows
        _prompt("prompt_pieces", P=2, M=8190, B=9, Hq=16, Hkv=4, cached=5000, page=16, slopes=True, pad=2),
        # documents with a prefix that sees itself whole, on an E4M3 cache, heads of 80 under a window
        _prompt("prompt_prefix_e4m3", P=2, M=6001, B=4, Hq=20, Hkv=4, D=80, kv="e4m3", cached=777, prefix=30, page=32, window=2048),
        # fp32 heads of 64, capped
        _prompt("prompt_fp32", P=2, M=2500, B=3, Hq=8, Hkv=2, D=64, dtype="fp32", cached=500, page=48, cap=30.0),
        # one new token for each sequence of a serving batch, capped scores, an empty padding row among them
        _decode("decode_cap", P=4, B=64, Hq=7, shortest=64, longest=16384, cap=50.0),
        # a bias by distance on an E4M3 cache with four key/value heads a shard
        _decode("decode_slopes_e4m3", P=2, B=96, Hq=16, Hkv=4, shortest=16, longest=8000, page=32, kv="e4m3", slopes=True),
        # both, fp32, a few short conversations: latency
        _decode("decode_fp32_both", P=2, B=3, Hq=8, Hkv=2, D=64, dtype="fp32", shortest=200, longest=900, page=48, cap=30.0, slopes=True),
        # one new token for each of 61 requests with an adapter of their own on the QKV projection, three padding rows: latency
        _lora("lora_tokens", P=4, M=64, K=3584, N=4608, R=16, adapters=61, pad=3),
        # the rows of nine prompts, three adapters among them, on the QKV projection
        _lora("lora_prompts", P=4, M=16384, K=3584, N=4608, R=16, adapters=9),
        # the output projection, its rows split over the shards, adapters of rank 64
        _lora("lora_out", P=2, M=3001, K=4096, N=4096, R=64, adapters=5, rowwise=True, pad=1),
        # fp32
        _lora("lora_fp32", P=2, M=300, K=1000, N=2304, R=8, adapters=7, dtype="fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("prompt", "decode", "lora"))
    P = rng.choice((1, 2, 4))
    dtype = rng.choice(("bf16", "bf16", "bf16", "fp32"))
    if op == "lora":
        M = _log(rng, 1, 16384)
        return _lora(None, P=P, M=M, K=8 * P * _log(rng, 16, 4096 // (8 * P)), N=8 * P * _log(rng, 16, 4608 // (8 * P)),
                     R=rng.choice((8, 16, 16, 32, 64, 128)), adapters=min(M, _log(rng, 1, 96)), rowwise=rng.random() < 0.4,
                     dtype=dtype, pad=rng.choice((0, 0, min(M - 1, 3))))
    D = rng.choice((64, 80, 96, 128, 128, 128, 256))
    Hkv = rng.choice((1, 1, 2, 4))
    group = rng.choice((1, 2, 4, 5, 7, 8, 16))
    kv = "e4m3" if dtype == "bf16" and rng.random() < 0.35 else "same"
    page = 16 * rng.choice((1, 1, 2, 3, 4, 8))
    row = P * Hkv * 2 * D * (4 if dtype == "fp32" else 2)
    window = rng.choice((0, 0, 0, _log(rng, 1, 4096)))
    cap = rng.choice((0.0, 0.0, 20.0, 50.0))
    slopes = rng.random() < 0.4
    if op == "decode":
        cap = cap or (0.0 if slopes else 30.0)  # without either it is the decoding step that was there before
        longest = min(_log(rng, 1, 131072), (350 << 20) // row)
        # padded to the longest, at most 2^27 elements of k in all
        B = max(1, min(_log(rng, 1, 256), (1 << 27) // (P * Hkv * D * longest), (350 << 20) // (row * longest)))
        shortest = longest if B == 1 else max(1, longest // rng.choice((1, 2, 30, 256)))
        return _decode(None, P=P, B=B, Hq=Hkv * group, Hkv=Hkv, D=D, dtype=dtype, kv=kv, shortest=shortest, longest=longest, page=page,
                       window=window, cap=cap, slopes=slopes)
    M = _log(rng, 1, 16384)
    B = max(1, min(64, M // _log(rng, 1, 4096)))
    c = _prompt(None, P=P, M=M, B=B, Hq=Hkv * group, Hkv=Hkv, D=D, dtype=dtype, kv=kv, cached=rng.choice((0, _log(rng, 1, 16384))),
                prefix=rng.choice((0, 0, 0, 15, 60)), page=page, window=window, cap=cap, slopes=slopes, pad=rng.choice((0, 0, min(M - 1, 2))))
    # no more than the largest listed case costs
    while work(c)["flops"] > (1e12 if dtype == "bf16" else 3e10) or sum(n + k for n, k in _spans(c)) * row > 1 << 30:
        c["M"], c["cached"] = max(c["pad"] + 1, c["M"] // 2), c["cached"] // 2
        c["B"] = min(c["B"], c["M"])
    return c


# ------------------------------------------------------------------ what follows from a case alone

def _dt(c):
    return BF if c["dtype"] == "bf16" else F32


def _lengths(c):
    """Lengths of a decode case's sequences: spread over their logarithm; from 16 on the first is an empty padding row."""
    B, lo, hi = c["B"], c["shortest"], c["longest"]
    n = [int(round(lo * (hi / lo) ** ((i + 1) / B))) for i in range(B)]
    return [0] + n[1:] if B >= 16 else n


def _counts(n, B):
    """A spread of n rows over B sequences."""
    at = [n * i * (i + B) // (2 * B * B) for i in range(B + 1)]
    return [at[i + 1] - at[i] for i in range(B)]


def _spans(c):
    """(new rows, keys cached before them) of a prompt case's sequences."""
    B = c["B"]
    return [(n, c["cached"] * (7 * i % B + 1) // B) for i, n in enumerate(_counts(c["M"] - c["pad"], B))]


def _prefix(c, length):
    return length * c["prefix"] // 100


def _visible(c, n, cached):
    """Keys [lo, hi) that each of a sequence's n new rows sees, int64 [n] each."""
    pos = cached + torch.arange(n)
    lo = (pos + 1 - c["window"]).clamp(min=0) if c["window"] else torch.zeros_like(pos)
    hi = (pos + 1).clamp(min=_prefix(c, cached + n))
    return lo, hi


def _request_of_row(c):
    """The adapter of each row of a lora case, -1 for padding."""
    ids = [i for i, n in enumerate(_counts(c["M"] - c["pad"], c["adapters"])) for _ in range(n)]
    return ids + [-1] * c["pad"]


def work(case):
    c, es = case, 2 if case["dtype"] == "bf16" else 4
    if c["op"] == "lora":
        ids = _request_of_row(c)
        rows, used = len([i for i in ids if i >= 0]), len({i for i in ids if i >= 0})
        wide = c["P"] * c["N"] if c["rowwise"] else c["N"]  # outputs of a row, of all shards
        x = rows * c["K"]
        return {"bytes": es * (x + used * c["R"] * (c["K"] + c["N"]) + 2 * c["M"] * wide) + 4 * c["M"],
                "flops": 2 * rows * c["R"] * (c["K"] + wide)}
    es_kv, extra = (1, 4) if c["kv"] == "e4m3" else (es, 0)
    key = c["P"] * c["Hkv"] * 2 * (c["D"] * es_kv + extra)
    if c["op"] == "decode":
        rows, pairs = c["B"], sum(min(n, c["window"]) if c["window"] else n for n in _lengths(c))
        keys = pairs
    else:
        rows, pairs, keys = c["M"] - c["pad"], 0, 0
        for n, cached in _spans(c):
            lo, hi = _visible(c, n, cached)
            if n:
                pairs, keys = pairs + int((hi - lo).sum()), keys + int(hi.max() - lo.min())
    return {"bytes": keys * key + 2 * c["P"] * rows * c["Hq"] * c["D"] * es + 4 * c["P"] * rows * c["Hq"],
            "flops": 4 * pairs * c["P"] * c["Hq"] * c["D"]}


# ------------------------------------------------------------------ inputs

def _pages(lengths, page, g):
    """A page table for sequences of these lengths over a pool in random order, and the pool's size (three pages to spare)."""
    n = [max(1, -(-x // page)) for x in lengths]
    total = sum(n) + 3
    ids = torch.randperm(total, generator=g, device="cuda").int()
    at = torch.tensor([0] + n[:-1]).cumsum(0)
    col = torch.arange(max(n))
    own_page = col[None, :] < torch.tensor(n)[:, None]
    table = ids[torch.where(own_page, at[:, None] + col[None, :], torch.zeros(1, dtype=torch.int64)).cuda()]
    return torch.where(own_page.cuda(), table, torch.zeros_like(table)), total


def _codes(x):
    """E4M3 codes (as bytes) and power-of-two row scales of bf16 rows: the least e >= -126 with max |x| <= 448 2^e."""
    m, e = torch.frexp(x.float().abs().amax(-1))
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-126)
    e = torch.where(m == 0, torch.full_like(e, -126), e)
    s = torch.ldexp(torch.ones_like(m), e)
    return (x.float() / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8), s


def _new_cache(c, total, g):
    """A cache that has been in use: every slot holds finite values."""
    shape = (c["P"], total, c["Hkv"], c["page"], c["D"])
    k, v = (torch.randn(shape, generator=g, device="cuda", dtype=BF if c["kv"] == "e4m3" else _dt(c)) for _ in range(2))
    if c["kv"] != "e4m3":
        return k, v, None, None
    (k, ks), (v, vs) = _codes(k), _codes(v)
    return k, v, ks, vs


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c}
    randn = lambda *shape: torch.randn(shape, generator=g, device="cuda", dtype=_dt(c))  # noqa: E731
    if c["op"] == "lora":
        P, M, K, N, R, n = c["P"], c["M"], c["K"], c["N"], c["R"], c["adapters"]
        # the loaded adapters in the order they came, not the rows'
        order = torch.randperm(n, generator=g, device="cuda").int()
        ids = torch.tensor(_request_of_row(c), dtype=torch.int64).cuda()
        s["ids"] = torch.where(ids >= 0, order[ids.clamp(min=0)], torch.full_like(order[:1], -1)).int()
        s["x"] = randn(P, M, K // P) if c["rowwise"] else randn(M, K)
        s["A"], s["B"] = randn(n, R, K) * K ** -0.5, randn(n, N, R) * R ** -0.5
        s["gains"] = 0.25 + torch.rand(n, generator=g, device="cuda")
        s["base"] = randn(P, M, N if c["rowwise"] else N // P)
        s["out"] = torch.empty_like(s["base"])
    else:
        order = torch.randperm(c["B"], generator=g, device="cuda").tolist()
        if c["op"] == "decode":
            lengths = [_lengths(c)[i] for i in order]
            rows = c["B"]
        else:
            s["spans"] = [_spans(c)[i] for i in order]
            lengths = [n + cached for n, cached in s["spans"]]
            rows = c["M"]
            s["visible"] = [[t.cuda()[:, None] for t in _visible(c, n, cached)] for n, cached in s["spans"]]
            s["starts"] = torch.tensor([0] + [n for n, _ in s["spans"]]).cumsum(0).int().cuda()
            s["prefix"] = torch.tensor([_prefix(c, n) for n in lengths]).int().cuda() if c["prefix"] else None
        s["table"], total = _pages(lengths, c["page"], g)
        s["lens"] = torch.tensor(lengths).int().cuda()
        s["cache"] = _new_cache(c, total, g)
        # scaled so that the weights of a long row are neither flat nor one key's alone, and that a cap is felt
        s["q"] = randn(c["P"], rows, c["Hq"], c["D"]) * (6.0 if c["cap"] else 1.5)
        s["scale"] = c["D"] ** -0.5
        # the usual geometric slopes over all shards' heads
        H = c["P"] * c["Hq"]
        s["slopes"] = (2.0 ** (-8.0 * torch.arange(1, H + 1) / H)).view(c["P"], c["Hq"]).cuda() if c["slopes"] else None
        s["out"] = torch.zeros(c["P"], rows, c["Hq"] * c["D"], dtype=_dt(c), device="cuda")
        s["lse"] = torch.zeros(c["P"], rows, c["Hq"], device="cuda")
    if own:
        _keep(s, c)
    return s


def _keep(s, c):
    """What a program that uses the framework keeps beside these: the workspace."""
    import sequence_tensor_transformer_gb300 as st

    if c["op"] == "lora":
        n = st.sptp_lora_workspace_size(c["P"], c["M"], c["K"], c["N"], c["R"], c["rowwise"])
    elif c["op"] == "decode":
        n = st.sptp_paged_attn_workspace_size(c["P"], c["B"], c["Hq"], c["Hkv"], c["D"])
    else:
        n = st.sptp_paged_attn_prompt_workspace_size(c["P"], c["M"], c["B"], c["Hq"], c["Hkv"], c["D"])
    s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------ one pass

def _gather(pool, scale, table):
    """The pool's rows of every sequence, in order, in 32 bits: [P, B, Hkv, length, D]."""
    x = pool[:, table]
    if scale is not None:
        x = x.view(torch.float8_e4m3fn).float() * scale[:, table][..., None]
    x = x.float()
    P, B, n, H, page, D = x.shape
    return x.transpose(2, 3).reshape(P, B, H, n * page, D)


def _weigh(scores, c, slopes, pos, lo, hi):
    """Scores (scaled) [..., rows, keys] to weights and their logarithmic sum; pos, lo, hi [..., rows, 1]: positions and visible keys."""
    at = torch.arange(scores.shape[-1], device="cuda")
    if c["cap"]:
        scores = c["cap"] * torch.tanh(scores / c["cap"])
    if slopes is not None:
        scores = scores - slopes * (pos - at).abs().float()
    scores = scores.masked_fill((at < lo) | (at >= hi), -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=torch.finfo(F32).min)
    w = torch.exp(scores - top)
    total = w.sum(-1, keepdim=True)
    lse = torch.where(total > 0, top + total.log(), torch.full_like(top, -math.inf))
    return w / total.clamp(min=1e-38), lse[..., 0]


def _plain_decode(s, c):
    k, v, ks, vs = s["cache"]
    table, lens = s["table"].long(), s["lens"].long()
    q = s["q"].float().view(c["P"], c["B"], c["Hkv"], -1, c["D"])
    scores = q @ _gather(k, ks, table).transpose(-1, -2) * s["scale"]
    hi = lens[None, :, None, None, None]
    lo = (hi - c["window"]).clamp(min=0) if c["window"] else torch.zeros_like(hi)
    slopes = None if s["slopes"] is None else s["slopes"].view(c["P"], 1, c["Hkv"], -1, 1)
    w, lse = _weigh(scores, c, slopes, hi - 1, lo, hi)
    o = w @ _gather(v, vs, table)
    return o.to(s["q"].dtype).reshape(c["P"], c["B"], -1), lse.reshape(c["P"], c["B"], -1)


def _plain_prompt(s, c):
    P, Hq, Hkv, D = c["P"], c["Hq"], c["Hkv"], c["D"]
    k, v, ks, vs = s["cache"]
    out, lse, row = s["out"], s["lse"], 0
    for b, (n, cached) in enumerate(s["spans"]):
        if n == 0:
            continue
        length = n + cached
        table = s["table"][b: b + 1, : -(-length // c["page"])].long()
        K, V = _gather(k, ks, table)[:, 0, :, None, :length], _gather(v, vs, table)[:, 0, :, None, :length]  # [P, Hkv, 1, keys, D]
        q = s["q"][:, row: row + n].float().view(P, n, Hkv, -1, D).permute(0, 2, 3, 1, 4)                   # [P, Hkv, group, n, D]
        lo, hi = s["visible"][b]
        pos = cached + torch.arange(n, device="cuda")[:, None]
        slopes = torch.zeros(P, Hkv, Hq // Hkv, 1, 1, device="cuda") if s["slopes"] is None else s["slopes"].view(P, Hkv, -1, 1, 1)
        # all heads at once, or one after another where their scores would take gigabytes
        if P * Hq * n * length <= 1 << 28:
            w, z = _weigh(q @ K.transpose(-1, -2) * s["scale"], c, slopes if c["slopes"] else None, pos, lo, hi)
            o = w @ V
        else:
            o, z = torch.empty_like(q), torch.empty(q.shape[:-1], device="cuda")
            for p in range(P):
                for h in range(Hkv):
                    for i in range(Hq // Hkv):
                        w, z[p, h, i] = _weigh(q[p, h, i] @ K[p, h, 0].T * s["scale"], c, slopes[p, h, i] if c["slopes"] else None, pos,
                                               lo, hi)
                        o[p, h, i] = w @ V[p, h, 0]
        out[:, row: row + n] = o.permute(0, 3, 1, 2, 4).reshape(P, n, Hq * D).to(out.dtype)
        lse[:, row: row + n] = z.permute(0, 3, 1, 2).reshape(P, n, Hq)
        row += n
    return out, lse


def _plain_lora(s, c):
    P, M, N, R, n = c["P"], c["M"], c["N"], c["R"], c["adapters"]
    ids = s["ids"].long()
    # every adapter's product with every row, those that are not a row's own cleared
    chosen = (ids[:, None] == torch.arange(n, device="cuda")[None, :]) * s["gains"]                        # [M, n]
    up = s["B"].float().transpose(1, 2).reshape(n * R, N)
    x = s["x"].float()
    if c["rowwise"]:
        down = s["A"].float().view(n * R, P, -1).permute(1, 2, 0)                                          # [P, K/P, n R]
        t = (x @ down).view(P, M, n, R) * chosen[None, :, :, None]
        delta = t.reshape(P, M, n * R) @ up
    else:
        t = (x @ s["A"].float().view(n * R, -1).T).view(M, n, R) * chosen[:, :, None]
        delta = (t.reshape(M, n * R) @ up).view(M, P, N // P).transpose(0, 1)
    return (s["base"].float() + delta).to(s["base"].dtype)


def run(state):
    s, c = state, state["case"]
    if own:
        import sequence_tensor_transformer_gb300 as st

        if c["op"] == "lora":
            return st.sptp_lora(s["x"], s["A"], s["B"], s["ids"], s["base"], gains=s["gains"], out=s["out"], workspace=s["ws"])
        if c["op"] == "decode":
            out, lse = st.sptp_paged_attn_decode(s["q"], s["cache"], s["table"], s["lens"], s["scale"], c["window"], out=s["out"],
                                                 lse=s["lse"], workspace=s["ws"], cap=c["cap"], slopes=s["slopes"])
        else:
            out, lse = st.sptp_paged_attn_prompt(s["q"], s["cache"], s["table"], s["lens"], s["starts"], s["scale"], c["window"],
                                                 cap=c["cap"], slopes=s["slopes"], prefix_lens=s["prefix"], out=s["out"], lse=s["lse"],
                                                 workspace=s["ws"])
    elif c["op"] == "lora":
        return _plain_lora(s, c)
    else:
        out, lse = (_plain_decode if c["op"] == "decode" else _plain_prompt)(s, c)
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------ the definition, in 64 bits

def exact(case, seed):
    c = case
    if work(c)["flops"] > 4e12:  # about 20 seconds
        return None
    s = prepare(case, seed)
    if c["op"] == "lora":
        y = s["base"].double()
        for a, gain in enumerate(s["gains"].tolist()):
            rows = (s["ids"] == a).nonzero()[:, 0]
            for p in range(c["P"]):
                if c["rowwise"]:
                    k = c["K"] // c["P"]
                    t = torch.einsum("mk,rk->mr", s["x"][p, rows].double(), s["A"][a, :, p * k: (p + 1) * k].double())
                    up = s["B"][a].double()
                else:
                    n = c["N"] // c["P"]
                    t = torch.einsum("mk,rk->mr", s["x"][rows].double(), s["A"][a].double())
                    up = s["B"][a, p * n: (p + 1) * n].double()
                y[p, rows] += gain * torch.einsum("mr,nr->mn", t, up)
        return y
    k, v, ks, vs = s["cache"]
    table, group = s["table"].long(), c["Hq"] // c["Hkv"]
    as64 = lambda t: (t.view(torch.float8_e4m3fn) if t.dtype == torch.uint8 else t).double()  # noqa: E731
    out, lse = s["out"].double().view(*s["q"].shape), s["lse"].double()
    spans = [(1 if n else 0, n - 1) for n in s["lens"].tolist()] if c["op"] == "decode" else s["spans"]
    row = 0
    for b, (n, cached) in enumerate(spans):
        first = b if c["op"] == "decode" else row
        row += n
        if n == 0 and c["op"] == "decode":
            out[:, b], lse[:, b] = 0, -math.inf
        for p in range(c["P"] if n else 0):
            at = torch.arange(n + cached, device="cuda")
            page, off = table[b, at // c["page"]], at % c["page"]
            K, V = as64(k[p][page, :, off]), as64(v[p][page, :, off])  # [keys, Hkv, D]
            if ks is not None:
                K, V = K * ks[p][page, :, off].double()[..., None], V * vs[p][page, :, off].double()[..., None]
            for r0 in range(0, n, 1024):
                r1 = min(n, r0 + 1024)
                pos = cached + torch.arange(r0, r1, device="cuda")
                end = pos + 1
                if c["op"] == "prompt" and c["prefix"]:
                    end = torch.maximum(end, torch.tensor((n + cached) * c["prefix"] // 100, device="cuda"))
                j0 = max(0, cached + r0 + 1 - c["window"]) if c["window"] else 0
                j1 = int(end.max())
                j = torch.arange(j0, j1, device="cuda")
                seen = j[None, :] < end[:, None]
                if c["window"]:
                    seen &= j[None, :] > pos[:, None] - c["window"]
                for h in range(c["Hq"]):
                    z = s["q"][p, first + r0: first + r1, h].double() @ K[j0:j1, h // group].T * s["scale"]
                    if c["cap"]:
                        z = torch.tanh(z / c["cap"]) * c["cap"]
                    if c["slopes"]:
                        z = z - float(s["slopes"][p, h]) * (pos[:, None] - j[None, :]).abs()
                    z = torch.where(seen, z, -math.inf)
                    l = torch.logsumexp(z, -1)
                    lse[p, first + r0: first + r1, h] = l
                    out[p, first + r0: first + r1, h] = torch.exp(z - l[:, None]) @ V[j0:j1, h // group]
    return {"out": out.reshape(*s["out"].shape), "lse": lse}
