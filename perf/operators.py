"""The attention operators between the QKV projection and the output projection: rotary positions, the rotation with the
append to a paged key-value cache, and the attention of one new token per sequence over that cache.

Sizes: the attention shape of this repository's benchmark (28 query and 4 key/value heads of 128 over P = 4 shards: 7 and 1 per
shard, prompts of 16384 rows), and generic ones around it.  A case's row counts and sequence lengths follow from the case alone
(a spread over their logarithm); the seed gives the values, the order of the sequences and the pages they live in.
"""
import math

import torch

own = False

BF, F32 = torch.bfloat16, torch.float32


# ------------------------------------------------------------------ cases

def _rope(name, **k):
    c = dict(op="rope", P=1, M=1, H=9, Hr=8, D=128, rot=128, inter=False, grad=False, dtype="bf16", far=4096, scaling="none",
             factor=1.0, gain=1.0)
    c.update(k)
    return dict(c, name=name) if name else c


def _append(name, **k):
    c = dict(op="append", P=1, M=1, Hq=8, Hkv=1, D=128, rot=128, inter=False, dtype="bf16", kv="same", B=1, far=4096, page=16,
             pad=0)
    c.update(k)
    return dict(c, name=name) if name else c


def _decode(name, **k):
    c = dict(op="decode", P=1, B=1, Hq=8, Hkv=1, D=128, dtype="bf16", kv="same", shortest=1, longest=1, page=16, window=0)
    c.update(k)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one new token: latency
        _rope("rope_token", P=4, M=1, far=32768),
        # the benchmark's prompt, every shard's q and k heads rotated, the v head copied through
        _rope("rope_prompt", P=4, M=16384, far=16384),
        # the gradient of an interleaved rotation of a part of odd-sized heads
        _rope("rope_grad_part", P=2, M=4097, H=20, Hr=16, D=80, rot=32, inter=True, grad=True, gain=1.0),
        # fp32, positions past a million, frequencies scaled by parts, with its gain
        _rope("rope_fp32_far", P=2, M=2500, H=24, Hr=20, D=64, rot=64, dtype="fp32", far=1 << 20, scaling="parts", factor=32.0,
              gain=1.3465735902799727),
        # one new token for each of 61 sequences in a batch padded to 64
        _append("append_tokens", P=4, M=64, Hq=7, B=61, far=4096, pad=3),
        # chunks of nine prompts, 16384 rows together
        _append("append_prompt", P=4, M=16384, Hq=7, B=9, far=8192, page=64),
        # the same into an E4M3 cache, four key/value heads a shard
        _append("append_e4m3", P=2, M=3001, Hq=16, Hkv=4, B=5, far=2000, page=32, kv="e4m3", pad=1),
        # one short conversation: latency
        _decode("decode_short", P=4, B=1, Hq=7, shortest=333, longest=333),
        # one long document: the length has to be split
        _decode("decode_long", P=4, B=1, Hq=7, shortest=131071, longest=131071, page=64),
        # a serving batch of mixed lengths, an empty padding row among them
        _decode("decode_batch", P=4, B=64, Hq=7, shortest=64, longest=16384, page=16),
        # the same kind of batch on an E4M3 cache with four key/value heads a shard
        _decode("decode_e4m3", P=2, B=96, Hq=16, Hkv=4, shortest=16, longest=8000, page=32, kv="e4m3"),
        # fp32, a sliding window, heads of 64
        _decode("decode_fp32_window", P=2, B=24, Hq=8, Hkv=2, D=64, dtype="fp32", shortest=100, longest=6000, page=48,
                window=2048),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "append", "decode"))
    P = rng.choice((1, 2, 4))
    D = rng.choice((64, 80, 96, 128, 128, 128, 256))
    Hkv = rng.choice((1, 1, 2, 4))
    group = rng.choice((1, 2, 4, 5, 7, 8, 16))
    dtype = rng.choice(("bf16", "bf16", "bf16", "fp32"))
    if op == "decode":
        kv = "e4m3" if dtype == "bf16" and rng.random() < 0.4 else "same"
        page = 16 * rng.choice((1, 1, 2, 3, 4, 8))
        longest = _log(rng, 1, 131072)
        row = P * Hkv * 2 * D * (4 if dtype == "fp32" else 2)
        longest = min(longest, (350 << 20) // row)
        # padded to the longest, at most 2^27 elements of k in all
        B = max(1, min(_log(rng, 1, 256), (1 << 27) // (P * Hkv * D * longest), (350 << 20) // (row * longest)))
        shortest = longest if B == 1 else max(1, longest // rng.choice((1, 2, 30, 256)))
        return _decode(None, P=P, B=B, Hq=Hkv * group, Hkv=Hkv, D=D, dtype=dtype, kv=kv, shortest=shortest, longest=longest, page=page,
                       window=rng.choice((0, 0, 0, _log(rng, 1, 4096))))
    rot = rng.choice((D, D, D // 2 // 16 * 16))
    most = (140 << 20) // (P * D * (4 if dtype == "fp32" else 2) * (group + 2) * Hkv)
    M = _log(rng, 1, min(16384, most))
    inter = rng.random() < 0.4
    far = _log(rng, 1024, 1 << 20 if op == "rope" else 16384)
    B = max(1, M // _log(rng, 1, 4096))
    if op == "append":  # at most 2^27 elements of k in the pool
        far = max(1, min(far, (1 << 27) // (P * Hkv * D * B)))
    if op == "rope":
        scaling = rng.choice(("none", "none", "linear", "ntk", "parts"))
        return _rope(None, P=P, M=M, H=(group + 2) * Hkv, Hr=(group + 1) * Hkv, D=D, rot=rot, inter=inter, grad=rng.random() < 0.4,
                     dtype=dtype, far=far, scaling=scaling, factor=1.0 if scaling == "none" else rng.choice((2.0, 8.0, 40.0)))
    return _append(None, P=P, M=M, Hq=group * Hkv, Hkv=Hkv, D=D, rot=rot, inter=inter, dtype=dtype,
                   kv="e4m3" if dtype == "bf16" and rng.random() < 0.4 else "same", B=B, far=far,
                   page=16 * rng.choice((1, 1, 2, 3, 4, 8)), pad=rng.choice((0, 0, min(M - 1, 2))))


# ------------------------------------------------------------------ what follows from a case alone

def _dt(c):
    return BF if c["dtype"] == "bf16" else F32


def _lengths(c):
    """Lengths of a decode case's sequences: spread over their logarithm; from 16 on the first is an empty padding row."""
    B, lo, hi = c["B"], c["shortest"], c["longest"]
    n = [int(round(lo * (hi / lo) ** ((i + 1) / B))) for i in range(B)]
    return [0] + n[1:] if B >= 16 else n


def _counts(c):
    """New rows of an append case's sequences: a spread of shares, together M - pad."""
    B, n = c["B"], c["M"] - c["pad"]
    at = [n * i * (i + B) // (2 * B * B) for i in range(B + 1)]
    return [at[i + 1] - at[i] for i in range(B)]


def _read(c):
    """Cache rows that a decode case has to read, per shard and key/value head."""
    return sum(min(n, c["window"]) if c["window"] else n for n in _lengths(c))


def _frequencies(c):
    """Angles a position, in radians, float64."""
    rot, theta, s = c["rot"], 1e4, c.get("factor", 1.0)
    f = theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    kind = c.get("scaling", "none")
    if kind == "linear":
        f = f / s
    elif kind == "ntk":
        f = (theta * s ** (rot / (rot - 2))) ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    elif kind == "parts":  # over an original length of 4096: below 1 turn scaled, above 32 turns kept, between them blended
        keep = ((4096 * f / (2 * math.pi) - 1.0) / 31.0).clamp(0, 1)
        f = keep * f + (1 - keep) * f / s
    return f


def work(case):
    c, es = case, 2 if case["dtype"] == "bf16" else 4
    if c["op"] == "rope":
        n = c["P"] * c["M"] * c["H"] * c["D"]
        return {"bytes": 2 * n * es + 4 * c["M"], "flops": 3 * c["P"] * c["M"] * c["Hr"] * c["rot"]}
    es_kv, extra = (1, 4) if c["kv"] == "e4m3" else (es, 0)
    if c["op"] == "append":
        rows = c["P"] * (c["M"] - c["pad"])
        q, kv = c["Hq"] * c["D"], c["Hkv"] * c["D"]
        return {"bytes": rows * ((q + 2 * kv) * es + q * es + 2 * (kv * es_kv + c["Hkv"] * extra)) + 12 * c["M"],
                "flops": 3 * rows * (c["Hq"] + c["Hkv"]) * c["rot"]}
    keys = _read(c)
    return {"bytes": keys * c["P"] * c["Hkv"] * 2 * (c["D"] * es_kv + extra) + 2 * c["P"] * c["B"] * c["Hq"] * c["D"] * es
            + 4 * c["P"] * c["B"] * c["Hq"],
            "flops": 4 * keys * c["P"] * c["Hq"] * c["D"]}


# ------------------------------------------------------------------ inputs

def _pages(lengths, page, g, total=None):
    """A page table for sequences of these lengths over a pool in random order, and the pool's size (three pages to spare, or as given)."""
    n = [max(1, -(-x // page)) for x in lengths]
    total = total or sum(n) + 3
    ids = torch.randperm(total, generator=g, device="cuda").int()
    at = torch.tensor([0] + n[:-1]).cumsum(0)
    col = torch.arange(max(n))
    own_page = col[None, :] < torch.tensor(n)[:, None]
    table = ids[torch.where(own_page, at[:, None] + col[None, :], torch.zeros(1, dtype=torch.int64)).cuda()]
    return torch.where(own_page.cuda(), table, torch.zeros_like(table)), total


def _codes(x):
    """E4M3 codes (as bytes) and power-of-two row scales of finished bf16 rows: the least e >= -126 with max |x| <= 448 2^e."""
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
    if c["op"] == "decode":
        order = torch.randperm(c["B"], generator=g, device="cuda")
        lengths = torch.tensor(_lengths(c))[order.cpu()]
        s["table"], total = _pages(lengths.tolist(), c["page"], g)
        s["lens"] = lengths.int().cuda()
        s["cache"] = _new_cache(c, total, g)
        # scaled so that the weights of a long row are neither flat nor one key's alone
        s["q"] = randn(c["P"], c["B"], c["Hq"], c["D"]) * 1.5
        s["scale"] = c["D"] ** -0.5
        s["out"] = torch.empty(c["P"], c["B"], c["Hq"] * c["D"], dtype=_dt(c), device="cuda")
        s["lse"] = torch.empty(c["P"], c["B"], c["Hq"], device="cuda")
    else:
        s["freq"] = _frequencies(c).cuda()
        if c["op"] == "rope":
            s["x"] = randn(c["P"], c["M"], c["H"], c["D"])
            s["pos"] = torch.randint(0, c["far"], (c["M"],), generator=g, device="cuda", dtype=torch.int32)
            s["out"] = torch.empty_like(s["x"])
        else:
            counts = torch.tensor(_counts(c))
            start = torch.randint(0, c["far"], (c["B"],), generator=g, device="cuda").cpu()
            seq = torch.repeat_interleave(torch.arange(c["B"]), counts)
            first = counts.cumsum(0) - counts
            n = seq.numel()
            pos = start[seq] + torch.arange(n) - first[seq]
            # a pool that holds every sequence at its longest
            s["table"], total = _pages((start + counts).tolist(), c["page"], g, sum(-(-(c["far"] + k) // c["page"]) for k in counts.tolist()))
            fill = torch.full((c["pad"],), -1)
            s["seq"], s["pos"] = torch.cat([seq, fill]).int().cuda(), torch.cat([pos, fill + 1]).int().cuda()
            s["rows"] = n  # the rows behind are padding
            s["qkv"] = randn(c["P"], c["M"], (c["Hq"] + 2 * c["Hkv"]) * c["D"])
            s["cache"] = _new_cache(c, total, g)
            s["q"] = torch.zeros(c["P"], c["M"], c["Hq"], c["D"], dtype=_dt(c), device="cuda")
    if own:
        _keep(s, c)
    return s


def _keep(s, c):
    """What a program that uses the framework keeps beside these: the rotation's table and the workspaces."""
    import sequence_tensor_transformer_gb300 as st

    if "freq" in s and c["rot"]:
        s["turns"] = st.sptp_rope_turns(c["rot"], 1e4, c.get("scaling", "none"), c.get("factor", 1.0), 4096)
    if c["op"] != "rope":
        n = st.SPTP_WS_HEADER_BYTES
        if c["op"] == "decode":
            n = st.sptp_paged_attn_workspace_size(c["P"], c["B"], c["Hq"], c["Hkv"], c["D"])
        s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------ one pass

def _turn(x, pos, freq, inter, grad, gain):
    """Rotates the first 2 * len(freq) elements of the last axis of x [P, M, heads, D] in 32 bits; angles in 64."""
    n = freq.numel()
    if n == 0:
        return x.float()
    a = pos.double()[:, None] * freq[None, :]
    cos, sin = (gain * a.cos()).float()[:, None, :], (gain * a.sin()).float()[:, None, :]
    if grad:
        sin = -sin
    x = x.float()
    part, rest = x[..., : 2 * n], x[..., 2 * n:]
    u, w = (part[..., 0::2], part[..., 1::2]) if inter else (part[..., :n], part[..., n:])
    y, z = u * cos - w * sin, u * sin + w * cos
    part = torch.stack((y, z), -1).flatten(-2) if inter else torch.cat((y, z), -1)
    return torch.cat((part, rest), -1)


def _plain_rope(s, c):
    x, hr = s["x"], c["Hr"]
    y = _turn(x[:, :, :hr], s["pos"], s["freq"], c["inter"], c["grad"], c["gain"]).to(x.dtype)
    return torch.cat((y, x[:, :, hr:]), 2)


def _plain_append(s, c):
    P, M, Hq, Hkv, D, n = c["P"], c["M"], c["Hq"], c["Hkv"], c["D"], s["rows"]
    x = s["qkv"].view(P, M, Hq + 2 * Hkv, D)[:, :n]
    y = _turn(x[:, :, : Hq + Hkv], s["pos"][:n], s["freq"], c["inter"], False, 1.0).to(x.dtype)
    s["q"][:, :n] = y[:, :, :Hq]
    k, v, ks, vs = s["cache"]
    pos = s["pos"][:n].long()
    pages, at = s["table"][s["seq"][:n].long(), pos // c["page"]].long(), pos % c["page"]
    new_k, new_v = y[:, :, Hq:], x[:, :, Hq + Hkv:]
    if ks is not None:
        (new_k, new_ks), (new_v, new_vs) = _codes(new_k), _codes(new_v)
        ks[:, pages, :, at], vs[:, pages, :, at] = new_ks.transpose(0, 1), new_vs.transpose(0, 1)
    k[:, pages, :, at], v[:, pages, :, at] = new_k.transpose(0, 1), new_v.transpose(0, 1)


def _gather(pool, scale, table):
    """The pool's rows of every sequence, in order, in 32 bits: [P, B, Hkv, length, D]."""
    x = pool[:, table]
    if scale is not None:
        x = x.view(torch.float8_e4m3fn).float() * scale[:, table][..., None]
    x = x.float()
    P, B, n, H, page, D = x.shape
    return x.transpose(2, 3).reshape(P, B, H, n * page, D)


def _plain_decode(s, c):
    k, v, ks, vs = s["cache"]
    table, lens = s["table"].long(), s["lens"][:, None]
    q = s["q"].float().view(c["P"], c["B"], c["Hkv"], -1, c["D"])
    scores = q @ _gather(k, ks, table).transpose(-1, -2) * s["scale"]
    at = torch.arange(scores.shape[-1], device="cuda")[None, :]
    seen = at < lens
    if c["window"]:
        seen &= at >= lens - c["window"]
    scores = scores.masked_fill(~seen[None, :, None, None, :], -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=torch.finfo(F32).min)
    w = torch.exp(scores - top)
    total = w.sum(-1, keepdim=True)
    o = (w @ _gather(v, vs, table)) / total.clamp(min=1e-38)
    lse = torch.where(total > 0, top + total.log(), torch.full_like(top, -math.inf))
    return o.to(s["q"].dtype).reshape(c["P"], c["B"], -1), lse.reshape(c["P"], c["B"], -1)


def run(state):
    s, c = state, state["case"]
    if own:
        import sequence_tensor_transformer_gb300 as st

        if c["op"] == "rope":
            return st.sptp_rope(s["x"], s["pos"], s.get("turns"), c["Hr"], interleaved=c["inter"], transpose=c["grad"],
                                gain=c["gain"], out=s["out"])
        if c["op"] == "decode":
            out, lse = st.sptp_paged_attn_decode(s["q"], s["cache"], s["table"], s["lens"], s["scale"], c["window"], out=s["out"],
                                                 lse=s["lse"], workspace=s["ws"])
            return {"out": out, "lse": lse}
        st.sptp_rope_append_kv(s["qkv"], s["pos"], s["seq"], s["table"], s.get("turns"), s["cache"], c["Hq"],
                               interleaved=c["inter"], q_out=s["q"], workspace=s["ws"])
    elif c["op"] == "rope":
        return _plain_rope(s, c)
    elif c["op"] == "decode":
        out, lse = _plain_decode(s, c)
        return {"out": out, "lse": lse}
    else:
        _plain_append(s, c)
    k, v, ks, vs = s["cache"]
    if ks is None:
        return {"q": s["q"], "k": k, "v": v}
    # the codes as the numbers they stand for, beside their rows' scales
    return {"q": s["q"], "k": k.view(torch.float8_e4m3fn), "v": v.view(torch.float8_e4m3fn), "k_scale": ks, "v_scale": vs}


# ------------------------------------------------------------------ the definition, in 64 bits

def _rotate64(x, pos, freq, inter, sign, gain):
    """x [..., D] with its pairs as complex numbers, times gain * exp(i * sign * pos * f)."""
    n = freq.numel()
    y = x.double().clone()
    if n == 0:
        return y
    turn = torch.polar(torch.full((pos.numel(), n), float(gain), dtype=torch.float64, device=x.device),
                       sign * pos.double().outer(freq))[:, None, :]
    re, im = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if inter else (slice(0, n), slice(n, 2 * n))
    z = torch.complex(y[..., re], y[..., im]) * turn
    y[..., re], y[..., im] = z.real, z.imag
    return y


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "rope":
        y = s["x"].double()
        for p in range(c["P"]):
            y[p, :, : c["Hr"]] = _rotate64(s["x"][p, :, : c["Hr"]], s["pos"], s["freq"], c["inter"], -1.0 if c["grad"] else 1.0, c["gain"])
        return y
    k, v, ks, vs = s["cache"]
    table = s["table"].long()
    as64 = lambda t: (t.view(torch.float8_e4m3fn) if t.dtype == torch.uint8 else t).double()  # noqa: E731
    if c["op"] == "append":
        q, k64, v64 = s["q"].double(), as64(k), as64(v)
        n, page, Hq, Hkv = s["rows"], c["page"], c["Hq"], c["Hkv"]
        pos, seq = s["pos"][:n].long(), s["seq"][:n].long()
        slot = table[seq, pos // page] * page + pos % page
        for p in range(c["P"]):
            x = s["qkv"][p, :n].view(n, Hq + 2 * Hkv, c["D"])
            q[p, :n] = _rotate64(x[:, :Hq], pos, s["freq"], c["inter"], 1.0, 1.0)
            for h in range(Hkv):
                for rows, pool, scales in ((_rotate64(x[:, Hq + h: Hq + h + 1], pos, s["freq"], c["inter"], 1.0, 1.0)[:, 0], k64, ks),
                                           (x[:, Hq + Hkv + h].double(), v64, vs)):
                    if scales is not None:  # the scale is that of the row's bf16 values
                        top = rows.to(BF).double().abs().amax(-1)
                        e = torch.ceil(torch.log2(top / 448)).clamp(min=-126)
                        rows = rows / 2.0 ** e[:, None]
                        scales[p].select(1, h)[slot // page, slot % page] = (2.0 ** e).float()
                    pool[p].select(1, h)[slot // page, slot % page] = rows
        if ks is None:
            return {"q": q, "k": k64, "v": v64}
        return {"q": q, "k": k64, "v": v64, "k_scale": ks.double(), "v_scale": vs.double()}
    out = torch.zeros(c["P"], c["B"], c["Hq"], c["D"], dtype=torch.float64, device="cuda")
    lse = torch.full((c["P"], c["B"], c["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
    group = c["Hq"] // c["Hkv"]
    for b, n in enumerate(s["lens"].tolist()):
        first = max(0, n - c["window"]) if c["window"] else 0
        if first >= n:
            continue
        at = torch.arange(first, n, device="cuda")
        page, off = table[b, at // c["page"]], at % c["page"]
        for p in range(c["P"]):
            K, V = as64(k[p][page, :, off]), as64(v[p][page, :, off])  # [keys, Hkv, D]
            if ks is not None:
                K, V = K * ks[p][page, :, off].double()[..., None], V * vs[p][page, :, off].double()[..., None]
            q = s["q"][p, b].double().view(c["Hkv"], group, c["D"])
            z = torch.einsum("hgd,nhd->hgn", q, K) * s["scale"]
            l = torch.logsumexp(z, -1)
            lse[p, b] = l.reshape(-1)
            out[p, b] = torch.einsum("hgn,nhd->hgd", torch.exp(z - l[..., None]), V).reshape(c["Hq"], c["D"])
    return {"out": out.reshape(c["P"], c["B"], -1), "lse": lse}
