"""Prompts' attention in 64 bits by torch, for sizes that the oracle's loops over rows are
too slow for, and the comparison with it (bounds: batch_cases.check)."""
import torch

from batch_cases import HALF, score_error


def on_gpu(a):
    return torch.from_numpy(a).cuda()


def modified(z, cap, slope, far):
    if cap:
        z = cap * torch.tanh(z / cap)
    return z - slope * far


def reference(c, rows_at_once=1024):
    """Yields (p, h, first row, out, lse, mean of |v|, (dots, far, keys)) as
    attn_oracle.paged_attn_prompt has them, a run of one sequence's rows at a time."""
    table = torch.from_numpy(c["table"]).cuda()
    for b, (n, length) in enumerate(zip(c["rows"].tolist(), c["lens"])):
        at = torch.arange(length, device="cuda")
        pages, off = table[b][at // c["page"]], at % c["page"]
        prefix = 0 if c["prefix"] is None else min(max(int(c["prefix"][b]), 0), length)
        for p in range(c["P"]):
            for h in range(c["Hq"]):
                kv = h * c["Hkv"] // c["Hq"]
                K, V = (on_gpu(c[x][p, :, kv])[pages, off] for x in ("k64", "v64"))
                slope = 0.0 if c["slopes"] is None else float(c["slopes"][p, h])
                for r0 in range(0, n, rows_at_once):
                    r = torch.arange(r0, min(n, r0 + rows_at_once), device="cuda")
                    pos = (length - n + r)[:, None]
                    seen = (at < torch.clamp(pos + 1, min=prefix)) & (pos >= 0)
                    if c["window"]:
                        seen &= at > pos - c["window"]
                    m = int(c["starts"][b]) + r0
                    q = on_gpu(c["q64"][p, m: m + len(r), h])
                    far = (pos - at).abs().double()
                    z = modified(q @ K.T * c["scale"], c["cap"], slope, far).masked_fill(~seen, -float("inf"))
                    lse = torch.logsumexp(z, 1)
                    w = torch.exp(z - torch.where(torch.isinf(lse), 0.0, lse)[:, None])
                    sizes = ((q.abs() @ K.abs().T * abs(c["scale"])).masked_fill(~seen, 0).amax(1),
                             (abs(slope) * far).masked_fill(~seen, 0).amax(1), seen.sum(1).double())
                    yield p, h, m, w @ V, lse, w @ V.abs(), sizes


def compare(c, out, lse, cap_error=None):
    """batch_cases.check against `reference`.  cap_error: how far the cap may put a score off,
    from the largest sum of |scale q_i k_ji|, instead of score_error's part of the cap."""
    P, M, Hq, D = c["P"], c["M"], c["Hq"], c["D"]
    out, untouched = out.view(P, M, Hq, D), torch.ones(M, dtype=torch.bool, device="cuda")
    for p, h, m, ref, rl, mean, (dots, far, keys) in reference(c):
        rows = slice(m, m + len(rl))
        untouched[rows] = False
        got, gl = out[p, rows, h].double(), lse[p, rows, h].double()
        assert not got.isnan().any() and not gl.isnan().any()
        es = score_error(D, dots, far, 0.0 if cap_error else c["cap"]) + keys * 2.0 ** -24
        if cap_error:
            es += cap_error(dots)
        rounded = 0.0 if c["kind"] == "fp32" else 2.0 ** -8
        tol = (rounded + 2 * es)[:, None] * mean + HALF[c["dtype"]] * ref.abs() * (1 + 2.0 ** -7)
        off = (got - ref).abs()
        assert (off <= tol).all(), (p, h, m, (off > tol).nonzero()[:3].tolist(), (off / tol.clamp(min=1e-30)).max().item())
        some = ~torch.isinf(rl)
        assert torch.equal(torch.isinf(gl), ~some) and not got[~some].any()
        assert ((gl - rl).abs()[some] <= (es + 2.0 ** -22 * rl.abs())[some]).all(), (gl - rl).abs()[some].max().item()
    assert (out[:, untouched] == 7.0).all() and (lse[:, untouched] == 7.0).all(), "a row of no sequence was written"
