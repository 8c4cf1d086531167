"""The largest pool that the calls take, 16 rows short of 2^31: its first and
last pages written and read, and a page outside it."""
import numpy as np
import pytest
import torch

import sequence_tensor_transformer_gb300 as st

import test_gpu_paged_attn as ta
import test_gpu_rope_cache as tr
from helpers import dev_tensor, host_f64, nan_workspace, to_f64
from oracle import attn_oracle as ao

pytestmark = pytest.mark.gpu

PAGES, PAGE = (1 << 27) - 1, 16


@pytest.mark.parametrize("kind,D", [("bf16", 8), ("e4m3", 16)])
def test_pool_of_almost_2_31_rows(kind, D):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    st.load_library()
    torch.cuda.set_device(0)
    if torch.cuda.mem_get_info()[0] < 110 << 30:
        pytest.skip("needs 110 GB of free memory")
    n, Hq = 100, 3
    code = torch.uint8 if kind == "e4m3" else torch.bfloat16
    k, v = (torch.empty(1, PAGES, 1, PAGE, D, dtype=code, device="cuda") for _ in range(2))
    scales = [torch.empty(1, PAGES, 1, PAGE, device="cuda") if kind == "e4m3" else None for _ in range(2)]
    cache = (k, v, *scales)
    pages = np.array([PAGES - 1, 0, 12345, PAGES // 2, PAGES - 2, 1, PAGES // 3])
    for t in cache:
        if t is not None:  # what the append does not write is not read
            t[:, torch.from_numpy(pages).cuda()] = 0xFF if t.dtype == torch.uint8 else float("nan")
    rng = np.random.default_rng(D)
    rows = tr.draw(rng, (1, n, (Hq + 2) * D), "bf16")
    q = st.sptp_rope_append_kv(dev_tensor(rows, "bf16"), ta.ints(range(n)), ta.ints([0] * n), ta.ints(pages[None]), None, cache, Hq)
    x = to_f64(rows, "bf16").reshape(n, Hq + 2, D)
    at = (pages[np.arange(n) // PAGE], np.arange(n) % PAGE)
    small = []
    for pool, scale, want in ((k, scales[0], x[:, Hq]), (v, scales[1], x[:, Hq + 1])):
        part = pool[0, torch.from_numpy(pages).cuda(), 0].cpu()  # [7, PAGE, D]
        if kind == "e4m3":
            s = scale[0, torch.from_numpy(pages).cuda(), 0].cpu().numpy()
            codes, sw = ao.quantise_rows(want)
            assert np.array_equal(part.numpy().reshape(-1, D)[:n], codes) and np.array_equal(s.reshape(-1)[:n], sw)
            wide = ao.dequantised(part.numpy(), s)
        else:
            wide = host_f64(part)
            assert np.array_equal(wide.reshape(-1, D)[:n], want)
        small.append(np.nan_to_num(wide)[None, :, None])
    last = q[:, -1:].contiguous()
    order = np.arange(7)[None]
    for bad in (None, 2, 6):
        table = pages[None].copy()
        kv = [s.copy() for s in small]
        if bad is not None:  # the first page past the pool: zero keys and values
            table[0, bad] = PAGES
            for s in kv:
                s[:, bad] = 0
        ws = nan_workspace(st.sptp_paged_attn_workspace_size(1, 1, Hq, 1, D))
        out, lse = st.sptp_paged_attn_decode(last, cache, ta.ints(table), ta.ints([n]), workspace=ws)
        assert st.sptp_read_device_status(ws) == (0 if bad is None else st.STATUS["shape"])
        c = dict(P=1, B=1, Hq=Hq, Hkv=1, D=D, page=PAGE, lens=np.array([n]), table=order, kind=kind, dtype="bf16", window=0,
                 scale=D ** -0.5, q64=host_f64(last), k64=kv[0], v64=kv[1])
        ta.check(c, out, lse)
    del k, v, scales, cache
    torch.cuda.empty_cache()
