"""Requests without rows (free places of a padded batch): what their lengths and page tables hold
does not matter in any of the target-side attention operators."""

import numpy as np
import pytest
import torch

from block_diffusion_speculative_gemm_b200 import dflash as D

from .test_attention_paged_gpu import Case, gen, i32, randn, row_ws

pytestmark = pytest.mark.gpu
STRAY = [(-1, -1), (-2**31, 2**31 - 1), (2**31 - 1, -5), (0, 10**6)]


@pytest.mark.parametrize("batch", [5, 45])
@pytest.mark.parametrize("rows", [1, 90])
def test_attention_of_a_padded_batch(batch, rows):
    live = [rows if r % 3 == 1 else 0 for r in range(batch)]
    ctx = [17 * r % 200 for r in range(batch)]
    c = Case(5 + rows, live, ctx, 8, 2, 64, "bf16", 16, kv_len=[
        a + b if a else 0 for a, b in zip(live, ctx)])
    want, wl = c.run()
    for r in range(batch):
        if live[r] == 0:
            c.start[r], c.len[r] = STRAY[r % len(STRAY)]
            c.tab[r] = -7
    out, lse = c.run()  # with a clean error word
    assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("batch,rows", [(5, 2), (45, 2), (5, 700)])
def test_rows_of_a_padded_batch(batch, rows):
    live = [rows if r % 3 == 1 else 0 for r in range(batch)]
    cu = np.cumsum([0] + live)
    start = np.array([7 * r for r in range(batch)])
    g, n = gen(3), int(cu[-1])
    k, v = randn(g, n, 2, 64), randn(g, n, 2, 64)
    table, ws = D.rope_table(1100, 64, 1e6), row_ws()
    pages = -(-(7 * batch + rows) // 16)
    tab = np.arange(batch * pages, dtype=np.int32).reshape(batch, pages)

    def run():
        ko = torch.empty_like(k)
        kp = torch.zeros(batch * pages, 2, 16, 64, dtype=torch.float16, device="cuda")
        vp = torch.zeros_like(kp)
        D.qk_norm_rope(None, k, None, None, table, i32(cu), i32(start), None, ko, ws)
        D.kv_append_paged(k, v, None, table, i32(cu), i32(start), kp, vp, i32(tab), ws)
        assert D.get_error(ws) == 0
        return ko, kp, vp

    want = run()
    for r in range(batch):
        if live[r] == 0:
            start[r] = STRAY[r % len(STRAY)][0]
            tab[r] = -7
    assert all(torch.equal(a, b) for a, b in zip(run(), want))
