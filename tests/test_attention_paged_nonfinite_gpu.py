"""Infinities and NaN in keys that only some rows of a paged attention call see, behind contexts
of 48 thousand keys: the answer is that of the formula, with a clean error word, and the other
request keeps its bits.  Tolerances as in test_attention_paged_gpu.py, against 64 bits on the GPU."""

import numpy as np
import pytest
import torch

from block_diffusion_speculative_gemm_b200 import dflash as D

from .test_attention_paged_gpu import F, Case, T, cu_of, gen, i32, randn

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def check(out, lse, q, K, V, start, scale, causal, window):
    """Rows q [n, heads, hd] at start.. over K, V [heads, keys, hd] of the same heads."""
    n, heads, hd = q.shape
    keys = K.shape[1]
    u = torch.finfo(q.dtype).eps / 2
    pos = torch.arange(start, start + n, device="cuda")[:, None]
    key = torch.arange(keys, device="cuda")[None]
    see = (key <= pos) if causal else torch.ones_like(key <= pos)
    if window:
        see = see & (key > pos - window)
    for h in range(heads):
        x, k, v = q[:, h].double(), K[h].double(), V[h].double()
        S = float((x.abs() @ k.abs().T).max()) * scale
        z = (x @ k.T * scale).masked_fill(~see, -INF)
        p = torch.softmax(z, -1)
        odd = ~torch.isfinite(v)
        ref = p @ v.masked_fill(odd, 0)
        mass = p @ v.masked_fill(odd, 0).abs()
        for j in odd.any(-1).nonzero()[:, 0].tolist():
            w = torch.where(odd[j][None] & see[:, j:j + 1], p[:, j:j + 1] * v[j][None], 0.0)
            ref = ref + w
        e = 2 * (hd + 4) * F * S + 2.0 ** -21
        fin = torch.isfinite(ref)
        got = out[:, h].double()
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        assert torch.equal(got[torch.isinf(ref)], ref[torch.isinf(ref)])
        tol = u * ref.abs() + 1.01 * mass * (u + 2 * e + 4 * (keys + 64) * F)
        if q.dtype == torch.float16:
            tol = tol + keys * 2.0 ** -25 * float(v.masked_fill(odd, 0).abs().max())
        assert ((got - ref).abs()[fin] <= tol[fin]).all()
        rl = torch.logsumexp(z, -1)
        assert ((lse[:, h].double() - rl).abs() <= e + 2 * (keys + 64) * F + 4 * F * rl.abs()).all()


# 74 kv heads x 2 requests: as many items as a B200 has multiprocessors, so that an item is a
# single run of keys for one CTA.  16 rows take the mma.sync kernel, 40 one query tile, 130 two.
@pytest.mark.parametrize("dtype,hd", [("bf16", 64), ("f16", 128)])
@pytest.mark.parametrize("rows", [16, 40, 130])
@pytest.mark.parametrize("causal,cut", [(True, 0), (True, 13), (False, 9)])
def test_values_that_some_rows_see_behind_long_contexts(dtype, hd, rows, causal, cut):
    nkv, page, keys = 74, 64, 48_000 if hd == 64 else 24_000
    g, dt, per = gen(rows), T[dtype], keys // page
    start, scale = keys - rows, hd ** -0.5
    # the window leaves the keys below `cut` behind for the first rows, more for later ones
    window = keys - rows + 1 - cut if cut else 0
    q = randn(g, 2 * rows, nkv, hd, std=2.0, dtype=dt)
    kp = randn(g, 2 * per, nkv, page, hd, dtype=dt)
    vp = randn(g, 2 * per, nkv, page, hd, dtype=dt)
    tab = torch.randperm(2 * per, generator=g, device="cuda").to(torch.int32).view(2, per)
    ws = D.attention_paged_workspace(2, 2 * rows, nkv, nkv, hd)
    out = torch.empty(2, 2 * rows, nkv, hd, dtype=dt, device="cuda")
    lse = torch.empty(2 * rows, nkv, device="cuda")

    def run(o):
        D.attention_paged(q, cu_of([rows, rows]), i32([start, start]), None, kp, vp, tab, o, ws,
                          causal=causal, window=window, lse=lse)
        assert D.get_error(ws) == 0

    run(out[0])
    # of request 0: the last rows' own keys, keys that the window passes, and one that all see
    last = keys - 1
    for at, d, val in ((last, 3, INF), (last - rows // 2, 3, -INF), (last - 1, hd - 1, NAN),
                       (cut + 4, 17, INF), (cut + rows // 2, 20, -INF), (cut + 1, 17, -INF),
                       (keys // 2, 40, INF)):
        vp[int(tab[0, at // page]), :, at % page, d] = val
    run(out[1])
    assert torch.equal(out[1][rows:], out[0][rows:])
    K, V = (p[tab[0].long()].permute(1, 0, 2, 3).reshape(nkv, keys, hd) for p in (kp, vp))
    heads = [0, 1, 36, 73]
    check(out[1][:rows][:, heads], lse[:rows][:, heads], q[:rows][:, heads], K[heads], V[heads],
          start, scale, causal, window)
    # the columns that hold none of them are those of the first call
    keep = torch.ones(hd, dtype=torch.bool, device="cuda")
    keep[[3, hd - 1, 17, 20, 40]] = False
    assert torch.equal(out[1][:rows][..., keep], out[0][:rows][..., keep])


@pytest.mark.parametrize("rows", [16, 200])
def test_keys_and_values_full_of_nan_that_later_rows_see(rows):
    # every value of the last half of the chunk's keys: the first half's rows are as without them
    nkv, hd, page, keys = 4, 64, 16, 20_000
    g = gen(rows)
    q = randn(g, rows, nkv, hd, std=2.0, dtype=torch.bfloat16)
    kp = randn(g, keys // page, nkv, page, hd, dtype=torch.bfloat16)
    vp = randn(g, keys // page, nkv, page, hd, dtype=torch.bfloat16)
    tab = torch.arange(keys // page, dtype=torch.int32, device="cuda").view(1, -1)
    ws = D.attention_paged_workspace(1, rows, nkv, nkv, hd)
    out = torch.empty(2, rows, nkv, hd, dtype=torch.bfloat16, device="cuda")
    for i in range(2):
        D.attention_paged(q, cu_of([rows]), i32([keys - rows]), None, kp, vp, tab, out[i], ws)
        assert D.get_error(ws) == 0
        flat = vp.permute(0, 2, 1, 3).reshape(keys, nkv, hd).clone()
        flat[keys - rows // 2:] = NAN
        vp.copy_(flat.view(keys // page, page, nkv, hd).permute(0, 2, 1, 3))
    half = rows - rows // 2
    assert torch.equal(out[1, :half], out[0, :half])
    assert torch.isnan(out[1, half:]).all() and torch.isfinite(out[0]).all()


@pytest.mark.parametrize("dtype,hd,page", [("bf16", 128, 64), ("f16", 64, 16)])
@pytest.mark.parametrize("rows", [[1, 3], [1] * 40, [33, 9], [300, 70, 1]])
def test_stored_keys_that_no_row_sees(dtype, hd, page, rows):
    # more keys stored than the causal rows see, and keys behind a window: NaN in all of them, and
    # pages that hold nothing else not mapped
    ctx = [50 + 23 * r for r in range(len(rows))]
    end = [a + b for a, b in zip(rows, ctx)]
    c = Case(hd + len(rows), rows, ctx, 8, 2, hd, dtype, page, kv_len=[t + 137 for t in end])
    c.check(*c.run(False), False)
    for window in (0, 45):
        want = c.run(True, window)
        c.check(*want, True, window)
        d = Case(hd + len(rows), rows, ctx, 8, 2, hd, dtype, page, kv_len=[t + 137 for t in end])
        for r, t in enumerate(end):
            first = max(0, ctx[r] - window + 1) if window else 0
            for key in [*range(first), *range(t, t + 137)]:
                at = int(d.tab[r, key // page])
                d.kp[at, :, key % page] = NAN
                d.vp[at, :, key % page] = NAN
            d.tab[r, : first // page] = -1
            d.tab[r, -(-t // page):] = d.n_pages
        got = d.run(True, window)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
