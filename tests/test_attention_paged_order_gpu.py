"""cu_rows that is not an ascending array inside [0, n_rows]: in every target-side attention
operator a request out of order writes nothing and sets DFLASH_DEV_ROWS, the others are as in a
call of their own.  Tolerances as in test_attention_paged_gpu.py."""

import numpy as np
import pytest
import torch

import oracle as O
from block_diffusion_speculative_gemm_b200 import dflash as D

from .test_attention_paged_gpu import F, Case, T, cu_of, f64, gen, i32, randn, row_ws

pytestmark = pytest.mark.gpu
OA = O.attention_paged


def in_order(cu, n_rows):
    """Request r is in order: no earlier entry is above cu[r], 0 <= cu[r] <= cu[r+1] <= n_rows."""
    return [cu[r] >= max(0, *cu[:r + 1]) and cu[r] <= cu[r + 1] <= n_rows
            for r in range(len(cu) - 1)]


def broken(kind, batch, per):
    """cu_rows of `batch` requests of `per` rows with one mistake, and n_rows."""
    n = batch * per
    cu = list(range(0, n + 1, per))
    mid = batch // 2
    if kind == "last descends":
        cu[-1] = cu[-2] - 1                     # its rows would pass for padding
    elif kind == "descends":
        cu[mid] = cu[mid + 1] + 1               # the request behind it begins inside another one
    elif kind == "end behind the rows":
        cu[-2] = n                              # the last request has no row below n_rows
        cu[-1] = n + 3
    elif kind == "far entry":
        cu[mid] = 2**31 - 1
    elif kind == "negative":
        cu[mid] = -2**31
    elif kind == "negative first":
        cu[0] = -1
    return cu, n


KINDS = ["last descends", "descends", "end behind the rows", "far entry", "negative",
         "negative first"]
# batches below and above 32 requests, the direct kernel and the ring of many rows
SIZES = [(3, 5), (40, 3), (3, 500), (70, 21)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("batch,per", SIZES)
def test_qk_norm_rope_rows_out_of_order(kind, batch, per):
    cu, n = broken(kind, batch, per)
    g = gen(batch)
    q, k = randn(g, n, 3, 64), randn(g, n, 1, 64)
    start = [7 * r % 50 for r in range(batch)]
    table = D.rope_table(60 + 2 * per, 64, 1e6)
    ws = row_ws()
    qo, ko = torch.full_like(q, 7), torch.full_like(k, 7)
    D.qk_norm_rope(q, k, None, None, table, i32(cu), i32(start), qo, ko, ws)
    assert D.get_error(ws) == D.DEV_ROWS
    want_q, want_k = torch.full_like(q, 7), torch.full_like(k, 7)
    ok = in_order(cu, n)
    assert not all(ok)
    for r in range(batch):
        if ok[r] and cu[r + 1] > cu[r]:
            s = slice(cu[r], cu[r + 1])
            D.qk_norm_rope(q[s], k[s], None, None, table, cu_of([cu[r + 1] - cu[r]]),
                           i32(start[r:r + 1]), want_q[s], want_k[s], ws)
    assert D.get_error(ws) == 0
    assert torch.equal(qo, want_q) and torch.equal(ko, want_k)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("batch,per", SIZES)
def test_kv_append_rows_out_of_order(kind, batch, per):
    cu, n = broken(kind, batch, per)
    g = gen(batch + 1)
    k, v = randn(g, n, 2, 64), randn(g, n, 2, 64)
    start = [7 * r % 50 for r in range(batch)]
    pages = -(-(50 + 2 * per) // 16)
    tab = np.arange(batch * pages, dtype=np.int32).reshape(batch, pages)
    ws = row_ws()
    kp = torch.full((batch * pages, 2, 16, 64), 7.0, dtype=torch.float16, device="cuda")
    vp = kp.clone()
    D.kv_append_paged(k, v, None, None, i32(cu), i32(start), kp, vp, i32(tab), ws)
    assert D.get_error(ws) == D.DEV_ROWS
    ref_k, ref_v = np.full(kp.shape, 7.0), np.full(vp.shape, 7.0)
    ok = in_order(cu, n)
    for r in range(batch):
        if ok[r]:
            s = slice(cu[r], cu[r + 1])
            OA.append(f64(k[s].half()), f64(v[s].half()), ref_k, ref_v, tab[r:r + 1],
                      [0, cu[r + 1] - cu[r]], start[r:r + 1])
    assert np.array_equal(f64(kp), ref_k) and np.array_equal(f64(vp), ref_v)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("batch,per", [(3, 2), (40, 3), (3, 150), (36, 17)])
def test_attention_rows_out_of_order(kind, batch, per):
    cu, n = broken(kind, batch, per)
    c = Case(batch, [per] * batch, [(31 * r) % 90 + per for r in range(batch)], 4, 2, 64, "bf16",
             16)
    c.cu = np.array(cu)
    out, lse = c.run(expect=D.DEV_ROWS)
    kp, vp = f64(c.kp), f64(c.vp)
    ok = in_order(cu, n)
    left = np.ones(n, bool)
    u = torch.finfo(T["bf16"]).eps / 2
    for r in range(batch):
        if not ok[r]:
            continue
        s = slice(cu[r], cu[r + 1])
        left[s] = False
        one = (c.tab[r:r + 1], [0, cu[r + 1] - cu[r]], c.start[r:r + 1], c.len[r:r + 1], 64 ** -0.5)
        ref, rl, mass = OA.attention(f64(c.q[s]), kp, vp, *one)
        e = 2 * (64 + 4) * F * OA.score_error(f64(c.q[s]), kp, *one) + 2.0 ** -21
        keys = int(c.len[r])
        tol = u * np.abs(ref) + 1.01 * mass * (u + 2 * e + 4 * (keys + 64) * F)
        assert (np.abs(f64(out[s]) - ref) <= tol).all()
        assert (np.abs(f64(lse[s]) - rl) <= e + 2 * (keys + 64) * F + 4 * F * np.abs(rl)).all()
    left = torch.from_numpy(left).cuda()
    assert (out[left] == 7).all() and (lse[left] == 7).all()
