"""The paths inside the target-side attention operators that small shapes do not reach: the ring
of bulk copies for many rows, items of one and of two query tiles in one batch, batches of more
than 32 requests, non-finite values that a row does see, repeated launches.  Tolerances as in
test_attention_paged_gpu.py."""

import numpy as np
import pytest
import torch

import oracle as O
from block_diffusion_speculative_gemm_b200 import dflash as D

from .test_attention_paged_gpu import (BASE, EPS, T, Case, check_rows, cu_of, f64, gen, i32,
                                       make_table, randn, row_ws)

pytestmark = pytest.mark.gpu
OA = O.attention_paged


# ---------------------------------------------------------------- row operators, many rows
@pytest.mark.parametrize("dtype,hd,nq,nkv", [("bf16", 128, 32, 8), ("f32", 128, 32, 8),
                                             ("f16", 64, 1, 1), ("f32", 64, 4, 2),
                                             ("bf16", 64, 90, 10)])
@pytest.mark.parametrize("rows", [[1300], [0, 700, 0, 613, 1], [k % 41 for k in range(70)]])
def test_qk_many_rows(dtype, hd, nq, nkv, rows):
    g, dt, n = gen(hd + nq), T[dtype], sum(rows)
    assert n > 1184  # more than 8 rows a multiprocessor
    start = np.array([(37 * r) % 501 for r in range(len(rows))])
    qkv = randn(g, n + 40, nq + 2 * nkv, hd, dtype=dt)
    q, k = qkv[:, :nq], qkv[:, nq:nq + nkv]
    gq, gk = (randn(g, hd, std=0.3).add(1).to(dt) for _ in range(2))
    table = D.rope_table(501 + max(rows), hd, BASE)
    pos = OA.positions(np.cumsum([0] + rows), start)
    ws = row_ws()
    for a, b, t in ((gq, gk, table), (gq, None, table), (None, gk, None), (None, None, table)):
        qo = torch.full((n + 40, nq, hd), 7.0, dtype=dt, device="cuda")
        ko = torch.full((n + 40, nkv, hd), 7.0, dtype=dt, device="cuda")
        D.qk_norm_rope(q, k, a, b, t, cu_of(rows), i32(start), qo, ko, ws, eps=EPS)
        assert D.get_error(ws) == 0
        base = BASE if t is not None else None
        check_rows(qo[:n], q[:n], a, pos, base, dt)
        check_rows(ko[:n], k[:n], b, pos, base, dt)
        assert (qo[n:] == 7).all() and (ko[n:] == 7).all()
    # one operand alone and in place: the same bits as the last call
    D.qk_norm_rope(None, k, None, None, table, cu_of(rows), i32(start), None, k, ws, eps=EPS)
    assert D.get_error(ws) == 0 and torch.equal(k[:n], ko[:n])


def test_qk_many_rows_errors_leave_the_request_alone():
    g = gen(6)
    rows = [500, 600, 400]
    q, k = randn(g, 1500, 4, 64), randn(g, 1500, 2, 64)
    table = D.rope_table(700, 64, BASE)
    ws = row_ws()
    want = torch.empty_like(q), torch.empty_like(k)
    D.qk_norm_rope(q, k, None, None, table, cu_of(rows), i32([0, 5, 9]), *want, ws)
    assert D.get_error(ws) == 0
    edges = [0, 500, 1100, 1500]
    for start, cu, bad, bits in [
            ([0, 101, 9], edges, 1, D.DEV_CTX_CAP),            # runs past the table
            ([0, -1, 9], edges, 1, D.DEV_CTX_CAP),
            ([0, 2**31 - 2, 9], edges, 1, D.DEV_CTX_CAP),
            ([0, 5, 9], [0, 500, 1100, 1501], 2, D.DEV_ROWS)]:  # ends behind the rows
        qo, ko = torch.full_like(q, 7), torch.full_like(k, 7)
        D.qk_norm_rope(q, k, None, None, table, i32(cu), i32(start), qo, ko, ws)
        assert D.get_error(ws) == bits
        for r in range(3):
            s = slice(edges[r], edges[r + 1])
            if r == bad:
                assert (qo[s] == 7).all() and (ko[s] == 7).all()
            else:
                assert torch.equal(qo[s], want[0][s]) and torch.equal(ko[s], want[1][s])


@pytest.mark.parametrize("dtype,cache,hd,nkv,page", [("bf16", "bf16", 128, 8, 64),
                                                     ("f32", "f16", 64, 2, 16),
                                                     ("f16", "bf16", 128, 1, 192),
                                                     ("f32", "bf16", 128, 20, 32)])
def test_append_many_rows(dtype, cache, hd, nkv, page):
    g, dt, ct = gen(page), T[dtype], T[cache]
    rows = [900, 0, 33, 1] + [11] * 40
    n = sum(rows)
    start = np.array([(53 * r + 11) % 90 for r in range(len(rows))])
    need = [-(-(int(s) + a) // page) for s, a in zip(start, rows)]
    tab, n_pages = make_table(g, need)
    kv = randn(g, n + 3, 2 * nkv, hd, dtype=dt)
    k, v = kv[:, :nkv], kv[:, nkv:]
    gk = randn(g, hd, std=0.3).add(1).to(dt)
    rope = D.rope_table(1000, hd, BASE)
    ws = row_ws()

    def run(tab, expect):
        kp = torch.full((n_pages, nkv, page, hd), 7.0, dtype=ct, device="cuda")
        vp = kp.clone()
        D.kv_append_paged(k, v, gk, rope, cu_of(rows), i32(start), kp, vp,
                          torch.from_numpy(tab).cuda(), ws, eps=EPS)
        assert D.get_error(ws) == expect
        return kp, vp

    kp, vp = run(tab, 0)
    cu = np.cumsum([0] + rows)
    pos = OA.positions(cu, start)
    kr = OA.norm_rope(f64(k[:n]), f64(gk), pos, BASE, EPS)
    tol = torch.finfo(ct).eps / 2 * np.abs(kr) + (hd + 16) * 2.0 ** -24 * OA.rotated_bound(
        f64(k[:n]), f64(gk), EPS) + 2.0 ** -25
    ref_k, ref_v = np.full(kp.shape, 7.0), np.full(vp.shape, 7.0)
    tol_k, vv = np.zeros(kp.shape), f64(v[:n].float().to(ct))
    OA.append(kr, vv, ref_k, ref_v, tab, cu, start)
    OA.append(tol, np.zeros_like(tol), tol_k, np.zeros(vp.shape), tab, cu, start)
    assert (np.abs(f64(kp) - ref_k) <= tol_k).all()
    assert np.array_equal(f64(vp), ref_v)
    # an unmapped page of the long request: none of its rows is written, all others are
    bad = tab.copy()
    bad[0, 3] = -1
    kb, vb = run(bad, D.DEV_PAGE)
    own = sorted(set(tab[0, :need[0]]))
    rest = np.setdiff1d(np.arange(n_pages), own)
    assert (kb[own] == 7).all() and (vb[own] == 7).all()
    assert torch.equal(kb[rest], kp[rest]) and torch.equal(vb[rest], vp[rest])


# ---------------------------------------------------------------- attention
@pytest.mark.parametrize("dtype,hd,nq,nkv,page", [("bf16", 128, 8, 2, 64), ("f16", 64, 8, 2, 16),
                                                  ("bf16", 64, 3, 3, 32), ("f16", 128, 7, 1, 128)])
def test_items_of_one_and_two_query_tiles(dtype, hd, nq, nkv, page):
    # long chunks (both query tiles), short ones (keys split over the tiles), with an odd and an
    # even number of 128-key runs, one run, and none
    rows = [300, 5, 1, 0, 70, 33, 129, 2]
    ctx = [100, 20, 640, 7, 0, 250, 511, 1023]
    c = Case(71, rows, ctx, nq, nkv, hd, dtype, page, pad=5)
    for causal, window in ((True, 0), (False, 0), (True, 130), (False, 70)):
        c.check(*c.run(causal, window), causal, window)


@pytest.mark.parametrize("batch", [33, 150])
@pytest.mark.parametrize("rows", [1, 9])
@pytest.mark.parametrize("hd", [64, 128])
def test_many_requests(batch, rows, hd):
    r = np.random.default_rng(batch)
    n = [rows if k % 7 else 0 for k in range(batch)]
    ctx = [int(x) for x in r.integers(0, 400, batch)]
    c = Case(batch, n, ctx, 8, 2, hd, "bf16", 16)
    c.check(*c.run(True, 0), True, 0)
    c.check(*c.run(True, 33), True, 33)


@pytest.mark.parametrize("rows", [1, 7])
def test_the_largest_batch(rows):
    # 4096 requests, most of them with a few rows, some with none, some without keys
    n = [rows if k % 9 else 0 for k in range(4096)]
    ctx = [k % 23 for k in range(4096)]
    c = Case(77, n, ctx, 4, 1, 64, "f16", 16, kv_len=[a + b if k % 13 else 0 for k, (a, b) in
                                                      enumerate(zip(n, ctx))])
    c.check(*c.run())
    with pytest.raises(D.DFlashError):
        ws = D.attention_paged_workspace(1, 1, 4, 1, 64)
        e = torch.zeros(4097, dtype=torch.int32, device="cuda")
        D.attention_paged(c.q[:1], torch.zeros(4098, dtype=torch.int32, device="cuda"), e, e, c.kp,
                          c.vp, torch.zeros(4097, 1, dtype=torch.int32, device="cuda"),
                          torch.empty_like(c.q[:1]), ws)


def test_one_long_chunk_among_single_tokens():
    # the average is far from every request: 40 single tokens and a chunk of 200
    c = Case(72, [1] * 20 + [200] + [1] * 20, [90 * (k % 11) for k in range(41)], 8, 2, 128,
             "bf16", 64)
    c.check(*c.run())
    c.check(*c.run(window=100), window=100)


@pytest.mark.parametrize("rows", [[2], [150]])
@pytest.mark.parametrize("hd", [64, 128])
def test_non_finite_values_that_rows_see(rows, hd):
    # a key with NaN and one with an infinity in sight: the rows that see them are NaN or
    # infinite as the formula says, the others are as without them
    c = Case(73, rows, [200], 8, 2, hd, "bf16", 32)
    n = rows[0]
    clean, _ = c.run()
    pg, sl = c.tab[0, (200 + n - 1) // 32], (200 + n - 1) % 32  # the last row's own key
    c.kp[pg, 0, sl, 3] = float("nan")
    out, lse = c.run()
    assert torch.isnan(out[-1, :4]).all() and torch.isnan(lse[-1, :4]).all()
    assert torch.isfinite(out[-1, 4:]).all()
    assert torch.equal(out[:-1], clean[:-1])
    c.kp[pg, 0, sl, 3] = 0.25
    c.vp[pg, 1, sl, 5] = float("inf")
    out, lse = c.run()
    assert (out[-1, 4:, 5] == float("inf")).all()
    assert torch.isfinite(lse).all() and torch.isfinite(out[:-1]).all()
    keep = torch.arange(hd, device="cuda") != 5
    assert torch.isfinite(out[-1][:, keep]).all()


@pytest.mark.parametrize("rows", [[1, 1], [8] * 12, [700, 30, 257]])
def test_repeated_launches_give_the_same_bits(rows):
    c = Case(74, rows, [900 - 60 * k % 800 for k in range(len(rows))], 32, 8, 128, "bf16", 64)
    n, b = c.q.shape[0], len(rows)
    ws = D.attention_paged_workspace(b, n, 32, 8, 128)
    args = (i32(c.cu), i32(c.start), i32(c.len), c.kp, c.vp, torch.from_numpy(c.tab).cuda())
    want, _ = c.run()
    outs = [torch.empty_like(want) for _ in range(8)]
    for rep in range(25):
        for o in outs:
            D.attention_paged(c.q, *args, o, ws)
        assert D.get_error(ws) == 0
        assert all(torch.equal(o, want) for o in outs)


def test_row_operators_repeat_and_overlap_streams():
    g = gen(75)
    rows = [1500, 700, 3]
    n = sum(rows)
    qkv = randn(g, n, 48, 128, dtype=torch.bfloat16)
    q, k = qkv[:, :32], qkv[:, 32:40]
    table = D.rope_table(1600, 128, BASE)
    gq = randn(g, 128, std=0.3).add(1).to(torch.bfloat16)
    cu, st = cu_of(rows), i32([0, 50, 9])
    spaces = [row_ws() for _ in range(2)]
    outs = [(torch.empty(n, 32, 128, dtype=torch.bfloat16, device="cuda"),
             torch.empty(n, 8, 128, dtype=torch.bfloat16, device="cuda")) for _ in range(6)]
    want = [torch.empty_like(x) for x in outs[0]]
    D.qk_norm_rope(q, k, gq, gq, table, cu, st, *want, spaces[0])
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for rep in range(40):
        for i, o in enumerate(outs):
            D.qk_norm_rope(q, k, gq, gq, table, cu, st, *o, spaces[i % 2], stream=streams[i % 2])
    torch.cuda.synchronize()
    assert all(D.get_error(w) == 0 for w in spaces)
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o, want))


# ---------------------------------------------------------------- refusals of the binding
def test_binding_refusals():
    c = Case(76, [2], [10], 4, 2, 64, "bf16", 16)
    ws = D.attention_paged_workspace(1, 2, 4, 2, 64)
    cu, st, ln, tab = i32(c.cu), i32(c.start), i32(c.len), torch.from_numpy(c.tab).cuda()
    out = torch.empty_like(c.q)
    good = [c.q, cu, st, ln, c.kp, c.vp, tab, out, ws]
    D.attention_paged(*good)

    def refused(kind, at, value, **kw):
        args = list(good)
        args[at] = value
        with pytest.raises(kind):
            D.attention_paged(*args, **kw)

    refused(ValueError, 0, c.q.transpose(1, 2))            # heads not contiguous
    refused(ValueError, 0, c.q[0])
    refused(TypeError, 0, c.q.double())
    refused(ValueError, 1, cu[:1])
    refused(TypeError, 1, cu.long())
    refused(TypeError, 3, ln.float())
    refused(TypeError, 4, c.kp.half())
    refused(ValueError, 5, c.vp[:-1])
    refused(ValueError, 6, tab[0])
    refused(ValueError, 7, out[:1])
    refused(TypeError, 8, ws.int())
    refused(D.DFlashError, 8, ws[:256])                     # too small
    refused(TypeError, 8, ws, lse=torch.empty(2, 4, device="cuda", dtype=torch.float16))
    refused(ValueError, 8, ws, lse=torch.empty(2, 3, device="cuda"))
    refused(ValueError, 8, ws, window=2**40)
    refused(D.DFlashError, 8, ws, window=-1)
    refused(D.DFlashError, 8, ws, scale=0.0)
    refused(TypeError, 8, ws, scale="x")
    torch.cuda.synchronize()
    assert D.get_error(ws) == 0
