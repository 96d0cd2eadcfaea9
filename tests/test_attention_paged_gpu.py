"""Target-side attention operators over paged K/V on the GPU, against oracle/attention_paged.py.

Tolerances.  u = finfo(type).eps / 2 is a rounding to the operands' type, f = 2^-24 one to fp32.

* norm + rotation: fp32 throughout, one rounding at the end.  The norm's factor is off by at
  most (hd + 8) f relative (a sum of hd squares, mean, root, products); a rotation sums two
  products with rounded table entries, 4 f of |a| + |b| more.  So
  |err| <= u |y| + (hd + 16) f (|a| + |b|).
* attention: every weight is rounded once (u relative; fp16 below its normal range 2^-25
  absolute, against a largest weight of at least 1), the result once.  A score is a sum of hd
  products on the tensor cores, whose adds may truncate (2 f each), and enters an exponential:
  relative weight error e = 2 (hd + 4) f S + 2^-21, S the largest sum of |q_d k_d| scale
  (2^-21: the exponential and the scaling), once in the numerator and once in the denominator.
  The sums over T keys add at most (T + 64) 2 f each.  With mass = sum p |v|:
  |err| <= u |y| + 1.01 mass (u + 2 e + 4 (T + 64) f) + T 2^-25 max|v| (fp16 only).
* lse: e + 2 (T + 64) f + 4 f |lse|.
"""

import numpy as np
import pytest
import torch

import oracle as O
from block_diffusion_speculative_gemm_b200 import dflash as D

pytestmark = pytest.mark.gpu

OA = O.attention_paged
F = 2.0 ** -24
BASE, EPS = 1e6, 1e-6
T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def f64(t):
    return t.detach().double().cpu().numpy()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cu_of(rows):
    return i32([0] + list(np.cumsum(rows)))


def make_table(g, need, spare=2, unmapped=-1):
    """A shuffled table of `need[r]` pages per request and the number of pages."""
    n_pages = sum(need) + spare
    perm = torch.randperm(n_pages, generator=g, device="cuda").cpu().numpy()
    tab = np.full((len(need), max(max(need), 1)), unmapped, np.int32)
    at = 0
    for r, n in enumerate(need):
        tab[r, :n] = perm[at:at + n]
        at += n
    return tab, n_pages


def row_ws():
    return D.new_workspace(D.attention_paged_workspace_size(0, 0, 1, 1, 64))


# ---------------------------------------------------------------- norms and rotation
def check_rows(got, x, gain, pos, base, dtype):
    ref = OA.norm_rope(f64(x), None if gain is None else f64(gain), pos, base, EPS)
    tol = torch.finfo(dtype).eps / 2 * np.abs(ref) + (x.shape[2] + 16) * F * OA.rotated_bound(
        f64(x), None if gain is None else f64(gain), EPS) + 2.0 ** -25 * (dtype == torch.float16)
    bad = np.abs(f64(got) - ref) > tol
    assert not bad.any(), (bad.sum(), np.abs(f64(got) - ref)[bad].max())


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("nq,nkv,rows,norm,rope,fused", [
    (32, 8, [1], True, True, True),
    (4, 2, [3, 0, 0, 17, 1, 0], True, True, True),
    (5, 1, [29], False, True, False),
    (7, 7, [2, 9], True, False, True),
    (1, 1, [0, 1, 1], False, False, False),
    (32, 8, [700, 611], True, True, True),        # the many-row schedule
    (3, 1, [k % 3 for k in range(70)], True, True, False),
    (2, 1, [k % 4 for k in range(1100)], True, True, False),
])
def test_qk_norm_rope(dtype, hd, nq, nkv, rows, norm, rope, fused):
    g = gen(hd + nq)
    dt, n, pad = T[dtype], sum(rows), 3
    start = np.array([(37 * r) % 501 for r in range(len(rows))])
    if fused:
        qkv = randn(g, n + pad, nq + 2 * nkv, hd, dtype=dt)
        q, k = qkv[:, :nq], qkv[:, nq:nq + nkv]
    else:
        q, k = randn(g, n + pad, nq, hd, dtype=dt), randn(g, n + pad, nkv, hd, dtype=dt)
    gq = randn(g, hd, std=0.3).add(1).to(dt) if norm else None
    gk = randn(g, hd, std=0.3).add(1).to(dt) if norm else None
    table = D.rope_table(501 + max(rows), hd, BASE) if rope else None
    qo = torch.full((n + pad, nq, hd), 7.0, dtype=dt, device="cuda")
    ko = torch.full((n + pad, nkv, hd), 7.0, dtype=dt, device="cuda")
    ws = row_ws()
    D.qk_norm_rope(q, k, gq, gk, table, cu_of(rows), i32(start), qo, ko, ws, eps=EPS)
    assert D.get_error(ws) == 0
    pos = OA.positions(np.cumsum([0] + rows), start)
    check_rows(qo[:n], q[:n], gq, pos, BASE if rope else None, dt)
    check_rows(ko[:n], k[:n], gk, pos, BASE if rope else None, dt)
    assert (qo[n:] == 7).all() and (ko[n:] == 7).all()  # padding rows stay as they were
    # in place, and each operand alone: the same bits
    D.qk_norm_rope(None, k, None, gk, table, cu_of(rows), i32(start), None, k, ws, eps=EPS)
    assert torch.equal(k[:n], ko[:n])
    D.qk_norm_rope(q, None, gq, None, table, cu_of(rows), i32(start), q, None, ws, eps=EPS)
    assert torch.equal(q[:n], qo[:n])
    assert D.get_error(ws) == 0


def test_qk_one_operand_normalised_and_far_positions():
    g = gen(5)
    q, k = randn(g, 4, 4, 128, dtype=torch.float32), randn(g, 4, 2, 128, dtype=torch.float32)
    gk = randn(g, 128, std=0.3).add(1)
    table = D.rope_table(200_004, 128, BASE)
    qo, ko, ws = torch.empty_like(q), torch.empty_like(k), row_ws()
    D.qk_norm_rope(q, k, None, gk, table, cu_of([4]), i32([200_000]), qo, ko, ws, eps=EPS)
    pos = np.arange(200_000, 200_004)
    check_rows(qo, q, None, pos, BASE, torch.float32)
    check_rows(ko, k, gk, pos, BASE, torch.float32)


def test_qk_errors_leave_the_request_alone():
    g = gen(6)
    q, k = randn(g, 9, 4, 64), randn(g, 9, 2, 64)
    table = D.rope_table(50, 64, BASE)
    ws = row_ws()
    want = torch.empty_like(q), torch.empty_like(k)
    D.qk_norm_rope(q, k, None, None, table, cu_of([3, 3, 3]), i32([0, 5, 9]), *want, ws)
    assert D.get_error(ws) == 0
    for start, cu, bad, bits in [
            ([0, 48, 9], [0, 3, 6, 9], 1, D.DEV_CTX_CAP),   # runs past the table
            ([0, -1, 9], [0, 3, 6, 9], 1, D.DEV_CTX_CAP),
            ([0, 2**31 - 2, 9], [0, 3, 6, 9], 1, D.DEV_CTX_CAP),
            ([0, 5, 9], [0, 3, 6, 12], 2, D.DEV_ROWS)]:     # ends behind the rows
        qo, ko = torch.full_like(q, 7), torch.full_like(k, 7)
        D.qk_norm_rope(q, k, None, None, table, i32(cu), i32(start), qo, ko, ws)
        assert D.get_error(ws) == bits
        for r in range(3):
            s = slice(3 * r, 3 * r + 3)
            if r == bad:
                assert (qo[s] == 7).all() and (ko[s] == 7).all()
            else:
                assert torch.equal(qo[s], want[0][s]) and torch.equal(ko[s], want[1][s])


def test_fp16_overflow_is_reported():
    x = torch.full((1, 2, 64), 60000.0, dtype=torch.float16, device="cuda")
    table = D.rope_table(4, 64, BASE)
    o, ws = torch.empty_like(x), row_ws()
    D.qk_norm_rope(x, None, None, None, table, cu_of([1]), i32([1]), o, None, ws)
    assert D.get_error(ws) == D.DEV_RANGE  # 60000 (cos 1 + sin 1) > 65504


# ---------------------------------------------------------------- append
@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("f32", "f16"), ("f16", "bf16"),
                                         ("bf16", "f16"), ("f32", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("page,hd,nkv,rows,norm", [
    (16, 64, 2, [1], True),
    (32, 128, 1, [5, 0, 40, 33], False),
    (64, 128, 8, [64, 63, 65, 1], True),
    (192, 64, 3, [200, 7], True),
    (16, 128, 8, [400, 1000], True),
])
def test_kv_append_paged(dtype, cache, page, hd, nkv, rows, norm):
    g = gen(page + hd)
    dt, ct, n = T[dtype], T[cache], sum(rows)
    start = np.array([(53 * r + 11) % 90 for r in range(len(rows))])
    need = [-(-(int(s) + a) // page) for s, a in zip(start, rows)]
    tab, n_pages = make_table(g, need)
    # pages below a chunk's first position are not the call's business
    for r, s in enumerate(start):
        tab[r, : s // page] = -5
    kv = randn(g, n + 2, 2 * nkv, hd, dtype=dt)
    k, v = kv[:, :nkv], kv[:, nkv:]
    gk = randn(g, hd, std=0.3).add(1).to(dt) if norm else None
    kp = randn(g, n_pages, nkv, page, hd, dtype=ct)
    vp = randn(g, n_pages, nkv, page, hd, dtype=ct)
    ref_k, ref_v = f64(kp), f64(vp)
    kp0, vp0 = kp.clone(), vp.clone()
    ws = row_ws()
    D.kv_append_paged(k, v, gk, D.rope_table(90 + max(rows), hd, BASE), cu_of(rows), i32(start),
                      kp, vp, torch.from_numpy(tab).cuda(), ws, eps=EPS)
    assert D.get_error(ws) == 0
    cu = np.cumsum([0] + rows)
    pos = OA.positions(cu, start)
    gg = None if gk is None else f64(gk)
    kr = OA.norm_rope(f64(k[:n]), gg, pos, BASE, EPS)
    OA.append(kr, f64(v[:n]), ref_k, ref_v, tab, cu, start)
    tol_k = np.zeros_like(ref_k)
    OA.append(torch.finfo(ct).eps / 2 * np.abs(kr)
              + (hd + 16) * F * OA.rotated_bound(f64(k[:n]), gg, EPS) + 2.0 ** -25,
              np.zeros_like(kr), tol_k, np.zeros_like(ref_k), tab, cu, start)
    assert (np.abs(f64(kp) - ref_k) <= tol_k).all()  # tolerance 0 wherever nothing is written
    written = tol_k > 0
    assert torch.equal(vp, torch.where(torch.from_numpy(written).cuda(),
                                       torch.from_numpy(ref_v).cuda().to(dt).float().to(ct), vp0))
    assert not written.all() and torch.equal(kp[~torch.from_numpy(written).cuda()],
                                             kp0[~torch.from_numpy(written).cuda()])


def test_append_errors_leave_the_request_alone():
    g = gen(9)
    k, v = randn(g, 30, 2, 64), randn(g, 30, 2, 64)
    table = D.rope_table(100, 64, BASE)
    ws = row_ws()
    tab = np.array([[0, 1, 2], [3, 4, 5], [6, 7, 8]], np.int32)
    cu, start = cu_of([10, 10, 10]), [0, 12, 30]

    def run(tab, start, cu=cu, rope=table):
        kp = torch.zeros(9, 2, 16, 64, dtype=torch.float16, device="cuda")
        vp = torch.zeros_like(kp)
        D.kv_append_paged(k, v, None, rope, cu, i32(start), kp, vp, torch.from_numpy(tab).cuda(),
                          ws)
        return kp, vp, D.get_error(ws)

    want_k, want_v, bits = run(tab, start)
    assert bits == 0
    cases = []
    for e in (-1, 9, 2**31 - 1):
        t = tab.copy()
        t[1, 1] = e  # positions 16..21 of request 1
        cases.append((t, start, D.DEV_PAGE))
    cases += [(tab, [0, 39, 30], D.DEV_CTX_CAP),   # behind the last page
              (tab, [0, -3, 30], D.DEV_CTX_CAP)]
    for t, st, want in cases:
        kp, vp, bits = run(t, st)
        assert bits == want
        assert (kp[3:6] == 0).all() and (vp[3:6] == 0).all()
        for s in (slice(0, 3), slice(6, 9)):
            assert torch.equal(kp[s], want_k[s]) and torch.equal(vp[s], want_v[s])
    # a rotation table that ends before the last request's rows
    kp, vp, bits = run(tab, start, rope=D.rope_table(39, 64, BASE))
    assert bits == D.DEV_CTX_CAP and (kp[6:] == 0).all() and torch.equal(kp[:6], want_k[:6])


# ---------------------------------------------------------------- attention
class Case:
    """Inputs of one attention call over shuffled pages, with NaN in every slot behind a
    request's keys."""

    def __init__(self, seed, rows, ctx, nq, nkv, hd, dtype, page, kv_len=None, pad=0, std=2.0,
                 fused=False):
        g = gen(seed)
        self.rows, self.dt, self.nq, self.nkv, self.hd, self.page = rows, T[dtype], nq, nkv, hd, page
        self.cu = np.cumsum([0] + rows)
        self.start = np.array(ctx)
        self.len = np.array([a + c for a, c in zip(rows, ctx)] if kv_len is None else kv_len)
        self.tab, self.n_pages = make_table(g, [-(-int(t) // page) for t in self.len])
        n = sum(rows) + pad
        if fused:
            self.q = randn(g, n, nq + 2 * nkv, hd, std=std, dtype=self.dt)[:, :nq]
        else:
            self.q = randn(g, n, nq, hd, std=std, dtype=self.dt)
        self.kp = randn(g, self.n_pages, nkv, page, hd, dtype=self.dt)
        self.vp = randn(g, self.n_pages, nkv, page, hd, dtype=self.dt)
        used = torch.zeros(self.n_pages, page, dtype=torch.bool, device="cuda")
        for r, t in enumerate(self.len):
            for j in range(0, int(t), page):
                used[self.tab[r, j // page], : min(page, int(t) - j)] = True
        self.kp.masked_fill_(~used[:, None, :, None], float("nan"))
        self.vp.masked_fill_(~used[:, None, :, None], float("nan"))

    def run(self, causal=True, window=0, scale=None, ws=None, kv_len="given", expect=0, out=None):
        n, b = self.q.shape[0], len(self.rows)
        ws = ws if ws is not None else D.attention_paged_workspace(b, n, self.nq, self.nkv, self.hd)
        out = out if out is not None else torch.full((n, self.nq, self.hd), 7.0, dtype=self.dt,
                                                     device="cuda")
        lse = torch.full((n, self.nq), 7.0, device="cuda")
        D.attention_paged(self.q, i32(self.cu), i32(self.start),
                          i32(self.len) if kv_len == "given" else None, self.kp, self.vp,
                          torch.from_numpy(self.tab).cuda(), out, ws, scale=scale, causal=causal,
                          window=window, lse=lse)
        assert D.get_error(ws) == expect
        return out, lse

    def check(self, out, lse, causal=True, window=0, scale=None):
        scale = self.hd ** -0.5 if scale is None else scale
        kp, vp, n = f64(self.kp), f64(self.vp), int(self.cu[-1])
        ref, rl, mass = OA.attention(f64(self.q[:n]), kp, vp, self.tab, self.cu, self.start,
                                     self.len, scale, causal, window)
        S = OA.score_error(f64(self.q[:n]), kp, self.tab, self.cu, self.start, self.len, scale)
        u, keys = torch.finfo(self.dt).eps / 2, int(self.len.max())
        e = 2 * (self.hd + 4) * F * S + 2.0 ** -21
        tol = u * np.abs(ref) + 1.01 * mass * (u + 2 * e + 4 * (keys + 64) * F)
        if self.dt == torch.float16:
            tol = tol + keys * 2.0 ** -25 * np.nanmax(np.abs(vp))
        got = f64(out[:n])
        assert np.array_equal(np.isnan(got), np.isnan(ref))
        fin = np.isfinite(ref) & np.isfinite(tol)
        assert np.array_equal(got[np.isinf(ref)], ref[np.isinf(ref)])
        err, lim = np.abs(got[fin] - ref[fin]), tol[fin]
        assert (err <= lim).all(), (err / np.maximum(lim, 1e-30)).max()
        gl = f64(lse[:n])
        assert np.array_equal(np.isneginf(gl), np.isneginf(rl))
        f = np.isfinite(rl)
        assert (np.abs(gl[f] - rl[f]) <= e + 2 * (keys + 64) * F + 4 * F * np.abs(rl[f])).all()
        assert (out[n:] == 7).all() and (lse[n:] == 7).all()  # padding rows stay as they were


SHAPES = [
    # rows per request, earlier positions, n_q, n_kv, page
    ([1], [0], 4, 2, 64),
    ([1], [2048], 32, 8, 64),
    ([1] * 9, [0, 1, 62, 63, 64, 65, 127, 500, 1999], 8, 2, 16),
    ([8] * 5, [0, 7, 56, 57, 900], 32, 8, 64),
    ([16, 16], [100, 3000], 32, 8, 128),
    ([5, 0, 1, 12, 0], [33, 9, 0, 250, 0], 6, 2, 32),
    ([130], [0], 4, 4, 64),
    ([97, 1, 301, 2], [0, 700, 31, 5], 28, 4, 32),
    ([257, 64], [1, 64], 5, 1, 192),
    ([3], [40], 64, 1, 16),
    ([700], [400], 2, 1, 64),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_attention_paged(dtype, hd, shape):
    rows, ctx, nq, nkv, page = SHAPES[shape]
    c = Case(shape + hd, rows, ctx, nq, nkv, hd, dtype, page, pad=shape % 3, fused=shape % 2 == 1)
    for causal, window in ((True, 0), (False, 0), (True, 17), (False, 300), (True, 1)):
        c.check(*c.run(causal, window), causal, window)


def test_attention_default_kv_len_and_scale():
    c = Case(3, [4, 9], [70, 0], 8, 2, 64, "bf16", 16)
    a, la = c.run(kv_len=None)
    b, lb = c.run()
    assert torch.equal(a, b) and torch.equal(la, lb)
    c.check(*c.run(scale=0.7), scale=0.7)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rows", [[3, 2, 4], [200, 40, 90]])
def test_attention_rows_that_see_nothing(hd, rows):
    # no keys at all; fewer keys than rows (causal rows still see the first ones); a window
    # that has left all keys behind for the last rows
    c = Case(4, rows, [0, 0, 50], 8, 2, hd, "bf16", 16, kv_len=[0, 1, 30])
    for causal, window in ((True, 0), (False, 0), (True, 21), (False, 25), (True, 5)):
        out, lse = c.run(causal, window)
        c.check(out, lse, causal, window)
        assert (out[: rows[0]] == 0).all() and (lse[: rows[0]] == float("-inf")).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rows,G", [([1, 6], 4), ([150], 2), ([16], 4)])
def test_masked_keys_do_not_reach_other_rows(dtype, hd, rows, G):
    # NaN and infinities in keys that only later rows see, and in keys the window has passed
    ctx = [90] * len(rows)
    c = Case(8, rows, ctx, 2 * G, 2, hd, dtype, 32)
    for r, n in enumerate(rows):
        last, mid = 90 + n - 1, 90 + n // 2
        for pos, val in ((last, float("nan")), (mid, float("inf")), (70, float("-inf"))):
            pg = c.tab[r, pos // 32]
            c.kp[pg, :, pos % 32] = float("nan") if val != val else 0.5
            c.vp[pg, :, pos % 32, : hd // 2] = val
    for causal, window in ((True, 10), (True, 0), (False, 12)):
        c.check(*c.run(causal, window), causal, window)


def test_nan_query_stays_in_its_row():
    c = Case(12, [9], [100], 8, 2, 128, "bf16", 64)
    c.q[3, 5, 7] = float("nan")
    out, lse = c.run()
    assert torch.isnan(out[3, 5]).all() and torch.isnan(lse[3, 5])
    keep = torch.ones(9, 8, dtype=torch.bool, device="cuda")
    keep[3, 5] = False
    assert torch.isfinite(out[keep]).all() and torch.isfinite(lse[keep]).all()


def test_pages_out_of_sight_need_not_be_mapped():
    # pages behind a sliding window were given back; pages behind kv_len never existed
    c = Case(13, [4, 130], [500, 300], 8, 2, 64, "f16", 16)
    want = c.run(window=40)
    c.check(*want, window=40)
    c.tab[0, : (500 - 39) // 16] = -1
    c.tab[1, : (300 - 39) // 16] = 10**6
    got = c.run(window=40)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_attention_errors_leave_the_request_alone():
    c = Case(14, [5, 6, 7], [40, 200, 90], 8, 2, 128, "bf16", 32)
    want, wl = c.run()
    tab, cu, start, length = c.tab.copy(), c.cu.copy(), c.start.copy(), c.len.copy()

    def broken(bits, keep):
        out, lse = c.run(expect=bits)
        for r in range(3):
            s = slice(int(cu[r]), int(cu[r + 1]))
            if r in keep:
                assert torch.equal(out[s], want[s]) and torch.equal(lse[s], wl[s])
            else:
                assert (out[s] == 7).all() and (lse[s] == 7).all()
        c.tab, c.cu, c.start, c.len = tab.copy(), cu.copy(), start.copy(), length.copy()

    # the other requests keep their division of work when request 1's keys stay counted
    for e in (-1, c.n_pages, -2**31):
        c.tab[1, 3] = e
        broken(D.DEV_PAGE, (0, 2))
    for bad in (-1, c.tab.shape[1] * 32 + 1, 2**31 - 1):
        c.len[1] = bad
        out, _ = c.run(expect=D.DEV_CTX_CAP)
        assert (out[5:11] == 7).all()
        assert torch.allclose(out[:5].float(), want[:5].float(), atol=0.05)
        assert torch.allclose(out[11:].float(), want[11:].float(), atol=0.05)
    c.len = length.copy()
    c.start[1] = -1
    assert (c.run(expect=D.DEV_CTX_CAP)[0][5:11] == 7).all()
    c.start = start.copy()
    c.cu = np.array([0, 5, 11, 19])  # the last request runs past the rows
    assert (c.run(expect=D.DEV_ROWS)[0][11:] == 7).all()
    c.cu = np.array([0, 11, 5, 18])  # descending: request 1 has no rows of its own
    c.run(expect=D.DEV_ROWS)


def test_attention_output_strides():
    c = Case(15, [3, 4], [20, 100], 8, 2, 128, "bf16", 64)
    want, _ = c.run()
    wide = torch.full((7, 8 * 128 + 64), 7.0, dtype=c.dt, device="cuda")
    c.run(out=wide.as_strided((7, 8, 128), (8 * 128 + 64, 128, 1)))
    assert torch.equal(wide[:, : 8 * 128].reshape(7, 8, 128), want)
    assert (wide[:, 8 * 128:] == 7).all()


def test_attention_is_deterministic_and_streams_are_independent():
    cases = [Case(16, [8] * 6, [300, 4, 900, 77, 1500, 10], 32, 8, 128, "bf16", 64),
             Case(17, [200, 31], [0, 600], 8, 2, 64, "f16", 16)]
    want = [c.run() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    spaces = [D.attention_paged_workspace(len(c.rows), c.q.shape[0], c.nq, c.nkv, c.hd)
              for c in cases]
    args = [(i32(c.cu), i32(c.start), i32(c.len), torch.from_numpy(c.tab).cuda()) for c in cases]
    outs = [[torch.empty_like(w[0]) for _ in range(5)] for w in want]
    torch.cuda.synchronize()
    for rep in range(5):
        for c, s, ws, (cu, st, ln, tab), o in zip(cases, streams, spaces, args, outs):
            D.attention_paged(c.q, cu, st, ln, c.kp, c.vp, tab, o[rep], ws, stream=s)
    torch.cuda.synchronize()
    for w, o, ws in zip(want, outs, spaces):
        assert D.get_error(ws) == 0
        for x in o:
            assert torch.equal(x, w[0])


def test_offsets_past_32_bits():
    # the used pages lie behind 2^31 elements (2^32 bytes) of each pool
    page, nkv, hd = 64, 8, 128
    n_pages = 2**31 // (page * nkv * hd) + 40
    kp = torch.empty(n_pages, nkv, page, hd, dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    tab = np.arange(n_pages - 35, n_pages, dtype=np.int32)[None, ::-1].copy()
    g = gen(20)
    k, v = randn(g, 2100, nkv, hd, dtype=torch.bfloat16), randn(g, 2100, nkv, hd,
                                                                dtype=torch.bfloat16)
    q = randn(g, 70, 32, hd, dtype=torch.bfloat16)
    tabd = torch.from_numpy(tab).cuda()
    ws = D.attention_paged_workspace(1, 2100, 32, nkv, hd)
    D.kv_append_paged(k, v, None, None, cu_of([2100]), i32([0]), kp, vp, tabd, ws)
    for rows in (1, 70):
        out = torch.empty(rows, 32, hd, dtype=torch.bfloat16, device="cuda")
        D.attention_paged(q[:rows], cu_of([rows]), i32([2100 - rows]), None, kp, vp, tabd, out, ws)
        assert D.get_error(ws) == 0
        low = torch.zeros(35, nkv, page, hd, dtype=torch.bfloat16, device="cuda")
        low_v = torch.zeros_like(low)
        low.copy_(kp[n_pages - 35:])
        low_v.copy_(vp[n_pages - 35:])
        want = torch.empty_like(out)
        D.attention_paged(q[:rows], cu_of([rows]), i32([2100 - rows]), None, low, low_v,
                          i32(tab - (n_pages - 35)), want, ws)
        assert torch.equal(out, want)
        assert torch.equal(low[34, :, 3].cpu(), k[3].cpu())  # the table runs backwards


# ---------------------------------------------------------------- the operators together
class Layer:
    """One attention layer's step as a target model runs it: norms and rotation of the queries,
    append of the keys and values, attention."""

    def __init__(self, batch, nq, nkv, hd, page, cap, dtype, max_rows):
        g = gen(30)
        self.nq, self.nkv, self.hd, self.dt = nq, nkv, hd, T[dtype]
        per = cap // page
        self.tab = torch.randperm(batch * per, generator=g, device="cuda").to(torch.int32).view(
            batch, per).contiguous()
        self.kp = torch.full((batch * per, nkv, page, hd), float("nan"), dtype=self.dt,
                             device="cuda")
        self.vp = self.kp.clone()
        self.gq, self.gk = (randn(g, hd, std=0.2).add(1).to(self.dt) for _ in range(2))
        self.rope = D.rope_table(cap, hd, BASE)
        self.ws = D.attention_paged_workspace(batch, max_rows, nq, nkv, hd)

    def step(self, qkv, cu, start, qr, out, window=0):
        q, k, v = qkv.split((self.nq, self.nkv, self.nkv), 1)
        D.qk_norm_rope(q, None, self.gq, None, self.rope, cu, start, qr, None, self.ws)
        D.kv_append_paged(k, v, self.gk, self.rope, cu, start, self.kp, self.vp, self.tab, self.ws)
        D.attention_paged(qr, cu, start, None, self.kp, self.vp, self.tab, out, self.ws,
                          window=window)


def layer_oracle(lay, qkv, window=0):
    """The whole sequence [n, heads, hd] of one request at once, K and V rounded to the cache
    type, q to the operand type; returns (out, tolerance)."""
    x = f64(qkv)
    n, hd, nq, nkv = x.shape[0], lay.hd, lay.nq, lay.nkv
    pos = np.arange(n)

    def rnd(y):
        return f64(torch.from_numpy(y).to(lay.dt))

    q = rnd(OA.norm_rope(x[:, :nq], f64(lay.gq), pos, BASE, EPS))
    k = rnd(OA.norm_rope(x[:, nq:nq + nkv], f64(lay.gk), pos, BASE, EPS))
    v = x[:, nq + nkv:]
    kp, vp = (np.ascontiguousarray(y.transpose(1, 0, 2))[None] for y in (k, v))
    return OA.attention(q, kp, vp, [[0]], [0, n], [0], [n], hd ** -0.5, True, window)


@pytest.mark.parametrize("dtype,hd,nq,nkv,page,window", [
    ("bf16", 128, 32, 8, 64, 0), ("f16", 64, 4, 2, 16, 0), ("bf16", 64, 14, 2, 32, 50)])
def test_prompt_chunks_blocks_and_tokens_equal_one_pass(dtype, hd, nq, nkv, page, window):
    # two requests: prompts in ragged chunks, then drafted blocks, then single tokens
    total = [150, 233]
    steps = [([90, 1], None), ([0, 140], None), ([43, 75], None), ([8, 8], None), ([8, 8], None),
             ([1, 1], None)]
    assert [sum(s[0][r] for s in steps) for r in range(2)] == total
    lay = Layer(2, nq, nkv, hd, page, 384, dtype, 200)
    g = gen(31)
    seq = [randn(g, n, nq + 2 * nkv, hd, dtype=T[dtype]) for n in total]
    got = [torch.empty(n, nq, hd, dtype=T[dtype], device="cuda") for n in total]
    at = [0, 0]
    for rows, _ in steps:
        n = sum(rows)
        qkv = torch.cat([seq[r][at[r]:at[r] + rows[r]] for r in range(2)]).contiguous()
        qr = torch.empty(n, nq, hd, dtype=T[dtype], device="cuda")
        out = torch.empty_like(qr)
        lay.step(qkv, cu_of(rows), i32(at), qr, out, window)
        first = 0
        for r in range(2):
            got[r][at[r]:at[r] + rows[r]] = out[first:first + rows[r]]
            first += rows[r]
            at[r] += rows[r]
    assert D.get_error(lay.ws) == 0
    u = torch.finfo(T[dtype]).eps / 2
    for r in range(2):
        ref, _, mass = layer_oracle(lay, seq[r], window)
        # the oracle's rounded q and k may sit one rounding step (2 u) away from the kernel's
        # where an fp32 result is next to a border; a normalised head has |x| <= sqrt(hd) gmax, so
        # a score (scale hd^-0.5) moves by at most 4 u sqrt(hd) gmax^2, a weight by that in the
        # numerator and in the denominator; the fp32 terms of the single call are below 1% of it
        gmax = float(max(lay.gq.abs().max(), lay.gk.abs().max()))
        move = 4 * u * lay.hd ** 0.5 * gmax ** 2
        tol = u * np.abs(ref) + mass * (1.01 * u + 2 * move)
        assert (np.abs(f64(got[r]) - ref) <= tol).all()


def test_captured_layer_step_replays_on_new_inputs():
    # a graph over the three calls, replayed with other rows, lengths and page tables; a padded
    # batch (fewer rows than captured) leaves the padding alone
    lay = Layer(3, 8, 2, 128, 64, 512, "bf16", 24)
    g = gen(33)
    qkv = torch.zeros(24, 12, 128, dtype=torch.bfloat16, device="cuda")
    qr = torch.zeros(24, 8, 128, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(qr)
    cu, start = cu_of([8, 8, 8]), i32([0, 0, 0])
    lay.kp.normal_()
    lay.vp.normal_()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        lay.step(qkv, cu, start, qr, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lay.step(qkv, cu, start, qr, out)
    other = torch.cuda.CUDAGraph()  # a second graph over the same workspace
    with torch.cuda.graph(other):
        lay.step(qkv, cu, start, qr, out)
    for rows, st in (([8, 8, 8], [3, 200, 500 - 8]), ([1, 0, 16], [70, 5, 9]), ([2, 1, 1], [0, 63, 64])):
        n = sum(rows)
        qkv.copy_(randn(g, 24, 12, 128))
        cu.copy_(cu_of(rows))
        start.copy_(i32(st))
        lay.tab.copy_(lay.tab[torch.randperm(3, generator=g, device="cuda")])
        kp, vp = lay.kp.clone(), lay.vp.clone()
        out.fill_(7)
        graph.replay()
        a, ka = out.clone(), lay.kp.clone()
        lay.kp.copy_(kp)
        lay.vp.copy_(vp)
        out.fill_(7)
        other.replay()
        assert torch.equal(a, out)
        lay.kp.copy_(kp)
        lay.vp.copy_(vp)
        out.fill_(7)
        lay.step(qkv, cu, start, qr, out)
        assert D.get_error(lay.ws) == 0
        assert torch.equal(a, out) and torch.equal(ka, lay.kp)
        assert (out[n:] == 7).all()


def test_current_device_is_checked():
    c = Case(40, [2], [10], 4, 2, 64, "bf16", 16)
    ws = D.attention_paged_workspace(1, 2, 4, 2, 64)
    with pytest.raises(ValueError):
        D.attention_paged(c.q, i32(c.cu).cpu(), i32(c.start), None, c.kp, c.vp,
                          torch.from_numpy(c.tab).cuda(), torch.empty_like(c.q), ws)
