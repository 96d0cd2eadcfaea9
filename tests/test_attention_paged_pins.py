"""CPU pins of oracle/attention_paged.py, and the refusals of the target-side attention calls.

No library call here reaches the GPU: every refusal happens on the host.
"""

import numpy as np
import pytest

import oracle as O
from block_diffusion_speculative_gemm_b200 import dflash as D

OA = O.attention_paged


# ---------------------------------------------------------------- oracle
def test_norm_rope_closed_forms():
    rng = np.random.default_rng(0)
    x = rng.normal(size=(5, 3, 8))
    pos = np.array([0, 1, 7, 100, 5])
    y = OA.norm_rope(x, None, pos, 1e4, 1e-6)
    assert np.allclose(y[0], x[0])                                   # position 0: identity
    assert np.allclose((y * y).sum(-1), (x * x).sum(-1))             # a rotation keeps the norm
    th = 7 * 1e4 ** (-2 * 1 / 8)                                     # pair 1 of 4 at position 7
    a, b = x[2, 0, 1], x[2, 0, 5]
    assert np.isclose(y[2, 0, 1], a * np.cos(th) - b * np.sin(th))
    assert np.isclose(y[2, 0, 5], b * np.cos(th) + a * np.sin(th))
    z = OA.norm_rope(x, np.ones(8), pos, None, 0.0)
    assert np.allclose((z * z).mean(-1), 1.0)
    assert np.allclose(OA.norm_rope(3 * x, np.ones(8), pos, None, 0.0), z)
    g = rng.normal(size=8)
    assert np.allclose(OA.norm_rope(x, g, pos, None, 0.0), z * g)


def test_scores_depend_on_relative_position():
    rng = np.random.default_rng(1)
    q, k = rng.normal(size=(1, 1, 16)), rng.normal(size=(1, 1, 16))

    def score(i, j):
        return float((OA.norm_rope(q, None, [i], 1e4, 0) * OA.norm_rope(k, None, [j], 1e4, 0)).sum())

    assert np.isclose(score(9, 4), score(109, 104))
    assert not np.isclose(score(9, 4), score(9, 5))


def _loops(q, K, V, lo, hi, scale):
    w = [np.exp(scale * sum(a * b for a, b in zip(q, K[j]))) for j in range(lo, hi)]
    return sum(x * V[j] for x, j in zip(w, range(lo, hi))) / sum(w), np.log(sum(w))


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 3), (False, 4)])
def test_attention_matches_loops(causal, window):
    rng = np.random.default_rng(2)
    P, hd, nq, nkv = 4, 8, 4, 2
    kp, vp = rng.normal(size=(2, 9, nkv, P, hd))
    tab = np.array([[5, 0, 3], [8, 1, -1]])
    cu, start, length = [0, 2, 5], [9, 3], [11, 6]
    q = rng.normal(size=(5, nq, hd))
    out, lse, _ = OA.attention(q, kp, vp, tab, cu, start, length, 0.4, causal, window)
    for r in range(2):
        K = np.concatenate([kp[t].transpose(1, 0, 2) for t in tab[r] if t >= 0])  # [T, nkv, hd]
        V = np.concatenate([vp[t].transpose(1, 0, 2) for t in tab[r] if t >= 0])
        for i in range(cu[r], cu[r + 1]):
            p = start[r] + i - cu[r]
            hi = min(length[r], p + 1) if causal else length[r]
            lo = max(0, p - window + 1) if window else 0
            for h in range(nq):
                o, l = _loops(q[i, h], K[:, h // 2], V[:, h // 2], lo, hi, 0.4)
                assert np.allclose(out[i, h], o) and np.isclose(lse[i, h], l)


def test_attention_special_cases():
    rng = np.random.default_rng(3)
    kp, vp = rng.normal(size=(2, 4, 1, 4, 8))
    q = rng.normal(size=(3, 2, 8))
    tab = np.array([[2, 1]])
    # one visible key: its value; no key: zeros and -inf; equal keys: the mean
    out, lse, _ = OA.attention(q, kp, vp, tab, [0, 3], [0], [1], 1.0)
    assert np.allclose(out, vp[2, 0, 0]) and np.isfinite(lse).all()
    out, lse, _ = OA.attention(q, kp, vp, tab, [0, 3], [0], [0], 1.0)
    assert (out == 0).all() and np.isneginf(lse).all()
    out, lse, _ = OA.attention(q, np.ones_like(kp), vp, tab, [0, 3], [5], [8], 1.0, causal=False)
    assert np.allclose(out, np.concatenate((vp[2, 0], vp[1, 0])).mean(0))
    # a window of one key: the row's own
    out, _, _ = OA.attention(q, kp, vp, tab, [0, 3], [4], [8], 1.0, window=1)
    assert np.allclose(out[1], vp[1, 0, 1])
    # what masked keys hold does not matter
    kp2, vp2 = kp.copy(), vp.copy()
    kp2[1, :, 3], vp2[1, :, 3] = np.nan, np.inf
    a = OA.attention(q, kp, vp, tab, [0, 3], [4], [8], 1.0)[0]
    assert np.array_equal(a, OA.attention(q, kp2, vp2, tab, [0, 3], [4], [8], 1.0)[0])


def test_append_then_gather_is_the_sequence():
    rng = np.random.default_rng(4)
    k, v = rng.normal(size=(2, 7, 2, 8))
    kp, vp = np.zeros((2, 5, 2, 4, 8))
    tab = np.array([[3, 1], [4, 0]])
    OA.append(k, v, kp, vp, tab, [0, 3, 7], [0, 2])
    assert np.array_equal(OA.gather(kp, tab[0], 3), k[:3].transpose(1, 0, 2))
    assert np.array_equal(OA.gather(vp, tab[1], 6)[:, 2:], v[3:].transpose(1, 0, 2))
    assert (kp[2] == 0).all()


# ---------------------------------------------------------------- refusals
P = 4096  # a fake device pointer: never dereferenced on these paths
BIG = 1 << 40


def _attn(**kw):
    a = dict(q=P, qs=32 * 128, dtype=D.BF16, cu=P, st=P, kl=P, batch=2, n=4, nq=32, nkv=8, hd=128,
             k=P, v=P, pages=10, page=64, tab=P, maxp=4, scale=0.1, causal=1, window=0, out=P,
             os=32 * 128, lse=None, ws=P, bytes=BIG)
    assert set(kw) <= set(a)
    a.update(kw)
    return D.lib().dflash_attention_paged(
        a["q"], a["qs"], a["dtype"], a["cu"], a["st"], a["kl"], a["batch"], a["n"], a["nq"],
        a["nkv"], a["hd"], a["k"], a["v"], a["pages"], a["page"], a["tab"], a["maxp"], a["scale"],
        a["causal"], a["window"], a["out"], a["os"], a["lse"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=0), D.OK),
    (dict(batch=0), D.EINVAL), (dict(n=-1), D.EINVAL), (dict(nkv=0), D.EINVAL),
    (dict(nq=30), D.EINVAL), (dict(q=None), D.EINVAL), (dict(out=None), D.EINVAL),
    (dict(cu=None), D.EINVAL), (dict(st=None), D.EINVAL), (dict(k=None), D.EINVAL),
    (dict(v=None), D.EINVAL), (dict(tab=None), D.EINVAL), (dict(ws=None), D.EINVAL),
    (dict(q=P + 8), D.EINVAL), (dict(k=P + 8), D.EINVAL), (dict(out=P + 2), D.EINVAL),
    (dict(ws=P + 64), D.EINVAL), (dict(qs=32 * 128 - 8), D.EINVAL), (dict(qs=32 * 128 + 4), D.EINVAL),
    (dict(os=100), D.EINVAL), (dict(lse=P + 2), D.EINVAL), (dict(dtype=7), D.EINVAL),
    (dict(scale=0.0), D.EINVAL), (dict(scale=-1.0), D.EINVAL), (dict(scale=float("nan")), D.EINVAL),
    (dict(scale=float("inf")), D.EINVAL), (dict(window=-1), D.EINVAL), (dict(pages=0), D.EINVAL),
    (dict(maxp=0), D.EINVAL), (dict(page=0), D.EINVAL),
    (dict(dtype=D.F32), D.EUNSUPPORTED), (dict(hd=96), D.EUNSUPPORTED),
    (dict(nq=65, nkv=1, qs=65 * 128, os=65 * 128), D.EUNSUPPORTED), (dict(page=48), D.EUNSUPPORTED),
    (dict(page=8), D.EUNSUPPORTED), (dict(page=96), D.EUNSUPPORTED),
    (dict(batch=4097), D.EUNSUPPORTED), (dict(pages=1 << 22), D.EUNSUPPORTED),
    (dict(maxp=(1 << 24) + 1), D.EUNSUPPORTED), (dict(bytes=1 << 12), D.EWORKSPACE),
])
def test_attention_refusals(kw, code):
    assert _attn(**kw) == code


def _qk(**kw):
    a = dict(q=P, qs=4 * 64, k=P, ks=2 * 64, dtype=D.F16, gq=P, gk=None, eps=1e-6, rope=P, maxpos=9,
             cu=P, st=P, batch=2, n=4, nq=4, nkv=2, hd=64, qo=P, qos=4 * 64, ko=P, kos=2 * 64, ws=P,
             bytes=BIG)
    assert set(kw) <= set(a)
    a.update(kw)
    return D.lib().dflash_qk_norm_rope(*list(a.values())[:21], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=0), D.OK), (dict(batch=0), D.EINVAL), (dict(nq=0, nkv=0), D.EINVAL),
    (dict(nq=-1), D.EINVAL), (dict(q=None), D.EINVAL), (dict(ko=None), D.EINVAL),
    (dict(q=P + 2), D.EINVAL), (dict(qs=4 * 64 + 4), D.EINVAL), (dict(kos=64), D.EINVAL),
    (dict(gq=P + 4), D.EINVAL), (dict(rope=P + 4), D.EINVAL), (dict(maxpos=0), D.EINVAL),
    (dict(eps=-1.0), D.EINVAL), (dict(eps=float("nan")), D.EINVAL), (dict(dtype=3), D.EINVAL),
    (dict(cu=None), D.EINVAL), (dict(st=None), D.EINVAL), (dict(ws=None), D.EINVAL),
    (dict(hd=32), D.EUNSUPPORTED), (dict(hd=256), D.EUNSUPPORTED), (dict(bytes=256), D.EWORKSPACE),
])
def test_qk_norm_rope_refusals(kw, code):
    assert _qk(**kw) == code


def _append(**kw):
    a = dict(k=P, ks=2 * 64, v=P, vs=2 * 64, dtype=D.F32, gk=P, eps=1e-6, rope=P, maxpos=9, cu=P,
             st=P, batch=2, n=4, nkv=2, hd=64, kp=P, vp=P, cache=D.F16, pages=4, page=16, tab=P,
             maxp=3, ws=P, bytes=BIG)
    assert set(kw) <= set(a)
    a.update(kw)
    return D.lib().dflash_kv_append_paged(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=0), D.OK), (dict(batch=0), D.EINVAL), (dict(nkv=0), D.EINVAL), (dict(k=None), D.EINVAL),
    (dict(vs=2 * 64 + 2), D.EINVAL), (dict(v=P + 8), D.EINVAL), (dict(kp=None), D.EINVAL),
    (dict(vp=P + 8), D.EINVAL), (dict(tab=None), D.EINVAL), (dict(dtype=9), D.EINVAL),
    (dict(cache=9), D.EINVAL), (dict(cache=D.F32), D.EUNSUPPORTED), (dict(hd=80), D.EUNSUPPORTED),
    (dict(page=24), D.EUNSUPPORTED), (dict(pages=1 << 28), D.EUNSUPPORTED),
    (dict(rope=None, maxpos=0, ws=None), D.EINVAL), (dict(bytes=8), D.EWORKSPACE),
])
def test_kv_append_refusals(kw, code):
    assert _append(**kw) == code


def test_rope_table_refusals():
    f = D.lib().dflash_rope_table
    assert f(None, 4, 64, 1e6, None) == D.EINVAL
    assert f(P, 0, 64, 1e6, None) == D.EINVAL
    assert f(P, 4, 63, 1e6, None) == D.EINVAL
    assert f(P, 4, 64, 0.0, None) == D.EINVAL
    assert f(P, 4, 64, float("inf"), None) == D.EINVAL


def test_workspace_sizes():
    f = D.attention_paged_workspace_size
    hdr = D.lib().dflash_verify_workspace_size(0, 8, 100)
    assert f(0, 0, 1, 1, 64) == hdr
    assert f(1, 1, 32, 8, 128) > hdr
    for bad in ((-1, 1, 32, 8, 128), (1, -1, 32, 8, 128), (1, 1, 32, 5, 128), (1, 1, 32, 8, 96),
                (1, 1, 0, 8, 128), (1, 1, 65, 1, 64)):
        assert f(*bad) == 0
    assert all(f(b, n, 32, 8, 128) % 256 == 0 for b in (1, 7, 300) for n in (1, 300, 5000))
    with pytest.raises(D.DFlashError):
        D.attention_paged_workspace(1, 1, 32, 5, 128)


def test_binding_refuses_host_tensors():
    import torch

    q = torch.zeros(2, 4, 64)
    with pytest.raises(ValueError):
        D.qk_norm_rope(q, None, None, None, None, torch.zeros(2, dtype=torch.int32),
                       torch.zeros(1, dtype=torch.int32), q, None, torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError):
        D.qk_norm_rope(None, None, None, None, None, None, None, None, None, None)
    with pytest.raises(TypeError):
        D.attention_paged([1], None, None, None, None, None, None, None, None)
