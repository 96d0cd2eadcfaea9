"""Cases of the target-side attention operators over a paged K/V cache, and their plain forms.

Three operators, used one after the other in every attention layer of the model whose hidden
states and logits the drafting calls consume:

* ``qk_norm_rope``: RMSNorm of every query and key head, then the rotate-half position rotation;
* ``kv_append_paged``: the chunk's keys (normalised and rotated on the way) and values written
  into the pages of a paged cache;
* ``attention_paged``: attention of each request's chunk of new tokens (one token, a drafted
  block, a prompt) over its paged cache.

Requests are ragged: ``cu_rows`` and ``start_pos`` say which rows belong to which request and at
which position they start, as in the injection calls.  The lengths come from the case (its
``mix``), the values from the seed.
"""

import math
import random

import torch

own = False

ROPE_BASE = 1e6
EPS = 1e-6
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------- cases
def _rows_case(op, name, batch, rows, ctx, nq, nkv, hd, dtype, page=64, norm=True, cache=None,
               mix=1):
    c = {"name": name, "op": op, "batch": batch, "rows_lo": rows[0], "rows_hi": rows[1],
         "ctx_lo": ctx[0], "ctx_hi": ctx[1], "nq": nq, "nkv": nkv, "hd": hd, "dtype": dtype,
         "norm": norm, "mix": mix}
    if op == "append":
        c.update(page=page, cache=cache or dtype)
    return c


def _attn_case(name, batch, rows, ctx, nq, nkv, hd, dtype, page=64, causal=True, window=0,
               lse=False, first_rows=0, mix=1):
    return {"name": name, "op": "attention", "batch": batch, "rows_lo": rows[0],
            "rows_hi": rows[1], "ctx_lo": ctx[0], "ctx_hi": ctx[1], "first_rows": first_rows,
            "nq": nq, "nkv": nkv, "hd": hd, "dtype": dtype, "page": page, "causal": causal,
            "window": window, "lse": lse, "mix": mix}


def listed():
    return [
        # one request generating one token (the concurrency-1 workload): latency only
        _rows_case("qk", "qk one token", 1, (1, 1), (2048, 2048), 32, 8, 128, "bf16"),
        # a small fp32 model, ragged odd chunks, rotation without norms
        _rows_case("qk", "qk ragged fp32 hd64", 7, (1, 301), (0, 777), 4, 2, 64, "f32",
                   norm=False, mix=2),
        # prompts of four requests: pure bandwidth
        _rows_case("qk", "qk prompt 4x4096", 4, (4096, 4096), (0, 0), 32, 8, 128, "bf16"),
        # a decode step of the concurrency-32 workload
        _rows_case("append", "append decode 32", 32, (1, 1), (512, 4096), 32, 8, 128, "bf16"),
        # fp32 projections of a small model into an fp16 cache of short pages, no key norm
        _rows_case("append", "append ragged hd64", 5, (1, 37), (0, 777), 4, 2, 64, "f32",
                   page=16, norm=False, cache="f16", mix=3),
        # prompts of four requests behind contexts of odd length
        _rows_case("append", "append prompt 4x4096", 4, (4096, 4096), (1, 999), 32, 8, 128,
                   "bf16", mix=4),
        # one token of one request at the concurrency-1 context: latency
        _attn_case("attn one token 2k", 1, (1, 1), (2048, 2048), 32, 8, 128, "bf16"),
        # the target's decode step at the concurrency-32 workload
        _attn_case("attn decode 32", 32, (1, 1), (512, 4096), 32, 8, 128, "bf16", mix=5),
        # the target's verify forward of 32 drafted blocks of 8, causal inside the block
        _attn_case("attn verify 32x8", 32, (8, 8), (512, 4096), 32, 8, 128, "bf16", lse=True,
                   mix=5),
        # verify of blocks of 16 behind the long contexts
        _attn_case("attn verify 4x16 32k", 4, (16, 16), (32768, 32768), 32, 8, 128, "f16"),
        # a scheduler's mixed batch: one long prompt chunk, short ragged chunks and single
        # tokens, with a sliding window and short pages
        _attn_case("attn mixed window", 13, (1, 45), (1, 4001), 32, 8, 64, "f16", page=16,
                   window=1500, lse=True, first_rows=1021, mix=6),
        # a whole prompt: tensor-core bound
        _attn_case("attn prompt 8k", 1, (8192, 8192), (0, 0), 32, 8, 128, "bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


HEADS = [(32, 8), (4, 2), (8, 8), (28, 4), (16, 2), (5, 1), (6, 2)]


def draw(rng):
    """One more case: chunk lengths from one token to thousands, contexts from none to 32k,
    every head layout, type, page size and mask."""
    nq, nkv = rng.choice(HEADS)
    hd = rng.choice((64, 128))
    page = rng.choice((16, 32, 64, 128, 192))
    mix = rng.randrange(1, 1 << 20)
    op = rng.choice(("qk", "append", "attention", "attention"))
    batch = _log(rng, 1, 64)
    if op != "attention":
        most = max(1, 16384 * 40 * 128 // (batch * (nq + nkv) * hd))
        hi = _log(rng, 1, min(8192, most))
        lo = rng.choice((1, hi, max(1, hi // 2)))
        ctx = _log(rng, 1, 16384)
        return {k: v for k, v in _rows_case(
            op, "", batch, (lo, hi), (rng.choice((0, ctx)), ctx), nq, nkv, hd,
            rng.choice(("bf16", "bf16", "f16", "f32")), page=page, norm=rng.random() < 0.7,
            cache=rng.choice(("bf16", "f16")), mix=mix).items() if k != "name"}
    causal = rng.random() < 0.8
    hi = _log(rng, 1, 4096)
    ctx = _log(rng, 1, 32768)
    while batch * hi * (ctx + hi) * nq > 1 << 30 or batch * (ctx + hi) * nkv * hd > 1 << 27:
        if batch > 1:
            batch = (batch + 1) // 2
        elif hi > 1 and hi * 4 > ctx:
            hi = (hi + 1) // 2
        else:
            ctx = max(1, ctx // 2)
    lo = rng.choice((1, hi, max(1, hi // 2)))
    return {k: v for k, v in _attn_case(
        "", batch, (lo, hi), (rng.choice((0, ctx, ctx // 2)), ctx), nq, nkv, hd,
        rng.choice(("bf16", "f16")), page=page, causal=causal,
        window=rng.choice((0, 0, _log(rng, 1, 4096))), lse=rng.random() < 0.5,
        mix=mix).items() if k != "name"}


def _lengths(case):
    """Rows and earlier positions of every request."""
    r = random.Random(case["mix"])
    rows = [r.randint(case["rows_lo"], case["rows_hi"]) for _ in range(case["batch"])]
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])]
    if case.get("first_rows"):
        rows[0] = case["first_rows"]
    return rows, ctx


# ---------------------------------------------------------------- inputs
def _pages(case, rows, ctx, gen):
    """A shuffled page table whose requests own just the pages they need, and the pool's size."""
    need = [-(-(n + t) // case["page"]) for n, t in zip(rows, ctx)]
    n_pages = sum(need) + 3
    perm = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    at = torch.arange(max(need), device="cuda")[None, :]
    n = torch.tensor(need, device="cuda")[:, None]
    first = torch.cumsum(n, 0) - n
    table = torch.where(at < n, perm[(first + at).clamp(max=n_pages - 1)],
                        torch.full((), -1, dtype=torch.int32, device="cuda"))
    return table.contiguous(), n_pages


def _rope(max_pos, hd):
    """cos and sin of p * base^(-2i/hd), evaluated in 64 bits: [2, max_pos, hd / 2]."""
    i = torch.arange(hd // 2, dtype=torch.float64, device="cuda")
    ang = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * ROPE_BASE ** (
        -2.0 * i / hd)
    return torch.stack((ang.cos(), ang.sin())).float()


def prepare(case, seed):
    rows, ctx = _lengths(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, nq, nkv, hd = DTYPES[case["dtype"]], case["nq"], case["nkv"], case["hd"]
    n = sum(rows)

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    s = {"case": case, "n": n}
    s["cu_rows"] = torch.tensor([0] + rows, device="cuda").cumsum(0).to(torch.int32)
    s["start_pos"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    if case["op"] == "attention":
        # keys after their norm, queries with a gain: scores of a few units' spread
        s["q"] = normal(n, nq, hd, std=2.5)
        s["table"], n_pages = _pages(case, rows, ctx, gen)
        s["k_pool"] = normal(n_pages, nkv, case["page"], hd)
        s["v_pool"] = normal(n_pages, nkv, case["page"], hd)
        s["kv_len"] = torch.tensor([a + b for a, b in zip(rows, ctx)], dtype=torch.int32,
                                   device="cuda")
        s["out"] = torch.empty(n, nq, hd, dtype=dt, device="cuda")
        s["lse"] = torch.empty(n, nq, device="cuda") if case["lse"] else None
    else:
        # the rows of a fused projection: [query heads | key heads | value heads]
        qkv = normal(n, nq + 2 * nkv, hd)
        s["q"], s["k"], s["v"] = qkv[:, :nq], qkv[:, nq:nq + nkv], qkv[:, nq + nkv:]
        s["g_q"] = normal(hd, std=0.2).add(1.0) if case["norm"] else None
        s["g_k"] = normal(hd, std=0.2).add(1.0) if case["norm"] else None
        s["rope"] = _rope(max(a + b for a, b in zip(rows, ctx)) + 1, hd)
        if case["op"] == "qk":
            s["q_out"] = torch.empty(n, nq, hd, dtype=dt, device="cuda")
            s["k_out"] = torch.empty(n, nkv, hd, dtype=dt, device="cuda")
        else:
            s["table"], n_pages = _pages(case, rows, ctx, gen)
            cdt = DTYPES[case["cache"]]
            s["k_pool"] = normal(n_pages, nkv, case["page"], hd, dtype=cdt)
            s["v_pool"] = normal(n_pages, nkv, case["page"], hd, dtype=cdt)
    if own:
        from block_diffusion_speculative_gemm_b200 import dflash as D

        s["D"] = D
        s["ws"] = D.attention_paged_workspace(case["batch"], n, nq, nkv, hd)
    return s


# ---------------------------------------------------------------- plain forms
def _row_requests(s):
    """Request and index inside its chunk of every row."""
    row = torch.arange(s["n"], device="cuda", dtype=torch.int32)
    req = torch.searchsorted(s["cu_rows"], row, right=True).long() - 1
    return req, row.long() - s["cu_rows"][req].long()


def _norm_rope(x, g, rope, pos):
    """RMSNorm over the head (when g is given) and the rotate-half rotation, in 32 bits."""
    y = x.float()
    if g is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * g.float()
    c, sn = rope[0][pos][:, None, :], rope[1][pos][:, None, :]
    a, b = y.chunk(2, -1)
    return torch.cat((a * c - b * sn, b * c + a * sn), -1)


def _plain_attention(s):
    case = s["case"]
    nq, nkv, hd, b = case["nq"], case["nkv"], case["hd"], case["batch"]
    G = nq // nkv
    req, i = _row_requests(s)
    rmax = int(case["first_rows"] or 0)
    rmax = max(rmax, case["rows_hi"])
    q = torch.zeros(b, rmax, nq, hd, device="cuda")
    q[req, i] = s["q"].float()
    q = q.view(b, rmax, nkv, G, hd).permute(0, 2, 3, 1, 4).reshape(b, nkv, G * rmax, hd)
    table = s["table"].long().clamp(min=0)

    def dense(pool):  # [b, nkv, T, hd]
        return pool[table].permute(0, 2, 1, 3, 4).reshape(b, nkv, -1, hd).float()

    sc = torch.matmul(q, dense(s["k_pool"]).transpose(-1, -2)).mul_(hd ** -0.5)
    T = sc.shape[-1]
    pos = s["start_pos"].long()[:, None] + torch.arange(rmax, device="cuda")  # [b, rmax]
    key = torch.arange(T, device="cuda")
    seen = (key < s["kv_len"].long()[:, None])[:, None, :].expand(b, rmax, T)
    if case["causal"]:
        seen = seen & (key <= pos[:, :, None])
    if case["window"]:
        seen = seen & (key > pos[:, :, None] - case["window"])
    sc = sc.view(b, nkv, G, rmax, T).masked_fill_(~seen[:, None, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = sc.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, nkv, G * rmax, T), dense(s["v_pool"])).view(b, nkv, G, rmax, hd)
    o = torch.where(l > 0, o / l, torch.zeros_like(o))
    out = o.permute(0, 3, 1, 2, 4).reshape(b, rmax, nq, hd)[req, i].to(s["q"].dtype)
    lse = (m + l.log())[..., 0].permute(0, 3, 1, 2).reshape(b, rmax, nq)[req, i]
    return (out, lse) if case["lse"] else out


def _plain(s):
    case = s["case"]
    if case["op"] == "attention":
        return _plain_attention(s)
    req, i = _row_requests(s)
    pos = s["start_pos"].long()[req] + i
    k = _norm_rope(s["k"], s["g_k"], s["rope"], pos)
    if case["op"] == "qk":
        return _norm_rope(s["q"], s["g_q"], s["rope"], pos).to(s["q"].dtype), k.to(s["k"].dtype)
    page, slot = s["table"][req, pos // case["page"]].long(), pos % case["page"]
    s["k_pool"][page, :, slot] = k.to(s["k_pool"].dtype)
    s["v_pool"][page, :, slot] = s["v"].float().to(s["v_pool"].dtype)
    return s["k_pool"], s["v_pool"]


def run(s):
    if not own:
        return _plain(s)
    case, D = s["case"], s["D"]
    if case["op"] == "qk":
        D.qk_norm_rope(s["q"], s["k"], s["g_q"], s["g_k"], s["rope"], s["cu_rows"],
                       s["start_pos"], s["q_out"], s["k_out"], s["ws"], eps=EPS)
        return s["q_out"], s["k_out"]
    if case["op"] == "append":
        D.kv_append_paged(s["k"], s["v"], s["g_k"], s["rope"], s["cu_rows"], s["start_pos"],
                          s["k_pool"], s["v_pool"], s["table"], s["ws"], eps=EPS)
        return s["k_pool"], s["v_pool"]
    D.attention_paged(s["q"], s["cu_rows"], s["start_pos"], s["kv_len"], s["k_pool"],
                      s["v_pool"], s["table"], s["out"], s["ws"], causal=case["causal"],
                      window=case["window"], lse=s["lse"])
    return (s["out"], s["lse"]) if case["lse"] else s["out"]


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    """From the definitions in 64 bits, request by request."""
    s = prepare(case, seed)
    rows, ctx = _lengths(case)
    nq, nkv, hd = case["nq"], case["nkv"], case["hd"]
    half = hd // 2
    freq = torch.tensor([ROPE_BASE ** (-2.0 * j / hd) for j in range(half)], dtype=torch.float64,
                        device="cuda")

    def turn(x, g, pos):
        y = x.double()
        if g is not None:
            y = y / torch.sqrt(y.square().sum(-1, keepdim=True) / hd + EPS) * g.double()
        z = torch.complex(y[..., :half], y[..., half:])
        ang = pos.double()[:, None] * freq
        z = z * torch.polar(torch.ones_like(ang), ang)[:, None, :]
        return torch.cat((z.real, z.imag), -1)

    res, res2, first = [], [], 0
    kp, vp = (s[x].double() if x in s else None for x in ("k_pool", "v_pool"))
    for r, (n, t) in enumerate(zip(rows, ctx)):
        part = slice(first, first + n)
        first += n
        pos = torch.arange(t, t + n, device="cuda")
        if case["op"] == "qk":
            res.append(turn(s["q"][part], s["g_q"], pos))
            res2.append(turn(s["k"][part], s["g_k"], pos))
            continue
        P = case["page"]
        pages = s["table"][r, : -(-(t + n) // P)].long()
        if case["op"] == "append":
            at, slot = pages[torch.div(pos, P, rounding_mode="floor")], pos % P
            kp[at, :, slot] = turn(s["k"][part], s["g_k"], pos)
            vp[at, :, slot] = s["v"][part].double()
            continue
        key = torch.arange(t + n, device="cuda")
        ok = torch.ones(n, t + n, dtype=torch.bool, device="cuda")
        if case["causal"]:
            ok &= key[None, :] <= pos[:, None]
        if case["window"]:
            ok &= key[None, :] > pos[:, None] - case["window"]
        out = torch.empty(n, nq, hd, dtype=torch.float64, device="cuda")
        lse = torch.empty(n, nq, dtype=torch.float64, device="cuda")
        for h in range(nq):
            K = kp[pages, h * nkv // nq].reshape(-1, hd)[: t + n]
            V = vp[pages, h * nkv // nq].reshape(-1, hd)[: t + n]
            z = s["q"][part, h].double() @ K.T / math.sqrt(hd)
            z.masked_fill_(~ok, -math.inf)
            lse[:, h] = torch.logsumexp(z, -1)
            out[:, h] = torch.nan_to_num(torch.softmax(z, -1)) @ V
        res.append(out)
        res2.append(lse)
    if case["op"] == "append":
        return kp, vp
    if case["op"] == "attention" and not case["lse"]:
        return torch.cat(res)
    return torch.cat(res), torch.cat(res2)


# ---------------------------------------------------------------- work
def work(case):
    rows, ctx = _lengths(case)
    n, nq, nkv, hd = sum(rows), case["nq"], case["nkv"], case["hd"]
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "qk":
        # rows in and out, the rotation table's rows
        return {"bytes": 2 * n * (nq + nkv) * hd * e + n * hd * 4,
                "flops": 8 * n * (nq + nkv) * hd}
    if case["op"] == "append":
        return {"bytes": n * 2 * nkv * hd * (e + 2) + n * hd * 4, "flops": 8 * n * nkv * hd}
    pairs, keys = 0, 0
    for a, t in zip(rows, ctx):
        w = case["window"] or a + t
        lo = max(0, t - w + 1)  # the first key any row sees
        keys += a + t - lo
        if case["causal"]:
            # sum over the rows at p = t .. t + a - 1 of min(p + 1, w)
            short = max(0, min(a, w - t))  # rows with p + 1 < = w
            pairs += short * t + short * (short + 1) // 2 + (a - short) * w
        else:
            # keys p - w + 1 .. a + t - 1, from 0 at the least
            short = max(0, min(a, w - t))
            rest = a - short
            pairs += short * (a + t)
            first = t + short  # position of the first row whose window starts behind key 0
            pairs += rest * (a + t + w - 1) - (rest * first + rest * (rest - 1) // 2)
    return {"bytes": 2 * keys * nkv * hd * e + 2 * n * nq * hd * e + (4 * n * nq if case["lse"]
                                                                     else 0),
            "flops": 4 * hd * nq * pairs}
