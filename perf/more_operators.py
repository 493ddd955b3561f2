"""Measured cases of the two operators between an attention block's projections: the norm of each
query and key head with the rotation by position in the same pass, and causal attention over packed
sequences with grouped heads, each forward and backward.

`prepare(case, seed)` makes what a program has in hand before the call, `run(state)` is one call,
either of the library (`own`) or written out in elementary torch operations in 32 bits, `exact`
evaluates the definition in 64 bits, and `work` counts the bytes and operations that a pass cannot
do without.
"""
import math
import random

import torch

own = False

EPS = 1e-6
ROPE_BASE = 1e6
ROW_BLOCK = 2048            # query rows of the plain form's score matrices
SCORE_ELEMENTS = 1 << 28    # elements of a score matrix held at once
EXACT_FLOPS = 3e12          # cases above it take too long in 64 bits


def listed():
    return [
        # ---- norm of the query and key heads, rotation by position ----
        # one decoded token: latency alone
        dict(name="rope_decode", op="rope", T=1, q_heads=32, kv_heads=8, dim=128, dtype="bf16", norm=True,
             pairs=False, fused=True, bwd=False),
        # a training batch of a fused query/key/value projection
        dict(name="rope_fwd_train", op="rope", T=8192, q_heads=32, kv_heads=8, dim=128, dtype="bf16", norm=True,
             pairs=False, fused=True, bwd=False),
        # its gradients, those of the norms' weights among them
        dict(name="rope_bwd_train", op="rope", T=8192, q_heads=32, kv_heads=8, dim=128, dtype="bf16", norm=True,
             pairs=False, fused=True, bwd=True),
        # an fp32 model with small heads, neighbouring elements turned, an odd number of tokens
        dict(name="rope_bwd_f32_pairs", op="rope", T=1023, q_heads=32, kv_heads=4, dim=64, dtype="f32", norm=True,
             pairs=True, fused=False, bwd=True),
        # ---- causal attention over packed sequences ----
        # one short prompt: the smallest call
        dict(name="attn_fwd_prompt", op="attn", tokens=17, lo=17, hi=17, lens_seed=0, pad=0, q_heads=32, kv_heads=8,
             dim=128, fused=True, bwd=False),
        # a microbatch of eight sequences of 128 tokens, small heads
        dict(name="attn_fwd_micro", op="attn", tokens=1024, lo=128, hi=128, lens_seed=0, pad=0, q_heads=32, kv_heads=4,
             dim=64, fused=False, bwd=False),
        # one training sequence
        dict(name="attn_fwd_train", op="attn", tokens=8192, lo=8192, hi=8192, lens_seed=0, pad=0, q_heads=32,
             kv_heads=8, dim=128, fused=True, bwd=False),
        # a packed batch of segments of 64 to 1024 tokens
        dict(name="attn_fwd_packed", op="attn", tokens=16384, lo=64, hi=1024, lens_seed=5, pad=0, q_heads=32,
             kv_heads=8, dim=128, fused=False, bwd=False),
        # one long document: the largest forward pass
        dict(name="attn_fwd_long", op="attn", tokens=32768, lo=32768, hi=32768, lens_seed=0, pad=0, q_heads=32,
             kv_heads=8, dim=128, fused=True, bwd=False),
        # the gradients of the microbatch, the packed batch (its last rows are padding) and the sequence
        dict(name="attn_bwd_micro", op="attn", tokens=1024, lo=128, hi=128, lens_seed=0, pad=0, q_heads=32, kv_heads=4,
             dim=64, fused=False, bwd=True),
        dict(name="attn_bwd_packed", op="attn", tokens=16384, lo=64, hi=1024, lens_seed=5, pad=101, q_heads=32,
             kv_heads=8, dim=128, fused=False, bwd=True),
        dict(name="attn_bwd_train", op="attn", tokens=8192, lo=8192, hi=8192, lens_seed=0, pad=0, q_heads=32,
             kv_heads=8, dim=128, fused=True, bwd=True),
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "attn", "attn"])
    while True:
        kv = rng.randint(1, 8)
        heads = dict(q_heads=kv * rng.choice([1, 2, 3, 4, 5, 6, 8]), kv_heads=kv, fused=rng.random() < 0.5)
        if op == "rope":
            c = dict(op=op, T=_log_int(rng, 1, 16384), dim=rng.choice([64, 128]), dtype=rng.choice(["bf16", "f32"]),
                     norm=rng.random() < 0.7, pairs=rng.random() < 0.4, bwd=rng.random() < 0.5, **heads)
            size = c["T"] * (c["q_heads"] + kv) * c["dim"] * (2 if c["dtype"] == "f32" else 1)
            if size <= 8192 * 40 * 128:
                return c
        else:
            tokens = _log_int(rng, 1, 32768)
            hi = _log_int(rng, 1, tokens)
            c = dict(op=op, tokens=tokens, lo=rng.randint(max(1, hi // 16), hi), hi=hi, lens_seed=rng.randrange(1 << 30),
                     pad=rng.choice([0, 0, rng.randint(1, 300)]), dim=rng.choice([64, 128, 128]),
                     bwd=rng.random() < 0.5, **heads)
            most = 4 * 32 * 128 * (8192 * 8193 / 2) * (2.5 if c["bwd"] else 4)
            if len(_lengths(c)) <= 2048 and work(c)["flops"] <= most:
                return c


def _lengths(case):
    """The lengths of an attention case's sequences: uniform in [lo, hi], the last one cut to the sum."""
    rng, left, out = random.Random(case["lens_seed"]), case["tokens"], []
    while left:
        out.append(min(left, rng.randint(case["lo"], case["hi"])))
        left -= out[-1]
    return out


def work(case):
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "rope":
        n, el = case["T"] * (hq + hk) * d, 2 if case["dtype"] == "bf16" else 4
        shared = case["T"] * (4 + 4 * d)   # positions and their cosines and sines
        vectors = (4 if case["bwd"] else 2) * 4 * d if case["norm"] else 0
        tensors = 3 if case["bwd"] and case["norm"] else 2
        return {"bytes": tensors * n * el + shared + vectors, "flops": (20 if case["bwd"] else 10) * n}
    t = case["tokens"]
    scores = sum(n * (n + 1) // 2 for n in _lengths(case)) * hq
    rows_q, rows_k = 2 * t * hq * d, 2 * t * hk * d
    if case["bwd"]:   # q, k, v, o, do and the statistics in, dq, dk, dv out; five products
        return {"bytes": 4 * rows_q + 4 * rows_k + 4 * t * hq, "flops": 10 * d * scores}
    return {"bytes": 2 * rows_q + 2 * rows_k + 4 * t * hq, "flops": 4 * d * scores}


# ------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _heads_of(buf, at, heads, dim):
    """Columns of a [T, width] buffer as [T, heads, dim], without a copy."""
    return buf[:, at:at + heads * dim].unflatten(1, (heads, dim))


def _split(buf, counts, dim):
    out, at = [], 0
    for n in counts:
        out.append(_heads_of(buf, at, n, dim))
        at += n * dim
    return out


def _place(make, rows, counts, dim, fused):
    """One [rows, heads, dim] tensor for each count: columns of one buffer (a fused projection's), or
    tensors of their own."""
    if fused:
        return _split(make(rows, sum(counts) * dim), counts, dim)
    return [make(rows, n * dim).unflatten(1, (n, dim)) for n in counts]


def _rope_table(positions, dim):
    """Cosines and sines [positions, dim / 2, 2], the angles in 64 bits."""
    inv = ROPE_BASE ** (-torch.arange(0, dim, 2, device="cuda", dtype=torch.float64) / dim)
    a = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * inv
    return torch.stack([a.cos(), a.sin()], dim=2).float().contiguous()


def _prepare_rope(case, g):
    T, hq, hk, d = case["T"], case["q_heads"], case["kv_heads"], case["dim"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    counts = [hq, hk, hk] if case["fused"] else [hq, hk]   # a fused buffer holds the values, too
    x = _place(lambda r, c: (2.0 * _randn(g, r, c)).to(dt), T, counts, d, case["fused"])
    n_pos = max(2 * T, 4096)
    # positions of two sequences, the second from the table's start, or of a decoded token far behind it
    pos = (torch.arange(T, device="cuda", dtype=torch.int32) + 2 * n_pos // 3) % n_pos
    s = dict(q=x[0], k=x[1], pos=pos, table=_rope_table(n_pos, d), n_pos=n_pos)
    s["gq"] = 1.0 + 0.1 * _randn(g, d) if case["norm"] else None
    s["gk"] = 1.0 + 0.1 * _randn(g, d) if case["norm"] else None
    if case["bwd"]:
        s["dyq"], s["dyk"] = (0.1 * _randn(g, T, hq, d)).to(dt), (0.1 * _randn(g, T, hk, d)).to(dt)
        s["dgq0"] = _randn(g, d) if case["norm"] else None
        s["dgk0"] = _randn(g, d) if case["norm"] else None
    if own:
        from bwd_adapter_adamw_gb300 import binding as L
        ld = s["q"].stride(0), s["k"].stride(0)
        s["desc"] = L.make_rope_desc(hq, hk, d, L.LORA_BF16 if case["dtype"] == "bf16" else L.LORA_F32,
                                     L.LORA_ROPE_PAIRS if case["pairs"] else L.LORA_ROPE_HALVES, EPS, ld_q=ld[0],
                                     ld_k=ld[1])
        if case["bwd"]:
            s["dq"], s["dk"] = _place(lambda r, c: torch.empty(r, c, dtype=dt, device="cuda"), T, counts, d,
                                      case["fused"])[:2]
            need = L.lora_rope_backward_workspace_size(s["desc"], T)
            s["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        else:
            s["yq"] = torch.empty(T, hq, d, dtype=dt, device="cuda")
            s["yk"] = torch.empty(T, hk, d, dtype=dt, device="cuda")
    return s


def _prepare_attn(case, g):
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
    lens = _lengths(case)
    T = case["tokens"] + case["pad"]
    # queries and keys behind their norms, spread enough for rows whose weight lies on a few keys
    x = _place(lambda r, c: (1.5 * _randn(g, r, c)).to(torch.bfloat16), T, [hq, hk, hk], d, case["fused"])
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    s = dict(q=x[0], k=x[1], v=x[2], starts=starts, T=T, scale=1.0 / math.sqrt(d),
             seq_start=torch.tensor(starts, dtype=torch.int32, device="cuda"))
    if case["bwd"]:
        o, lse = _plain_attn_forward(s, case)
        s["o"], s["lse"] = o, lse
        s["do"] = (0.1 * _randn(g, T, hq, d)).to(torch.bfloat16)
    if own:
        from bwd_adapter_adamw_gb300 import binding as L
        s["desc"] = L.make_attn_desc(hq, hk, d, scale=s["scale"], ld_q=s["q"].stride(0), ld_k=s["k"].stride(0),
                                     ld_v=s["v"].stride(0))
        s["plan"] = torch.empty(L.lora_attn_plan_size(T, len(lens)), dtype=torch.uint8, device="cuda")
        L.lora_attn_plan_build(T, len(lens), s["seq_start"], s["plan"])
        if case["bwd"]:
            s["dq"], s["dk"], s["dv"] = _place(lambda r, c: torch.zeros(r, c, dtype=torch.bfloat16, device="cuda"), T,
                                               [hq, hk, hk], d, case["fused"])
            need = L.lora_attn_backward_workspace_size(s["desc"], T)
            s["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        else:
            s["o"] = torch.zeros(T, hq, d, dtype=torch.bfloat16, device="cuda")
            s["lse"] = torch.zeros(hq, T, device="cuda")
    return s


def prepare(case, seed):
    make = _prepare_rope if case["op"] == "rope" else _prepare_attn
    return dict(make(case, _gen(seed)), case=case)


# ------------------------------------------------------------------------------- one call
def _run_own(s):
    from bwd_adapter_adamw_gb300 import binding as L
    c = s["case"]
    if c["op"] == "rope" and not c["bwd"]:
        L.lora_rope_forward(s["desc"], c["T"], s["q"], s["k"], s["gq"], s["gk"], s["pos"], s["table"], s["n_pos"],
                            s["yq"], s["yk"])
        return s["yq"], s["yk"]
    if c["op"] == "rope":
        dgq, dgk = (s["dgq0"].clone(), s["dgk0"].clone()) if c["norm"] else (None, None)
        L.lora_rope_backward(s["desc"], c["T"], s["q"], s["k"], s["gq"], s["gk"], s["pos"], s["table"], s["n_pos"],
                             s["dyq"], s["dyk"], s["dq"], s["dk"], dgq, dgk, s["ws"])
        return (s["dq"], s["dk"], dgq, dgk) if c["norm"] else (s["dq"], s["dk"])
    n_seq = len(s["starts"]) - 1
    if not c["bwd"]:
        L.lora_attn_forward(s["desc"], s["T"], n_seq, s["plan"], s["q"], s["k"], s["v"], s["o"], s["lse"])
        return s["o"], s["lse"]
    L.lora_attn_backward(s["desc"], s["T"], n_seq, s["plan"], s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"],
                         s["dq"], s["dk"], s["dv"], s["ws"])
    return s["dq"], s["dk"], s["dv"]


def _turn(x, cos, sin, pairs):
    """x [T, heads, dim] with each pair of elements turned by its angle."""
    a, b = (x[..., 0::2], x[..., 1::2]) if pairs else x.chunk(2, dim=-1)
    u, v = a * cos - b * sin, a * sin + b * cos
    return torch.stack([u, v], dim=-1).flatten(-2) if pairs else torch.cat([u, v], dim=-1)


def _plain_rope(s, c):
    cs = s["table"][s["pos"].long()][:, None]
    cos, sin = cs[..., 0], cs[..., 1]
    out, sums = [], []
    for x, gamma, dy, dg0 in ((s["q"], s["gq"], s.get("dyq"), s.get("dgq0")),
                              (s["k"], s["gk"], s.get("dyk"), s.get("dgk0"))):
        dt = x.dtype
        if c["norm"]:
            xf = x.float()
            rstd = 1.0 / torch.sqrt((xf * xf).mean(dim=-1, keepdim=True) + EPS)
            xhat = xf * rstd
        if not c["bwd"]:
            out.append(_turn(xhat * gamma if c["norm"] else x.float(), cos, sin, c["pairs"]).to(dt))
            continue
        g = _turn(dy.float(), cos, -sin, c["pairs"])
        if c["norm"]:
            sums.append(dg0 + (g * xhat).sum(dim=(0, 1)))
            g = g * gamma
            g = rstd * (g - xhat * (g * xhat).mean(dim=-1, keepdim=True))
        out.append(g.to(dt))
    return (*out, *sums)


def _blocks(s, c):
    """Pieces of the score matrices: rows a .. b of a sequence from row t0, query heads h0 .. h1."""
    hq, per = c["q_heads"], c["q_heads"] // c["kv_heads"]
    for t0, t1 in zip(s["starts"], s["starts"][1:]):
        for a in range(0, t1 - t0, ROW_BLOCK):
            b = min(a + ROW_BLOCK, t1 - t0)
            step = max(1, min(hq, SCORE_ELEMENTS // ((b - a) * b)) // per) * per
            for h0 in range(0, hq, step):
                yield t0, a, b, h0, min(hq, h0 + step)


def _kv_of(x, t0, b, h0, h1, per):
    """Rows t0 .. t0 + b of the key or value heads of query heads h0 .. h1, in 32 bits, [heads, b, dim]."""
    return x[t0:t0 + b, h0 // per:h1 // per].float().transpose(0, 1).repeat_interleave(per, dim=0)


def _plain_scores(s, t0, a, b, h0, h1, per):
    q = s["q"][t0 + a:t0 + b, h0:h1].float().transpose(0, 1)
    k = _kv_of(s["k"], t0, b, h0, h1, per)
    scores = (q @ k.transpose(1, 2)) * s["scale"]
    late = torch.arange(b, device="cuda")[None, :] > torch.arange(a, b, device="cuda")[:, None]
    return q, k, scores.masked_fill_(late, float("-inf"))


def _plain_attn_forward(s, c):
    hq, per = c["q_heads"], c["q_heads"] // c["kv_heads"]
    o = torch.zeros(s["T"], hq, c["dim"], dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(hq, s["T"], device="cuda")
    for t0, a, b, h0, h1 in _blocks(s, c):
        _, _, p = _plain_scores(s, t0, a, b, h0, h1, per)
        top = p.amax(dim=-1, keepdim=True)
        p = p.sub_(top).exp_()
        total = p.sum(dim=-1, keepdim=True)
        v = _kv_of(s["v"], t0, b, h0, h1, per)
        o[t0 + a:t0 + b, h0:h1] = ((p @ v) / total).transpose(0, 1).to(torch.bfloat16)
        lse[h0:h1, t0 + a:t0 + b] = (top + total.log())[..., 0]
    return o, lse


def _plain_attn_backward(s, c):
    hq, hk, d = c["q_heads"], c["kv_heads"], c["dim"]
    per = hq // hk
    dq = torch.zeros(s["T"], hq, d, dtype=torch.bfloat16, device="cuda")
    dk, dv = torch.zeros(2, s["T"], hk, d, device="cuda").unbind(0)
    for t0, a, b, h0, h1 in _blocks(s, c):
        q, k, p = _plain_scores(s, t0, a, b, h0, h1, per)
        rows, kv = slice(t0 + a, t0 + b), slice(h0 // per, h1 // per)
        p = p.sub_(s["lse"][h0:h1, rows, None]).exp_()
        do = s["do"][rows, h0:h1].float().transpose(0, 1)
        o = s["o"][rows, h0:h1].float().transpose(0, 1)
        dv[t0:t0 + b, kv] += (p.transpose(1, 2) @ do).unflatten(0, (-1, per)).sum(dim=1).transpose(0, 1)
        dp = do @ _kv_of(s["v"], t0, b, h0, h1, per).transpose(1, 2)
        ds = p.mul_(dp.sub_((do * o).sum(dim=-1, keepdim=True)))
        dq[rows, h0:h1] = ((ds @ k) * s["scale"]).transpose(0, 1).to(torch.bfloat16)
        dk[t0:t0 + b, kv] += (ds.transpose(1, 2) @ q).unflatten(0, (-1, per)).sum(dim=1).transpose(0, 1) * s["scale"]
    return dq, dk.to(torch.bfloat16), dv.to(torch.bfloat16)


def run(state):
    if own:
        return _run_own(state)
    c = state["case"]
    if c["op"] == "rope":
        return _plain_rope(state, c)
    return _plain_attn_backward(state, c) if c["bwd"] else _plain_attn_forward(state, c)


# --------------------------------------------------------------------- the definition in 64 bits
def _exact_rope(s, c):
    cs = torch.view_as_complex(s["table"].double())[s["pos"].long()]   # e^(i angle), [T, dim / 2]
    d = c["dim"]
    order = torch.arange(d, device="cuda")
    order = order.view(-1, 2) if c["pairs"] else order.view(2, -1).t()   # the elements of each pair
    dy = s.get("dyq"), s.get("dyk")
    out, sums = [], []
    for i, (x, gamma) in enumerate(((s["q"], s["gq"]), (s["k"], s["gk"]))):
        x = x.double()
        w = gamma.double() if c["norm"] else torch.ones(d, device="cuda", dtype=torch.float64)
        r = (x.square().mean(-1) + EPS) ** -0.5 if c["norm"] else torch.ones_like(x[..., 0])
        source = torch.einsum("thd,th,d->thd", x, r, w) if not c["bwd"] else dy[i].double()
        turn = cs if not c["bwd"] else cs.conj()
        z = torch.view_as_complex(source[..., order].contiguous()) * turn[:, None]
        y = torch.empty_like(x)
        y[..., order] = torch.view_as_real(z)
        if c["bwd"] and c["norm"]:
            sums.append((s["dgq0"], s["dgk0"])[i].double() + torch.einsum("thd,thd,th->d", y, x, r))
            y = torch.einsum("thd,d->thd", y, w)
            y = torch.einsum("thd,th->thd", y, r) - torch.einsum("thd,th->thd", x, r ** 3 * (y * x).mean(-1))
        out.append(y)
    return (*out, *sums)


def _exact_attn(s, c):
    """One query head at a time, in runs of rows."""
    hq, d, T = c["q_heads"], c["dim"], s["T"]
    per = hq // c["kv_heads"]
    new = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device="cuda")   # noqa: E731
    o, lse = new(T, hq, d), new(hq, T)
    dq, dk, dv = new(T, hq, d), new(T, hq // per, d), new(T, hq // per, d)
    for first, last in zip(s["starts"], s["starts"][1:]):
        for h in range(hq):
            k, v = s["k"][first:last, h // per].double(), s["v"][first:last, h // per].double()
            for r0 in range(first, last, 4096):
                r1 = min(last, r0 + 4096)
                n = r1 - first
                z = torch.einsum("id,jd->ij", s["q"][r0:r1, h].double(), k[:n]) * s["scale"]
                allowed = torch.ones(r1 - r0, n, dtype=torch.bool, device="cuda").tril(r0 - first)
                if not c["bwd"]:
                    lse[h, r0:r1] = torch.logsumexp(z.where(allowed, -torch.inf), dim=1)
                    w = torch.exp(z - lse[h, r0:r1, None]) * allowed
                    o[r0:r1, h] = torch.einsum("ij,jd->id", w, v[:n])
                    continue
                w = torch.exp(z.where(allowed, -torch.inf) - s["lse"][h, r0:r1, None].double())
                g = s["do"][r0:r1, h].double()
                dv[first:r1, h // per] += torch.einsum("ij,id->jd", w, g)
                delta = torch.einsum("id,id->i", g, s["o"][r0:r1, h].double())
                w = w * (torch.einsum("id,jd->ij", g, v[:n]) - delta[:, None]) * s["scale"]
                dq[r0:r1, h] = torch.einsum("ij,jd->id", w, k[:n])
                dk[first:r1, h // per] += torch.einsum("ij,id->jd", w, s["q"][r0:r1, h].double())
    return (dq, dk, dv) if c["bwd"] else (o, lse)


def exact(case, seed):
    if case["op"] == "attn" and work(case)["flops"] > EXACT_FLOPS:
        return None
    s = prepare(case, seed)
    return _exact_rope(s, case) if case["op"] == "rope" else _exact_attn(s, case)
