"""Measured cases of three operators that surround an adapted linear layer: the frozen product over
an E4M3 base with a scale for each block of 128, layer norm with its backward pass, and the
orthogonalised (Newton-Schulz) update of the adapters.

`prepare(case, seed)` makes what a program has in hand before the call, `run(state)` is one call,
either of the library (`own`) or written out in elementary torch operations in 32 bits, `exact`
evaluates the definition in 64 bits, and `work` counts the bytes and operations that a pass cannot
do without.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
BLOCK = 128
NS = (3.4445, -4.7750, 2.0315)   # coefficients of the Newton-Schulz step
NS_STEPS = 5


def listed():
    return [
        # ---- frozen product, E4M3 base with 128-blocks ----
        # one token through a key projection: the smallest call, latency alone
        dict(name="product_decode_kv", op="product", T=1, in_dim=2560, out_dim=1024, dx=False),
        # one token through a wide gate projection: streams the weight
        dict(name="product_decode_gate", op="product", T=1, in_dim=4096, out_dim=14336, dx=False),
        # a serving batch, an odd number of tokens, through a down projection
        dict(name="product_serve_down", op="product", T=37, in_dim=9728, out_dim=2560, dx=False),
        # a training batch forward through a gate projection: the largest product
        dict(name="product_train_fwd", op="product", T=8192, in_dim=4096, out_dim=14336, dx=False),
        # the input gradient of a ragged batch, the contraction not a multiple of the block
        dict(name="product_train_dx_odd", op="product", T=1003, in_dim=2560, out_dim=1552, dx=True),
        # the input gradient of a training batch
        dict(name="product_train_dx", op="product", T=4096, in_dim=1536, out_dim=4096, dx=True),
        # ---- layer norm ----
        # one token in serving
        dict(name="norm_fwd_decode", op="norm", T=1, dim=2560, kind="layer", dtype="bf16", bwd=False),
        # a training batch, forward and backward
        dict(name="norm_fwd_train", op="norm", T=8192, dim=4096, kind="layer", dtype="bf16", bwd=False),
        dict(name="norm_bwd_train", op="norm", T=8192, dim=4096, kind="layer", dtype="bf16", bwd=True),
        # an fp32 model's root-mean-square norm, an odd number of tokens
        dict(name="norm_bwd_f32_rms", op="norm", T=1023, dim=2048, kind="rms", dtype="f32", bwd=True),
        # ---- orthogonalised update ----
        # 22 layers of a key projection's rank-8 adapters
        dict(name="muon_rank8", op="muon", layers=22, in_dim=2048, out_dim=256, rank=8),
        # 32 layers of a gate projection's rank-64 adapters: the largest update
        dict(name="muon_rank64", op="muon", layers=32, in_dim=4096, out_dim=14336, rank=64),
    ]


def _log_int(rng, lo, hi, step=1):
    """An integer of [lo, hi], a multiple of step, spread over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi // step * step, max(-(-lo // step) * step, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["product", "product", "norm", "muon"])
    while True:
        if op == "product":
            c = dict(op=op, T=_log_int(rng, 1, 8192), in_dim=_log_int(rng, 64, 14336, 16),
                     out_dim=_log_int(rng, 64, 14336, 16), dx=rng.random() < 0.5)
            if c["T"] * c["in_dim"] * c["out_dim"] <= 8192 * 4096 * 14336:
                return c
        elif op == "norm":
            c = dict(op=op, T=_log_int(rng, 1, 16384), dim=_log_int(rng, 64, 16384, 8),
                     kind=rng.choice(["layer", "rms"]), dtype=rng.choice(["bf16", "f32"]),
                     bwd=rng.random() < 0.6)
            if c["T"] * c["dim"] * (2 if c["dtype"] == "f32" else 1) <= 8192 * 4096:
                return c
        else:
            c = dict(op=op, layers=_log_int(rng, 1, 32), in_dim=_log_int(rng, 64, 14336, 8),
                     out_dim=_log_int(rng, 64, 14336, 8), rank=4 * rng.randint(1, 16))
            if c["layers"] * c["rank"] * (c["in_dim"] + c["out_dim"]) <= 32 * 64 * (4096 + 14336):
                return c


def work(case):
    if case["op"] == "product":
        T, n_in, n_out = case["T"], case["in_dim"], case["out_dim"]
        scales = 4 * -(-n_in // BLOCK) * -(-n_out // BLOCK)
        return {"bytes": 2 * T * (n_in + n_out) + n_in * n_out + scales, "flops": 2 * T * n_in * n_out}
    if case["op"] == "norm":
        n, el = case["T"] * case["dim"], 2 if case["dtype"] == "bf16" else 4
        vectors = (2 if case["kind"] == "layer" else 1) * 4 * case["dim"]
        if case["bwd"]:   # X, dY and the statistics in, dX out, the weights in, their gradients in and out
            return {"bytes": 3 * n * el + 8 * case["T"] + 4 * case["dim"] + 2 * vectors, "flops": 14 * n}
        return {"bytes": 2 * n * el + 8 * case["T"] + vectors, "flops": 8 * n}
    # parameters and momentum in and out, gradients in; the Gram matrix and one product by a
    # rank x rank matrix are the least a Newton-Schulz sequence can do on the long axis
    n = case["layers"] * case["rank"] * (case["in_dim"] + case["out_dim"])
    return {"bytes": 20 * n, "flops": 4 * case["rank"] * n}


# ------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, T, dim):
    """A residual stream's values: unit normal, one channel in 64 twenty times larger."""
    x = _randn(g, T, dim)
    x[:, ::64] *= 20.0
    return x


def _blocks(x, rows, cols):
    """x [R, C] as [R / rows, rows, C / cols, cols], zeros past its ends."""
    R, C = x.shape
    pad = torch.zeros(-(-R // rows) * rows, -(-C // cols) * cols, dtype=x.dtype, device=x.device)
    pad[:R, :C] = x
    return pad.view(pad.shape[0] // rows, rows, pad.shape[1] // cols, cols)


def _quantize(x, rows, cols):
    """E4M3 codes of x [R, C] and one scale for each rows x cols block: r = 448 / amax,
    codes = e4m3(x r), scale = amax / 448 (r = scale = 1 where amax is 0 or r is not finite)."""
    R, C = x.shape
    b = _blocks(x, rows, cols)
    amax = b.abs().amax(dim=(1, 3))
    r = E4M3_MAX / amax
    fine = (amax > 0) & torch.isfinite(r)
    one = torch.ones_like(amax)
    r, scale = torch.where(fine, r, one), torch.where(fine, amax / E4M3_MAX, one)
    codes = (b * r[:, None, :, None]).to(torch.float8_e4m3fn)
    codes = codes.view(torch.uint8).reshape(b.shape[0] * rows, b.shape[2] * cols)[:R, :C]
    return codes.contiguous(), scale.contiguous()


def _dequantize(codes, scale, rows, cols):
    R, C = codes.shape
    b = _blocks(codes, rows, cols).view(torch.float8_e4m3fn).float() * scale[:, None, :, None]
    return b.view(b.shape[0] * rows, b.shape[2] * cols)[:R, :C]


def _prepare_product(case, g):
    T, n_in, n_out = case["T"], case["in_dim"], case["out_dim"]
    W8, sw = _quantize(_randn(g, n_out, n_in) / math.sqrt(n_in), BLOCK, BLOCK)
    if case["dx"]:
        x = 0.1 * _randn(g, T, n_out)
    else:
        x = _activations(g, T, n_in)
    s = dict(X=x.to(torch.bfloat16), W8=W8, sw=sw)
    if own:
        from bwd_adapter_adamw_gb300 import binding as L
        s["Y"] = torch.empty(T, n_in if case["dx"] else n_out, dtype=torch.bfloat16, device="cuda")
        need = L.lora_block_product_workspace_size(T, n_out, n_in, case["dx"])
        s["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    return s


def _prepare_norm(case, g):
    T, dim, dt = case["T"], case["dim"], torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    layer = case["kind"] == "layer"
    s = dict(X=(_activations(g, T, dim) + 0.25).to(dt), gamma=1.0 + 0.1 * _randn(g, dim), eps=1e-5,
             beta=0.1 * _randn(g, dim) if layer else None)
    if case["bwd"]:
        # the statistics that the forward pass kept; the gradients of earlier chunks
        x = s["X"].float()
        mean = x.mean(dim=1) if layer else torch.zeros(T, device="cuda")
        var = ((x - mean[:, None]) ** 2).mean(dim=1)
        s["stats"] = torch.stack([mean, torch.rsqrt(var + s["eps"])], dim=1).contiguous()
        s["dY"] = (0.1 * _randn(g, T, dim)).to(dt)
        s["dgamma0"] = _randn(g, dim)
        s["dbeta0"] = _randn(g, dim) if layer else None
    if own:
        from bwd_adapter_adamw_gb300 import binding as L
        s["desc"] = L.make_norm_desc(dim, L.LORA_NORM_LAYER if layer else L.LORA_NORM_RMS,
                                     L.LORA_BF16 if case["dtype"] == "bf16" else L.LORA_F32, s["eps"])
        s["out"] = torch.empty(T, dim, dtype=dt, device="cuda")
        if case["bwd"]:
            need = L.lora_norm_backward_workspace_size(s["desc"], T)
            s["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        else:
            s["stats"] = torch.empty(T, 2, device="cuda")
    return s


def _prepare_muon(case, g):
    n, r, n_in, n_out = case["layers"], case["rank"], case["in_dim"], case["out_dim"]
    # gradients whose singular values fall off, as those of a projection over correlated tokens do
    fall = torch.exp(-2.0 * torch.arange(r, device="cuda", dtype=torch.float32) / r)

    def grad(dim):   # [n, r, dim]
        return torch.matmul(_randn(g, n, r, r) * fall, _randn(g, n, r, dim)) / r

    na, nb = n * r * n_in, n * n_out * r
    params = torch.cat([_randn(g, na) * math.sqrt(2.0 / n_in), _randn(g, nb) * 0.1])
    grads = torch.cat([grad(n_in).reshape(-1), grad(n_out).transpose(1, 2).reshape(-1)])
    mom = torch.cat([grad(n_in).reshape(-1), grad(n_out).transpose(1, 2).reshape(-1)]) * 1e-3
    s = dict(params=params, grads=grads, mom=mom, na=na, n=n, r=r, n_in=n_in, n_out=n_out,
             scale_norm=torch.tensor([1.0 / 1024, 1.0], dtype=torch.float64, device="cuda"),
             status=torch.zeros(1, dtype=torch.int32, device="cuda"),
             lr=2e-3, wd=0.01, mu=0.95, ratio=4.0)
    if own:
        from bwd_adapter_adamw_gb300 import binding as L
        s["groups"] = L.make_groups([dict(offset=0, n_a=na, n_b=nb, grad_scale=1.0 / 1024, max_norm=1.0,
                                          lr=s["lr"], step=10)])
        mats = [dict(offset=i * r * n_in, rows=r, cols=n_in, kind=L.LORA_KIND_A) for i in range(n)]
        mats += [dict(offset=na + i * n_out * r, rows=n_out, cols=r, kind=L.LORA_KIND_B) for i in range(n)]
        s["mats"] = L.make_mats(mats)
        s["hp"] = L.make_muon_hp(momentum=s["mu"], weight_decay=s["wd"], plus_ratio=s["ratio"])
        need = L.lora_muon_workspace_size(s["mats"])
        s["ws"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    return s


def prepare(case, seed):
    make = {"product": _prepare_product, "norm": _prepare_norm, "muon": _prepare_muon}[case["op"]]
    return dict(make(case, _gen(seed)), case=case)


# ------------------------------------------------------------------------------- one call
def _run_own(s):
    from bwd_adapter_adamw_gb300 import binding as L
    c = s["case"]
    if c["op"] == "product":
        L.lora_block_product(c["T"], c["out_dim"], c["in_dim"], s["X"], s["W8"], s["sw"], s["Y"], c["dx"], s["ws"])
        return s["Y"]
    if c["op"] == "norm" and not c["bwd"]:
        L.lora_norm_forward(s["desc"], c["T"], s["X"], s["gamma"], s["beta"], s["out"], s["stats"])
        return s["out"], s["stats"]
    if c["op"] == "norm":
        dgamma = s["dgamma0"].clone()
        dbeta = None if s["dbeta0"] is None else s["dbeta0"].clone()
        L.lora_norm_backward(s["desc"], c["T"], s["X"], s["gamma"], s["dY"], s["stats"], None, s["out"],
                             dgamma, dbeta, s["ws"])
        return (s["out"], dgamma) if dbeta is None else (s["out"], dgamma, dbeta)
    L.lora_muon_step(s["params"], s["grads"], s["mom"], s["groups"], s["mats"], s["hp"], s["scale_norm"],
                     s["status"], False, s["ws"])
    return s["params"], s["mom"]


def _plain_product(s, dx):
    X8, sx = _quantize(s["X"].float(), 1, BLOCK)
    x = _dequantize(X8, sx, 1, BLOCK)
    w = _dequantize(s["W8"], s["sw"], BLOCK, BLOCK)
    return (x @ w if dx else x @ w.t()).to(torch.bfloat16)


def _plain_norm_forward(s):
    x = s["X"].float()
    layer = s["beta"] is not None
    mean = x.mean(dim=1, keepdim=True) if layer else torch.zeros_like(x[:, :1])
    xc = x - mean
    rstd = 1.0 / torch.sqrt((xc * xc).mean(dim=1, keepdim=True) + s["eps"])
    y = xc * rstd * s["gamma"]
    if layer:
        y = y + s["beta"]
    return y.to(s["X"].dtype), torch.cat([mean, rstd], dim=1)


def _plain_norm_backward(s):
    x, dy = s["X"].float(), s["dY"].float()
    mean, rstd = s["stats"][:, :1], s["stats"][:, 1:]
    xhat = (x - mean) * rstd
    g = dy * s["gamma"]
    dx = g - xhat * (g * xhat).mean(dim=1, keepdim=True)
    dgamma = s["dgamma0"] + (dy * xhat).sum(dim=0)
    if s["dbeta0"] is None:
        return (dx * rstd).to(s["X"].dtype), dgamma
    dx = (dx - g.mean(dim=1, keepdim=True)) * rstd
    return dx.to(s["X"].dtype), dgamma, s["dbeta0"] + dy.sum(dim=0)


def _orthogonalize(u):
    """Newton-Schulz sequence of u [n, r, dim], r <= dim, from u / ||u||."""
    a, b, c = NS
    norm = u.square().sum(dim=(1, 2), keepdim=True).sqrt()
    x = u / torch.where(norm > 0, norm, torch.ones_like(norm))
    for _ in range(NS_STEPS):
        gram = x @ x.transpose(1, 2)
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x


def _plain_muon(s):
    n, r, n_in, n_out, na = s["n"], s["r"], s["n_in"], s["n_out"], s["na"]
    c = s["scale_norm"][0].float()
    gh = c * s["grads"]
    s["mom"].mul_(s["mu"]).add_(gh)
    u = gh + s["mu"] * s["mom"]
    uA, uB = u[:na].view(n, r, n_in), u[na:].view(n, n_out, r)
    oA = _orthogonalize(uA)
    oB = _orthogonalize(uB.transpose(1, 2)).transpose(1, 2)
    p, lr = s["params"], s["lr"]
    p[:na] -= lr * s["wd"] * p[:na] + lr * math.sqrt(max(1.0, r / n_in)) * oA.reshape(-1)
    p[na:] -= lr * s["ratio"] * math.sqrt(max(1.0, n_out / r)) * oB.reshape(-1)
    return p, s["mom"]


def run(state):
    if own:
        return _run_own(state)
    c = state["case"]
    if c["op"] == "product":
        return _plain_product(state, c["dx"])
    if c["op"] == "norm":
        return _plain_norm_backward(state) if c["bwd"] else _plain_norm_forward(state)
    return _plain_muon(state)


# --------------------------------------------------------------------- the definition in 64 bits
def _e4m3_round(v):
    """The nearest E4M3 value (ties to even) of v in float64."""
    _, e = torch.frexp(v)
    ulp = torch.exp2((e - 1).clamp(min=-6).double() - 3.0)
    return (torch.round(v / ulp) * ulp).clamp(-E4M3_MAX, E4M3_MAX)


def _e4m3_value(codes):
    """Values of E4M3 codes in float64: sign, 4 exponent bits (bias 7), 3 fraction bits."""
    c = codes.to(torch.int64)
    e, f = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e > 0, (8.0 + f) * torch.exp2(e.double() - 10.0), f * 2.0 ** -9)
    return torch.where(c >= 128, -mag, mag)


def _exact_product(s, dx):
    x = s["X"].float()
    T, K = x.shape
    nb = -(-K // BLOCK)
    ids = torch.arange(K, device="cuda") // BLOCK
    amax = torch.zeros(T, nb, device="cuda").index_reduce_(1, ids, x.abs(), "amax")
    # the scales and the scaled values are 32-bit numbers by definition
    r, sc = E4M3_MAX / amax, amax / E4M3_MAX
    plain = ~((amax > 0) & torch.isfinite(r))
    r, sc = r.masked_fill(plain, 1.0), sc.masked_fill(plain, 1.0)
    xq = _e4m3_round((x * r[:, ids]).double()) * sc.double()[:, ids]
    rows = torch.arange(s["W8"].shape[0], device="cuda") // BLOCK
    cols = torch.arange(s["W8"].shape[1], device="cuda") // BLOCK
    w = _e4m3_value(s["W8"]) * s["sw"].double()[rows][:, cols]
    return xq @ w if dx else xq @ w.t()


def _exact_norm(s, case):
    x = s["X"].double()
    layer = case["kind"] == "layer"
    gamma = s["gamma"].double()
    if not case["bwd"]:
        mean = x.mean(1) if layer else torch.zeros(x.shape[0], device="cuda", dtype=torch.float64)
        rstd = ((x - mean[:, None]).square().mean(1) + s["eps"]) ** -0.5
        y = (x - mean[:, None]) * rstd[:, None] * gamma
        return (y + s["beta"].double() if layer else y), torch.stack([mean, rstd], dim=1)
    mean, rstd = s["stats"].double().unbind(1)
    dy = s["dY"].double()
    xhat = torch.einsum("td,t->td", x - mean[:, None], rstd)
    g = torch.einsum("td,d->td", dy, gamma)
    proj = torch.einsum("td,td->t", g, xhat) / x.shape[1]
    dx = g - torch.einsum("t,td->td", proj, xhat)
    if layer:
        dx = dx - g.mean(1)[:, None]
    dx = torch.einsum("td,t->td", dx, rstd)
    dgamma = s["dgamma0"].double() + torch.einsum("td,td->d", dy, xhat)
    return (dx, dgamma, s["dbeta0"].double() + dy.sum(0)) if layer else (dx, dgamma)


def _exact_muon(s):
    a, b, c = NS
    na, n = s["na"], s["n"]
    g = s["grads"].double() * s["scale_norm"][0]
    m = s["mu"] * s["mom"].double() + g
    u = g + s["mu"] * m
    p = s["params"].double()

    def update(lo, hi, rows, cols):
        x = u[lo:hi].view(n, rows, cols)
        norm = x.flatten(1).norm(dim=1)
        x = x / norm.where(norm > 0, torch.ones_like(norm))[:, None, None]
        for _ in range(NS_STEPS):   # on the smaller side's Gram matrix
            if rows <= cols:
                q = torch.einsum("nij,nkj->nik", x, x)
                x = a * x + torch.einsum("nij,njk->nik", b * q + c * torch.bmm(q, q), x)
            else:
                q = torch.einsum("nji,njk->nik", x, x)
                x = a * x + torch.einsum("nij,njk->nik", x, b * q + c * torch.bmm(q, q))
        return math.sqrt(max(1.0, rows / cols)) * x.reshape(-1)

    lr = s["lr"]
    pa = p[:na] - lr * s["wd"] * p[:na] - lr * update(0, na, s["r"], s["n_in"])
    pb = p[na:] - lr * s["ratio"] * update(na, u.numel(), s["n_out"], s["r"])
    return torch.cat([pa, pb]), m


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "product":
        return _exact_product(s, case["dx"])
    if case["op"] == "norm":
        return _exact_norm(s, case)
    return _exact_muon(s)
