"""Layer norm and RMS norm, forward and backward, against float64.

fp32: a value passes through a few fp32 roundings and sums of at most 16384 terms held in lanes
and trees, so the 2-norm of an output's error stays under 2e-6 of the output's (statistics and
gradients too). bf16 outputs add one rounding: 3e-3.
"""
import numpy as np
import pytest
import torch

from oracle import sublayer_oracle as S

pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bwd_adapter_adamw_gb300 import binding
    return binding


def _inputs(T, dim, dtype, seed):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, dim)) * np.exp(rng.uniform(-2, 2, (T, 1))) + 0.5
    dy = rng.standard_normal((T, dim))
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    return (torch.from_numpy(x).to(dt), torch.from_numpy(dy).to(dt),
            torch.from_numpy(1 + 0.2 * rng.standard_normal(dim)).float(),
            torch.from_numpy(0.2 * rng.standard_normal(dim)).float())


def _desc(L, dim, rms, dtype, eps=EPS):
    return L.make_norm_desc(dim, L.LORA_NORM_RMS if rms else L.LORA_NORM_LAYER,
                            L.LORA_BF16 if dtype == "bf16" else L.LORA_F32, eps)


def _forward(L, d, x, gamma, beta):
    y = torch.empty_like(x, device="cuda")
    st = torch.empty(x.shape[0], 2, device="cuda")
    L.lora_norm_forward(d, x.shape[0], x.cuda(), gamma.cuda(), None if beta is None else beta.cuda(), y, st)
    return y, st


def _backward(L, d, x, gamma, dy, st, add=None, want_dx=True, dg=None, db=None):
    dx = torch.empty_like(x, device="cuda") if want_dx else None
    ws = torch.empty(max(16, L.lora_norm_backward_workspace_size(d, x.shape[0])), dtype=torch.uint8, device="cuda")
    L.lora_norm_backward(d, x.shape[0], x.cuda(), gamma.cuda(), dy.cuda(), st, add, dx, dg, db, ws)
    return dx


def _off(got, ref):
    got = got.double().cpu().numpy()
    return np.linalg.norm(got - ref) / max(np.linalg.norm(ref), 1e-300)


SHAPES = [(1, 8), (1, 2560), (3, 64), (7, 136), (33, 520), (200, 1032), (5, 2056), (17, 4096),
          (2, 8200), (3, 16384), (1023, 256), (2500, 264), (2500, 1544), (2100, 3592)]


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,dim", SHAPES)
def test_forward_and_backward(L, T, dim, dtype, rms):
    x, dy, gamma, beta = _inputs(T, dim, dtype, T * 31 + dim)
    beta = None if rms else beta
    d = _desc(L, dim, rms, dtype)
    y, st = _forward(L, d, x, gamma, beta)
    rng = np.random.default_rng(1)
    g0, b0 = rng.standard_normal(dim).astype(np.float32), rng.standard_normal(dim).astype(np.float32)
    dg = torch.from_numpy(g0).cuda()
    db = None if rms else torch.from_numpy(b0).cuda()
    dx = _backward(L, d, x, gamma, dy, st, dg=dg, db=db)
    torch.cuda.synchronize()
    tol = 2e-6 if dtype == "f32" else 3e-3
    ry, mean, rstd = S.norm_forward(x.double().numpy(), gamma.numpy(), None if rms else beta.numpy(), EPS, rms)
    rdx, rdg, rdb = S.norm_backward(x.double().numpy(), gamma.numpy(), dy.double().numpy(), EPS, rms)
    assert _off(y, ry) <= tol
    # a mean near zero cancels: its error is held against the row's size
    size = np.abs(x.double().numpy()).max(1)
    assert np.all(np.abs(st[:, 0].double().cpu().numpy() - mean) <= 1e-6 * size)
    assert _off(st[:, 1], rstd) <= 2e-6
    # dX of a row of 8 equal-sized terms cancels too: against its terms' size
    ref_size = np.linalg.norm(dy.double().numpy() * gamma.numpy() * rstd[:, None])
    assert np.linalg.norm(dx.double().cpu().numpy() - rdx) <= tol * ref_size
    terms = np.linalg.norm(np.abs(dy.double().numpy() * (x.double().numpy() - mean[:, None]) * rstd[:, None]).sum(0) + np.abs(g0))
    assert np.linalg.norm(dg.double().cpu().numpy() - (g0 + rdg)) <= 2e-6 * terms
    if db is not None:
        assert np.linalg.norm(db.double().cpu().numpy() - (b0 + rdb)) <= 2e-6 * np.linalg.norm(np.abs(dy.double().numpy()).sum(0) + np.abs(b0))


@pytest.mark.parametrize("rms", [False, True])
def test_gradients_against_differences(L, rms):
    """The fp32 gradients against central differences of the float64 forward: h = 1e-4 leaves an
    error of h^2 times a third derivative of order one."""
    T, dim = 5, 24
    x, dy, gamma, beta = _inputs(T, dim, "f32", 3)
    beta = None if rms else beta
    d = _desc(L, dim, rms, "f32")
    _, st = _forward(L, d, x, gamma, beta)
    dg = torch.zeros(dim, device="cuda")
    db = None if rms else torch.zeros(dim, device="cuda")
    dx = _backward(L, d, x, gamma, dy, st, dg=dg, db=db).double().cpu().numpy()
    f = lambda x_, g_, b_: float((S.norm_forward(x_, g_, b_, EPS, rms)[0] * dy.double().numpy()).sum())   # noqa: E731
    X, Gm = x.double().numpy(), gamma.double().numpy()
    B = None if rms else beta.double().numpy()
    h = 1e-4
    for (t, i) in [(0, 0), (2, 5), (4, 23)]:
        e = np.zeros_like(X)
        e[t, i] = h
        assert abs((f(X + e, Gm, B) - f(X - e, Gm, B)) / (2 * h) - dx[t, i]) <= 1e-5 * max(1.0, np.abs(dx[t]).max())
    for i in [0, 7, 23]:
        e = np.zeros(dim)
        e[i] = h
        want = (f(X, Gm + e, B) - f(X, Gm - e, B)) / (2 * h)
        assert abs(want - dg[i].item()) <= 1e-5 * max(1.0, abs(want))
        if not rms:
            want = (f(X, Gm, B + e) - f(X, Gm, B - e)) / (2 * h)
            assert abs(want - db[i].item()) <= 1e-5 * max(1.0, abs(want))


def test_residual_gradient_in_place_and_partial_outputs(L):
    T, dim = 300, 1032
    x, dy, gamma, beta = _inputs(T, dim, "bf16", 4)
    d = _desc(L, dim, False, "bf16")
    _, st = _forward(L, d, x, gamma, beta)
    res = torch.randn(T, dim, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    dg, db = torch.zeros(dim, device="cuda"), torch.zeros(dim, device="cuda")
    both = _backward(L, d, x, gamma, dy, st, add=res, dg=dg, db=db)
    inplace = res.clone()
    ws = torch.empty(L.lora_norm_backward_workspace_size(d, T), dtype=torch.uint8, device="cuda")
    L.lora_norm_backward(d, T, x.cuda(), gamma.cuda(), dy.cuda(), st, inplace, inplace, None, None, ws)
    only = torch.zeros(dim, device="cuda")
    _backward(L, d, x, gamma, dy, st, want_dx=False, dg=only)
    onlyb = torch.zeros(dim, device="cuda")
    _backward(L, d, x, gamma, dy, st, want_dx=False, db=onlyb)
    torch.cuda.synchronize()
    rdx, _, _ = S.norm_backward(x.double().numpy(), gamma.numpy(), dy.double().numpy(), EPS, False)
    assert _off(both, rdx + res.double().cpu().numpy()) <= 3e-3
    assert torch.equal(both, inplace)
    assert torch.equal(dg, only) and torch.equal(db, onlyb)


@pytest.mark.parametrize("rms", [False, True])
def test_constant_rows_zero_rows_and_a_large_mean(L, rms):
    dim = 512
    x = torch.zeros(5, dim)
    x[1] = 3.0                                        # variance zero (layer norm)
    x[2] = 1e4 + torch.randn(dim, generator=torch.Generator().manual_seed(2))   # cancels in x^2
    x[3] = 1e-20
    x[4] = 1e15
    gamma = torch.ones(dim)
    d = _desc(L, dim, rms, "f32")
    y, st = _forward(L, d, x, gamma, None)
    torch.cuda.synchronize()
    ry, _, rstd = S.norm_forward(x.double().numpy(), gamma.numpy(), None, EPS, rms)
    assert torch.isfinite(y).all()
    got = y.double().cpu().numpy()
    for r in range(5):
        # a constant row's centred values are the mean's rounding, up to 2^-23 of it, times rstd
        slack = 0.0 if rms else float(x[r].abs().max()) * 2.0 ** -23 * rstd[r]
        assert np.abs(got[r] - ry[r]).max() <= 2e-6 * max(1.0, np.abs(ry[r]).max()) + slack


def test_nonfinite_rows_stay_in_their_rows(L):
    T, dim = 40, 520
    x, dy, gamma, beta = _inputs(T, dim, "bf16", 6)
    d = _desc(L, dim, False, "bf16")
    y0, st0 = _forward(L, d, x, gamma, beta)
    xb = x.clone()
    xb[7, 3] = float("nan")
    xb[20, 500] = float("inf")
    y1, st1 = _forward(L, d, xb, gamma, beta)
    dx0 = _backward(L, d, x, gamma, dy, st0)
    dx1 = _backward(L, d, xb, gamma, dy, st1)
    torch.cuda.synchronize()
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[[7, 20]] = False
    assert torch.equal(y0[keep], y1[keep]) and torch.equal(dx0[keep], dx1[keep])
    assert torch.isnan(y1[7].float()).all() and torch.isnan(y1[20].float()).any()


def test_reruns_bitwise_equal_on_another_stream(L):
    T, dim = 3000, 2056
    x, dy, gamma, beta = _inputs(T, dim, "bf16", 8)
    x, dy, gamma, beta = x.cuda(), dy.cuda(), gamma.cuda(), beta.cuda()
    d = _desc(L, dim, False, "bf16")
    outs = []
    ws = torch.empty(L.lora_norm_backward_workspace_size(d, T), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for st in (torch.cuda.current_stream(), torch.cuda.Stream()):
        y, dx, stats = torch.empty_like(x), torch.empty_like(x), torch.empty(T, 2, device="cuda")
        dg, db = torch.zeros(dim, device="cuda"), torch.zeros(dim, device="cuda")
        torch.cuda.synchronize()
        L.lora_norm_forward(d, T, x, gamma, beta, y, stats, stream=st)
        L.lora_norm_backward(d, T, x, gamma, dy, stats, None, dx, dg, db, ws, stream=st)
        torch.cuda.synchronize()
        outs.append((y, stats, dx, dg, db))
    for a, b in zip(*outs):
        assert torch.equal(a, b)
