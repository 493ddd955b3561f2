"""Refusals of the operators between an attention block's projections, which come before any launch, and
the oracle's own pins: its gradients against differences, its attention against a softmax written out."""
import numpy as np
import pytest

from oracle import attention_oracle as A

FAKE = 1 << 20   # an aligned non-null address; never dereferenced (validation fails first)


@pytest.fixture(scope="module")
def L():
    from bwd_adapter_adamw_gb300 import build
    build.build()
    from bwd_adapter_adamw_gb300 import binding
    return binding


def test_rope_table_refusals(L):
    f = lambda n=4, d=64, i=FAKE, t=FAKE: L.lora_rope_table(n, d, i, t, stream=0, check=False)   # noqa: E731
    assert f(n=0) == f(n=-1) == f(d=0) == f(i=None) == f(t=None) == L.LORA_ERR_INVALID
    assert f(d=96) == f(n=(1 << 24) + 1) == L.LORA_ERR_UNSUPPORTED
    assert f(i=FAKE + 8) == f(t=FAKE + 4) == L.LORA_ERR_ALIGN


def _rope(L, d, T=3, n_pos=8, ws_bytes=1 << 30, bwd=False, **kw):
    a = dict(Q=FAKE, K=FAKE, gq=FAKE, gk=FAKE, pos=FAKE, table=FAKE, YQ=FAKE, YK=FAKE, dQ=FAKE, dK=FAKE, dgq=FAKE,
             dgk=FAKE, ws=FAKE)
    a.update(kw)
    if bwd:
        return L.lora_rope_backward(d, T, a["Q"], a["K"], a["gq"], a["gk"], a["pos"], a["table"], n_pos, a["YQ"], a["YK"],
                                    a["dQ"], a["dK"], a["dgq"], a["dgk"], a["ws"], ws_bytes, stream=0, check=False)
    return L.lora_rope_forward(d, T, a["Q"], a["K"], a["gq"], a["gk"], a["pos"], a["table"], n_pos, a["YQ"], a["YK"],
                               stream=0, check=False)


@pytest.mark.parametrize("bwd", [False, True])
def test_rope_refusals(L, bwd):
    ok = L.make_rope_desc(4, 2, 64)
    f = lambda d=ok, **kw: _rope(L, d, bwd=bwd, **kw)   # noqa: E731
    mk = L.make_rope_desc
    assert f(T=0) == L.LORA_OK
    for d in (mk(0, 2, 64), mk(4, -1, 64), mk(4, 2, 0), mk(4, 2, 64, dtype=L.LORA_BF16_FP8), mk(4, 2, 64, layout=2),
              mk(4, 2, 64, eps=-1.0), mk(4, 2, 64, eps=float("nan")), mk(4, 2, 64, eps=float("inf")),
              mk(4, 2, 64, ld_q=248), mk(4, 2, 64, ld_yk=120), mk(4, 2, 64, ld_k=-128)):
        assert f(d) == L.LORA_ERR_INVALID
    for d in (mk(4, 2, 96), mk((1 << 13) + 1, 0, 64), mk(1 << 13, 1, 64), mk(4, 2, 64, ld_q=1 << 33)):
        assert f(d) == L.LORA_ERR_UNSUPPORTED
    assert f(mk(4, 2, 64, ld_q=260)) == f(mk(4, 2, 64, dtype=L.LORA_F32, ld_yq=258)) == L.LORA_ERR_ALIGN
    assert f(T=-1) == f(n_pos=0) == L.LORA_ERR_INVALID
    assert f(T=1 << 31) == f(n_pos=(1 << 24) + 1) == L.LORA_ERR_UNSUPPORTED
    for name in ["Q", "K", "gq", "gk", "pos", "table", "YQ", "YK"] + (["dQ", "dK", "ws"] if bwd else []):
        assert f(**{name: None}) == L.LORA_ERR_INVALID, name
        assert f(**{name: FAKE + 4}) == L.LORA_ERR_ALIGN, name
    assert f(mk(4, 0, 64), K=None, YK=None, dK=None, T=0) == L.LORA_OK
    if bwd:
        assert f(ws_bytes=100) == L.LORA_ERR_WORKSPACE
        assert f(gq=None, gk=None) == L.LORA_ERR_INVALID        # gradients of weights that are not there
        assert f(gq=None, gk=None, dgq=None, dgk=None, Q=None, K=None, T=0) == L.LORA_OK
        assert f(dgq=None, dgk=None, T=0) == L.LORA_OK
        assert L.lora_rope_backward_workspace_size(mk(4, 2, 96), 3) == 0
        assert L.lora_rope_backward_workspace_size(ok, 3) > 0


def test_plan_refusals(L):
    f = lambda T=100, n=3, s=FAKE, p=FAKE, b=1 << 20: L.lora_attn_plan_build(T, n, s, p, b, stream=0, check=False)   # noqa: E731
    assert f(T=-1) == f(n=0) == f(n=-4) == f(s=None) == f(p=None) == L.LORA_ERR_INVALID
    assert f(T=1 << 31) == f(n=(1 << 24) + 1) == L.LORA_ERR_UNSUPPORTED
    assert f(s=FAKE + 2) == f(p=FAKE + 8) == L.LORA_ERR_ALIGN
    assert f(b=64) == L.LORA_ERR_WORKSPACE
    assert L.lora_attn_plan_size(-1, 1) == L.lora_attn_plan_size(5, 0) == 0
    assert L.lora_attn_plan_size(0, 1) > 0
    # room for the tiles of any table: 128-row and 256-row tiles of 16 bytes
    assert L.lora_attn_plan_size(1000, 5) >= 16 * (1000 // 128 + 5 + 1000 // 256 + 5) + 8 * 5


@pytest.mark.parametrize("bwd", [False, True])
def test_attention_refusals(L, bwd):
    def f(d=L.make_attn_desc(4, 2, 64), T=3, n=1, ws_bytes=1 << 30, **kw):
        a = {k: FAKE for k in ("plan", "Q", "K", "V", "O", "lse", "dO", "dQ", "dK", "dV", "ws")}
        a.update(kw)
        if bwd:
            return L.lora_attn_backward(d, T, n, a["plan"], a["Q"], a["K"], a["V"], a["O"], a["lse"], a["dO"], a["dQ"],
                                        a["dK"], a["dV"], a["ws"], ws_bytes, stream=0, check=False)
        return L.lora_attn_forward(d, T, n, a["plan"], a["Q"], a["K"], a["V"], a["O"], a["lse"], stream=0, check=False)
    mk = L.make_attn_desc
    assert f(T=0) == L.LORA_OK
    for d in (mk(0, 1, 64), mk(4, 0, 64), mk(4, 3, 64), mk(4, 2, -64), mk(4, 2, 64, dtype=9), mk(4, 2, 64, scale=0.0),
              mk(4, 2, 64, scale=-1.0), mk(4, 2, 64, scale=float("nan")), mk(4, 2, 64, scale=float("inf")),
              mk(4, 2, 64, ld_q=248), mk(4, 2, 64, ld_k=64), mk(4, 2, 64, ld_v=-8), mk(4, 2, 64, ld_o=8)):
        assert f(d) == L.LORA_ERR_INVALID
    for d in (mk(4, 2, 96), mk(4, 2, 256), mk(4, 2, 64, dtype=L.LORA_F32), mk(4, 2, 64, dtype=L.LORA_BF16_FP8),
              mk(1 << 14, 1, 128), mk(4, 2, 64, ld_k=1 << 33)):
        assert f(d) == L.LORA_ERR_UNSUPPORTED
    for kw in (dict(ld_q=260), dict(ld_k=132), dict(ld_v=129), dict(ld_o=268)):
        assert f(mk(4, 2, 64, **kw)) == L.LORA_ERR_ALIGN
    assert f(T=-1) == f(n=0) == L.LORA_ERR_INVALID
    assert f(T=1 << 31) == f(n=1 << 25) == L.LORA_ERR_UNSUPPORTED
    for name in ["plan", "Q", "K", "V", "O", "lse"] + (["dO", "dQ", "dK", "dV", "ws"] if bwd else []):
        assert f(**{name: None}) == L.LORA_ERR_INVALID, name
        assert f(**{name: FAKE + 8}) == L.LORA_ERR_ALIGN, name
    if bwd:
        assert f(ws_bytes=16) == L.LORA_ERR_WORKSPACE
        assert L.lora_attn_backward_workspace_size(mk(4, 2, 96), 3) == 0
        assert L.lora_attn_backward_workspace_size(mk(4, 2, 64), 1000) >= 4 * 4000


def _slope(f, x, d, h=1e-5):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


@pytest.mark.parametrize("pairs", [False, True])
def test_oracle_rope_gradients_against_differences(pairs):
    """Differences of step 1e-5 in float64: the cubic part is 1e-10 of the derivatives' sizes (order 10 here),
    the rounding 2^-52 of the sum over 1e-5: 1e-7 holds both."""
    rng = np.random.default_rng(1)
    T, H, D = 5, 3, 8
    x, dy, gamma = rng.standard_normal((T, H, D)), rng.standard_normal((T, H, D)), 1 + 0.3 * rng.standard_normal(D)
    cs = A.rope_table(40, 100.0 ** -np.linspace(0, 1, D // 2))[rng.integers(0, 40, T)]
    dx, dg = A.rope_backward(x, gamma, cs, dy, 1e-3, pairs)
    f = lambda a, g: float((A.rope_forward(a, g, cs, 1e-3, pairs) * dy).sum())   # noqa: E731
    for _ in range(3):
        d, e = rng.standard_normal(x.shape), rng.standard_normal(D)
        assert abs(_slope(lambda a: f(a, gamma), x, d) - (dx * d).sum()) <= 1e-7
        assert abs(_slope(lambda g: f(x, g), gamma, e) - (dg * e).sum()) <= 1e-7
    d = rng.standard_normal(x.shape)
    h, _ = A.rope_backward(None, None, cs, dy, 0.0, pairs)
    assert abs(_slope(lambda a: f(a, None), x, d) - (h * d).sum()) <= 1e-7


def test_oracle_rope_turns_by_relative_position():
    """The product of a turned query and a turned key depends on the difference of their positions alone, and a
    turn keeps lengths."""
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((2, 1, 1, 16))
    t = A.rope_table(100, 50.0 ** -np.linspace(0, 1, 8))
    for pairs in (False, True):
        at = lambda x, n: A.rope_forward(x, None, t[n:n + 1], 0.0, pairs)[0, 0]   # noqa: E731
        assert abs(at(q, 30) @ at(k, 10) - at(q, 75) @ at(k, 55)) <= 1e-12
        assert abs(np.linalg.norm(at(q, 63)) - np.linalg.norm(q)) <= 1e-13
        assert np.array_equal(at(q, 0), q[0, 0])


def test_oracle_attention_against_a_loop_and_differences():
    rng = np.random.default_rng(3)
    T, H, K, D = 9, 4, 2, 3
    starts, scale = [0, 4, 4, 8], 0.7
    q, k, v, do = (rng.standard_normal((T, n, D)) for n in (H, K, K, H))
    o, lse = A.attention_forward(q, k, v, starts, scale)
    for h in range(H):
        for a, b in zip(starts, starts[1:]):
            for i in range(a, b):
                w = [np.exp(scale * sum(q[i, h, d] * k[j, h // 2, d] for d in range(D))) for j in range(a, i + 1)]
                want = sum(x * v[j, h // 2] for x, j in zip(w, range(a, i + 1))) / sum(w)
                assert np.abs(o[i, h] - want).max() <= 1e-13 and abs(lse[h, i] - np.log(sum(w))) <= 1e-13
    assert np.isnan(o[8]).all() and np.isnan(lse[:, 8]).all()
    grads = A.attention_backward(q, k, v, o, np.nan_to_num(lse), do, starts, scale)
    loss = lambda *a: float((A.attention_forward(*a, starts, scale)[0] * do)[:8].sum())   # noqa: E731
    for i in range(3):   # as for the rotation: step 1e-5, derivatives of order 10
        d = rng.standard_normal((q, k, v)[i].shape)
        args = [q, k, v]
        f = lambda x: loss(*[x if n == i else a for n, a in enumerate(args)])   # noqa: E731
        assert abs(_slope(f, args[i], d) - (grads[i] * d).sum()) <= 1e-7
