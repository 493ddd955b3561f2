"""Argument checks of the operators around the adapted linear: every refusal comes before any
launch, so these run without a GPU. And the oracle's own pins for them."""
import numpy as np
import pytest

from oracle import sublayer_oracle as S

FAKE = 1 << 20   # an aligned non-null address; never dereferenced (validation fails first)


@pytest.fixture(scope="module")
def L():
    from bwd_adapter_adamw_gb300 import build
    build.build()
    from bwd_adapter_adamw_gb300 import binding
    return binding


def _product(L, T=4, out=64, n_in=64, ws_bytes=1 << 30, **kw):
    a = dict(X=FAKE, W8=FAKE, sw=FAKE, Y=FAKE, ws=FAKE)
    a.update(kw)
    return L.lora_block_product(T, out, n_in, a["X"], a["W8"], a["sw"], a["Y"], False, a["ws"],
                                ws_bytes, stream=0, check=False)


def test_block_product_refusals(L):
    assert _product(L, T=-1) == L.LORA_ERR_INVALID
    assert _product(L, out=0) == L.LORA_ERR_INVALID
    assert _product(L, out=24) == L.LORA_ERR_ALIGN
    assert _product(L, n_in=40) == L.LORA_ERR_ALIGN
    assert _product(L, T=(1 << 31)) == L.LORA_ERR_UNSUPPORTED
    assert _product(L, n_in=1 << 21) == L.LORA_ERR_UNSUPPORTED
    for name in ("X", "W8", "sw", "Y", "ws"):
        assert _product(L, **{name: None}) == L.LORA_ERR_INVALID
        assert _product(L, **{name: FAKE + 8}) == L.LORA_ERR_ALIGN
    assert _product(L, ws_bytes=16) == L.LORA_ERR_WORKSPACE
    assert _product(L, T=0) == L.LORA_OK                # nothing to do, nothing launched
    assert L.lora_block_product_workspace_size(4, 24, 64) == 0
    assert L.lora_block_product_workspace_size(4, 64, 64) > 0
    q = lambda **kw: L.lora_block_quantize(kw.get("src", FAKE), kw.get("rows", 2), kw.get("K", 32),   # noqa: E731
                                           FAKE, FAKE, stream=0, check=False)
    assert q(K=24) == L.LORA_ERR_ALIGN
    assert q(rows=-1) == L.LORA_ERR_INVALID
    assert q(src=None) == L.LORA_ERR_INVALID
    assert q(rows=0) == L.LORA_OK
    assert L.lora_block_quantize_weight(FAKE, 40, 64, FAKE, FAKE, stream=0, check=False) == L.LORA_ERR_ALIGN
    assert L.lora_block_quantize_weight(FAKE, 64, 64, None, FAKE, stream=0, check=False) == L.LORA_ERR_INVALID


def test_norm_refusals(L):
    def fwd(d, T=3, **kw):
        a = dict(X=FAKE, gamma=FAKE, beta=FAKE, Y=FAKE, stats=FAKE)
        a.update(kw)
        return L.lora_norm_forward(d, T, a["X"], a["gamma"], a["beta"], a["Y"], a["stats"], stream=0, check=False)

    def bwd(d, T=3, ws_bytes=1 << 30, **kw):
        a = dict(X=FAKE, gamma=FAKE, dY=FAKE, stats=FAKE, add=None, dX=FAKE, dg=FAKE, db=FAKE, ws=FAKE)
        a.update(kw)
        return L.lora_norm_backward(d, T, a["X"], a["gamma"], a["dY"], a["stats"], a["add"], a["dX"],
                                    a["dg"], a["db"], a["ws"], ws_bytes, stream=0, check=False)

    ok = L.make_norm_desc(64)
    rms = L.make_norm_desc(64, L.LORA_NORM_RMS)
    for f in (fwd, bwd):
        assert f(L.make_norm_desc(0)) == L.LORA_ERR_INVALID
        assert f(L.make_norm_desc(64, 2)) == L.LORA_ERR_INVALID
        assert f(L.make_norm_desc(64, 0, L.LORA_BF16_FP8)) == L.LORA_ERR_INVALID
        assert f(L.make_norm_desc(64, eps=-1.0)) == L.LORA_ERR_INVALID
        assert f(L.make_norm_desc(64, eps=float("nan"))) == L.LORA_ERR_INVALID
        assert f(L.make_norm_desc(60)) == L.LORA_ERR_ALIGN
        assert f(L.make_norm_desc(L.LORA_NORM_MAX_DIM + 8)) == L.LORA_ERR_UNSUPPORTED
        assert f(ok, T=-1) == L.LORA_ERR_INVALID
        assert f(ok, T=1 << 31) == L.LORA_ERR_UNSUPPORTED
        assert f(ok, X=None) == L.LORA_ERR_INVALID
        assert f(ok, gamma=FAKE + 4) == L.LORA_ERR_ALIGN
        assert f(ok, stats=None) == L.LORA_ERR_INVALID
        assert f(ok, T=0) == L.LORA_OK
    assert fwd(rms) == L.LORA_ERR_INVALID               # an RMS norm has no shift
    assert bwd(rms) == L.LORA_ERR_INVALID
    assert bwd(ok, dX=None, dg=None, db=None) == L.LORA_ERR_INVALID
    assert bwd(ok, dX=None, add=FAKE) == L.LORA_ERR_INVALID
    assert bwd(ok, dY=None) == L.LORA_ERR_INVALID
    assert bwd(ok, ws_bytes=16) == L.LORA_ERR_WORKSPACE
    assert bwd(ok, db=FAKE + 8) == L.LORA_ERR_ALIGN


def test_muon_refusals(L):
    groups = L.make_groups([dict(offset=0, n_a=1024, n_b=1024, grad_scale=1.0, lr=0.1)])

    def step(mats, hp=None, ws_bytes=1 << 20, **kw):
        a = dict(p=FAKE, g=FAKE, m=FAKE, sn=FAKE, st=FAKE, ws=FAKE)
        a.update(kw)
        return L.lora_muon_step(a["p"], a["g"], a["m"], groups, L.make_mats(mats), hp or L.make_muon_hp(),
                                a["sn"], a["st"], False, a["ws"], ws_bytes, stream=0, check=False)

    mat = lambda **kw: dict(dict(offset=0, rows=8, cols=64, group=0, kind=0), **kw)   # noqa: E731
    assert step([mat(rows=0)]) == L.LORA_ERR_INVALID
    assert step([mat(offset=-4)]) == L.LORA_ERR_INVALID
    assert step([mat(kind=2)]) == L.LORA_ERR_INVALID
    assert step([mat(group=1)]) == L.LORA_ERR_INVALID
    assert step([mat(rows=6)]) == L.LORA_ERR_UNSUPPORTED
    assert step([mat(rows=68, cols=128)]) == L.LORA_ERR_UNSUPPORTED
    assert step([mat(offset=2)]) == L.LORA_ERR_ALIGN
    assert step([mat(offset=2048 - 256)]) == L.LORA_ERR_INVALID          # past the group's end
    assert step([mat(), mat(offset=256)]) == L.LORA_ERR_INVALID          # overlapping
    assert step([mat(offset=1024), mat(offset=768)]) == L.LORA_ERR_INVALID
    assert step([mat()], L.make_muon_hp(momentum=1.0)) == L.LORA_ERR_INVALID
    assert step([mat()], L.make_muon_hp(steps=0)) == L.LORA_ERR_INVALID
    assert step([mat()], L.make_muon_hp(steps=9)) == L.LORA_ERR_INVALID
    assert step([mat()], L.make_muon_hp(adjust=2)) == L.LORA_ERR_INVALID
    assert step([mat()], L.make_muon_hp(coef=(float("nan"), 0.0, 0.0))) == L.LORA_ERR_INVALID
    for name in ("p", "g", "m", "sn", "st", "ws"):
        assert step([mat()], **{name: None}) == L.LORA_ERR_INVALID
    assert step([mat()], p=FAKE + 8) == L.LORA_ERR_ALIGN
    assert step([mat()], ws_bytes=0) == L.LORA_ERR_WORKSPACE
    assert step([]) == L.LORA_OK
    assert L.lora_muon_workspace_size(L.make_mats([mat(rows=6)])) == 0


# ---- the oracle's pins ------------------------------------------------------------------------
def test_oracle_blocks():
    x = np.zeros((130, 260), np.float32)
    x[5, 7] = -2.0
    x[129, 259] = 3.0
    c, s = S.quantize_blocks(x, 128, 128)
    assert s.shape == (2, 3) and s[0, 0] == np.float32(2.0) * (np.float32(1) / np.float32(448)) and s[0, 1] == 1.0
    d = S.dequantize_blocks(c, s, 128, 128)
    assert np.allclose(d[5, 7], -2.0, rtol=1e-6) and np.allclose(d[129, 259], 3.0, rtol=1e-6)
    assert np.count_nonzero(d) == 2
    rng = np.random.default_rng(0)
    w = rng.standard_normal((40, 300)).astype(np.float32)
    c, s = S.quantize_blocks(w, 1, 128)
    assert np.abs(S.dequantize_blocks(c, s, 1, 128) - w).max() <= 2.0 ** -4 * np.abs(w).max()


@pytest.mark.parametrize("rms", [False, True])
def test_oracle_norm_gradient_against_differences(rms):
    rng = np.random.default_rng(1)
    x, dy = rng.standard_normal((3, 6)), rng.standard_normal((3, 6))
    gamma = 1 + 0.1 * rng.standard_normal(6)
    dx, dg, db = S.norm_backward(x, gamma, dy, 1e-5, rms)
    f = lambda x_, g_, b_: float((S.norm_forward(x_, g_, b_, 1e-5, rms)[0] * dy).sum())   # noqa: E731
    z = np.zeros(6)
    for t in range(3):
        for i in range(6):
            e = np.zeros_like(x)
            e[t, i] = 1e-5
            assert abs((f(x + e, gamma, z) - f(x - e, gamma, z)) / 2e-5 - dx[t, i]) < 1e-7
    for i in range(6):
        e = np.zeros(6)
        e[i] = 1e-5
        assert abs((f(x, gamma + e, z) - f(x, gamma - e, z)) / 2e-5 - dg[i]) < 1e-7
        assert abs((f(x, gamma, z + e) - f(x, gamma, z - e)) / 2e-5 - db[i]) < 1e-7


def test_oracle_newton_schulz():
    rng = np.random.default_rng(2)
    u = rng.standard_normal((6, 40))
    x, gain = S.newton_schulz(u)
    # the sequence acts on the singular values alone
    U, s, V = np.linalg.svd(u / np.linalg.norm(u), full_matrices=False)
    for _ in range(5):
        s = 3.4445 * s - 4.7750 * s ** 3 + 2.0315 * s ** 5
    assert np.allclose(x, (U * s) @ V, atol=1e-12)
    assert np.allclose(S.newton_schulz(u.T)[0], x.T, atol=1e-12)
    assert np.allclose(S.newton_schulz(1e-20 * u)[0], x, atol=1e-9)
    # the cubic-quintic (2, -1.5, 0.5) converges to the orthogonal factor
    y, _ = S.newton_schulz(u, (2.0, -1.5, 0.5), 40)
    assert np.allclose(y, U @ V, atol=1e-9) and gain > 1.0


def test_block_scaled_base_sizes_and_refusals(L):
    """dtype LORA_BF16_BLK8: one copy of codes with a scale per block; no DoRA, no slots, no fused group."""
    d = L.make_desc(272, 400, 8, 1.0, L.LORA_BF16_BLK8)
    assert L.lora_prepared_weight_size(d) == 400 * 272 + 4 * 4 * 3
    assert L.lora_workspace_size(d, 100) > 0
    for bad in (L.make_desc(24, 64, 8, 1.0, L.LORA_BF16_BLK8), L.make_desc(64, 40, 8, 1.0, L.LORA_BF16_BLK8),
                L.make_desc(64, 64, 8, 1.0, L.LORA_BF16_BLK8, dora=True),
                L.make_desc(64, (1 << 20) + 16, 8, 1.0, L.LORA_BF16_BLK8)):
        assert L.lora_prepared_weight_size(bad) == 0 and L.lora_workspace_size(bad, 16) == 0
    assert L.lora_dora_norm_workspace_size(d) == 0
    F = 1 << 20   # never touched: every call is refused on the host
    for args, status in (((d, None, 4, F, None, None, F, F, None, None, F, F, F, 1 << 30), L.LORA_ERR_INVALID),
                         ((d, None, 4, F, None, F, F, F, None, None, F, F, F, 16), L.LORA_ERR_WORKSPACE),
                         ((d, None, 4, F + 2, None, F, F, F, None, None, F, F, F, 1 << 30), L.LORA_ERR_ALIGN)):
        with pytest.raises(L.LoraError) as e:
            L.lora_forward(*args, stream=0)
        assert e.value.status == status
