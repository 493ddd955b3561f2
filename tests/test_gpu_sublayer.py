"""The adapted linear over a block-scaled E4M3 base (LORA_BF16_BLK8), and the sublayer step that runs
the norm, the projections and the orthogonalised update together, against float64.

The frozen terms are compared with the oracle's product of the same codes, everything else with
the oracle's formulas; the bars are the library's bf16 ones (2e-2 on outputs and gradients, 1e-2 on
the post-step parameters)."""
import numpy as np
import pytest
import torch

from oracle import lora_oracle as O
from oracle import sublayer_oracle as S
from tests.helpers import TOL_BF16, TOL_BF16_STEP, rel_err, to64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bwd_adapter_adamw_gb300 import binding
    return binding


def _bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16)


def _problem(T, in_d, out_d, r, seed):
    rng = np.random.default_rng(seed)
    X = _bf16(rng.standard_normal((T, in_d)))
    W = _bf16(rng.standard_normal((out_d, in_d)) / np.sqrt(in_d))
    dY = _bf16(0.1 * rng.standard_normal((T, out_d)))
    A = rng.uniform(-np.sqrt(6 / in_d), np.sqrt(6 / in_d), (r, in_d)).astype(np.float32)
    B = (0.1 * rng.standard_normal((out_d, r))).astype(np.float32)
    return X, W, dY, A, B


@pytest.mark.parametrize("T,in_d,out_d,r,p", [(384, 256, 384, 16, 0.0), (512, 528, 256, 8, 0.1),
                                              (257, 1024, 528, 64, 0.0), (5, 272, 400, 36, 0.3),
                                              (130, 144, 1040, 4, 0.0),
                                              (2048, 640, 2816, 64, 0.0), (2816, 2560, 384, 64, 0.2),
                                              (200, 2064, 400, 64, 0.2), (140, 400, 4112, 36, 0.1)])
def test_blk8_forward_backward(L, T, in_d, out_d, r, p):
    from bwd_adapter_adamw_gb300.step import Linear, LoraStep
    X, W, dY, A, B = _problem(T, in_d, out_d, r, T + in_d)
    s = O.lora_scale(2.0 * r, r, False)
    lin = Linear(0, 0, X.cuda(), W.cuda(), dY.cuda())
    step = LoraStep([lin], rank=r, scale=s, dtype="bf16blk8", tokens=T, chunks=1, dropout_p=p,
                    seed=5, max_norm=1.0, hp=L.make_hp(), device="cuda")
    lin.A.copy_(torch.from_numpy(A))
    lin.B.copy_(torch.from_numpy(B))
    step.prepare_weights()
    step.forward_backward(opt_step=2)
    torch.cuda.synchronize()
    assert L.lora_device_error() == 0
    keep = O.dropout_keep(p, 5, 2, 0, 0, 0, T, in_d) if p > 0 else None
    q = O.dropout_q(p) if p > 0 else 1.0
    Xf, Wf, dYf = X.float().numpy(), W.float().numpy(), dY.float().numpy()
    c, sc = S.quantize_blocks(Wf, 128, 128)
    buf = lin.Wp.cpu().numpy()
    assert np.array_equal(buf[:out_d * in_d].reshape(out_d, in_d), c)
    assert np.array_equal(buf[out_d * in_d:].view(np.float32).reshape(sc.shape), sc)
    # LoRA terms: what the oracle's forward and backward add to a frozen weight of zeros
    f0 = O.lora_forward(to64(Xf), np.zeros_like(to64(Wf)), A, B, s, keep, q)
    b = O.lora_backward(to64(Xf), np.zeros_like(to64(Wf)), A, B, to64(dYf), s, keep, q)
    assert rel_err(lin.Y, S.block_product(Xf, c, sc, False)[0] + f0.Y) <= TOL_BF16
    assert rel_err(lin.dX, S.block_product(dYf, c, sc, True)[0] + b.dX) <= TOL_BF16
    assert rel_err(lin.gA, b.dA) <= TOL_BF16
    assert rel_err(lin.gB, b.dB) <= TOL_BF16


def test_blk8_from_checkpoint_codes_without_a_bf16_weight(L):
    T, in_d, out_d, r = 200, 272, 400, 8
    X, W, _, A, B = _problem(T, in_d, out_d, r, 3)
    c, sc = S.quantize_blocks(W.float().numpy(), 128, 128)
    d = L.make_desc(in_d, out_d, r, 2.0, L.LORA_BF16_BLK8)
    n = L.lora_prepared_weight_size(d)
    assert n == out_d * in_d + 4 * sc.size
    Wp = torch.empty(n, dtype=torch.uint8)
    Wp[:out_d * in_d] = torch.from_numpy(c.reshape(-1))
    Wp[out_d * in_d:] = torch.from_numpy(sc.reshape(-1).view(np.uint8))
    Wp = Wp.cuda()
    Ad, Bd = torch.from_numpy(A).cuda(), torch.from_numpy(B).cuda()
    Y = torch.empty(T, out_d, dtype=torch.bfloat16, device="cuda")
    H = torch.empty(T, r, device="cuda")
    ws = torch.empty(L.lora_workspace_size(d, T), dtype=torch.uint8, device="cuda")
    L.lora_forward(d, None, T, X.cuda(), None, Wp, Ad, Bd, None, None, Y, H, ws)
    torch.cuda.synchronize()
    f0 = O.lora_forward(to64(X.float().numpy()), np.zeros((out_d, in_d)), A, B, 2.0)
    assert rel_err(Y, S.block_product(X.float().numpy(), c, sc, False)[0] + f0.Y) <= TOL_BF16


@pytest.mark.parametrize("T,in_d,out_d,dx", [(300, 14336, 512, False), (129, 2560, 1008, False),
                                             (260, 528, 4112, True), (131, 1040, 272, False),
                                             (140, 144, 2064, True), (640, 1936, 400, False)])
def test_product_of_few_tiles_and_long_contractions(L, T, in_d, out_d, dx):
    """Sizes whose tiles are shared by a cluster: against the oracle, and reruns bitwise equal."""
    rng = np.random.default_rng(T + in_d)
    X = _bf16(rng.standard_normal((T, out_d if dx else in_d)))
    W = _bf16(rng.standard_normal((out_d, in_d)) / np.sqrt(in_d))
    c, sc = S.quantize_blocks(W.float().numpy(), 128, 128)
    cd, sd, Xd = torch.from_numpy(c).cuda(), torch.from_numpy(sc).cuda(), X.cuda()
    ws = torch.empty(L.lora_block_product_workspace_size(T, out_d, in_d, dx), dtype=torch.uint8, device="cuda")
    Y = [torch.full((T, in_d if dx else out_d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for y in Y:
        L.lora_block_product(T, out_d, in_d, Xd, cd, sd, y, dx, ws)
    assert L.lora_device_check() == L.LORA_OK
    assert torch.equal(Y[0], Y[1])
    assert rel_err(Y[0], S.block_product(X.float().numpy(), c, sc, dx)[0]) <= TOL_BF16


@pytest.mark.parametrize("T,in_d,out_d,dx", [(29, 3456, 10816, False), (100, 3456, 10816, False),
                                             (29, 3456, 10816, True), (500, 2560, 4096, False),
                                             (8, 2560, 4096, False)])
def test_product_reruns_are_bitwise_equal(L, T, in_d, out_d, dx):
    """Many reruns, alone and on three streams at once: a stage that is overwritten before its last
    reader is done shows as a few different elements."""
    g = torch.Generator(device="cuda").manual_seed(T + in_d)
    X = torch.randn(T, out_d if dx else in_d, generator=g, device="cuda").to(torch.bfloat16)
    X[:, ::64] *= 20
    W = (torch.randn(out_d, in_d, generator=g, device="cuda") / in_d ** 0.5).to(torch.bfloat16)
    c = torch.empty(out_d, in_d, dtype=torch.uint8, device="cuda")
    sc = torch.empty(-(-out_d // 128), -(-in_d // 128), device="cuda")
    L.lora_block_quantize_weight(W, out_d, in_d, c, sc)
    n, streams = L.lora_block_product_workspace_size(T, out_d, in_d, dx), [torch.cuda.Stream() for _ in range(3)]
    ws = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in streams]
    Y = [torch.empty(T, in_d if dx else out_d, dtype=torch.bfloat16, device="cuda") for _ in streams]
    L.lora_block_product(T, out_d, in_d, X, c, sc, Y[0], dx, ws[0])
    want = Y[0].clone()
    torch.cuda.synchronize()
    for k in range(150):
        for st, w, y in list(zip(streams, ws, Y))[:1 if k < 75 else 3]:
            with torch.cuda.stream(st):
                for _ in range(3):
                    L.lora_block_product(T, out_d, in_d, X, c, sc, y, dx, w)
        torch.cuda.synchronize()
        for y in Y[:1 if k < 75 else 3]:
            assert torch.equal(y, want)


@pytest.mark.parametrize("T,dim,dt", [(2100, 4096, torch.bfloat16), (2100, 2048, torch.float32), (700, 8192, torch.bfloat16)])
def test_norm_backward_reruns_are_bitwise_equal(L, T, dim, dt):
    g = torch.Generator(device="cuda").manual_seed(dim)
    x, dy = (torch.randn(T, dim, generator=g, device="cuda").to(dt) for _ in range(2))
    gamma, st = torch.rand(dim, generator=g, device="cuda"), torch.empty(T, 2, device="cuda")
    d = L.make_norm_desc(dim, L.LORA_NORM_LAYER, L.LORA_BF16 if dt == torch.bfloat16 else L.LORA_F32)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    ws = torch.empty(L.lora_norm_backward_workspace_size(d, T), dtype=torch.uint8, device="cuda")
    L.lora_norm_forward(d, T, x, gamma, None, y, st)
    want = None
    for _ in range(100):
        dg, db = torch.zeros(dim, device="cuda"), torch.zeros(dim, device="cuda")
        for a, b, out in ((dg, db, dx), (dg, db, None)):   # the second: the token sums alone
            L.lora_norm_backward(d, T, x, gamma, dy, st, None, out, a, b, ws)
        got = (dx.clone(), dg, db)
        want = want or got
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_blk8_refusals(L):
    bad = lambda *a, **k: L.lora_prepared_weight_size(L.make_desc(*a, **k))   # noqa: E731
    assert bad(64, 64, 8, 1.0, L.LORA_BF16_BLK8) > 0
    assert bad(24, 64, 8, 1.0, L.LORA_BF16_BLK8) == 0            # in % 16 != 0
    assert bad(64, 64, 8, 1.0, L.LORA_BF16_BLK8, dora=True) == 0
    d = L.make_desc(64, 64, 8, 1.0, L.LORA_BF16_BLK8)
    A = torch.zeros(8, 64)
    projs = L.make_projs([dict(A=A, B=A, out=64)])
    assert L.lora_fused_workspace_size(d, 16, projs) == 0
    slots = L.make_slots([dict(A=A, B=A, rank=8, scale=1.0)])
    assert L.multi_lora_workspace_size(d, 16, 1, slots) == 0
    assert L.lora_dora_norm_workspace_size(d) == 0
    F = 1 << 20
    with pytest.raises(L.LoraError) as e:
        L.lora_dora_norm(d, F, F, F, F, F, 1 << 30, stream=0)
    assert e.value.status == L.LORA_ERR_UNSUPPORTED


@pytest.mark.parametrize("T", [4, 40, 200, 300, 1000])
def test_product_short_wait_bound_reports_timeout_and_recovers(L, T):
    """Waits shortened to one cycle run out on an ordinary launch: the status says so, and with the
    default bound the same call is right again."""
    out_d, in_d = 2560, 4096
    rng = np.random.default_rng(T)
    X = _bf16(rng.standard_normal((T, in_d))).cuda()
    W = _bf16(rng.standard_normal((out_d, in_d)) / 64).cuda()
    c = torch.empty(out_d, in_d, dtype=torch.uint8, device="cuda")
    sc = torch.empty(out_d // 128, in_d // 128, device="cuda")
    L.lora_block_quantize_weight(W, out_d, in_d, c, sc)
    Y = torch.empty(T, out_d, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(L.lora_block_product_workspace_size(T, out_d, in_d), dtype=torch.uint8, device="cuda")
    L.lora_block_product(T, out_d, in_d, X, c, sc, Y, False, ws)
    want = Y.clone()
    assert L.lora_device_error(reset=True) == 0
    try:
        L.lora_set_wait_limit(1)
        L.lora_block_product(T, out_d, in_d, X, c, sc, Y, False, ws)
        status = L.lora_device_check()
    finally:
        L.lora_set_wait_limit(0)
    flags = L.lora_device_error(reset=True)
    assert status == L.LORA_ERR_TIMEOUT and flags != 0 and (flags & ~0x7) == 0
    L.lora_block_product(T, out_d, in_d, X, c, sc, Y, False, ws)
    assert L.lora_device_check() == L.LORA_OK
    assert torch.equal(Y, want)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_sublayer_step(L, kind):
    """Norm, two block-scaled projections with adapters, the residual's gradient, the global clip, the
    orthogonalised update of A and B and AdamW on the norm's parameters, two steps."""
    from bwd_adapter_adamw_gb300.step import Linear, SublayerStep
    T, dim, outs, r, lr, rms = 300, 272, (400, 144), 16, 1e-2, kind == "rms"
    rng = np.random.default_rng(7)
    x = _bf16(rng.standard_normal((T, dim)) * 2 + 0.3)
    res = _bf16(0.1 * rng.standard_normal((T, dim)))
    pr = [_problem(T, dim, o, r, 20 + o) for o in outs]
    lins = [Linear(0, i, None, p[1].cuda(), p[2].cuda()) for i, p in enumerate(pr)]
    s = O.lora_scale(2.0 * r, r, False)
    st = SublayerStep(x.cuda(), lins, kind=kind, muon=L.make_muon_hp(plus_ratio=2.0), rank=r, scale=s,
                      dtype="bf16blk8", tokens=T, chunks=1, max_norm=0.5, hp=L.make_hp(), device="cuda")
    st.prepare_weights()
    A, B, m = [p[3].astype(np.float64) for p in pr], [p[4].astype(np.float64) for p in pr], {}
    for l, p in zip(lins, pr):
        l.A.copy_(torch.from_numpy(p[3]))
        l.B.copy_(torch.from_numpy(p[4]))
    g, b = np.ones(dim), None if rms else np.zeros(dim)
    adam = {k: (np.zeros(dim), np.zeros(dim)) for k in ("g", "b")}
    for t in range(2):
        st.run(t, lr, res.cuda())
        torch.cuda.synchronize()
        xf = to64(x.float().numpy())
        h = _bf16(S.norm_forward(xf, g, b, 1e-5, rms)[0]).float().numpy()
        dh, grads = np.zeros((T, dim)), {}
        for i, p in enumerate(pr):
            c, sc = S.quantize_blocks(p[1].float().numpy(), 128, 128)
            dy, z = p[2].float().numpy(), np.zeros((outs[i], dim))
            f0 = O.lora_forward(to64(h), z, A[i], B[i], s)
            bk = O.lora_backward(to64(h), z, A[i], B[i], to64(dy), s)
            assert rel_err(lins[i].Y, S.block_product(h, c, sc, False)[0] + f0.Y) <= TOL_BF16
            dh += S.block_product(dy, c, sc, True)[0] + bk.dX
            grads["A", i], grads["B", i] = bk.dA, bk.dB
        dx, dg, db = S.norm_backward(xf, g, dh, 1e-5, rms)
        assert rel_err(st.dX, dx + to64(res.float().numpy())) <= TOL_BF16
        grads["g"] = dg
        if not rms:
            grads["b"] = db
        norm = np.sqrt(sum(float((v ** 2).sum()) for v in grads.values())) / T
        cs = (1 / T) * (0.5 / norm if norm > 0.5 else 1.0)
        assert abs(st.scale_norm[0].item() - cs) <= 2e-2 * cs
        for i in range(len(pr)):
            A[i], m["A", i] = S.muon_update(A[i], grads["A", i], m.get(("A", i), 0 * A[i]), c=cs, lr=lr, kind="A", ratio=2.0)
            B[i], m["B", i] = S.muon_update(B[i], grads["B", i], m.get(("B", i), 0 * B[i]), c=cs, lr=lr, kind="B", ratio=2.0)
            assert rel_err(lins[i].A, A[i]) <= TOL_BF16_STEP
            assert rel_err(lins[i].B, B[i]) <= TOL_BF16_STEP
        for k, dev in (("g", st.gamma), ("b", st.beta)):
            if k == "b" and rms:
                continue
            m1, v1 = adam[k]
            gh = cs * grads[k]
            m1, v1 = 0.9 * m1 + 0.1 * gh, 0.999 * v1 + 0.001 * gh ** 2
            adam[k] = (m1, v1)
            u = (m1 / (1 - 0.9 ** (t + 1))) / (np.sqrt(v1 / (1 - 0.999 ** (t + 1))) + 1e-8)
            if k == "g":
                g = g - lr * u
            else:
                b = b - lr * u
            # near-zero gradients make Adam's first steps a sign: at most 2 lr per step of difference
            got = to64(dev)
            ref = g if k == "g" else b
            assert np.mean(np.abs(got - ref) > 0.05 * lr) <= 0.02 and np.abs(got - ref).max() <= 2.1 * lr * (t + 1)
            if k == "g":
                g = got
            else:
                b = got
        assert float(st.arena.grads.abs().max()) == 0.0
        for i in range(len(pr)):   # the next step from the device's state
            A[i], B[i] = to64(lins[i].A), to64(lins[i].B)
