"""The attention sublayer's step: norm, adapted q / k / v, head norms with rotation, packed causal
attention, adapted output projection, and all of it backward.

Each stage is checked against float64 on the step's own inputs of that stage (which are rounded to bf16), so
that a stage's bar is its operator's: the library's bf16 ones for the projections, the norms' 3e-3 in the
2-norm, one rounding (2^-8) and fp32 arithmetic for the rotation, the attention's element-wise bounds."""
import numpy as np
import pytest
import torch

from oracle import attention_oracle as A
from oracle import lora_oracle as O
from oracle import sublayer_oracle as S
from tests.helpers import TOL_BF16, rel_err, to64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bwd_adapter_adamw_gb300 import binding
    return binding


def make(starts, pad, dim=256, hq=4, hk=2, hd=64, seed=0, **kw):
    from bwd_adapter_adamw_gb300.step import AttentionStep, Linear
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")   # noqa: E731
    T = starts[-1] + pad
    X = rnd(T, dim).to(torch.bfloat16)
    lin = lambda i, o, n: Linear(0, i, None, (rnd(o, n) / n ** 0.5).to(torch.bfloat16), None)   # noqa: E731
    q, k, v, o = lin(0, hq * hd, dim), lin(1, hk * hd, dim), lin(2, hk * hd, dim), lin(3, dim, hq * hd)
    o.dY = (0.1 * rnd(T, dim)).to(torch.bfloat16)
    if pad:
        o.dY[-pad:] = 0
    kw = dict(dict(rank=8, scale=2.0, dtype="bf16", tokens=T, chunks=1, max_norm=0.5, kind="rms"), **kw)
    st = AttentionStep(X, q, k, v, o, q_heads=hq, kv_heads=hk, head_dim=hd,
                       seq_start=torch.tensor(starts, dtype=torch.int32, device="cuda"), **kw)
    st.prepare_weights()
    for l in st.linears:
        l.A.copy_(rnd(*l.A.shape) / l.in_dim ** 0.5)
        l.B.copy_(0.1 * rnd(*l.B.shape))
    st.gamma.copy_(1 + 0.2 * rnd(dim))
    for gm in (st.gamma_q, st.gamma_k):
        if gm is not None:
            gm.copy_(1 + 0.2 * rnd(hd))
    return st, rnd


def close(got, ref, bar):
    got = to64(got)
    return np.linalg.norm(got - ref) <= bar * np.linalg.norm(ref)


def check(st, starts, dX_res=None, pairs=False):
    T, hd, hq, hk = st.T, st.head_dim, st.q_heads, st.kv_heads
    live = np.zeros(T, bool)
    live[:starts[-1]] = True
    rms = st.beta is None
    h, mean, rstd = S.norm_forward(to64(st.X_in), to64(st.gamma), None if rms else to64(st.beta), 1e-5, rms)
    assert close(st.H_norm, h, 3e-3)
    f, b = {}, {}
    for n, l in (("q", st.q), ("k", st.k), ("v", st.v), ("o", st.o)):
        x, W, Aa, B = (to64(t) for t in (l.X, l.W, l.A, l.B))
        assert rel_err(l.Y, O.lora_forward(x, W, Aa, B, 2.0).Y) <= TOL_BF16, n
        back = O.lora_backward(x, W, Aa, B, to64(l.dY), 2.0)
        assert rel_err(l.dX, back.dX) <= TOL_BF16, n
        assert rel_err(l.gA, back.dA) <= TOL_BF16 and rel_err(l.gB, back.dB) <= TOL_BF16, n
    pos = np.concatenate([np.arange(e - s) for s, e in zip(starts, starts[1:])] + [np.zeros(T - starts[-1], int)])
    inv = 10000.0 ** (-np.arange(0, hd, 2) / hd)
    cs = A.rope_table(T, inv)[pos]
    u = (hd + 24) * 2.0 ** -24   # the rotation's fp32 arithmetic, with the table's own rounding
    heads = lambda t, n: to64(t).reshape(T, n, hd)   # noqa: E731
    for l, y, n, gm in ((st.q, st.Qr, hq, st.gamma_q), (st.k, st.Kr, hk, st.gamma_k)):
        x, gam = heads(l.Y, n), None if gm is None else to64(gm)
        ref = A.rope_forward(x, gam, cs, 1e-6, pairs)
        size = np.abs(x).max(-1, keepdims=True) * 2 * (1 if gm is None else np.abs(gam).max() / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6))
        assert np.all(np.abs(heads(y, n) - ref)[live] <= (2.0 ** -8 * np.abs(ref) + 2 * u * size)[live])
        assert not heads(y, n)[~live].any()
    q, k, v = heads(st.Qr, hq), heads(st.Kr, hk), heads(st.v.Y, hk)
    scale = float(np.float32(hd ** -0.5))
    o, lse = A.attention_forward(q, k, v, starts, scale)
    eo, el = A.attention_bounds(q, k, v, np.nan_to_num(o), np.nan_to_num(lse), np.zeros_like(q), starts, scale, False)
    assert np.all(np.abs(heads(st.o.X, hq) - o)[live] <= (2.0 ** -8 * np.abs(o) + eo * 1.01)[live])
    assert np.all(np.abs(to64(st.lse) - lse)[:, live] <= el[:, live])
    assert not heads(st.o.X, hq)[~live].any()
    od, ld, do = heads(st.o.X, hq), to64(st.lse), heads(st.o.dX, hq)
    want = A.attention_backward(q, k, v, od, ld, do, starts, scale)
    room = A.attention_bounds(q, k, v, od, ld, do, starts, scale, True)
    for got, n, ref, e in zip((st.dQr, st.dKr, st.v.dY), (hq, hk, hk), want, room):
        assert np.all(np.abs(heads(got, n) - ref) <= 2.0 ** -8 * np.abs(ref) + e * 1.01)
    for l, dy, n, gm, dg in ((st.q, st.dQr, hq, st.gamma_q, st.dgamma_q), (st.k, st.dKr, hk, st.gamma_k, st.dgamma_k)):
        gam = None if gm is None else to64(gm)
        ref, sums = A.rope_backward(heads(l.Y, n)[live], gam, cs[live], heads(dy, n)[live], 1e-6, pairs)
        assert close(heads_t(l.dY, n, hd)[live], ref, 3e-3)
        assert not heads(l.dY, n)[~live].any()
        if gm is not None:
            assert close(dg, sums, 1e-4)
    dh = sum(to64(l.dX) for l in (st.q, st.k, st.v))
    dx, dgam, dbet = S.norm_backward(to64(st.X_in), to64(st.gamma), dh, 1e-5, rms)
    res = 0 if dX_res is None else to64(dX_res)
    assert close(st.dX, dx + res, 8e-3)          # the sum of the three gradients is rounded, too
    assert close(st.dgamma, dgam, 8e-3)


def heads_t(t, n, hd):
    return t.float().cpu().view(t.shape[0], n, hd)


@pytest.mark.parametrize("starts,pad,kw", [([0, 200], 0, {}), ([0, 77, 77, 300, 301], 30, dict(pairs=True, kind="layer")),
                                           ([0, 129, 260], 5, dict(head_norm=False, n_streams=3)),
                                           ([0, 64, 300], 0, dict(hq=3, hk=3, hd=128, dim=384))])
def test_every_stage(L, starts, pad, kw):
    st, rnd = make(starts, pad, **kw)
    res = rnd(*st.X_in.shape).to(torch.bfloat16)
    st.forward_backward(0, res)
    torch.cuda.synchronize()
    assert L.lora_device_error() == 0
    check(st, starts, res, kw.get("pairs", False))
    # the update takes every parameter, and a second step runs from it
    before = st.arena.params.clone()
    st.optimizer_step(1e-3, 0)
    torch.cuda.synchronize()
    assert int(st.status.item()) == 0 and not bool(st.arena.grads.any())
    moved = st.arena.params != before
    assert moved.float().mean() > 0.99
    st.run(1, 1e-3, res)
    torch.cuda.synchronize()
    assert int(st.status.item()) == 0 and bool(torch.isfinite(st.arena.params).all())


def test_forward_alone_and_replayed(L):
    """The serving call gives the training forward's output; a captured step repeats an eager one bit for bit."""
    starts = [0, 100, 333]
    st, _ = make(starts, 0)
    st.forward_backward(0)
    torch.cuda.synchronize()
    want = [t.clone() for t in (st.o.Y, st.dX, st.arena.grads)]
    st.o.Y.zero_()
    st.forward()
    assert torch.equal(st.o.Y, want[0])
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        st.arena.grads.zero_()
        st.forward_backward(0)
    for _ in range(2):
        st.dX.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (st.o.Y, st.dX, st.arena.grads)))


def test_refusals(L):
    from bwd_adapter_adamw_gb300.step import AttentionStep, Linear
    X = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    W = lambda o, i: torch.zeros(o, i, dtype=torch.bfloat16, device="cuda")   # noqa: E731
    lin = lambda i, o, n, dY=None: Linear(0, i, None, W(o, n), dY)   # noqa: E731
    s = torch.tensor([0, 8], dtype=torch.int32, device="cuda")

    def build(X=X, kq=128, o_in=128, start=s, dY=X, **kw):
        kw = dict(dict(rank=8, scale=1.0, dtype="bf16", tokens=8, chunks=1), **kw)
        return AttentionStep(X, lin(0, kq, 64), lin(1, 64, 64), lin(2, 64, 64), lin(3, 64, o_in, dY), q_heads=2, kv_heads=1,
                             head_dim=64, seq_start=start, **kw)
    build()
    for kw in (dict(X=X.float(), dtype="f32"), dict(kq=64), dict(o_in=64), dict(start=s.long()), dict(start=s[:1]),
               dict(dY=X[:4]), dict(pos=s.long()), dict(pos=s), dict(tokens=9),
               dict(start=s.cpu()), dict(pos=torch.zeros(8, dtype=torch.int32)), dict(inv_freq=torch.ones(3))):
        with pytest.raises(ValueError):
            build(**kw)


@pytest.mark.parametrize("captured", [False, True])
def test_another_batch_of_the_same_step(L, captured):
    """set_sequences gives a step another batch: rows that are padding in it, after they were in a sequence, add
    nothing to any gradient, in eager and in captured steps. The caller's own table is not read again."""
    first, second = [0, 100, 333], [0, 31, 260]
    st, rnd = make(first, 0)
    dY = st.o.dY.clone()
    graph = torch.cuda.CUDAGraph()
    if captured:
        st.forward_backward(0)
        torch.cuda.synchronize()
        st.arena.grads.zero_()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            st.arena.grads.zero_()
            st.forward_backward(0)

    def step():
        if captured:
            graph.replay()
        else:
            st.arena.grads.zero_()
            st.forward_backward(0)
        torch.cuda.synchronize()

    step()
    check(st, first)
    table = torch.tensor(second, dtype=torch.int32, device="cuda")
    st.o.dY[second[-1]:] = 0
    st.set_sequences(table)
    table.zero_()
    step()
    check(st, second)
    st.o.dY.copy_(dY)
    st.set_sequences(torch.tensor(first, dtype=torch.int32, device="cuda"))
    step()
    check(st, first)
    with pytest.raises(ValueError):
        st.set_sequences(torch.tensor([0, 333], dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        st.set_sequences(torch.tensor(first, device="cuda"))
