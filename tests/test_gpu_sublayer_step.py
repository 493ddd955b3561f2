"""The sublayer step: what it adds up, and that its options mean what they mean in LoraStep."""
import numpy as np
import pytest
import torch

from oracle import sublayer_oracle as S
from tests.helpers import to64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bwd_adapter_adamw_gb300 import binding
    return binding


def _step(L, T, dim, outs, dtype="bf16", **kw):
    from bwd_adapter_adamw_gb300.step import Linear, SublayerStep
    g = torch.Generator(device="cuda").manual_seed(4)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")   # noqa: E731
    X = rnd(T, dim).to(dt)
    lins = [Linear(0, i, None, (rnd(o, dim) / dim ** 0.5).to(dt), (0.1 * rnd(T, o)).to(dt)) for i, o in enumerate(outs)]
    kw = dict(dict(rank=8, scale=2.0, dtype=dtype, tokens=T, chunks=1, max_norm=0.5), **kw)
    st = SublayerStep(X, lins, **kw)
    st.prepare_weights()
    for l in lins:
        l.A.copy_(rnd(*l.A.shape) / dim ** 0.5)
        l.B.copy_(0.1 * rnd(*l.B.shape))
    st.gamma.copy_(1 + 0.2 * rnd(dim))
    return st


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("outs", [(144,), (400, 144), (256,) * 6, (64,) * 16])
def test_input_gradient_is_rounded_once(L, outs, kind):
    """A residual's gradient a hundred times the projections' contributions. Against float64 from the
    projections' own input gradients an element of dX may be off by its rounding (2^-8 of it), by the
    rounding of the projections' sum (2^-8 of it) carried through the norm's formula term by term, and by
    fp32 arithmetic (2^-18 of the terms' sizes)."""
    T, dim = 300, 272
    st = _step(L, T, dim, outs, kind=kind)
    st.forward_backward(0)
    g = torch.Generator(device="cuda").manual_seed(9)
    res = (100 * st.dX.float().std() * torch.randn(T, dim, generator=g, device="cuda")).to(torch.bfloat16)
    st.arena.grads.zero_()
    st.forward_backward(0, res)
    torch.cuda.synchronize()
    dh = sum(to64(l.dX) for l in st.linears)
    x, gamma, rms = to64(st.X_in), to64(st.gamma), kind == "rms"
    dx, dg, db = S.norm_backward(x, gamma, dh, 1e-5, rms)
    _, mean, rstd = S.norm_forward(x, gamma, None, 1e-5, rms)
    xh = np.abs((x - mean[:, None]) * rstd[:, None])
    size = np.abs(dh) * np.abs(gamma)
    through = rstd[:, None] * (size + (0 if rms else size.mean(1, keepdims=True)) + xh * (size * xh).mean(1, keepdims=True))
    want = dx + to64(res)
    assert np.all(np.abs(to64(st.dX) - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -18) * through)
    assert np.linalg.norm(to64(st.dgamma) - dg) <= (2.0 ** -8 + 2.0 ** -18) * np.linalg.norm((np.abs(dh) * xh).sum(0))
    if not rms:
        assert np.linalg.norm(to64(st.dbeta) - db) <= (2.0 ** -8 + 2.0 ** -18) * np.linalg.norm(np.abs(dh).sum(0))


@pytest.mark.parametrize("n,count", [(1, 8), (2, 4096), (3, 8 * 1001), (4, 1 << 20), (7, 264), (16, 8 * 12345)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sum_of_tensors(L, n, count, dtype):
    """In order in fp32: n - 1 roundings of 2^-24 of the running sum at most, then one to bf16 (2^-8)."""
    g = torch.Generator(device="cuda").manual_seed(n + count)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    src = [(torch.randn(count, generator=g, device="cuda") * 10.0 ** (k % 3)).to(dt) for k in range(n)]
    dst = torch.full((count + 16,), 7.0, dtype=dt, device="cuda")
    L.lora_sum(src, count, L.LORA_F32 if dtype == "f32" else L.LORA_BF16, dst)
    ref, mag = sum(to64(s) for s in src), sum(np.abs(to64(s)) for s in src)
    got = to64(dst)[:count]
    assert np.all(np.abs(got - ref) <= (2.0 ** -8 * np.abs(ref) if dtype == "bf16" else 0) + n * 2.0 ** -23 * mag)
    assert bool((dst[count:] == 7.0).all())
    again = src[0].clone()
    L.lora_sum([again] + src[1:], count, L.LORA_F32 if dtype == "f32" else L.LORA_BF16, again)   # in place
    assert torch.equal(again, dst[:count])


@pytest.mark.parametrize("per_chunk", [False, True])
def test_streams_and_chunks_mean_what_they_mean_in_lora_step(L, per_chunk, monkeypatch):
    """The same projections as a LoraStep over the norm's output, with dropout keyed by chunk: outputs and
    gradients bitwise equal, calls spread over the streams, chunk by chunk where asked."""
    from bwd_adapter_adamw_gb300.step import Linear, LoraStep
    kw = dict(n_streams=3, chunks=3, dropout_p=0.2, seed=11)
    st = _step(L, 384, 272, (400, 144, 256, 64), **kw)
    st.beta.normal_()
    calls, forward = [], L.lora_forward

    def counted(d, c, n, *a, **k):
        calls.append((n, k["stream"].cuda_stream))
        return forward(d, c, n, *a, **k)
    monkeypatch.setattr(L, "lora_forward", counted)
    st.forward_backward(5, per_chunk_calls=per_chunk)
    torch.cuda.synchronize()
    assert len({s for _, s in calls}) == 3
    assert [n for n, _ in calls] == ([128] * 12 if per_chunk else [384] * 4)
    one = LoraStep([Linear(l.layer, l.proj_id, st.H_norm, l.W, l.dY, l.Wp) for l in st.linears], rank=8, scale=2.0,
                   dtype="bf16", tokens=384, max_norm=0.5, **kw)
    for a, b in zip(one.linears, st.linears):
        a.A.copy_(b.A)
        a.B.copy_(b.B)
    one.forward_backward(5, per_chunk)
    torch.cuda.synchronize()
    for a, b in zip(one.linears, st.linears):
        for x, y in ((a.Y, b.Y), (a.dX, b.dX), (a.gA, b.gA), (a.gB, b.gB)):
            assert torch.equal(x, y)
    Y = [l.Y.clone() for l in st.linears]
    calls.clear()
    st.forward(5)
    torch.cuda.synchronize()
    assert len({s for _, s in calls}) == 3
    if not per_chunk:
        assert all(torch.equal(a, l.Y) for a, l in zip(Y, st.linears))
