"""Attention's backward pass in calls that follow one another: same buffers, other contents."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bwd_adapter_adamw_gb300 import binding
    return binding


@pytest.mark.parametrize("lens,hq,hk,dim", [([128] * 8, 32, 4, 64), ([640, 1, 300], 8, 2, 128), ([1500], 9, 9, 64)])
@pytest.mark.parametrize("captured", [False, True])
def test_statistics_of_every_call_are_its_own(L, lens, hq, hk, dim, captured):
    """Forward and backward over the same addresses, with other contents each time: dQ's kernel, which begins beside the
    one ahead, finds this call's log sums and delta, not the call's before."""
    from tests.test_gpu_attention import Batch
    bs = [Batch(L, lens, hq, hk, dim, seed=s) for s in (1, 2)]
    want = []
    for b in bs:
        b.forward()
        b.backward()
        torch.cuda.synchronize()
        want.append([x.clone() for x in (b.o, b.lse, b.dq, b.dk, b.dv)])
    a = Batch(L, lens, hq, hk, dim, seed=3)
    outs = [[torch.zeros_like(x) for x in want[0]] for _ in range(8)]

    def calls():
        for i, out in enumerate(outs):
            b = bs[i % 2]
            for x, y in ((a.q, b.q), (a.k, b.k), (a.v, b.v), (a.do, b.do)):
                x.copy_(y)
            a.forward()
            a.backward()
            for x, y in zip(out, (a.o, a.lse, a.dq, a.dk, a.dv)):
                x.copy_(y)
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
            calls()
        for _ in range(3):
            graph.replay()
    else:
        for _ in range(3):
            calls()
    torch.cuda.synchronize()
    assert L.lora_device_error() == 0
    for i, out in enumerate(outs):
        assert all(torch.equal(x, y) for x, y in zip(out, want[i % 2])), i


def test_positions_of_padding_are_not_read(L):
    """Positions that a caller gives for tokens of no sequence, past the table or before it, change nothing: padding's
    turned rows stay zero and no gradient takes a NaN from them."""
    from tests.test_gpu_attention_step import make
    starts, pad = [0, 70, 200], 30
    outs = []
    for junk in (-1, 3, 1 << 20):
        st, _ = make(starts, pad)
        pos = torch.cat([torch.arange(70), torch.arange(130), torch.full((pad,), junk)]).int().cuda()
        st.set_sequences(st.seq_start.clone(), pos)
        st.forward_backward(0)
        torch.cuda.synchronize()
        outs.append([t.clone() for t in (st.Qr, st.Kr, st.o.Y, st.dX, st.arena.grads)])
    assert bool(torch.isfinite(outs[0][-1]).all())
    for other in outs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(outs[0], other))


@pytest.mark.parametrize("lens,hq,hk,dim", [([8] * 128, 32, 4, 64), ([8] * 128, 32, 8, 128), ([1] * 700, 8, 1, 64)])
def test_many_short_sequences_take_persistent_ctas(L, lens, hq, hk, dim):
    """Every sequence has a key tile of its own, however short: few tokens in many sequences are many items. They take the
    form that a large batch takes, bit for bit (clusters that share a group's heads add their sums in another order)."""
    from tests.test_gpu_attention import Batch
    a = Batch(L, lens, hq, hk, dim, seed=6)
    b = Batch(L, lens, hq, hk, dim, seed=6, pad=60 * 128)
    for x, y in ((b.q, a.q), (b.k, a.k), (b.v, a.v), (b.do, a.do)):
        x[:a.T] = y
    for x in (a, b):
        x.forward()
        x.backward()
    torch.cuda.synchronize()
    assert L.lora_device_error() == 0
    for x, y in ((a.o, b.o), (a.dq, b.dq), (a.dk, b.dk), (a.dv, b.dv)):
        assert torch.equal(x, y[:a.T])
