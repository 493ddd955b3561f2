"""Causal attention over packed sequences, forward and backward, against float64.

Each element is held to the bound of oracle.attention_oracle.attention_bounds (operands rounded to bf16,
sums and exponentials in fp32) plus its own rounding: 2^-8 of the value in bf16.
"""
import numpy as np
import pytest
import torch

from oracle import attention_oracle as A

pytestmark = pytest.mark.gpu
ROUND = 2.0 ** -8


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bwd_adapter_adamw_gb300 import binding
    return binding


def starts_of(lens):
    return [0] + list(np.cumsum(lens).tolist())


class Batch:
    """Inputs of a packed batch on the GPU, the outputs' buffers, and one call of each direction."""

    def __init__(self, L, lens, hq, hk, dim, pad=0, fused=False, seed=0, spread=1.5, starts=None, rows=None):
        self.L, self.hq, self.hk, self.dim = L, hq, hk, dim
        self.starts = starts_of(lens) if starts is None else starts
        self.T = (self.starts[-1] + pad) if rows is None else rows
        g = torch.Generator().manual_seed(seed)
        rnd = lambda h, f: (f * torch.randn(self.T, h, dim, generator=g)).to(torch.bfloat16)   # noqa: E731
        q, k, v, do = rnd(hq, spread), rnd(hk, spread), rnd(hk, 1.0), rnd(hq, 0.5)
        self.fused = fused
        self.q, self.k, self.v = self.place(q, k, v)
        self.do = do.cuda()
        self.o = torch.full((self.T, hq, dim), 77.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((hq, self.T), 77.0, device="cuda")
        self.dq, self.dk, self.dv = self.place(*(torch.full_like(x, 77.0) for x in (q, k, v)))
        self.plan_now()

    def place(self, q, k, v):
        if not self.fused:
            return q.cuda(), k.cuda(), v.cuda()
        w = torch.full((self.T, (self.hq + 2 * self.hk) * self.dim + 8), 77.0, dtype=torch.bfloat16, device="cuda")
        out, at = [], 0
        for x in (q, k, v):
            n = x.shape[1] * self.dim
            w[:, at:at + n] = x.flatten(1).cuda()
            out.append(w[:, at:at + n].unflatten(1, (x.shape[1], self.dim)))
            at += n
        return out

    def plan_now(self):
        L = self.L
        self.n_seq = len(self.starts) - 1
        self.desc = L.make_attn_desc(self.hq, self.hk, self.dim, ld_q=self.q.stride(0), ld_k=self.k.stride(0),
                                     ld_v=self.v.stride(0))
        self.table = torch.tensor(self.starts, dtype=torch.int32, device="cuda")
        self.plan = torch.empty(L.lora_attn_plan_size(self.T, self.n_seq), dtype=torch.uint8, device="cuda")
        L.lora_attn_plan_build(self.T, self.n_seq, self.table, self.plan)
        self.ws = torch.empty(L.lora_attn_backward_workspace_size(self.desc, self.T), dtype=torch.uint8, device="cuda")

    def forward(self):
        self.L.lora_attn_forward(self.desc, self.T, self.n_seq, self.plan, self.q, self.k, self.v, self.o, self.lse)

    def backward(self):
        self.L.lora_attn_backward(self.desc, self.T, self.n_seq, self.plan, self.q, self.k, self.v, self.o, self.lse,
                                  self.do, self.dq, self.dk, self.dv, self.ws)

    def host(self):
        return [x.double().cpu().numpy() for x in (self.q, self.k, self.v)]

    def inside(self):
        m = np.zeros(self.T, bool)
        for a, b in zip(self.starts, self.starts[1:]):
            m[a:b] = True
        return m

    def check_forward(self):
        q, k, v = self.host()
        scale = float(np.float32(self.dim ** -0.5))
        o, lse = A.attention_forward(q, k, v, self.starts, scale)
        m = self.inside()
        eo, el = A.attention_bounds(q, k, v, np.nan_to_num(o), np.nan_to_num(lse), np.zeros_like(q), self.starts, scale, False)
        got, gl = self.o.double().cpu().numpy(), self.lse.double().cpu().numpy()
        assert np.all(np.abs(got - o)[m] <= (ROUND * np.abs(o) + eo * (1 + ROUND))[m])
        assert np.all(np.abs(gl - lse)[:, m] <= el[:, m])
        assert np.all(got[~m] == 77.0) and np.all(gl[:, ~m] == 77.0)

    def exact_statistics(self):
        """The forward's outputs as they would be without its roundings but the last."""
        q, k, v = self.host()
        o, lse = A.attention_forward(q, k, v, self.starts, float(np.float32(self.dim ** -0.5)))
        self.o.copy_(torch.from_numpy(np.nan_to_num(o)))
        self.lse.copy_(torch.from_numpy(np.nan_to_num(lse)))

    def check_backward(self):
        q, k, v = self.host()
        scale = float(np.float32(self.dim ** -0.5))
        o, lse, do = (x.double().cpu().numpy() for x in (self.o, self.lse, self.do))
        want = A.attention_backward(q, k, v, o, lse, do, self.starts, scale)
        room = A.attention_bounds(q, k, v, o, lse, do, self.starts, scale, True)
        m = self.inside()
        for name, got, ref, e in zip(("dq", "dk", "dv"), (self.dq, self.dk, self.dv), want, room):
            got = got.double().cpu().numpy()
            off = np.abs(got - ref) - (ROUND * np.abs(ref) + e * (1 + ROUND))
            assert np.all(off[m] <= 0), (name, float(off[m].max()), int((off[m] > 0).sum()))
            assert np.all(got[~m] == 77.0), name


# lengths, query heads, key heads, head size, rows of padding, one buffer
BATCHES = [([1], 2, 1, 64, 0, False), ([1], 1, 1, 128, 5, True), ([17], 4, 2, 128, 0, False), ([127], 2, 2, 64, 1, True),
           ([128], 4, 1, 128, 0, False), ([129], 3, 1, 128, 0, True), ([256], 2, 2, 64, 0, False),
           ([257], 8, 1, 64, 3, False), ([383, 1, 0, 130], 4, 4, 128, 7, True), ([1] * 9, 6, 2, 128, 0, False),
           ([0, 0, 5, 0], 2, 1, 64, 2, False), ([300, 0, 64, 513], 4, 2, 64, 100, True),
           ([640, 200], 5, 1, 128, 0, False), ([1100], 2, 1, 128, 0, True), ([900, 31, 128], 6, 3, 64, 9, False),
           ([64, 65, 66, 67, 68] * 3, 8, 2, 128, 30, True),
           # more items than SMs: several for each CTA, in both forms of a pair
           ([700, 1, 900, 0, 333, 566], 16, 8, 64, 11, False), ([900, 410, 640], 9, 9, 128, 0, True),
           ([600] * 4, 8, 8, 128, 60, False), ([1300, 129, 700], 16, 16, 64, 0, True)]


@pytest.mark.parametrize("batch", range(len(BATCHES)))
def test_forward(L, batch):
    lens, hq, hk, dim, pad, fused = BATCHES[batch]
    b = Batch(L, lens, hq, hk, dim, pad, fused, seed=batch)
    b.forward()
    torch.cuda.synchronize()
    assert L.lora_device_error() == 0
    b.check_forward()
    first = b.o.clone(), b.lse.clone()
    b.forward()
    assert torch.equal(first[0], b.o) and torch.equal(first[1], b.lse)


@pytest.mark.parametrize("batch", range(len(BATCHES)))
def test_backward(L, batch):
    lens, hq, hk, dim, pad, fused = BATCHES[batch]
    b = Batch(L, lens, hq, hk, dim, pad, fused, seed=100 + batch)
    b.exact_statistics()
    b.backward()
    torch.cuda.synchronize()
    assert L.lora_device_error() == 0
    b.check_backward()
    first = [x.clone() for x in (b.dq, b.dk, b.dv)]
    b.backward()
    assert all(torch.equal(x, y) for x, y in zip(first, (b.dq, b.dk, b.dv)))
