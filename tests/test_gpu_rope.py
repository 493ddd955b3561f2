"""Norm of each query and key head with the rotation by position, forward and backward, against float64.

A value passes through the squares' sum (dim fp32 additions, relative 2^-24 each at most: dim 2^-24), a
square root and a division (2^-22 together), three products and one addition (2^-22 of the terms' sizes).
E = (dim + 16) 2^-24 of |a c| + |b s| covers it, and the backward pass's second sum with it. bf16 outputs add
a rounding of 2^-8. The weights' gradients add n = T heads terms: at most 2 E of the terms' sizes, and n 2^-24
of them in the worst order (n < 2^20 here; lanes, CTAs and trees keep the order's part far below).
"""
import numpy as np
import pytest
import torch

from oracle import attention_oracle as A

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bwd_adapter_adamw_gb300 import binding
    return binding


class Heads:
    def __init__(self, L, T, hq, hk, dim, dtype="bf16", pairs=False, norm=True, fused=False, seed=0, n_pos=500, pos=None):
        self.L, self.T, self.hq, self.hk, self.dim, self.pairs, self.norm, self.n_pos = L, T, hq, hk, dim, pairs, norm, n_pos
        self.dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
        size = torch.exp(rnd(T, hq + hk, 1))
        x = (rnd(T, hq + hk, dim) * size).to(self.dt).cuda()
        if fused:
            w = torch.full((T, (hq + hk) * dim + 16), 77.0, dtype=self.dt, device="cuda")
            w[:, :(hq + hk) * dim] = x.flatten(1)
            self.q = w[:, :hq * dim].unflatten(1, (hq, dim))
            self.k = w[:, hq * dim:(hq + hk) * dim].unflatten(1, (hk, dim)) if hk else None
        else:
            self.q, self.k = x[:, :hq].clone(), x[:, hq:].clone() if hk else None
        self.gq, self.gk = ((1 + 0.2 * rnd(dim)).cuda(), (1 + 0.2 * rnd(dim)).cuda()) if norm else (None, None)
        self.dyq, self.dyk = rnd(T, hq, dim).to(self.dt).cuda(), rnd(T, hk, dim).to(self.dt).cuda()
        self.pos = (torch.randint(0, n_pos, (T,), generator=g) if pos is None else torch.tensor(pos)).int().cuda()
        inv = 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
        self.table = torch.empty(n_pos, dim // 2, 2, device="cuda")
        L.lora_rope_table(n_pos, dim, inv.cuda(), self.table)
        self.cs = self.table.double().cpu().numpy()[self.pos.cpu().numpy().clip(0, n_pos - 1)]
        ld = self.q.stride(0), self.k.stride(0) if hk else 0
        self.desc = L.make_rope_desc(hq, hk, dim, L.LORA_BF16 if dtype == "bf16" else L.LORA_F32,
                                     L.LORA_ROPE_PAIRS if pairs else L.LORA_ROPE_HALVES, EPS, ld_q=ld[0], ld_k=ld[1])
        self.yq, self.yk = torch.full_like(self.dyq, 77.0), torch.full_like(self.dyk, 77.0)
        self.dq = torch.full((T, ld[0]), 77.0, dtype=self.dt, device="cuda")
        self.dk = torch.full((T, max(ld[1], 1)), 77.0, dtype=self.dt, device="cuda")
        self.dgq0, self.dgk0 = rnd(dim).cuda(), rnd(dim).cuda()
        self.ws = torch.empty(L.lora_rope_backward_workspace_size(self.desc, T), dtype=torch.uint8, device="cuda")

    def forward(self, stream=None):
        self.L.lora_rope_forward(self.desc, self.T, self.q, self.k, self.gq, self.gk, self.pos, self.table, self.n_pos,
                                 self.yq, self.yk if self.hk else None, stream=stream)

    def backward(self):
        self.dgq, self.dgk = (self.dgq0.clone(), self.dgk0.clone()) if self.norm else (None, None)
        self.L.lora_rope_backward(self.desc, self.T, self.q if self.norm else None, self.k if self.norm else None, self.gq,
                                  self.gk, self.pos, self.table, self.n_pos, self.dyq, self.dyk if self.hk else None,
                                  self.dq, self.dk if self.hk else None, self.dgq, self.dgk if self.hk else None, self.ws)

    def sides(self):
        for n in ("q", "k")[:2 if self.hk else 1]:
            yield n, getattr(self, n).double().cpu().numpy(), getattr(self, "g" + n), getattr(self, "hq" if n == "q" else "hk")

    def live(self):
        return (self.pos >= 0).cpu().numpy()

    def err(self, ref, size):
        e = (self.dim + 16) * 2.0 ** -24 * size
        return e + (2.0 ** -8 * (np.abs(ref) + e) if self.dt == torch.bfloat16 else 2.0 ** -24 * np.abs(ref))

    def sizes(self, x):
        """|a| + |b| of each pair, an upper bound of the turned terms."""
        a, b = A._pairs(self.dim, self.pairs)
        s = np.empty_like(x)
        s[..., a] = s[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
        return s

    def check_forward(self):
        m = self.live()
        for n, x, gamma, _ in self.sides():
            gam = gamma.double().cpu().numpy() if self.norm else None
            ref = A.rope_forward(x, gam, self.cs, EPS, self.pairs)
            h = x / np.sqrt((x * x).mean(-1, keepdims=True) + EPS) * gam if self.norm else x
            got = getattr(self, "y" + n).double().cpu().numpy()
            assert np.all((np.abs(got - ref) <= self.err(ref, self.sizes(h)))[m]), n
            assert np.all(got[~m] == 77.0)

    def check_backward(self):
        m = self.live()
        for n, x, gamma, heads in self.sides():
            x = x[m]
            dy = getattr(self, "dy" + n).double().cpu().numpy()[m]
            gam = gamma.double().cpu().numpy() if self.norm else None
            ref, dg = A.rope_backward(x, gam, self.cs[m], dy, EPS, self.pairs)
            size = self.sizes(dy)
            if self.norm:
                r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)
                xh = np.abs(x) * r
                g = size * np.abs(gam)
                terms = (size * xh).sum((0, 1))
                size = r * (g + xh * (g * xh).mean(-1, keepdims=True)) * 2
            buf = getattr(self, "d" + n)
            got = buf[:, :heads * self.dim].unflatten(1, (heads, self.dim)).double().cpu().numpy()
            assert np.all(np.abs(got[m] - ref) <= self.err(ref, size)), n
            assert np.all(got[~m] == 77.0) and bool((buf[:, heads * self.dim:] == 77.0).all())
            if self.norm:
                d0 = getattr(self, f"dg{n}0").double().cpu().numpy()
                got = getattr(self, "dg" + n).double().cpu().numpy()
                room = (2 * (self.dim + 16) + x.shape[0] * heads) * 2.0 ** -24 * (terms + np.abs(d0))
                assert np.all(np.abs(got - d0 - dg) <= room), n


SHAPES = [(1, 1, 1, 64), (1, 32, 8, 128), (3, 5, 3, 64), (7, 4, 0, 128), (33, 3, 1, 256), (130, 32, 4, 64), (257, 9, 9, 128),
          (2600, 6, 2, 128), (3001, 2, 1, 64), (1500, 33, 5, 64), (5000, 1, 0, 256), (700, 40, 40, 128)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pairs,norm,fused", [(False, True, False), (True, True, True), (False, False, True), (True, False, False)])
def test_forward_and_backward(L, shape, dtype, pairs, norm, fused):
    h = Heads(L, *shape, dtype=dtype, pairs=pairs, norm=norm, fused=fused, seed=sum(shape))
    h.forward()
    h.backward()
    torch.cuda.synchronize()
    h.check_forward()
    h.check_backward()
    first = [x.clone() for x in (h.yq, h.dq, h.dk)] + ([h.dgq.clone()] if norm else [])
    h.forward()
    h.backward()
    again = [h.yq, h.dq, h.dk] + ([h.dgq] if norm else [])
    assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("norm,times", [(False, 40), (True, 40), (False, 900), (True, 900)])
def test_padding_and_positions_past_the_table(L, norm, times):
    """Padding rows, which may hold anything, are left as they were and add to no gradient; a position past
    the table gives NaN there."""
    pos = [4, -1, 499, 0, -7, 499, 20] * times
    h = Heads(L, len(pos), 6, 2, 128, norm=norm, seed=2, pos=pos)
    pad = h.pos < 0
    for x in (h.q, h.k, h.dyq, h.dyk):
        x[pad] = float("nan")
    h.forward()
    h.backward()
    h.check_forward()
    h.check_backward()
    h.pos[3] = 500
    h.pos[5] = 1 << 30
    far = h.pos >= 500
    h.forward()
    h.backward()
    torch.cuda.synchronize()
    for y in (h.yq, h.yk, h.dq, h.dk):
        bad = torch.isnan(y.flatten(1)).all(1)
        assert torch.equal(bad, far)
    if norm:
        assert bool(torch.isnan(h.dgq).all()) and bool(torch.isnan(h.dgk).all())


@pytest.mark.parametrize("T", [77, 3000])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place(L, dtype, T):
    """Outputs over inputs of the same strides: y over x, dx over dy."""
    h = Heads(L, T, 8, 2, 128, dtype=dtype, seed=5)
    h.forward()
    h.backward()
    q, k, dyq, dyk = h.q.clone(), h.k.clone(), h.dyq.clone(), h.dyk.clone()
    L.lora_rope_forward(h.desc, h.T, q, k, h.gq, h.gk, h.pos, h.table, h.n_pos, q, k)
    L.lora_rope_backward(h.desc, h.T, h.q, h.k, h.gq, h.gk, h.pos, h.table, h.n_pos, dyq, dyk, dyq, dyk, None, None, h.ws)
    assert torch.equal(q, h.yq) and torch.equal(k, h.yk)
    assert torch.equal(dyq.flatten(1), h.dq) and torch.equal(dyk.flatten(1), h.dk)


def test_gradient_of_one_weight_alone(L):
    h = Heads(L, 50, 4, 2, 64, seed=6)
    h.backward()
    only = h.dgk0.clone()
    L.lora_rope_backward(h.desc, h.T, h.q, h.k, h.gq, h.gk, h.pos, h.table, h.n_pos, h.dyq, h.dyk, h.dq, h.dk, None, only, h.ws)
    assert torch.equal(only, h.dgk)


def test_table_at_far_positions(L):
    """Angles in double: 2^-24 of rounding plus the angle's own 2^-52."""
    n, dim = 200_003, 64
    inv = 500000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    t = torch.empty(n, dim // 2, 2, device="cuda")
    L.lora_rope_table(n, dim, inv.cuda(), t)
    want = A.rope_table(n, inv.numpy())
    assert np.abs(t.double().cpu().numpy() - want).max() <= 2.0 ** -24 + n * 2.0 ** -51


def test_rows_past_32_bits(L):
    """Offsets of more than 2^31 elements from the start of a wide buffer."""
    T, hq, hk, dim, width = 530_000, 1, 1, 64, 4096
    w = torch.zeros(T, width, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(T, width, dtype=torch.bfloat16, device="cuda")
    last = torch.randn(3, width, device="cuda").to(torch.bfloat16)
    w[-3:] = last
    d = L.make_rope_desc(hq, hk, dim, ld_q=width, ld_k=width, ld_yq=width, ld_yk=width)
    h = Heads(L, 3, hq, hk, dim, norm=False, pos=[1, 2, 3])
    pos = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    pos[-3:] = h.pos
    L.lora_rope_forward(d, T, w, w[:, dim:], None, None, pos, h.table, h.n_pos, y, y[:, dim:])
    h.q, h.k = last[:, None, :dim].clone(), last[:, None, dim:2 * dim].clone()
    h.forward()
    assert torch.equal(y[-3:, :dim], h.yq[:, 0]) and torch.equal(y[-3:, dim:2 * dim], h.yk[:, 0])
    assert not bool(y[:-3].any())


def test_captured_on_another_stream(L):
    h = Heads(L, 300, 8, 4, 128, seed=11)
    h.forward()
    h.backward()
    want = [x.clone() for x in (h.yq, h.yk, h.dq, h.dk, h.dgq)]
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        h.forward()
        h.backward()
    for _ in range(2):
        for x in (h.yq, h.yk, h.dq, h.dk):
            x.fill_(0.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (h.yq, h.yk, h.dq, h.dk, h.dgq)))
