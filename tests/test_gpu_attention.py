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


@pytest.mark.parametrize("hq,hk,dim", [(2, 1, 128), (3, 1, 64)])
def test_maxima_that_grow_and_fall(L, hq, hk, dim):
    """Scores whose maximum grows by more than the reference's slack with every tile (O is rescaled each time),
    stays, or falls; a row whose weight lies on one key alone."""
    lens = [700]
    for seed, ramp in enumerate((lambda i: 1.0 + i / 40.0, lambda i: 18.0 - i / 40.0, lambda i: 1.0 + 17.0 * (i == 300))):
        b = Batch(L, lens, hq, hk, dim, seed=40 + seed, spread=1.0)
        f = torch.tensor([ramp(i) for i in range(700)], device="cuda")
        base = torch.randn(dim, generator=torch.Generator().manual_seed(seed)).cuda()
        b.k.copy_((base + 0.1 * b.k.float()) * f[:, None, None])
        b.q.copy_(base + 0.1 * b.q.float())
        b.forward()
        b.check_forward()
        b.exact_statistics()
        b.backward()
        b.check_backward()


@pytest.mark.parametrize("hq,hk,dim", [(4, 2, 128), (3, 3, 64)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -3e38])
def test_other_sequences_and_padding_do_not_reach_a_row(L, hq, hk, dim, bad):
    """Sequences full of `bad` beside, between and behind good ones, and padding full of it: the good ones'
    rows are those of a batch without them, bit for bit."""
    lens = [130, 70, 257, 1, 200]
    good = [0, 2, 4]

    def fill(b, v):
        for k in range(len(lens)):
            if k not in good:
                for x in (b.q, b.k, b.v, b.do, b.o):
                    x[b.starts[k]:b.starts[k + 1]] = v
        for x in (b.q, b.k, b.v, b.do, b.o):
            x[b.starts[-1]:] = v
    outs = []
    for v in (0.0, bad):
        b = Batch(L, lens, hq, hk, dim, pad=140, seed=7)
        b.exact_statistics()
        fill(b, v)
        if v != 0.0:
            for k in range(len(lens)):
                if k not in good:
                    b.lse[:, b.starts[k]:b.starts[k + 1]] = v
            b.lse[:, b.starts[-1]:] = v
        b.backward()
        rows = torch.cat([torch.arange(b.starts[k], b.starts[k + 1]) for k in good]).cuda()
        got = [x[rows].clone() for x in (b.dq, b.dk, b.dv)]
        b.o.fill_(77.0)
        b.lse.fill_(77.0)
        b.forward()
        got += [b.o[rows].clone(), b.lse[:, rows].clone()]
        pad = slice(b.starts[-1], b.T)
        assert bool((b.o[pad] == 77.0).all()) and bool((b.dq[pad] == 77.0).all()) and bool((b.dv[pad] == 77.0).all())
        outs.append(got)
    assert all(torch.equal(x, y) for x, y in zip(*outs))
    assert all(bool(torch.isfinite(x.float()).all()) for x in outs[1])


def test_scores_of_minus_infinity_weigh_nothing(L):
    """Keys whose scores overflow to -inf in fp32: the other keys' softmax, and NaN where a row has none else."""
    b = Batch(L, [300], 2, 1, 64, seed=3)
    b.q.copy_(b.q.float().abs() + 0.1)
    b.k[:150] = -3e38
    b.forward()
    torch.cuda.synchronize()
    o, lse = A.attention_forward(*[x[150:] for x in b.host()], [0, 150], float(np.float32(64 ** -0.5)))
    got = b.o.double().cpu().numpy()
    assert np.isnan(got[:150]).all()
    eo, _ = A.attention_bounds(*[x[150:] for x in b.host()], o, lse, np.zeros_like(o), [0, 150], 0.125, False)
    assert np.all(np.abs(got[150:] - o) <= ROUND * np.abs(o) + eo * (1 + ROUND))


@pytest.mark.parametrize("starts,rows", [([0, 100, 60, 250], 250), ([-5, 90, 1000], 200), ([50, 50, 20, 20], 130),
                                         ([30, 130, 131, 400], 450), ([7, 7], 40)])
def test_tables_out_of_order_or_range(L, starts, rows):
    """Offsets are clamped to the tokens, and a sequence begins no earlier than those before it end."""
    end, want = 0, []
    for a, b in zip(starts, starts[1:]):
        a, b = max(0, min(rows, a)), max(0, min(rows, b))
        a = max(a, end)
        if b > a:
            want.append((a, b))
        end = max(end, b)
    b = Batch(L, None, 4, 2, 64, seed=2, starts=starts, rows=rows)
    b.forward()
    got, gl = b.o.double().cpu().numpy(), b.lse.double().cpu().numpy()
    q, k, v = b.host()
    inside = np.zeros(rows, bool)
    for s, e in want:
        inside[s:e] = True
        o, lse = A.attention_forward(q[s:e], k[s:e], v[s:e], [0, e - s], 0.125)
        eo, el = A.attention_bounds(q[s:e], k[s:e], v[s:e], o, lse, np.zeros_like(o), [0, e - s], 0.125, False)
        assert np.all(np.abs(got[s:e] - o) <= ROUND * np.abs(o) + eo * (1 + ROUND))
        assert np.all(np.abs(gl[:, s:e] - lse) <= el)
    assert np.all(got[~inside] == 77.0) and np.all(gl[:, ~inside] == 77.0)


def test_plan_of_other_tokens_or_sequences(L):
    """A plan built for another T or n_seq, or never built: nothing is written."""
    b, other = Batch(L, [200, 100], 4, 2, 64, seed=1), Batch(L, [200, 100, 50], 4, 2, 64, seed=2)
    b.exact_statistics()
    keep = b.o.clone(), b.lse.clone()
    for plan in (other.plan, Batch(L, [100, 100, 100], 4, 2, 64).plan, Batch(L, [290, 9], 4, 2, 64).plan,
                 torch.zeros_like(other.plan)):
        b.plan = plan
        b.o.fill_(77.0)
        b.lse.fill_(77.0)
        b.forward()
        assert bool((b.o == 77.0).all()) and bool((b.lse == 77.0).all())
        b.o.copy_(keep[0])
        b.lse.copy_(keep[1])
        b.backward()
        assert all(bool((x == 77.0).all()) for x in (b.dq, b.dk, b.dv))
    assert L.lora_device_check() == L.LORA_OK


def torch_reference(b, h):
    """(o, lse, dq of head h, and dk, dv of its key head's group) in float64 on the GPU."""
    per = b.hq // b.hk
    g = h // per
    scale = float(np.float32(b.dim ** -0.5))
    dk, dv = torch.zeros(b.T, b.dim, dtype=torch.float64, device="cuda"), torch.zeros(b.T, b.dim, dtype=torch.float64, device="cuda")
    out = None
    for hh in range(g * per, (g + 1) * per):
        o, lse, dq = torch.zeros_like(dk), torch.zeros(b.T, dtype=torch.float64, device="cuda"), torch.zeros_like(dk)
        for s, e in zip(b.starts, b.starts[1:]):
            q, k, v, do = b.q[s:e, hh].double(), b.k[s:e, g].double(), b.v[s:e, g].double(), b.do[s:e, hh].double()
            z = (q @ k.T * scale).masked_fill(torch.ones(e - s, e - s, dtype=torch.bool, device="cuda").triu(1), -torch.inf)
            lse[s:e] = z.logsumexp(1)
            p = (z - lse[s:e, None]).exp()
            o[s:e] = p @ v
            dp = do @ v.T - (do * o[s:e]).sum(1, keepdim=True)
            ds = p * dp * scale
            dq[s:e] = ds @ k
            dk[s:e] += ds.T @ q
            dv[s:e] += p.T @ do
        if hh == h:
            out = o, lse, dq
    return (*out, dk, dv)


@pytest.mark.parametrize("lens,hq,hk,dim", [([8192], 8, 8, 128), ([5000, 3192], 16, 2, 64), ([4097, 1, 2047, 2048], 6, 2, 128)])
def test_long_sequences(L, lens, hq, hk, dim):
    """Whole forward and backward, the backward from the forward's own outputs, in the 2-norm: two operands rounded
    to bf16 (2^-8 each at most, of random sign) and the output's rounding, 3 x 2^-8 in all; O's rounding in delta
    adds as much to dq and dk."""
    b = Batch(L, lens, hq, hk, dim, seed=1)
    b.forward()
    b.backward()
    torch.cuda.synchronize()
    assert L.lora_device_error() == 0
    for h in (0, hq - 1):
        g = h // (hq // hk)
        o, lse, dq, dk, dv = torch_reference(b, h)
        off = lambda x, y: float((x.double() - y).norm() / y.norm())   # noqa: E731
        assert off(b.o[:, h], o) <= 3 * ROUND and off(b.lse[h], lse) <= 1e-5
        assert off(b.dq[:, h], dq) <= 6 * ROUND and off(b.dk[:, g], dk) <= 6 * ROUND and off(b.dv[:, g], dv) <= 3 * ROUND


def test_rows_past_32_bits(L):
    """Sequences more than 2^31 elements behind the start of wide buffers."""
    width, T, hq, hk, dim = 8192, 270_000, 2, 1, 64
    w = torch.zeros(T, width, dtype=torch.bfloat16, device="cuda")
    small = Batch(L, [200, 90], hq, hk, dim, seed=4)
    at = T - small.T
    for x, c in ((small.q, 0), (small.k, 128), (small.v, 192), (small.do, 512)):
        w[at:, c:c + x.shape[1] * dim] = x.flatten(1)
    view = lambda c, h: w[:, c:c + h * dim].unflatten(1, (h, dim))   # noqa: E731
    d = L.make_attn_desc(hq, hk, dim, ld_q=width, ld_k=width, ld_v=width, ld_o=width)
    table = torch.tensor([at, at + 200, T], dtype=torch.int32, device="cuda")
    plan = torch.empty(L.lora_attn_plan_size(T, 2), dtype=torch.uint8, device="cuda")
    L.lora_attn_plan_build(T, 2, table, plan)
    lse = torch.zeros(hq, T, device="cuda")
    L.lora_attn_forward(d, T, 2, plan, view(0, hq), view(128, hk), view(192, hk), view(256, hq), lse)
    small.forward()
    small.backward()
    assert torch.equal(w[at:, 256:384], small.o.flatten(1)) and torch.equal(lse[:, at:], small.lse)
    ws = torch.empty(L.lora_attn_backward_workspace_size(d, T), dtype=torch.uint8, device="cuda")
    L.lora_attn_backward(d, T, 2, plan, view(0, hq), view(128, hk), view(192, hk), view(256, hq), lse, view(512, hq),
                         view(640, hq), view(768, hk), view(832, hk), ws)
    assert torch.equal(w[at:, 640:768], small.dq.flatten(1))
    # (the few tokens' call shares a group's heads between CTAs and adds their sums in another order)
    for c, x in ((768, small.dk), (832, small.dv)):
        x.copy_(w[at:, c:c + dim].unflatten(1, (1, dim)))
    small.check_backward()
    assert not bool(w[:at].any())


def test_one_plan_on_two_streams_and_in_graphs(L):
    """Two layers' calls at once over one plan, each with its own workspace, eager and captured: each layer's own
    results."""
    lens = [300, 500, 129, 95]
    a, b = (Batch(L, lens, 8, 2, 64, pad=3, seed=s) for s in (1, 2))
    for x in (a, b):
        x.forward()
        x.backward()
    torch.cuda.synchronize()
    outs = lambda x: (x.o, x.lse, x.dq, x.dk, x.dv)   # noqa: E731
    want = [[t.clone() for t in outs(x)] for x in (a, b)]
    b.plan = a.plan
    streams = [torch.cuda.Stream() for _ in range(2)]
    for rep in range(5):
        for x in (a, b):
            for t in outs(x):
                t.fill_(77.0)
        torch.cuda.synchronize()
        for x, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                x.forward()
                x.backward()
        torch.cuda.synchronize()
        assert all(torch.equal(t, u) for x, w in zip((a, b), want) for t, u in zip(outs(x), w))
    graphs = []
    for x, s in zip((a, b), streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            x.forward()
            x.backward()
        graphs.append(g)
    for x in (a, b):
        for t in outs(x):
            t.fill_(77.0)
    torch.cuda.synchronize()
    for g, s in zip(graphs, streams):
        with torch.cuda.stream(s):
            g.replay()
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(t, u) for x, w in zip((a, b), want) for t, u in zip(outs(x), w))


@pytest.mark.parametrize("lens,hq,hk,dim", [([640], 8, 1, 128), ([2048], 32, 8, 128), ([300, 17, 900], 16, 4, 64)])
def test_calls_in_a_row_wait_for_one_another(L, lens, hq, hk, dim):
    """The backward pass's last kernel begins beside the one ahead of it: what follows in the stream, here a second
    batch with the same workspace and a kernel that overwrites the queries, still finds both complete."""
    a, b = Batch(L, lens, hq, hk, dim, seed=1), Batch(L, lens, hq, hk, dim, seed=2)
    b.ws = a.ws
    want = []
    for x in (a, b):
        x.forward()
        x.backward()
        torch.cuda.synchronize()
        want.append([y.clone() for y in (x.dq, x.dk, x.dv)])
    kept, other = a.q.clone(), torch.full_like(a.q, 3.0)
    desc = L.make_rope_desc(hq, 0, dim)
    pos = torch.zeros(a.T, dtype=torch.int32, device="cuda")
    table = torch.tensor([[1.0, 0.0]], device="cuda").repeat(1, dim // 2, 1)   # no rotation: a copy
    copy = lambda src, dst: L.lora_rope_forward(desc, a.T, src, None, None, None, pos, table, 1, dst, None)   # noqa: E731
    for x in (a, b):
        for y in (x.dq, x.dk, x.dv):
            y.fill_(77.0)
    torch.cuda.synchronize()
    for _ in range(20):
        a.backward()
        copy(other, a.q)
        copy(kept, a.q)
        b.backward()
    torch.cuda.synchronize()
    for x, w in zip((a, b), want):
        assert all(torch.equal(g, y) for g, y in zip((x.dq, x.dk, x.dv), w))


def test_many_sequences(L):
    """More sequences than the plan's threads, most of them of one token or none."""
    g = torch.Generator().manual_seed(0)
    lens = torch.randint(0, 4, (3000,), generator=g).tolist()
    lens[1777] = 400
    b = Batch(L, lens, 2, 1, 64, pad=5, seed=8, spread=1.0)
    b.forward()
    b.check_forward()
    b.exact_statistics()
    b.backward()
    b.check_backward()


LIMITS = [1, 300, 1000, 3000, 10000, 30000, 100000]   # cycles; a launch takes up to about 100000


@pytest.mark.parametrize("lens,hq,hk,dim", [([500, 129, 700], 4, 2, 128), ([300, 300], 8, 1, 64), ([1500], 8, 8, 128),
                                            ([640], 3, 3, 64), ([1100, 1300], 9, 9, 64)])
def test_waits_that_run_out(L, lens, hq, hk, dim):
    """Under a short bound of the pipeline waits, on correct launches: every element of the outputs is its value or
    as it was, the device reports it, and the next call is right."""
    b = Batch(L, lens, hq, hk, dim, seed=5)
    b.exact_statistics()
    keep = b.o.clone(), b.lse.clone()
    b.backward()
    want = [x.clone() for x in (b.dq, b.dk, b.dv)]
    b.forward()
    fwd = b.o.clone(), b.lse.clone()
    seen = []
    assert L.lora_device_error(reset=True) == 0
    for limit in LIMITS:
        for x in (b.dq, b.dk, b.dv):
            x.fill_(77.0)
        b.o.copy_(keep[0])
        b.lse.copy_(keep[1])
        try:
            L.lora_set_wait_limit(limit)
            b.backward()
            back = L.lora_device_check()
            b.o.fill_(77.0)
            b.lse.fill_(77.0)
            L.lora_device_error(reset=True)
            b.forward()
            forw = L.lora_device_check()
        finally:
            L.lora_set_wait_limit(0)
        L.lora_device_error(reset=True)
        seen.append((back, forw))
        for got, w in zip((b.dq, b.dk, b.dv, b.o, b.lse), (*want, *fwd)):
            assert bool(((got == w) | (got == 77.0)).all())
        if back == L.LORA_OK:
            assert all(torch.equal(x, w) for x, w in zip((b.dq, b.dk, b.dv), want))
        if forw == L.LORA_OK:
            assert torch.equal(b.o, fwd[0]) and torch.equal(b.lse, fwd[1])
    assert seen[0] == (L.LORA_ERR_TIMEOUT, L.LORA_ERR_TIMEOUT)
    b.o.copy_(keep[0])
    b.lse.copy_(keep[1])
    b.backward()
    assert L.lora_device_check() == L.LORA_OK
    assert all(torch.equal(x, w) for x, w in zip((b.dq, b.dk, b.dv), want))
