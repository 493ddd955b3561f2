"""The orthogonalised (Newton-Schulz) update against float64.

Tolerance. The long-axis operands are held with at least 16 significant bits, so each of the
roundings of u, of X after a stage and of a stage's polynomial moves X by at most 2^-16 of its
Frobenius norm (1 at the start), and the sequence multiplies a direction by at most the largest
gain f(sigma) / sigma over the matrix's singular values. Four such roundings and the fp32
arithmetic of the small matrices (another such share) bound the error's Frobenius norm by
5 gain 2^-16.
"""
import numpy as np
import pytest
import torch

from oracle import sublayer_oracle as S

pytestmark = pytest.mark.gpu

LR, MU, WD, C = 0.5, 0.95, 0.01, 1.0 / 64


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bwd_adapter_adamw_gb300 import binding
    return binding


def _grad(rng, rows, cols, fall=0.0, rank=None):
    s, n = min(rows, cols), max(rows, cols)
    k = s if rank is None else rank
    g = (rng.standard_normal((s, k)) * np.exp(-fall * np.arange(k) / k)) @ rng.standard_normal((k, n))
    return (g if rows == s else g.T).astype(np.float32)


class Problem:
    """Matrices [(rows, cols, kind, group)], side by side in the arenas with gaps of 8 elements."""

    def __init__(self, L, mats, seed=0, fall=0.0, rank=None, grad=None, statuses=None, gap=8,
                 momentum=True):
        rng = np.random.default_rng(seed)
        self.L, self.mats = L, []
        n_groups = 1 + max(m[3] for m in mats)
        at, ranges = 0, []
        p, g, m = [], [], []
        for gi in range(n_groups):
            lo = at
            for (r, c, kind, group) in mats:
                if group != gi:
                    continue
                self.mats.append(dict(offset=at, rows=r, cols=c, group=gi, kind=L.LORA_KIND_A if kind == "A" else L.LORA_KIND_B))
                at += r * c + gap
                p.append(0.1 * rng.standard_normal(r * c + gap))
                g.append(np.concatenate([(_grad(rng, r, c, fall, rank) if grad is None else grad(rng, r, c)).reshape(-1), np.full(gap, 7.0)]))
                m.append(1e-2 * np.concatenate([_grad(rng, r, c, fall, rank).reshape(-1) * momentum, np.full(gap, 7.0)]))
            ranges.append((lo, at - lo))
        f = lambda v: torch.from_numpy(np.concatenate(v).astype(np.float32)).cuda()   # noqa: E731
        self.p, self.g, self.m = f(p), f(g), f(m)
        self.groups = L.make_groups([dict(offset=o, n_a=n, grad_scale=C, lr=LR * (1 + i)) for i, (o, n) in enumerate(ranges)])
        self.sn = torch.tensor([C * (1 + 0.5 * i) if k == 0 else 1.0 for i in range(n_groups) for k in range(2)], dtype=torch.float64, device="cuda")
        self.st = torch.tensor(statuses or [0] * n_groups, dtype=torch.int32, device="cuda")
        self.before = [v.double().cpu().numpy() for v in (self.p, self.g, self.m)]

    def run(self, zero=False, stream=None, **kw):
        L = self.L
        mats = L.make_mats(self.mats)
        ws = torch.empty(max(16, L.lora_muon_workspace_size(mats)), dtype=torch.uint8, device="cuda")
        hp = L.make_muon_hp(momentum=MU, weight_decay=WD, plus_ratio=4.0, **kw)
        L.lora_muon_step(self.p, self.g, self.m, self.groups, mats, hp, self.sn, self.st, zero, ws, stream=stream)
        torch.cuda.synchronize()

    def check(self, zero=False, **kw):
        L = self.L
        p, g, m = (v.double().cpu().numpy() for v in (self.p, self.g, self.m))
        p0, g0, m0 = self.before
        touched = np.zeros(p.size, bool)
        adjust = "rms" if kw.pop("adjust", 0) == L.LORA_MUON_ADJUST_RMS else "aspect"
        for e in self.mats:
            if self.st[e["group"]].item() != 0:
                continue
            sl = slice(e["offset"], e["offset"] + e["rows"] * e["cols"])
            touched[sl] = True
            shape = (e["rows"], e["cols"])
            lr, c = LR * (1 + e["group"]), C * (1 + 0.5 * e["group"])
            kind = "A" if e["kind"] == L.LORA_KIND_A else "B"
            rp, rm = S.muon_update(p0[sl].reshape(shape), g0[sl].reshape(shape), m0[sl].reshape(shape),
                                   c=c, lr=lr, kind=kind, mu=MU, wd=WD, ratio=4.0, adjust=adjust, **kw)
            u = c * g0[sl] + MU * rm.reshape(-1) if kw.get("nesterov", True) else rm.reshape(-1)
            _, gain = S.newton_schulz(u.reshape(shape), kw.get("coef", (3.4445, -4.7750, 2.0315)), kw.get("steps", 5))
            rows, cols = shape
            s = np.sqrt(max(1.0, rows / cols)) if adjust == "aspect" else 0.2 * np.sqrt(max(shape))
            step = lr * s * (4.0 if kind == "B" else 1.0)
            tol = step * 5 * gain * 2.0 ** -16 + 1e-6 * np.linalg.norm(rp)
            assert np.isfinite(p[sl]).all()
            assert np.linalg.norm(p[sl] - rp.reshape(-1)) <= tol, (shape, kind, np.linalg.norm(p[sl] - rp.reshape(-1)) / step, gain)
            assert np.linalg.norm(m[sl] - rm.reshape(-1)) <= 1e-6 * max(np.linalg.norm(rm), 1e-30)
            assert np.all(g[sl] == (0.0 if zero else g0[sl]))
        for now, was in ((p, p0), (g, g0), (m, m0)):
            assert np.array_equal(now[~touched], was[~touched])


SHAPES = [(4, 64), (64, 4), (4, 4), (8, 8), (8, 2048), (256, 8), (12, 100), (100, 12), (16, 1536),
          (4096, 16), (20, 516), (32, 2560), (1024, 32), (36, 72), (48, 1000), (64, 64), (64, 1024),
          (4096, 64), (64, 14336), (14336, 64), (60, 20000)]


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_one_matrix(L, rows, cols):
    kind = "A" if rows <= cols else "B"
    pr = Problem(L, [(rows, cols, kind, 0)], seed=rows + cols)
    pr.run()
    pr.check()


@pytest.mark.parametrize("fall", [3.0, 8.0])
@pytest.mark.parametrize("rows,cols", [(8, 512), (512, 16), (64, 768), (1536, 64)])
def test_falling_spectra(L, rows, cols, fall):
    pr = Problem(L, [(rows, cols, "A" if rows < cols else "B", 0)], seed=1, fall=fall)
    pr.run()
    pr.check()


@pytest.mark.parametrize("rows,cols,rank", [(64, 1024, 1), (64, 1024, 5), (512, 16, 3), (8, 64, 1)])
def test_rank_deficient_gradients(L, rows, cols, rank):
    pr = Problem(L, [(rows, cols, "A", 0)], seed=2, rank=rank)
    pr.run()
    pr.check()


def test_many_matrices_groups_and_kinds(L):
    mats = []
    for i in range(70):
        r = [4, 8, 16, 32, 64][i % 5]
        mats += [(r, 64 + 8 * (i % 7), "A", i % 3), (128 + 8 * (i % 5), r, "B", i % 3)]
    pr = Problem(L, mats, seed=3)
    pr.run(zero=True)
    pr.check(zero=True)


def test_more_matrices_than_one_launch_holds(L):
    pr = Problem(L, [(4, 16, "A", 0)] * 700, seed=4, gap=0)
    pr.run()
    pr.check()


def test_rejected_groups_are_left_untouched(L):
    pr = Problem(L, [(8, 128, "A", 0), (64, 512, "A", 1), (256, 16, "B", 2)], seed=5,
                 statuses=[0, L.LORA_ERR_NONFINITE, 0])
    pr.g[pr.mats[1]["offset"] + 5] = float("nan")
    pr.before[1] = pr.g.double().cpu().numpy()
    pr.run(zero=True)
    torch.cuda.synchronize()
    g1 = slice(pr.mats[1]["offset"], pr.mats[1]["offset"] + 64 * 512)
    assert torch.isnan(pr.g[g1]).sum() == 1
    pr.g[pr.mats[1]["offset"] + 5] = 0.0
    pr.before[1][pr.mats[1]["offset"] + 5] = 0.0
    pr.check(zero=True)


@pytest.mark.parametrize("rows,cols", [(8, 64), (64, 1024), (1024, 64)])
def test_zero_update_leaves_decay_alone(L, rows, cols):
    pr = Problem(L, [(rows, cols, "A", 0)], seed=6, grad=lambda rng, r, c: np.zeros((r, c)), momentum=False)
    pr.run()
    pr.check()


@pytest.mark.parametrize("size", [1e-30, 1e-12, 1e12, 1e30])
@pytest.mark.parametrize("rows,cols", [(8, 128), (512, 64)])
def test_update_does_not_depend_on_the_gradients_size(L, rows, cols, size):
    pr = Problem(L, [(rows, cols, "B", 0)], seed=7, momentum=False,
                 grad=lambda rng, r, c: _grad(rng, r, c) * size)
    pr.run()
    pr.check()


@pytest.mark.parametrize("size", [1e-30, 1.0, 1e30])
@pytest.mark.parametrize("rows,cols", [(64, 10240), (12288, 64), (40, 14336), (64, 30000)])
def test_tiles_past_the_chips_room(L, rows, cols, size):
    """One matrix whose CTAs hold all their tiles, or move some through memory, also where u is
    rescaled on its way."""
    pr = Problem(L, [(rows, cols, "A", 0)], seed=11, momentum=False,
                 grad=lambda rng, r, c: _grad(rng, r, c) * size)
    pr.run()
    pr.check()


def test_long_chains_of_matrices(L):
    """More matrices than clusters, of unequal lengths: the CTAs go from one to the next."""
    mats = [(64, 2048 + 128 * (i % 5), "A", 0) for i in range(90)] + [(700 + 60 * i, 48, "B", 1) for i in range(70)]
    pr = Problem(L, mats, seed=12)
    pr.run(zero=True)
    pr.check(zero=True)


@pytest.mark.parametrize("kw", [dict(steps=1), dict(steps=2), dict(steps=3), dict(steps=4),
                                dict(steps=8), dict(nesterov=False), dict(adjust=1),
                                dict(coef=(2.0, -1.5, 0.5), steps=6)])
@pytest.mark.parametrize("rows,cols", [(8, 300), (640, 64)])
def test_hyperparameters(L, rows, cols, kw):
    pr = Problem(L, [(rows, cols, "A", 0)], seed=8)
    pr.run(**kw)
    pr.check(**kw)


def test_result_is_near_orthogonal(L):
    """Five steps take every singular value above 0.005 of the norm into [0.68, 1.21] (the map's
    interval around one), so the update's rows are near orthonormal."""
    pr = Problem(L, [(64, 4096, "A", 0)], seed=9, momentum=False)
    pr.run()
    p0 = pr.before[0][:64 * 4096]
    x = -(pr.p[:64 * 4096].double().cpu().numpy() - p0 * (1 - LR * WD)) / LR
    sv = np.linalg.svd(x.reshape(64, 4096), compute_uv=False)
    u = np.linalg.svd(pr.before[1][:64 * 4096].reshape(64, 4096), compute_uv=False)
    above = int(np.sum(u / np.linalg.norm(u) > 0.005))
    assert above >= 60 and sv[above - 1] > 0.67 and sv.max() < 1.22


def test_reruns_bitwise_equal_on_another_stream(L):
    mats = [(8, 512, "A", 0), (64, 4096, "A", 0), (14336, 64, "B", 1), (256, 32, "B", 1)]
    a, b = Problem(L, mats, seed=10), Problem(L, mats, seed=10)
    torch.cuda.synchronize()
    a.run()
    b.run(stream=torch.cuda.Stream())
    assert torch.equal(a.p, b.p) and torch.equal(a.m, b.m)
