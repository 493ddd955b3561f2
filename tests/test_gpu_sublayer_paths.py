"""The block-scaled product, the norms and the update where each form of their kernels is chosen: every
tile width with several tiles per CTA, both directions, shared contractions, odd numbers of rows where
two go together, matrices past the chip's room on CUDA cores, late stages over spilled tiles.

Bars: those of the operators' own tests. The update's after more than two stages: a rounding of u, one of X
after each stage but the last, one of each stage's polynomial, and one such share for fp32 arithmetic, each at
most 2^-16 of the largest gain.
"""
import numpy as np
import pytest
import torch

from oracle import sublayer_oracle as S
from tests import test_gpu_block_product as P
from tests import test_gpu_muon as M
from tests import test_gpu_norm as N

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bwd_adapter_adamw_gb300 import binding
    return binding


# T, out, in, dx: 256-wide tiles, fewer than CTAs and several per CTA; 128-wide tiles in two rounds; a
# contraction shared by a cluster; one token whose weight streams behind the quantisation; a contraction too
# long for the one-launch form
@pytest.mark.parametrize("T,out_d,in_d,dx", [(1003, 1552, 2560, True), (1003, 2560, 400, False),
                                             (2050, 2576, 272, False), (2050, 272, 2576, True),
                                             (10200, 384, 144, False), (10200, 144, 384, True),
                                             (200, 400, 4112, False), (200, 4112, 400, True),
                                             (300, 272, 2064, False), (131, 2064, 1040, True),
                                             (1, 8208, 4112, False), (1, 4112, 8208, True),
                                             (3, 144, 12304, False), (5, 12304, 144, True)])
def test_product(L, T, out_d, in_d, dx):
    rng = np.random.default_rng(T * 1009 + out_d * 31 + in_d + dx)
    c, s = P._weight(rng, out_d, in_d)
    X = P._acts(rng, T, out_d if dx else in_d)
    cd, sd, Xd = torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(), X.cuda()
    Y = P._run(L, Xd, cd, sd, out_d, in_d, dx)
    again = P._run(L, Xd, cd, sd, out_d, in_d, dx)
    torch.cuda.synchronize()
    ref, mag = S.block_product(X.float().numpy(), c, s, dx)
    P._check(Y, ref, mag)
    assert torch.equal(Y, again) and L.lora_device_error() == 0


@pytest.mark.parametrize("T,out_d,in_d", [(1, 14336, 4096), (1, 1024, 2560), (37, 2560, 9728)])
def test_product_of_inputs_that_change_in_place(L, T, out_d, in_d):
    """Activations, codes and scales written right ahead of each call, by turns, into the same buffers."""
    g = torch.Generator(device="cuda").manual_seed(T + in_d)

    def inputs():
        X = torch.randn(T, in_d, generator=g, device="cuda").to(torch.bfloat16)
        W = (torch.randn(out_d, in_d, generator=g, device="cuda") / in_d ** 0.5).to(torch.bfloat16)
        c = torch.empty(out_d, in_d, dtype=torch.uint8, device="cuda")
        s = torch.empty(-(-out_d // 128), -(-in_d // 128), device="cuda")
        L.lora_block_quantize_weight(W, out_d, in_d, c, s)
        return X, c, s
    sets = [inputs() for _ in range(2)]
    want = [P._run(L, *v, out_d, in_d, False) for v in sets]
    X, c, s = (torch.empty_like(v) for v in sets[0])
    ws = torch.empty(L.lora_block_product_workspace_size(T, out_d, in_d), dtype=torch.uint8, device="cuda")
    Y = torch.empty_like(want[0])
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for k in range(300):
        for dst, src in zip((X, c, s), sets[k % 2]):
            dst.copy_(src)
        L.lora_block_product(T, out_d, in_d, X, c, s, Y, False, ws)
        differ += (Y != want[k % 2]).sum()
    assert differ.item() == 0


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("T,dim,dtype", [(3701, 2048, "bf16"), (7303, 1024, "bf16"), (14601, 512, "bf16"),
                                         (1827, 4096, "bf16"), (3701, 1024, "f32"), (7303, 512, "f32"),
                                         (14601, 256, "f32"), (1827, 2048, "f32"), (2051, 1000, "bf16"),
                                         (2051, 2000, "bf16"), (2051, 3000, "bf16"), (2051, 4000, "bf16"),
                                         (2051, 500, "f32"), (2051, 1500, "f32")])
def test_norm_of_odd_numbers_of_rows(L, T, dim, dtype, rms):
    N.test_forward_and_backward(L, T, dim - dim % 8, dtype, rms)


@pytest.mark.parametrize("size", [1e-30, 1.0, 1e30])
@pytest.mark.parametrize("rows,cols", [(16, 50000), (50008, 16), (12, 70000), (8, 80000), (128256, 8), (4, 210000),
                                       (210004, 4)])
def test_update_on_cuda_cores_past_the_chips_room(L, rows, cols, size):
    pr = M.Problem(L, [(rows, cols, "A" if rows < cols else "B", 0)], seed=14, momentum=size == 1.0,
                   grad=lambda rng, r, c: M._grad(rng, r, c) * size)
    pr.run(zero=True)
    pr.check(zero=True)


@pytest.mark.parametrize("steps", [6, 7, 8])
@pytest.mark.parametrize("rows,cols", [(64, 14336), (12288, 64), (40, 30000)])
def test_late_stages_over_spilled_tiles(L, rows, cols, steps):
    pr = M.Problem(L, [(rows, cols, "A", 0)], seed=15)
    pr.run(steps=steps)
    n = rows * cols
    p0, g0, m0 = (v[:n].reshape(rows, cols) for v in pr.before)
    want, m = S.muon_update(p0, g0, m0, c=M.C, lr=M.LR, kind="A", mu=M.MU, wd=M.WD, ratio=4.0, steps=steps)
    _, gain = S.newton_schulz(M.C * g0 + M.MU * m, steps=steps)
    stages = -(-steps // 3)
    got = pr.p[:n].double().cpu().numpy().reshape(rows, cols)
    tol = M.LR * max(1.0, rows / cols) ** 0.5 * (2 * stages + 1) * gain * 2.0 ** -16 + 1e-6 * np.linalg.norm(want)
    assert np.linalg.norm(got - want) <= tol, (np.linalg.norm(got - want), tol)
    assert np.linalg.norm(pr.m[:n].double().cpu().numpy() - m.reshape(-1)) <= 1e-6 * np.linalg.norm(m)
