"""Bounded waits of the operators around the adapted linear, on correct launches.

The bound of the pipeline waits is shortened (a test hook), from one cycle up to about the time of a
whole launch, so that ordinary waits run out at different places; nothing is broken on purpose. What
such a call may have written is then checked element by element, the status is reported, and with the
default bound back the same call is right on the same context.
"""
import pytest
import torch

from tests.test_gpu_muon import Problem

pytestmark = pytest.mark.gpu

LIMITS = [1, 100, 300, 1000, 3000, 10000, 30000, 100000]   # cycles; a launch takes up to about 400000


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bwd_adapter_adamw_gb300 import binding
    return binding


def _short(L, limit, call):
    """call() under the bound; the status that the device reports for it."""
    assert L.lora_device_error(reset=True) == 0
    try:
        L.lora_set_wait_limit(limit)
        call()
        status = L.lora_device_check()
    finally:
        L.lora_set_wait_limit(0)
    flags = L.lora_device_error(reset=True)
    assert (flags & ~0x7) == 0 and (flags != 0) == (status == L.LORA_ERR_TIMEOUT)
    assert status in (L.LORA_OK, L.LORA_ERR_TIMEOUT)
    return status


# clusters of several CTAs, one CTA per matrix, tiles past the chip's room, several matrices per cluster
UPDATES = [[(64, 14336, "A", 0), (4096, 64, "B", 0), (64, 4096, "A", 0)], [(64, 30000, "A", 0)],
           [(64, 128, "A", 0)] * 40, [(48, 2560 + 128 * (i % 3), "A", 0) for i in range(120)]]


@pytest.mark.parametrize("mats", range(len(UPDATES)))
@pytest.mark.parametrize("size", [1.0, 1e-30])   # the latter: u is rescaled on its way
def test_update_writes_right_parameters_or_none(L, mats, size):
    def problem():
        pr = Problem(L, UPDATES[mats], seed=13, momentum=size == 1.0)
        pr.g *= size
        return pr
    old, new = problem(), problem()
    new.run(zero=True)
    seen = []
    for limit in LIMITS:
        pr = problem()
        seen.append(_short(L, limit, lambda: pr.run(zero=True)))
        for got, was, now in ((pr.p, old.p, new.p), (pr.m, old.m, new.m), (pr.g, old.g, new.g)):
            assert bool(((got == was) | (got == now)).all())
        if seen[-1] == L.LORA_OK:
            assert torch.equal(pr.p, new.p)
    assert seen[0] == L.LORA_ERR_TIMEOUT
    again = problem()
    again.run(zero=True)
    assert L.lora_device_check() == L.LORA_OK
    assert torch.equal(again.p, new.p) and torch.equal(again.m, new.m)


@pytest.mark.parametrize("T,dim,dtype", [(2100, 4096, "bf16"), (1023, 2048, "f32"), (700, 8192, "bf16"),
                                         (3000, 256, "bf16"), (40, 16384, "f32")])
def test_norm_backward_writes_right_rows_and_no_partial_sums(L, T, dim, dtype):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(dim)
    x, dy = (torch.randn(T, dim, generator=g, device="cuda").to(dt) for _ in range(2))
    gamma, st = torch.rand(dim, generator=g, device="cuda"), torch.empty(T, 2, device="cuda")
    d = L.make_norm_desc(dim, L.LORA_NORM_LAYER, L.LORA_BF16 if dtype == "bf16" else L.LORA_F32)
    L.lora_norm_forward(d, T, x, gamma, None, torch.empty_like(x), st)
    ws = torch.empty(L.lora_norm_backward_workspace_size(d, T), dtype=torch.uint8, device="cuda")
    dx, grads = torch.empty_like(x), torch.empty(2 * dim, device="cuda")

    def call():
        dx.fill_(77.0)
        grads.fill_(1.0)
        L.lora_norm_backward(d, T, x, gamma, dy, st, None, dx, grads[:dim], grads[dim:], ws)

    call()
    want, sums = dx.clone(), grads.clone()
    seen = []
    for limit in LIMITS:
        seen.append(_short(L, limit, call))
        assert bool(((dx == 77.0) | (dx == want)).all())
        if seen[-1] == L.LORA_OK:
            assert torch.equal(dx, want) and torch.equal(grads, sums)
        else:
            assert bool(torch.isnan(grads).all())
            groups = L.make_groups([dict(offset=0, n_mag=2 * dim, grad_scale=1.0, max_norm=1.0, lr=1e-3, step=0)])
            sn, status = torch.zeros(2, dtype=torch.float64, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
            pw = torch.empty(L.lora_grad_prepare_workspace_size(groups), dtype=torch.uint8, device="cuda")
            L.lora_grad_prepare(grads, groups, sn, status, pw)
            assert status.item() == L.LORA_ERR_NONFINITE
    assert seen[0] == L.LORA_ERR_TIMEOUT
    call()
    assert L.lora_device_check() == L.LORA_OK
    assert torch.equal(dx, want) and torch.equal(grads, sums)


# the fused and the streaming form, tiles shared by a cluster, tiles of 128 and of 256 outputs
@pytest.mark.parametrize("dx", [False, True])
@pytest.mark.parametrize("T,out_d,in_d", [(1, 2560, 4096), (8, 2560, 4096), (12, 2560, 4096), (37, 2560, 9728),
                                          (100, 4096, 2560), (129, 2560, 2560), (300, 512, 7168), (1000, 2560, 4096)])
def test_product_writes_right_values_or_none(L, T, out_d, in_d, dx):
    g = torch.Generator(device="cuda").manual_seed(T + in_d)
    X = torch.randn(T, out_d if dx else in_d, generator=g, device="cuda").to(torch.bfloat16)
    W = (torch.randn(out_d, in_d, generator=g, device="cuda") / in_d ** 0.5).to(torch.bfloat16)
    c = torch.empty(out_d, in_d, dtype=torch.uint8, device="cuda")
    sc = torch.empty(-(-out_d // 128), -(-in_d // 128), device="cuda")
    L.lora_block_quantize_weight(W, out_d, in_d, c, sc)
    ws = torch.empty(L.lora_block_product_workspace_size(T, out_d, in_d, dx), dtype=torch.uint8, device="cuda")
    Y = torch.empty(T, in_d if dx else out_d, dtype=torch.bfloat16, device="cuda")

    def call():
        Y.fill_(1e30)
        L.lora_block_product(T, out_d, in_d, X, c, sc, Y, dx, ws)

    old = torch.full_like(Y, 1e30)
    call()
    want = Y.clone()
    seen = []
    for limit in LIMITS * 3:
        seen.append(_short(L, limit, call))
        assert bool(((Y == want) | (Y == old) | torch.isnan(Y)).all())
        if seen[-1] == L.LORA_OK:
            assert torch.equal(Y, want)
    assert seen[0] == L.LORA_ERR_TIMEOUT
    call()
    assert L.lora_device_check() == L.LORA_OK
    assert torch.equal(Y, want)
