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
