"""Host-side behaviour of the operators around the adapted linear and of the step that runs them:
refusals, memory that runs out, what the step hands to the library. No GPU."""
import os
import subprocess
import sys

import pytest

FAKE = 1 << 20   # an aligned non-null address; never dereferenced (validation fails first)
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def L():
    from bwd_adapter_adamw_gb300 import build
    build.build()
    from bwd_adapter_adamw_gb300 import binding
    return binding


@pytest.mark.parametrize("offset", [(1 << 63) - 4, (1 << 63) - 512, (1 << 62), 2048 + 4, 2048])
def test_update_refuses_matrices_whose_end_overflows(L, offset):
    groups = L.make_groups([dict(offset=0, n_a=1024, n_b=1024, grad_scale=1.0, lr=0.1)])
    mats = L.make_mats([dict(offset=offset, rows=8, cols=64, kind=L.LORA_KIND_A)])
    assert L.lora_muon_step(FAKE, FAKE, FAKE, groups, mats, L.make_muon_hp(), FAKE, FAKE, False, FAKE, 1 << 30,
                            stream=0, check=False) == L.LORA_ERR_INVALID
    if offset > (1 << 63) - 512:
        assert L.lora_muon_workspace_size(mats) == 0


def test_memory_that_runs_out_is_a_status(L):
    """Two million matrices with 24 MB of address space left: the update's host tables do not fit."""
    code = """
import ctypes as C, resource, sys
import numpy as np
sys.path.insert(0, %r)
from bwd_adapter_adamw_gb300 import binding as L
n = 2000000
a = np.zeros(n, dtype=[("offset", "i8"), ("rows", "i8"), ("cols", "i8"), ("group", "i4"), ("kind", "i4")])
assert a.itemsize == C.sizeof(L.lora_mat)
a["offset"], a["rows"], a["cols"] = 16 * np.arange(n), 4, 4
mats = (L.lora_mat * n).from_buffer(a)
groups = L.make_groups([dict(offset=0, n_a=16 * n, grad_scale=1.0, lr=0.1)])
back = (L.lora_mat * n).from_buffer(a[::-1].copy())
size = [int(l.split()[1]) for l in open("/proc/self/status") if l.startswith("VmSize")][0] << 10
resource.setrlimit(resource.RLIMIT_AS, (size + (24 << 20), resource.getrlimit(resource.RLIMIT_AS)[1]))
F = 1 << 20
assert L.lora_muon_workspace_size(mats) == 0
assert L.lora_muon_workspace_size(back) == 0
for m in (mats, back):
    st = L.lora_muon_step(F, F, F, groups, m, L.make_muon_hp(), F, F, False, F, 1 << 30, stream=0, check=False)
    assert st == L.LORA_ERR_UNSUPPORTED, st
print("ok")
""" % ROOT
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", (r.returncode, r.stderr[-500:])


CSRC = os.path.join(ROOT, "bwd_adapter_adamw_gb300", "csrc")


def test_what_is_found_per_device_is_kept_per_device(tmp_path):
    """Attributes are set once on each device and again after a failure; values are found per device."""
    src = tmp_path / "t.cpp"
    src.write_text("""
#include "per_device.h"
#include <cassert>
#include <initializer_list>
int main() {
  std::atomic<uint64_t> done{0};
  int calls = 0, status = 0;
  auto set = [&] { ++calls; return status; };
  for (int dev : {0, 1, 0, 1, 63, 63, 0}) assert(lora::once_on_device(done, dev, 0, set) == 0);
  assert(calls == 3);
  status = 7;                                       // a device that fails is asked again
  assert(lora::once_on_device(done, 5, 0, set) == 7 && lora::once_on_device(done, 5, 0, set) == 7 && calls == 5);
  status = 0;
  assert(lora::once_on_device(done, 5, 0, set) == 0 && lora::once_on_device(done, 5, 0, set) == 0 && calls == 6);
  for (int dev : {-1, 64, 64}) assert(lora::once_on_device(done, dev, 0, set) == 0);
  assert(calls == 9);
  static lora::DeviceValues<4> v;
  int found = 0;
  for (int dev = 0; dev < 3; ++dev)
    for (int k = 0; k < 2; ++k) assert(v.get(dev, 3, [&] { ++found; return 10 * dev; }) == 10 * dev);
  assert(found == 3);
  assert(v.get(0, 2, [] { return -1; }) == -1 && v.get(0, 2, [] { return 4; }) == 4);
  return 0;
}
""")
    exe = str(tmp_path / "t")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", exe], check=True)
    assert subprocess.run([exe]).returncode == 0


def test_no_launcher_keeps_a_devices_state_for_the_process():
    """Every place that sets a kernel's attribute or asks how many clusters are resident does so through
    the helpers that keep it per device, or through a table by device."""
    import re
    for f in sorted(os.listdir(CSRC)):
        text = open(os.path.join(CSRC, f)).read()
        plain = re.findall(r"static (?:bool|int|cudaError_t|std::atomic<int>) \w+(?:\[[^\]]*\])*\s*(?:=[^;(]*|=[^;]*\([^;]*)?;", text)
        assert all("[64]" in p for p in plain), (f, plain)


def test_sum_refusals(L):
    def call(n=2, src=None, count=64, dtype=None, dst=FAKE):
        return L.lora_sum([FAKE] * n if src is None else src, count, L.LORA_BF16 if dtype is None else dtype, dst,
                          stream=0, check=False)
    assert call(n=0) == L.LORA_ERR_INVALID
    assert call(n=L.LORA_SUM_MAX + 1) == L.LORA_ERR_UNSUPPORTED
    assert call(src=[FAKE, None]) == L.LORA_ERR_INVALID
    assert call(src=[FAKE, FAKE + 8]) == L.LORA_ERR_ALIGN
    assert call(dst=None) == L.LORA_ERR_INVALID
    assert call(dst=FAKE + 2) == L.LORA_ERR_ALIGN
    assert call(count=-8) == L.LORA_ERR_INVALID
    assert call(count=12) == L.LORA_ERR_ALIGN
    assert call(count=1 << 41) == L.LORA_ERR_UNSUPPORTED
    assert call(dtype=L.LORA_BF16_FP8) == L.LORA_ERR_INVALID
    assert call(count=0) == L.LORA_OK


def _sublayer(L, T=16, dim=64, outs=(32, 48), in_dims=None, dt=None, **kw):
    import torch

    from bwd_adapter_adamw_gb300.step import Linear, SublayerStep
    dt = torch.bfloat16 if dt is None else dt
    lins = [Linear(0, i, None, torch.zeros(o, d, dtype=dt), torch.zeros(T, o, dtype=dt))
            for i, (o, d) in enumerate(zip(outs, in_dims or [dim] * len(outs)))]
    kw = dict(dict(rank=8, scale=1.0, dtype="bf16", tokens=T, chunks=1, device="cpu"), **kw)
    return SublayerStep(kw.pop("X", torch.zeros(T, dim, dtype=dt)), lins, **kw)


def test_sublayer_step_refuses_shapes_that_do_not_fit(L):
    """The library takes pointers: a projection of another width would read past the norm's output."""
    import torch
    assert _sublayer(L).n_mag == 2 * 64 and _sublayer(L, kind="rms").n_mag == 64
    for kw in (dict(in_dims=[64, 72]), dict(X=torch.zeros(8, 64, dtype=torch.bfloat16)), dict(tokens=32),
               dict(X=torch.zeros(16, 72, dtype=torch.bfloat16)), dict(X=torch.zeros(16, 128, dtype=torch.bfloat16)[:, ::2]),
               dict(X=torch.zeros(16, 64)), dict(dtype="f32"), dict(dt=torch.float16),
               dict(X=torch.zeros(16, 64, dtype=torch.bfloat16), dt=torch.float32), dict(outs=()), dict(outs=(8,) * (L.LORA_SUM_MAX + 1)),
               dict(kind="batch")):
        with pytest.raises(ValueError):
            _sublayer(L, **kw)
    st = _sublayer(L)
    for res in (torch.zeros(16, 72, dtype=torch.bfloat16), torch.zeros(16, 64), True):
        with pytest.raises(ValueError):
            st.forward_backward(0, res)


def test_sublayer_step_takes_decay_and_ratio_from_its_adamw_settings(L):
    """A and B take the orthogonalised update: with no settings of its own, the decay and the LoRA+ ratio
    of the step's `hp`, which LoraStep gives to AdamW."""
    st = _sublayer(L, hp=L.make_hp(plus_ratio=4.0, weight_decay=0.25))
    assert (st.muon.plus_ratio, st.muon.weight_decay) == (4.0, 0.25)
    st = _sublayer(L, hp=L.make_hp(plus_ratio=4.0), muon=L.make_muon_hp(plus_ratio=2.0))
    assert st.muon.plus_ratio == 2.0


def test_sublayer_step_allocates_one_arena(L, monkeypatch):
    from bwd_adapter_adamw_gb300 import step as S
    made = []

    class Counted(S.Arena):
        def __init__(self, n, device):
            made.append(n)
            super().__init__(n, device)
    monkeypatch.setattr(S, "Arena", Counted)
    st = _sublayer(L)
    assert made == [8 * 64 * 2 + 8 * (32 + 48) + 2 * 64]
    base = st.n_a + st.n_b
    assert st.gamma.data_ptr() == st.arena.params.data_ptr() + 4 * base
    assert st.dbeta.data_ptr() == st.arena.grads.data_ptr() + 4 * (base + 64)
    assert st.linears[1].B.data_ptr() == st.arena.params.data_ptr() + 4 * (st.n_a + 8 * 32)
    with pytest.raises(ValueError):
        _sublayer(L, dora=True)
