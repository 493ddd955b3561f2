"""The rotation's backward pass where the norms of queries and keys share one weight and one gradient."""
import pytest
import torch

from tests.test_gpu_rope import Heads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bwd_adapter_adamw_gb300 import binding
    return binding


@pytest.mark.parametrize("T,hq,hk,dim,dtype", [(1, 4, 2, 64, "bf16"), (700, 6, 3, 128, "f32"), (4000, 8, 8, 256, "bf16"),
                                               (50, 3, 0, 64, "f32")])
def test_one_gradient_array_takes_both_sums(L, T, hq, hk, dim, dtype):
    """The array takes the queries' sum, then the keys': the same two fp32 additions as into arrays of their own, of which
    the second starts from the first's result. Many reruns, each the same."""
    h = Heads(L, T, hq, hk, dim, dtype=dtype, seed=T)
    start, ks = h.dgq0, []
    h.gk = h.gq if hk else h.gk

    def call(dgq, dgk):
        L.lora_rope_backward(h.desc, T, h.q, h.k, h.gq, h.gk, h.pos, h.table, h.n_pos, h.dyq, h.dyk if hk else None, h.dq,
                             h.dk if hk else None, dgq, dgk, h.ws)
    first, only_k = start.clone(), torch.zeros_like(start)
    call(first, None)
    call(None, only_k)
    want = first + only_k
    for _ in range(20):
        both = start.clone()
        call(both, both)
        ks.append(both)
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in ks)
