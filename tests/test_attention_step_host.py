"""What AttentionStep refuses before it allocates or launches anything (no GPU is needed to find it)."""
import pytest
import torch


def build(dim=64, q_heads=4, kv_heads=2, head_dim=64, T=8, **kw):
    from bwd_adapter_adamw_gb300 import build as b
    b.build()
    from bwd_adapter_adamw_gb300.step import AttentionStep, Linear
    t = lambda *s: torch.zeros(s, dtype=torch.bfloat16)   # noqa: E731
    q, k, v = (Linear(0, i, None, t(n * head_dim, dim), None) for i, n in enumerate((q_heads, kv_heads, kv_heads)))
    o = Linear(0, 3, None, t(dim, q_heads * head_dim), t(T, dim))
    kw = dict(dict(rank=8, scale=1.0, dtype="bf16", tokens=T, chunks=1), **kw)
    try:
        return AttentionStep(t(T, dim), q, k, v, o, q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim,
                             seq_start=torch.tensor([0, T], dtype=torch.int32), **kw)
    finally:
        assert q.dY is None and k.dY is None and v.dY is None and o.X is None


@pytest.mark.parametrize("kw", [dict(head_dim=256), dict(head_dim=32), dict(head_dim=96), dict(q_heads=3, kv_heads=2),
                                dict(q_heads=2, kv_heads=4), dict(q_heads=0, kv_heads=1), dict(kv_heads=0),
                                dict(head_eps=-1.0), dict(head_eps=float("nan")), dict(n_pos=0),
                                dict(n_pos=(1 << 24) + 1), dict(inv_freq=torch.ones(31))])
def test_shapes_that_the_operators_refuse(kw):
    """The rotation takes heads of 256 and heads that do not divide, the attention does not: the step refuses them when it
    is made, with the projections as they were."""
    with pytest.raises(ValueError):
        build(**kw)
