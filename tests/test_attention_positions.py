"""Positions of a packed batch's tokens, as AttentionStep makes them of the sequences' table, against the header's rule
written out: offsets are clamped to the tokens, and a sequence begins no earlier than those before it end."""
import random

import pytest
import torch


def rule(starts, T):
    pos, end = [-1] * T, 0
    for a, b in zip(starts, starts[1:]):
        a, b = max(0, min(T, a)), max(0, min(T, b))
        for i in range(max(a, end), b):
            pos[i] = i - max(a, end)
        end = max(end, b)
    return pos


def positions(starts, T):
    from bwd_adapter_adamw_gb300 import build
    build.build()
    from bwd_adapter_adamw_gb300.step import AttentionStep
    return AttentionStep._positions(torch.tensor(starts, dtype=torch.int32), T).tolist()


@pytest.mark.parametrize("starts,T", [([0, 4, 9], 9), ([0, 4, 4, 7], 9), ([2, 5], 9), ([5, 3, 10], 10), ([0, 6, 3, 9], 9),
                                      ([-4, 3, 80], 9), ([9, 9], 9), ([7, 7, 2, 2], 9), ([8, 1, 0, 6], 9), ([0, 1], 1)])
def test_positions_follow_the_plan(starts, T):
    assert positions(starts, T) == rule(starts, T)


def test_positions_of_any_table():
    rng = random.Random(5)
    for _ in range(300):
        T = rng.randint(1, 20)
        starts = [rng.randint(-3, T + 3) for _ in range(rng.randint(2, 7))]
        assert positions(starts, T) == rule(starts, T), (starts, T)
