"""Counts that the window and cache bindings take: whole numbers of any type, and nothing cut off silently."""
import numpy as np
import pytest
import torch

from flashattention_bf16_fwd_b200 import build as fa_build

INT_MAX = 2**31 - 1


@pytest.fixture(scope="module")
def scope():
    fa_build.build()
    from flashattention_bf16_fwd_b200 import _scope
    return _scope


@pytest.mark.parametrize("n,want", [(0, 0), (7, 7), (7.0, 7), (np.int64(5), 5), (np.float32(5), 5), (torch.tensor(3), 3), (True, 1), (-2, -1),
                                    (INT_MAX, INT_MAX), (2**31, INT_MAX), (10**30, INT_MAX), (1e12, INT_MAX), (-2**40, -1), (-1e12, -1)])
def test_whole_numbers(scope, n, want):
    assert scope.count(n) == want


@pytest.mark.parametrize("n", [3.7, 0.5, -0.5, np.float64(1.25), float("nan"), torch.tensor(2.5)])
def test_others_are_refused(scope, n):
    with pytest.raises(ValueError):
        scope.count(n)
    with pytest.raises((ValueError, OverflowError)):
        scope.count(float("inf"))


def test_calls_refuse_them_too(scope):
    from flashattention_bf16_fwd_b200 import cache
    bf, i32 = torch.bfloat16, torch.int32
    kp, table, lens = torch.zeros(7, 2, 16, 64, dtype=bf), torch.zeros(3, 5, dtype=i32), torch.zeros(3, dtype=i32)
    with pytest.raises(ValueError, match="whole"):
        cache.attention_decode(torch.zeros(3, 4, 64, dtype=bf), kp, kp, table, lens, window=2.5)
    with pytest.raises(ValueError, match="whole"):
        cache.cache_reserve(torch.zeros(7, dtype=i32), table, lens, lens, 16.5)
    with pytest.raises(ValueError, match="whole"):
        cache.cache_free(torch.zeros(7, dtype=i32), table, lens, lens, 16.5)


@pytest.mark.gpu
def test_window_calls_refuse_them_too(scope):
    from flashattention_bf16_fwd_b200 import window
    q = torch.zeros(1, 2, 100, 64, dtype=torch.bfloat16, device="cuda")
    o, lse = window.attention_window_fwd(q, q, q, 10.0)
    for kw in (dict(window=9.5), dict(window=9, sinks=0.5), dict(window=9, fix_mode=1.5)):
        with pytest.raises(ValueError, match="whole"):
            window.attention_window_fwd(q, q, q, **kw)
    with pytest.raises(ValueError, match="whole"):
        window.attention_window_bwd(q, q, q, o, lse, q, 9.5)
    with pytest.raises(ValueError, match="whole"):
        window.attention_window_bwd(q, q, q, o, lse, q, 9, 0.5)
