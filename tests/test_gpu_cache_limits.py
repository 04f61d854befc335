"""The cache at the largest tables that its calls accept, a row with room for nearly 2^31 tokens: where a count of
tokens is rounded up to pages or tiles, it passes 2^31."""
import numpy as np
import pytest
import torch

from oracle import paged64

pytestmark = pytest.mark.gpu
FA_ERR_PAGES = -13
PAGE, M = 24, 89478485                                  # M * PAGE = 2^31 - 8


@pytest.fixture(scope="module")
def fa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from flashattention_bf16_fwd_b200 import cache, fa as binding
    binding.cache = cache
    assert binding.fa_check_device_error() == 0
    return binding


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_reserve(fa):
    refs, lens = i32([0] * 40), i32([0])
    table = torch.full((1, M), -1, dtype=torch.int32, device="cuda")
    assert fa.cache.cache_reserve(refs, table, lens, i32([M * PAGE]), PAGE).item() == M - 40
    assert lens.item() == 0 and not refs.any() and (table == -1).all()
    assert fa.cache.cache_reserve(refs, table, lens, i32([M * PAGE + 1]), PAGE).item() == -1
    assert fa.fa_check_device_error() == FA_ERR_PAGES
    lens.fill_(M * PAGE - 60)                           # 12 tokens into the last page but two
    assert fa.cache.cache_reserve(refs, table, lens, i32([60]), PAGE).item() == 0
    assert lens.item() == M * PAGE and table[0, -3:].tolist() == [-1, 0, 1] and refs.tolist() == [1, 1] + [0] * 38
    assert fa.fa_check_device_error() == 0


def test_free_and_compact(fa):
    P = 1000
    kp, vp = (torch.randn(1, P, 1, PAGE, 64, device="cuda").half() for _ in range(2))
    held = torch.arange(M, device="cuda") % 600 + 400   # pages 400 to 999
    table, lens = held.int().view(1, M).contiguous(), i32([M * PAGE])
    refs = torch.bincount(held, minlength=P).int()
    want = torch.arange(P, device="cuda")
    want[600:] = torch.arange(400, device="cuda")       # 600 pages in use: the last 400 move to the first numbers
    moved = kp[0, 600:].clone()
    assert fa.cache.cache_compact(kp, vp, refs, table, lens).item() == 600
    assert fa.fa_check_device_error() == 0
    assert torch.equal(table[0].long(), want[held]) and torch.equal(kp[0, :400], moved)
    fa.cache.cache_free(refs, table, lens, i32([0]), PAGE)
    assert fa.fa_check_device_error() == 0
    assert not refs.any() and (table == -1).all() and lens.item() == 0


@pytest.mark.parametrize("d,H,dt", [(64, 2, torch.bfloat16), (128, 12, torch.float16)])
@pytest.mark.parametrize("page,rows", [(8, 2**28 - 1), (PAGE, M)])
def test_decode(fa, d, H, dt, page, rows):
    """The newest of 2^31 - 8 tokens, with the 100 before it and three sinks; a length past the table's row counts as
    the row's."""
    g = torch.Generator().manual_seed(d + page)
    n, window, sinks = rows * page, 100, 3
    first = (n - window) // page                        # page entries from here on
    held = rows - first
    kp, vp = (torch.randn(held + 1, 1, page, d, generator=g).to(dt) for _ in range(2))
    q = torch.randn(1, H, d, generator=g).to(dt)
    table = torch.full((1, rows), -1, dtype=torch.int32, device="cuda")
    table[0, 0] = held
    table[0, first:] = torch.arange(held, dtype=torch.int32)
    flat = [torch.cat([x[held, 0, :sinks], x[:held].transpose(0, 1).reshape(-1, d)[-window:]]) for x in (kp, vp)]
    ref, ref_lse, weight, reach = paged64.decode(q, flat[0][None, None], flat[1][None, None], [[0]], [window + sinks], d ** -0.5)
    for length in (n, 2**31 - 1):
        o, lse = fa.cache.attention_decode(q.cuda(), kp.cuda(), vp.cuda(), table, i32([length]), window=window, sinks=sinks)
        assert fa.fa_check_device_error() == (0 if length == n else FA_ERR_PAGES)
        # the bounds of test_gpu_cache.py
        e = 2.0 ** -23 * (d + 8) * reach + 2.0 ** -22 * (4 + 2 * reach)
        tol = torch.finfo(dt).eps / 2 * np.abs(ref) + (2 * e[..., None] + 2.0 ** -15) * weight
        assert (np.abs(o.double().cpu().numpy() - ref) <= tol).all()
        assert (np.abs(lse.double().cpu().numpy() - ref_lse) <= e + 2.0 ** -23 * np.abs(ref_lse)).all()
