"""The largest sizes that the window and cache calls accept: sequences of millions of tokens, 8192 sequences, pages of
32768 tokens, 256 query heads over one.  Some rows of each against 64 bits; the bounds are those of
oracle/window64.py and of tests/test_gpu_cache.py."""
import numpy as np
import pytest
import torch

from oracle import paged64, window64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from flashattention_bf16_fwd_b200 import cache, fa as binding, window
    binding.cache, binding.window = cache, window
    assert binding.fa_check_device_error() == 0
    return binding


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def within(got, want, tol, what):
    over = np.abs(got.double().cpu().numpy() - want) / np.maximum(tol, 1e-300)
    assert over.max() <= 1, (what, over.max())


@pytest.mark.parametrize("H,Hkv,N,d,dt", [(4, 2, 8388607, 64, torch.bfloat16), (1, 1, 16777215, 128, torch.float16)])
def test_window_over_millions_of_tokens(fa, H, Hkv, N, d, dt):
    """Pieces of 500 tokens at the end, in the middle and at the start, against the attention of each piece alone: its
    rows from the 100th on see nothing before it, and its keys up to the 100th from its end nothing after it does."""
    window, n = 100, 500
    g = torch.Generator(device="cuda").manual_seed(1)
    q, do = (torch.randn(1, H, N, d, generator=g, device="cuda", dtype=dt) for _ in range(2))
    k, v = (torch.randn(1, Hkv, N, d, generator=g, device="cuda", dtype=dt) for _ in range(2))
    o, lse = fa.window.attention_window_fwd(q, k, v, window)
    dq, dk, dv = fa.window.attention_window_bwd(q, k, v, o, lse, do, window)
    assert fa.fa_check_device_error() == 0
    for at in (N - n, N // 2 + 77, 0):
        x = [t[:, :, at:at + n].cpu() for t in (q, k, v, do)]
        first = 0 if at == 0 else window                # rows that see no token before `at`
        last = n if at + n == N else n - window         # keys that no query after the piece sees
        eps = torch.finfo(dt).eps
        want, want_lse, tol, tol_lse = window64.forward(*x[:3], window, 0, d ** -0.5, eps)
        within(o[:, :, at + first:at + n], want[:, :, first:], tol[:, :, first:], ("o", at))
        within(lse[:, :, at + first:at + n], want_lse[:, :, first:], tol_lse[:, :, first:], ("lse", at))
        # rows before `first` see other keys than in the piece: they count for nothing in what is compared
        want, tol = window64.backward(*x, window, 0, d ** -0.5, eps)
        within(dq[:, :, at + first:at + n], want[0][:, :, first:], tol[0][:, :, first:], ("dq", at))
        for got, i, name in ((dk, 1, "dk"), (dv, 2, "dv")):
            within(got[:, :, at + first:at + last], want[i][:, :, first:last], tol[i][:, :, first:last], (name, at))


def check_decode(o, lse, q, kp, vp, table, lens, seqs, window=0, sinks=0):
    """Sequences `seqs` of a batch."""
    d = q.shape[-1]
    q, table, lens = q[seqs], table[seqs], lens[seqs]
    ref, ref_lse, weight, reach = paged64.decode(q, kp, vp, table.tolist(), lens.tolist(), d ** -0.5, window, sinks)
    e = 2.0 ** -23 * (d + 8) * reach + 2.0 ** -22 * (4 + 2 * reach)
    full = lens.numpy() > 0
    within(o[seqs][torch.from_numpy(full)], ref[full], (torch.finfo(q.dtype).eps / 2 * np.abs(ref) + (2 * e[..., None] + 2.0 ** -15) * weight)[full], "o")
    within(lse[seqs][torch.from_numpy(full)], ref_lse[full], (e + 2.0 ** -23 * np.abs(ref_lse))[full], "lse")
    assert (o[seqs][torch.from_numpy(~full)] == 0).all() and (lse[seqs][torch.from_numpy(~full)] == -np.inf).all()


@pytest.mark.parametrize("H,Hkv,d,window,sinks", [(2, 1, 64, 0, 0), (34, 2, 128, 20, 3)])
def test_8192_sequences(fa, H, Hkv, d, window, sinks):
    """Prompts, forks, decoding, and all of it ended again."""
    S, page, M, P = 8192, 8, 12, 40000
    g = torch.Generator().manual_seed(H)
    refs, lens, table = i32([0] * P), i32([0] * S), torch.full((S, M), -1, dtype=torch.int32, device="cuda")
    add = torch.randint(0, 70, (S,), generator=g, dtype=torch.int32)
    add[S // 2:] = 0
    kp, vp = (torch.randn(P, Hkv, page, d, generator=g).bfloat16().cuda() for _ in range(2))
    assert fa.cache.cache_reserve(refs, table, lens, add.cuda(), page).item() == 0
    src, dst = torch.randperm(S // 2, generator=g).int().cuda(), torch.arange(S // 2, S).int().cuda()
    assert fa.cache.cache_fork(kp, vp, refs, table, lens, src, dst).item() == 0
    held = -(-lens // page)
    assert lens.tolist() == add[:S // 2].tolist() + add[src.cpu().long()].tolist()
    assert refs.sum().item() == held.sum().item() == (table >= 0).sum().item()
    q = torch.randn(S, H, d, generator=g).bfloat16()
    o, lse = fa.cache.attention_decode(q.cuda(), kp, vp, table, lens, window=window, sinks=sinks)
    assert fa.fa_check_device_error() == 0
    seqs = torch.cat([torch.arange(6), torch.randint(0, S, (60,), generator=g), torch.arange(S - 6, S)])
    check_decode(o.cpu(), lse.cpu(), q, kp.cpu(), vp.cpu(), table.cpu(), lens.cpu(), seqs, window, sinks)
    fa.cache.cache_free(refs, table, lens, torch.arange(S - 1, -1, -1).int().cuda(), page)
    assert fa.fa_check_device_error() == 0
    assert not refs.any() and not lens.any() and (table == -1).all()


@pytest.mark.parametrize("H,Hkv,d,page,lens", [(256, 1, 64, 16, [300, 1]), (256, 1, 128, 16, [77, 0, 200]), (96, 2, 128, 64, [500]),
                                               (4, 2, 64, 32768, [40000, 1, 32768]), (3, 1, 128, 32760, [33000])])
def test_many_heads_and_large_pages(fa, H, Hkv, d, page, lens):
    g = torch.Generator().manual_seed(page)
    held = [-(-n // page) for n in lens]
    table, at = torch.full((len(lens), max(held) + 1), -1, dtype=torch.int32), 0
    for s, n in enumerate(held):
        table[s, :n] = torch.arange(at, at + n)
        at += n
    kp, vp = (torch.randn(at, Hkv, page, d, generator=g).half() for _ in range(2))
    q, n = torch.randn(len(lens), H, d, generator=g).half(), torch.tensor(lens, dtype=torch.int32)
    o, lse = fa.cache.attention_decode(*(t.cuda() for t in (q, kp, vp, table, n)))
    assert fa.fa_check_device_error() == 0
    check_decode(o.cpu(), lse.cpu(), q, kp, vp, table, n, torch.arange(len(lens)))
