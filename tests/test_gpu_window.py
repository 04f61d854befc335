"""Sliding-window attention with sinks on the GPU against the 64-bit oracle,
element by element, within the bounds that oracle/window64.py derives."""
import numpy as np
import pytest
import torch

from oracle import window64

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def fa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from flashattention_bf16_fwd_b200 import fa as binding, window
    binding.window = window
    assert binding.fa_check_device_error() == 0
    return binding


def draw(B, H, Hkv, N, d, dt, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(B, h, N, d, generator=g).to(DT[dt]) for h in (H, Hkv, Hkv, H)]


def within(got, want, tol, what):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), what
    over = np.abs(got - want) / np.maximum(tol, 1e-300)
    at = np.unravel_index(over.argmax(), over.shape)
    assert over.max() <= 1, f"{what}{list(map(int, at))}: {got[at]} for {want[at]}, {over.max():.3f} times the bound"


def check(fa, x, window, sinks, fix=1, scale=None, bwd=True):
    q, k, v, do = x
    eps = torch.finfo(q.dtype).eps
    scale_ = q.shape[-1] ** -0.5 if scale is None else scale
    dev = [t.cuda() for t in x]
    o, lse = fa.window.attention_window_fwd(*dev[:3], window, sinks, scale=scale, fix_mode=fix)
    assert fa.fa_check_device_error() == 0
    want, want_lse, tol, tol_lse = window64.forward(q, k, v, window, sinks, scale_, eps)
    within(o, want, tol, "o")
    within(lse, want_lse, tol_lse, "lse")
    if bwd:
        grads = fa.window.attention_window_bwd(*dev[:3], o, lse, dev[3], window, sinks, scale=scale)
        assert fa.fa_check_device_error() == 0
        want, tol = window64.backward(q, k, v, do, window, sinks, scale_, eps)
        for got, w, t, name in zip(grads, want, tol, ("dq", "dk", "dv")):
            within(got, w, t, name)
        return (o, lse) + grads
    return o, lse


CASES = [  # B, H, Hkv, N, d, window, sinks, type
    (1, 1, 1, 1, 64, 1, 0, "bf16"),
    (1, 2, 1, 1, 128, 5, 3, "fp16"),
    (2, 2, 2, 127, 64, 16, 4, "bf16"),
    (1, 2, 2, 128, 128, 128, 0, "bf16"),
    (1, 2, 1, 129, 64, 1, 0, "fp16"),
    (1, 3, 3, 257, 64, 1, 1, "bf16"),
    (1, 2, 2, 300, 128, 100, 0, "bf16"),
    (1, 2, 2, 512, 64, 128, 4, "bf16"),
    (1, 2, 2, 513, 128, 129, 4, "fp16"),
    (1, 4, 2, 640, 64, 130, 130, "bf16"),
    (2, 4, 1, 700, 128, 127, 5, "bf16"),
    (1, 2, 2, 777, 64, 257, 128, "fp16"),
    (1, 2, 1, 900, 64, 64, 300, "bf16"),
    (1, 2, 2, 640, 128, 5000, 0, "bf16"),
    (1, 1, 1, 640, 64, 640, 7, "fp16"),
    (1, 2, 2, 400, 64, 30, 5000, "bf16"),
    (1, 3, 1, 2100, 64, 200, 4, "bf16"),
    (1, 2, 1, 1900, 128, 90, 3, "fp16"),
    (1, 2, 2, 1500, 64, 2, 129, "bf16"),
    (1, 8, 1, 700, 64, 300, 4, "bf16"),          # windows and far parts cut, some parts empty
    (1, 4, 1, 2500, 128, 600, 140, "bf16"),
    (1, 5, 1, 1300, 64, 400, 0, "fp16"),
    (2, 8, 1, 100, 64, 30, 4, "bf16"),           # one query tile: dQ has one step, dK and dV are in parts
    (3, 6, 2, 128, 128, 200, 0, "fp16"),
    (1, 4, 4, 66, 128, 3, 2, "bf16"),
]


@pytest.mark.parametrize("B,H,Hkv,N,d,window,sinks,dt", CASES)
def test_window(fa, B, H, Hkv, N, d, window, sinks, dt):
    check(fa, draw(B, H, Hkv, N, d, dt, N + window), window, sinks)


@pytest.mark.parametrize("B,H,Hkv,N,d,window,sinks,dt", [
    (3, 2, 1, 1, 64, 7, 16, "bf16"), (2, 4, 2, 2, 128, 2, 1, "bf16"), (1, 3, 3, 3, 64, 8, 0, "fp16"), (4, 2, 2, 8, 64, 9, 0, "bf16"),
    (2, 6, 2, 300, 64, 1, 0, "bf16"), (1, 2, 2, 700, 128, 5, 3, "bf16"), (2, 2, 1, 400, 128, 2, 6, "fp16"), (1, 4, 1, 500, 64, 1, 9, "bf16")])
def test_gradients_of_rows_that_see_few_keys(fa, B, H, Hkv, N, d, window, sinks, dt):
    """Rows of up to 8 keys have a D without O's rounding; one that sees a key alone has no gradient but dv."""
    q, k, v, do = draw(B, H, Hkv, N, d, dt, N + d)
    dev = [t.cuda() for t in (q, k, v, do)]
    o, lse = fa.window.attention_window_fwd(*dev[:3], window, sinks)
    grads = fa.window.attention_window_bwd(*dev[:3], o, lse, dev[3], window, sinks)
    assert fa.fa_check_device_error() == 0
    want, tol = window64.backward(q, k, v, do, window, sinks, d ** -0.5, torch.finfo(DT[dt]).eps, few=8)
    for got, w, t, name in zip(grads, want, tol, ("dq", "dk", "dv")):
        within(got, w, t, name)


@pytest.mark.parametrize("fix", range(6))
@pytest.mark.parametrize("d,dt", [(64, "bf16"), (128, "fp16")])
def test_fix_modes_on_repeated_maxima(fa, fix, d, dt):
    """Every fix_mode on rows whose maximum is repeated: the sinks are copies of one long key, and keys repeat
    inside the window and across its border."""
    x = draw(1, 2, 2, 500, d, dt, fix)
    k = x[1]
    k[:, :, 1:3] = k[:, :, 0:1] = 4 * k[:, :, 0:1]
    k[:, :, 130::3] = k[:, :, 129:-1:3][:, :, :k[:, :, 130::3].shape[2]]
    check(fa, x, 140, 3, fix=fix, bwd=False)


@pytest.mark.parametrize("N,d,window,sinks,dt", [
    (129, 64, 1, 0, "bf16"), (256, 128, 100, 3, "fp16"), (257, 64, 128, 0, "bf16"), (383, 128, 130, 140, "bf16"), (640, 64, 129, 4, "fp16"),
    (777, 64, 191, 5, "bf16"), (900, 128, 257, 1, "fp16"), (1030, 64, 2000, 0, "bf16")])
def test_many_heads_are_as_few(fa, N, d, window, sinks, dt):
    """With more query tiles than CTAs two share one, or follow one another in it; the bits are those of a call with
    few heads, where each has its own."""
    q, k, v, _ = (t.cuda() for t in draw(2, 150, 75, N, d, dt, N))
    for fix in range(6):
        o, lse = fa.window.attention_window_fwd(q, k, v, window, sinks, fix_mode=fix)
        for b, h in ((0, 0), (0, 77), (1, 40), (1, 149)):
            few = fa.window.attention_window_fwd(q[b:b + 1, h:h + 1].contiguous(), k[b:b + 1, h // 2:h // 2 + 1].contiguous(),
                                                 v[b:b + 1, h // 2:h // 2 + 1].contiguous(), window, sinks, fix_mode=fix)
            assert torch.equal(o[b, h], few[0][0, 0]) and torch.equal(lse[b, h], few[1][0, 0]), (fix, b, h)
    assert fa.fa_check_device_error() == 0


@pytest.mark.parametrize("B,H,Hkv,N,d,window,sinks,dt", [
    (8, 12, 12, 900, 64, 200, 4, "bf16"), (6, 48, 24, 650, 128, 100, 140, "fp16"), (4, 64, 32, 1024, 64, 3, 260, "bf16")])
def test_backward_of_many_heads(fa, B, H, Hkv, N, d, window, sinks, dt):
    """Enough heads that the sinks' queries behind the window go with those in it: some heads against the oracle, and
    dk and dv the same bits again."""
    q, k, v, do = draw(B, H, Hkv, N, d, dt, N)
    dev = [t.cuda() for t in (q, k, v, do)]
    o, lse = fa.window.attention_window_fwd(*dev[:3], window, sinks)
    grads = fa.window.attention_window_bwd(*dev[:3], o, lse, dev[3], window, sinks)
    assert fa.fa_check_device_error() == 0
    again = fa.window.attention_window_bwd(*dev[:3], o, lse, dev[3], window, sinks)
    assert torch.equal(grads[1], again[1]) and torch.equal(grads[2], again[2])
    g, eps = H // Hkv, torch.finfo(DT[dt]).eps
    for b, x in ((0, 0), (B - 1, Hkv - 1), (B // 2, Hkv // 2)):
        hs = slice(x * g, x * g + g)
        want, tol = window64.backward(q[b:b + 1, hs], k[b:b + 1, x:x + 1], v[b:b + 1, x:x + 1], do[b:b + 1, hs], window, sinks,
                                      d ** -0.5, eps)
        for got, w, t, name in zip((grads[0][b:b + 1, hs], grads[1][b:b + 1, x:x + 1], grads[2][b:b + 1, x:x + 1]), want, tol,
                                   ("dq", "dk", "dv")):
            within(got, w, t, name)


def test_window_as_wide_as_the_sequence_is_causal_attention(fa):
    """The same tiles in the same order: the bits are those of attention_fwd in the modes that share its softmax."""
    for d, N in ((64, 900), (128, 777)):
        x = [t.cuda() for t in draw(1, 4, 2, N, d, "bf16", 3)]
        for fix in (0, 2, 3, 4, 5):
            o, lse = fa.window.attention_window_fwd(*x[:3], N, 0, fix_mode=fix)
            o2, lse2 = fa.attention_fwd(*x[:3], causal=True, fix_mode=fix)
            assert torch.equal(o, o2) and torch.equal(lse, lse2), fix


@pytest.mark.parametrize("d,dt", [(64, "bf16"), (128, "bf16"), (64, "fp16"), (128, "fp16")])
def test_rising_and_falling_scores(fa, d, dt):
    """Scores that rise by more than the shift's headroom from tile to tile, or fall by thousands: every key tile
    moves the shift, or none after the first does and P underflows."""
    for sign in (1, -1):
        x = draw(1, 2, 2, 900, d, dt, 12)
        x[0][..., 0] = 16
        x[1][..., 0] = torch.linspace(-20, 20, 900) * sign
        check(fa, x, 500, 130, scale=0.5, bwd=False)


def test_many_items_and_repeats(fa):
    """More items than CTAs, so that the pipelines run on across items: sampled heads against the oracle, and
    the same bits on every repeat (dQ, whose order of sums varies, within a rounding of the type)."""
    for d, dt in ((64, "bf16"), (128, "fp16")):
        B, H, Hkv, N, window, sinks = 4, 12, 6, 1111, 150, 4
        x = draw(B, H, Hkv, N, d, dt, 5)
        dev = [t.cuda() for t in x]
        first = None
        for _ in range(5):
            o, lse = fa.window.attention_window_fwd(*dev[:3], window, sinks)
            grads = fa.window.attention_window_bwd(*dev[:3], o, lse, dev[3], window, sinks)
            assert fa.fa_check_device_error() == 0
            if first is None:
                first = (o, lse) + grads
            for i, (a, b) in enumerate(zip((o, lse) + grads, first)):
                if i != 2:
                    assert torch.equal(a, b), i
        eps = torch.finfo(DT[dt]).eps
        for b, g in ((0, 0), (3, 5)):
            s = [x[0][b:b + 1, 2 * g:2 * g + 2], x[1][b:b + 1, g:g + 1], x[2][b:b + 1, g:g + 1], x[3][b:b + 1, 2 * g:2 * g + 2]]
            want, want_lse, tol, tol_lse = window64.forward(*s[:3], window, sinks, d ** -0.5, eps)
            within(first[0][b:b + 1, 2 * g:2 * g + 2], want, tol, "o")
            within(first[1][b:b + 1, 2 * g:2 * g + 2], want_lse, tol_lse, "lse")
            want, tol = window64.backward(*s, window, sinks, d ** -0.5, eps)
            within(first[2][b:b + 1, 2 * g:2 * g + 2], want[0], tol[0], "dq")
            within(first[3][b:b + 1, g:g + 1], want[1], tol[1], "dk")
            within(first[4][b:b + 1, g:g + 1], want[2], tol[2], "dv")


def test_gradients_against_differences(fa):
    """The kernel's gradients along random directions against differences of the 64-bit forward."""
    B, H, Hkv, N, d, window, sinks = 1, 4, 2, 400, 64, 70, 3
    x = draw(B, H, Hkv, N, d, "fp16", 8)
    grads = check(fa, x, window, sinks)[2:]
    _, tol = window64.backward(*x, window, sinks, d ** -0.5, torch.finfo(torch.float16).eps)
    r = np.random.default_rng(2)
    y, do = [t.double().numpy() for t in x[:3]], x[3].double().numpy()
    for n in range(3):
        u, step = r.standard_normal(y[n].shape), 1e-4
        f = [float((do * window64.forward(*[z + t * u if i == n else z for i, z in enumerate(y)], window, sinks, d ** -0.5,
                                          2.0 ** -10)[0]).sum()) for t in (step, -step)]
        got = float((grads[n].double().cpu().numpy() * u).sum())
        # the difference itself is off by step^2 times a third derivative of order sum |do| (about 1e5 values)
        assert abs(got - (f[0] - f[1]) / (2 * step)) <= float((tol[n] * np.abs(u)).sum()) + 1e-3


def test_large_scores_and_a_first_tile_that_a_row_does_not_see(fa):
    """Scores down to some hundreds below zero: rows whose first key tiles are hidden start from nothing, not
    from a shift of 0."""
    x = draw(1, 2, 2, 600, 64, "bf16", 4)
    x[0].abs_()
    x[1].abs_().neg_()
    check(fa, [x[0] * 4, x[1] * 4, x[2], x[3]], 129, 0, scale=1.0, bwd=False)


def test_other_stream_and_own_workspace(fa):
    x = draw(1, 4, 2, 700, 64, "bf16", 6)
    dev = [t.cuda() for t in x]
    o, lse = fa.window.attention_window_fwd(*dev[:3], 100, 4)
    want = fa.window.attention_window_bwd(*dev[:3], o, lse, dev[3], 100, 4)
    ws = torch.full((fa.window.fa_window_bwd_workspace_size(1, 4, 2, 700, 64, 100, 4),), 255, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    o2, lse2 = fa.window.attention_window_fwd(*dev[:3], 100, 4, stream=stream)
    got = fa.window.attention_window_bwd(*dev[:3], o2, lse2, dev[3], 100, 4, stream=stream.cuda_stream, workspace=ws)
    torch.cuda.synchronize()
    assert fa.fa_check_device_error() == 0
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])


def test_training_step_in_a_graph(fa):
    """Forward and backward captured and replayed on new inputs."""
    x = [t.cuda() for t in draw(1, 2, 1, 500, 64, "bf16", 1)]
    step = lambda: (lambda o, lse: (o, lse) + fa.window.attention_window_bwd(*x[:3], o, lse, x[3], 90, 4))(
        *fa.window.attention_window_fwd(*x[:3], 90, 4))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (2, 3):
        for t, new in zip(x, draw(1, 2, 1, 500, 64, "bf16", seed)):
            t.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        assert fa.fa_check_device_error() == 0
        cpu = [t.cpu() for t in x]
        want, want_lse, tol, tol_lse = window64.forward(*cpu[:3], 90, 4, 0.125, 2.0 ** -7)
        within(out[0], want, tol, "o")
        want, tol = window64.backward(*cpu, 90, 4, 0.125, 2.0 ** -7)
        for got, w, t, name in zip(out[2:], want, tol, ("dq", "dk", "dv")):
            within(got, w, t, name)


def test_prefill_then_decoding_behind_the_same_window(fa):
    """A prompt through the windowed forward, then tokens one by one from the cache: every position's output is
    the windowed attention's."""
    from flashattention_bf16_fwd_b200 import cache
    H, Hkv, N, d, window, sinks, page, prompt = 4, 2, 300, 64, 70, 4, 16, 270
    q, k, v, _ = draw(1, H, Hkv, N, d, "bf16", 9)
    want, want_lse, tol, tol_lse = window64.forward(q, k, v, window, sinks, d ** -0.5, 2.0 ** -7)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    qd, kd, vd = (t[0].transpose(0, 1).contiguous().cuda() for t in (q, k, v))       # [N, heads, d]
    o, _ = fa.window.attention_window_fwd(*(t[:, :, :prompt].contiguous().cuda() for t in (q, k, v)), window, sinks)
    within(o, want[:, :, :prompt], tol[:, :, :prompt], "prompt")
    kp, vp = (torch.full((40, Hkv, page, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    refs, lens = torch.zeros(40, dtype=torch.int32, device="cuda"), i32([0])
    table = torch.full((1, 20), -1, dtype=torch.int32, device="cuda")
    cache.cache_reserve(refs, table, lens, i32([prompt]), page)
    cache.cache_append(kd[:prompt], vd[:prompt], kp, vp, table, lens, i32([0, prompt]))
    for i in range(prompt, N):
        cache.cache_reserve(refs, table, lens, i32([1]), page)
        cache.cache_append(kd[i:i + 1], vd[i:i + 1], kp, vp, table, lens)
        o, lse = cache.attention_decode(qd[i:i + 1], kp, vp, table, lens, window=window, sinks=sinks)
        within(o[0], want[0, :, i], tol[0, :, i], i)
        within(lse[0], want_lse[0, :, i], tol_lse[0, :, i], i)
    assert fa.fa_check_device_error() == 0


def test_two_streams_at_once(fa):
    """Training steps and decoding on two streams at the same time, each with its own tensors: as one after the other."""
    from flashattention_bf16_fwd_b200 import cache
    jobs = []
    for seed, (H, Hkv, N, d, dt, win) in enumerate([(8, 4, 1500, 64, "bf16", 200), (6, 2, 1300, 128, "fp16", 333)]):
        x = [t.cuda() for t in draw(2, H, Hkv, N, d, dt, seed)]
        S, page = 40, 16
        kp, vp = (torch.randn(400, Hkv, page, d, device="cuda").to(DT[dt]) for _ in range(2))
        table = torch.randint(0, 400, (S, 20), dtype=torch.int32, device="cuda")
        lens = torch.randint(0, 320, (S,), dtype=torch.int32, device="cuda")
        qd = torch.randn(S, H, d, device="cuda").to(DT[dt])

        def job(x=x, win=win, qd=qd, kp=kp, vp=vp, table=table, lens=lens):
            o, lse = fa.window.attention_window_fwd(*x[:3], win, 4)
            grads = fa.window.attention_window_bwd(*x[:3], o, lse, x[3], win, 4)
            return (o, lse, *grads[1:], *cache.attention_decode(qd, kp, vp, table, lens))
        jobs.append(job)
    want = [job() for job in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(10):
        got = []
        for job, stream in zip(jobs, streams):
            with torch.cuda.stream(stream):
                got.append([job() for _ in range(3)])
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            for one in g:
                assert all(torch.equal(a, b) for a, b in zip(one, w))
    assert fa.fa_check_device_error() == 0
