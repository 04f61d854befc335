"""dQ of the windowed backward from call to call.  dQ is the one output that several CTAs add up in an order that
varies, in an accumulator that an earlier launch clears, so that repeats, old contents of a workspace and calls that
run at the same time could show in it and nowhere else.

Two calls add the same FP32 terms, a key tile each, in two orders: either sum of T terms is off by at most T 2^-24
times the sum of their sizes, and is then rounded to the element type by half a step, eps / 2 |dQ| (in fp16 2^-25 at
least).  So two results differ by at most
    eps / 2 (|a| + |b|) + 2^-24 (fp16) + 2 T 2^-24 size,   size = scale sum_j |dS_ij| |K_j|
and |dS| = P |dP - D| <= P (|dO||V| + sum |dO||O|), 2 % more for the roundings of P, dP and O.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def fa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from flashattention_bf16_fwd_b200 import cache, fa as binding, window
    binding.cache, binding.window = cache, window
    assert binding.fa_check_device_error() == 0
    return binding


def draw(B, H, Hkv, N, d, dt, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(B, h, N, d, generator=g).to(DT[dt]).cuda() for h in (H, Hkv, Hkv, H)]


def spread(x, window, sinks):
    """2 T 2^-24 size of every element, in 64 bits, head by head."""
    q, k, v, do = x
    B, H, N, d = q.shape
    g, scale = H // k.shape[1], d ** -0.5
    i = torch.arange(N, device="cuda")
    hidden = (i[None, :] > i[:, None]) | ((i[:, None] - i[None, :] >= window) & (i[None, :] >= sinks))
    out = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    for b in range(B):
        for h in range(H):
            qq, kk, vv, dd = (t.double() for t in (q[b, h], k[b, h // g], v[b, h // g], do[b, h]))
            p = torch.softmax((scale * qq @ kk.T).masked_fill(hidden, float("-inf")), 1)
            ds = p * (dd.abs() @ vv.abs().T + (dd * (p @ vv)).abs().sum(1, keepdim=True))
            out[b, h] = 1.02 * scale * ds @ kk.abs()
    return out * (2 * -(-N // 128) * 2.0 ** -24)


def same(a, b, noise):
    eps = torch.finfo(a.dtype).eps
    tol = eps / 2 * (a.double().abs() + b.double().abs()) + noise + (2.0 ** -24 if a.dtype is torch.float16 else 0.0)
    over = (a.double() - b.double()).abs() - tol
    assert torch.isfinite(a).all() and (over <= 0).all(), over.max().item()


SHAPES = [(4, 12, 6, 1111, 64, 150, 4, "bf16"), (4, 12, 6, 1111, 128, 150, 4, "fp16"), (8, 12, 12, 900, 64, 200, 4, "bf16"),
          (1, 8, 1, 700, 64, 300, 4, "bf16"), (2, 8, 1, 100, 64, 30, 4, "bf16"), (4, 64, 32, 1024, 64, 3, 260, "bf16")]


@pytest.mark.parametrize("B,H,Hkv,N,d,window,sinks,dt", SHAPES)
def test_repeats(fa, B, H, Hkv, N, d, window, sinks, dt):
    x = draw(B, H, Hkv, N, d, dt, N + d)
    noise = spread(x, window, sinks)
    o, lse = fa.window.attention_window_fwd(*x[:3], window, sinks)
    first = fa.window.attention_window_bwd(*x[:3], o, lse, x[3], window, sinks)
    for _ in range(5):
        again = fa.window.attention_window_bwd(*x[:3], o, lse, x[3], window, sinks)
        same(again[0], first[0], noise)
        assert torch.equal(again[1], first[1]) and torch.equal(again[2], first[2])
    assert fa.fa_check_device_error() == 0


@pytest.mark.parametrize("B,H,Hkv,N,d,window,sinks,dt", SHAPES)
def test_a_workspace_with_old_contents(fa, B, H, Hkv, N, d, window, sinks, dt):
    """NaN everywhere, then what another call's inputs have left."""
    x, y = draw(B, H, Hkv, N, d, dt, 1), draw(B, H, Hkv, N, d, dt, 2)
    noise = spread(x, window, sinks)
    o, lse = fa.window.attention_window_fwd(*x[:3], window, sinks)
    want = fa.window.attention_window_bwd(*x[:3], o, lse, x[3], window, sinks)
    other = fa.window.attention_window_fwd(*y[:3], window, sinks)
    ws = torch.full((fa.window.fa_window_bwd_workspace_size(B, H, Hkv, N, d, window, sinks),), 255, dtype=torch.uint8,
                    device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    for on in (None, stream):
        if on is None:
            torch.cuda.synchronize()
        got = fa.window.attention_window_bwd(*x[:3], o, lse, x[3], window, sinks, stream=on, workspace=ws)
        fa.window.attention_window_bwd(*y[:3], *other, y[3], window, sinks, stream=on, workspace=ws)
        again = fa.window.attention_window_bwd(*x[:3], o, lse, x[3], window, sinks, stream=on, workspace=ws)
        torch.cuda.synchronize()
        for g in (got, again):
            same(g[0], want[0], noise)
            assert torch.equal(g[1], want[1]) and torch.equal(g[2], want[2])
    assert fa.fa_check_device_error() == 0


def test_two_streams_at_once(fa):
    jobs = []
    for seed, (H, Hkv, N, d, dt, window) in enumerate([(8, 4, 1500, 64, "bf16", 200), (6, 2, 1300, 128, "fp16", 333)]):
        x = draw(2, H, Hkv, N, d, dt, seed)

        def job(x=x, window=window):
            o, lse = fa.window.attention_window_fwd(*x[:3], window, 4)
            return (o, lse) + fa.window.attention_window_bwd(*x[:3], o, lse, x[3], window, 4)
        jobs.append((job, spread(x, window, 4)))
    want = [job() for job, _ in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(10):
        got = []
        for (job, _), stream in zip(jobs, streams):
            with torch.cuda.stream(stream):
                got.append([job() for _ in range(3)])
        torch.cuda.synchronize()
        for runs, w, (_, noise) in zip(got, want, jobs):
            for one in runs:
                same(one[2], w[2], noise)
                assert all(torch.equal(a, b) for i, (a, b) in enumerate(zip(one, w)) if i != 2)
    assert fa.fa_check_device_error() == 0


@pytest.mark.parametrize("B,H,Hkv,N,d,window,sinks,dt", SHAPES)
def test_both_ways_through_the_binding(fa, monkeypatch, B, H, Hkv, N, d, window, sinks, dt):
    x = draw(B, H, Hkv, N, d, dt, 5)
    o, lse = fa.window.attention_window_fwd(*x[:3], window, sinks)
    fast = fa.window.attention_window_bwd(*x[:3], o, lse, x[3], window, sinks)

    class Never:
        window_bwd = staticmethod(lambda *a: None)
    monkeypatch.setattr(fa.window, "_fast", Never())
    other = fa.window.attention_window_bwd(*x[:3], o, lse, x[3], window, sinks)
    same(other[0], fast[0], spread(x, window, sinks))
    assert torch.equal(other[1], fast[1]) and torch.equal(other[2], fast[2])
    assert fa.fa_check_device_error() == 0


def test_graph_replays_in_one_workspace(fa):
    """A backward captured with a workspace that an eager call uses between the replays."""
    B, H, Hkv, N, d, window, sinks, dt = SHAPES[2]
    x, y = draw(B, H, Hkv, N, d, dt, 1), draw(B, H, Hkv, N, d, dt, 2)
    noise = spread(x, window, sinks)
    o, lse = fa.window.attention_window_fwd(*x[:3], window, sinks)
    other = fa.window.attention_window_fwd(*y[:3], window, sinks)
    ws = torch.empty(fa.window.fa_window_bwd_workspace_size(B, H, Hkv, N, d, window, sinks), dtype=torch.uint8, device="cuda")
    want = fa.window.attention_window_bwd(*x[:3], o, lse, x[3], window, sinks, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fa.window.attention_window_bwd(*x[:3], o, lse, x[3], window, sinks, workspace=ws)
    for _ in range(3):
        fa.window.attention_window_bwd(*y[:3], *other, y[3], window, sinks, workspace=ws)
        graph.replay()
        same(got[0], want[0], noise)
        assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    assert fa.fa_check_device_error() == 0
