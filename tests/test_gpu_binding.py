"""The compiled way through the window and cache bindings: what it does beside the call itself."""
import os
import subprocess
import sys
import threading
import time

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from flashattention_bf16_fwd_b200 import cache, fa as binding, window
    binding.cache, binding.window = cache, window
    assert binding.fa_check_device_error() == 0
    return binding


def calls(fa):
    """One small call of each entry point; the cache's leave it as it is."""
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    rand = lambda *s: torch.randn(*s, device="cuda").bfloat16()
    q, k, v, do = (rand(1, 2, 100, 64) for _ in range(4))
    kp, vp, new = rand(1, 9, 2, 8, 64), rand(1, 9, 2, 8, 64), rand(2, 2, 64)
    refs, table, lens = i32([1, 1] + [0] * 7), i32([[0, 1], [-1, -1]]), i32([10, 0])
    zero, one = i32([0, 0]), i32([1])
    o, lse = fa.window.attention_window_fwd(q, k, v, 20, 2)
    return {
        "window_fwd": lambda: fa.window.attention_window_fwd(q, k, v, 20, 2),
        "window_bwd": lambda: fa.window.attention_window_bwd(q, k, v, o, lse, do, 20, 2),
        "decode": lambda: fa.cache.attention_decode(new, kp[0], vp[0], table, lens),
        "append": lambda: fa.cache.cache_append(new, new, kp[0], vp[0], table, lens),
        "reserve": lambda: fa.cache.cache_reserve(refs, table, lens, zero, 8),
        "fork": lambda: fa.cache.cache_fork(kp, vp, refs, table, lens, one, one),
        "free": lambda: fa.cache.cache_free(refs, table, lens, one, 8),
        "compact": lambda: fa.cache.cache_compact(kp, vp, refs, table, lens),
    }


@pytest.mark.parametrize("name", ["window_fwd", "window_bwd", "decode", "append", "reserve", "fork", "free", "compact"])
def test_other_threads_run_while_a_launch_waits(fa, name):
    """A stream that is busy for half a second or more and its queue of launches full: the call waits for room, and
    another Python thread goes on meanwhile."""
    call = calls(fa)[name]
    for _ in range(3):
        call()
    torch.cuda.synchronize()
    gaps, stop = [], threading.Event()

    def tick():
        last = time.perf_counter()
        while not stop.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gaps.append(now - last)
            last = now
    other = threading.Thread(target=tick)
    torch.cuda._sleep(1_500_000_000)                    # cycles of a clock of at most 2 GHz
    other.start()
    longest = 0.0
    for _ in range(2500):
        begin = time.perf_counter()
        call()
        longest = max(longest, time.perf_counter() - begin)
    stop.set()
    other.join()
    torch.cuda.synchronize()
    assert fa.fa_check_device_error() == 0
    assert longest > 0.3, "no launch waited"
    assert max(gaps) < longest / 2                      # a call that keeps the others out makes a gap as long as it waits


def test_two_threads_at_once(fa):
    """Steps of two Python threads, each with its own stream and tensors, are those of one after the other."""
    from test_gpu_window_dq import draw, same, spread
    jobs = []
    for seed, (H, Hkv, N, d, dt, window) in enumerate([(8, 4, 900, 64, "bf16", 200), (6, 2, 700, 128, "fp16", 333)]):
        x = draw(1, H, Hkv, N, d, dt, seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(x[0].dtype)
        q, k, v = rand(9, H, d), rand(9, Hkv, d), rand(9, Hkv, d)

        def job(x=x, q=q, k=k, v=v, window=window, Hkv=Hkv, d=d):
            """A training step, and a cache from its first token on."""
            o, lse = fa.window.attention_window_fwd(*x[:3], window, 4)
            out = [o, lse, *fa.window.attention_window_bwd(*x[:3], o, lse, x[3], window, 4)]
            kp, vp = (torch.zeros(2, 60, Hkv, 8, d, dtype=q.dtype, device="cuda") for _ in range(2))
            refs, lens = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (60, 9))
            table = torch.full((9, 6), -1, dtype=torch.int32, device="cuda")
            one = torch.ones(9, dtype=torch.int32, device="cuda")
            one[6:] = 0
            src, dst = torch.arange(3, device="cuda").int(), torch.arange(6, 9, device="cuda").int()
            for _ in range(11):
                out.append(fa.cache.cache_reserve(refs, table, lens, one, 8))
                fa.cache.cache_append(k, v, kp[1], vp[1], table, lens)
                out += fa.cache.attention_decode(q, kp[1], vp[1], table, lens, window=5, sinks=1)
            out.append(fa.cache.cache_fork(kp, vp, refs, table, lens, src, dst))
            fa.cache.cache_free(refs, table, lens, src, 8)
            out.append(fa.cache.cache_compact(kp, vp, refs, table, lens))
            return out + [kp, vp, refs, table, lens]
        jobs.append((job, spread(x, window, 4)))
    want = [job() for job, _ in jobs]
    torch.cuda.synchronize()
    got, failed, start = [None, None], [], threading.Barrier(2)

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait(60)
                got[i] = [jobs[i][0]() for _ in range(8)]
        except Exception as e:                          # reported by the test's own thread
            failed.append(e)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed and fa.fa_check_device_error() == 0
    for runs, w, (_, noise) in zip(got, want, jobs):
        for one in runs:
            same(one[2], w[2], noise)
            assert all(torch.equal(a, b) for i, (a, b) in enumerate(zip(one, w)) if i != 2)


FAILED_LAUNCH = """
import ctypes, sys, torch
from flashattention_bf16_fwd_b200 import cache, fa, window
from tests.test_gpu_binding import calls
fa.cache, fa.window = cache, window
rt = ctypes.CDLL(next(line.split()[-1] for line in open("/proc/self/maps") if "libcudart.so" in line))
tried = []
class Lib:
    def __getattr__(self, x):
        tried.append(x)
        return lambda *a: 0
real = cache.lib
for name, call in calls(fa).items():
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        for _ in range(2):                               # memory of this stream's own is at hand
            call()
        stream.synchronize()
        tried.clear()
        cache.lib = window.lib = Lib()
        handle, graph = ctypes.c_void_p(stream.cuda_stream), ctypes.c_void_p()
        assert rt.cudaStreamBeginCapture(handle, 2) == 0
        assert rt.cudaStreamSynchronize(handle) != 0     # breaks the capture off: launches into it are refused
        try:
            call()
            said = "nothing"
        except fa.FAError as e:
            said = e
        cache.lib = window.lib = real
        assert rt.cudaStreamEndCapture(handle, ctypes.byref(graph)) != 0
        rt.cudaGetLastError()
        print(name, "|", said, "|", tried)
        call()
        stream.synchronize()
"""


def test_a_failed_launch_is_said_and_not_tried_again(fa):
    """A call whose launch failed may have run in part: a second one could pass over what the first has left.  (A
    stream whose capture was broken off refuses launches; in a process of its own.)"""
    r = subprocess.run([sys.executable, "-c", FAILED_LAUNCH], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0, r.stderr
    names = {"window_fwd": "fa_window_fwd", "window_bwd": "fa_window_bwd", "decode": "fa_decode", "append": "fa_cache_append",
             "reserve": "fa_cache_reserve", "fork": "fa_cache_fork", "free": "fa_cache_free", "compact": "fa_cache_compact"}
    assert r.stdout.splitlines() == [f"{name} | {fa.FAError(call, -7)} | []" for name, call in names.items()]
