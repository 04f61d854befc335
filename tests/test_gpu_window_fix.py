"""The windowed forward's fix_mode 1 keeps every exponential below 1: a row's shift is the maximum + delta + headroom
when the maximum + delta passes the shift in use, and stays until then.  What that does to O is small (other
roundings of P_bar), but not to be missed: the mode is followed step by step in 64 bits, with its roundings, and the
kernel's O has to agree with it, and not with the same steps without delta.

Scores are small whole numbers, exact in FP32, so that the followed P is the kernel's but for ex2's error, 2^-20 at
most with the rest of the arithmetic's.  A P that lies that close to the border between two values of the element
format may be rounded to either: a step times |V|.  FP32 sums of up to some hundred terms add less than 2^-18 of
their size, and O is rounded by half a step."""
import numpy as np
import pytest
import torch

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
DELTA = {"bf16": -np.log2(1 - 2.0 ** -8), "fp16": -np.log2(1 - 2.0 ** -11)}
HEADROOM = {"bf16": 8.0, "fp16": 4.0}
CASES = [(100, 64, 40, 3, "bf16"), (128, 128, 128, 0, "bf16"), (300, 128, 90, 4, "bf16"), (700, 64, 200, 130, "bf16"),
         (100, 128, 40, 3, "fp16"), (300, 64, 90, 4, "fp16"), (700, 128, 200, 130, "fp16")]
SCALE = 0.25


def draw(N, d, dt, seed):
    """q and k in whole numbers, the keys longer from tile to tile, so that maxima repeat and shifts move."""
    g = torch.Generator().manual_seed(seed)
    q, k = (torch.randint(-1, 2, (1, 1, N, d), generator=g).float() for _ in range(2))
    k[:, :, 128:] *= 2
    k[:, :, 384:] *= 2
    return q.to(DT[dt]), k.to(DT[dt]), torch.randn(1, 1, N, d, generator=g).to(DT[dt])


def f32(x):
    return np.asarray(x, dtype=np.float32).astype(np.float64)


def follow(q, k, v, window, sinks, dt, delta):
    """O before its rounding, and what the kernel's may be off by."""
    q, k, v = (t[0, 0].double().numpy() for t in (q, k, v))
    N = len(q)
    s = q @ k.T
    i, j = np.arange(N)[:, None], np.arange(N)[None, :]
    s = np.where((j <= i) & ((i - j < window) | (j < sinks)), s, -np.inf)
    sl2, delta = f32(SCALE * 1.4426950408889634), f32(delta)
    bits, least = (8, -126) if dt == "bf16" else (11, -14)
    ms, l = np.full((N, 1), -np.inf), np.zeros((N, 1))
    o, off, size = np.zeros(v.shape), np.zeros(v.shape), np.zeros(v.shape)
    for t in range(0, N, 128):
        x, vv = s[:, t:t + 128], v[t:t + 128]
        top = f32(x.max(1, keepdims=True) * sl2 + delta)
        moved = top > ms
        shift = np.where(moved, f32(top + HEADROOM[dt]), ms)
        with np.errstate(invalid="ignore"):
            alpha = np.where(moved, np.exp2(ms - shift), 1.0)
            p = np.where(x > -np.inf, np.exp2(f32(x * sl2 - shift)), 0.0)
        ulp = np.exp2(np.maximum(np.floor(np.log2(np.maximum(p, 1e-300))), least) - (bits - 1))
        border = np.abs(p / ulp - np.floor(p / ulp) - 0.5) * ulp <= 2.0 ** -20 * p
        rounded = np.rint(p / ulp) * ulp
        assert (rounded < 1).all() or delta == 0
        o = o * alpha + rounded @ vv
        l = l * alpha + p.sum(1, keepdims=True)
        off = off * alpha + (border * ulp) @ np.abs(vv)
        size = size * alpha + p @ np.abs(vv)
        ms = shift
    o, off, size = o / l, off / l, size / l
    half = torch.finfo(DT[dt]).eps / 2
    off = off + 2.0 ** -18 * size
    return o, off + np.maximum(half * (np.abs(o) + off), 0.0 if dt == "bf16" else 2.0 ** -25)


@pytest.mark.parametrize("N,d,window,sinks,dt", CASES)
def test_the_steps_tell_a_missing_delta(N, d, window, sinks, dt):
    """On the CPU: with and without delta differ by more than both bounds in many places."""
    x = draw(N, d, dt, N + d)
    o, tol = follow(*x, window, sinks, dt, DELTA[dt])
    plain, tol_plain = follow(*x, window, sinks, dt, 0.0)
    assert (np.abs(o - plain) > tol + tol_plain).sum() > 20


@pytest.mark.gpu
@pytest.mark.parametrize("N,d,window,sinks,dt", CASES)
def test_shift_above_the_maximum(N, d, window, sinks, dt):
    from flashattention_bf16_fwd_b200 import fa, window as win
    x = draw(N, d, dt, N + d)
    o, _ = win.attention_window_fwd(*(t.cuda() for t in x), window, sinks, scale=SCALE)
    assert fa.fa_check_device_error() == 0
    got = o[0, 0].double().cpu().numpy()
    want, tol = follow(*x, window, sinks, dt, DELTA[dt])
    over = np.abs(got - want) / tol
    assert over.max() <= 1, over.max()
    plain, tol_plain = follow(*x, window, sinks, dt, 0.0)
    assert (np.abs(got - plain) > tol_plain).sum() > 20
