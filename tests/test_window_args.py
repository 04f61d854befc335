"""The windowed attention's C calls and binding refuse bad arguments on the
host; its 64-bit oracle agrees with the causal one and with differences."""
import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

from flashattention_bf16_fwd_b200 import build as fa_build
from oracle import attention_bwd, attention_fwd, window64

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NULL, SHAPE, HEADDIM, ALIGN, FIXMODE, WORKSPACE, ARG, DEVICE, WINDOW = -1, -2, -3, -4, -5, -6, -9, -10, -15
A, MIS = 0x10000, 0x10008


@pytest.fixture(scope="module")
def win():
    fa_build.build()
    from flashattention_bf16_fwd_b200 import window
    return window


def test_header_and_binding_name_the_same_calls(win, tmp_path):
    text = open(os.path.join(ROOT, "include", "fa_b200_window.h")).read()
    declared = sorted(re.findall(r"FA_API\s+[\w\s\*]+?\b(fa_\w+)\s*\(", text))
    assert declared == sorted(win.EXPORTED)
    from flashattention_bf16_fwd_b200 import fa
    so = ctypes.CDLL(fa.LIB_PATH)
    for name in declared:
        assert hasattr(so, name), name
    assert fa.fa_status_string(WINDOW) not in ("", "unknown status")
    if shutil.which("gcc"):
        src = tmp_path / "a.c"
        src.write_text('#include "fa_b200_window.h"\nint main(void) { return FA_ERR_WINDOW == -15 ? 0 : 1; }\n')
        r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I",
                            os.path.join(ROOT, "include"), "-c", str(src), "-o", str(tmp_path / "a.o")],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr


FWD = [("q", A), ("k", A), ("v", A), ("o", A), ("lse", A), ("B", 1), ("H", 4), ("Hkv", 2), ("N", 300), ("d", 64),
       ("window", 64), ("sinks", 4), ("scale", 0.125), ("fix", 1), ("elem", 0), ("stream", None)]
BWD = [("q", A), ("k", A), ("v", A), ("o", A), ("lse", A), ("do", A), ("dq", A), ("dk", A), ("dv", A), ("ws", A),
       ("wsz", 1 << 30), ("B", 1), ("H", 4), ("Hkv", 2), ("N", 300), ("d", 64), ("window", 64), ("sinks", 4),
       ("scale", 0.125), ("elem", 0), ("stream", None)]


def call(win, name, defaults, **kw):
    assert set(kw) <= {n for n, _ in defaults}
    return getattr(win.lib, name)(*[kw.get(n, v) for n, v in defaults])


@pytest.mark.parametrize("name,args", [("fa_window_fwd", FWD), ("fa_window_bwd", BWD)])
def test_arguments(win, name, args):
    for arg, default in args:
        if default == A:
            assert call(win, name, args, **{arg: None}) == (WORKSPACE if arg == "ws" else NULL), arg
            if arg != "lse":
                assert call(win, name, args, **{arg: MIS}) == (WORKSPACE if arg == "ws" else ALIGN), arg
    for kw, want in ((dict(d=96), HEADDIM), (dict(N=0), SHAPE), (dict(Hkv=3), SHAPE), (dict(Hkv=8), SHAPE),
                     (dict(H=1 << 18, Hkv=1 << 18, N=1 << 7), SHAPE), (dict(window=0), WINDOW), (dict(window=-5), WINDOW),
                     (dict(sinks=-1), WINDOW), (dict(scale=0.0), ARG), (dict(scale=float("inf")), ARG),
                     (dict(elem=2), ARG)):
        assert call(win, name, args, **kw) == want, kw
    if name == "fa_window_fwd":
        assert call(win, name, args, fix=6) == FIXMODE
        assert call(win, name, args, fix=-1) == FIXMODE
    else:
        need = win.fa_window_bwd_workspace_size(1, 4, 2, 300, 64, 64, 4)
        assert need > 0 and call(win, name, args, wsz=need - 1) == WORKSPACE
    if not torch.cuda.is_available():
        assert call(win, name, args) == DEVICE


def test_workspace_size(win):
    size = win.fa_window_bwd_workspace_size
    up = lambda x: -(-x // 256) * 256
    rows = 8 * 12 * 1024
    base = up(rows * 64 * 4) + up(rows * 4)
    assert size(8, 12, 12, 1024, 64, 256, 0) == base
    assert size(8, 12, 12, 1024, 64, 5000, 4) == base          # no query is past the window
    # 8 query tiles, 3 in a window, 5 behind it, the same item; with half the heads a part beside the window's
    assert size(8, 12, 12, 1024, 64, 256, 4) == base
    assert size(4, 12, 12, 1024, 64, 256, 4) == base // 2 + up(48 * 2 * 4 * 2 * 64 * 4)
    # 16 query tiles, 2 in a window, 14 behind it in four parts
    assert size(8, 12, 12, 2048, 64, 128, 4) == 2 * base + up(96 * 5 * 4 * 2 * 64 * 4)
    # one head: its tiles of 3, 2 and 1 steps in parts of two steps, the least length
    assert size(1, 1, 1, 300, 64, 256, 0) == up(300 * 64 * 4) + up(300 * 4) + up(2 * 300 * 2 * 64 * 4)
    assert size(1, 1, 1, 256, 64, 256, 0) == up(256 * 64 * 4) + up(256 * 4)
    # four heads over one: 12 steps a tile, in six parts of all rows
    assert size(1, 4, 1, 300, 64, 256, 0) == up(1200 * 64 * 4) + up(1200 * 4) + up(6 * 300 * 2 * 64 * 4)
    assert size(2, 4, 2, 1000, 64, 0, 4) == 0
    assert size(2, 4, 3, 1000, 64, 64, 4) == 0
    assert size(1, 1, 1, 1 << 20, 64, 10**12, 10**12) == size(1, 1, 1, 1 << 20, 64, 1 << 20, 1 << 20)


def test_binding_refuses(win):
    q = torch.zeros(1, 4, 128, 64, dtype=torch.bfloat16)
    lse = torch.zeros(1, 4, 128)
    for k, v in ((q[:, :3], q[:, :3]), (q.half(), q), (q.transpose(2, 3).contiguous().transpose(2, 3), q)):
        with pytest.raises(ValueError):
            win.attention_window_fwd(q, k, v, 16)
    with pytest.raises(ValueError):
        win.attention_window_fwd(q.float(), q.float(), q.float(), 16)
    with pytest.raises(ValueError):
        win.attention_window_bwd(q, q, q, q, lse.half(), q, 16)
    with pytest.raises(ValueError):
        win.attention_window_bwd(q, q, q, q[:, :2], lse, q, 16)
    with pytest.raises(ValueError, match="CUDA"):
        win.attention_window_fwd(q, q, q, 16)


def inputs(B, H, Hkv, N, d, seed=0):
    r = np.random.default_rng(seed)
    return [r.standard_normal((B, h, N, d)) for h in (H, Hkv, Hkv, H)]


def test_oracle_is_causal_attention_where_the_window_is_wide():
    q, k, v, do = inputs(1, 2, 2, 40, 8)
    o, lse, _, _ = window64.forward(q, k, v, 40, 0, 0.3, 2.0 ** -8)
    want, want_lse = attention_fwd(q, k, v, True, 0.3)
    assert np.allclose(o, want, atol=1e-12) and np.allclose(lse, want_lse, atol=1e-12)
    got, _ = window64.backward(q, k, v, do, 40, 0, 0.3, 2.0 ** -8)
    for a, b in zip(got, attention_bwd(q, k, v, do, True, 0.3)):
        assert np.allclose(a, b, atol=1e-12)


def test_oracle_mask_by_hand():
    want = ["10000", "11000", "11100", "10110", "10011"]
    assert [[int(c) for c in row] for row in want] == window64.visible(5, 2, 1).astype(int).tolist()


@pytest.mark.parametrize("window,sinks", [(1, 0), (5, 2), (3, 9), (30, 0)])
def test_oracle_gradients_against_differences(window, sinks):
    q, k, v, do = x = inputs(1, 4, 2, 23, 8, seed=window)
    grads, _ = window64.backward(*x, window, sinks, 0.4, 2.0 ** -8)
    r = np.random.default_rng(1)
    for n in range(3):
        u, step = r.standard_normal(x[n].shape), 1e-5
        f = [float((do * window64.forward(*[y + t * u if i == n else y for i, y in enumerate(x[:3])], window, sinks, 0.4,
                                          2.0 ** -8)[0]).sum()) for t in (step, -step)]
        assert abs((f[0] - f[1]) / (2 * step) - float((grads[n] * u).sum())) < 1e-6
