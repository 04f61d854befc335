"""The paged cache's C calls and binding refuse bad arguments on the host: no
GPU, no launch.  A valid call without an sm_100 device returns FA_ERR_DEVICE."""
import ctypes
import os
import re

import pytest
import torch

from flashattention_bf16_fwd_b200 import build as fa_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, HEADDIM, ALIGN, WORKSPACE, ARG, DEVICE, CSHAPE = 0, -1, -2, -3, -4, -6, -9, -10, -14
A, MIS16, MIS4 = 0x10000, 0x10008, 0x10002      # fake device addresses, never dereferenced


@pytest.fixture(scope="module")
def fa():
    fa_build.build()
    from flashattention_bf16_fwd_b200 import cache, fa as binding
    binding.cache = cache
    return binding


def test_header_and_binding_name_the_same_calls(fa):
    text = open(os.path.join(ROOT, "include", "fa_b200_cache.h")).read()
    declared = sorted(re.findall(r"FA_API\s+[\w\s\*]+?\b(fa_\w+)\s*\(", text))
    assert declared == sorted(fa.cache.EXPORTED)
    so = ctypes.CDLL(fa.LIB_PATH)
    for name in declared:
        assert hasattr(so, name), name
    for code in (-13, -14):
        assert fa.fa_status_string(code) not in ("", "unknown status")


def test_header_is_c(tmp_path):
    import shutil
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("needs a C compiler")
    src = tmp_path / "a.c"
    src.write_text('#include "fa_b200_cache.h"\nint main(void) { return FA_ERR_PAGES == -13 ? 0 : 1; }\n')
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I",
                        os.path.join(ROOT, "include"), "-c", str(src), "-o", str(tmp_path / "a.o")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def call(fa, name, defaults, **kw):
    assert set(kw) <= {n for n, _ in defaults}, kw
    return getattr(fa.lib, name)(*[kw.get(n, v) for n, v in defaults])


DECODE = [("q", A), ("k", A), ("v", A), ("table", A), ("lens", A), ("o", A), ("lse", A), ("ws", A), ("wsz", 1 << 30),
          ("S", 4), ("H", 8), ("Hkv", 2), ("d", 64), ("P", 100), ("page", 16), ("M", 50), ("q_stride", 512),
          ("window", 0), ("sinks", 0), ("scale", 0.125), ("elem", 0), ("stream", None)]
APPEND = [("k", A), ("v", A), ("kp", A), ("vp", A), ("table", A), ("lens", A), ("cu", A), ("T", 9), ("S", 4),
          ("Hkv", 2), ("d", 64), ("P", 100), ("page", 16), ("M", 50), ("ks", 128), ("vs", 128), ("stream", None)]
RESERVE = [("refs", A), ("table", A), ("lens", A), ("add", A), ("missing", A), ("S", 4), ("P", 100), ("page", 16),
           ("M", 50), ("stream", None)]
FORK = [("kp", A), ("vp", A), ("refs", A), ("table", A), ("lens", A), ("src", A), ("dst", A), ("missing", A),
        ("ws", A), ("wsz", 1 << 30), ("F", 2), ("L", 3), ("S", 4), ("Hkv", 2), ("d", 64), ("P", 100), ("page", 16),
        ("M", 50), ("stream", None)]
FREE = [("refs", A), ("table", A), ("lens", A), ("seqs", A), ("F", 2), ("S", 4), ("P", 100), ("page", 16), ("M", 50),
        ("stream", None)]
COMPACT = [("kp", A), ("vp", A), ("refs", A), ("table", A), ("lens", A), ("live", A), ("ws", A), ("wsz", 1 << 30),
           ("L", 3), ("S", 4), ("Hkv", 2), ("d", 64), ("P", 100), ("page", 16), ("M", 50), ("stream", None)]
ALL = {"fa_decode": DECODE, "fa_cache_append": APPEND, "fa_cache_reserve": RESERVE, "fa_cache_fork": FORK,
       "fa_cache_free": FREE, "fa_cache_compact": COMPACT}


@pytest.mark.parametrize("name", ALL)
def test_pointers(fa, name):
    for arg, default in ALL[name]:
        if default != A:
            continue
        got = call(fa, name, ALL[name], **{arg: None})
        if arg == "cu":
            assert got == CSHAPE          # 9 tokens for 4 sequences need their boundaries
        else:
            assert got == (WORKSPACE if arg == "ws" else NULL), arg
        wide = arg in ("q", "k", "v", "kp", "vp", "o", "refs", "ws")
        got = call(fa, name, ALL[name], **{arg: MIS16 if wide else MIS4})
        assert got == (WORKSPACE if arg == "ws" else ALIGN), arg


@pytest.mark.parametrize("name", ALL)
def test_sizes(fa, name):
    names = [n for n, _ in ALL[name]]
    bad = [("page", 0), ("page", 12), ("page", 4), ("page", 32776), ("page", -8), ("S", 0), ("S", 8193), ("P", 0),
           ("M", 0), ("M", 1 << 27), ("P", 1 << 30), ("F", 0), ("F", 5), ("L", 0), ("T", -1), ("M", (1 << 31) - 1)]
    for arg, value in bad:
        if arg in names and not (arg == "P" and value > 0 and "Hkv" not in names):
            assert call(fa, name, ALL[name], **{arg: value}) == CSHAPE, (arg, value)
    if "d" in names:
        assert call(fa, name, ALL[name], d=96) == HEADDIM
        assert call(fa, name, ALL[name], Hkv=0) == SHAPE
    if "wsz" in names:
        assert call(fa, name, ALL[name], wsz=16) == WORKSPACE


def test_decode_arguments(fa):
    dec = lambda **kw: call(fa, "fa_decode", DECODE, **kw)
    assert dec(H=9) == SHAPE
    assert dec(H=1) == SHAPE
    assert dec(S=1, M=1 << 26, H=128, Hkv=2, q_stride=128 * 64) == CSHAPE       # 2^31 tiles over one sequence's heads
    for kw in (dict(q_stride=504), dict(q_stride=516), dict(window=-1), dict(window=4, sinks=-1), dict(sinks=3)):
        assert dec(**kw) == CSHAPE, kw
    for kw in (dict(scale=0.0), dict(scale=float("nan")), dict(scale=-1.0), dict(elem=2), dict(elem=-1)):
        assert dec(**kw) == ARG, kw
    assert fa.cache.fa_decode_workspace_size(4, 8, 3, 64) == 0
    assert fa.cache.fa_decode_workspace_size(0, 8, 2, 64) == 0
    assert fa.cache.fa_decode_workspace_size(8193, 8, 2, 64) == 0
    need = fa.cache.fa_decode_workspace_size(4, 8, 2, 64)
    assert need > 0 and dec(wsz=need - 1) == WORKSPACE
    assert fa.cache.fa_cache_workspace_size(0, 5) == 0 and fa.cache.fa_cache_workspace_size(5, 0) == 0


def test_append_arguments(fa):
    app = lambda **kw: call(fa, "fa_cache_append", APPEND, **kw)
    for kw in (dict(ks=120), dict(vs=120), dict(ks=130), dict(vs=132), dict(ks=1 << 31)):
        assert app(**kw) == CSHAPE, kw


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU behaviour")
@pytest.mark.parametrize("name", ALL)
def test_valid_call_without_gpu_reports_device_error(fa, name):
    assert call(fa, name, ALL[name]) == DEVICE


def tensors(**kw):
    c = dict(q=torch.zeros(3, 4, 64, dtype=torch.bfloat16), k_pages=torch.zeros(7, 2, 16, 64, dtype=torch.bfloat16),
             v_pages=torch.zeros(7, 2, 16, 64, dtype=torch.bfloat16), table=torch.zeros(3, 5, dtype=torch.int32),
             lens=torch.zeros(3, dtype=torch.int32))
    c.update(kw)
    return c


def test_binding_refuses(fa):
    bf, i32 = torch.bfloat16, torch.int32
    for kw in (dict(q=torch.zeros(3, 4, 128, dtype=bf)), dict(q=torch.zeros(3, 3, 64, dtype=bf)),
               dict(q=torch.zeros(3, 4, 64)), dict(q=torch.zeros(4, 4, 64, dtype=bf)),
               dict(k_pages=torch.zeros(7, 2, 16, 64)), dict(v_pages=torch.zeros(6, 2, 16, 64, dtype=bf)),
               dict(k_pages=torch.zeros(7, 2, 64, 16, dtype=bf).transpose(2, 3)),
               dict(table=torch.zeros(3, 5, dtype=torch.int64)), dict(table=torch.zeros(5, 3, dtype=i32).T),
               dict(lens=torch.zeros(4, dtype=i32)), dict(q=torch.zeros(3, 64, 4, dtype=bf).transpose(1, 2))):
        with pytest.raises(ValueError):
            fa.cache.attention_decode(**tensors(**kw))
    with pytest.raises(ValueError, match="CUDA"):          # valid, but on the CPU
        fa.cache.attention_decode(**tensors())
    c = tensors()
    kv = torch.zeros(3, 2, 64, dtype=bf)
    with pytest.raises(ValueError):
        fa.cache.cache_append(kv[:2], kv[:2], c["k_pages"], c["v_pages"], c["table"], c["lens"])
    with pytest.raises(ValueError):
        fa.cache.cache_append(kv, kv.half(), c["k_pages"], c["v_pages"], c["table"], c["lens"])
    with pytest.raises(ValueError):
        fa.cache.cache_append(kv, kv, c["k_pages"], c["v_pages"], c["table"], c["lens"], torch.zeros(3, dtype=i32))
    refs, one = torch.zeros(7, dtype=i32), torch.zeros(3, dtype=i32)
    with pytest.raises(ValueError):
        fa.cache.cache_reserve(refs.long(), c["table"], c["lens"], one, 16)
    with pytest.raises(ValueError):
        fa.cache.cache_reserve(refs, c["table"], c["lens"], one[:2], 16)
    with pytest.raises(ValueError):
        fa.cache.cache_fork(c["k_pages"], c["v_pages"], refs[:5], c["table"], c["lens"], one[:1], one[:1])
    with pytest.raises(ValueError):
        fa.cache.cache_fork(c["k_pages"], c["v_pages"], refs, c["table"], c["lens"], one[:2], one[:1])
    with pytest.raises(ValueError):
        fa.cache.cache_free(refs, c["table"], c["lens"], one.float(), 16)
    with pytest.raises(ValueError):
        fa.cache.cache_compact(c["k_pages"], c["v_pages"].half(), refs, c["table"], c["lens"])
