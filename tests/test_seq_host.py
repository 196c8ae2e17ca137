"""CPU-only checks of the language-model operators' C entry points and of their binding: argument
validation, sizes of workspaces, struct layouts.  Every call here is refused, or empty, before
anything is launched: its pointers are numbers that nothing reads."""
import ctypes
import os
import shutil
import subprocess

import pytest

import linear_attention_diffusion_litela_b200 as ll
from linear_attention_diffusion_litela_b200 import seq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED = 1, 2
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from linear_attention_diffusion_litela_b200.build import build
    build()
    return ll.lib()


def refused(lib, status, code, words):
    assert status == code
    assert words in lib.lite_la_last_error().decode(), lib.lite_la_last_error()


# ---------------------------------------------------------------------------------------
# head norms with rotation

NORM = dict(qkv=1 * MB, out=2 * MB, wq=3 * MB, wk=3 * MB + 512, cos=4 * MB, sin=5 * MB, pos=6 * MB, pos_bytes=8, B=2, N=3,
            Hq=4, Hk=2, Hv=2, d=64, rot=32, table=100, inter=0, eps=1e-6)


def norm_fwd(lib, **change):
    a = dict(NORM, **change)
    return lib.lite_la_qk_norm_rope_fwd(*(a[n] for n in NORM), None)


def norm_bwd(lib, dout=7 * MB, dwq=8 * MB, dwk=8 * MB + 512, ws=9 * MB, ws_bytes=MB, **change):
    a = dict(NORM, **change)
    rest = [a[n] for n in ("cos", "sin", "pos", "pos_bytes", "B", "N", "Hq", "Hk", "Hv", "d", "rot", "table", "inter", "eps")]
    return lib.lite_la_qk_norm_rope_bwd(a["qkv"], dout, a["out"], a["wq"], a["wk"], dwq, dwk, *rest, ws, ws_bytes, None)


@pytest.mark.parametrize("code,words,change", [
    (INVALID, "must be >= 0", dict(B=-1)), (INVALID, "must be >= 0", dict(N=-1)), (INVALID, "must be >= 0", dict(Hq=-2)),
    (INVALID, "must be >= 0", dict(Hk=-1)), (INVALID, "must be >= 0", dict(Hv=-1)),
    (INVALID, "65535", dict(B=65536)), (INVALID, "65535", dict(Hq=65536)), (INVALID, "2^30", dict(N=(1 << 30) + 1)),
    (UNSUPPORTED, "d must be", dict(d=16, rot=16)), (UNSUPPORTED, "d must be", dict(d=256)),
    (UNSUPPORTED, "rot must be", dict(rot=8)), (UNSUPPORTED, "rot must be", dict(rot=80)),
    (UNSUPPORTED, "rot must be", dict(rot=-16)),
    (INVALID, "eps", dict(eps=float("nan"))), (INVALID, "eps", dict(eps=-1.0)), (INVALID, "eps", dict(eps=float("inf"))),
    (INVALID, "at least one position", dict(table=0)), (INVALID, "position_bytes", dict(pos_bytes=2)),
    (INVALID, "shorter than N", dict(pos=0, table=2)),
    (INVALID, "null buffer", dict(qkv=0)), (INVALID, "null buffer", dict(out=0)),
    (INVALID, "null cos or sin", dict(cos=0)), (INVALID, "null cos or sin", dict(sin=0)),
    (INVALID, "16-byte aligned", dict(qkv=MB + 8)), (INVALID, "16-byte aligned", dict(out=2 * MB + 2)),
    (INVALID, "16-byte aligned", dict(cos=4 * MB + 4)), (INVALID, "aligned to their elements", dict(wq=3 * MB + 2)),
    (INVALID, "aligned to their elements", dict(pos=6 * MB + 4)),
    (INVALID, "overlaps qkv", dict(out=MB + 16)),
    (INVALID, "overlaps a weight", dict(out=3 * MB)), (INVALID, "overlaps a weight", dict(out=4 * MB)),
    (INVALID, "overlaps a weight", dict(out=6 * MB)),
])
def test_norm_refusals(lib, code, words, change):
    refused(lib, norm_fwd(lib, **change), code, words)
    refused(lib, norm_bwd(lib, **change), code, words)


@pytest.mark.parametrize("words,change", [
    ("null buffer", dict(dout=0)), ("16-byte aligned", dict(dout=7 * MB + 2)),
    ("overlaps qkv or dout", dict(dout=2 * MB + 16)),
    ("overlaps qkv or dout", dict(out=MB)),                 # dqkv may be dout, not qkv
    ("4-byte aligned", dict(dwq=8 * MB + 1)), ("workspace missing", dict(ws=0)),
    ("workspace missing", dict(ws_bytes=1000)), ("workspace missing", dict(ws=9 * MB + 4)),
    ("workspace overlaps an output", dict(ws=2 * MB)), ("workspace overlaps an output", dict(ws=8 * MB)),
    ("workspace overlaps an input", dict(ws=MB)), ("workspace overlaps an input", dict(ws=7 * MB)),
    ("outputs overlap", dict(dwk=8 * MB)), ("outputs overlap", dict(dwq=2 * MB)),
    ("overlaps an input", dict(dwq=MB)), ("overlaps an input", dict(dwk=3 * MB)),
])
def test_norm_gradient_refusals(lib, words, change):
    refused(lib, norm_bwd(lib, **change), INVALID, words)


def test_norm_empty_calls(lib):
    for change in (dict(B=0), dict(N=0), dict(Hq=0, Hk=0, Hv=0)):
        assert norm_fwd(lib, qkv=0, out=0, **change) == 0
    assert [lib.lite_la_qk_norm_rope_workspace_bytes(d) > 0 for d in (16, 32, 64, 128, 256)] == [0, 1, 1, 1, 0]


# ---------------------------------------------------------------------------------------
# the gated delta rule

VIEWS = ("q", "k", "v", "out")
DELTA = dict(q=(1 * MB, 0, 256, 64), k=(2 * MB, 0, 256, 64), v=(3 * MB, 0, 512, 64), out=(4 * MB, 0, 512, 64), g=5 * MB,
             beta=6 * MB, g_sb=0, g_st=8, b_sb=0, b_st=8, si=7 * MB, so=8 * MB, cu=0, B=1, N=200, Hk=4, Hv=8, d=64,
             scale=0.125, zero_tail=0, ws=16 * MB, ws_bytes=16 * MB)
SAVED = 64 * MB
GRADS = dict(dout=(9 * MB, 0, 512, 64), dq=(10 * MB, 0, 256, 64), dk=(11 * MB, 0, 256, 64), dv=(12 * MB, 0, 512, 64),
             dg=13 * MB, dbeta=13 * MB + 65536, dso=14 * MB, dsi=15 * MB)


def delta(**change):
    a = dict(DELTA, **change)
    return seq._DELTA_ARGS.pack(*(x for n in VIEWS for x in a[n]), *(a[n] for n in DELTA if n not in VIEWS))


def grads(**change):
    a = dict(GRADS, **change)
    return seq._DELTA_GRADS.pack(*(x for n in ("dout", "dq", "dk", "dv") for x in a[n]),
                                 *(a[n] for n in ("dg", "dbeta", "dso", "dsi")))


def test_struct_layouts(tmp_path):
    """What the binding packs is what the header declares."""
    cxx = shutil.which("g++") or shutil.which("c++")
    cuda = "/usr/local/cuda/include"
    if cxx is None or not os.path.exists(os.path.join(cuda, "cuda_runtime_api.h")):
        pytest.skip("no C++ compiler or CUDA headers")
    fields = {"lite_la_delta_args": [(8 * 4 * 4, "g"), (128 + 16, "g_batch_stride"), (176, "state_in"), (192, "cu_seqlens"),
                                     (200, "B"), (220, "scale"), (224, "zero_tail"), (232, "workspace")],
              "lite_la_delta_grads": [(0, "dout"), (32, "dq"), (128, "dg"), (144, "dstate_out"), (152, "dstate_in")]}
    size = {"lite_la_delta_args": seq._DELTA_ARGS.size, "lite_la_delta_grads": seq._DELTA_GRADS.size}
    text = '#include <cstddef>\n#include "litela.h"\n'
    for name, fs in fields.items():
        text += 'static_assert(sizeof(%s) == %d, "size");\n' % (name, size[name])
        for off, f in fs:
            text += 'static_assert(offsetof(%s, %s) == %d, "%s");\n' % (name, f, off, f)
    src = tmp_path / "layout.cpp"
    src.write_text(text)
    subprocess.run([cxx, "-fsyntax-only", "-I" + os.path.join(ROOT, "include"), "-I" + cuda, str(src)], check=True)


BAD_DELTA = [
    (INVALID, "must be >= 0", dict(B=-1)), (INVALID, "must be >= 0", dict(N=-1)), (INVALID, "must be >= 0", dict(Hk=-4)),
    (INVALID, "must be >= 0", dict(Hv=-8)), (INVALID, "65535", dict(B=65536)), (INVALID, "65535", dict(Hv=65536)),
    (INVALID, "2^30", dict(N=(1 << 30) + 1)),
    (UNSUPPORTED, "d must be", dict(d=48)), (UNSUPPORTED, "d must be", dict(d=256)), (UNSUPPORTED, "d must be", dict(d=0)),
    (UNSUPPORTED, "multiple of Hk", dict(Hk=3)), (UNSUPPORTED, "multiple of Hk", dict(Hk=0)),
    (UNSUPPORTED, "multiple of Hk", dict(Hk=16)),
    (INVALID, "scale", dict(scale=float("inf"))), (INVALID, "scale", dict(scale=float("nan"))),
    (INVALID, "too many sequences", dict(B=65535, Hv=65535, Hk=1)),
    (INVALID, "null q, k, v", dict(q=(0, 0, 256, 64))), (INVALID, "null q, k, v", dict(k=(0, 0, 256, 64))),
    (INVALID, "null q, k, v", dict(v=(0, 0, 512, 64))),
    (INVALID, "views must be 16-byte", dict(q=(MB + 2, 0, 256, 64))), (INVALID, "multiples of 8", dict(k=(2 * MB, 0, 260, 64))),
    (INVALID, "multiples of 8", dict(v=(3 * MB, 0, -512, 64))), (INVALID, "multiples of 8", dict(v=(3 * MB, 0, 512, 63))),
    (INVALID, "extent overflows", dict(q=(MB, 0, 1 << 62, 64))),
    (INVALID, "null g or beta", dict(g=0)), (INVALID, "null g or beta", dict(beta=0)),
    (INVALID, "g and beta must be 4-byte", dict(g=5 * MB + 2)), (INVALID, "strides of g", dict(g_st=-8)),
    (INVALID, "strides of g", dict(b_sb=-1)), (INVALID, "gate's extent", dict(g_st=1 << 61)),
    (INVALID, "gate's extent", dict(b_st=1 << 61)),
    (INVALID, "states must be 16-byte", dict(si=7 * MB + 4)), (INVALID, "cu_seqlens must be 4-byte", dict(cu=20 * MB + 2)),
    (INVALID, "packed tokens need a sequence", dict(cu=20 * MB, B=0)),
]
BAD_FORWARD = [
    (INVALID, "null q, k, v, out", dict(out=(0, 0, 512, 64))),
    (INVALID, "output view overlaps itself", dict(out=(4 * MB, 0, 256, 64))),
    (INVALID, "output view overlaps itself", dict(out=(4 * MB, 0, 0, 64))),
    (INVALID, "output view overlaps itself", dict(out=(4 * MB, 0, 512, 32))),
    (INVALID, "out overlaps an input", dict(out=(3 * MB, 0, 512, 64))),
    (INVALID, "out overlaps an input", dict(out=(5 * MB, 0, 512, 64))),
    (INVALID, "a state overlaps out", dict(si=4 * MB)), (INVALID, "a state overlaps out", dict(so=4 * MB + 16)),
    (INVALID, "state_out overlaps an input", dict(so=2 * MB)), (INVALID, "state_out overlaps state_in", dict(so=7 * MB + 16)),
]


@pytest.mark.parametrize("code,words,change", BAD_DELTA)
def test_delta_refusals(lib, code, words, change):
    args = delta(**change)
    refused(lib, lib.lite_la_gated_delta_fwd(args, None), code, words)
    refused(lib, lib.lite_la_gated_delta_fwd_save(args, SAVED, 64 * MB, None), code, words)
    refused(lib, lib.lite_la_gated_delta_bwd(args, grads(), SAVED, 64 * MB, None), code, words)


@pytest.mark.parametrize("code,words,change", BAD_FORWARD)
def test_delta_forward_refusals(lib, code, words, change):
    refused(lib, lib.lite_la_gated_delta_fwd(delta(**change), None), code, words)
    refused(lib, lib.lite_la_gated_delta_fwd_save(delta(**change), SAVED, 64 * MB, None), code, words)


@pytest.mark.parametrize("words,change", [
    ("workspace missing", dict(ws=0)), ("workspace missing", dict(ws_bytes=100)), ("workspace missing", dict(ws=16 * MB + 8)),
    ("overlaps a buffer", dict(ws=4 * MB)), ("overlaps a buffer", dict(ws=MB)), ("overlaps a buffer", dict(ws=8 * MB)),
    ("overlaps a buffer", dict(ws=7 * MB)),
])
def test_delta_workspace_refusals(lib, words, change):
    refused(lib, lib.lite_la_gated_delta_fwd(delta(**change), None), INVALID, words)


@pytest.mark.parametrize("words,saved,size", [
    ("saved missing", 0, 64 * MB), ("saved missing", SAVED, 1000), ("saved missing", SAVED + 8, 64 * MB),
    ("saved overlaps", 3 * MB, 64 * MB), ("saved overlaps", 7 * MB, 64 * MB),
])
def test_delta_saved_refusals(lib, words, saved, size):
    refused(lib, lib.lite_la_gated_delta_fwd_save(delta(), saved, size, None), INVALID, words)
    refused(lib, lib.lite_la_gated_delta_bwd(delta(), grads(), saved, size, None), INVALID, words)


@pytest.mark.parametrize("words,change,args", [
    ("null q, k, v, out or gradient", dict(dout=(0, 0, 512, 64)), {}),
    ("null q, k, v, out or gradient", dict(dq=(0, 0, 256, 64)), {}),
    ("output view overlaps itself", dict(dk=(11 * MB, 0, 64, 64)), {}), ("multiples of 8", dict(dv=(12 * MB, 0, 516, 64)), {}),
    ("null dg or dbeta", dict(dg=0), {}), ("null dg or dbeta", dict(dbeta=0), {}),
    ("dg and dbeta must be 4-byte", dict(dg=13 * MB + 2), {}),
    ("the states' gradients must be", dict(dso=14 * MB + 4), {}), ("the states' gradients must be", dict(dsi=15 * MB + 4), {}),
    ("workspace missing", {}, dict(ws=0)), ("workspace missing", {}, dict(ws_bytes=100)),
    ("workspace overlaps", {}, dict(ws=2 * MB)),
    ("different memory", dict(dq=(11 * MB, 0, 256, 64)), {}), ("different memory", dict(dv=(10 * MB, 0, 512, 64)), {}),
    ("output overlaps an input", dict(dq=(9 * MB, 0, 256, 64)), {}), ("output overlaps an input", dict(dv=(3 * MB, 0, 512, 64)), {}),
    ("output overlaps an input", dict(dg=14 * MB), {}), ("output overlaps an input", dict(dsi=3 * MB), {}),
    ("output overlaps an input", dict(dk=(64 * MB, 0, 256, 64)), {}),
    ("outputs overlap", dict(dg=12 * MB), {}), ("outputs overlap", dict(dbeta=13 * MB), {}),
    ("outputs overlap", {}, dict(ws=10 * MB)), ("dstate_in overlaps dstate_out in part", dict(dsi=14 * MB + 16), {}),
])
def test_delta_gradient_refusals(lib, words, change, args):
    refused(lib, lib.lite_la_gated_delta_bwd(delta(**args), grads(**change), SAVED, 64 * MB, None), INVALID, words)


def test_delta_gradient_needs_its_struct(lib):
    refused(lib, lib.lite_la_gated_delta_bwd(delta(), None, SAVED, 64 * MB, None), INVALID, "null grads")
    refused(lib, lib.lite_la_gated_delta_bwd(None, grads(), SAVED, 64 * MB, None), INVALID, "null args")
    refused(lib, lib.lite_la_gated_delta_fwd(None, None), INVALID, "null args")


STEP = dict(B=4, N=1, q=(1 * MB, 256, 0, 64), k=(2 * MB, 256, 0, 64), v=(3 * MB, 512, 0, 64), out=(4 * MB, 512, 0, 64), g_sb=8,
            b_sb=8, g_st=0, b_st=0, si=8 * MB, so=8 * MB)


@pytest.mark.parametrize("words,change,slots,pool", [
    ("pool must be >= 0", {}, 0, -1), ("takes no cu_seqlens", dict(cu=20 * MB), 0, 4), ("output view overlaps itself", dict(N=2), 0, 4),
    ("needs N = 1", dict(N=2, out=(4 * MB, 1024, 512, 64)), 0, 4),
    ("needs N = 1", dict(N=0), 0, 4), ("same pool", dict(so=7 * MB), 0, 4), ("same pool", dict(si=0, so=0), 0, 4),
    ("same pool", dict(so=0), 0, 4), ("fewer states", {}, 0, 3), ("fewer states", dict(si=0, so=0), 0, 0),
    ("state_indices must be 4-byte", {}, 20 * MB + 2, 4), ("out overlaps an input", {}, 4 * MB, 4),
    ("a state overlaps out", dict(si=4 * MB, so=4 * MB), 0, 4), ("state_out overlaps an input", dict(si=3 * MB, so=3 * MB), 0, 4),
    ("state_out overlaps an input", {}, 8 * MB + 64, 4), ("must be >= 0", dict(B=-1), 0, 4),
    ("null g or beta", dict(beta=0), 0, 4),
])
def test_step_refusals(lib, words, change, slots, pool):
    refused(lib, lib.lite_la_gated_delta_step(delta(**dict(STEP, **change)), slots or None, pool, None), INVALID, words)


def test_delta_empty_calls(lib):
    for change in (dict(B=0), dict(Hk=0, Hv=0), dict(B=0, N=0, cu=20 * MB)):
        assert lib.lite_la_gated_delta_fwd(delta(**change), None) == 0
        assert lib.lite_la_gated_delta_fwd_save(delta(**change), None, 0, None) == 0
        assert lib.lite_la_gated_delta_bwd(delta(**change), grads(), None, 0, None) == 0
    assert lib.lite_la_gated_delta_step(delta(**dict(STEP, B=0)), None, 4, None) == 0


def test_delta_workspace_sizes(lib):
    """Nothing for the recurrence, and as many chunks as the lengths can need at most for the rest."""
    size, saved, back = (lib.lite_la_gated_delta_workspace_bytes, lib.lite_la_gated_delta_saved_bytes,
                         lib.lite_la_gated_delta_bwd_workspace_bytes)
    assert size(8, 1, 4, 8, 64, 0) == 0 and size(1, 32, 4, 8, 64, 0) == 0
    one = size(1, 64, 1, 1, 64, 0)
    assert one > 0
    assert size(1, 65, 1, 1, 64, 0) >= 2 * one - 512 and size(3, 64, 2, 4, 64, 0) <= 12 * one
    # 3 sequences in 130 tokens: 2 whole chunks and 3 started ones
    assert 5 * one - 1024 <= size(3, 130, 1, 1, 64, 1) <= 5 * one
    for f in (size, saved, back):
        assert all(f(*bad) == 0 for bad in ((-1, 64, 1, 1, 64, 0), (1, -64, 1, 1, 64, 0), (1, 64, 1, 1, 48, 0),
                                            (1, 64, 0, 0, 64, 0), (0, 64, 1, 1, 64, 1)))
        assert f(1, 1 << 20, 64, 64, 128, 0) > 1 << 32     # no 32-bit sizes
    assert saved(1, 64, 1, 1, 64, 0) >= 66 * 1024 + 4 * 64 * 64 + 256 * 64


# ---------------------------------------------------------------------------------------
# the binding's own checks: CPU tensors, wrong types and shapes are refused before the library is called

def test_binding_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    q = torch.zeros(1, 5, 2, 64, dtype=torch.bfloat16)
    g = torch.zeros(1, 5, 2)
    for call in (lambda: ll.lite_la_qk_norm_rope_fwd(q.view(1, 5, 128), 1, 1, d=64),
                 lambda: ll.lite_la_qk_norm_rope(q.view(1, 5, 128), 1, 1, d=64),
                 lambda: ll.lite_la_gated_delta_fwd(q, q, q, g, g),
                 lambda: ll.lite_la_gated_delta(q, q, q, g, g),
                 lambda: ll.lite_la_gated_delta_fwd_save(q, q, q, g, g),
                 lambda: ll.lite_la_gated_delta_bwd(q, q, q, g, g, q, None),
                 lambda: ll.lite_la_gated_delta_step(q[:, 0], q[:, 0], q[:, 0], g[:, 0], g[:, 0], torch.zeros(1, 2, 64, 64))):
        with pytest.raises(TypeError):
            call()


def test_struct_arguments_are_bytes(lib):
    assert lib.lite_la_gated_delta_fwd.argtypes[0] in (ctypes.c_char_p, ctypes.c_void_p)
