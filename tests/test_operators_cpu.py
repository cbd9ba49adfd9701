"""Refusals of the operators between the adapted linears, checked without a
device: the C entry points before any launch, and the binding's own checks."""
import ctypes

import pytest
import torch

BF16 = torch.bfloat16
P = ctypes.c_void_p
BIG = 1 << 20


@pytest.fixture(scope="module")
def am():
    from adapter_merge_b200 import build
    build.build()
    import adapter_merge_b200
    adapter_merge_b200.lib()
    return adapter_merge_b200


def at(i, off=0):
    """A made-up, 1 MiB spaced device address (nothing is read before a launch)."""
    return (i + 1) * BIG * 64 + off


def project(am, **kw):
    a = dict(x=at(0), T=4, K=64, ldx=64, W=at(1), N=32, ldw=64, bias=None, res=None, ldr=0, y=at(2), ldy=32, flags=0)
    a.update(kw)
    return am.lib().adafuse_project(a["x"], a["T"], a["K"], a["ldx"], a["W"], a["N"], a["ldw"], a["bias"], a["res"],
                                    a["ldr"], a["y"], a["ldy"], a["flags"], None, None)


def gated(am, **kw):
    a = dict(x=at(0), T=4, K=64, ldx=64, W=at(1), U=at(3), N=32, ldw=64, bg=None, bu=None, y=at(2), ldy=32, flags=2)
    a.update(kw)
    return am.lib().adafuse_gated_project(a["x"], a["T"], a["K"], a["ldx"], a["W"], a["U"], a["N"], a["ldw"], a["bg"],
                                          a["bu"], a["y"], a["ldy"], a["flags"], None, None)


@pytest.mark.parametrize("kw", [
    {"x": None}, {"W": None}, {"y": None}, {"T": -1}, {"K": 0}, {"N": 0}, {"K": -8}, {"flags": 1 << 9},
    {"flags": 1 << 5}, {"ldx": 56}, {"ldw": 56}, {"ldy": 24}, {"y": at(0)}, {"y": at(1)}, {"y": at(0, 128)},
])
def test_projections_refuse_bad_arguments(am, kw):
    assert project(am, **kw) == am.ERR_INVALID_ARG
    assert gated(am, **kw) == am.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    {"K": 60, "ldx": 60, "ldw": 60}, {"N": 36, "ldy": 36}, {"x": at(0, 8)}, {"W": at(1, 2)}, {"y": at(2, 8)},
    {"ldx": 68}, {"ldw": 70}, {"ldy": 36}, {"flags": 5}, {"flags": 7}, {"T": 1 << 31},
    {"ldx": 1 << 38}, {"ldw": 1 << 40}, {"ldy": 1 << 60}, {"N": (1 << 31) - 8, "ldy": 1 << 32},
    {"K": (1 << 31) - 8, "ldx": 1 << 32, "ldw": 1 << 32},
])
def test_projections_refuse_what_they_do_not_support(am, kw):
    assert project(am, **kw) == am.ERR_UNSUPPORTED
    assert gated(am, **kw) == am.ERR_UNSUPPORTED


def test_projections_refuse_overlaps_and_options(am):
    bad = am.ERR_INVALID_ARG
    assert gated(am, U=None) == bad and gated(am, U=at(2)) == bad and gated(am, flags=2 | am.OUT_F32) == bad
    assert gated(am, bg=at(2)) == bad and gated(am, bu=at(2, 64)) == bad and project(am, bias=at(2)) == bad
    assert project(am, bias=at(4, 2)) == am.ERR_UNSUPPORTED
    # a residual overlaps y unless it is y itself: another offset or stride, or fp32 results
    assert project(am, res=at(2, 16), ldr=32) == bad
    assert project(am, res=at(2), ldr=40) == bad
    assert project(am, res=at(2), ldr=32, flags=am.OUT_F32) == bad
    assert project(am, res=at(2), ldr=0) == bad
    assert project(am, res=at(3), ldr=24) == bad
    # x as its own residual and result
    assert project(am, N=64, ldy=64, y=at(0), res=at(0), ldr=64) == bad
    # columns of one buffer that cross
    assert project(am, x=at(5), ldx=128, y=at(5, 112), ldy=128) == bad
    assert project(am, T=0, x=None, W=None, y=None) == am.OK
    assert gated(am, T=0, x=None, W=None, y=None) == am.OK


def epilogue(am, **kw):
    a = dict(y=at(0), T=4, n=24, ldy=24, bias=None, up=None, ldu=0, res=None, ldr=0, out=at(1), ldo=24, flags=0)
    a.update(kw)
    return am.lib().adafuse_epilogue(a["y"], a["T"], a["n"], a["ldy"], a["bias"], a["up"], a["ldu"], a["res"], a["ldr"],
                                     a["out"], a["ldo"], a["flags"], None)


def test_epilogue_refusals(am):
    bad = am.ERR_INVALID_ARG
    for kw in ({"y": None}, {"out": None}, {"T": -1}, {"n": 0}, {"flags": 1 << 6}, {"ldy": 23}, {"ldo": 20},
               {"ldo": 0}, {"up": at(2), "ldu": 5}, {"res": at(2), "ldr": 5}, {"y": at(0, 1)}, {"out": at(1, 1)},
               {"y": at(0, 2), "flags": am.IN_F32}, {"out": at(1, 2), "flags": am.OUT_F32}, {"bias": at(3, 1)},
               {"out": at(0, 2)}, {"out": at(0), "ldo": 32}, {"out": at(0), "flags": am.IN_F32},
               {"out": at(0), "flags": am.OUT_F32}, {"bias": at(1)}, {"up": at(1, 48), "ldu": 24},
               {"res": at(1), "ldr": 24, "flags": am.IN_F32 | am.OUT_F32}, {"res": at(1), "ldr": 0}):
        assert epilogue(am, **kw) == bad, kw
    assert epilogue(am, flags=5) == am.ERR_UNSUPPORTED
    assert epilogue(am, n=1 << 31, ldy=1 << 31, ldo=1 << 31) == am.ERR_UNSUPPORTED
    assert epilogue(am, T=1 << 31) == am.ERR_UNSUPPORTED and epilogue(am, ldo=1 << 38) == am.ERR_UNSUPPORTED
    assert epilogue(am, T=0, y=None, out=None) == am.OK


def rotary(am, q=None, k=None, T=4, D=16, rot=16, pos=at(8), freq=at(9), flags=0):
    return am.lib().adafuse_rotary(q, k, T, D, rot, pos, freq, 1.0, 1e-6, flags, None)


def heads(am, src=at(0), out=at(1), its=32, ihs=16, ots=32, ohs=16, weight=None, n=2):
    return ctypes.byref(am.Heads(src, out, its, ihs, ots, ohs, weight, n))


def test_rotary_refusals(am):
    bad, un = am.ERR_INVALID_ARG, am.ERR_UNSUPPORTED
    ok = heads(am)
    assert rotary(am) == bad and rotary(am, ok, T=-1) == bad and rotary(am, ok, D=0) == bad
    assert rotary(am, ok, rot=-2) == bad and rotary(am, ok, flags=1) == bad
    assert rotary(am, ok, rot=15) == un and rotary(am, ok, rot=18) == un and rotary(am, ok, D=1026, rot=16) == un
    assert rotary(am, ok, pos=None) == bad and rotary(am, ok, freq=None) == bad
    assert rotary(am, ok, pos=at(8, 4)) == bad and rotary(am, ok, pos=at(8, 2), flags=am.POS_I32) == bad
    assert rotary(am, ok, freq=at(9, 4)) == bad
    for kw in ({"src": None}, {"out": None}, {"n": 0}, {"src": at(0, 1)}, {"out": at(1, 1)}, {"weight": at(2, 1)},
               {"its": -32}, {"ots": -32}, {"ihs": -16}, {"ohs": -16}, {"ots": 0}, {"ohs": 0}, {"ohs": 8}, {"ots": 24},
               {"out": at(0, 2)}, {"out": at(0), "ots": 48}, {"weight": at(1)}, {"out": at(8)}, {"out": at(9)}):
        assert rotary(am, heads(am, **kw)) == bad, kw
        assert rotary(am, heads(am, src=at(4), out=at(5)), heads(am, **kw)) == bad, kw
    assert rotary(am, heads(am, n=70000)) == un and rotary(am, ok, T=1 << 31) == un
    assert rotary(am, heads(am, its=1 << 38)) == un and rotary(am, heads(am, ots=1 << 40)) == un
    # the two outputs meet, or one output meets the other's input
    assert rotary(am, heads(am), heads(am, src=at(4), out=at(1))) == bad
    assert rotary(am, heads(am), heads(am, src=at(4), out=at(0))) == bad
    assert rotary(am, heads(am), heads(am, src=at(1), out=at(4))) == bad
    # heads of q and k side by side: windows that cross, a token stride that breaks the pattern
    side = dict(its=96, ihs=48, ots=96, ohs=48)
    assert rotary(am, heads(am, src=at(3), out=at(3), **side),
                  heads(am, src=at(3, 16), out=at(3, 16), **side)) == bad
    odd = dict(its=100, ihs=48, ots=100, ohs=48)
    assert rotary(am, heads(am, src=at(3), out=at(3), **odd), heads(am, src=at(3, 40), out=at(3, 40), **odd)) == bad
    assert rotary(am, heads(am, n=2, ots=1 << 37, ohs=16), T=1 << 30) == bad      # rows that reach over the inputs
    assert rotary(am, ok, T=0) == am.OK


def test_binding_refusals(am):
    z = lambda *s, dtype=BF16: torch.zeros(s, dtype=dtype)
    x, W = z(4, 64), z(32, 64)
    freq, pos, q = torch.ones(8, dtype=torch.float64), torch.arange(4), z(4, 2, 16)
    calls = [
        lambda: am.project(x, W),                                   # not on a device
        lambda: am.project(x.float(), W),
        lambda: am.project(x[0], W),
        lambda: am.project(x, z(32, 72)),
        lambda: am.project(z(64, 4).t(), W),
        lambda: am.project(x, W, activation="swish"),
        lambda: am.project(x, W, activation=[]),
        lambda: am.project(x, W, bias=z(31)),
        lambda: am.project(x, W, bias=z(32, dtype=torch.float32)),
        lambda: am.project(x, W, residual=z(3, 32)),
        lambda: am.project(x, W, out=z(4, 40)),
        lambda: am.project(x, W, out_dtype=torch.float16),
        lambda: am.project(x, W, out=z(4, 32), out_dtype=torch.float32),
        lambda: am.project(x, W, status=z(1)),
        lambda: am.gated_project(x, W, z(32, 72)),
        lambda: am.gated_project(x, W, z(32, 80)[:, :64]),
        lambda: am.gated_project(x, W, W, bias_up=z(8)),
        lambda: am.gated_project(x, W, W, out=z(4, 32, dtype=torch.float32)),
        lambda: am.gated_project(x, W, W),
        lambda: am.epilogue(x),
        lambda: am.epilogue(x.double()),
        lambda: am.epilogue(x, up=x.float()),
        lambda: am.epilogue(x, residual=x.float()),
        lambda: am.epilogue(x, bias=z(63)),
        lambda: am.epilogue(x, out=z(4, 63)),
        lambda: am.epilogue(x, activation="tanh"),
        lambda: am.rotary(q, None, pos, freq),
        lambda: am.rotary(x, None, pos, freq),
        lambda: am.rotary(q, None, pos[:3], freq),
        lambda: am.rotary(q, None, pos.float(), freq),
        lambda: am.rotary(q, None, pos, freq.float()),
        lambda: am.rotary(q, None, pos, freq, layout="pairs"),
        lambda: am.rotary(q, None, pos, freq, k_weight=z(16)),
        lambda: am.rotary_frequencies(7),
        lambda: am.rotary_frequencies(0),
        lambda: am.rotary_frequencies(8, scaling="cubic"),
        lambda: am.rotary_frequencies(8, factor=0),
        lambda: am.rotary_frequencies(2, scaling="base", factor=2),
        lambda: am.rotary_frequencies(8, scaling="wavelength", fast_turns=1, slow_turns=1),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was accepted")


def test_reduce_output_adds_to_row_parallel_sums_only():
    from adapter_merge_b200 import tp
    y, b = torch.zeros(2, 8), torch.zeros(8, dtype=BF16)
    assert tp.reduce_output(tp.COLUMN, y) is y and tp.reduce_output(tp.ROW, y) is y
    for kw in ({"bias": b}, {"residual": y.to(BF16)}):
        with pytest.raises(ValueError):
            tp.reduce_output(tp.COLUMN, y, **kw)
