"""What of the operators between the adapted linears needs no device, at the
ends of its range."""
import math
import os
import subprocess
import sys

import pytest
import torch

import adapter_merge_b200 as am
from adapter_merge_b200 import build as ambuild


@pytest.mark.parametrize("dim", [2, 8, 64, 128, 256])
@pytest.mark.parametrize("base", [1.5, 100.0, 10000.0, 500000.0])
@pytest.mark.parametrize("length", [1, 4, 64, 4096, 65536, 131072, 10 ** 7])
@pytest.mark.parametrize("fast,slow", [(32.0, 1.0), (4.0, 0.5)])
def test_wavelength_scaling_by_the_turns_of_each_pair(dim, base, length, fast, slow):
    """Each pair by its own turns: at least `fast` keeps its frequency, at most
    `slow` is slowed by the whole factor, and between them the share falls
    along the pairs by one step each, from a whole pair outside to one outside."""
    factor = 8.0
    w, mult = am.rotary_frequencies(dim, base=base, scaling="wavelength", factor=factor, original_length=length,
                                    fast_turns=fast, slow_turns=slow)
    assert mult == pytest.approx(0.1 * math.log(factor) + 1)
    index = lambda turns: dim * math.log(length / (turns * 2 * math.pi), base) / 2      # the pair that makes so many
    for i in range(dim // 2):
        f = base ** (-2 * i / dim)
        turns = length * f / (2 * math.pi)
        share = (1 - float(w[i]) / f) / (1 - 1 / factor)        # 0: kept, 1: slowed by the whole factor
        if turns >= fast:
            assert share == pytest.approx(0, abs=1e-12)
        elif turns <= slow:
            assert share == pytest.approx(1, abs=1e-12)
        else:
            lo, hi = max(math.floor(index(fast) + 1e-9), 0), math.ceil(index(slow) - 1e-9)
            assert share == pytest.approx((i - lo) / (hi - lo), abs=1e-9)


def test_wavelength_scaling_of_long_contexts():
    """The slowest pair of 128 turns 2.41 times within 131072 positions: pair 63
    of a ramp from 45 to 70, not its end."""
    w, _ = am.rotary_frequencies(128, scaling="wavelength", factor=8.0, original_length=131072)
    f, _ = am.rotary_frequencies(128)
    assert float(w[63] / f[63]) == pytest.approx(1 - 18 / 25 * 7 / 8, abs=1e-12)


@pytest.mark.parametrize("base", [1.0, 0.5])
def test_wavelength_scaling_needs_frequencies_that_fall(base):
    with pytest.raises(ValueError):
        am.rotary_frequencies(64, base=base, scaling="wavelength", factor=2.0)


# ------------------------------------------------------------------ refusals

@pytest.fixture(scope="module")
def lib():
    ambuild.build()
    return am.lib()


def at(i):
    """A made-up device address, 1 TiB apart (nothing is read before a launch)."""
    return (i + 1) << 40


def test_sums_too_long_for_one_accumulator_are_refused(lib):
    """bf16 results keep one fp32 accumulator that rounds towards zero; fp32
    results add up parts, and take any d_in (refused further on, without a device)."""
    project = lambda K, flags: lib.adafuse_project(at(0), 4, K, K, at(1), 32, K, None, None, 0, at(2), 32, flags, None,
                                                   None)
    gated = lambda K: lib.adafuse_gated_project(at(0), 4, K, K, at(1), at(3), 32, K, None, None, at(2), 32, 2, None,
                                                None)
    for K in (131080, 1 << 20):
        assert project(K, 0) == project(K, 1) == gated(K) == am.ERR_UNSUPPORTED
    if not torch.cuda.is_available():
        assert project(131072, 0) == gated(131072) == project(1 << 20, am.OUT_F32) == am.ERR_DEVICE


# ------------------------------------------------------------------ build

def recorded(monkeypatch, tmp_path, fail=None):
    """Builds into tmp_path by a compiler that only writes its output; the commands."""
    ran = []
    tmp_path = tmp_path / "package"
    tmp_path.mkdir()
    (tmp_path.parent / "include").mkdir()
    (tmp_path.parent / "include" / "adafuse.h").touch()

    def run(cmd):
        if fail and fail in os.path.basename(cmd[0]):
            raise subprocess.CalledProcessError(1, cmd)
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(ambuild, "HERE", str(tmp_path))
    monkeypatch.setattr(ambuild, "LIB", str(tmp_path / "libadafuse.so"))
    monkeypatch.setattr(ambuild.subprocess, "check_call", run)
    return ran


def test_the_library_is_built_without_torch_or_a_host_compiler(monkeypatch, tmp_path):
    ran = recorded(monkeypatch, tmp_path, fail="g++")
    with pytest.raises(subprocess.CalledProcessError):
        ambuild.build()
    assert len(ran) == 1 and os.path.exists(ambuild.LIB)
    ran.clear()
    monkeypatch.setitem(sys.modules, "torch", None)
    assert ambuild.build(force=True) == ambuild.LIB
    assert len(ran) == 1 and "nvcc" in ran[0][0]


def test_a_binding_serves_the_torch_that_it_was_built_for(monkeypatch, tmp_path):
    ran = recorded(monkeypatch, tmp_path)
    first = ambuild.build_binding()
    assert ambuild.build_binding() == first and len(ran) == 1
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    assert not os.path.exists(ambuild.binding_path())
    monkeypatch.setattr(am, "_native", None)
    monkeypatch.setattr(am, "lib", lambda: None)
    with pytest.raises(RuntimeError, match="not built"):
        am._operators()
    second = ambuild.build_binding()
    assert second != first and len(ran) == 2
