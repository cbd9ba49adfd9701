"""The operators between the adapted linears at the ends of their ranges: tails
of the activations, far positions, long sums, and calls whose CTAs leave while
the other one of a pair has just finished.
"""
from fractions import Fraction

import pytest
import torch

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
HALF = torch.finfo(BF16).eps / 2       # 2^-8
STEP = 2.0 ** -23


@pytest.fixture(scope="module")
def am(cuda_device):
    from adapter_merge_b200 import build
    build.build()
    import adapter_merge_b200
    adapter_merge_b200.lib()
    return adapter_merge_b200


def rnd(*shape, seed=0, std=1.0, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + sum(shape))
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


@pytest.mark.parametrize("T", [513, 600, 640, 1025])
def test_pairs_whose_second_cta_stores_nothing_last(am, T):
    """1 to 128 tokens in the last tile: the pair's second CTA gives its
    accumulator back and is done at once.  Many calls back to back, so that each
    finds shared memory that the last one has just left."""
    assert 1 <= T % 256 <= 128
    x, W, U = rnd(T, 128), rnd(1024, 128, seed=1, std=0.05), rnd(1024, 128, seed=2, std=0.05)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for f in (lambda: am.project(x, W, status=status), lambda: am.project(x, W, out_dtype=F32, status=status),
              lambda: am.gated_project(x, W, U, status=status)):
        first = f()
        assert all(torch.equal(first, y) for y in [f() for _ in range(40)])
    assert int(status) == 0


# ------------------------------------------------------------------ rotation

def arctan_inverse(n, bits):
    """arctan(1 / n) * 2^bits by its series, a few units of the last place off."""
    term = (1 << bits) // n
    total, k = term, 1
    while term:
        term //= -n * n
        k += 2
        total += term // k
    return total


BITS = 400
PI = Fraction(4 * (4 * arctan_inverse(5, BITS) - arctan_inverse(239, BITS)), 1 << BITS)    # Machin


def angle(p, f):
    """p f modulo 2 pi, the product and the reduction in rational numbers."""
    turns = p * Fraction(f) / (2 * PI)
    return float((turns - round(turns)) * 2 * PI)


FAR = [0, 1, -1, 4097, 2 ** 31 - 1, -2 ** 31, 2 ** 33 + 1, 2 ** 40, -2 ** 40 - 7, 2 ** 50, -2 ** 50, 2 ** 53 + 1,
       3 * 10 ** 18, 2 ** 62, -2 ** 62 + 12345, 2 ** 63 - 1, -2 ** 63]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("freq", [
    [10000.0 ** (-i / 64) for i in range(64)], [500000.0 ** (-i / 16) / 8 for i in range(16)],
    [1.0, -1.0, 0.3, -0.01, 6.283185307179586, -6.283185307179586, 1000.25, 1048575.9, 1e-9, -1e-15, 0.0, 2.0 ** -60],
    [3.0], [0.1, 0.7, 1.3]])
def test_rotary_of_far_positions(am, layout, freq):
    """Every int64 position, against angles reduced in rational numbers: the
    stated |p f| 2^-103 of the reduction, fp32 sines and cosines (two steps), of
    an angle rounded to fp32 (half a step of at most pi), two products and a
    sum, and one rounding to bf16."""
    n, T = len(freq), len(FAR)
    x = rnd(T, 2, 2 * n, seed=n)
    pos = torch.tensor(FAR, device="cuda")
    f = torch.tensor(freq, dtype=F64, device="cuda")
    y, _ = am.rotary(x, None, pos, f, layout=layout)
    turn = torch.tensor([[angle(p, v) for v in freq] for p in FAR], dtype=F64, device="cuda")[:, None, :]
    a, b = (slice(0, n), slice(n, 2 * n)) if layout == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    p, q = x[..., a].to(F64), x[..., b].to(F64)
    for got, want in ((y[..., a], p * turn.cos() - q * turn.sin()), (y[..., b], p * turn.sin() + q * turn.cos())):
        err = (8 * STEP + (pos.to(F64)[:, None] * f).abs()[:, None, :] * 2.0 ** -103) * (p.abs() + q.abs())
        assert bool(((got.to(F64) - want).abs() <= err + HALF * (want.abs() + err)).all())


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D", [8, 64, 7])
def test_frequencies_that_are_no_numbers_reach_their_own_pairs(am, layout, D):
    x, pos = rnd(5, 3, D), torch.tensor([0, 1, -3, 2 ** 40, 7], device="cuda")
    n = D // 2 if D % 2 == 0 else 2
    f = torch.full((n,), 0.25, dtype=F64, device="cuda")
    good, _ = am.rotary(x, None, pos, f, layout=layout)
    for i, bad in enumerate((float("nan"), float("inf"), -float("inf"))):
        g = f.clone()
        g[i % n] = bad
        y, _ = am.rotary(x, None, pos, g, layout=layout)
        pair = [i % n, i % n + n] if layout == "half" else [2 * (i % n), 2 * (i % n) + 1]
        rest = [j for j in range(D) if j not in pair]
        assert bool(y[..., pair].isnan().all()) and torch.equal(y[..., rest], good[..., rest])


# ------------------------------------------------------------------ activations

def act64(v, name):
    """Without cancellation or overflow in the tails."""
    if name == "gelu":
        return 0.5 * v * torch.special.erfc(-v / 2 ** 0.5)
    w = v if name == "silu" else (8 / torch.pi) ** 0.5 * (v + 0.044715 * v ** 3)
    return v * torch.special.expit(w)


def act_error(v, name):
    """Relative error of an activation in fp32, in units of 2^-23.
    gelu, v Q(v) with Q(-|v|) = exp(-v^2 / 2) t P(t): the square's rounding is
    0.25 v^2 in the exponent, __expf is off by 2 + 1.173 v^2 / 2 (its documented
    bound); t by 2.5 (a sum and __fdividef's 2), which counts up to 1.1 times;
    P by 0.3 of its fit and 2 of its rounding; three products: 0.84 v^2 + 10.
    silu and gelu_tanh, v / (1 + exp(-w)): __expf is off by 2 + 1.173 |w|, its
    product and the sum by 0.5 each, the division by 2; where exp(-|w|) is below
    2^-126 it is a multiple of 2^-149 (one of at least 2^13 of them here) and off
    by another 2^10.  gelu_tanh's w is off by 3 relative (a square, a product, a
    sum with a share of both, two products: 0.5 each, and its two constants')."""
    if name == "gelu":
        return (0.84 * v * v + 10) * STEP
    w = v if name == "silu" else (8 / torch.pi) ** 0.5 * (v + 0.044715 * v ** 3)
    e = (1.173 if name == "silu" else 1.173 + 3.5) * w.abs() + 7
    return (e + torch.where(w < -87.3, 1024.0, 0.0)) * STEP


TAILS = {"gelu": (-12.8, 14.0), "silu": (-91.5, 100.0), "gelu_tanh": (-10.3, 14.0)}


@pytest.mark.parametrize("name", TAILS)
def test_activations_keep_their_digits_in_the_tails(am, name):
    """Relative to the result, down to where it leaves fp32's normal numbers."""
    lo, hi = TAILS[name]
    v = torch.linspace(lo, hi, 1 << 16, device="cuda", dtype=F32).view(256, 256)
    want = act64(v.to(F64), name)
    rel = act_error(v.to(F64), name)
    y = am.epilogue(v, activation=name, out_dtype=F32)
    assert bool(((y.to(F64) - want).abs() <= rel * want.abs() + 2.0 ** -126).all())
    y = am.epilogue(v, activation=name)
    assert bool(((y.to(F64) - want).abs() <= (rel + HALF * (1 + rel)) * want.abs() + 2.0 ** -126).all())
    # the same behind products with a one in each row, of values that bf16 holds
    b = v.to(BF16).view(512, 128)
    eye = torch.eye(128, dtype=BF16, device="cuda")
    want, rel = act64(b.to(F64), name), act_error(b.to(F64), name)
    for T in (5, 512):
        bound = rel[:T] * want[:T].abs() + 2.0 ** -126
        y = am.project(b[:T], eye, activation=name, out_dtype=F32)
        assert bool(((y.to(F64) - want[:T]).abs() <= bound).all())
        y = am.gated_project(b[:T], eye, torch.zeros_like(eye), activation=name,
                             bias_up=torch.ones(128, dtype=BF16, device="cuda"))
        assert bool(((y.to(F64) - want[:T]).abs() <= bound + HALF * (1 + rel[:T]) * want[:T].abs()).all())


# ------------------------------------------------------------------ long sums

@pytest.mark.parametrize("T,N", [(16, 512), (300, 256)])
def test_longest_sums(am, T, N):
    """Sums of products of one sign, whose partial sums are as large as they can
    be, by the accumulator's rounding towards zero: at most a sixteenth of a
    bf16 rounding of 2^-8 for the longest that are taken.  Projected onto the
    exact results, with rows of every scale within a step, the roundings
    themselves average out (each uniform in 2^-8 of its value: 1.1e-3 / sqrt(TN)
    = 1.3e-5)."""
    K = 131072
    scale = 1 + torch.rand(T, 1, device="cuda", generator=torch.Generator("cuda").manual_seed(T))
    x = (rnd(T, K, dtype=F32).abs() * scale).to(BF16)
    W = rnd(N, K, seed=1, std=0.02).abs()
    want = sum(x[:, k:k + 16384].to(F64) @ W[:, k:k + 16384].to(F64).t() for k in range(0, K, 16384))
    off = lambda y: float((y.to(F64) * want).sum() / (want * want).sum() - 1)
    one = torch.ones(N, dtype=BF16, device="cuda")
    assert abs(off(am.project(x, W))) < HALF / 16
    assert abs(off(am.gated_project(x, torch.zeros_like(W), W, bias_gate=one, activation="relu"))) < HALF / 16
    assert abs(off(am.project(x, W, out_dtype=F32))) < 1.5e-6
    x, W = torch.cat([x, x], 1), torch.cat([W, W], 1)
    assert abs(off(am.project(x, W, out_dtype=F32) / 2)) < 1.5e-6
    for call in (lambda: am.project(x, W), lambda: am.gated_project(x, W, W)):
        with pytest.raises(am.AdafuseError):
            call()
