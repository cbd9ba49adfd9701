"""GPU parity of the operators between the adapted linears (projection, gated
projection, epilogue, rotation of queries and keys) against plain 64-bit
computations of their formulas.

Tolerances count roundings.  A bf16 output is off by at most half a step,
2^-8 of its value, after fp32 arithmetic whose error is bounded from the sums
of absolute values: the tensor core rounds each step of 16 products towards
zero, so a sum over n columns is taken as off by at most (n / 8 + 8) 2^-23
times the sum of |x w|; an activation has a slope of at most 1.13 and adds a
few fp32 steps of its argument.
"""
import math

import pytest
import torch

import synth

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
HALF = torch.finfo(BF16).eps / 2       # 2^-8
STEP = 2.0 ** -23
ACTS = [None, "relu", "silu", "gelu", "gelu_tanh"]


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


def act64(v, name):
    if name == "relu":
        return torch.where(v < 0, torch.zeros_like(v), v)
    if name == "silu":
        return v / (1 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1 + torch.erf(v / math.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return v


def product64(x, W, bias, part=None):
    """x W^T + bias in 64 bits and the bound of the fp32 error."""
    x, W = x.to(F64), W.to(F64)
    n = x.shape[1] if part is None else min(part, x.shape[1])
    v = x @ W.t()
    e = (x.abs() @ W.abs().t()) * ((n / 8 + 8 + x.shape[1] / n) * STEP)
    if bias is not None:
        v = v + bias.to(F64)
    return v, e + STEP * v.abs()


def after_act(v, e, name):
    return (v, e) if name is None else (act64(v, name), 1.13 * e + 4 * STEP * v.abs())


def check(got, want, err, what=""):
    if got.dtype == BF16:
        err = err + HALF * (want.abs() + err)
    else:
        err = err + STEP * want.abs()
    bad = ~((got.to(F64) - want).abs() <= err + 1e-38)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {bad.nonzero()[0].tolist()}, "
                           f"got {got[bad][0].item()} want {want[bad][0].item()}")


def check_project(am, T, K, N, act=None, bias=False, residual=False, f32=False, seed=0):
    x, W = rnd(T, K, seed=seed), rnd(N, K, seed=seed + 1, std=0.05)
    b = rnd(N, seed=seed + 2) if bias else None
    r = rnd(T, N, seed=seed + 3) if residual else None
    y = am.project(x, W, bias=b, activation=act, residual=r, out_dtype=F32 if f32 else None)
    v, e = after_act(*product64(x, W, b, 512 if f32 else None), act)
    if r is not None:
        v = v + r.to(F64)
        e = e + STEP * v.abs()
    assert y.dtype == (F32 if f32 else BF16) and y.shape == (T, N)
    check(y, v, e, f"project {T}x{K}->{N}")


def check_gated(am, T, K, N, act="silu", bias=False, seed=0):
    x, Wg, Wu = rnd(T, K, seed=seed), rnd(N, K, seed=seed + 1, std=0.05), rnd(N, K, seed=seed + 2, std=0.05)
    bg, bu = (rnd(N, seed=seed + 3), rnd(N, seed=seed + 4)) if bias else (None, None)
    y = am.gated_project(x, Wg, Wu, bias_gate=bg, bias_up=bu, activation=act)
    a, ea = after_act(*product64(x, Wg, bg), act)
    u, eu = product64(x, Wu, bu)
    check(y, a * u, a.abs() * eu + u.abs() * ea + ea * eu + STEP * (a * u).abs(), f"gated {T}x{K}->{N}")


# ------------------------------------------------------------------ projections

@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 33, 64, 65, 128, 129, 255, 256, 257, 300, 515])
def test_project_token_counts(am, T):
    check_project(am, T, 200, 264, residual=True, seed=T)
    check_project(am, T, 1096, 136, bias=True, act="silu", f32=True, seed=T)


@pytest.mark.parametrize("K,N", [(8, 8), (56, 8), (64, 128), (72, 120), (128, 136), (512, 4096), (4096, 256),
                                 (1376, 4096), (11008, 24), (4096, 4096), (5120, 13824)])
def test_project_widths(am, K, N):
    check_project(am, 1, K, N, seed=1)
    check_project(am, 19, K, N, bias=True, residual=True, seed=2)
    check_project(am, 130, K, N, f32=True, seed=3)


@pytest.mark.parametrize("T", [1, 17, 33, 48, 64, 80, 96, 112, 128, 144, 160, 176, 192, 208, 224, 240, 256, 272, 500])
def test_projections_over_many_laps_of_a_ring(am, T):
    """Rings of every depth, walked many times by one CTA, alone and in clusters."""
    check_project(am, T, 13824, 128, seed=T)
    check_project(am, T, 8192, 1024, f32=True, seed=T)
    check_project(am, T, 2048, 13824, seed=T)
    check_gated(am, T, 13824, 128, seed=T)
    check_gated(am, T, 2048, 13824, seed=T)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T", [3, 270])
def test_project_activations(am, act, T):
    check_project(am, T, 192, 272, act=act, bias=True, residual=True)
    check_project(am, T, 192, 272, act=act, f32=True)


@pytest.mark.parametrize("T,K,N", [(512, 1024, 2048), (1000, 520, 1336), (2049, 4096, 1024), (4096, 256, 512),
                                   (777, 64, 8), (1500, 2048, 5000), (300, 4096, 11008)])
def test_project_prompts(am, T, K, N):
    check_project(am, T, K, N, residual=True, seed=5)
    check_project(am, T, K, N, bias=True, act="gelu", seed=6)
    check_project(am, T, K, N, f32=True, seed=7)


@pytest.mark.parametrize("T", [1, 2, 16, 17, 64, 100, 128, 129, 256, 300, 600])
def test_gated_token_counts(am, T):
    check_gated(am, T, 200, 264, seed=T)
    check_gated(am, T, 1096, 136, bias=True, act="gelu_tanh", seed=T)


@pytest.mark.parametrize("K,N", [(8, 8), (64, 128), (72, 136), (512, 4096), (4096, 11008), (5120, 13824)])
def test_gated_widths(am, K, N):
    check_gated(am, 1, K, N, seed=1)
    check_gated(am, 40, K, N, bias=True, seed=2)


@pytest.mark.parametrize("act", ACTS)
def test_gated_activations(am, act):
    check_gated(am, 5, 192, 272, act=act, bias=True)
    check_gated(am, 700, 192, 272, act=act)


@pytest.mark.parametrize("T,K,N", [(512, 1024, 2048), (1000, 520, 1336), (2049, 4096, 1024), (777, 64, 8)])
def test_gated_prompts(am, T, K, N):
    check_gated(am, T, K, N, seed=5)


def test_gated_biases_are_independent(am):
    x, Wg, Wu = rnd(9, 64), rnd(40, 64, seed=1), rnd(40, 64, seed=2)
    b = rnd(40, seed=3)
    for kw in ({"bias_gate": b}, {"bias_up": b}):
        y = am.gated_project(x, Wg, Wu, **kw)
        a, ea = after_act(*product64(x, Wg, kw.get("bias_gate")), "silu")
        u, eu = product64(x, Wu, kw.get("bias_up"))
        check(y, a * u, a.abs() * eu + u.abs() * ea + ea * eu + STEP * (a * u).abs())


@pytest.mark.parametrize("T", [1, 37, 300, 1100])
def test_projections_of_strided_views_touch_nothing_else(am, T):
    """Operands and results that are columns of wider buffers, filled with NaN
    around what may be read, and unchanged around what is written."""
    K, N = 264, 328
    nan = float("nan")

    def view(rows, cols, seed, left=8, right=24, std=1.0, dtype=BF16):
        buf = torch.full((rows + 2, left + cols + right), nan, dtype=dtype, device="cuda")
        v = buf[1:rows + 1, left:left + cols]
        v.copy_(rnd(rows, cols, seed=seed, std=std, dtype=dtype))
        return buf, v

    _, x = view(T, K, 1)
    _, W = view(N, K, 2, std=0.05)
    _, U = view(N, K, 3, std=0.05)
    _, r = view(T, N, 4)
    for dtype in (BF16, F32):
        buf = torch.full((T + 2, N + 40), 3.0, dtype=dtype, device="cuda")
        y = buf[1:T + 1, 16:16 + N]
        assert am.project(x, W, residual=r, out=y) is y
        v, e = product64(x, W, None, 512 if dtype == F32 else None)
        check(y, v + r.to(F64), e + STEP * v.abs() + STEP * r.abs())
        y.fill_(3.0)
        assert bool((buf == 3.0).all())
    buf = torch.full((T + 2, N + 40), 3.0, dtype=BF16, device="cuda")
    y = buf[1:T + 1, 16:16 + N]
    am.gated_project(x, W, U, out=y)
    a, ea = after_act(*product64(x, W, None), "silu")
    u, eu = product64(x, U, None)
    check(y, a * u, a.abs() * eu + u.abs() * ea + ea * eu + STEP * (a * u).abs())
    y.fill_(3.0)
    assert bool((buf == 3.0).all())


@pytest.mark.parametrize("T", [1, 50, 400])
def test_project_residual_in_place_and_broadcast(am, T):
    x, W = rnd(T, 128), rnd(256, 128, seed=1, std=0.05)
    v, e = product64(x, W, None)
    stream = rnd(T, 256, seed=2)
    want = v + stream.to(F64)
    assert am.project(x, W, residual=stream, out=stream) is stream
    check(stream, want, e + STEP * want.abs())
    one = rnd(1, 256, seed=3)
    y = am.project(x, W, residual=one.expand(T, 256))
    want = v + one.to(F64)
    check(y, want, e + STEP * want.abs())


@pytest.mark.parametrize("T", [5, 300, 700])
def test_bad_values_stay_in_their_rows_and_columns(am, T):
    """A token of NaN and one of infinities, and a row of W of NaN, reach their
    own results only."""
    x, W, U = rnd(T, 192), rnd(160, 192, seed=1), rnd(160, 192, seed=2)
    for f in (lambda: am.project(x, W, activation="silu"), lambda: am.gated_project(x, W, U)):
        good = f()
        x2, W2 = x.clone(), W.clone()
        x2[2] = float("nan")
        x2[T - 1] = float("inf")
        W2[7] = float("nan")
        saved, savedW = x, W
        x, W = x2, W2
        bad = f()
        x, W = saved, savedW
        rows = [t for t in range(T) if t not in (2, T - 1)]
        cols = [o for o in range(160) if o != 7]
        assert torch.equal(good[rows][:, cols], bad[rows][:, cols])
        assert bool(bad[2].isnan().all()) and bool(bad[:, 7].isnan().all())
        assert not bool(bad[T - 1].isfinite().logical_and(bad[T - 1] != 0).any())


@pytest.mark.parametrize("T", [1, 64, 200, 1030])
def test_projections_are_deterministic(am, T):
    x, W, U = rnd(T, 2048), rnd(1032, 2048, seed=1), rnd(1032, 2048, seed=2)
    for f in (lambda: am.project(x, W), lambda: am.project(x, W, out_dtype=F32), lambda: am.gated_project(x, W, U)):
        first = f()
        for _ in range(5):
            assert torch.equal(first, f())


def test_fp32_sums_stay_near_fp32_over_long_rows(am):
    """Parts of at most 512 columns: an error that grows with d_in would be
    1.2e-5 relative at 11008 columns (measured for one accumulator)."""
    for T, N in ((4, 256), (200, 256), (600, 256), (16, 13824), (100, 13824), (256, 5120), (1500, 1024)):
        x, W = rnd(T, 11008), rnd(N, 11008, seed=1, std=0.02)
        want = x.to(F64) @ W.to(F64).t()
        y = am.project(x, W, out_dtype=F32).to(F64)
        assert float((y - want).norm() / want.norm()) < 1.5e-6


# ------------------------------------------------------------------ epilogue

@pytest.mark.parametrize("T,n", [(1, 1), (1, 8), (3, 7), (64, 11008), (33, 1000), (5, 13824), (2000, 24), (1, 40000)])
@pytest.mark.parametrize("f32_in,f32_out", [(False, False), (True, False), (False, True), (True, True)])
def test_epilogue_shapes_and_types(am, T, n, f32_in, f32_out):
    kind = F32 if f32_in else BF16
    y, up, r, b = rnd(T, n, dtype=kind), rnd(T, n, seed=1, dtype=kind), rnd(T, n, seed=2), rnd(n, seed=3)
    for act in ACTS:
        for bias, u, res in ((None, None, None), (b, up, None), (b, None, r), (None, up, r)):
            got = am.epilogue(y, bias=bias, activation=act, up=u, residual=res, out_dtype=F32 if f32_out else None)
            v = y.to(F64) if bias is None else y.to(F64) + bias.to(F64)
            v, e = after_act(v, STEP * v.abs(), act)
            if u is not None:
                v, e = v * u.to(F64), e * u.to(F64).abs() + STEP * (v * u.to(F64)).abs()
            if res is not None:
                v = v + res.to(F64)
                e = e + STEP * v.abs()
            check(got, v, e, f"epilogue {T}x{n} {act}")


def test_epilogue_strides_broadcast_and_in_place(am):
    T, n = 21, 88
    buf = rnd(T, 3 * n + 1)
    for off in (0, 1):             # 16-byte groups, and single elements
        y, up = buf[:, off:off + n], buf[:, n + off:2 * n + off]
        got = am.epilogue(y, activation="silu", up=up)
        v = act64(y.to(F64), "silu")
        check(got, v * up.to(F64), 8 * STEP * (v * up.to(F64)).abs() + 4 * STEP * (y * up).to(F64).abs())
    one = rnd(1, n, seed=1)
    y = rnd(T, n, seed=2)
    check(am.epilogue(y, residual=one.expand(T, n)), y.to(F64) + one.to(F64), STEP * (y.abs() + one.abs()).to(F64))
    for name in ("y", "up", "residual"):
        t = {"y": rnd(T, n, seed=3), "up": rnd(T, n, seed=4), "residual": rnd(T, n, seed=5)}
        want = am.epilogue(**t)
        got = am.epilogue(**t, out=t[name])
        assert got is t[name] and torch.equal(got, want)


def test_epilogue_of_one_row_for_all_tokens(am):
    T, n = 70, 96
    y, up, r = rnd(1, n), rnd(1, n, seed=1), rnd(1, n, seed=2)
    got = am.epilogue(y.expand(T, n), activation="relu", up=up.expand(T, n), residual=r.expand(T, n))
    assert torch.equal(got, am.epilogue(y, activation="relu", up=up, residual=r).expand(T, n))


def test_offsets_past_32_bits(am):
    """5 GB of outputs: rows whose element offsets, and byte offsets, pass 2^31 and 2^32."""
    T, K, N = 600_000, 64, 4096
    x, W = rnd(T, K), rnd(N, K, seed=1, std=0.05)
    y = am.project(x, W)
    rows = torch.tensor([0, 262_143, 262_144, 524_287, 524_288, T - 257, T - 1], device="cuda")
    check(y[rows], *product64(x[rows], W, None))
    z = am.epilogue(y, activation="relu", residual=y, out=y)
    assert z is y
    v, e = product64(x[rows], W, None)
    check(y[rows], act64(v, "relu") + v, 2 * e + 3 * HALF * v.abs())
    freq, _ = am.rotary_frequencies(64, device="cuda")
    pos = torch.arange(T, device="cuda")
    q = y.view(T, 64, 64)
    want = rotary64(q[rows], None, pos[rows], freq, "half", 1.0, 0)
    am.rotary(q, None, pos, freq, q_out=q)
    check(q[rows], *want)


def test_epilogue_extremes(am):
    inf, nan = float("inf"), float("nan")
    y = torch.tensor([[0.0, -0.0, inf, nan, 1e4, -1e4, 90.0, -90.0]], device="cuda")
    got = am.epilogue(y, activation="silu", out_dtype=F32)[0].tolist()
    assert got[:2] == [0, 0] and got[2] == inf and math.isnan(got[3]) and got[4:6] == [1e4, 0] and got[6] == 90
    assert abs(got[7]) < 1e-36
    got = am.epilogue(y, activation="gelu", out_dtype=F32)[0].tolist()
    assert got[2] == inf and math.isnan(got[3]) and got[4:] == [1e4, 0, 90, 0]
    got = am.epilogue(y, activation="relu", out_dtype=F32)[0].tolist()
    assert got[2] == inf and math.isnan(got[3]) and got[4:] == [1e4, 0, 90, 0]
    big = torch.tensor([[3.4e38, 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8]], device="cuda")
    assert am.epilogue(big)[0].tolist() == [inf, 1.0, 1 + 2.0 ** -6]      # one rounding, ties to even


# ------------------------------------------------------------------ rotation

def rotary64(x, weight, positions, freq, layout, factor, eps):
    """The formula in 64 bits and the bound of the fp32 error."""
    x, D, n = x.to(F64), x.shape[2], freq.shape[0]
    e = torch.zeros_like(x)
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.to(F64)
        e = x.abs() * ((D / 2 + 8) * STEP / 2)
    a, b = (slice(0, n), slice(n, 2 * n)) if layout == "half" else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    # exact turns: positions and frequencies as they are, reduced in 64 bits
    angle = (positions.to(F64)[:, None] * freq)[:, None, :]
    c, s = angle.cos() * factor, angle.sin() * factor
    y, ey = x.clone(), e.clone()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    both = (e[..., a] + e[..., b] + (x[..., a].abs() + x[..., b].abs()) * 8 * STEP) * abs(factor)
    ey[..., a] = both
    ey[..., b] = both
    return y, ey


def check_rotary(am, T, Hq, Hk, D, rot, layout, norm=False, factor=1.0, pos=None, seed=0, dtype=torch.int64):
    q, k = rnd(T, Hq, D, seed=seed), rnd(T, Hk, D, seed=seed + 1)
    wq, wk = (rnd(D, seed=seed + 2), rnd(D, seed=seed + 3)) if norm else (None, None)
    if pos is None:
        pos = torch.randint(-5000, 1 << 20, (T,), device="cuda", generator=torch.Generator("cuda").manual_seed(seed))
    freq, _ = am.rotary_frequencies(rot, device="cuda") if rot else (torch.empty(0, dtype=F64, device="cuda"), 1)
    qo, ko = am.rotary(q, k, pos.to(dtype), freq, layout=layout, factor=factor, q_weight=wq, k_weight=wk)
    for got, x, w in ((qo, q, wq), (ko, k, wk)):
        check(got, *rotary64(x, w, pos, freq, layout, factor, 1e-6), f"rotary {T} {Hq} {Hk} {D} {rot} {layout}")


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 64), (64, 64), (80, 80), (96, 96), (112, 56), (256, 256), (192, 96),
                                   (2, 2), (6, 4), (7, 2), (33, 32), (320, 320), (512, 512), (1024, 1024), (1000, 500),
                                   (128, 0)])
def test_rotary_head_sizes(am, layout, D, rot):
    check_rotary(am, 5, 3, 2, D, rot, layout, seed=1)
    check_rotary(am, 5, 4, 1, D, rot, layout, norm=True, factor=1.2, seed=2)


@pytest.mark.parametrize("T,Hq,Hk", [(1, 1, 1), (1, 32, 8), (2, 40, 40), (64, 32, 32), (1183, 8, 1), (2500, 5, 5),
                                     (5000, 1, 1)])
def test_rotary_tokens_and_heads(am, T, Hq, Hk):
    for norm in (False, True):
        check_rotary(am, T, Hq, Hk, 128, 128, "half", norm=norm, seed=3)
        check_rotary(am, T, Hq, Hk, 80, 40, "interleaved", norm=norm, seed=4)


def test_rotary_positions(am):
    far = torch.tensor([0, 1, -1, 2 ** 20, 2 ** 31 - 1, -2 ** 31], device="cuda")
    check_rotary(am, 6, 2, 2, 64, 64, "half", pos=far)
    check_rotary(am, 6, 2, 2, 64, 64, "half", pos=far, dtype=torch.int32)
    # whole turns come back to the start exactly, however far
    x = rnd(4, 1, 4)
    turns = torch.tensor([0, 2 ** 40, -2 ** 50, 2 ** 62], device="cuda")
    freq = torch.full((2,), 2 * math.pi, dtype=F64, device="cuda")
    y, none = am.rotary(x, None, turns[:1].expand(4).contiguous(), freq)
    assert none is None and torch.equal(x, y)
    # frequencies outside one turn, zero and negative ones
    freq = torch.tensor([0.0, -0.3, 100.0, 2 * math.pi * 3 + 0.1], dtype=F64, device="cuda")
    x, pos = rnd(9, 2, 8), torch.arange(9, device="cuda") * 11
    y, _ = am.rotary(x, None, pos, freq)
    check(y, *rotary64(x, None, pos, freq, "half", 1.0, 0))


def test_rotary_by_minus_p_undoes_p(am):
    """Cached keys move to new positions by rotating them by the difference."""
    freq, _ = am.rotary_frequencies(128, device="cuda")
    x = rnd(50, 4, 128)
    pos = torch.arange(50, device="cuda") * 997
    y, _ = am.rotary(x, None, pos, freq)
    z, _ = am.rotary(y, None, -pos, freq)
    pair = x.view(50, 4, 2, 64).to(F64).norm(dim=2).repeat(1, 1, 2)
    assert bool(((z.to(F64) - x.to(F64)).abs() <= HALF * (x.to(F64).abs() + 1.5 * pair)).all())


@pytest.mark.parametrize("D,lead", [(128, 0), (128, 8), (80, 4), (64, 1)])
def test_rotary_in_place_in_a_fused_buffer(am, D, lead):
    """q and k as columns of the rows that one projection wrote, rotated where
    they are; v and what surrounds them stay."""
    T, Hq, Hk = 13, 4, 2
    buf = rnd(T, lead + (Hq + 2 * Hk) * D + 8)
    was = buf.clone()
    q = buf[:, lead:lead + Hq * D].unflatten(1, (Hq, D))
    k = buf[:, lead + Hq * D:lead + (Hq + Hk) * D].unflatten(1, (Hk, D))
    pos = torch.arange(T, device="cuda") + 100
    freq, _ = am.rotary_frequencies(D, device="cuda")
    wq, wk = rnd(D, seed=1), rnd(D, seed=2)
    want = am.rotary(q, k, pos, freq, q_weight=wq, k_weight=wk)
    check(want[0], *rotary64(q, wq, pos, freq, "half", 1.0, 1e-6))
    got = am.rotary(q, k, pos, freq, q_weight=wq, k_weight=wk, q_out=q, k_out=k)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(buf[:, :lead], was[:, :lead])
    assert torch.equal(buf[:, lead + (Hq + Hk) * D:], was[:, lead + (Hq + Hk) * D:])
    # keys into a head-major cache, one norm only
    cache = torch.full((Hk, T + 3, D), 7.0, dtype=BF16, device="cuda")
    am.rotary(q, k, pos, freq, k_weight=wk, k_out=cache[:, 1:T + 1].transpose(0, 1))
    check(cache[:, 1:T + 1].transpose(0, 1), *rotary64(k, wk, pos, freq, "half", 1.0, 1e-6))
    assert bool((cache[:, 0] == 7).all()) and bool((cache[:, T + 1:] == 7).all())


@pytest.mark.parametrize("T,heads", [(1, 1), (1, 4), (9, 1), (9, 4)])
def test_rotary_in_place_with_q_k_v_of_a_head_side_by_side(am, T, heads):
    D = 64
    buf = rnd(T, heads, 3, D)
    was = buf.clone()
    q, k = buf[:, :, 0], buf[:, :, 1]
    pos, (freq, _) = torch.arange(T, device="cuda") + 5, am.rotary_frequencies(D, device="cuda")
    want = am.rotary(q, k, pos, freq)
    am.rotary(q, k, pos, freq, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(buf[:, :, 2], was[:, :, 2])
    # one token or one head: a stride that is not used says nothing
    x = rnd(1, 2, D)
    y = torch.as_strided(x, (1, 2, D), (7 * D, D, 1))
    want, _ = am.rotary(x, None, pos[:1], freq)
    am.rotary(x, None, pos[:1], freq, q_out=y)
    assert torch.equal(x, want)


def test_norm_of_zero_tiny_and_huge_heads(am):
    x = torch.zeros(3, 1, 64, dtype=BF16, device="cuda")
    x[1] = 1e-4
    x[2] = 1e17
    w = torch.ones(64, dtype=BF16, device="cuda")
    freq, _ = am.rotary_frequencies(64, device="cuda")
    pos = torch.zeros(3, dtype=torch.int64, device="cuda")
    y, _ = am.rotary(x, None, pos, freq, q_weight=w)
    check(y, *rotary64(x, w, pos, freq, "half", 1.0, 1e-6))


def test_frequency_scalings(am):
    f, m = am.rotary_frequencies(128)
    assert m == 1.0 and f[0] == 1 and abs(float(f[1]) - 10000 ** (-2 / 128)) < 1e-15
    assert torch.equal(am.rotary_frequencies(128, scaling="linear", factor=4)[0], f / 4)
    b, m = am.rotary_frequencies(128, scaling="base", factor=4)
    assert m == 1.0 and b[0] == 1 and abs(float(b[-1] / f[-1]) - 0.25) < 1e-12
    w, m = am.rotary_frequencies(128, scaling="wavelength", factor=8)
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(w[turns > 40], f[turns > 40]) and torch.allclose(w[turns < 0.9], f[turns < 0.9] / 8, rtol=1e-14)
    assert bool((w <= f).all()) and bool((w >= f / 8 * (1 - 1e-12)).all())
    assert m == pytest.approx(0.1 * math.log(8) + 1)


# ------------------------------------------------------------------ calls

def everything(am, x, W, U, pos, freq):
    """The operators as a layer uses them, each reading what the last one wrote."""
    T, H = x.shape
    q = am.project(x, W, residual=x)
    a, _ = am.rotary(q.view(T, -1, 64), None, pos, freq)
    h = am.gated_project(a.reshape(T, H), W, U)
    return am.epilogue(h, activation="gelu", up=q, residual=x)


def test_no_tokens(am):
    e = lambda *s: torch.empty(s, dtype=BF16, device="cuda")
    assert am.project(e(0, 64), e(32, 64)).shape == (0, 32)
    assert am.gated_project(e(0, 64), e(32, 64), e(32, 64)).shape == (0, 32)
    assert am.epilogue(e(0, 5), up=e(0, 5)).shape == (0, 5)
    freq, _ = am.rotary_frequencies(64, device="cuda")
    q, k = am.rotary(e(0, 2, 64), e(0, 1, 64), torch.empty(0, dtype=torch.int64, device="cuda"), freq)
    assert q.shape == (0, 2, 64) and k.shape == (0, 1, 64)


@pytest.mark.parametrize("T", [2, 300])
def test_another_stream_and_a_captured_graph(am, T):
    H = 512
    x, W, U = rnd(T, H), rnd(H, H, seed=1, std=0.05), rnd(H, H, seed=2, std=0.05)
    pos, (freq, _) = torch.arange(T, device="cuda"), am.rotary_frequencies(64, device="cuda")
    want = everything(am, x, W, U, pos, freq)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = am.project(x, W, stream=side)
    z = am.epilogue(y, activation="silu", stream=side.cuda_stream)
    side.synchronize()
    ref = am.epilogue(am.project(x, W), activation="silu")
    assert torch.equal(z, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = everything(am, x, W, U, pos, freq)
    got.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    x.copy_(rnd(T, H, seed=9))
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, everything(am, x, W, U, pos, freq))


def test_calls_on_two_streams_at_once(am):
    """No call keeps anything that another could disturb."""
    x, W, U = rnd(40, 4096), rnd(4096, 4096, seed=1, std=0.02), rnd(4096, 4096, seed=2, std=0.02)
    X = rnd(700, 4096, seed=3)
    a, b, c = am.project(x, W), am.gated_project(x, W, U), am.project(X, W)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    out = []
    for _ in range(20):
        out.append((am.project(x, W, stream=streams[0]), am.gated_project(x, W, U, stream=streams[1]),
                    am.project(X, W, stream=streams[2])))
    torch.cuda.synchronize()
    for p, q, r in out:
        assert torch.equal(p, a) and torch.equal(q, b) and torch.equal(r, c)


def test_a_wait_that_gives_up_is_reported(am):
    """The test hook withholds one load: the call ends, says so, and the next is right."""
    for T, gated in ((3, False), (3, True), (600, False), (600, True)):
        x, W, U = rnd(T, 512), rnd(256, 512, seed=1), rnd(256, 512, seed=2)
        good = am.gated_project(x, W, U) if gated else am.project(x, W)
        y = torch.zeros_like(good)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        if gated:
            rc = am.lib().adafuse_gated_project(x.data_ptr(), T, 512, 512, W.data_ptr(), U.data_ptr(), 256, 512, None,
                                                None, y.data_ptr(), 256, am.TEST_STALL | 2, status.data_ptr(), None)
        else:
            rc = am.lib().adafuse_project(x.data_ptr(), T, 512, 512, W.data_ptr(), 256, 512, None, None, 0,
                                          y.data_ptr(), 256, am.TEST_STALL, status.data_ptr(), None)
        torch.cuda.synchronize()
        assert rc == 0 and int(status) == am.STATUS_TIMEOUT
        status.zero_()
        again = am.gated_project(x, W, U, status=status) if gated else am.project(x, W, status=status)
        assert torch.equal(again, good) and int(status) == 0


def test_row_parallel_shards_of_a_projection(am):
    """Two shards of the input columns, fp32 partial sums, added (in place of
    the all-reduce), then bias and residual with the one rounding."""
    from adapter_merge_b200 import tp
    T, K, N = 37, 512, 264
    x, W, b, r = rnd(T, K), rnd(N, K, seed=1, std=0.05), rnd(N, seed=2), rnd(T, N, seed=3)
    parts = []
    for rank in range(2):
        i0, i1 = tp.block(K, rank, 2)
        parts.append(am.project(x[:, i0:i1], W[:, i0:i1], out_dtype=F32))
    y = parts[0] + parts[1]
    v, e = product64(x, W, None, 512)
    want = v + b.to(F64) + r.to(F64)
    err = e + 4 * STEP * (v.abs() + b.to(F64).abs() + r.to(F64).abs())
    check(tp.reduce_output(tp.ROW, y, bias=b, residual=r), want, err)
    assert tp.reduce_output(tp.ROW, y, out=r, bias=b, residual=r) is r
    check(r, want, err)
    check(tp.reduce_output(tp.ROW, y, out=r), v, err)


# ------------------------------------------------------------------ a layer

def test_a_layer_merged_and_unmerged(am, cuda_device):
    """One decoder layer of a request whose tokens share a selection, both ways:
    the merged weights through project / gated_project, and the unmerged apply
    with the epilogue, with the rotation between."""
    H, F, heads, T, E, r, k = 256, 512, 4, 24, 4, 8, 2
    D = H // heads
    shapes = [(3 * H, H), (H, H), (F, H), (F, H), (H, F)]         # qkv, o, gate, up, down
    cfg = synth.custom(shapes, E, r, k, T, name="layer")
    w = synth.make_weights(cfg, 0, device=cuda_device)
    Wo = [torch.empty_like(t) for t in w.W_views]
    x, W_r = rnd(T, H), rnd(E, H, seed=1, std=H ** -0.5, dtype=F32)
    idx, gate = am.pregate(x, W_r, k, pool=True)
    wq, wk = 1 + rnd(D, seed=2, std=0.1), 1 + rnd(D, seed=3, std=0.1)
    pos, (freq, m) = torch.arange(T, device="cuda") + 777, am.rotary_frequencies(D, scaling="linear", factor=2.0,
                                                                                 device="cuda")

    def mix(qkv):
        q, kk, v = (t.unflatten(1, (heads, D)) for t in qkv.split(H, dim=1))
        q, kk = am.rotary(q, kk, pos, freq, factor=m, q_weight=wq, k_weight=wk)
        s = torch.einsum("thd,shd->hts", q.float(), kk.float()) / D ** 0.5
        s = s.masked_fill(torch.ones(T, T, device="cuda").triu(1).bool(), float("-inf")).softmax(-1)
        return torch.einsum("hts,shd->thd", s, v.float()).reshape(T, H).to(BF16).contiguous()

    plan = am.Plan(list(zip(w.W_views, Wo, w.A_views, w.B_views)), E, r)
    plan.merge(idx[0], gate[0])
    a = am.project(mix(am.project(x, Wo[0])), Wo[1], residual=x)
    merged = am.project(am.gated_project(a, Wo[2], Wo[3]), Wo[4], residual=a)

    sel, g = idx.expand(T, k).contiguous(), gate.expand(T, k).contiguous()

    def apply(which, inputs):
        p = am.Plan([(w.W_views[i], Wo[i], w.A_views[i], w.B_views[i]) for i in which], E, r)
        ys = [torch.empty(T, shapes[i][0], dtype=BF16, device="cuda") for i in which]
        p.apply(inputs, ys, T, sel, g, torch.empty(p.workspace_bytes(T, k), dtype=torch.uint8, device="cuda"))
        assert p.status() == (0, 0)
        return ys

    qkv, = apply([0], [x])
    o, = apply([1], [mix(qkv)])
    a2 = am.epilogue(o, residual=x, out=o)
    yg, yu = apply([2, 3], [a2, a2])
    h = am.epilogue(yg, activation="silu", up=yu)
    d, = apply([4], [h])
    unmerged = am.epilogue(d, residual=a2)
    assert plan.status() == (0, 0)

    # the same layer in 64 bits
    dW = [wv.to(F64) + sum(float(gate[0, s]) * w.B_views[i][int(idx[0, s])].to(F64) @ w.A_views[i][int(idx[0, s])].to(F64)
                           for s in range(k)) for i, wv in enumerate(w.W_views)]
    x64 = x.to(F64)
    q, kk, v = (t.unflatten(1, (heads, D)) for t in (x64 @ dW[0].t()).split(H, dim=1))
    q, kk = (rotary64(t, n, pos, freq, "half", m, 1e-6)[0] for t, n in ((q, wq), (kk, wk)))
    s = torch.einsum("thd,shd->hts", q, kk) / D ** 0.5
    s = s.masked_fill(torch.ones(T, T, device="cuda").triu(1).bool(), float("-inf")).softmax(-1)
    a64 = torch.einsum("hts,shd->thd", s, v).reshape(T, H) @ dW[1].t() + x64
    want = (act64(a64 @ dW[2].t(), "silu") * (a64 @ dW[3].t())) @ dW[4].t() + a64
    # six roundings to bf16 (merged weights or outputs) on the way, none amplified: a few half steps of the whole
    for got in (merged, unmerged):
        assert float((got.to(F64) - want).norm() / want.norm()) < 6 * HALF
