"""GPU parity of the gated feed-forward and its backward pass against fp64.

Bounds, per output and to first order, with u half a step of the element type
(2^-11 fp16, 2^-8 bf16), e = 2^-23 (one fp32 step, which also covers sums that
truncate) and sums of n terms erring by at most (n + 64) e of the sum of
magnitudes:

  h, g       eh = (C + 64) e (|x| |Wh|^T + |bh|), eg alike
  GELU       |GELU'| <= 1.13;  the erf approximation errs by 1.5e-7 in erf and
             2^-21 relative through exp and the reciprocal:
             eG = 1.13 eg + |g| 6e-7
  y          |h| eG + |GELU| eh + u |y|
  GELU'      |GELU''| <= 0.8:  eS = 0.8 eg + (1 + |g|) 6e-7
  P = [dh, dg] before rounding: |dy| eG, |dy| (|h| eS + |GELU'| eh)
  P rounded  + u |P| (+ half a subnormal step, fp16)
  dx         sum over P's columns of (error of P) |W| + (2F + 64) e |P| |W| + u |dx|
  dW         sum over rows of (error of P) |x| + (T + 64) e |P|^T |x| + u |dW|
  db         sum over rows of P's unrounded error + (T + 64) e |P|
"""
import pytest

from oracle import unet_ops

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import diffusion_unet_attention_b200 as sd  # noqa: E402

DEV = torch.device("cuda:0")
HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
SUB = {torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}
E32 = 2.0 ** -23


def make(seed, T, C, F, dtype, bias=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, C, generator=g).to(dtype).to(DEV)
    w = (torch.randn(2 * F, C, generator=g) / C ** 0.5).to(dtype).to(DEV)
    b = (0.2 * torch.randn(2 * F, generator=g)).to(DEV) if bias else None
    dy = (0.3 * torch.randn(T, F, generator=g)).to(dtype).to(DEV)
    return x, w, b, dy


def within(got, ref, bound, what):
    assert got.shape == ref.shape, what
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    assert bool((err <= bound + 1e-30).all()), f"{what}: off by {float((err / (bound + 1e-30)).max()):.2f} of its bound"


def parts(x, w, b):
    """h, g, their errors, GELU and its slope, in fp64 (the oracle's formulas, as torch tensors)."""
    x, w = x.double(), w.double()
    F = w.shape[0] // 2
    b = torch.zeros(2 * F, dtype=torch.float64, device=DEV) if b is None else b.double()
    p, mag = x @ w.T + b, x.abs() @ w.abs().T + b.abs()
    e = (x.shape[1] + 64) * E32 * mag
    h, g = p[:, :F], p[:, F:]
    cdf = 0.5 * torch.erfc(-g / 2 ** 0.5)
    slope = cdf + g * torch.exp(-g * g / 2) / (2 * torch.pi) ** 0.5
    return h, g, e[:, :F], e[:, F:], g * cdf, slope


def check_forward(x, w, b, y, dtype, what=""):
    h, g, eh, eg, gelu, _ = parts(x, w, b)
    eG = 1.13 * eg + g.abs() * 6e-7
    ref = h * gelu
    within(y, ref, h.abs() * eG + gelu.abs() * eh + HALF_STEP[dtype] * ref.abs() + SUB[dtype], f"y {what}")


def check_backward(x, w, b, dy, got, dtype, what=""):
    h, g, eh, eg, gelu, slope = parts(x, w, b)
    d, u, T, F2 = dy.double(), HALF_STEP[dtype], x.shape[0], w.shape[0]
    eG, eS = 1.13 * eg + g.abs() * 6e-7, 0.8 * eg + (1 + g.abs()) * 6e-7
    P = torch.cat([d * gelu, d * h * slope], 1)
    eP = torch.cat([d.abs() * eG, d.abs() * (h.abs() * eS + slope.abs() * eh)], 1)
    eR = eP + u * P.abs() + SUB[dtype]
    W, X = w.double(), x.double()
    dx, dw, db = got
    within(dx, P @ W, eR @ W.abs() + (F2 + 64) * E32 * (P.abs() @ W.abs()) + u * (P @ W).abs() + SUB[dtype], f"dx {what}")
    ref = P.T @ X
    within(dw, ref, eR.T @ X.abs() + (T + 64) * E32 * (P.abs().T @ X.abs()) + u * ref.abs() + SUB[dtype], f"dw {what}")
    if b is None:
        assert db is None
    else:
        within(db, P.sum(0), eP.sum(0) + (T + 64) * E32 * P.abs().sum(0), f"db {what}")


# one row; rows and columns below, at and past a tile; the smallest widths;
# contractions of one partial step and of many; the UNet's widths
SHAPES = [(1, 8, 8), (1, 320, 1280), (3, 40, 24), (127, 64, 128), (128, 128, 128), (129, 72, 136), (200, 320, 1280),
          (77, 768, 264), (300, 1280, 640), (64, 1280, 5120), (2048, 64, 96), (4097, 320, 320), (8192, 320, 1280),
          (513, 648, 2560), (1500, 8, 2048), (5000, 136, 8)]


@pytest.mark.parametrize("dtype", list(HALF_STEP))
@pytest.mark.parametrize("T,C,F", SHAPES)
def test_forward_and_backward(T, C, F, dtype):
    x, w, b, dy = make(T + 7 * C + F, T, C, F, dtype)
    check_forward(x, w, b, sd.gated_ff(x, w, b), dtype)
    got = sd.gated_ff_backward(dy, x, w, b)
    check_backward(x, w, b, dy, got, dtype)
    for a, c in zip(got, sd.gated_ff_backward(dy, x, w, b)):
        assert torch.equal(a, c)            # fixed order of every sum


@pytest.mark.parametrize("dtype", list(HALF_STEP))
def test_without_bias_and_with_leading_dimensions(dtype):
    x, w, _, dy = make(3, 2 * 33, 64, 72, dtype, bias=False)
    y = sd.gated_ff(x.view(2, 33, 64), w)
    assert y.shape == (2, 33, 72)
    check_forward(x, w, None, y.view(66, 72), dtype)
    got = sd.gated_ff_backward(dy.view(2, 33, 72), x.view(2, 33, 64), w)
    check_backward(x, w, None, dy, (got[0].view(66, 64), got[1], got[2]), dtype)


def test_agrees_with_the_separate_passes():
    """The same result as the projection followed by `geglu`, within the
    rounding of the stored projection that the fused form does not make."""
    x, w, b, _ = make(9, 500, 320, 640, torch.float16)
    p = (x.float() @ w.float().T + b).half()
    sep = sd.geglu(p).double()
    h, g, _, _, gelu, slope = parts(x, w, b)
    u = HALF_STEP[torch.float16]
    err = (sd.gated_ff(x, w, b).double() - sep).abs()
    assert bool((err <= u * (3.2 * (h * gelu).abs() + (h * slope * g).abs()) + 1e-4 * u * h.abs() + 1e-5).all())


def test_rows_past_the_end_and_neighbouring_memory():
    """Outputs inside a larger buffer: nothing outside them is written."""
    T, C, F = 131, 72, 136
    x, w, b, _ = make(17, T, C, F, torch.bfloat16)
    big = torch.full((T * F + 4096,), 3.0, dtype=torch.bfloat16, device=DEV)
    y = big[1024:1024 + T * F].view(T, F)
    sd.gated_ff(x, w, b, out=y)
    check_forward(x, w, b, y, torch.bfloat16)
    assert bool((big[:1024] == 3).all()) and bool((big[1024 + T * F:] == 3).all())


def test_not_finite_values_stay_in_their_row():
    x, w, b, dy = make(23, 300, 64, 256, torch.float16)
    clean, grads = sd.gated_ff(x, w, b), sd.gated_ff_backward(dy, x, w, b)
    x2 = x.clone()
    x2[140, 3] = float("nan")
    y = sd.gated_ff(x2, w, b)
    keep = torch.arange(300, device=DEV) != 140
    assert torch.equal(y[keep], clean[keep]) and torch.isnan(y[140]).all()
    dx = sd.gated_ff_backward(dy, x2, w, b)[0]
    assert torch.equal(dx[keep], grads[0][keep])


def test_infinite_bias_of_rows_that_do_not_exist():
    """A tile's rows past T see the bias alone; an infinite one must not reach the sums."""
    x, w, b, dy = make(29, 5, 64, 128, torch.bfloat16)
    b = b.clone()
    b[128 + 7] = float("inf")               # gate of column 7: GELU = inf, its slope NaN
    db = sd.gated_ff_backward(dy, x, w, b)[2]
    ok = torch.ones(256, dtype=torch.bool, device=DEV)
    ok[[7, 128 + 7]] = False
    b0 = b.clone()
    b0[128 + 7] = 0
    assert torch.equal(db[ok], sd.gated_ff_backward(dy, x, w, b0)[2][ok])


def test_no_rows():
    _, w, b, _ = make(1, 1, 64, 72, torch.float16)
    x, dy = torch.empty(0, 64, dtype=torch.float16, device=DEV), torch.empty(0, 72, dtype=torch.float16, device=DEV)
    assert sd.gated_ff(x, w, b).shape == (0, 72)
    dx, dw, db = sd.gated_ff_backward(dy, x, w, b)
    assert dx.shape == (0, 64) and not dw.any() and not db.any() and db.shape == (144,)


def test_gradient_against_differences():
    """Directional central differences of the fp64 definition, on inputs exact in fp16."""
    import numpy as np
    x, w, b, dy = make(31, 12, 16, 24, torch.float16)
    got = [t.double().cpu().numpy() for t in sd.gated_ff_backward(dy, x, w, b)]
    at = [t.double().cpu().numpy() for t in (x, w, b)]
    d = dy.double().cpu().numpy()
    f = lambda v: float((unet_ops.geglu(v[0] @ v[1].T + v[2]) * d).sum())   # noqa: E731
    rng, step = np.random.default_rng(1), 1e-5
    for k in range(3):
        v = rng.normal(size=at[k].shape)
        num = (f([a + step * v if i == k else a for i, a in enumerate(at)])
               - f([a - step * v if i == k else a for i, a in enumerate(at)])) / (2 * step)
        # two roundings to fp16 (P, the output): 2 * 2^-11 of the terms' magnitude; db has none
        assert abs(num - float((got[k] * v).sum())) <= (2 ** -10 if k < 2 else 1e-5) * np.abs(got[k] * v).sum() + 1e-4


def test_two_streams_at_once_and_captured():
    x, w, b, dy = make(37, 700, 320, 640, torch.bfloat16)
    want = (sd.gated_ff(x, w, b),) + sd.gated_ff_backward(dy, x, w, b)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append((sd.gated_ff(x, w, b),) + sd.gated_ff_backward(dy, x, w, b))
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(a, c) for a, c in zip(r, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = (sd.gated_ff(x, w, b),) + sd.gated_ff_backward(dy, x, w, b)
    for t in held:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(held, want))


def test_refusals():
    x, w, b, dy = make(41, 16, 64, 72, torch.float16)
    with pytest.raises(TypeError):
        sd.gated_ff(x.float(), w.float(), b)
    with pytest.raises(ValueError):
        sd.gated_ff(x, w.bfloat16(), b)
    with pytest.raises(ValueError):
        sd.gated_ff(x, w[:, :56], b)
    with pytest.raises(ValueError):
        sd.gated_ff(x, w, b[:72])
    with pytest.raises(ValueError):
        sd.gated_ff(x, w.cpu(), b)
    with pytest.raises(sd.SdattnError):
        sd.gated_ff(x[:, :60], w[:, :60], b)          # C not a multiple of 8
    with pytest.raises(sd.SdattnError):
        sd.gated_ff(x, w[:140], b[:140])              # F = 70
    with pytest.raises(ValueError):
        sd.gated_ff_backward(dy[:8], x, w, b)
    odd = torch.zeros(16 * 64 + 1, dtype=torch.float16, device=DEV)[1:].view(16, 64)
    with pytest.raises(sd.SdattnError):
        sd.gated_ff(odd, w, b)                        # not on a 16-byte boundary


def test_no_device_error_after_gated_ff():
    status, detail = sd.device_error()
    assert status == "SDATTN_OK", (status, hex(detail))


def test_gates_of_every_size():
    """One row per gate, h = 1: infinities, not-a-numbers, far tails and zeros."""
    vals = [float("inf"), float("nan"), 100.0, 30.0, 8.0, 5.6, 3.0, 1.0, 1e-20, 0.0, -1e-20, -1.0, -3.0, -5.6, -8.0, -30.0]
    x = torch.eye(16, dtype=torch.float16, device=DEV)
    w = torch.zeros(32, 16, dtype=torch.float16, device=DEV)
    b = torch.cat([torch.ones(16), torch.tensor(vals)]).to(DEV)
    y = sd.gated_ff(x, w, b)[0].double()
    assert torch.isinf(y[0]) and torch.isnan(y[1])
    g = torch.tensor(vals[2:], dtype=torch.float64, device=DEV)
    ref = g * 0.5 * torch.erfc(-g / 2 ** 0.5)
    u = HALF_STEP[torch.float16]
    assert bool(((y[2:] - ref).abs() <= u * ref.abs() + 1.2e-7 + SUB[torch.float16]).all())


@pytest.mark.parametrize("dtype", list(HALF_STEP))
@pytest.mark.parametrize("T,C,F", [(500, 1280, 5048), (8300, 320, 1240)])
def test_more_tiles_than_pairs(T, C, F, dtype):
    """A few tiles of CTA pairs behind the last full wave, the last column tile narrow."""
    x, w, b, dy = make(T + 7 * C + F, T, C, F, dtype)
    check_forward(x, w, b, sd.gated_ff(x, w, b), dtype)
    got = sd.gated_ff_backward(dy, x, w, b)
    check_backward(x, w, b, dy, got, dtype)
    assert all(torch.equal(p, q) for p, q in zip(got, sd.gated_ff_backward(dy, x, w, b)))


def test_pairs_back_to_back():
    """Short launches of CTA pairs, one after the other and mixed with single
    CTAs whose barriers lie elsewhere in shared memory: every CTA must have all
    that arrives in its memory behind it when it leaves.  An arrival that came
    late would complete a phase of a later kernel's barrier."""
    a = make(43, 8192, 320, 1280, torch.float16)
    b = make(44, 77, 128, 72, torch.bfloat16)
    calls = [lambda: (sd.gated_ff(*a[:3]),), lambda: sd.gated_ff_backward(a[3], *a[:3]),
             lambda: (sd.gated_ff(*b[:3]),), lambda: (sd.adapter_linear(a[0], a[1], a[2]),),
             lambda: sd.gated_ff_backward(b[3], *b[:3])]
    want = [[t.clone() for t in f()] for f in calls]
    check_forward(*a[:3], want[0][0], torch.float16)
    check_backward(*a, want[1], torch.float16)
    for turn in range(100):
        got = [f() for f in calls]
        if turn % 20 == 19:
            for g, w in zip(got, want):
                assert all(torch.equal(p, q) for p, q in zip(g, w)), turn
    status, detail = sd.device_error()
    assert status == "SDATTN_OK", (status, hex(detail))


@pytest.mark.parametrize("dtype", list(HALF_STEP))
def test_a_gate_of_minus_infinity(dtype):
    """The formula gives not-a-number there, and so does `geglu`; gates far
    below zero give zero, the largest finite ones themselves."""
    x = torch.eye(16, dtype=dtype, device=DEV)
    w = torch.zeros(32, 16, dtype=dtype, device=DEV)
    gates = torch.full((16,), 1.0)
    gates[:6] = torch.tensor([float("-inf"), float("inf"), 3e38, -20.0, -1e4, -3e38])
    b = torch.cat([torch.ones(16), gates]).to(DEV)
    y = sd.gated_ff(x, w, b)
    assert torch.isnan(sd.geglu(b.to(dtype)[None])[0, 0])
    assert torch.isnan(y[:, 0]).all() and (y[:, 1] == float("inf")).all()
    assert torch.equal(y[:, 2], torch.full((16,), 3e38, device=DEV).to(dtype))
    assert (y[:, 3:6].abs() <= 1e-13).all()
    db = sd.gated_ff_backward(torch.full_like(x, 1 / 16), x, w, b)[2]      # sums of 16 equal rows
    assert torch.isnan(db[0]) and torch.isnan(db[16]) and not db[3:6].any() and not db[19:22].any()
    assert db[1] == float("inf") and torch.isfinite(db[2:16]).all() and torch.isfinite(db[18:]).all()
