"""GPU parity of the layer norm and its backward pass against fp64.

Bars, from the arithmetic: the kernels compute in fp32 (unit roundoff 2^-24)
and round y and dx once to the element type (half a step: 2^-11, 2^-8 or
2^-24 of the value).  The fp32 part is a row sum of C terms (error at most C
2^-24 of the sum of magnitudes, in practice about log C steps), so per output

  |y - ref|  <= u |ref| + k 2^-24 (|z gamma| + |beta|) + k 2^-24 r (|x| + |m|) |gamma|

with k = 64 (a lane's chain of at most 40 additions plus the tree over lanes,
for the mean and again for the variance); the last term is the mean's own
error, which matters where |x| is large beside the row's deviation.  The
weight's gradients are sums over rows of fp32 products in a fixed order:
|error| <= (64 + T / 512 rows of one lane's chain) 2^-24 sum_t |term|, where
each term carries the error of its z.
"""
import numpy as np
import pytest

from oracle import unet_ops

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import diffusion_unet_attention_b200 as sd  # noqa: E402

DEV = torch.device("cuda:0")
HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DTYPES = list(HALF_STEP)
E32 = 2.0 ** -24
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 0.0, torch.float32: 0.0}   # half a subnormal step


def make(seed, T, C, dtype, offset=0.5):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, C, generator=g, dtype=torch.float64) * torch.exp(0.5 * torch.randn(T, 1, generator=g, dtype=torch.float64))
         + offset).to(dtype)
    dy = (0.3 * torch.randn(T, C, generator=g, dtype=torch.float64)).to(dtype)
    gamma = 1.0 + 0.2 * torch.randn(C, generator=g)
    beta = 0.2 * torch.randn(C, generator=g)
    return x, dy, gamma, beta


def forward_bound(x, gamma, beta, ref, eps, dtype):
    m = x.mean(-1, keepdims=True)
    r = 1.0 / np.sqrt(((x - m) ** 2).mean(-1, keepdims=True) + eps)
    z = (x - m) * r
    return (HALF_STEP[dtype] * np.abs(ref) + TINY[dtype]
            + 64 * E32 * (np.abs(z * gamma) + np.abs(beta) + r * (np.abs(x) + np.abs(m)) * np.abs(gamma)))


def backward_check(x, dy, stats, gamma, got, dtype, what):
    xs, ds, ss, gs = (t.double().cpu().numpy() for t in (x, dy, stats, gamma))
    dx, dg, db = (t.double().cpu().numpy() for t in got)
    rx, rg, rb = unet_ops.layer_norm_backward(ds, xs, ss, gs)
    T, C = xs.shape
    m, r = ss[:, :1], ss[:, 1:]
    z, e = (xs - m) * r, ds * gs
    ez = E32 * 4 * r * (np.abs(xs) + np.abs(m))                  # error of one z
    scale = np.abs(e) + np.abs(e).mean(-1, keepdims=True) + np.abs(z) * np.abs(e * z).mean(-1, keepdims=True)
    slip = ez * np.abs(e * z).mean(-1, keepdims=True) + np.abs(z) * (np.abs(e) * ez).mean(-1, keepdims=True)
    bnd = HALF_STEP[dtype] * np.abs(rx) + TINY[dtype] + r * (64 * E32 * scale + slip)
    assert np.all(np.abs(dx - rx) <= bnd), f"{what}: dx off by {np.max(np.abs(dx - rx) / bnd):.2f} of its bound"
    k = (64 + T / 512) * E32
    bg = k * np.abs(ds * z).sum(0) + (np.abs(ds) * ez).sum(0)
    bb = k * np.abs(ds).sum(0)
    assert np.all(np.abs(dg - rg) <= bg + 1e-30), f"{what}: dgamma"
    assert np.all(np.abs(db - rb) <= bb + 1e-30), f"{what}: dbeta"


# rows of one value, odd rows, rows at each lane count, at the borders of the
# register plans (32 lanes x 5 accesses, a CTA per row) and the longest
SHAPES = [(1, 1), (3, 2), (5, 7), (1, 8), (77, 33), (8192, 320), (154, 768), (513, 640), (130, 1280), (40, 1288), (9, 641),
          (19, 513), (6, 4095), (3, 8192), (2, 8191), (4800, 72), (5000, 26), (1200, 1000)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,C", SHAPES)
def test_forward_and_backward(T, C, dtype):
    x, dy, gamma, beta = make(T * 31 + C, T, C, dtype)
    eps = 1e-5
    y, stats = sd.layer_norm(x.to(DEV), gamma.to(DEV), beta.to(DEV), eps, return_stats=True)
    xr = x.double().numpy()
    gr, br = gamma.double().numpy(), beta.double().numpy()
    ref, sref = unet_ops.layer_norm(xr, gr, br, eps)
    bnd = forward_bound(xr, gr, br, ref, eps, dtype)
    err = np.abs(y.double().cpu().numpy() - ref)
    assert np.all(err <= bnd), f"y off by {np.max(err / bnd):.2f} of its bound"
    st = stats.double().cpu().numpy()
    assert np.all(np.abs(st[:, 0] - sref[:, 0]) <= 64 * E32 * np.abs(xr).mean(-1) + 1e-30)
    got = sd.layer_norm_backward(dy.to(DEV), x.to(DEV), stats, gamma.to(DEV))
    backward_check(x, dy, stats, gamma, got, dtype, f"{T, C}")
    # no atomics: the same bits again
    again = sd.layer_norm_backward(dy.to(DEV), x.to(DEV), stats, gamma.to(DEV))
    for a, b in zip(got, again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", DTYPES)
def test_without_parameters_and_leading_dimensions(dtype):
    x, dy, _, _ = make(3, 6 * 5, 48, dtype)
    x, dy = x.view(2, 3, 5, 48).to(DEV), dy.view(2, 3, 5, 48).to(DEV)
    y, stats = sd.layer_norm(x, return_stats=True)
    assert y.shape == x.shape and stats.shape == (2, 3, 5, 2)
    one, zero = torch.ones(48, device=DEV), torch.zeros(48, device=DEV)
    assert torch.equal(y, sd.layer_norm(x, one, zero))
    for a, b in zip(sd.layer_norm_backward(dy, x, stats), sd.layer_norm_backward(dy, x, stats, one)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("C", [40, 320, 4096])
def test_unaligned_and_strided_views(dtype, C):
    """A view that starts off a 16-byte boundary and a transposed one give the
    results of their contiguous copies."""
    flat = make(11, 9, C, dtype)[0].reshape(-1).to(DEV)
    odd = torch.empty(flat.numel() + 1, dtype=dtype, device=DEV)[1:]
    odd.copy_(flat)
    want = sd.layer_norm(flat.view(9, C)).double()
    got = sd.layer_norm(odd.view(9, C)).double()
    # another access width adds in another order: a rounding step apart at most
    assert (got - want).abs().max() <= 2 * HALF_STEP[dtype] * want.abs().max() + 64 * E32 * 8
    turned = flat.view(9, C).t().contiguous().t()
    assert torch.equal(sd.layer_norm(turned), sd.layer_norm(flat.view(9, C)))


def test_constant_rows_give_beta():
    """Rows without deviation: z is exactly 0 whatever eps."""
    x = torch.full((5, 320), 7.0, dtype=torch.float16, device=DEV)
    beta = torch.linspace(-1, 1, 320, device=DEV)
    assert torch.equal(sd.layer_norm(x, torch.ones(320, device=DEV), beta), beta.half().expand(5, 320))


def test_no_rows():
    x = torch.empty(0, 320, dtype=torch.float16, device=DEV)
    y, stats = sd.layer_norm(x, return_stats=True)
    assert y.shape == (0, 320) and stats.shape == (0, 2)
    dx, dg, db = sd.layer_norm_backward(x, x, stats)
    assert dx.shape == (0, 320) and not dg.any() and not db.any() and dg.shape == (320,)


def test_not_finite_rows_stay_their_own():
    x, _, gamma, beta = make(21, 12, 320, torch.float16)
    clean = sd.layer_norm(x.to(DEV), gamma.to(DEV), beta.to(DEV))
    x[3, 5], x[7, 0] = float("inf"), float("nan")
    y = sd.layer_norm(x.to(DEV), gamma.to(DEV), beta.to(DEV))
    rows = torch.tensor([i for i in range(12) if i not in (3, 7)], device=DEV)
    assert torch.equal(y[rows], clean[rows])
    assert torch.isnan(y[7]).all() and torch.isnan(y[3]).all()


def test_gradient_against_differences():
    """Central differences of the fp64 definition along random directions:
    the analytic directional derivative agrees to the differences' own error."""
    x, dy, gamma, beta = make(5, 6, 56, torch.float32)
    y, stats = sd.layer_norm(x.to(DEV), gamma.to(DEV), beta.to(DEV), return_stats=True)
    dx, dg, db = (t.double().cpu().numpy() for t in sd.layer_norm_backward(dy.to(DEV), x.to(DEV), stats, gamma.to(DEV)))
    rng = np.random.default_rng(0)
    xs, ds, gs, bs = (t.double().numpy() for t in (x, dy, gamma, beta))
    f = lambda a, b, c: float((unet_ops.layer_norm(a, b, c, 1e-5)[0] * ds).sum())   # noqa: E731
    h = 1e-5
    for which, grad in ((0, dx), (1, dg), (2, db)):
        v = rng.normal(size=(xs, gs, bs)[which].shape)
        at = [[a + (s * h * v if k == which else 0) for k, a in enumerate((xs, gs, bs))] for s in (1, -1)]
        num = (f(*at[0]) - f(*at[1])) / (2 * h)
        # h^2 f''' / 6 is about 1e-9 here, fp32's own error 1e-6 of the terms
        assert abs(num - float((grad * v).sum())) <= 1e-5 * np.abs(grad * v).sum()


def test_captured_and_replayed_with_new_values():
    x, dy, gamma, beta = make(8, 512, 320, torch.bfloat16)
    xd, dd, gd, bd = x.to(DEV), dy.to(DEV), gamma.to(DEV), beta.to(DEV)

    def step():
        y, stats = sd.layer_norm(xd, gd, bd, return_stats=True)
        return (y,) + sd.layer_norm_backward(dd, xd, stats, gd)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    xd.copy_(make(9, 512, 320, torch.bfloat16)[0])
    want = step()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(held, want):
        assert torch.equal(a, b)


def test_refusals():
    x = torch.zeros(4, 320, dtype=torch.float16, device=DEV)
    st = torch.zeros(4, 2, device=DEV)
    with pytest.raises(TypeError):
        sd.layer_norm(x.double())
    with pytest.raises(ValueError):
        sd.layer_norm(x, torch.ones(319, device=DEV))
    with pytest.raises(ValueError):
        sd.layer_norm(x, out=torch.empty(4, 320, device=DEV))
    with pytest.raises(sd.SdattnError):
        sd.layer_norm(torch.zeros(2, 8200, dtype=torch.float16, device=DEV))
    with pytest.raises(sd.SdattnError):
        sd.layer_norm(x, eps=-1.0)
    with pytest.raises(ValueError):
        sd.layer_norm_backward(x.float(), x, st)
    with pytest.raises(ValueError):
        sd.layer_norm_backward(x, x, st[:3])
    with pytest.raises(ValueError):
        sd.layer_norm_backward(x, x, st.cpu())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("C", [77, 1000, 1001, 4095])
def test_constant_rows_of_large_values(dtype, C):
    """z is 0 where no value of a row differs, whatever the mean's rounding."""
    v = torch.tensor([1999.0, 1234.5, 777.7, -1601.3, 3.1], dtype=dtype, device=DEV)
    y, stats = sd.layer_norm(v[:, None].repeat(1, C), return_stats=True)
    # the deviations are a few steps of the value, their mean right to 2^-20 of them, and r at most 317
    assert bool((y.double().abs() <= 317 * 2.0 ** -20 * 64 * E32 * v.double().abs()[:, None]).all())
    assert bool(((stats[:, 0].double() - v.double()).abs() <= 2 * E32 * v.double().abs()).all())


@pytest.mark.parametrize("C", [320, 1000, 1001, 4095])
def test_small_deviations_from_a_large_mean(C):
    """fp32 rows around 1000 with deviations of 0.01.  x - m is exact (both
    within a factor of two), so what errs is the deviations' mean, their squares
    and the product: 64 steps of |d| + mean |d|, not of |x|."""
    x = (1000 + 0.01 * torch.randn(40, C, generator=torch.Generator().manual_seed(C), dtype=torch.float64)).float()
    xs = x.double().numpy()
    ref = unet_ops.layer_norm(xs, np.ones(C), np.zeros(C), 1e-6)[0]
    d = np.abs(xs - xs.mean(-1, keepdims=True))
    r = 1 / np.sqrt((d ** 2).mean(-1, keepdims=True) + 1e-6)
    y = sd.layer_norm(x.to(DEV), eps=1e-6).double().cpu().numpy()
    bnd = E32 * np.abs(ref) + 64 * E32 * (r * (d + d.mean(-1, keepdims=True)) + np.abs(ref))
    assert np.all(np.abs(y - ref) <= bnd), np.max(np.abs(y - ref) / bnd)
