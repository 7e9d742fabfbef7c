"""GPU parity of the projection with low-rank adapters against fp64.

Bound per output, to first order, u half a step of the element type (2^-11
fp16, 2^-8 bf16), e = 2^-23 (an fp32 step, which also covers sums that
truncate), sums of n terms erring by at most (n + 64) e of the magnitudes:

  z = s x D^T     ez = s (C + 64) e (|x| |D|^T);  rounded once: + u |z| (+ half a subnormal step, fp16)
  y               (C + 64) e (|x| |W|^T + |bias|) + ez_rounded |U|^T + (R + 64) e |z| |U|^T + u |y|
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import diffusion_unet_attention_b200 as sd  # noqa: E402

DEV = torch.device("cuda:0")
HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
SUB = {torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}
E32 = 2.0 ** -23


def make(seed, G, N, C, K, R, L, dtype, bias=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(G, N, C, generator=g).to(dtype).to(DEV)
    w = (torch.randn(K, C, generator=g) / C ** 0.5).to(dtype).to(DEV)
    b = (0.2 * torch.randn(K, generator=g)).to(DEV) if bias else None
    down = (torch.randn(L, R, C, generator=g) / C ** 0.5).to(dtype).to(DEV)
    up = (torch.randn(L, K, R, generator=g) / R ** 0.5).to(dtype).to(DEV)
    scale = (0.25 + torch.rand(L, generator=g)).to(DEV)
    ids = torch.randint(-1, L, (G,), generator=g, dtype=torch.int32).to(DEV)
    return x, w, b, down, up, scale, ids


def check(y, x, w, b, down, up, scale, ids, dtype, what=""):
    X, W, u = x.double(), w.double(), HALF_STEP[dtype]
    C = X.shape[-1]
    ref, bnd = X @ W.T, (C + 64) * E32 * (X.abs() @ W.abs().T)
    if b is not None:
        ref, bnd = ref + b.double(), bnd + (C + 64) * E32 * b.double().abs()
    for r, i in enumerate(ids.tolist()):
        if not 0 <= i < down.shape[0]:
            continue
        D, U, s = down[i].double(), up[i].double(), 1.0 if scale is None else float(scale[i])
        z = s * (X[r] @ D.T)
        ez = s * (C + 64) * E32 * (X[r].abs() @ D.abs().T) + u * z.abs() + SUB[dtype]
        ref[r] += z @ U.T
        bnd[r] += ez @ U.abs().T + (D.shape[0] + 64) * E32 * (z.abs() @ U.abs().T)
    bnd += u * ref.abs() + SUB[dtype]
    err = (y.double() - ref).abs()
    assert y.shape == ref.shape and torch.isfinite(y).all(), what
    assert bool((err <= bnd + 1e-30).all()), f"{what}: off by {float((err / (bnd + 1e-30)).max()):.2f} of its bound"


# G requests of N rows: one of one, one row each (many adapters a tile, some
# tiles with more than a phase holds), requests that straddle tiles, tiles of
# one request, odd widths, every slot size, ranks of several slots
SHAPES = [(1, 1, 8, 8, 8, 1), (1, 1, 320, 320, 16, 3), (48, 1, 1280, 1280, 32, 12), (300, 1, 64, 136, 8, 200),
          (130, 1, 128, 64, 128, 140), (2, 77, 768, 320, 8, 2), (5, 77, 320, 640, 24, 4), (3, 129, 72, 200, 40, 2),
          (2, 4096, 320, 320, 16, 2), (16, 64, 1280, 1280, 64, 8), (7, 50, 136, 72, 72, 5), (4, 300, 64, 2560, 256, 3),
          (40, 9, 200, 48, 48, 17)]


@pytest.mark.parametrize("dtype", list(HALF_STEP))
@pytest.mark.parametrize("G,N,C,K,R,L", SHAPES)
def test_parity(G, N, C, K, R, L, dtype):
    a = make(G + 3 * N + C + K + R, G, N, C, K, R, L, dtype)
    y = sd.adapter_linear(*a)
    check(y, *a, dtype)
    assert torch.equal(y, sd.adapter_linear(*a))


@pytest.mark.parametrize("dtype", list(HALF_STEP))
@pytest.mark.parametrize("T,C,K", [(1, 8, 8), (154, 768, 320), (1000, 320, 1280), (129, 1280, 72)])
def test_plain_projection(T, C, K, dtype):
    x, w, b = make(T + C, T, 1, C, K, 8, 1, dtype)[:3]
    ids = torch.full((T,), -1, dtype=torch.int32)
    zero = torch.zeros(1, 8, C, dtype=dtype, device=DEV), torch.zeros(1, K, 8, dtype=dtype, device=DEV)
    y = sd.adapter_linear(x, w, b)
    check(y, x, w, b, *zero, None, ids, dtype)
    # no request with an adapter, and no adapters at all, are the same call
    assert torch.equal(y, sd.adapter_linear(x, w, b, *zero, None, ids.to(DEV)))
    assert torch.equal(y[:, 0], sd.adapter_linear(x[:, 0], w, b))
    assert torch.equal(y, sd.adapter_linear(x, w, b, zero[0][:0], zero[1][:0], None, ids.to(DEV)))


def test_ids_outside_the_adapters_take_the_projection_alone():
    x, w, b, down, up, scale, ids = make(3, 6, 40, 64, 72, 16, 3, torch.float16)
    ids = torch.tensor([0, 3, -1, 2147483647, -2147483648, 2], dtype=torch.int32, device=DEV)
    y = sd.adapter_linear(x, w, b, down, up, scale, ids)
    check(y, x, w, b, down, up, scale, ids, torch.float16)


def test_rows_of_ragged_requests():
    """Requests of 1, 200, 3, 77 and 128 rows: one id a row."""
    lens, who = [1, 200, 3, 77, 128], [2, 0, -1, 2, 1]
    T = sum(lens)
    x, w, b, down, up, scale, _ = make(5, T, 1, 320, 320, 16, 3, torch.bfloat16)
    ids = torch.tensor([a for n, a in zip(lens, who) for _ in range(n)], dtype=torch.int32, device=DEV)
    y = sd.adapter_linear(x[:, 0], w, b, down, up, scale, ids)
    check(y[:, None], x, w, b, down, up, scale, ids, torch.bfloat16)


def test_default_scale_and_leading_dimensions():
    x, w, b, down, up, _, ids = make(7, 3, 24, 64, 80, 8, 2, torch.float16)
    y = sd.adapter_linear(x.view(3, 4, 6, 64), w, None, down, up, None, ids)
    assert y.shape == (3, 4, 6, 80)
    check(y.view(3, 24, 80), x, w, None, down, up, None, ids, torch.float16)


def test_a_row_that_is_not_finite_stays_its_own():
    x, w, b, down, up, scale, _ = make(9, 200, 1, 64, 136, 16, 40, torch.float16)
    ids = (torch.arange(200, dtype=torch.int32) % 41 - 1).to(DEV)
    clean = sd.adapter_linear(x, w, b, down, up, scale, ids)
    x2 = x.clone()
    x2[77, 0, 5], x2[131, 0, 0] = float("inf"), float("nan")
    y = sd.adapter_linear(x2, w, b, down, up, scale, ids)
    keep = torch.ones(200, dtype=torch.bool, device=DEV)
    keep[[77, 131]] = False
    assert torch.equal(y[keep], clean[keep]) and torch.isnan(y[131]).all()


def test_an_adapter_that_is_not_finite_stays_with_its_requests():
    x, w, b, down, up, scale, _ = make(11, 10, 30, 64, 72, 16, 4, torch.bfloat16)
    ids = torch.tensor([0, 1, 2, 3, -1, 0, 1, 2, 3, -1], dtype=torch.int32, device=DEV)
    clean = sd.adapter_linear(x, w, b, down, up, scale, ids)
    down2 = down.clone()
    down2[2, 1] = float("nan")
    y = sd.adapter_linear(x, w, b, down2, up, scale, ids)
    keep = ids != 2
    assert torch.equal(y[keep], clean[keep]) and torch.isnan(y[2]).all()


def test_nothing_outside_the_output_is_written():
    G, N, C, K = 3, 43, 72, 136
    x, w, b, down, up, scale, ids = make(13, G, N, C, K, 8, 2, torch.float16)
    big = torch.full((G * N * K + 4096,), 3.0, dtype=torch.float16, device=DEV)
    y = big[1024:1024 + G * N * K].view(G, N, K)
    sd.adapter_linear(x, w, b, down, up, scale, ids, out=y)
    check(y, x, w, b, down, up, scale, ids, torch.float16)
    assert bool((big[:1024] == 3).all()) and bool((big[1024 + G * N * K:] == 3).all())


def test_captured_with_other_requests_on_replay():
    """A captured call reads ids, scale and adapters anew on every replay."""
    x, w, b, down, up, scale, ids = make(17, 8, 64, 320, 320, 16, 5, torch.float16)
    sd.adapter_linear(x, w, b, down, up, scale, ids)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = sd.adapter_linear(x, w, b, down, up, scale, ids)
    for turn in range(3):
        ids.copy_(torch.tensor([(turn + k) % 6 - 1 for k in range(8)], dtype=torch.int32))
        scale.mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        check(y, x, w, b, down, up, scale, ids, torch.float16)


def test_no_requests():
    x, w, b, down, up, scale, ids = make(19, 2, 4, 64, 72, 8, 2, torch.float16)
    assert sd.adapter_linear(x[:0], w, b, down, up, scale, ids[:0]).shape == (0, 4, 72)
    assert sd.adapter_linear(x[:, :0], w, b, down, up, scale, ids).shape == (2, 0, 72)


def test_refusals():
    x, w, b, down, up, scale, ids = make(23, 4, 8, 64, 72, 8, 2, torch.float16)
    for bad in [dict(ids=ids.long()), dict(ids=ids[:3]), dict(ids=ids.cpu()), dict(up=up[:, :64]), dict(down=down.bfloat16()),
                dict(down=None), dict(w=w.bfloat16()), dict(scale=scale[:1]), dict(ids=None), dict(bias=b[:64])]:
        kw = dict(w=w, bias=b, down=down, up=up, scale=scale, ids=ids)
        kw.update(bad)
        with pytest.raises(ValueError):
            sd.adapter_linear(x, **kw)
    with pytest.raises(TypeError):
        sd.adapter_linear(x.float(), w.float(), b)
    with pytest.raises(sd.SdattnError):
        sd.adapter_linear(x, w, b, down[:, :4], up[:, :, :4], scale, ids)      # rank 4, not padded
    with pytest.raises(sd.SdattnError):
        sd.adapter_linear(x, w[:70], b[:70])                                    # K = 70


def test_no_device_error_after_adapters():
    status, detail = sd.device_error()
    assert status == "SDATTN_OK", (status, hex(detail))


def test_few_rows_without_an_adapter_among_them():
    """The per-row form (fewer than 16 rows a request) where some or all requests have none."""
    x, w, b, down, up, scale, _ = make(29, 70, 3, 128, 200, 40, 6, torch.float16)
    for ids in (torch.full((70,), -1), torch.arange(70) % 8 - 1):
        ids = ids.to(torch.int32).to(DEV)
        y = sd.adapter_linear(x, w, b, down, up, scale, ids)
        check(y, x, w, b, down, up, scale, ids, torch.float16)


def test_many_adapters_in_a_tile_of_long_requests():
    """Requests of 16 rows, eight adapters a tile, ranks that fill a phase
    each: tiles of an even and an odd number of phases, one after the other."""
    for R, L in ((64, 8), (64, 3), (16, 8), (200, 5)):
        x, w, b, down, up, scale, _ = make(31 + R + L, 600, 16, 64, 200, R, L, torch.bfloat16)
        ids = (torch.randint(-1, L, (600,), generator=torch.Generator().manual_seed(R)).to(torch.int32)).to(DEV)
        y = sd.adapter_linear(x, w, b, down, up, scale, ids)
        check(y, x, w, b, down, up, scale, ids, torch.bfloat16)


def test_two_streams_at_once():
    a = make(37, 48, 1, 320, 640, 32, 12, torch.float16)
    want = sd.adapter_linear(*a)
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append([sd.adapter_linear(*a) for _ in range(3)])
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for ys in got for y in ys)


@pytest.mark.parametrize("dtype", list(HALF_STEP))
@pytest.mark.parametrize("R", [8, 16, 72])
def test_up_matrices_that_are_not_finite_stay_with_their_requests(R, dtype):
    """Several requests a tile, one of whose U holds infinities and NaN."""
    x, w, b, down, up, scale, _ = make(41 + R, 12, 30, 64, 136, R, 4, dtype)
    ids = torch.tensor([0, 1, 2, 3, -1, 0, 1, 2, 3, -1, 2, 1], dtype=torch.int32, device=DEV)
    clean = sd.adapter_linear(x, w, b, down, up, scale, ids)
    up2 = up.clone()
    up2[2, :, 1], up2[2, 5, 3] = float("inf"), float("nan")
    y = sd.adapter_linear(x, w, b, down, up2, scale, ids)
    assert torch.equal(y[ids != 2], clean[ids != 2])
    assert not torch.isfinite(y[ids == 2]).any() and torch.isnan(y[ids == 2][..., 5]).all()


def test_an_infinite_product_is_infinite_whatever_the_padding():
    """Rank 8 fills half a slot: its other half must not turn an infinity into NaN."""
    x, w, _, down, up, _, _ = make(43, 4, 40, 64, 72, 8, 2, torch.float16)
    x, w, down, up = x.abs() + 1, w.abs() + 0.5, down.abs() + 0.5, up.abs() + 0.5
    x[1, 7, 3] = float("inf")
    ids = torch.tensor([0, 1, 0, -1], dtype=torch.int32, device=DEV)
    y = sd.adapter_linear(x, w, None, down, up, None, ids)
    assert torch.isinf(y[1, 7]).all() and torch.isfinite(y[0]).all() and torch.isfinite(y[1, :7]).all()


def workspace(G, N, C, K, R, L):
    from ctypes import byref
    from diffusion_unet_attention_b200 import _lib
    return sd.load_library().sdattn_adapter_linear_workspace_bytes(byref(_lib.AdapterDesc(G * N, C, K, L, R, N, 0)))


@pytest.mark.parametrize("dtype", list(HALF_STEP))
@pytest.mark.parametrize("G,N,C,K,R,L", [(4096, 1, 320, 320, 72, 160), (1300, 3, 72, 136, 72, 300), (256, 4, 640, 640, 128, 256),
                                         (4000, 2, 72, 136, 200, 90), (7, 16, 320, 328, 256, 7)])
def test_many_adapters_a_tile_in_one_launch(G, N, C, K, R, L, dtype):
    """Short requests in the one-launch form: up to 128 adapters in a tile of
    128 rows, each of several slots; a tile of fewer rows too (7 x 16)."""
    assert workspace(G, N, C, K, R, L) == 0
    x, w, b, down, up, scale, _ = make(G + R, G, N, C, K, R, L, dtype)
    ids = ((torch.arange(G) * 37) % (L + 1) - 1).to(torch.int32).to(DEV)      # all different in a tile
    y = sd.adapter_linear(x, w, b, down, up, scale, ids)
    check(y, x, w, b, down, up, scale, ids, dtype)
    assert torch.equal(y, sd.adapter_linear(x, w, b, down, up, scale, ids))


@pytest.mark.parametrize("G,N,C,K,R,L", [(64, 1, 1600, 2560, 128, 32), (64, 1, 1560, 2520, 128, 32), (300, 1, 1280, 1280, 64, 200)])
def test_per_row_form_of_wide_adapters(G, N, C, K, R, L):
    assert workspace(G, N, C, K, R, L) == G * N * R * 4
    a = make(G + R, G, N, C, K, R, L, torch.float16)
    check(sd.adapter_linear(*a), *a, torch.float16)


@pytest.mark.parametrize("dtype", list(HALF_STEP))
@pytest.mark.parametrize("G,N,C,K,R,L", [(2, 77, 768, 320, 8, 2), (16, 64, 320, 320, 16, 8), (9, 40, 128, 136, 40, 4),
                                         (5, 64, 320, 328, 72, 3), (3, 300, 64, 200, 256, 2)])
def test_the_low_rank_product_is_held_in_two_parts(G, N, C, K, R, L, dtype):
    """Where the shared projection is zero y is z U^T alone, and sums that
    cancel show z's own rounding: 2^-13 (bf16) or 2^-19 (fp16, and half a
    subnormal step) of |z| |U|^T beside the fp32 sums' and y's own half step."""
    x, w, _, down, up, scale, ids = make(53 + R, G, N, C, K, R, L, dtype)
    ids = (torch.arange(G, device=DEV, dtype=torch.int32)) % L
    up[:, :, R // 2:] = -up[:, :, :R // 2]                  # pairs of ranks whose products nearly cancel
    down[:, R // 2:] = down[:, :R // 2]
    down[:, 0] *= 1.5
    y = sd.adapter_linear(x, torch.zeros_like(w), None, down, up, scale, ids).double()
    part = {torch.float16: 2.0 ** -19, torch.bfloat16: 2.0 ** -13}[dtype]
    for g, i in enumerate(ids.tolist()):
        X, D, U, s = x[g].double(), down[i].double(), up[i].double(), float(scale[i])
        z = s * (X @ D.T)
        ez = s * (C + 64) * E32 * (X.abs() @ D.abs().T) + part * z.abs() + SUB[dtype]
        ref = z @ U.T
        bnd = ez @ U.abs().T + (2 * R + 64) * E32 * (z.abs() @ U.abs().T) + HALF_STEP[dtype] * ref.abs() + SUB[dtype]
        assert bool(((y[g] - ref).abs() <= bnd).all()), f"off by {float(((y[g] - ref).abs() / bnd).max()):.2f} of its bound"


@pytest.mark.parametrize("dtype", list(HALF_STEP))
def test_an_infinite_up_matrix_gives_infinity(dtype):
    """z of few bits (exact in one part) and of many, times one infinity."""
    x, w, _, down, up, _, _ = make(59, 2, 40, 64, 72, 16, 1, dtype)
    x[0] = 0
    x[0, :, 0], down[0] = 2.0, down[0].abs() + 0.25
    down[0, :, 0] = 0.5                                     # request 0: z = 1 in every rank
    x[1] = x[1].abs() + 0.5
    up[0, 3, 5], up[0, 7, 2] = float("inf"), float("-inf")
    y = sd.adapter_linear(x, w, None, down, up, None, torch.zeros(2, dtype=torch.int32, device=DEV))
    assert (y[..., 3] == float("inf")).all() and (y[..., 7] == float("-inf")).all()
    rest = [k for k in range(72) if k not in (3, 7)]
    assert torch.isfinite(y[..., rest]).all()
