"""Argument checks of the transformer block's operators, decided on the host
before anything is enqueued (the pointers below are never dereferenced), and
what their Python entry points refuse without a GPU."""
import ctypes

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    from diffusion_unet_attention_b200 import _lib, build
    build.build()
    return _lib.load()


OK = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 1)
OFF4 = ctypes.c_void_p((1 << 20) + 4)


def ln(T=64, C=320, dtype=0, eps=1e-5):
    from diffusion_unet_attention_b200 import _lib
    return ctypes.byref(_lib.LNDesc(T, C, dtype, eps))


@pytest.mark.parametrize("kw,status", [(dict(T=-1), 1), (dict(C=0), 1), (dict(eps=-1e-5), 1), (dict(eps=float("nan")), 1),
                                       (dict(dtype=3), 2), (dict(C=8193), 2), (dict(T=1 << 31), 2)])
def test_layer_norm_descriptor(lib, kw, status):
    d = ln(**kw)
    assert lib.sdattn_layer_norm(d, OK, OK, OK, OK, OK, None) == status
    assert lib.sdattn_layer_norm_bwd(d, OK, OK, OK, OK, OK, OK, OK, OK, 1 << 30, None) == status
    assert lib.sdattn_layer_norm_bwd_workspace_bytes(d) == 0


def test_layer_norm_pointers(lib):
    fwd, bwd = lib.sdattn_layer_norm, lib.sdattn_layer_norm_bwd
    assert fwd(None, OK, OK, OK, OK, OK, None) == 1
    assert fwd(ln(), None, OK, OK, OK, OK, None) == 1
    assert fwd(ln(), OK, OK, OK, None, OK, None) == 1
    assert fwd(ln(), ODD, OK, OK, OK, OK, None) == 3
    assert fwd(ln(), OK, ODD, OK, OK, OK, None) == 3
    assert fwd(ln(), OK, OK, OK, OK, OFF4, None) == 3
    assert fwd(ln(T=0), None, None, None, None, None, None) == 0     # nothing to do
    assert lib.sdattn_layer_norm_bwd_workspace_bytes(ln(T=3)) == 0
    need = lib.sdattn_layer_norm_bwd_workspace_bytes(ln())
    assert need >= 2 * 320 * 4
    assert bwd(ln(), OK, OK, OK, None, OK, OK, OK, None, need, None) in (4, 5)      # 5: no device to plan for
    assert bwd(ln(), None, OK, OK, OK, OK, OK, OK, OK, need, None) == 1
    assert bwd(ln(), OK, OK, None, OK, OK, OK, OK, OK, need, None) == 1
    assert bwd(ln(), OK, OK, OK, OK, OK, None, OK, OK, need, None) == 1
    assert bwd(ln(dtype=2), OK, ctypes.c_void_p((1 << 20) + 2), OK, OK, OK, OK, OK, OK, need, None) == 3


def test_python_refuses_cpu_tensors():
    import diffusion_unet_attention_b200 as sd
    x = torch.zeros(4, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        sd.layer_norm(x)
    with pytest.raises(ValueError):
        sd.layer_norm_backward(x, x, torch.zeros(4, 2))


def ff(T=64, C=320, F=1280, dtype=0):
    from diffusion_unet_attention_b200 import _lib
    return ctypes.byref(_lib.FFDesc(T, C, F, dtype))


@pytest.mark.parametrize("kw,status", [(dict(T=-1), 1), (dict(C=0), 1), (dict(F=0), 1), (dict(C=12), 2), (dict(F=20), 2),
                                       (dict(dtype=2), 2), (dict(T=1 << 27), 2), (dict(C=65544), 2)])
def test_gated_ff_descriptor(lib, kw, status):
    d = ff(**kw)
    assert lib.sdattn_gated_ff(d, OK, OK, OK, OK, None) == status
    assert lib.sdattn_gated_ff_bwd(d, OK, OK, OK, OK, OK, OK, OK, OK, 1 << 40, None) == status
    assert lib.sdattn_gated_ff_bwd_workspace_bytes(d) == 0


def test_gated_ff_pointers(lib):
    fwd, bwd = lib.sdattn_gated_ff, lib.sdattn_gated_ff_bwd
    assert fwd(None, OK, OK, OK, OK, None) == 1
    assert fwd(ff(), None, OK, OK, OK, None) == 1
    assert fwd(ff(), OK, OK, OK, None, None) == 1
    for k in range(4):
        args = [OFF4 if i == k else OK for i in range(4)]
        assert fwd(ff(), *args, None) == 3
    assert fwd(ff(T=0), None, None, None, None, None) == 0
    assert lib.sdattn_gated_ff_bwd_workspace_bytes(ff(T=0)) > 0
    need = lib.sdattn_gated_ff_bwd_workspace_bytes(ff())
    assert need >= 64 * 2560 * 2                              # the projection's gradient in 16 bits
    assert bwd(ff(), OK, OK, OK, OK, OK, OK, OK, OK, need - 1, None) == 4
    assert bwd(ff(), OK, OK, OK, OK, OK, OK, OK, None, need, None) == 4
    assert bwd(ff(), OK, OK, OK, OK, None, OK, OK, OK, need, None) == 1
    assert bwd(ff(), OK, OK, OK, OK, OK, None, OK, OK, need, None) == 1
    assert bwd(ff(), OFF4, OK, OK, OK, OK, OK, OK, OK, need, None) == 3
    assert bwd(ff(), OK, OK, OK, OK, OK, OK, ctypes.c_void_p((1 << 20) + 2), OK, need, None) == 3


def ad(T=64, C=320, K=320, L=2, R=16, rows=32, dtype=0):
    from diffusion_unet_attention_b200 import _lib
    return ctypes.byref(_lib.AdapterDesc(T, C, K, L, R, rows, dtype))


@pytest.mark.parametrize("kw,status", [(dict(T=-1), 1), (dict(C=0), 1), (dict(K=0), 1), (dict(L=-1), 1), (dict(rows=0), 1),
                                       (dict(rows=48), 1), (dict(L=0), 1), (dict(R=0), 1), (dict(C=12), 2), (dict(K=20), 2),
                                       (dict(R=4), 2), (dict(R=264), 2), (dict(dtype=2), 2), (dict(T=1 << 27), 2)])
def test_adapter_descriptor(lib, kw, status):
    assert lib.sdattn_adapter_linear(ad(**kw), OK, OK, OK, OK, OK, OK, OK, OK, None, 0, None) == status
    assert lib.sdattn_adapter_linear_workspace_bytes(ad(**kw)) == 0


def test_adapter_pointers(lib):
    def f(d, *ptrs, ws=None, n=0):
        return lib.sdattn_adapter_linear(d, *ptrs, ws, n, None)

    assert f(None, OK, OK, OK, OK, OK, OK, OK, OK) == 1
    for k in (0, 1, 3, 4, 7):                      # X, W, D, U, Y
        assert f(ad(), *[None if i == k else OK for i in range(8)]) == 1
        assert f(ad(), *[OFF4 if i == k else OK for i in range(8)]) == 3
    assert f(ad(), OK, OK, OK, OK, OK, OK, None, OK) == 1              # adapters without ids
    assert f(ad(L=0, R=0), OK, OK, OK, OK, OK, OK, OK, OK) == 1        # ids without adapters
    assert f(ad(), OK, OK, OK, OK, OK, OK, ctypes.c_void_p((1 << 20) + 2), OK) == 3
    assert f(ad(T=0), *[None] * 8) == 0
    # requests of a few rows need a workspace: z [T][R] in fp32
    few = dict(T=48, rows=1, R=32, L=12)
    assert lib.sdattn_adapter_linear_workspace_bytes(ad(T=48, rows=1, R=32)) == 0   # two adapters at most
    assert lib.sdattn_adapter_linear_workspace_bytes(ad(**few)) == 48 * 32 * 4
    assert lib.sdattn_adapter_linear_workspace_bytes(ad()) == 0
    assert f(ad(**few), *[OK] * 8) == 4
    assert f(ad(**few), *[OK] * 8, ws=OK, n=48 * 32 * 4 - 1) == 4
    assert f(ad(**few), *[OK] * 8, ws=OFF4, n=48 * 32 * 4) == 3


def test_adapter_form_follows_its_cost(lib):
    """Single rows with an adapter each take the per-row form (it has a
    workspace) at widths on both sides of 64 MB of adapters read, 35 us as
    against 340; many rows of few ranks that may share adapters do not."""
    ws = lib.sdattn_adapter_linear_workspace_bytes
    for C, K in ((1560, 2520), (1600, 2560)):
        assert ws(ad(T=64, rows=1, C=C, K=K, R=128, L=32)) == 64 * 128 * 4
    assert ws(ad(T=300, rows=1, C=1280, K=1280, R=64, L=200)) == 300 * 64 * 4
    assert ws(ad(T=16384, rows=1, R=8, L=16)) == 0
    assert ws(ad(T=(1 << 27) - 1, rows=1, C=8, K=8, R=256, L=1 << 20)) == 0      # never more than 64 MB
