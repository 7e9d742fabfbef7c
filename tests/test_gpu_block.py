"""The UNet's transformer block out of the library's calls, as it is used:

    x1 = x + O(attention(Q, K, V of LN1(x)))        Q, K, V, O: projections with
    y  = x1 + W2 gated_ff(LN2(x1))                  each request's own adapter

against the same block in fp64 on the same 16-bit inputs, and the gradients of
its feed-forward half against autograd in fp64.

Tolerances (relative Frobenius norm).  Every stored 16-bit tensor errs by at
most u (2^-11 fp16, 2^-8 bf16) of its values, and the operators between them
pass a relative error on with a gain of about 1 (norms, projections with
orthogonal-like weights, attention averages) on these inputs.  On the longest
path LN1, z, V, attention's P and O, z, O, x1, LN2, gated_ff, W2 and y are
rounded: 12 roundings, so 12 u if every one were at its worst and of one sign.
The gradients pass 5 (the block's dy times W2, P, dx of the gate, its norm's dx,
and the inputs LN and x1 they are taken at); sums of the weight's gradients are
fp32 of operands with those errors.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import diffusion_unet_attention_b200 as sd  # noqa: E402

DEV = torch.device("cuda:0")
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
HEADS = 8


def weights(seed, C, dtype, L, R):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)      # noqa: E731
    p = {k: (n(C, C) / C ** 0.5).to(dtype).to(DEV) for k in "qkvo"}
    p["w1"], p["b1"] = (n(8 * C, C) / C ** 0.5).to(dtype).to(DEV), (0.1 * n(8 * C)).to(DEV)
    p["w2"], p["b2"] = (n(C, 4 * C) / (4 * C) ** 0.5).to(dtype).to(DEV), (0.1 * n(C)).to(DEV)
    for k in ("g1", "g2"):
        p[k] = (1 + 0.1 * n(C)).to(DEV)
    for k in ("e1", "e2"):
        p[k] = (0.1 * n(C)).to(DEV)
    for k in "qkvo":
        p["d" + k] = (n(L, R, C) / C ** 0.5).to(dtype).to(DEV)
        p["u" + k] = (0.5 * n(L, C, R) / R ** 0.5).to(dtype).to(DEV)
    p["s"] = torch.linspace(0.5, 1.0, L).to(DEV)
    return p


def block(x, p, ids):
    B, N, C = x.shape
    d = C // HEADS
    h = sd.layer_norm(x, p["g1"], p["e1"])
    q, k, v = (sd.adapter_linear(h, p[c], None, p["d" + c], p["u" + c], p["s"], ids)
               .view(B, N, HEADS, d).transpose(1, 2) for c in "qkv")
    a = sd.flash(q, k, v).transpose(1, 2).reshape(B, N, C)
    x1 = x + sd.adapter_linear(a, p["o"], None, p["do"], p["uo"], p["s"], ids)
    y = sd.gated_ff(sd.layer_norm(x1, p["g2"], p["e2"]), p["w1"], p["b1"])
    return x1 + sd.adapter_linear(y, p["w2"], p["b2"])


def ln64(x, g, e):
    m = x.mean(-1, keepdim=True)
    return (x - m) / torch.sqrt(((x - m) ** 2).mean(-1, keepdim=True) + 1e-5) * g + e


def ff64(h, w1, b1):
    t = h @ w1.T + b1
    a, g = t.chunk(2, -1)
    return a * g * 0.5 * torch.erfc(-g / math.sqrt(2))


def block64(x, p, ids):
    p = {k: v.double() for k, v in p.items()}
    x = x.double()
    B, N, C = x.shape
    d = C // HEADS

    def proj(h, c):
        y = h @ p[c].T
        z = torch.stack([h[i] @ p["d" + c][a].T @ p["u" + c][a].T * p["s"][a] if a >= 0 else torch.zeros_like(h[i])
                         for i, a in enumerate(ids.tolist())])
        return y + z

    h = ln64(x, p["g1"], p["e1"])
    q, k, v = (proj(h, c).view(B, N, HEADS, d).transpose(1, 2) for c in "qkv")
    a = (torch.softmax(q @ k.transpose(-1, -2) / math.sqrt(d), -1) @ v).transpose(1, 2).reshape(B, N, C)
    x1 = x + proj(a, "o")
    return x1 + ff64(ln64(x1, p["g2"], p["e2"]), p["w1"], p["b1"]) @ p["w2"].T + p["b2"]


def frob(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("dtype", list(U))
@pytest.mark.parametrize("B,N,C", [(3, 256, 320), (2, 77, 640), (1, 1, 320)])
def test_block(B, N, C, dtype):
    p = weights(B + N + C, C, dtype, 2, 16)
    x = torch.randn(B, N, C, generator=torch.Generator().manual_seed(N)).to(dtype).to(DEV)
    ids = torch.tensor([1, -1, 0][:B], dtype=torch.int32, device=DEV)
    assert frob(block(x, p, ids), block64(x, p, ids)) <= 12 * U[dtype]


def test_block_captured():
    """The whole block in one CUDA graph, replayed on other inputs and other adapters."""
    C, dtype = 320, torch.float16
    p = weights(5, C, dtype, 3, 8)
    x = torch.randn(2, 256, C).to(dtype).to(DEV)
    ids = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    block(x, p, ids)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block(x, p, ids)
    for turn in range(2):
        x.copy_(torch.randn(2, 256, C).to(dtype))
        ids.copy_(torch.tensor([2, turn - 1], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert frob(y, block64(x, p, ids)) <= 12 * U[dtype]


@pytest.mark.parametrize("dtype", list(U))
@pytest.mark.parametrize("T,C", [(512, 320), (77, 640)])
def test_feed_forward_half_trains(T, C, dtype):
    """One training step's gradients of y = x + W2 gated_ff(LN(x)) from a given dL/dy."""
    p = weights(T + C, C, dtype, 1, 8)
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, C, generator=g).to(dtype).to(DEV)
    dy = (0.1 * torch.randn(T, C, generator=g)).to(dtype).to(DEV)
    h, stats = sd.layer_norm(x, p["g2"], p["e2"], return_stats=True)
    da = sd.adapter_linear(dy, p["w2"].t().contiguous())          # dL/d gated_ff = dy W2
    dh, dw1, db1 = sd.gated_ff_backward(da, h, p["w1"], p["b1"])
    dx, dg, de = sd.layer_norm_backward(dh, x, stats, p["g2"])
    dx = dx + dy
    leaves = [t.double().requires_grad_() for t in (x, p["w1"], p["b1"], p["g2"], p["e2"])]
    y = leaves[0] + ff64(ln64(leaves[0], leaves[3], leaves[4]), leaves[1], leaves[2]) @ p["w2"].double().T
    y.backward(dy.double())
    for got, leaf, name in zip((dx, dw1, db1, dg, de), leaves, ("dx", "dw1", "db1", "dgamma", "dbeta")):
        assert frob(got, leaf.grad) <= 6 * U[dtype], name


def test_no_device_error_after_block():
    status, detail = sd.device_error()
    assert status == "SDATTN_OK", (status, hex(detail))


def test_an_output_over_an_input_is_refused():
    x = torch.randn(40, 64, dtype=torch.float16, device=DEV)
    both = torch.zeros(200, 64, dtype=torch.float16, device=DEV)
    w = both[:64]
    with pytest.raises(ValueError, match="overlap"):
        sd.layer_norm(x, out=x)
    with pytest.raises(ValueError, match="overlap"):
        sd.adapter_linear(x, w, out=x)
    with pytest.raises(ValueError, match="overlap"):
        sd.adapter_linear(x, w, out=both[63:103])
    with pytest.raises(ValueError, match="overlap"):
        sd.gated_ff(x, torch.cat([w, w]), out=x)
    assert sd.adapter_linear(x, w, out=both[64:104]).eq(0).all()


@pytest.mark.parametrize("oracle_fn", ["layer_norm", "geglu", "geglu_backward", "layer_norm_backward"])
def test_smoke_checks_every_output(oracle_fn, monkeypatch):
    """An oracle whose output is off by 1% must fail smoke()."""
    import __graft_entry__ as entry
    from oracle import unet_ops
    right = getattr(unet_ops, oracle_fn)

    def wrong(*a):
        r = right(*a)
        if oracle_fn == "geglu":
            return 1.01 * r
        k = 0 if oracle_fn == "layer_norm" else 1            # y; dw; dgamma
        return tuple(1.01 * t if i == k else t for i, t in enumerate(r))

    entry.smoke()
    monkeypatch.setattr(unet_ops, oracle_fn, wrong)
    with pytest.raises(AssertionError, match="rel_frob"):
        entry.smoke()
