"""The affine MSR epilogue and its gradient against fp64: the formula (torch's autograd on the
definition) and central differences; and a training step's chain with the retention's gradient.

Bars.  fp32 results: max|err|/rms <= 1e-5 (a row's statistics are sums of d_v <= 1024 terms in fp32,
relative error below 1024 * 2^-24 = 6e-5 of the sum of magnitudes in the worst order and about
sqrt(1024) * 2^-24 = 2e-6 in the mean; eps 1e-5 keeps 1/sd below 320 and rows here have sd ~ 1).
bf16 results: the same net of half a step of rounding, 2^-8 of the value.  dweight, dbias: fp32 sums.
"""
import numpy as np
import pytest
import torch

import linear_attention_sequence_chunkwise_b200 as rn
import oracle
import synth_inputs as si
from gpu_util import TOL_BF16, TOL_F32, require_gpu
from serving_util import errors

pytestmark = pytest.mark.gpu
TOL = 1e-5


@pytest.fixture(autouse=True)
def _gpu(cuda_lib):
    require_gpu()


def inputs(tokens, heads, dv, dtype, seed, affine=True):
    y, g, d = (si.randn((tokens, heads, dv), seed + i, dtype) for i in range(3))
    y = (y.float() + 0.5).to(y.dtype)
    w, b = (1.0 + 0.3 * si.randn((heads, dv), seed + 3, "f32"), 0.3 * si.randn((heads, dv), seed + 4, "f32")) if affine \
        else (None, None)
    return y, g, d, w, b


def definition(y, g, w, b, eps):
    y, g = y.double().requires_grad_(), g.double().requires_grad_()
    w = torch.ones(y.shape[1:]) if w is None else w
    b = torch.zeros(y.shape[1:]) if b is None else b
    w, b = w.double().requires_grad_(), b.double().requires_grad_()
    m = y.mean(-1, keepdim=True)
    var = ((y - m) ** 2).mean(-1, keepdim=True)
    out = (w * (y - m) / torch.sqrt(var + eps) + b) * g * torch.sigmoid(g)
    return out, (y, g, w, b)


SHAPES = [(1, 1, 8), (1, 1, 1), (3, 2, 7), (64, 16, 512), (130, 3, 100), (1000, 8, 256), (33, 2, 1024), (57, 5, 264),
          (20, 1, 1001), (4097, 1, 64), (513, 4, 128), (9, 300, 40), (77, 2, 33)]


@pytest.mark.parametrize("tokens,heads,dv", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("affine", [True, False])
def test_matches_definition(tokens, heads, dv, dtype, affine):
    y, g, d, w, b = inputs(tokens, heads, dv, dtype, tokens + dv, affine)
    out, leaves = definition(y, g, w, b, 1e-5)
    grads = torch.autograd.grad(out, leaves, d.double())
    dev = [None if t is None else t.cuda() for t in (y, g, w, b, d)]
    got = rn.msr_affine(*dev[:4])
    ggot = rn.msr_affine_backward(*dev)
    torch.cuda.synchronize()
    e = [errors(got, out.detach().numpy())] + [errors(x, r.numpy()) for x, r in zip(ggot, grads)]
    if dv == 1:  # y - mean is 0: dy is 0 in exact arithmetic, and dweight too
        assert float(ggot[0].abs().max()) == 0.0 and float(ggot[2].abs().max()) == 0.0
        e[1] = e[3] = 0.0
    print(f"msr {tokens}x{heads}x{dv} {dtype}: out/dy/dg/dw/db " + " ".join(f"{x:.1e}" for x in e))
    assert max(e) <= TOL, e
    if not affine:
        assert errors(got, oracle.msr_epilogue(y, g, heads, 1e-5)) <= TOL


def test_unaligned_rows_and_tails():
    """Buffers off a 16-byte boundary take the scalar path: the same values."""
    y, g, d, w, b = inputs(40, 3, 64, "bf16", 9)

    def shift(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        flat[1:] = t.flatten().cuda()
        return flat[1:].view(t.shape)
    a = rn.msr_affine(y.cuda(), g.cuda(), w.cuda(), b.cuda())
    s = rn.msr_affine(shift(y), shift(g), shift(w), shift(b))
    ga = rn.msr_affine_backward(y.cuda(), g.cuda(), w.cuda(), b.cuda(), d.cuda())
    gs = rn.msr_affine_backward(shift(y), shift(g), shift(w), shift(b), shift(d))
    torch.cuda.synchronize()
    for x, z in zip((a, *ga), (s, *gs)):
        assert errors(x, z.double().cpu().numpy()) <= 2.0 ** -7  # two roundings of nearly the same value


def test_central_differences():
    """Directional derivatives of the forward in fp32 by central differences: h^2 truncation (h = 1e-2,
    third derivatives of order 1: ~1e-4) and 2^-24 |sum| / h of rounding."""
    y, g, d, w, b = inputs(12, 2, 24, "f32", 21)
    dev = [t.cuda() for t in (y, g, w, b)]
    grads = rn.msr_affine_backward(*dev, d.cuda())
    h = 1e-2
    for i, name in enumerate("ygwb"):
        u = si.randn(tuple(dev[i].shape), 30 + i, "f32").cuda()
        lo, hi = list(dev), list(dev)
        hi[i], lo[i] = dev[i] + h * u, dev[i] - h * u
        f = lambda a: (rn.msr_affine(*a).double() * d.cuda().double()).sum().item()  # noqa: E731
        num, ana = (f(hi) - f(lo)) / (2 * h), (grads[i].double() * u.double()).sum().item()
        scale = float(grads[i].double().norm() * u.double().norm())
        assert abs(num - ana) <= 2e-3 * scale, (name, num, ana)


@pytest.mark.parametrize("which", ["none", "w", "b"])
def test_optional_sums_no_workspace_and_empty(which):
    y, g, d, w, b = (t.cuda() for t in inputs(50, 2, 64, "bf16", 41))
    full = rn.msr_affine_backward(y, g, w, b, d)
    dy, dg = torch.empty_like(y), torch.empty_like(g)
    s = torch.full((2, 64), 7.0, device="cuda")
    rn.retnet_msr_affine_backward(y, g, w, b, d, dy, dg, s if which == "w" else None, s if which == "b" else None)
    torch.cuda.synchronize()
    assert torch.equal(dy, full[0]) and torch.equal(dg, full[1])
    if which != "none":
        assert torch.equal(s, full[2] if which == "w" else full[3])
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert rn.msr_affine(e, e, w, b).shape == e.shape
    out = rn.msr_affine_backward(e, e, w, b, e)
    torch.cuda.synchronize()
    assert not out[2].any() and not out[3].any()


def test_same_bits_in_a_graph_and_in_place():
    y, g, d, w, b = (t.cuda() for t in inputs(700, 4, 128, "bf16", 51))
    want, grads = rn.msr_affine(y, g, w, b), rn.msr_affine_backward(y, g, w, b, d)
    out = [torch.empty_like(y) for _ in range(3)] + [torch.empty(4, 128, device="cuda") for _ in range(2)]
    ws = torch.empty(rn.retnet_msr_affine_workspace_size(y.shape), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rn.retnet_msr_affine(y, g, w, b, out[0])
        rn.retnet_msr_affine_backward(y, g, w, b, d, *out[1:], workspace=ws)
    for _ in range(2):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, z) for a, z in zip(out, (want, *grads)))
    y2 = y.clone()
    rn.retnet_msr_affine(y2, g, w, b, y2)
    torch.cuda.synchronize()
    assert torch.equal(y2, want)


def test_rows_of_one_value_and_large_values():
    """A constant row has y - mean = 0 and sd = sqrt(eps); rows of magnitude 1e4 lose nothing to the
    uncentred square."""
    y, g, d, w, b = inputs(6, 2, 48, "f32", 61)
    y[0] = 3.0
    y[1] = 0.0
    y[2] += 1e4
    out, leaves = definition(y, g, w, b, 1e-5)
    grads = torch.autograd.grad(out, leaves, d.double())
    dev = [t.cuda() for t in (y, g, w, b, d)]
    got, gg = rn.msr_affine(*dev[:4]), rn.msr_affine_backward(*dev)
    torch.cuda.synchronize()
    # row 2: the sum of 48 values of 1e4 rounds by half a step of 8e4 (2^-8) some 36 times and of 4.8e5
    # (2^-6) some three times: the mean is off by up to 0.14 / 48 = 3e-3, the output by up to
    # |w g sigmoid(g)| <= 5 times that, against an rms of about 0.6
    keep = [0, 1, 3, 4, 5]
    assert errors(got[keep], out.detach().numpy()[keep]) <= TOL
    assert errors(got[2], out.detach().numpy()[2]) <= 3e-2
    for x, r in zip(gg[:2], grads[:2]):
        assert np.isfinite(x.cpu().numpy()).all()
        assert errors(x[keep][1:], r.numpy()[keep][1:]) <= TOL * 316  # row 1: 1/sd = 316 scales every rounding


def test_training_chain():
    """Retention forward, affine epilogue, and both gradients chained: dq, dk, dv, dgate, dweight, dbias of
    a scalar loss against fp64 autograd through the quadratic form."""
    B, L, h, dk, dv = 2, 96, 2, 64, 64
    flags = rn.F_XPOS | rn.F_SCALE_SQRT_D | rn.F_NORM_D
    q, k, v = si.qkv(B, L, h, dk, dv, 71, "f32")
    gate, d = si.randn((B * L, h, dv), 72, "f32"), si.randn((B * L, h, dv), 73, "f32")
    w, b = 1.0 + 0.2 * si.randn((h, dv), 74, "f32"), 0.2 * si.randn((h, dv), 75, "f32")
    g, th = si.gamma_schedule(h), si.theta_schedule(dk)
    dev = [t.cuda() for t in (q, k, v)]
    o = rn.retention_chunkwise(*dev, g, th, 64, flags)
    y = o.flatten(0, 1)
    dy, dgate, dw, db = rn.msr_affine_backward(y, gate.cuda(), w.cuda(), b.cuda(), d.cuda())
    grads = [torch.empty_like(t) for t in dev]
    rn.retnet_retention_backward(*dev, dy.view(B, L, h, dv), *grads, g, th, 0, flags)
    torch.cuda.synchronize()
    q, k, v = (t.double().requires_grad_() for t in (q, k, v))
    p = torch.arange(L, dtype=torch.float64)
    z = torch.polar(torch.ones(L, dk // 2, dtype=torch.float64), p[:, None] * torch.from_numpy(th).double())
    rot = lambda x: torch.view_as_real(torch.view_as_complex(x.unflatten(-1, (-1, 2))) * z[:, None]).flatten(-2)  # noqa: E731
    gam = torch.from_numpy(g).double()
    n = p[:, None] - p[None]
    D = torch.where(n >= 0, gam[:, None, None] ** n.clamp(min=0), 0.0)
    c = torch.sqrt((1 - gam[:, None] ** (p + 1)) / (1 - gam[:, None])) * dk ** 0.5
    ref = torch.einsum("bnhd,bmhd->bhnm", rot(q), rot(k)) * D / c[..., None]
    ref = torch.einsum("bhnm,bmhe->bnhe", ref, v).flatten(0, 1)
    m = ref.mean(-1, keepdim=True)
    gd, wd, bd = (t.double().requires_grad_() for t in (gate, w, b))
    out = (wd * (ref - m) / torch.sqrt(((ref - m) ** 2).mean(-1, keepdim=True) + 1e-5) + bd) * gd * torch.sigmoid(gd)
    want = torch.autograd.grad(out, (q, k, v, gd, wd, bd), d.double())
    e = [errors(x, r.numpy()) for x, r in zip((*grads, dgate, dw, db), want)]
    print("chain dq/dk/dv/dgate/dw/db " + " ".join(f"{x:.1e}" for x in e))
    # the normalisation divides by a row's deviation, as small as 1e-2 of the outputs' rms here: the
    # retention's bar, times the ten that its smallest rows magnify it by
    assert max(e) <= 10 * TOL_F32 and TOL_F32 < TOL_BF16
