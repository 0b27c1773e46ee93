"""Refusals of the packed, single-token, slot-copy and affine-MSR entry points (no GPU needed): each
bad argument gets its documented status before any device is touched."""
import ctypes

import numpy as np
import pytest
import torch

import linear_attention_sequence_chunkwise_b200 as rn
from linear_attention_sequence_chunkwise_b200 import _build

FAKE = 0x10000  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return rn.load()


def _fp(a):
    return a.tobytes()


def _dims(**kw):
    d = dict(tokens=10, seqs=2, heads=4, heads_kv=2, d_k=16, d_v=8, slots=5, stride_q=64, stride_k=32, stride_v=16,
             stride_o=32)
    d.update(kw)
    return rn.PackedDims(**d)


G2, TH8 = np.full(2, 0.9, np.float32), np.ones(8, np.float32)
BIG = 1 << 40


def _packed(lib, d=None, q=FAKE, o=FAKE, dtype=0, gamma=G2, theta=TH8, flags=rn.F_XPOS, cu=FAKE, slots=FAKE, pos=FAKE,
            pool=FAKE, ws=FAKE, ws_bytes=BIG):
    return lib.retnet_retention_packed(q, FAKE, FAKE, o, d or _dims(), dtype, _fp(gamma),
                                       None if theta is None else _fp(theta), flags, cu, slots, pos, pool, ws, ws_bytes,
                                       None)


def _step(lib, d=None, dtype=0, flags=0, slots=FAKE, pos=FAKE, pool=FAKE, gamma=G2):
    return lib.retnet_retention_step_slots(FAKE, FAKE, FAKE, FAKE, d or _dims(tokens=2), dtype, _fp(gamma), None, flags,
                                           slots, pos, pool, None)


BAD_DIMS = [dict(tokens=-1), dict(tokens=1 << 31), dict(seqs=-1), dict(seqs=65536), dict(heads=0), dict(heads_kv=0),
            dict(heads=3), dict(heads=258, stride_q=1 << 20, stride_o=1 << 20), dict(d_k=0), dict(d_v=0),
            dict(d_k=514, stride_q=1 << 20, stride_k=1 << 20), dict(d_v=1025, stride_v=1 << 20, stride_o=1 << 20),
            dict(slots=0), dict(stride_q=63), dict(stride_k=31), dict(stride_v=15), dict(stride_o=31)]


@pytest.mark.parametrize("bad", BAD_DIMS)
def test_packed_shapes(lib, bad):
    assert _packed(lib, _dims(**bad)) == 2
    assert _step(lib, _dims(**{"tokens": 2, **bad})) == 2


def test_packed_refusals(lib):
    assert _packed(lib, dtype=2) == 3
    assert _packed(lib, flags=64) == 4
    assert _packed(lib, flags=rn.F_NORM_R) == 5
    assert _packed(lib, _dims(d_k=15, stride_q=60), flags=rn.F_XPOS) == 4  # odd d_k with xPos
    assert _packed(lib, gamma=np.array([0.9, 1.0], np.float32)) == 4
    assert _packed(lib, theta=None) == 1
    assert _packed(lib, theta=np.full(8, np.inf, np.float32)) == 4
    for name in ("q", "o", "cu", "slots", "pool", "ws"):
        assert _packed(lib, **{name: None}) == 1, name
    assert _packed(lib, q=FAKE + 2) == 4 and _packed(lib, q=FAKE + 1, dtype=1) == 4
    assert _packed(lib, cu=FAKE + 2) == 4 and _packed(lib, slots=FAKE + 2) == 4 and _packed(lib, pos=FAKE + 4) == 4
    assert _packed(lib, pool=FAKE + 4) == 4 and _packed(lib, ws=FAKE + 8) == 4
    n = rn.retnet_packed_workspace_size((10, 2, 4, 2, 16, 8))
    assert n > 0 and _packed(lib, ws_bytes=n - 1) == 4
    assert _packed(lib, _dims(tokens=0), q=None) == 0 and _packed(lib, _dims(seqs=0), cu=None) == 0  # no work


def test_packed_kernel_choice(lib):
    f = rn.F_XPOS | rn.F_SCALE_SQRT_D | rn.F_NORM_D
    g = np.array([1 - 2.0 ** -5, 0.999], np.float32)
    def kern(dims=(300, 3, 4, 2, 128, 192), dtype=rn.BF16, flags=f, gamma=g, strides=None):
        return rn.retnet_packed_kernel(dims, dtype, flags, gamma, strides)
    assert kern() == 1 and kern((1, 1, 2, 2, 64, 64)) == 1 and kern((9, 2, 2, 2, 256, 512)) == 1
    assert kern(dtype=rn.F32) == 0 and kern(flags=f | rn.F_PRECISE) == 0
    assert kern((300, 3, 4, 2, 96, 192)) == 0 and kern((300, 3, 4, 2, 128, 200)) == 0
    assert kern(gamma=np.array([0.93, 0.999], np.float32)) == 0  # 0.93^128 < 2^-12
    assert kern(strides=(520, 256, 384, 768)) == 1 and kern(strides=(516, 256, 384, 768)) == 0
    assert kern(dtype=7) == -3 and kern((300, 3, 3, 2, 128, 192)) == -2 and kern(flags=rn.F_NORM_R) == -5
    assert kern(gamma=np.array([1.0, 0.9], np.float32)) == -4 and kern(gamma=None) == -1


def test_step_refusals(lib):
    assert _step(lib, _dims(tokens=3)) == 2  # tokens != seqs
    assert _step(lib, dtype=5) == 3
    assert _step(lib, flags=rn.F_NORM_R) == 5
    assert _step(lib, slots=None) == 1 and _step(lib, pool=None) == 1
    assert _step(lib, pool=FAKE + 8) == 4 and _step(lib, pos=FAKE + 4) == 4
    assert _step(lib, _dims(tokens=0, seqs=0), slots=None) == 0


def test_slots_copy_refusals(lib):
    def call(pool=FAKE, slots=4, floats=16, src=FAKE, dst=FAKE, n=2):
        return lib.retnet_state_slots_copy(pool, slots, floats, src, dst, n, None)
    assert call(slots=0) == 2 and call(floats=0) == 2 and call(n=-1) == 2 and call(n=rn.MAX_SLOT_PAIRS + 1) == 2
    assert call(pool=None) == 1 and call(src=None) == 1 and call(dst=None) == 1
    assert call(pool=FAKE + 4) == 4 and call(src=FAKE + 2) == 4
    assert call(n=0, pool=None) == 0


def test_msr_affine_refusals(lib):
    def fwd(y=FAKE, g=FAKE, w=FAKE, out=FAKE, tokens=3, heads=2, dv=8, eps=1e-5, dtype=0):
        return lib.retnet_msr_affine(y, g, w, None, out, tokens, heads, dv, eps, dtype, None)

    def bwd(dout=FAKE, dy=FAKE, dw=FAKE, ws=FAKE, n=BIG, tokens=3, heads=2, dv=8, eps=1e-5, dtype=0):
        return lib.retnet_msr_affine_backward(FAKE, FAKE, None, None, dout, dy, FAKE, dw, None, tokens, heads, dv, eps,
                                              dtype, ws, n, None)
    for f in (fwd, bwd):
        assert f(dtype=3) == 3 and f(tokens=-1) == 2 and f(heads=0) == 2 and f(dv=0) == 2 and f(dv=1025) == 2
        assert f(tokens=1 << 30, heads=4) == 2
        assert f(eps=-1.0) == 4 and f(eps=float("nan")) == 4
    assert fwd(y=None) == 1 and fwd(out=None) == 1 and fwd(y=FAKE + 2) == 4 and fwd(y=FAKE + 1, dtype=1) == 4
    assert fwd(w=FAKE + 2) == 4 and fwd(tokens=0, y=None) == 0
    assert bwd(dout=None) == 1 and bwd(dy=None) == 1 and bwd(ws=None) == 1 and bwd(ws=FAKE + 4) == 4
    need = rn.retnet_msr_affine_workspace_size((3, 2, 8))
    assert bwd(n=need - 1) == 4


def test_binding_refusals():
    """Wrong shapes, types, layouts and host tensors raise before the library is called; where everything
    else is right, host tensors are what is refused."""
    q, k, v, o = torch.zeros(4, 4, 16), torch.zeros(4, 2, 16), torch.zeros(4, 2, 8), torch.zeros(4, 4, 8)
    pool, cu = torch.zeros(5, 2, 16, 8), torch.zeros(3, dtype=torch.int32)
    sl, pos = torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int64)
    good = dict(q=q, k=k, v=v, o=o, pool=pool, cu_seqlens=cu, slots=sl, pos=pos, gamma=G2, theta=TH8)
    wide = torch.zeros(4, 200)
    cases = [({}, "CUDA tensors"), (dict(q=wide[:, 3:67].unflatten(1, (4, 16))), "CUDA tensors"),
             (dict(pos=None, theta=None), "CUDA tensors"), (dict(gamma=[0.9, 0.8]), "CUDA tensors"),
             (dict(gamma=torch.full((2,), 0.9, dtype=torch.float64)), "CUDA tensors"),
             (dict(q=torch.zeros(4, 16, 4).transpose(1, 2)), "heads of a row"),
             (dict(q=torch.zeros(1, 4, 16).expand(4, 4, 16)), "rows must not overlap"),
             (dict(k=k[:, :1]), "shape mismatch"), (dict(o=o[:3]), "shape mismatch"), (dict(q=q[0]), "three dimensions"),
             (dict(o=o.bfloat16()), "one dtype"), (dict(pool=pool.double()), "pool"), (dict(pool=pool[:, :, :8]), "pool"),
             (dict(pool=pool.transpose(2, 3)), "pool"), (dict(cu_seqlens=cu.long()), "cu_seqlens"),
             (dict(cu_seqlens=cu[:2]), "cu_seqlens"), (dict(slots=sl[:, None]), "slots"), (dict(pos=pos.int()), "pos"),
             (dict(gamma=G2[:1]), "gamma has 1 entries"), (dict(theta=TH8[:7]), "theta has 7 entries"),
             (dict(workspace=torch.zeros(8, 8, dtype=torch.uint8).t()), "workspace")]
    for change, why in cases:
        with pytest.raises(ValueError, match=why):
            rn.retnet_retention_packed(**{**good, **change})
    step = {n: good[n] for n in ("q", "k", "v", "o", "pool", "gamma", "theta")}
    step.update(slots=torch.zeros(4, dtype=torch.int32), pos=None)
    for change, why in (({}, "CUDA tensors"), (dict(slots=sl), "slots"), (dict(pos=pos), "pos"), (dict(v=v[:2]), "shape mismatch")):
        with pytest.raises(ValueError, match=why):
            rn.retnet_retention_step_slots(**{**step, **change})
    for args, why in (((pool, sl, sl), "CUDA tensors"), ((pool.double(), sl, sl), "float32"), ((pool, sl, sl[:1]), "dst"),
                      ((pool, sl.long(), sl), "src"), ((pool.transpose(0, 1), sl, sl), "contiguous")):
        with pytest.raises(ValueError, match=why):
            rn.retnet_state_slots_copy(*args)
    y, w = torch.zeros(3, 2, 8), torch.zeros(2, 8)
    for args, why in (((y, y, w, w, y), "CUDA tensors"), ((y, y[:, :, :4], None, None, y), "one shape"),
                      ((y, y.bfloat16(), None, None, y), "one shape"), ((y, y, torch.zeros(8), None, y), "float32"),
                      ((y, y, w.double(), None, y), "float32"), ((y[0], y, None, None, y), "tokens"),
                      ((y.transpose(0, 1), y, None, None, y), "contiguous")):
        with pytest.raises(ValueError, match=why):
            rn.retnet_msr_affine(*args)
        with pytest.raises(ValueError, match=why):
            rn.retnet_msr_affine_backward(*args, y, y)
        with pytest.raises(ValueError, match=why):
            rn.msr_affine_backward(*args)
    with pytest.raises(ValueError, match="float32"):
        rn.retnet_msr_affine_backward(y, y, w, w, y, y, y, torch.zeros(3, 8))
