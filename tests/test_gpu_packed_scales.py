"""Packed tensor-core outputs for q and k far from unit size, against the fp64 oracle.

Bars, max|err|/rms: 1e-2 for bf16 outputs net of their own rounding (the framework's bar for bf16 inputs),
1e-4 for the pool.  q and k are rounded to fp16 after they are brought to its range by powers of two, so
their size does not matter; states are rounded as they are, so v and k keep them above 1e-3 here.
"""
import numpy as np
import pytest
import torch

import linear_attention_sequence_chunkwise_b200 as rn
from gpu_util import TOL_BF16, TOL_F32, require_gpu
from serving_util import FLAGS, case, cu_of, errors, reference, split

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(cuda_lib):
    require_gpu()
    for f in (rn.retnet_slot_errors, rn.retnet_debug_wait_timeouts, rn.retnet_fp16_range_errors):
        f(clear=True)
    yield
    assert rn.retnet_slot_errors(clear=True) == 0
    assert rn.retnet_debug_wait_timeouts(clear=True) == 0
    assert rn.retnet_fp16_range_errors(clear=True) == 0


def run(lens, heads, dk, dv, seed, gamma, by_q, by_k, by_v=1.0, pos=None, pool_std=0.5):
    """Output and pool of a call on the GPU and of the oracle; by_*: factors of q, k, v (numbers, or one a row)."""
    fused, pool, slots, pos, gamma, theta = case(lens, heads, heads, dk, dv, "bf16", seed, gamma=gamma, pos=pos,
                                                 pool_std=pool_std)
    q, k, v = split(fused, heads, heads, dk, dv)
    row = lambda by: torch.as_tensor(by, dtype=torch.float64).reshape(-1, 1, 1)  # noqa: E731
    q, k, v = ((x.double() * row(by)).bfloat16() for x, by in ((q, by_q), (k, by_k), (v, by_v)))
    assert rn.retnet_packed_kernel((q.shape[0], len(lens), heads, heads, dk, dv), rn.BF16, FLAGS, gamma) == 1
    ref = reference(q, k, v, pool, lens, slots, pos, gamma, theta, FLAGS)
    o, p = torch.full((q.shape[0], heads, dv), 0.25, dtype=torch.bfloat16, device="cuda"), pool.cuda()
    rn.retnet_retention_packed(q.cuda(), k.cuda(), v.cuda(), o, p, cu_of(lens).cuda(),
                               torch.tensor(slots, dtype=torch.int32).cuda(), torch.tensor(pos).cuda(), gamma, theta)
    torch.cuda.synchronize()
    return o, p, ref


@pytest.mark.parametrize("gamma", [[0.94, 0.945], [1 - 2.0 ** -5, 1 - 2.0 ** -9]])
@pytest.mark.parametrize("by_q,by_k", [(1e-2, 1e-2), (1e-3, 1e-2), (1e-4, 1e-2), (1e-2, 1.0), (1.0, 1e-2), (1e-30, 1.0)])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (256, 128)])
def test_small_q_and_k(gamma, by_q, by_k, dk, dv):
    o, p, (ref, after) = run([300, 128, 77], 2, dk, dv, 400 + dk, gamma, by_q, by_k, pool_std=0.5 * by_k)
    eo, ep = errors(o, ref), errors(p, after)
    print(f"gamma {gamma[0]} q {by_q} k {by_k}: o {eo:.2e} pool {ep:.2e}")
    assert eo <= TOL_BF16 and ep <= TOL_F32


@pytest.mark.parametrize("by_q,by_k,by_v", [(1e6, 1e-2, 1.0), (1e30, 1e-2, 1.0), (1e-3, 1e6, 1e-6), (1e4, 1e4, 1e-4)])
def test_large_q_and_k(by_q, by_k, by_v):
    """q and k past fp16's 65504 are finite operands (the states, k times v, stay within)."""
    o, p, (ref, after) = run([300, 128, 77], 2, 128, 64, 411, [0.94, 0.99], by_q, by_k, by_v, pool_std=0.5 * by_k * by_v)
    eo, ep = errors(o, ref), errors(p, after)
    print(f"q {by_q} k {by_k} v {by_v}: o {eo:.2e} pool {ep:.2e}")
    assert eo <= TOL_BF16 and ep <= TOL_F32


@pytest.mark.parametrize("dk", [64, 128, 256])
def test_tokens_of_different_sizes(dk):
    """Rows of q and k whose sizes differ by up to 2^8 (exact factors): each output row, its own factor of q
    taken off, meets the bar."""
    lens = [260, 90]
    rng = np.random.default_rng(dk)
    by_q, by_k = (2.0 ** rng.integers(-4, 5, sum(lens) + 2) for _ in range(2))
    o, p, (ref, after) = run(lens, 2, dk, 64, 420 + dk, [0.94, 0.97], by_q, by_k)
    off = by_q[:, None, None]
    scaled = (o.double().cpu() / torch.from_numpy(off)).bfloat16()  # exact: powers of two
    assert errors(scaled, ref / off) <= TOL_BF16 and errors(p, after) <= TOL_F32


def test_one_token_of_zeros_and_one_not_finite():
    """All-zero rows (a padding token), and one row that is not finite in a sequence of its own."""
    by = np.ones(192)
    by[3] = 0.0
    by[130:] = 0.0
    o, p, (ref, after) = run([130, 60], 2, 64, 64, 431, [0.94, 0.97], by, by)
    assert errors(o[:130], ref[:130]) <= TOL_BF16 and errors(p, after) <= TOL_F32
    o, p, (ref, after) = run([100, 60], 2, 64, 64, 432, [0.94, 0.97], 1e-3, 1.0)
    fused, pool, slots, pos, gamma, theta = case([100, 60], 2, 2, 64, 64, "bf16", 432, gamma=[0.94, 0.97])
    q, k, v = split(fused, 2, 2, 64, 64)
    q = (q.double() * 1e-3).bfloat16()
    q[120] = float("inf")
    o2 = torch.full_like(o, 0.25)
    rn.retnet_retention_packed(q.cuda(), k.cuda(), v.cuda(), o2, pool.cuda(), cu_of([100, 60]).cuda(),
                               torch.tensor(slots, dtype=torch.int32).cuda(), torch.tensor(pos).cuda(), gamma, theta)
    torch.cuda.synchronize()
    assert rn.retnet_fp16_range_errors(clear=True) > 0
    assert torch.equal(o2[:100], o[:100]) and not torch.isfinite(o2[120]).any()


@pytest.mark.parametrize("dk", [64, 128, 256])
def test_a_token_that_is_not_finite_costs_its_neighbours_nothing(dk):
    """Tokens that share their power of two with one whose q is infinite, or that come before one whose k is,
    meet the bar at sizes that need it."""
    fused, pool, slots, pos, gamma, theta = case([128, 70], 2, 2, dk, 64, "bf16", 440 + dk, gamma=[0.94, 0.945], pos=[0, 0])
    q, k, v = split(fused, 2, 2, dk, 64)
    q, k = ((x.double() * 1e-4).bfloat16() for x in (q, k))
    ref, _ = reference(q, k, v, pool, [128, 70], slots, pos, gamma, theta, FLAGS)
    q[100], q[101, 0, 3], k[128 + 50] = float("inf"), float("nan"), float("-inf")
    o = torch.full((q.shape[0], 2, 64), 0.25, dtype=torch.bfloat16, device="cuda")
    rn.retnet_retention_packed(q.cuda(), k.cuda(), v.cuda(), o, pool.cuda(), cu_of([128, 70]).cuda(),
                               torch.tensor(slots, dtype=torch.int32).cuda(), torch.tensor(pos).cuda(), gamma, theta)
    torch.cuda.synchronize()
    assert rn.retnet_fp16_range_errors(clear=True) > 0
    good = [i for i in range(128 + 50) if i not in (100, 101)]
    assert errors(o[good], ref[good]) <= TOL_BF16
    assert not torch.isfinite(o[100]).any() and not torch.isfinite(o[101, 0]).any() and torch.isfinite(o[101, 1]).all()


@pytest.mark.parametrize("by_q,by_k,by_v", [(1e-33, 1.0, 1.0), (1.0, 1e-33, 1e33), (1e33, 1.0, 1e-33)])
def test_the_ends_of_the_range(by_q, by_k, by_v):
    """Powers of two near the ends of fp32's range (for k, a chunk that starts at position 0: no state is read)."""
    lens, pos = ([300, 128], None) if by_k == 1.0 and by_v == 1.0 else ([128, 77], [0, 0])
    o, p, (ref, after) = run(lens, 2, 64, 64, 451, [0.94, 0.99], by_q, by_k, by_v, pos=pos, pool_std=0.5 * by_k * by_v)
    eo, ep = errors(o, ref), errors(p, after)
    print(f"q {by_q} k {by_k} v {by_v}: o {eo:.2e} pool {ep:.2e}")
    assert eo <= TOL_BF16 and ep <= TOL_F32
