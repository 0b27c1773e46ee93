"""The waits of the packed tensor-core kernels: results against the fp64 oracle, and no wait gives up."""
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


class Call:
    """One packed bf16 call on the GPU, to be made again and again on the same inputs."""

    def __init__(self, lens, heads, dk, dv, seed, gamma=None, **kw):
        gamma = np.linspace(0.95, 0.9999, heads) if gamma is None else gamma
        self.fused, self.pool, self.slots, self.pos, self.gamma, self.theta = case(lens, heads, heads, dk, dv, "bf16", seed,
                                                                                   gamma=gamma, **kw)
        self.lens, self.dims = lens, (heads, heads, dk, dv)
        self.q, self.k, self.v = split(self.fused.cuda(), *self.dims)
        self.cu, self.pos_d = cu_of(lens).cuda(), torch.tensor(self.pos).cuda()
        self.slots_d = torch.tensor(self.slots, dtype=torch.int32).cuda()
        assert rn.retnet_packed_kernel((self.fused.shape[0], len(lens), *self.dims), rn.BF16, FLAGS, self.gamma) == 1

    def run(self):
        o = torch.full((self.q.shape[0], self.dims[0], self.dims[3]), 0.25, dtype=torch.bfloat16, device="cuda")
        p = self.pool.cuda()
        rn.retnet_retention_packed(self.q, self.k, self.v, o, p, self.cu, self.slots_d, self.pos_d, self.gamma, self.theta)
        return o, p

    def reference(self):
        return reference(*split(self.fused, *self.dims), self.pool, self.lens, self.slots, self.pos, self.gamma, self.theta,
                         FLAGS)


@pytest.mark.parametrize("lens,heads,dk,dv", [
    ([128 * 6 + 65, 128 * 5, 128 * 4 + 64, 128 * 7 + 1] * 2, 24, 64, 64),  # walks by sequence, the shortest products
    ([128 * 9 + 100, 128 * 8], 4, 64, 64),                                  # chunks dealt out
    ([128 * 5 + 3] * 6, 16, 128, 128),
    ([128 * 6 + 120] * 2, 8, 256, 256),
])
def test_chunks_of_one_and_two_steps_many_times(lens, heads, dk, dv):
    """The waits of the data warps (tests/test_packed_steps.py) as they run: the same bits every time."""
    call = Call(lens, heads, dk, dv, 300 + dk + len(lens))
    ref, after = call.reference()
    o, p = call.run()
    assert errors(o, ref) <= TOL_BF16 and errors(p, after) <= TOL_F32
    for _ in range(100):
        again = call.run()
        assert torch.equal(again[0], o) and torch.equal(again[1], p)


@pytest.mark.parametrize("lens,heads,dk,dv", [
    ([700, 130, 1, 0, 400], 24, 64, 64),  # a walk by sequence
    ([1100, 900], 2, 64, 192),            # chunks dealt out, then the scan
    ([700, 500] * 4, 8, 128, 256),        # by sequence, 64 state values a thread
    ([900, 1030], 2, 256, 128),           # dealt out, two blocks of d_k, two teams
])
def test_waits_that_give_up_return_and_leave_no_trace(lens, heads, dk, dv):
    """With a budget of 500 SM cycles (a testing aid) the warps' waits for one another give up: the call
    returns, counts them, and a later call has the bits of an earlier one."""
    call = Call(lens, heads, dk, dv, 340 + dk + dv)
    o, p = call.run()
    assert rn.retnet_debug_wait_timeouts(clear=True) == 0
    rn.retnet_debug_set_wait_budget(500)
    try:
        call.run()  # (its outputs and slots are undefined)
        torch.cuda.synchronize()
        gave_up = rn.retnet_debug_wait_timeouts(clear=True)
    finally:
        rn.retnet_debug_set_wait_budget(0)
    rn.retnet_fp16_range_errors(clear=True)  # (so are the operands of the call that gave up)
    print(f"waits that gave up: {gave_up}")
    assert gave_up > 0
    again = call.run()
    assert torch.equal(again[0], o) and torch.equal(again[1], p)


def test_waits_do_not_count_the_states_running_time():
    """Output CTAs start beside the walk over the states and wait for it, however long it takes: with one
    prompt of 40000 tokens among empty sequences, walked for some 1e6 SM cycles, and a budget of 2e5 (a step
    of the walk takes 4e3, an output CTA 3e4) no wait gives up."""
    lens = [0] * 100 + [40000] + [0] * 99
    call = Call(lens, 2, 64, 64, 371, slots=[0] * 100 + [1] + [0] * 99, pos=[0] * 100 + [7] + [0] * 99, n_slots=2)
    o, p = call.run()
    torch.cuda.synchronize()
    rn.retnet_debug_set_wait_budget(200000)
    try:
        again = call.run()
        torch.cuda.synchronize()
    finally:
        rn.retnet_debug_set_wait_budget(0)
    assert rn.retnet_debug_wait_timeouts(clear=True) == 0
    assert torch.equal(again[0], o) and torch.equal(again[1], p)


@pytest.mark.parametrize("lens,heads,dv", [([700, 130, 300] * 4, 24, 64), ([900, 400] * 6, 16, 128)])
def test_range_report_sees_only_the_states(lens, heads, dv):
    """A walk with d_k 64 uses half of the lanes of its accumulators: what another call left in the other
    half is not reported as out of fp16's range."""
    call = Call(lens, heads, 64, dv, 381)
    call.run()
    assert rn.retnet_fp16_range_errors(clear=True) == 0
    leave = Call([128] * 296, 8, 64, 128, 382)
    for x in (leave.q, leave.k, leave.v):
        x.fill_(float("nan"))
    for _ in range(3):
        leave.run()
        assert rn.retnet_fp16_range_errors(clear=True) > 0
        call.run()
        assert rn.retnet_fp16_range_errors(clear=True) == 0
