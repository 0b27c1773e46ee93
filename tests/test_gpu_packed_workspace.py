"""The packed call within the workspace that retnet_packed_call_workspace_size names, and what it allocates."""
import numpy as np
import pytest
import torch

import linear_attention_sequence_chunkwise_b200 as rn
from gpu_util import TOL_BF16, TOL_F32, require_gpu
from serving_util import FLAGS, case, cu_of, errors, reference, split

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,hq,kv,dk,dv,dtype,offset", [
    ([300, 41, 0, 200], 4, 4, 128, 128, "bf16", 0),   # by sequence
    ([700, 900], 1, 1, 128, 128, "bf16", 0),          # chunks dealt out
    ([300, 41], 2, 2, 64, 64, "bf16", 1),             # bf16 off 16-byte addresses: CUDA cores
    ([300, 41], 4, 2, 40, 24, "f32", 0), ([1], 1, 1, 1, 1, "f32", 0), ([600], 1, 1, 256, 256, "f32", 0)])
def test_the_named_workspace_does(cuda_lib, lens, hq, kv, dk, dv, dtype, offset):
    require_gpu()
    flags = FLAGS if dk % 2 == 0 else rn.F_SCALE_SQRT_D | rn.F_NORM_D
    fused, pool, slots, pos, gamma, theta = case(lens, hq, kv, dk, dv, dtype, 500 + dk, gamma=np.linspace(0.95, 0.999, kv))
    ref, after = reference(*split(fused, hq, kv, dk, dv), pool, lens, slots, pos, gamma, theta, flags)
    rows, width = fused.shape
    flat = torch.zeros(fused.numel() + 8, dtype=fused.dtype, device="cuda")
    place = flat[offset:offset + fused.numel()].view(rows, width)
    place.copy_(fused)
    q, k, v = split(place, hq, kv, dk, dv)
    aligned = all(x.data_ptr() % 16 == 0 for x in (q, k, v))
    assert not (aligned and offset)
    code, strides = rn.BF16 if dtype == "bf16" else rn.F32, (width,) * 3 + (hq * dv,)
    dims = (rows, len(lens), hq, kv, dk, dv)
    n = rn.retnet_packed_call_workspace_size(dims, code, flags if aligned else flags | rn.F_PRECISE, gamma, strides)
    cu, sl, ps = cu_of(lens).cuda(), torch.tensor(slots, dtype=torch.int32).cuda(), torch.tensor(pos).cuda()

    def call(ws):
        o, p = torch.full((rows, hq, dv), 0.25, dtype=fused.dtype, device="cuda"), pool.cuda()
        torch.cuda.synchronize()
        torch.cuda.empty_cache()  # (a cached block may be up to 1 MB larger than what is asked for)
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        rn.retnet_retention_packed(q, k, v, o, p, cu, sl, ps, gamma, theta, flags, workspace=ws)
        torch.cuda.synchronize()
        return o, p, torch.cuda.max_memory_allocated() - before
    held = torch.full((n + 4096,), 77, dtype=torch.uint8, device="cuda")
    o, p, used = call(held[:n])
    assert errors(o, ref) <= (TOL_BF16 if dtype == "bf16" else TOL_F32) and errors(p, after) <= TOL_F32
    assert used == 0 and bool((held[n:] == 77).all())
    o2, p2, used = call(None)
    assert torch.equal(o, o2) and torch.equal(p, p2)
    assert n <= used <= n + 512  # (the allocator's granularity)
    with pytest.raises(rn.RetnetError):
        call(held[:n - 1])
