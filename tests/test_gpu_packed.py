"""Packed retention (retnet_retention_packed) against the fp64 oracle, sequence by sequence.

Bars, max|err|/rms: 1e-4 for fp32 results and for the fp32 pool (fp32 arithmetic); for bf16 outputs
net of their own rounding 1e-2 (the framework's bar for bf16 inputs).
"""
import numpy as np
import pytest
import torch

import linear_attention_sequence_chunkwise_b200 as rn
import synth_inputs as si
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


def run(fused, pool, lens, slots, pos, gamma, theta, hq, kv, dk, dv, flags=FLAGS, stream=None, workspace=None, fill=0.25):
    q, k, v = split(fused.cuda(), hq, kv, dk, dv)
    o = torch.full((q.shape[0], hq, dv), fill, dtype=q.dtype, device="cuda")
    p = pool.cuda()
    rn.retnet_retention_packed(q, k, v, o, p, cu_of(lens).cuda(), torch.tensor(slots, dtype=torch.int32).cuda(),
                               None if pos is None else torch.tensor(pos).cuda(), gamma, theta, flags,
                               workspace=workspace, stream=stream)
    torch.cuda.synchronize()
    return o, p


def check(lens, hq, kv, dk, dv, dtype, seed, flags=FLAGS, tensor_cores=None, **kw):
    fused, pool, slots, pos, gamma, theta = case(lens, hq, kv, dk, dv, dtype, seed, **kw)
    q, k, v = split(fused, hq, kv, dk, dv)
    if tensor_cores is not None:
        dims, width = (q.shape[0], len(lens), hq, kv, dk, dv), fused.shape[1]
        kernel = rn.retnet_packed_kernel(dims, rn.BF16 if dtype == "bf16" else rn.F32, flags, gamma, (width,) * 3 + (hq * dv,))
        assert kernel == int(tensor_cores)
    ref, after = reference(q, k, v, pool, lens, slots, pos, gamma, theta, flags)
    o, p = run(fused, pool, lens, slots, pos, gamma, theta, hq, kv, dk, dv, flags)
    eo, ep = errors(o, ref), errors(p, after)
    print(f"packed lens={lens} h={hq}/{kv} dk={dk} dv={dv} {dtype}: o {eo:.2e} pool {ep:.2e}")
    assert eo <= (TOL_BF16 if dtype == "bf16" else TOL_F32) and ep <= TOL_F32
    # rows of no sequence and slots of no sequence with tokens keep their bits
    idle = torch.from_numpy(np.isnan(ref).all(axis=(1, 2)))
    assert bool((o.cpu()[idle] == 0.25).all()) and int(idle.sum()) >= 2
    named = {s for s, n in zip(slots, lens) if n and s >= 0}
    rest = [s for s in range(pool.shape[0]) if s not in named]
    assert torch.equal(p.cpu()[rest], pool[rest])


LENS = [[1], [2, 1], [64, 63, 65], [128, 127, 129, 0, 1], [300], [256, 257, 255], [0, 0, 5, 0], [511, 513, 40, 1, 0, 130],
        [1100, 17]]


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("hq,kv,dk,dv,dtype", [(2, 2, 64, 64, "bf16"), (2, 1, 128, 128, "bf16"), (3, 3, 32, 40, "f32")])
def test_lengths(lens, hq, kv, dk, dv, dtype):
    check(lens, hq, kv, dk, dv, dtype, 100 + sum(lens), tensor_cores=dtype == "bf16")


@pytest.mark.parametrize("hq,kv,dk,dv,dtype", [
    (4, 1, 128, 64, "bf16"), (6, 2, 64, 192, "bf16"), (2, 2, 256, 64, "bf16"), (2, 1, 256, 256, "bf16"),
    (1, 1, 128, 320, "bf16"), (2, 2, 256, 512, "bf16"),
    (2, 2, 16, 8, "bf16"), (1, 1, 1, 1, "f32"), (2, 2, 7, 5, "f32"), (8, 2, 80, 120, "f32"), (1, 1, 512, 130, "f32"),
    (2, 1, 66, 129, "bf16"), (1, 1, 96, 1024, "f32"),
])
def test_heads_and_widths(hq, kv, dk, dv, dtype):
    flags = FLAGS if dk % 2 == 0 else rn.F_SCALE_SQRT_D | rn.F_NORM_D
    check([130, 1, 0, 300, 77], hq, kv, dk, dv, dtype, 7 * dk + dv, flags=flags,
          tensor_cores=dtype == "bf16" and dk in (64, 128, 256) and dv % 64 == 0)


@pytest.mark.parametrize("flags", [0, rn.F_XPOS, rn.F_SCALE_SQRT_D, rn.F_NORM_D, FLAGS, FLAGS | rn.F_PRECISE])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_flags(flags, dtype):
    check([140, 33, 5], 2, 2, 64, 64, dtype, 31, flags=flags)


@pytest.mark.parametrize("gamma", [[0.5, 0.9], [1e-3, 0.94], [0.97, 1 - 2.0 ** -24], [1e-30, 0.3]])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decays(gamma, dtype):
    check([400, 257], 2, 2, 64, 64, dtype, 41, gamma=gamma)


@pytest.mark.parametrize("lens,kv,dk,dv", [
    ([700, 900], 1, 128, 128),           # few heads: states chunk by chunk, then the scan
    ([700, 900], 1, 256, 256),           # two blocks of d_k
    ([500, 1, 640, 0, 257], 24, 64, 64),  # many heads: a walk by sequence
    ([300] * 7, 8, 128, 256),
    ([1300], 2, 64, 320),                # 64 columns left over behind two slices of 128
])
def test_walks(lens, kv, dk, dv):
    """Both walks over the states (by chunk, by sequence) at every block of d_k and slice of d_v."""
    gamma = np.linspace(0.95, 0.9999, kv)  # (the schedule reaches 1 in fp32 at the 24th head)
    check(lens, kv, kv, dk, dv, "bf16", dk + dv + len(lens), tensor_cores=True, gamma=gamma)


@pytest.mark.parametrize("offset,pad", [(8, 0), (0, 8), (1, 0), (0, 4)])
def test_alignments(offset, pad):
    """Outputs and inputs off a 32-byte boundary (16-byte stores), and off a 16-byte one (CUDA cores)."""
    lens, hq, kv, dk, dv = [200, 60], 2, 2, 64, 128
    fused, pool, slots, pos, gamma, theta = case(lens, hq, kv, dk, dv, "bf16", 55)
    ref, after = reference(*split(fused, hq, kv, dk, dv), pool, lens, slots, pos, gamma, theta, FLAGS)
    rows, width = fused.shape

    def place(t):
        flat = torch.zeros(rows * (t.shape[1] + pad) + offset, dtype=t.dtype, device="cuda")
        view = flat[offset:].view(rows, t.shape[1] + pad)[:, :t.shape[1]]
        view.copy_(t)
        return view
    q, k, v = split(place(fused), hq, kv, dk, dv)
    o = place(torch.zeros(rows, hq * dv, dtype=torch.bfloat16)).unflatten(1, (hq, dv))
    p = pool.cuda()
    rn.retnet_retention_packed(q, k, v, o, p, cu_of(lens).cuda(), torch.tensor(slots, dtype=torch.int32).cuda(),
                               torch.tensor(pos).cuda(), gamma, theta)
    torch.cuda.synchronize()
    assert errors(o, ref) <= TOL_BF16 and errors(p, after) <= TOL_F32


def test_fp16_range_is_counted():
    """bf16 magnitudes beyond fp16's range: the outputs may be infinite and are counted; the states are not
    affected, and neither is another sequence."""
    lens, hq, kv, dk, dv = [150, 150], 2, 2, 64, 64
    fused, pool, slots, pos, gamma, theta = case(lens, hq, kv, dk, dv, "bf16", 65, pos=[0, 3])
    fused[20:40] *= 1e5
    ref, after = reference(*split(fused, hq, kv, dk, dv), pool, lens, slots, pos, gamma, theta, FLAGS)
    o, p = run(fused, pool, lens, slots, pos, gamma, theta, hq, kv, dk, dv)
    assert rn.retnet_fp16_range_errors(clear=True) > 0
    assert errors(o[150:300], ref[150:300]) <= TOL_BF16
    for s in slots:
        assert errors(p[s], after[s]) <= TOL_F32


def test_two_calls_at_once():
    """Two streams, each with its own workspace and slots, many times over: the same bits as one by one."""
    args = []
    for seed, lens, dk, dv in ((201, [300, 77, 513], 128, 128), (202, [64, 700], 64, 256)):
        fused, pool, slots, pos, gamma, theta = case(lens, 4, 4, dk, dv, "bf16", seed)
        args.append((fused, pool, lens, slots, pos, gamma, theta, 4, 4, dk, dv))
    want = [run(*a) for a in args]
    streams = [torch.cuda.Stream() for _ in args]
    outs = []
    for a, s in zip(args, streams):
        fused, pool, lens, slots, pos, gamma, theta, hq, kv, dk, dv = a
        q, k, v = split(fused.cuda(), hq, kv, dk, dv)
        outs.append([(torch.full((q.shape[0], hq, dv), 0.25, dtype=q.dtype, device="cuda"), pool.cuda()) for _ in range(6)])
        a += (q, k, v, cu_of(lens).cuda(), torch.tensor(slots, dtype=torch.int32).cuda(), torch.tensor(pos).cuda())
        args[streams.index(s)] = a
    torch.cuda.synchronize()
    for i in range(6):
        for a, s, o in zip(args, streams, outs):
            q, k, v, cu, sl, ps = a[11:]
            rn.retnet_retention_packed(q, k, v, o[i][0], o[i][1], cu, sl, ps, a[5], a[6], FLAGS, stream=s)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        for got in o:
            assert torch.equal(w[0], got[0]) and torch.equal(w[1], got[1])


def test_far_positions():
    check([200, 130], 2, 2, 64, 64, "bf16", 51, pos=[1 << 30, (1 << 33) + 7])


def test_positions_default_to_zero_and_stale_slots_are_not_read():
    """pos=None: every sequence starts from zeros, even where its slot holds NaN."""
    lens, hq, kv, dk, dv = [70, 5], 2, 2, 64, 64
    for dtype, tol in (("bf16", TOL_BF16), ("f32", TOL_F32)):
        fused, pool, slots, _, gamma, theta = case(lens, hq, kv, dk, dv, dtype, 61)
        q, k, v = split(fused, hq, kv, dk, dv)
        ref, after = reference(q, k, v, pool, lens, slots, [0, 0], gamma, theta, FLAGS)
        pool[slots] = float("nan")
        o, p = run(fused, pool, lens, slots, None, gamma, theta, hq, kv, dk, dv)
        assert errors(o, ref) <= tol and errors(p[slots], after[slots]) <= TOL_F32


def test_non_finite_rows_of_others_stay_out():
    """Rows behind the last sequence and other sequences' rows hold inf and NaN: no other output sees them."""
    lens, hq, kv, dk, dv = [100, 60, 130], 2, 2, 64, 64
    for dtype, tol in (("bf16", TOL_BF16), ("f32", TOL_F32)):
        fused, pool, slots, pos, gamma, theta = case(lens, hq, kv, dk, dv, dtype, 71)
        q, k, v = split(fused, hq, kv, dk, dv)
        ref, after = reference(q, k, v, pool, lens, slots, pos, gamma, theta, FLAGS)
        fused[100:160] = float("nan")  # the second sequence
        fused[120, :] = float("inf")
        fused[290:] = float("nan")
        o, p = run(fused, pool, lens, slots, pos, gamma, theta, hq, kv, dk, dv)
        keep = [0, 2]
        rows = list(range(100)) + list(range(160, 290))
        assert errors(o[rows], ref[rows]) <= tol
        assert errors(p[[slots[i] for i in keep]], after[[slots[i] for i in keep]]) <= TOL_F32
        assert torch.isfinite(o[rows]).all()
        assert bool((o[290:] == 0.25).all())
    rn.retnet_fp16_range_errors(clear=True)  # the second sequence's own operands are not finite


def test_padded_sequences_and_refused_ones():
    """slot -1 is left out silently; a slot out of range or named twice, or a negative position, is left
    out and counted; the others are as without them."""
    lens, hq, kv, dk, dv = [40, 30, 50, 20, 10, 60], 2, 2, 64, 64
    slots, pos = [3, -1, 99, 3, 1, 2], [0, 5, 9, 7, -4, 11]
    for dtype, tol in (("bf16", TOL_BF16), ("f32", TOL_F32)):
        fused, pool, _, _, gamma, theta = case(lens, hq, kv, dk, dv, dtype, 81)
        q, k, v = split(fused, hq, kv, dk, dv)
        used = [3, -1, -1, -1, -1, 2]
        ref, after = reference(q, k, v, pool, lens, used, [0, 0, 0, 0, 0, 11], gamma, theta, FLAGS)
        o, p = run(fused, pool, lens, slots, pos, gamma, theta, hq, kv, dk, dv)
        assert rn.retnet_slot_errors(clear=True) == 3
        assert errors(o, ref) <= tol and errors(p[[2, 3]], after[[2, 3]]) <= TOL_F32
        assert bool((o[40:210 - 60] == 0.25).all())
        assert torch.equal(p.cpu()[[0, 1, 4]], pool[[0, 1, 4]])


@pytest.mark.parametrize("cu", [[0, 50, 40, 90], [-1, 20, 30, 90], [0, 20, 30, 93], [5, 4, 3, 2]])
def test_cu_seqlens_out_of_order_do_nothing(cu):
    hq, kv, dk, dv = 2, 2, 64, 64
    for dtype in ("bf16", "f32"):
        fused, pool, slots, pos, gamma, theta = case([30, 30, 30], hq, kv, dk, dv, dtype, 91)
        q, k, v = split(fused.cuda(), hq, kv, dk, dv)
        o, p = torch.full((92, hq, dv), 0.25, dtype=q.dtype, device="cuda"), pool.cuda()
        rn.retnet_retention_packed(q, k, v, o, p, torch.tensor(cu, dtype=torch.int32).cuda(),
                                   torch.tensor(slots, dtype=torch.int32).cuda(), torch.tensor(pos).cuda(), gamma, theta)
        assert rn.retnet_slot_errors(clear=True) == 1
        assert bool((o == 0.25).all()) and torch.equal(p.cpu(), pool)


def test_empty_sequences_may_share_a_slot():
    """Padding of a batch to a fixed number of sequences: empty ones, all on slot 0."""
    lens, hq, kv, dk, dv = [0, 20, 0, 30, 0], 1, 1, 64, 64
    fused, pool, _, _, gamma, theta = case(lens, hq, kv, dk, dv, "bf16", 95)
    q, k, v = split(fused, hq, kv, dk, dv)
    slots, pos = [0, 0, 0, 2, 0], [0, 3, 0, 4, 0]
    ref, after = reference(q, k, v, pool, lens, slots, pos, gamma, theta, FLAGS)
    o, p = run(fused, pool, lens, slots, pos, gamma, theta, hq, kv, dk, dv)
    assert errors(o, ref) <= TOL_BF16 and errors(p, after) <= TOL_F32


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_in_pieces_equals_the_whole(dtype):
    """A prompt cut at odd places and continued from its slot gives the whole prompt's outputs and state."""
    total, hq, kv, dk, dv = 700, 2, 2, 64, 128
    fused, pool, slots, _, gamma, theta = case([total], hq, kv, dk, dv, dtype, 101, behind=0)
    whole, after = run(fused, pool, [total], slots, [0], gamma, theta, hq, kv, dk, dv)
    p, at = pool.clone(), 0
    outs = []
    for n in (1, 129, 256, 300, 14):
        o, p = run(fused[at:at + n], p.cpu(), [n], slots, [at], gamma, theta, hq, kv, dk, dv)
        outs.append(o)
        at += n
    tol = TOL_BF16 if dtype == "bf16" else TOL_F32
    assert errors(torch.cat(outs), whole.double().cpu().numpy()) <= 2 * tol
    assert errors(p[slots], after[slots].double().cpu().numpy()) <= TOL_F32


def test_bitwise_repeatable_and_on_its_stream():
    """The same bits on another stream, in another workspace filled with NaN, as part of a captured graph
    that is replayed with other lengths, slots and positions."""
    hq, kv, dk, dv = 2, 2, 128, 128
    lens_a, lens_b = [300, 41, 0], [129, 5, 207]
    for dtype in ("bf16", "f32"):
        fused, pool, slots, pos, gamma, theta = case(lens_a, hq, kv, dk, dv, dtype, 111)
        fused, rows = fused.cuda(), fused.shape[0]
        q, k, v = split(fused, hq, kv, dk, dv)

        def eager(lens, sl, ps):
            return run(fused, pool, lens, sl, ps, gamma, theta, hq, kv, dk, dv)
        want_a, want_b = eager(lens_a, slots, pos), eager(lens_b, slots[::-1], pos[::-1])
        ws = torch.full((rn.retnet_packed_workspace_size((rows, 3, hq, kv, dk, dv)),), 255, dtype=torch.uint8, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = run(fused, pool, lens_a, slots, pos, gamma, theta, hq, kv, dk, dv, stream=side, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(want_a, got))
        cu, sl, ps = cu_of(lens_a).cuda(), torch.tensor(slots, dtype=torch.int32).cuda(), torch.tensor(pos).cuda()
        o, p = torch.empty_like(want_a[0]), pool.cuda()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            rn.retnet_retention_packed(q, k, v, o, p, cu, sl, ps, gamma, theta, FLAGS, workspace=ws)
        for lens, s, t, want in ((lens_a, slots, pos, want_a), (lens_b, slots[::-1], pos[::-1], want_b)):
            cu.copy_(cu_of(lens))
            sl.copy_(torch.tensor(s, dtype=torch.int32))
            ps.copy_(torch.tensor(t))
            o.fill_(0.25)
            p.copy_(pool)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, want[0]) and torch.equal(p, want[1])


def test_matches_the_dense_call():
    """Equal lengths and zero starts: retnet_retention_chunkwise's results, up to its bar."""
    b, L, h, dk, dv = 3, 320, 2, 64, 64
    q, k, v = si.qkv(b, L, h, dk, dv, 121, "bf16")
    g, th = si.gamma_schedule(h), si.theta_schedule(dk)
    dense, so, _ = rn.retention_chunkwise(q.cuda(), k.cuda(), v.cuda(), g, th, 64, FLAGS, return_state=True)
    o, pool = torch.empty(b * L, h, dv, dtype=torch.bfloat16, device="cuda"), torch.empty(b, h, dk, dv, device="cuda")
    rn.retnet_retention_packed(q.cuda().flatten(0, 1), k.cuda().flatten(0, 1), v.cuda().flatten(0, 1), o, pool,
                               cu_of([L] * b).cuda(), torch.arange(b, dtype=torch.int32).cuda(), None, g, th)
    torch.cuda.synchronize()
    assert errors(o.view(b, L, h, dv), dense.double().cpu().numpy()) <= 2 * TOL_BF16
    assert errors(pool, so.double().cpu().numpy()) <= TOL_BF16


def test_many_sequences():
    """More sequences than a plan's threads, lengths 0 to 9, and a pool past 2^31 bytes."""
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 10, 700).tolist()
    hq, kv, dk, dv = 2, 1, 64, 64
    n_slots = 140000  # 140000 * 16 KB = 2.3 GB
    slots = (n_slots - 1 - rng.permutation(1000)[:700]).tolist()
    fused, _, _, pos, gamma, theta = case(lens, hq, kv, dk, dv, "bf16", 131, slots=slots, n_slots=1)
    q, k, v = split(fused, hq, kv, dk, dv)
    small = si.randn((1000, kv, dk, dv), 132, "f32")
    ref, after = reference(q, k, v, small, lens, [s - (n_slots - 1000) for s in slots], pos, gamma, theta, FLAGS)
    p = torch.zeros(n_slots, kv, dk, dv, device="cuda")
    p[-1000:] = small.cuda()
    o = torch.full((fused.shape[0], hq, dv), 0.25, dtype=torch.bfloat16, device="cuda")
    rn.retnet_retention_packed(*split(fused.cuda(), hq, kv, dk, dv), o, p, cu_of(lens).cuda(),
                               torch.tensor(slots, dtype=torch.int32).cuda(), torch.tensor(pos).cuda(), gamma, theta)
    torch.cuda.synchronize()
    assert errors(o, ref) <= TOL_BF16 and errors(p[-1000:], after) <= TOL_F32
    assert not p[:-1000].any()


@pytest.mark.parametrize("length,kv,dk,dv,dtype,gamma,run_of,start", [
    (256, 1, 64, 64, "bf16", 0.94, 128, 0),    # tensor cores, a walk by sequence
    (640, 1, 64, 64, "bf16", 0.94, 128, 70),   # chunk by chunk, then the scan
    (240, 1, 64, 64, "bf16", 0.94, 128, 70),   # a short last chunk
    (128, 2, 64, 64, "f32", 0.8, 64, 0),       # CUDA cores
    (512, 1, 256, 128, "f32", 0.8, 256, 70),
])
def test_small_after_large(length, kv, dk, dv, dtype, gamma, run_of, start):
    """A state that was 2^12 times larger a run ago leaves no rounding of that size behind: every entry
    within 2e-5 of the decayed sum of magnitudes (128 fp32 additions of at most 2^-23 each, 1.5e-5, and
    a few 1e-7 for the decay factors, exponents up to 12 in fp32)."""
    fused, pool, slots, _, _, theta = case([length], kv, kv, dk, dv, dtype, length + dk, behind=0)
    last = (length - 1) // run_of * run_of
    fused[last - run_of:last, kv * dk:] *= 64.0  # k and v
    g = np.full(kv, gamma, dtype=np.float32)
    q, k, v = split(fused, kv, kv, dk, dv)
    assert rn.retnet_packed_kernel((length, 1, kv, kv, dk, dv), rn.BF16 if dtype == "bf16" else rn.F32, 0, g) == (dtype == "bf16")
    _, p = run(fused, pool, [length], slots, [start], g, theta, kv, kv, dk, dv, flags=0)
    decay = g.astype(np.float64)[:, None] ** np.arange(length - 1, -1, -1)  # (kv, length)
    k64, v64 = k.double().numpy(), v.double().numpy()
    before = pool[slots[0]].double().numpy() * (g.astype(np.float64) ** length)[:, None, None] * (start > 0)
    ref = np.einsum("ht,thi,thj->hij", decay, k64, v64) + before
    size = np.einsum("ht,thi,thj->hij", decay, abs(k64), abs(v64)) + abs(before)
    err = (abs(p[slots[0]].double().cpu().numpy() - ref) / size).max()
    print(f"{err:.2e}")
    assert err <= 2e-5


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_positions_up_to_the_limit(dtype):
    """The largest position is computed (frequencies that are powers of two: exact angles in the
    reference); one more is left out and counted."""
    lens, hq, kv, dk, dv = [150, 20, 1], 2, 2, 64, 64
    theta = (2.0 ** -np.arange(dk // 2)).astype(np.float32)
    fused, pool, slots, _, gamma, _ = case(lens, hq, kv, dk, dv, dtype, 111)
    q, k, v = split(fused, hq, kv, dk, dv)
    used = [slots[0], -1, slots[2]]
    pos = [rn.MAX_POSITION, rn.MAX_POSITION + 1, rn.MAX_POSITION]
    ref, after = reference(q, k, v, pool, lens, used, pos, gamma, theta, FLAGS)
    o, p = run(fused, pool, lens, slots, pos, gamma, theta, hq, kv, dk, dv)
    assert rn.retnet_slot_errors(clear=True) == 1
    assert errors(o, ref) <= (TOL_BF16 if dtype == "bf16" else TOL_F32) and errors(p, after) <= TOL_F32
    assert bool((o[150:170] == 0.25).all()) and torch.equal(p[slots[1]].cpu(), pool[slots[1]])
