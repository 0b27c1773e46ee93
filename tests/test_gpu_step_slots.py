"""The single-token form over pool slots (retnet_retention_step_slots) and slot copies
(retnet_state_slots_copy) against the fp64 oracle, and a serving run of them together.

Bars, max|err|/rms: 1e-4 for fp32 results and the pool; bf16 outputs 1e-4 net of their own rounding
(fp32 arithmetic on exact bf16 inputs).
"""
import numpy as np
import pytest
import torch

import linear_attention_sequence_chunkwise_b200 as rn
import oracle
import synth_inputs as si
from gpu_util import TOL_BF16, TOL_F32, require_gpu
from serving_util import FLAGS, case, cu_of, errors, reference, split

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(cuda_lib):
    require_gpu()
    rn.retnet_slot_errors(clear=True)
    yield
    assert rn.retnet_slot_errors(clear=True) == 0


def step(fused, pool, slots, pos, gamma, theta, hq, kv, dk, dv, flags=FLAGS):
    q, k, v = split(fused.cuda(), hq, kv, dk, dv)
    o, p = torch.full((q.shape[0], hq, dv), 0.25, dtype=q.dtype, device="cuda"), pool.cuda()
    rn.retnet_retention_step_slots(q, k, v, o, p, torch.tensor(slots, dtype=torch.int32).cuda(),
                                   None if pos is None else torch.tensor(pos).cuda(), gamma, theta, flags)
    torch.cuda.synchronize()
    return o, p


@pytest.mark.parametrize("rows,hq,kv,dk,dv,dtype", [
    (1, 1, 1, 64, 64, "bf16"), (3, 8, 8, 128, 128, "bf16"), (64, 4, 4, 256, 512, "bf16"), (37, 16, 4, 100, 130, "f32"),
    (5, 2, 1, 64, 36, "f32"), (2, 12, 2, 48, 33, "bf16"), (2, 16, 1, 66, 64, "f32"), (3, 24, 1, 128, 128, "bf16"),
    (1, 1, 1, 1, 1, "f32"), (2, 2, 2, 7, 3, "f32"), (1, 9, 1, 512, 1024, "bf16"), (80, 8, 4, 128, 128, "bf16")])
def test_step_matches_oracle(rows, hq, kv, dk, dv, dtype):
    flags = FLAGS if dk % 2 == 0 else rn.F_SCALE_SQRT_D | rn.F_NORM_D
    fused, pool, slots, pos, gamma, theta = case([1] * rows, hq, kv, dk, dv, dtype, 11 * dk + dv + rows, behind=0)
    if rows >= 5:
        slots[1] = slots[-1] = -1
    q, k, v = split(fused, hq, kv, dk, dv)
    ref, after = reference(q, k, v, pool, [1] * rows, slots, pos, gamma, theta, flags)
    o, p = step(fused, pool, slots, pos, gamma, theta, hq, kv, dk, dv, flags)
    eo, ep = errors(o, ref), errors(p, after)
    print(f"step rows={rows} h={hq}/{kv} dk={dk} dv={dv} {dtype}: o {eo:.2e} pool {ep:.2e}")
    assert eo <= TOL_F32 and ep <= TOL_F32
    idle = torch.from_numpy(np.isnan(ref).all(axis=(1, 2)))
    assert bool((o.cpu()[idle] == 0.25).all())
    rest = [s for s in range(pool.shape[0]) if s not in slots]
    assert torch.equal(p.cpu()[rest], pool[rest])


def test_step_refuses_bad_rows():
    hq, kv, dk, dv = 2, 2, 64, 64
    fused, pool, _, _, gamma, theta = case([1] * 6, hq, kv, dk, dv, "f32", 5, behind=0, n_slots=7)
    slots, pos = [2, 7, 2, -1, 4, 5], [3, 4, 5, -9, -1, 0]
    pool[5] = float("nan")  # position 0: not read
    q, k, v = split(fused, hq, kv, dk, dv)
    ref, after = reference(q, k, v, pool, [1] * 6, [2, -1, -1, -1, -1, 5], [3, 0, 0, 0, 0, 0], gamma, theta, FLAGS)
    o, p = step(fused, pool, slots, pos, gamma, theta, hq, kv, dk, dv)
    assert rn.retnet_slot_errors(clear=True) == 3  # 7 is out of range, 2 again, position -1
    assert errors(o, ref) <= TOL_F32 and errors(p, after) <= TOL_F32
    assert bool((o[1:5] == 0.25).all())


def test_step_without_positions_and_at_far_ones():
    hq, kv, dk, dv = 2, 2, 64, 64
    fused, pool, slots, _, gamma, theta = case([1] * 3, hq, kv, dk, dv, "f32", 6, behind=0)
    q, k, v = split(fused, hq, kv, dk, dv)
    for pos in (None, [1 << 31, (1 << 40) + 3, 1]):
        ref, after = reference(q, k, v, pool, [1] * 3, slots, pos or [0] * 3, gamma, theta, FLAGS)
        o, p = step(fused, pool, slots, pos, gamma, theta, hq, kv, dk, dv)
        assert errors(o, ref) <= TOL_F32 and errors(p, after) <= TOL_F32


def test_step_positions_up_to_the_limit():
    hq, kv, dk, dv = 2, 2, 64, 64
    theta = (2.0 ** -np.arange(dk // 2)).astype(np.float32)  # exact angles in the reference
    fused, pool, slots, _, gamma, _ = case([1] * 3, hq, kv, dk, dv, "f32", 9, behind=0)
    q, k, v = split(fused, hq, kv, dk, dv)
    pos = [rn.MAX_POSITION, rn.MAX_POSITION + 1, 3]
    ref, after = reference(q, k, v, pool, [1] * 3, [slots[0], -1, slots[2]], pos, gamma, theta, FLAGS)
    o, p = step(fused, pool, slots, pos, gamma, theta, hq, kv, dk, dv)
    assert rn.retnet_slot_errors(clear=True) == 1
    assert errors(o, ref) <= TOL_F32 and errors(p, after) <= TOL_F32 and bool((o[1] == 0.25).all())


def test_pool_past_32_bit_offsets():
    """Slots behind 2^31 floats (8.6 GB) are reached by the step and by the copy."""
    kv, dk, dv = 1, 256, 512
    n = (1 << 31) // (kv * dk * dv) + 3
    pool = torch.zeros(n, kv, dk, dv, device="cuda")
    first = si.randn((kv, dk, dv), 7, "f32")
    pool[n - 1] = first.cuda()
    fused, _, _, _, gamma, theta = case([1], 1, kv, dk, dv, "bf16", 8, behind=0, slots=[0], n_slots=1)
    q, k, v = split(fused, 1, kv, dk, dv)
    ref, after = reference(q, k, v, first[None], [1], [0], [9], gamma, theta, FLAGS)
    o = torch.empty(1, 1, dv, dtype=torch.bfloat16, device="cuda")
    rn.retnet_retention_step_slots(*(x.cuda() for x in (q, k, v)), o, pool,
                                   torch.tensor([n - 1], dtype=torch.int32).cuda(), torch.tensor([9]).cuda(), gamma, theta)
    rn.retnet_state_slots_copy(pool, torch.tensor([n - 1], dtype=torch.int32).cuda(),
                               torch.tensor([n - 2], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert errors(o, ref) <= TOL_F32
    assert errors(pool[n - 1], after[0]) <= TOL_F32 and torch.equal(pool[n - 2], pool[n - 1])
    assert not pool[:2].any()


# ---- slot copies: exact -----------------------------------------------------------------------

def copy_ref(pool, src, dst, n_slots):
    out, seen, bad = pool.clone(), set(), 0
    for s, d in zip(src, dst):
        if d < 0:
            continue
        dup = d in seen
        seen.add(d)
        if d >= n_slots or s >= n_slots or dup:
            bad += 1
            continue
        out[d] = pool[s] if s >= 0 else 0.0
    return out, bad


def copy_case(kind, n, slots, rng):
    order = rng.permutation(slots).tolist()
    if kind == "fork":
        return [order[0]] * n, order[1:n + 1]
    if kind == "compact":
        return order[:n], order[n:2 * n]
    if kind == "rotate":
        return order[:n], order[1:n] + order[:1]
    if kind == "beam":
        return [int(rng.choice(order[:n])) for _ in range(n)], order[:n]
    if kind == "free":
        return [-1] * n, order[:n]
    return [-1 if i % 3 == 0 else int(rng.choice(order[:n])) for i in range(n)], \
        [-1 if i % 4 == 3 else order[i] for i in range(n)]


@pytest.mark.parametrize("kind", ["fork", "compact", "rotate", "beam", "free", "mixed"])
@pytest.mark.parametrize("n,shape", [(1, (1, 16, 8)), (2, (3, 7, 5)), (7, (8, 128, 128)), (65, (2, 33, 31)), (300, (1, 20, 12)),
                                     (1024, (1, 4, 6)), (1024, (1, 64, 64))])
def test_slots_copy(kind, n, shape):
    rng = np.random.default_rng(n)
    slots = 2 * n + 1
    pool = si.randn((slots, *shape), n, "f32")
    src, dst = copy_case(kind, n, slots, rng)
    want, bad = copy_ref(pool, src, dst, slots)
    assert bad == 0
    p = pool.cuda()
    rn.retnet_state_slots_copy(p, torch.tensor(src, dtype=torch.int32).cuda(), torch.tensor(dst, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert torch.equal(p.cpu(), want)


def test_slots_copy_refuses_bad_pairs():
    pool = si.randn((6, 1, 8, 8), 3, "f32")
    src, dst = [0, 1, 9, 3, 2, -1, 4], [1, 1, 2, 6, -1, 0, 4]
    want, bad = copy_ref(pool, src, dst, 6)
    p = pool.cuda()
    rn.retnet_state_slots_copy(p, torch.tensor(src, dtype=torch.int32).cuda(), torch.tensor(dst, dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert bad == 3 and rn.retnet_slot_errors(clear=True) == 3
    assert torch.equal(p.cpu(), want)


# ---- together ---------------------------------------------------------------------------------

def test_serving_run():
    """Two prompts of ragged lengths, the first forked into three samples, five decode steps of all four
    sequences, a beam reorder in place, three more steps (captured and replayed), then one sequence freed:
    every output and state against the oracle run over each sequence's whole history."""
    hq, kv, dk, dv = 4, 2, 64, 64
    lens = [150, 37]
    fused, pool, _, _, gamma, theta = case(lens, hq, kv, dk, dv, "bf16", 200, behind=0, n_slots=6)
    pool[:] = float("nan")  # nothing in a slot is read before it was written
    o, p = torch.empty(187, hq, dv, dtype=torch.bfloat16, device="cuda"), pool.cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    q, k, v = split(fused.cuda(), hq, kv, dk, dv)
    rn.retnet_retention_packed(q, k, v, o, p, cu_of(lens).cuda(), i32([4, 1]), None, gamma, theta)
    rn.retnet_state_slots_copy(p, i32([4, 4]), i32([0, 5]))
    seqs = [4, 0, 5, 1]  # slots
    history = {0: [fused[:150]], 1: [fused[:150]], 2: [fused[:150]], 3: [fused[150:]]}
    pos = torch.tensor([150, 150, 150, 37]).cuda()
    tokens = torch.empty(5, fused.shape[1], dtype=torch.bfloat16, device="cuda")
    tq, tk, tv = split(tokens, hq, kv, dk, dv)
    ot = torch.zeros(5, hq, dv, dtype=torch.bfloat16, device="cuda")
    slots = i32(seqs + [-1])  # a row of padding
    pos = torch.cat((pos, pos[:1]))

    def call():
        rn.retnet_retention_step_slots(tq, tk, tv, ot, p, slots, pos, gamma, theta)
        pos.add_(1)

    def check_step(i):
        for r in range(4):
            h = torch.cat(history[r])
            a, b, c = split(h, hq, kv, dk, dv)
            empty = torch.zeros(1, kv, dk, dv)
            ref, after = reference(a, b, c, empty, [len(h)], [0], [0], gamma, theta, FLAGS)
            # the state comes from a packed prompt on 16-bit operands at most: its bar is TOL_BF16's
            assert errors(ot[r], ref[-1]) <= TOL_BF16, (i, r)
            assert errors(p[seqs[r]], after[0]) <= TOL_F32, (i, r)

    def new_tokens(i):
        t = si.randn((5, fused.shape[1]), 300 + i, "bf16")
        tokens.copy_(t)
        for r in range(4):
            history[r].append(t[r:r + 1])
    for i in range(5):
        new_tokens(i)
        call()
        torch.cuda.synchronize()
        check_step(i)
    # rows 0..2 become copies of rows 2, 0, 2; in place
    rn.retnet_state_slots_copy(p, i32([5, 4, 5]), i32([4, 0, 5]))
    history[0], history[1], history[2] = list(history[2]), list(history[0]), list(history[2])
    graph = torch.cuda.CUDAGraph()
    at = pos.clone()
    with torch.cuda.graph(graph):
        call()
    assert torch.equal(pos, at)  # capturing ran nothing
    for i in range(5, 8):
        new_tokens(i)
        graph.replay()
        torch.cuda.synchronize()
        check_step(i)
    assert not ot[4].any()
    rn.retnet_state_slots_copy(p, i32([-1]), i32([1]))
    torch.cuda.synchronize()
    assert not p[1].any() and torch.isnan(p[[2, 3]]).all()


def test_calls_right_behind_one_another():
    """Launches overlap their predecessor's tail: a chain of all the calls, each reading what the one before
    wrote, gives the same bits unsynchronised, with a synchronisation after every call, and captured."""
    hq, kv, dk, dv = 4, 4, 128, 128
    lens = [90, 0, 300, 1]
    fused, pool, _, _, gamma, theta = case(lens, hq, kv, dk, dv, "bf16", 210, behind=0, n_slots=8)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    x = fused.cuda()
    q, k, v = split(x, hq, kv, dk, dv)
    cu, slots, back, rows = cu_of(lens).cuda(), i32([0, 1, 2, 3]), i32([4, 5, 6, 7]), i32([4, 6, 7])
    pos = torch.full((4,), 5).cuda()
    w, b = torch.rand(hq, dv, device="cuda"), torch.rand(hq, dv, device="cuda")
    ws = torch.empty(rn.retnet_packed_workspace_size((q.shape[0], 4, hq, kv, dk, dv)), dtype=torch.uint8, device="cuda")

    def chain(p, o, sync):
        for _ in range(4):
            for call in (lambda: rn.retnet_retention_packed(q, k, v, o, p, cu, slots, pos, gamma, theta, workspace=ws),
                         lambda: rn.retnet_state_slots_copy(p, slots, back),
                         lambda: rn.retnet_retention_step_slots(q[:3], k[:3], v[:3], o[:3], p, rows, pos[:3], gamma, theta),
                         lambda: rn.retnet_msr_affine(o, o, w, b, o),
                         lambda: rn.retnet_state_slots_copy(p, back, slots)):
                call()
                if sync:
                    torch.cuda.synchronize()
    results = []
    for how in ("sync", "eager", "graph"):
        p, o = pool.cuda(), torch.zeros(q.shape[0], hq, dv, dtype=torch.bfloat16, device="cuda")
        if how == "graph":
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                chain(p, o, False)
            graph.replay()
        else:
            chain(p, o, how == "sync")
        torch.cuda.synchronize()
        results.append((p, o))
    for p, o in results[1:]:
        assert torch.equal(p, results[0][0]) and torch.equal(o, results[0][1])
    assert torch.isfinite(results[0][0]).all() and torch.isfinite(results[0][1]).all()


def test_captured_behind_copies_and_joined_streams():
    """Each call captured right behind a memset, a copy and a join with another stream's work, and read by a
    copy right behind it: replays give the eager results."""
    hq, kv, dk, dv = 2, 2, 64, 64
    lens = [30, 200]
    fused, pool, _, _, gamma, theta = case(lens, hq, kv, dk, dv, "bf16", 220, behind=0, n_slots=4)
    source, start = fused.cuda(), pool.cuda()
    x, p = torch.empty_like(source), torch.empty_like(start)
    q, k, v = split(x, hq, kv, dk, dv)
    i32 = lambda t: torch.tensor(t, dtype=torch.int32).cuda()  # noqa: E731
    cu, slots, other, pos = cu_of(lens).cuda(), i32([0, 3]), i32([1, 2]), torch.tensor([4, 0]).cuda()
    w = torch.rand(hq, dv, device="cuda")
    o, kept = torch.empty(230, hq, dv, dtype=torch.bfloat16, device="cuda"), [torch.empty_like(start) for _ in range(3)]
    out, last = torch.empty_like(o), torch.empty_like(o)
    ws = torch.empty(rn.retnet_packed_workspace_size((230, 2, hq, kv, dk, dv)), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()

    def work():
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            x.copy_(source)
        p.copy_(start)
        o.zero_()
        here.wait_stream(side)
        rn.retnet_retention_packed(q, k, v, o, p, cu, slots, pos, gamma, theta, workspace=ws)
        kept[0].copy_(p)
        rn.retnet_state_slots_copy(p, slots, other)
        kept[1].copy_(p)
        o[:2].zero_()
        rn.retnet_retention_step_slots(q[:2], k[:2], v[:2], o[:2], p, other, pos, gamma, theta)
        kept[2].copy_(p)
        out.zero_()
        rn.retnet_msr_affine(o, q.contiguous(), w, None, out)
        last.copy_(out)
    work()
    torch.cuda.synchronize()
    want = [t.clone() for t in (*kept, last)]
    for t in (*kept, last, x, p, o, out):
        t.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, (*kept, last)):
        assert torch.equal(a, b)


def test_step_equals_packed_of_one_token():
    hq, kv, dk, dv = 4, 2, 64, 64
    fused, pool, slots, pos, gamma, theta = case([1] * 9, hq, kv, dk, dv, "f32", 15, behind=0)
    o, p = step(fused, pool, slots, pos, gamma, theta, hq, kv, dk, dv)
    q, k, v = split(fused.cuda(), hq, kv, dk, dv)
    o2, p2 = torch.empty_like(o), pool.cuda()
    rn.retnet_retention_packed(q, k, v, o2, p2, cu_of([1] * 9).cuda(), torch.tensor(slots, dtype=torch.int32).cuda(),
                               torch.tensor(pos).cuda(), gamma, theta)
    torch.cuda.synchronize()
    assert errors(o2, o.double().cpu().numpy()) <= TOL_F32 and errors(p2, p.double().cpu().numpy()) <= TOL_F32


def test_oracle_is_the_dense_step():
    """The reference used here agrees with the oracle called on a dense batch (a check of the test)."""
    fused, pool, slots, _, gamma, theta = case([1, 1], 2, 2, 16, 8, "f32", 16, behind=0)
    q, k, v = split(fused, 2, 2, 16, 8)
    ref, after = reference(q, k, v, pool, [1, 1], slots, [4, 4], gamma, theta, FLAGS)
    o, s, _ = oracle.recurrent(q[:, None], k[:, None], v[:, None], gamma, theta, 4, FLAGS, pool[slots])
    assert np.allclose(ref, o[:, 0]) and np.allclose(after[slots], s)
