"""Cases and plain forms of the packed-serving and MSR-training operators.

Four operators, by the field "op" of a case:
  packed  retention (linear attention with a decay per head) over prompts of ragged lengths packed in one
          token axis, each continuing from or starting a state slot of a pool
  step    one token for each of many sequences, every row with its own slot and position
  slots   copying, forking, compacting and freeing the pool's slots
  msr     the MSR epilogue with a learnable affine, swish(g) * (w * GroupNorm_h(y) + b), forward
          alone or forward and backward

``run`` computes them in elementary torch operations in fp32 (angles and decay exponents in fp64), or, where
``own`` is true, by the calls a user makes.  ``exact`` evaluates the definitions token by token in fp64.
"""
import math
import random

import torch

own = False

CHUNK = 128  # tokens a chunk of the plain chunked form
EPS = 1e-5
XPOS, SCALE, NORM_D = 1, 2, 4
FLAGS = XPOS | SCALE | NORM_D
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # a few short prompts and continued turns (one of them empty, one of a single token): latency counts
        dict(name="packed_turns", op="packed", dtype="bf16", tokens=157, seqs=6, heads=8, heads_kv=8, d_k=128, d_v=128,
             slots=16, mix=1),
        # a prefill batch of ragged prompts at the eight-head 128-wide configuration
        dict(name="packed_prompts", op="packed", dtype="bf16", tokens=12289, seqs=9, heads=8, heads_kv=8, d_k=128,
             d_v=128, slots=24, mix=2),
        # two long documents at the sixteen-head configuration (d_k 256, d_v 512)
        dict(name="packed_documents", op="packed", dtype="bf16", tokens=16381, seqs=2, heads=16, heads_kv=16, d_k=256,
             d_v=512, slots=4, mix=3),
        # fp32, odd widths, keys and values shared by groups of four query heads
        dict(name="packed_shared_f32", op="packed", dtype="f32", tokens=2999, seqs=5, heads=8, heads_kv=2, d_k=80,
             d_v=120, slots=8, mix=4),
        # three conversations answering at once: latency counts
        dict(name="step_few", op="step", dtype="bf16", rows=3, padded=0, heads=8, heads_kv=8, d_k=128, d_v=128, slots=9),
        # the decode batch of 64 at the sixteen-head configuration, two of its rows padding
        dict(name="step_batch", op="step", dtype="bf16", rows=64, padded=2, heads=16, heads_kv=16, d_k=256, d_v=512,
             slots=80),
        # fp32, odd widths, shared keys and values
        dict(name="step_shared_f32", op="step", dtype="f32", rows=37, padded=3, heads=16, heads_kv=4, d_k=100, d_v=130,
             slots=50),
        # one prompt's state forked into a few samples
        dict(name="slots_fork", op="slots", kind="fork", pairs=4, heads_kv=8, d_k=128, d_v=128, slots=12),
        # a beam reorder in place, frees among it, at the sixteen-head configuration
        dict(name="slots_reorder", op="slots", kind="reorder", pairs=61, heads_kv=16, d_k=256, d_v=512, slots=72),
        # the epilogue of one decode batch: latency counts
        dict(name="msr_decode", op="msr", dtype="bf16", tokens=64, heads=16, d_v=512, train=False),
        # a training step's epilogue at the eight-head 256-wide configuration, forward and backward
        dict(name="msr_train", op="msr", dtype="bf16", tokens=16384, heads=8, d_v=256, train=True),
        # the same in fp32 at odd sizes
        dict(name="msr_train_f32", op="msr", dtype="f32", tokens=1501, heads=6, d_v=100, train=True),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["packed", "packed", "step", "slots", "msr", "msr"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    kv = rng.randint(1, 8)
    group = rng.choice([1, 1, 2, 4]) if kv <= 4 else 1
    if op == "packed":
        big = dtype == "bf16"
        return dict(op=op, dtype=dtype, tokens=_log_uniform(rng, 24, 9000 if big else 2500), seqs=rng.randint(1, 12),
                    heads=kv * group, heads_kv=kv, d_k=rng.choice([64, 128, 256] if big else [16, 48, 64, 90]),
                    d_v=rng.choice([64, 128, 192, 256] if big else [24, 64, 101, 128]), slots=16,
                    mix=rng.randint(0, 1 << 20))
    if op == "step":
        rows = _log_uniform(rng, 1, 60)
        return dict(op=op, dtype=dtype, rows=rows, padded=rng.randint(0, rows // 4), heads=kv * group, heads_kv=kv,
                    d_k=2 * rng.randint(8, 128), d_v=rng.choice([rng.randint(16, 256), 64 * rng.randint(1, 4)]),
                    slots=rows + rng.randint(0, 12))
    if op == "slots":
        pairs = _log_uniform(rng, 2, 120)
        return dict(op=op, kind=rng.choice(["fork", "reorder", "compact"]), pairs=pairs, heads_kv=kv,
                    d_k=2 * rng.randint(8, 64), d_v=2 * rng.randint(8, 64), slots=2 * pairs + rng.randint(0, 20))
    return dict(op=op, dtype=dtype, tokens=_log_uniform(rng, 1, 8000), heads=rng.randint(1, 8),
                d_v=rng.choice([rng.randint(8, 256), 64 * rng.randint(1, 4)]), train=rng.random() < 0.7)


def _lengths(case):
    """Ragged lengths that sum to case["tokens"], an empty one and one of a single token where there are enough."""
    n, total = case["seqs"], case["tokens"]
    rng = random.Random(case["mix"])
    lens = [0] * n
    if n >= 4:
        lens[1], lens[2] = 1, 0
    free = [i for i in range(n) if not (n >= 4 and i in (1, 2))]
    weights = [math.exp(rng.uniform(0.0, 1.5)) for _ in free]
    left = total - sum(lens)
    for i, w in zip(free, weights):
        lens[i] = int(left * w / sum(weights))
    lens[free[-1]] += total - sum(lens)
    return lens


def _continues(i):
    """Whether sequence i starts from a state in its slot (two of three do) or at position 0."""
    return i % 3 != 0


def _schedules(heads, d_k):
    gamma = torch.tensor([1.0 - 2.0 ** (-5 - i) for i in range(heads)], dtype=torch.float32)
    theta = torch.tensor([10000.0 ** (-2.0 * j / d_k) for j in range(d_k // 2)], dtype=torch.float32)
    return gamma, theta


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    rng = random.Random(int(seed))
    op = case["op"]

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)

    if op == "msr":
        dt, shape = DTYPES[case["dtype"]], (case["tokens"], case["heads"], case["d_v"])
        s = dict(case=dict(case), y=normal(*shape, dtype=dt), g=normal(*shape, dtype=dt),
                 weight=1.0 + 0.2 * normal(*shape[1:]), bias=0.2 * normal(*shape[1:]))
        if case["train"]:
            s["dout"] = normal(*shape, dtype=dt)
        return s

    kv, dk, dv, slots = case["heads_kv"], case["d_k"], case["d_v"], case["slots"]
    pool = 2.0 * normal(slots, kv, dk, dv)
    if op == "slots":
        n, kind = case["pairs"], case["kind"]
        order = rng.sample(range(slots), slots)
        if kind == "fork":  # one live slot into n free ones
            src, dst = [order[0]] * n, order[1:n + 1]
        elif kind == "compact":  # live slots into free ones; the slots left behind are not touched
            src, dst = order[:n], order[n:2 * n]
        else:  # a beam's parents: any slot of the beam, several times or not at all; some are freed
            dst = order[:n]
            src = [-1 if rng.random() < 0.1 else rng.choice(dst) for _ in range(n)]
        return dict(case=dict(case), pool=pool, src=torch.tensor(src, dtype=torch.int32, device="cuda"),
                    dst=torch.tensor(dst, dtype=torch.int32, device="cuda"))

    dt, hq = DTYPES[case["dtype"]], case["heads"]
    gamma, theta = _schedules(kv, dk)
    if op == "packed":
        lens = _lengths(case)
        n, rows = len(lens), case["tokens"] + 3  # three rows of padding behind the last sequence
        cu = [0]
        for x in lens:
            cu.append(cu[-1] + x)
        pos = [rng.randint(1, 6000) if _continues(i) else 0 for i in range(n)]
        index = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), longest=max(lens))
    else:
        n = rows = case["rows"]
        pos = [rng.randint(1, 9000) if _continues(i) else 0 for i in range(n)]
        index = {}
    slot = rng.sample(range(slots), n)
    if op == "step" and case["padded"]:  # the batch's last rows hold no sequence
        slot[n - case["padded"]:] = [-1] * case["padded"]
    # q, k, v are views of one fused projection's output
    fused = normal(rows, (hq + kv) * dk + kv * dv, dtype=dt)
    q = fused[:, :hq * dk].unflatten(1, (hq, dk))
    k = fused[:, hq * dk:(hq + kv) * dk].unflatten(1, (kv, dk))
    v = fused[:, (hq + kv) * dk:].unflatten(1, (kv, dv))
    return dict(case=dict(case), q=q, k=k, v=v, o=torch.full((rows, hq, dv), 0.5, dtype=dt, device="cuda"), pool=pool,
                slots=torch.tensor(slot, dtype=torch.int32, device="cuda"),
                pos=torch.tensor(pos, dtype=torch.int64, device="cuda"), gamma=gamma.numpy(), theta=theta.numpy(),
                gamma_dev=gamma.cuda(), theta_dev=theta.cuda(), **index)


# ---- the framework's calls -----------------------------------------------------------------

def _run_own(s):
    import linear_attention_sequence_chunkwise_b200 as rn
    case = s["case"]
    if case["op"] == "packed":
        rn.retnet_retention_packed(s["q"], s["k"], s["v"], s["o"], s["pool"], s["cu_seqlens"], s["slots"], s["pos"],
                                   s["gamma"], s["theta"], FLAGS)
        return {"o": s["o"], "pool": s["pool"]}
    if case["op"] == "step":
        rn.retnet_retention_step_slots(s["q"], s["k"], s["v"], s["o"], s["pool"], s["slots"], s["pos"], s["gamma"],
                                       s["theta"], FLAGS)
        return {"o": s["o"], "pool": s["pool"]}
    if case["op"] == "slots":
        rn.retnet_state_slots_copy(s["pool"], s["src"], s["dst"])
        return {"pool": s["pool"]}
    out = rn.msr_affine(s["y"], s["g"], s["weight"], s["bias"], EPS)
    if not case["train"]:
        return {"out": out}
    dy, dg, dw, db = rn.msr_affine_backward(s["y"], s["g"], s["weight"], s["bias"], s["dout"], EPS)
    return {"out": out, "dy": dy, "dg": dg, "dweight": dw, "dbias": db}


# ---- the plain forms -----------------------------------------------------------------------

def _rotate(x, angle):
    """Pairs (2j, 2j+1) of x's last axis turned by angle (fp64, broadcast over x's leading axes)."""
    c, n = torch.cos(angle).float(), torch.sin(angle).float()
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack((a * c - b * n, a * n + b * c), dim=-1).flatten(-2)


def _power(gamma, n):
    """gamma^n in fp64; n any broadcastable integer tensor."""
    return torch.exp(torch.log(gamma.double()) * n)


def _row_factor(gamma, d_k, p):
    """1/sqrt(d_k) / c_p, c_p^2 = sum_{j<=p} gamma^j, in fp64."""
    return torch.rsqrt((1.0 - _power(gamma, p + 1)) / (1.0 - gamma.double())) / math.sqrt(d_k)


def _packed(s):
    case, q, k, v, pool, o = s["case"], s["q"], s["k"], s["v"], s["pool"], s["o"]
    rows, hq, dk = q.shape
    kv, dv = v.shape[1:]
    G, C = hq // kv, CHUNK
    gamma, theta, pos = s["gamma_dev"], s["theta_dev"].double(), s["pos"]
    start, lens = s["cu_seqlens"][:-1].long(), (s["cu_seqlens"][1:] - s["cu_seqlens"][:-1]).long()
    n, m = len(lens), -(-s["longest"] // C)
    c0 = torch.arange(m, device="cuda") * C  # a chunk's first token
    r = torch.arange(C, device="cuda")
    t = c0[:, None] + r  # (m, C): token of its sequence
    valid = t < lens[:, None, None]  # (n, m, C)
    tok = torch.where(valid, start[:, None, None] + t, 0)
    p = pos[:, None, None] + t
    angle = p.double()[..., None, None] * theta  # (n, m, C, 1, dk/2)
    keep = valid[..., None, None]
    qc = torch.where(keep, _rotate(q[tok].float(), angle), 0.0).unflatten(3, (kv, G))  # (n, m, C, kv, G, dk)
    kc = torch.where(keep, _rotate(k[tok].float(), angle), 0.0)  # (n, m, C, kv, dk)
    vc = torch.where(keep, v[tok].float(), 0.0)
    # every chunk's own state, decayed to its end; then the states before each chunk
    end = torch.minimum(c0 + C, lens[:, None])  # (n, m)
    left = (end[..., None] - 1 - t).clamp(min=0)  # tokens behind t in its chunk
    own_state = torch.einsum("nmchd,nmche->nmhde", kc * _power(gamma, left[..., None]).float()[..., None], vc)
    slots = s["slots"].long()
    first = torch.where((pos > 0)[:, None, None, None], pool[slots], 0.0)  # (n, kv, dk, dv)
    gap = c0[:, None] - c0[None, :] - C  # tokens between the end of chunk c' and the start of chunk c
    between = torch.where((gap >= 0)[..., None], _power(gamma, gap.clamp(min=0)[..., None]), 0.0).float()
    before = torch.einsum("cxh,nxhde->nchde", between, own_state)
    before = before + _power(gamma, c0[:, None]).float()[..., None, None] * first[:, None]
    rest = (lens[:, None] - end).clamp(min=0)
    last = torch.einsum("nmh,nmhde->nhde", _power(gamma, rest[..., None]).float(), own_state)
    last = last + _power(gamma, lens[:, None]).float()[..., None, None] * first
    # outputs: the masked product inside the chunk, and the state before it
    near = r[:, None] - r[None, :]
    decay = torch.where((near >= 0)[..., None], _power(gamma, near.clamp(min=0)[..., None]), 0.0).float()  # (C, C, kv)
    scores = torch.einsum("nmrhgd,nmchd->nmhgrc", qc, kc) * decay.permute(2, 0, 1)[:, None]
    oc = torch.einsum("nmhgrc,nmche->nmrhge", scores, vc)
    xi = _power(gamma, (r + 1)[:, None]).float()[..., None, None]  # (C, kv, 1, 1)
    oc = oc + torch.einsum("nmrhgd,nmhde->nmrhge", qc, before) * xi
    oc = oc * _row_factor(gamma, dk, p[..., None]).float()[..., None, None]
    # rows behind the last sequence keep what they held: row `rows` takes the padding's writes
    full = torch.cat((o, o[:1]))
    full[torch.where(valid, tok, rows)] = oc.flatten(3, 4).to(o.dtype)
    o.copy_(full[:rows])
    pool[slots] = torch.where((lens > 0)[:, None, None, None], last, pool[slots])
    return {"o": o, "pool": pool}


def _step(s):
    q, k, v, pool, o, pos = s["q"], s["k"], s["v"], s["pool"], s["o"], s["pos"]
    hq, dk = q.shape[1:]
    kv = k.shape[1]
    live = s["slots"] >= 0
    at = torch.where(live, s["slots"], pool.shape[0]).long()  # padding goes to one slot more
    wide = torch.cat((pool, pool[:1]))
    gamma, angle = s["gamma_dev"], pos.double()[:, None, None] * s["theta_dev"].double()
    qr, kr = _rotate(q.float(), angle).unflatten(1, (kv, hq // kv)), _rotate(k.float(), angle)
    old = torch.where((pos > 0)[:, None, None, None], wide[at], 0.0)
    state = gamma[:, None, None] * old + kr[..., None] * v.float()[:, :, None]
    wide[at] = state
    pool.copy_(wide[:-1])
    out = torch.einsum("nhgd,nhde->nhge", qr, state) * _row_factor(gamma, dk, pos[:, None]).float()[..., None, None]
    o.copy_(torch.where(live[:, None, None], out.flatten(1, 2).to(o.dtype), o))
    return {"o": o, "pool": pool}


def _slots(s):
    pool, src, dst = s["pool"], s["src"].long(), s["dst"].long()
    pool[dst] = torch.where((src >= 0)[:, None, None, None], pool[src.clamp(min=0)], 0.0)
    return {"pool": pool}


def _msr(s):
    y, g, w, b = s["y"].float(), s["g"].float(), s["weight"], s["bias"]
    dt = s["y"].dtype
    mean = y.mean(dim=-1, keepdim=True)
    rstd = torch.rsqrt((y - mean).square().mean(dim=-1, keepdim=True) + EPS)
    xhat = (y - mean) * rstd
    norm = xhat * w + b
    sig = torch.sigmoid(g)
    out = (g * sig * norm).to(dt)
    if not s["case"]["train"]:
        return {"out": out}
    dout = s["dout"].float()
    dn = dout * g * sig
    dg = dout * norm * sig * (1.0 + g * (1.0 - sig))
    dx = dn * w
    dy = rstd * (dx - dx.mean(dim=-1, keepdim=True) - xhat * (dx * xhat).mean(dim=-1, keepdim=True))
    return {"out": out, "dy": dy.to(dt), "dg": dg.to(dt), "dweight": (dn * xhat).sum(dim=0), "dbias": dn.sum(dim=0)}


def run(state):
    if own:
        return _run_own(state)
    return {"packed": _packed, "step": _step, "slots": _slots, "msr": _msr}[state["case"]["op"]](state)


# ---- costs and the definitions in fp64 -----------------------------------------------------

def work(case):
    op = case["op"]
    if op == "msr":
        size = 2 if case["dtype"] == "bf16" else 4
        n, params = case["tokens"] * case["heads"] * case["d_v"], case["heads"] * case["d_v"] * 4
        # y, g read and out written; backward: y, g, dout read, dy, dg written
        passes, p = (3, 2) if not case["train"] else (8, 6)
        return {"bytes": passes * n * size + p * params, "flops": (40 if case["train"] else 14) * n}
    one = 4 * case["heads_kv"] * case["d_k"] * case["d_v"]
    if op == "slots":
        read = 1 if case["kind"] == "fork" else case["pairs"]
        return {"bytes": (read + case["pairs"]) * one, "flops": 0}
    size = 2 if case["dtype"] == "bf16" else 4
    token = ((case["heads"] + case["heads_kv"]) * case["d_k"] + (case["heads"] + case["heads_kv"]) * case["d_v"]) * size
    flops = 2 * (case["heads"] + case["heads_kv"]) * case["d_k"] * case["d_v"]
    if op == "packed":
        lens = _lengths(case)
        states = sum((2 if _continues(i) else 1) for i, x in enumerate(lens) if x)
        return {"bytes": case["tokens"] * token + states * one, "flops": case["tokens"] * flops}
    live = case["rows"] - case["padded"]
    states = sum(2 if _continues(i) else 1 for i in range(live))
    return {"bytes": live * token + states * one, "flops": live * flops}


def _turn64(x, angle):
    z = torch.view_as_complex(x.double().unflatten(-1, (-1, 2)).contiguous())
    return torch.view_as_real(z * torch.polar(torch.ones_like(angle), angle)).flatten(-2)


def _token64(state, q, k, v, p, gamma, theta, group):
    """One token of each of n sequences: (output, new state) by o = f q (g S + k^T v), all in fp64."""
    angle = p.double()[:, None, None] * theta
    q, k, v = _turn64(q, angle), _turn64(k, angle), v.double()
    n, hq, dk = q.shape
    state = state * gamma[:, None, None]
    out = torch.matmul(q.reshape(n, hq // group, group, dk), state)
    out = out + (q.reshape(n, hq // group, group, dk) * k[:, :, None]).sum(-1, keepdim=True) * v[:, :, None]
    state.add_(k[..., None] * v[:, :, None])
    seen = -torch.expm1((p.double()[:, None] + 1.0) * torch.log(gamma)) / (1.0 - gamma)
    return (out / torch.sqrt(dk * seen)[:, :, None, None]).reshape(n, hq, -1), state


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "msr":
        y, g, w, b = (s[x].double().requires_grad_() for x in ("y", "g", "weight", "bias"))
        var, mean = torch.var_mean(y, dim=-1, unbiased=False, keepdim=True)
        out = (w * ((y - mean) / torch.sqrt(var + EPS)) + b) * (g / (1.0 + torch.exp(-g)))
        if not case["train"]:
            return {"out": out.detach()}
        dy, dg, dw, db = torch.autograd.grad(out, (y, g, w, b), s["dout"].double())
        return {"out": out.detach(), "dy": dy, "dg": dg, "dweight": dw, "dbias": db}
    pool = s["pool"].double()
    if op == "slots":
        old = pool.clone()
        for a, d in zip(s["src"].tolist(), s["dst"].tolist()):
            pool[d] = old[a] if a >= 0 else 0.0
        return {"pool": pool}
    gamma, theta, group = s["gamma_dev"].double(), s["theta_dev"].double(), case["heads"] // case["heads_kv"]
    o = s["o"].double()
    slots, pos = s["slots"].tolist(), s["pos"].tolist()
    if op == "step":
        live = [i for i, x in enumerate(slots) if x >= 0]
        lens, start = [1] * len(live), live
    else:
        cu = s["cu_seqlens"].tolist()
        live = [i for i in range(len(slots)) if cu[i + 1] > cu[i]]
        lens, start = [cu[i + 1] - cu[i] for i in live], [cu[i] for i in live]
    if max(lens, default=0) * len(live) * pool[0].numel() > 9e11:
        return None
    # the longest first, so that the sequences still running are a prefix
    order = sorted(range(len(live)), key=lambda i: -lens[i])
    at = [slots[live[i]] for i in order]
    state = torch.stack([pool[slots[live[i]]] * (pos[live[i]] > 0) for i in order])
    p0 = torch.tensor([pos[live[i]] for i in order], device="cuda")
    first = torch.tensor([start[i] for i in order], device="cuda")
    lens = [lens[i] for i in order]
    running = len(lens)
    for t in range(lens[0]):
        while lens[running - 1] <= t:
            running -= 1
        row = first[:running] + t
        out, new = _token64(state[:running], s["q"][row], s["k"][row], s["v"][row], p0[:running] + t, gamma, theta, group)
        o[row], state[:running] = out, new
    pool[at] = state
    return {"o": o, "pool": pool}
