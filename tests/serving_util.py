"""Shared by the tests of the packed, single-token and slot-copy calls: cases and their fp64 results."""
import numpy as np
import torch

import linear_attention_sequence_chunkwise_b200 as rn
import oracle
import synth_inputs as si

FLAGS = rn.F_XPOS | rn.F_SCALE_SQRT_D | rn.F_NORM_D


def reference(q, k, v, pool, lens, slots, pos, gamma, theta, flags, start=None):
    """Outputs (fp64, NaN in rows of no sequence) and pool after packed retention, sequence by sequence
    through the oracle's recurrent form; keys, values and states repeated over their query heads."""
    rows, hq, dk = q.shape
    kv, dv = v.shape[1:]
    group = hq // kv
    out = np.full((rows, hq, dv), np.nan)
    after = pool.double().numpy().copy()
    before = after.copy()
    at = 0
    for i, n in enumerate(lens):
        r = slice(at if start is None else start[i], (at if start is None else start[i]) + n)
        at += n
        if n == 0 or slots[i] < 0:
            continue
        rep = lambda x: x[r].repeat_interleave(group, dim=1)[None]  # noqa: E731
        s0 = None
        if pos[i] > 0:
            s0 = np.repeat(before[slots[i]], group, axis=0)[None]
        g = np.repeat(gamma, group)
        if pos[i] <= 100000:
            o, s, _ = oracle.recurrent(q[r][None], rep(k), rep(v), g, theta, pos[i], flags, s0)
        else:  # the oracle counts up to a position: far ones are rotated and divided by c_p's closed form here
            p = pos[i] + np.arange(n, dtype=np.float64)[:, None]
            a = p.astype(np.longdouble) * theta.astype(np.longdouble)  # 64-bit significands: exact up to 2^40
            z = (np.cos(a).astype(float) + 1j * np.sin(a).astype(float))[:, None] if flags & rn.F_XPOS else 1.0

            def turn(x):
                x = x.double().numpy()[0]
                y = (x[..., 0::2] + 1j * x[..., 1::2]) * z
                return np.stack((y.real, y.imag), axis=-1).reshape(1, *x.shape)
            o, s, _ = oracle.recurrent(turn(q[r][None]), turn(rep(k)), rep(v), g, theta, 0, flags & rn.F_SCALE_SQRT_D, s0)
            if flags & rn.F_NORM_D:
                o /= np.sqrt((1.0 - g.astype(np.float64) ** (p + 1.0)) / (1.0 - g.astype(np.float64)))[..., None]
        out[r] = o[0]
        after[slots[i]] = s[0, ::group]
    return out, after


def case(lens, hq, kv, dk, dv, dtype, seed, slots=None, pos=None, n_slots=None, behind=2, gamma=None, pool_std=0.5):
    """Inputs on the CPU: q, k, v as views of one fused projection, a pool, slots, positions."""
    n, rows = len(lens), sum(lens) + behind
    fused = si.randn((rows, (hq + kv) * dk + kv * dv), seed, dtype)
    n_slots = n_slots or n + 3
    rng = np.random.default_rng(seed)
    if slots is None:
        slots = rng.permutation(n_slots)[:n].tolist()
    if pos is None:
        pos = [0 if i % 3 == 0 else int(rng.integers(1, 5000)) for i in range(n)]
    pool = si.randn((n_slots, kv, dk, dv), seed + 1, "f32", std=pool_std)
    gamma = si.gamma_schedule(kv) if gamma is None else np.asarray(gamma, dtype=np.float32)
    return fused, pool, list(slots), list(pos), gamma, si.theta_schedule(dk)


def split(fused, hq, kv, dk, dv):
    q, k, v = fused.split((hq * dk, kv * dk, kv * dv), dim=1)
    return q.unflatten(1, (hq, dk)), k.unflatten(1, (kv, dk)), v.unflatten(1, (kv, dv))


def cu_of(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)


def errors(got, ref):
    """max|got - ref| / rms(ref) over the elements that ref has; a bf16 result's own rounding (half a
    step, 2^-8 of the value) comes off first."""
    g = got.detach().double().cpu().numpy()
    keep = ~np.isnan(ref)
    if not keep.any():
        return 0.0
    g, r = g[keep], ref[keep]
    d = np.abs(g - r)
    if got.dtype == torch.bfloat16:
        d = np.maximum(d - 2.0 ** -8 * np.abs(r), 0.0)
    return float(d.max() / max(np.sqrt((r ** 2).mean()), 1e-300))
