"""Float64 oracle of the paged serving calls: plain numpy and loops, written
from the definitions (the page bookkeeping as a host scheduler would do it,
the rotation as complex numbers, the attention with both maps materialised).
It shares no code with the CUDA path."""
from __future__ import annotations

import numpy as np


def paged_step(ctx, new, table, ring, pool, page, T):
    """(table, ring, pool, cu_q, kv_lens, positions, slots, info) after the step; the inputs are left alone."""
    table, ring = np.array(table), np.array(ring)
    S, width = table.shape
    F = len(ring)
    head, count = int(pool[0]), int(pool[1])
    ceil = lambda a: -(-a // page)
    tokens = taken = freed = bad = 0
    for c, n in zip(ctx, new):
        c, n = int(c), int(n)
        if c < 0 or n < -1 or c + n > 2 ** 31 - 1:
            bad |= 8
            continue
        if max(ceil(c), ceil(c + max(n, 0))) > width:
            bad |= 2
        if n < 0:
            freed += ceil(c)
        else:
            tokens += n
            taken += ceil(c + n) - ceil(c)
    bad |= 1 if taken > count else 0
    bad |= 4 if tokens > T else 0
    bad |= 16 if head < 0 or head >= F or count < 0 or count + freed > F else 0
    info = [min(x, 2 ** 31 - 1) for x in (tokens, taken, freed)] + [bad]
    if bad:
        return (table, ring, [head, count], [0] * (S + 1), [0] * S, [-1] * T, [-1] * T, info)
    cu, kv, pos, slots = [0], [], [], []
    out_at, in_at = head, head + count
    for s in range(S):
        c, n = int(ctx[s]), int(new[s])
        if n < 0:
            for j in range(ceil(c)):
                ring[in_at % F] = table[s, j]
                in_at += 1
            cu.append(cu[-1])
            kv.append(0)
            continue
        for j in range(ceil(c), ceil(c + n)):
            table[s, j] = ring[out_at % F]
            out_at += 1
        for p in range(c, c + n):
            pos.append(p)
            slots.append(int(table[s, p // page]) * page + p % page)
        cu.append(cu[-1] + n)
        kv.append(c + n)
    pos += [-1] * (T - len(pos))
    slots += [-1] * (T - len(slots))
    return table, ring, [out_at % F, count - taken + freed], cu, kv, pos, slots, info


def rope_frequencies(rot, base, scaling="plain", factor=1.0, orig_len=4096, beta_fast=32.0, beta_slow=1.0):
    """(theta'_j, the factor on cos and sin)."""
    j = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    theta = base ** (-2 * j / rot)
    if scaling == "linear":
        return theta / factor, 1.0
    if scaling == "yarn":
        turns = orig_len * theta / (2 * np.pi)
        g = np.clip((turns - beta_slow) / (beta_fast - beta_slow), 0, 1)
        return theta * g + theta / factor * (1 - g), 0.1 * np.log(factor) + 1
    return theta, 1.0


def rope(x, pos, theta, m=1.0, half=False, inverse=False):
    """x [T, rows..., d] with channel pairs turned by pos * theta; rows with a negative position as they are."""
    x = np.asarray(x, dtype=np.float64)
    r = 2 * len(theta)
    pos = np.asarray(pos)
    turn = m * np.exp((-1j if inverse else 1j) * pos[:, None] * theta[None, :])
    turn = turn.reshape((len(pos),) + (1,) * (x.ndim - 2) + (r // 2,))
    a, b = (x[..., :r // 2], x[..., r // 2:r]) if half else (x[..., 0:r:2], x[..., 1:r:2])
    z = (a + 1j * b) * turn
    y = x.copy()
    if half:
        y[..., :r // 2], y[..., r // 2:r] = z.real, z.imag
    else:
        y[..., 0:r:2], y[..., 1:r:2] = z.real, z.imag
    y[pos < 0] = x[pos < 0]
    return y


def extend(q, k_cache, v_cache, table, cu_q, kv_lens, lam, lambda_init, rms_w, eps, causal=True, c2=None,
           p_err=None, out_err=0.0):
    """[T, H, 2d]; rows of no request are nan.  c2: the coefficient of map 2 (default -lam).  Pages out of range
    read as zeros; keys that the table has no entry for are left out.

    With p_err, also a bound of the error of an implementation whose weights are off by at most p_err relative
    (and whose result is rounded by at most out_err relative): the sum o of c_i p_i v is off by at most
    e = p_err * sum |c_i| p_i |v| a channel, so o / sqrt(mean o^2 + eps) by at most
    (e + |o| r(e) / r) / r / (1 - r(e) / r) with r = sqrt(mean o^2 + eps) and r(e) = sqrt(mean e^2): r changes by at
    most r(e)."""
    T, H, _, d = q.shape
    P, page, Hkv = k_cache.shape[:3]
    c2 = -lam if c2 is None else c2
    out = np.full((T, H, 2 * d), np.nan)
    tol = np.zeros((T, H, 2 * d))
    for s in range(len(kv_lens)):
        n, L = int(cu_q[s + 1] - cu_q[s]), int(kv_lens[s])
        held = min(L, table.shape[1] * page)
        k, v = np.zeros((held, Hkv, 2, d)), np.zeros((held, Hkv, 2 * d))
        for i in range(held):
            pg = int(table[s, i // page])
            if 0 <= pg < P:
                k[i], v[i] = k_cache[pg, i % page], v_cache[pg, i % page]
        for i in range(n):
            t = int(cu_q[s]) + i
            see = held if not causal else min(held, max(0, L - n + i + 1))
            for h in range(H):
                g = h // (H // Hkv)
                o, e = np.zeros(2 * d), np.zeros(2 * d)
                for m, c in ((0, 1.0), (1, c2)):
                    if see:
                        x = k[:see, g, m] @ q[t, h, m] / np.sqrt(d)
                        w = np.exp(x - x.max())
                        o += c * (w / w.sum()) @ v[:see, g]
                        if p_err is not None:
                            e += p_err * abs(c) * (w / w.sum()) @ np.abs(v[:see, g])
                rms = np.sqrt((o * o).mean() + eps)
                out[t, h] = (1 - lambda_init) * rms_w * o / rms
                if p_err is not None and see:
                    ne = np.sqrt((e * e).mean())
                    shrink = max(1 - ne / rms, 1e-3)
                    tol[t, h] = np.abs((1 - lambda_init) * rms_w) * (e + np.abs(o) * ne / rms) / rms / shrink
                    tol[t, h] += out_err * (np.abs(out[t, h]) + tol[t, h])
    return out if p_err is None else (out, tol)
