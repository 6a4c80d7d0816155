"""Slow numpy fp64 restatement of rotary positions in their usual forms, of attention over a prefix
that several sequences share, and of drawing the next token.  Test infrastructure only: it shares no
code with the CUDA path."""
import math

import numpy as np

PLAIN, LINEAR, BASE, WAVES, RAMP = range(5)


# ---- rotary positions ------------------------------------------------------------------------
def theta(rot, base, scaling=PLAIN, factor=1.0, original_len=0.0, low=0.0, high=0.0):
    """The angle pair i turns per position, for each of the rot / 2 pairs."""
    out = []
    for i in range(rot // 2):
        if scaling == BASE:
            out.append((base * factor ** (rot / (rot - 2))) ** (-2 * i / rot))
            continue
        t = base ** (-2 * i / rot)
        slow = t / factor
        if scaling == LINEAR:
            t = slow
        elif scaling == WAVES:
            turns = original_len * t / (2 * math.pi)          # of the original context
            if turns < low:
                t = slow
            elif turns <= high:
                g = (turns - low) / (high - low)
                t = g * t + (1 - g) * slow
        elif scaling == RAMP:
            pair = lambda turns: rot * math.log(original_len / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
            lo, hi = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rot - 1)
            r = min(max((i - lo) / ((hi - lo) or 0.001), 0.0), 1.0)
            t = (1 - r) * t + r * slow
        out.append(t)
    return np.array(out)


def rotate(x, pos, theta_, half, amplitude=1.0):
    """x [n, heads, hd]: pair i of the first 2 len(theta_) channels turned by pos * theta_i."""
    y = np.array(x, np.float64)
    m = len(theta_)
    a, b = (np.arange(m), np.arange(m) + m) if half else (2 * np.arange(m), 2 * np.arange(m) + 1)
    ang = np.asarray(pos, np.float64)[:, None, None] * theta_
    c, s = np.cos(ang) * amplitude, np.sin(ang) * amplitude
    u, w = y[..., a].copy(), y[..., b].copy()
    y[..., a], y[..., b] = u * c - w * s, u * s + w * c
    return y


# ---- shared prefix ---------------------------------------------------------------------------
def shared_attention(q, last, prefixes, seq0, own_k, own_v):
    """q [n_seq, n_q, H, hd], last [n_seq, n_q], prefixes: per group (k, v) [rows, Hkv, hd]; group g
    has sequences [seq0[g], seq0[g + 1]); own_k, own_v [n_seq, cap, Hkv, hd].  Returns the output
    and sum_i p_i |v_i| of the same shape."""
    n, nq, H, hd = q.shape
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    for g, (kp, vp) in enumerate(prefixes):
        for s in range(seq0[g], seq0[g + 1]):
            for j in range(nq):
                m = int(last[s, j]) + 1
                if m < 0:
                    continue
                k, v = np.concatenate([kp, own_k[s, :m]]), np.concatenate([vp, own_v[s, :m]])
                if not len(k):
                    continue
                G = H // k.shape[1]
                for h in range(H):
                    z = k[:, h // G].astype(np.float64) @ q[s, j, h].astype(np.float64) / math.sqrt(hd)
                    p = np.exp(z - z.max())
                    p /= p.sum()
                    out[s, j, h], mag[s, j, h] = p @ v[:, h // G], p @ np.abs(v[:, h // G])
    return out, mag


# ---- sampling --------------------------------------------------------------------------------
def sample(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """One row: (token, ln of its share, ids kept, distance of the nearest decision: how far, as a share
    of the weight, the draw and the top_p border are from falling otherwise)."""
    x = np.asarray(x, np.float64)
    order = [i for i in np.argsort(-x, kind="stable") if x[i] > -np.inf]
    if not order:
        return -1, -np.inf, 0, 1.0
    top, T = x[order[0]], float(temperature)
    w = {i: (1.0 if x[i] == top else math.exp((x[i] - top) / T) if T > 0 and np.isfinite(top) else 0.0) for i in order}
    if T == 0:
        order = order[:1]
    if top_k > 0:
        order = order[:top_k]
    near = 1.0
    if top_p < 1:
        total, run, keep = math.fsum(w[i] for i in order), 0.0, []
        for i in order:
            if keep and run >= top_p * total:
                break
            keep.append(i)
            run += w[i]
            near = min(near, abs(run - top_p * total) / total)
        order = keep
    if min_p > 0:
        near = min(near, min(abs(w[i] - min(min_p, 1.0)) for i in order if w[i] < 1) if any(w[i] < 1 for i in order) else 1.0)
        order = [i for i in order if w[i] >= min(min_p, 1.0)]
    ids = sorted(order)
    total = math.fsum(w[i] for i in ids)
    run, token = 0.0, ids[-1]
    for i in ids:
        run += w[i]
        near = min(near, abs(run - u * total) / total if i != ids[-1] else 1.0)
        if run > u * total:
            token = i
            break
    return token, math.log(w[token] / total), len(ids), near
