"""Slow numpy fp64 restatement of the 8-bit block-scaled KV cache, attention over it, eviction
by accumulated weight, and the rules on logits.  Test infrastructure only: it shares no code
with the CUDA path.

A cache is a dict: codes "k", "v" int64 [n_seq, Hkv, cap, hd], scales "ks", "vs" float32
[n_seq, Hkv, cap / block], and "block".  Scales are fp32 values (the stored quantity); every
decision and sum is taken in fp64."""
import numpy as np

MIN_SCALE = np.float32(1e-8)


def empty(n_seq, hkv, cap, hd, block):
    z = lambda: np.zeros((n_seq, hkv, cap, hd), np.int64)  # noqa: E731
    s = lambda: np.zeros((n_seq, hkv, cap // block), np.float32)  # noqa: E731
    return {"k": z(), "v": z(), "ks": s(), "vs": s(), "block": block}


def _scale(amax):
    return max(np.float32(np.float32(amax) / np.float32(127)), MIN_SCALE)


def _nearest(num, den):
    return np.clip(np.rint(num / den), -127, 127).astype(np.int64)


def append(c, k, v, start, count=None):
    """k, v: [n_seq, n_rows, Hkv, hd]; rows past the capacity are dropped, non-finite is 0."""
    n_seq, hkv, cap, _ = c["k"].shape
    blk = c["block"]
    for x, codes, scale in ((k, c["k"], c["ks"]), (v, c["v"], c["vs"])):
        x = np.where(np.isfinite(x), x, 0.0).astype(np.float64)
        for s in range(n_seq):
            a = int(start[s])
            if a < 0:
                continue
            n = x.shape[1] if count is None else min(max(int(count[s]), 0), x.shape[1])
            e = min(a + n, cap)
            for b in range(a // blk, -(-e // blk) if e > a else 0):
                lo, hi = max(a, b * blk), min(e, (b + 1) * blk)
                for h in range(hkv):
                    new = x[s, lo - a:hi - a, h]
                    sc = _scale(np.abs(new).max())
                    if lo > b * blk:
                        old = scale[s, h, b]
                        if sc > old:
                            r = slice(b * blk, lo)
                            codes[s, h, r] = _nearest(codes[s, h, r] * np.float64(old), np.float64(sc))
                        sc = max(sc, old)
                    codes[s, h, lo:hi] = _nearest(new, np.float64(sc))
                    scale[s, h, b] = sc


def values(codes, scale, block):
    return codes * np.repeat(scale.astype(np.float64), block, axis=2)[..., None]


def attention(c, q, last):
    """q: [n_seq, n_q, H, hd], last: [n_seq, n_q].  Returns out [n_seq, n_q, H, hd], the weights
    [n_seq, Hkv, cap], sum_i p_i |v_i| (same shape as out) and, per query, two figures that
    roundings scale with: the largest sum_c |q_c k_c| / sqrt(hd) over the keys it sees, and the
    largest p_i times the scale of v_i."""
    n_seq, nq, H, hd = q.shape
    hkv, cap = c["k"].shape[1:3]
    g = H // hkv
    out, mag, zmag = np.zeros(q.shape), np.zeros(q.shape), np.zeros((n_seq, nq, H))
    top = np.zeros((n_seq, nq, H))
    w = np.zeros((n_seq, hkv, cap))
    for s in range(n_seq):
        for j in range(nq):
            n = int(last[s, j]) + 1
            if n <= 0 or n > cap:
                continue
            nb = -(-n // c["block"])
            for h in range(H):
                kh = h // g
                sl = lambda codes, scale: (codes[s, kh, :n] * np.repeat(  # noqa: E731
                    np.maximum(scale[s, kh, :nb].astype(np.float64), float(MIN_SCALE)), c["block"])[:n, None])
                K, V = sl(c["k"], c["ks"]), sl(c["v"], c["vs"])
                z = K @ q[s, j, h] / np.sqrt(hd)
                p = np.exp(z - z.max())
                p /= p.sum()
                out[s, j, h] = p @ V
                mag[s, j, h] = p @ np.abs(V)
                zmag[s, j, h] = (np.abs(K) @ np.abs(q[s, j, h])).max() / np.sqrt(hd)
                top[s, j, h] = (p * np.repeat(np.maximum(c["vs"][s, kh, :nb], MIN_SCALE), c["block"])[:n]).max()
                w[s, kh, :n] += p
    return out, w, mag, zmag, top


def evict(c, length, weights, n_keep, n_sink, n_recent, dst_cap):
    """Returns (dst cache, dst_len, dst_weights, kept)."""
    n_seq, hkv, cap, hd = c["k"].shape
    blk = c["block"]
    d = empty(n_seq, hkv, dst_cap, hd, blk)
    kept = np.full((n_seq, hkv, n_keep), -1, np.int64)
    dw = np.zeros((n_seq, hkv, dst_cap), np.float32)
    dl = np.zeros(n_seq, np.int64)
    for s in range(n_seq):
        n = min(max(int(length[s]), 0), cap)
        m = dl[s] = min(n, n_keep)
        for h in range(hkv):
            w = weights[s, h, :n].astype(np.float64)
            rank = np.where(np.isnan(w) | (w < 0), 0.0, w)
            if n <= n_keep:
                rows = np.arange(n)
            else:
                lo, hi = n_sink, n - n_recent
                best = lo + np.argsort(-rank[lo:hi], kind="stable")[:n_keep - n_sink - n_recent]
                rows = np.sort(np.concatenate([np.arange(lo), best, np.arange(hi, n)]))
            kept[s, h, :m] = rows
            dw[s, h, :m] = weights[s, h, rows]
            for codes, scale, dc, ds in ((c["k"], c["ks"], d["k"], d["ks"]), (c["v"], c["vs"], d["v"], d["vs"])):
                # a moved value is the fp32 product of its code and scale
                x = (codes[s, h, rows].astype(np.float32) * scale[s, h, rows // blk][:, None]).astype(np.float64)
                for b in range(-(-m // blk)):
                    r = slice(b * blk, min(m, (b + 1) * blk))
                    ds[s, h, b] = _scale(np.abs(x[r]).max())
                    dc[s, h, r] = _nearest(x[r], np.float64(ds[s, h, b]))
    return d, dl, dw, kept


def logits(x, history=None, prompt_len=0, repetition=1.0, presence=0.0, frequency=0.0, bias=(), mask=None, vocab=None):
    """One row in fp64: history a list of ids, bias a list of (id, value), mask a bool array."""
    x = np.array(x, np.float64)
    ids = np.asarray([] if history is None else history, np.int64)
    ok = (ids >= 0) & (ids < len(x))
    seen = np.unique(ids[ok])
    x[seen] = np.where(x[seen] > 0, x[seen] / repetition, x[seen] * repetition)
    made, count = np.unique(ids[prompt_len:][ok[prompt_len:]], return_counts=True)
    x[made] -= frequency * count + presence
    for i, b in bias:
        if 0 <= i < len(x):
            x[i] += b
    if mask is not None:
        x[~mask] = -np.inf
    return x


def token(y):
    """The lowest id of the largest value (NaN never), -1 if none is above -inf."""
    y = np.where(np.isnan(y), -np.inf, y)
    return int(np.argmax(y)) if y.max() > -np.inf else -1
