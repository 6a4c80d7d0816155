"""Workloads of the operators behind a batch of answers sampled from one blended prompt: rotary
positions in other layouts and scalings than the blend's own, attention over a prefix that a
batch shares with each answer's own rows behind it, and the choice of the next token from given
random numbers.

Each workload has a plain form (elementary torch operations in fp32, 64 bits for the sampling's
weights and sums, rounded once at the end) and the library's own calls.  `own` chooses between them.

Formulas (n = row, s = sequence, h = KV head, G = query heads per KV head):

  rope     (x1, x2) -> (x1 c - x2 s, x1 s + x2 c), c and s = a cos, a sin of position * theta_i; pairs
           (2i, 2i + 1) or (i, i + rot / 2) of a head's first rot channels, the others as they are.
           theta_i = base^(-2i / rot), scaled for long contexts by a factor f:
             linear   theta / f
             base     with base f^(rot / (rot - 2)) in place of base
             waves    w = 2 pi / theta, L = original length: theta for w < L / high, theta / f for
                      w > L / low, between them g theta + (1 - g) theta / f, g = (L / w - low) / (high - low)
             ramp     d(b) = rot ln(L / (2 pi b)) / (2 ln base), lo = max(floor d(high), 0),
                      hi = min(ceil d(low), rot - 1), r = clamp((i - lo) / (hi - lo), 0, 1) (hi = lo: + 0.001):
                      (1 - r) theta + r theta / f
           k (rotated) and v go to rows of a cache; inverse: the angle negated
  shared   o[s, j] = sum_i softmax_i(q[s, j] . k[i] / sqrt(hd)) v[i], i over the prefix rows of the
           group of s and the rows 0..last[s, j] of s's own cache; last = -2: padding, zeros
  sample   w_i = exp((l_i - max l) / T), in order of falling logit, then rising id: the first top_k, of
           those the fewest whose weight reaches top_p of theirs, of those the ones with w >= min_p;
           token = first of them by id whose running weight exceeds u * their weight; its log share,
           and how many are kept.  T = 0: the lowest id of the largest logit
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # a decoding step of 64 answers: q | k | v as one projection leaves them, K and V into their caches (latency)
        dict(name="rope_token_yi", op="rope", rows=64, h=56, hkv=8, hd=128, rot=128, layout="half", scaling="ramp",
             factor=8.0, pos="far", to="cache", packed=True, inverse=False, dtype="bf16"),
        # a long prompt's rows, an odd number of them (the largest)
        dict(name="rope_prompt_yi", op="rope", rows=16001, h=56, hkv=8, hd=128, rot=128, layout="half", scaling="waves",
             factor=8.0, pos="run", to="cache", packed=True, inverse=False, dtype="bf16"),
        # chunk caches of another layout moved to their new positions, half of each head rotated
        dict(name="rope_pool_7b", op="rope", rows=3840, h=0, hkv=32, hd=128, rot=64, layout="half", scaling="none",
             factor=1.0, pos="delta", to="gather", packed=False, inverse=False, dtype="bf16"),
        # the gradient of a rotation, or cached keys turned back
        dict(name="rope_back_f32", op="rope", rows=1001, h=4, hkv=4, hd=64, rot=32, layout="interleaved", scaling="linear",
             factor=4.0, pos="run", to="rows", packed=False, inverse=True, dtype="f32"),
        # the first tokens of four answers sampled from one 4096-row prompt
        dict(name="shared_token_7b", op="shared", groups=1, n_seq=4, n_q=1, h=32, hkv=32, hd=128, prefix=4096, cap=64,
             dtype="bf16"),
        # 64 answers to one long prompt, further on, grouped heads
        dict(name="shared_token_yi_b64", op="shared", groups=1, n_seq=64, n_q=1, h=56, hkv=8, hd=128, prefix=16384, cap=512,
             dtype="bf16"),
        # four prompts of different lengths with eight answers each, four drafted tokens checked at once
        dict(name="shared_draft_13b", op="shared", groups=4, n_seq=32, n_q=4, h=40, hkv=40, hd=128, prefix=8192, cap=700,
             dtype="bf16"),
        # eight questions of up to 96 tokens about the same documents (the largest)
        dict(name="shared_ask_yi", op="shared", groups=1, n_seq=8, n_q=96, h=56, hkv=8, hd=128, prefix=16000, cap=96,
             dtype="bf16"),
        # the exact mode
        dict(name="shared_f32", op="shared", groups=2, n_seq=6, n_q=3, h=4, hkv=4, hd=64, prefix=1000, cap=100,
             dtype="f32"),
        # the next token of one answer
        dict(name="sample_7b", op="sample", rows=1, vocab=32000, k=50, p=0.95, min_p=0.0, heat=0.8, closed=0.0,
             dtype="f32"),
        # a batch over a large vocabulary, half of it closed by a grammar
        dict(name="sample_yi_b64", op="sample", rows=64, vocab=64000, k=0, p=0.9, min_p=0.02, heat=1.0, closed=0.5,
             dtype="bf16"),
        # a large batch over a larger one, settings that differ by row
        dict(name="sample_large_b256", op="sample", rows=256, vocab=131072, k=1000, p=0.98, min_p=0.001, heat=1.2,
             closed=0.0, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "shared", "shared", "sample"])
    hkv, g = rng.choice([(32, 1), (40, 1), (8, 7), (4, 1), (8, 4), (2, 4)])
    if op == "rope":
        hd = rng.choice([128, 128, 64])
        to = rng.choice(["cache", "rows", "gather"])
        rows = _log(rng, 1, 16000)
        case = dict(op=op, rows=rows, h=0 if to == "gather" else hkv * g, hkv=hkv, hd=hd,
                    rot=rng.choice([hd, hd, hd // 2, hd // 4]), layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "base", "waves", "ramp"]), factor=rng.choice([2.0, 4.0, 8.0]),
                    pos="delta" if to == "gather" else rng.choice(["run", "far"]), to=to,
                    packed=to != "gather" and rng.random() < 0.6, inverse=rng.random() < 0.25,
                    dtype=rng.choice(["bf16", "bf16", "f32"]))
        while work(case)["bytes"] > 59e7:          # (the largest listed one's)
            case["rows"] = case["rows"] // 2 + 1
        return case
    if op == "shared":
        hd = rng.choice([128, 128, 64])
        dtype = rng.choice(["bf16", "bf16", "bf16", "bf16", "f32"])
        groups = rng.choice([1, 1, 1, 2, rng.randint(3, 8)])
        n_seq = max(groups, _log(rng, 1, 64))
        n_q = rng.choice([1, 1, 1, rng.randint(2, 8), rng.randint(9, 100)])
        prefix, cap = _log(rng, 64, 16384), _log(rng, 1, 1024)
        cap = max(cap, n_q)
        if dtype == "f32":          # exact arithmetic: small work only
            n_seq, n_q, prefix = max(groups, min(n_seq, 8)), min(n_q, 8), min(prefix, 2000)
            hkv, g = rng.choice([(4, 1), (2, 4)])
        case = dict(op=op, groups=groups, n_seq=n_seq, n_q=n_q, h=hkv * g, hkv=hkv, hd=hd, prefix=prefix, cap=cap,
                    dtype=dtype)
        # at most the work of the largest listed ones
        while work(case)["flops"] > 27e10 or work(case)["bytes"] > 77e7:
            if n_seq * case["cap"] > 2 * groups * case["prefix"]:
                case["cap"] = max(n_q, case["cap"] // 2)
            case["prefix"] = case["prefix"] * 3 // 4 + 1
        return case
    return dict(op=op, rows=_log(rng, 1, 128), vocab=rng.choice([32000, 64000, 131072, 5000, rng.randint(3, 131072)]),
                k=rng.choice([0, 0, 1, 40, 1000]), p=rng.choice([1.0, 1.0, 0.9, 0.95, 0.5]),
                min_p=rng.choice([0.0, 0.0, 0.05, 0.3]), heat=rng.choice([0.0, 0.6, 1.0, 1.5]),
                closed=rng.choice([0.0, 0.0, 0.5, 0.9]), dtype=rng.choice(["f32", "bf16"]))


# ---------------------------------------------------------------------------- inputs
_BASE, _ORIGINAL, _FAR = 5.0e6, 16384, 131072      # rotary base, original and scaled context length
_CAP = 256                                         # rows of an answer's cache in the rope workloads


def _rope_numbers(case):
    """low, high and the amplitude of the scaling rule."""
    if case["scaling"] == "waves":
        return 1.0, 4.0, 1.0
    if case["scaling"] == "ramp":
        return 1.0, 32.0, 0.1 * math.log(case["factor"]) + 1.0
    return 0.0, 0.0, 1.0


def _theta(case):
    """The angle a position adds to pair i, in 64 bits."""
    rot, f, rule = case["rot"], case["factor"], case["scaling"]
    low, high, _ = _rope_numbers(case)
    i = torch.arange(rot // 2, dtype=torch.float64)
    base = _BASE * f ** (rot / (rot - 2)) if rule == "base" else _BASE
    t = base ** (-2 * i / rot)
    if rule == "linear":
        t = t / f
    elif rule == "waves":
        w = 2 * math.pi / t
        mix = (_ORIGINAL / w - low) / (high - low)
        t = torch.where(w < _ORIGINAL / high, t, torch.where(w > _ORIGINAL / low, t / f, mix * t + (1 - mix) * t / f))
    elif rule == "ramp":
        dim = lambda b: rot * math.log(_ORIGINAL / (2 * math.pi * b)) / (2 * math.log(_BASE))  # noqa: E731
        lo, hi = max(math.floor(dim(high)), 0), min(math.ceil(dim(low)), rot - 1)
        r = ((i - lo) / (hi - lo if hi != lo else 0.001)).clamp(0, 1)
        t = (1 - r) * t + r * t / f
    return t


def _lens(case):
    """Own rows of each sequence: none for the first (where there are others), then spread up to the whole cache."""
    n, cap, nq = case["n_seq"], case["cap"], case["n_q"]
    return [cap if n == 1 else max(0 if nq == 1 else nq, cap * ((i * 7) % n) // (n - 1)) for i in range(n)]


def _queries(case):
    """Queries each sequence brings: all, but shorter questions where there are many rows of them."""
    n, nq = case["n_seq"], case["n_q"]
    return [nq if nq < 9 else max(1, nq - (nq * i) // (2 * n)) for i in range(n)]


def _prefixes(case):
    """(row0, rows) of each prefix: the first one whole, the others down to a half, and gaps between them."""
    out, at = [], 0
    for g in range(case["groups"]):
        n = case["prefix"] - (case["prefix"] * g) // (2 * case["groups"])
        out.append((at, n))
        at += n + 3 * (g % 2)
    return out


def _seq0(case):
    n, g = case["n_seq"], case["groups"]
    return [n * i // g for i in range(g + 1)]


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _kv(g, n, hkv, hd, k_like):
    """K and V rows as a model leaves them: keys with a few strong channels, token norms that vary."""
    x = _normal(g, n, hkv, hd)
    if k_like:
        x *= 1 + 3 * (torch.rand(hkv, hd, generator=g, device="cuda") < 0.04)
    x *= 0.5 + torch.rand(n, 1, 1, generator=g, device="cuda")
    return x.reshape(n, hkv * hd)


def prepare(case, seed):
    g = _generator(seed)
    st = {"case": case}
    {"rope": _prepare_rope, "shared": _prepare_shared, "sample": _prepare_sample}[case["op"]](st, case, g)
    if own:   # the handles, tables and scratch that such a program keeps between calls
        _handles(st, case)
    return st


def _prepare_rope(st, case, g):
    n, h, hkv, hd, dt = (case[k] for k in ("rows", "h", "hkv", "hd", "dtype"))
    dt = _DT[dt]
    i32 = lambda t: t.to(device="cuda", dtype=torch.int32)  # noqa: E731
    if case["to"] == "gather":          # a pool of chunk rows, each slot's rows in a run
        n_src = n + n // 3 + 1
        st["k"], st["v"] = _kv(g, n_src, hkv, hd, True).to(dt), _kv(g, n_src, hkv, hd, False).to(dt)
        st["src_row"] = i32((torch.arange(n, device="cuda") + torch.randint(n_src, (1,), generator=g, device="cuda")) % n_src)
        st["q"] = None
    else:
        x = torch.cat([_normal(g, n, h * hd), _kv(g, n, hkv, hd, True), _kv(g, n, hkv, hd, False)], 1).to(dt)
        q, k, v = x.split([h * hd, hkv * hd, hkv * hd], 1)
        st["q"], st["k"], st["v"] = (q, k, v) if case["packed"] else (q.contiguous(), k.contiguous(), v.contiguous())
        st["src_row"] = None
    if case["pos"] == "far":            # one row of each of many answers, well behind their prompts
        st["pos"] = i32(_FAR - 1 - (torch.rand(n, generator=g, device="cuda").pow(3) * (_FAR - 2)).long())
    elif case["pos"] == "run":
        st["pos"] = i32(torch.arange(n, device="cuda") + torch.randint(_FAR - n, (1,), generator=g, device="cuda"))
    else:                               # offsets of chunk slots: forwards, some of them back
        slots = (torch.randint(-_FAR // 4, _FAR, (n // 480 + 1,), generator=g, device="cuda"))
        st["pos"] = i32(slots.repeat_interleave(480)[:n])
    rows = n
    st["kv_row"] = None
    if case["to"] == "cache":           # few rows: one for each answer's cache; many: a run of one cache
        if n <= 512:
            rows = n * _CAP
            st["kv_row"] = i32(torch.arange(n, device="cuda") * _CAP + torch.randint(_CAP, (n,), generator=g, device="cuda"))
        else:
            rows = n + 100
            st["kv_row"] = i32(torch.arange(n, device="cuda") + 77)
    st["q_out"] = None if st["q"] is None else torch.empty(n, h * hd, dtype=dt, device="cuda")
    st["k_out"] = torch.zeros(rows, hkv * hd, dtype=dt, device="cuda")
    st["v_out"] = torch.zeros(rows, hkv * hd, dtype=dt, device="cuda")
    if not own:
        p = torch.arange(_FAR, device="cuda", dtype=torch.float64)
        angle = p[:, None] * _theta(case).cuda()
        st["table"] = (torch.stack([angle.cos(), angle.sin()], 2) * _rope_numbers(case)[2]).float()


def _prepare_shared(st, case, g):
    n, nq, h, hkv, hd, cap, dt = (case[k] for k in ("n_seq", "n_q", "h", "hkv", "hd", "cap", "dtype"))
    dt = _DT[dt]
    row0, rows = _prefixes(case)[-1]
    st["k"], st["v"] = _kv(g, row0 + rows, hkv, hd, True).to(dt), _kv(g, row0 + rows, hkv, hd, False).to(dt)
    st["own_k"], st["own_v"] = (_kv(g, n * cap, hkv, hd, kl).to(dt).reshape(n, cap, hkv * hd) for kl in (True, False))
    # scores of standard deviation about 1.5: some rows draw most of the attention
    st["q"] = (_normal(g, n, nq, h, hd) * 1.1).to(dt)
    last = []
    for m, l in zip(_queries(case), _lens(case)):
        # the newest rows of each answer (their own keys are in the cache); what is shorter is padded
        last.append([l - m + j if nq > 1 else l - 1 for j in range(m)] + [-2] * (nq - m))
    st["last"] = torch.tensor(last, dtype=torch.int32, device="cuda")
    st["o"] = torch.empty_like(st["q"])


def _prepare_sample(st, case, g):
    n, V, dt = case["rows"], case["vocab"], _DT[case["dtype"]]
    x = _normal(g, n, V) * 2.2
    # a few ids stand out, by more in some rows than in others
    x += torch.rand(n, V, generator=g, device="cuda").pow(200) * 12 * torch.rand(n, 1, generator=g, device="cuda")
    closed = torch.rand(n, V, generator=g, device="cuda") < case["closed"]
    closed[:, V // 2] = False
    x[closed] = float("-inf")
    st["logits"] = x.to(dt)
    r = lambda: torch.rand(n, generator=g, device="cuda")  # noqa: E731
    vary = n > 1 and case["heat"] > 0
    st["temperature"] = case["heat"] * (0.7 + 0.6 * r()) if vary else torch.full((n,), case["heat"], device="cuda")
    st["top_k"] = torch.full((n,), case["k"], dtype=torch.int32, device="cuda")
    st["top_p"] = torch.full((n,), case["p"], device="cuda")
    st["min_p"] = torch.full((n,), case["min_p"], device="cuda")
    if n > 8:                            # every eighth row without a limit on the count
        st["top_k"][::8] = 0
        st["min_p"][3::8] = 0.0
    st["u"] = r()
    st["token"] = torch.zeros(n, dtype=torch.int32, device="cuda")
    st["kept"] = torch.zeros(n, dtype=torch.int32, device="cuda")
    st["logprob"] = torch.zeros(n, device="cuda")


def _handles(st, case):
    from non_prefix_kv_gb300 import binding as B
    st["B"] = B
    dt = B.CB_BF16 if case["dtype"] == "bf16" else B.CB_F32
    if case["op"] == "sample":
        st["rules"] = B.sample_rules(temperature=st["temperature"], top_k=st["top_k"], top_p=st["top_p"], min_p=st["min_p"])
        return
    h, hkv, hd = case["h"] or case["hkv"], case["hkv"], case["hd"]
    st["dims"] = B.cb_dims(h * hd, h, hkv, hd, 1024, 1024, _BASE, 1e-5, dt)
    if case["op"] == "rope":
        low, high, amp = _rope_numbers(case)
        rule = {"none": B.CB_ROPE_PLAIN, "linear": B.CB_ROPE_LINEAR, "base": B.CB_ROPE_BASE, "waves": B.CB_ROPE_WAVES,
                "ramp": B.CB_ROPE_RAMP}[case["scaling"]]
        st["spec"] = B.rope_spec(B.CB_ROPE_HALF if case["layout"] == "half" else B.CB_ROPE_INTERLEAVED, case["rot"], _BASE,
                                 scaling=rule, factor=case["factor"], original_len=_ORIGINAL, low=low, high=high,
                                 amplitude=amp)
        st["cos_sin"] = torch.empty(_FAR * case["rot"], device="cuda")
        B.cb_rope_table_scaled(st["cos_sin"], _FAR, st["spec"])
    else:
        st["shared"] = B.shared_kv(st["k"], st["v"], [r for r, _ in _prefixes(case)], [m for _, m in _prefixes(case)],
                                   _seq0(case), st["own_k"], st["own_v"])
        st["ws"] = torch.empty(B.cb_shared_workspace_bytes(st["shared"], st["dims"], case["n_q"]), dtype=torch.uint8,
                               device="cuda")


# ---------------------------------------------------------------------------- one pass
def run(st):
    return {"rope": _rope, "shared": _shared, "sample": _sample}[st["case"]["op"]](st)


def _rope(st):
    case = st["case"]
    if own:
        st["B"].cb_rope_rows(st["q"], st["k"], st["v"], st["pos"], st["q_out"], st["k_out"], st["v_out"], st["dims"],
                             st["spec"], st["cos_sin"], _FAR, src_row=st["src_row"], kv_row=st["kv_row"],
                             inverse=case["inverse"])
        return [t for t in (st["q_out"], st["k_out"], st["v_out"]) if t is not None]
    p = st["pos"].long()
    cs = st["table"][p.abs()]
    c, s = cs[:, None, :, 0], cs[:, None, :, 1] * torch.where(p < 0, -1.0, 1.0)[:, None, None]
    if case["inverse"]:
        s = -s
    src = slice(None) if st["src_row"] is None else st["src_row"].long()
    out = []
    if st["q"] is not None:
        out.append(_turn(st["q"], c, s, case))
    k, v = _turn(st["k"][src], c, s, case), st["v"][src]
    row = slice(0, case["rows"]) if st["kv_row"] is None else st["kv_row"].long()
    st["k_out"][row], st["v_out"][row] = k, v
    return out + [st["k_out"], st["v_out"]]


def _turn(x, c, s, case):
    n, hd, rot = x.shape[0], case["hd"], case["rot"]
    y = x.reshape(n, -1, hd).float()
    a = y[..., :rot]
    x1, x2 = (a[..., :rot // 2], a[..., rot // 2:]) if case["layout"] == "half" else (a[..., 0::2], a[..., 1::2])
    y1, y2 = x1 * c - x2 * s, x1 * s + x2 * c
    a = torch.cat([y1, y2], 2) if case["layout"] == "half" else torch.stack([y1, y2], 3).flatten(2)
    return torch.cat([a, y[..., rot:]], 2).reshape(n, -1).to(x.dtype)


def _shared(st):
    case = st["case"]
    n, nq, h, hkv, hd, cap = (case[k] for k in ("n_seq", "n_q", "h", "hkv", "hd", "cap"))
    if own:
        st["B"].cb_shared_attention(st["q"], st["last"], nq, st["shared"], st["dims"], st["o"], st["ws"])
        return st["o"]
    g = h // hkv
    q = st["q"].float().reshape(n, nq, hkv, g, hd).permute(2, 0, 1, 3, 4) * (1 / math.sqrt(hd))   # [hkv, n, nq, g, hd]
    heads = lambda t: t.float().reshape(*t.shape[:-1], hkv, hd)  # noqa: E731
    out = []
    for (row0, rows), a, b in zip(_prefixes(case), _seq0(case), _seq0(case)[1:]):
        if a == b:
            continue
        m = b - a
        kp, vp = (heads(t[row0:row0 + rows]).permute(1, 0, 2) for t in (st["k"], st["v"]))         # [hkv, rows, hd]
        ko, vo = (heads(t[a:b]).permute(2, 0, 1, 3) for t in (st["own_k"], st["own_v"]))           # [hkv, m, cap, hd]
        z = q[:, a:b].reshape(hkv, m * nq * g, hd)
        last = st["last"][a:b].repeat_interleave(g, 1)[None, :, :, None]
        sp = (z @ kp.transpose(1, 2)).reshape(hkv, m, nq * g, rows)
        so = z.reshape(hkv, m, nq * g, hd) @ ko.transpose(2, 3)
        so.masked_fill_(torch.arange(cap, device="cuda") > last, float("-inf"))
        top = sp.amax(3, keepdim=True)
        if cap:
            top = torch.maximum(top, so.amax(3, keepdim=True))
        sp.sub_(top).exp_()
        so.sub_(top).exp_()
        o = (sp.reshape(hkv, m * nq * g, rows) @ vp).reshape(hkv, m, nq * g, hd) + so @ vo
        o /= sp.sum(3, keepdim=True) + so.sum(3, keepdim=True)
        o.masked_fill_(last == -2, 0)
        out.append(o.reshape(hkv, m, nq, g, hd).permute(1, 2, 0, 3, 4).reshape(m, nq, h, hd).to(st["q"].dtype))
        del sp, so, o
    return torch.cat(out)


def _sample(st):
    case = st["case"]
    if own:
        st["B"].cb_sample_token(st["logits"], st["u"], st["rules"], st["token"], st["logprob"], st["kept"])
        return st["token"], st["logprob"], st["kept"]
    x = st["logits"].double()
    n, V = x.shape
    x, ids = torch.sort(x, dim=1, descending=True, stable=True)
    greedy = st["temperature"] == 0
    heat = torch.where(greedy, torch.ones_like(st["temperature"]), st["temperature"]).double()[:, None]
    w = ((x - x[:, :1]) / heat).exp()
    i = torch.arange(V, device="cuda")
    k = torch.where(st["top_k"] > 0, st["top_k"], torch.full_like(st["top_k"], V))
    k = torch.where(greedy, torch.ones_like(k), k)[:, None]
    keep = (x > float("-inf")) & (i < k)
    w = torch.where(keep, w, torch.zeros((), device="cuda", dtype=torch.float64))
    before = w.cumsum(1) - w
    p = st["top_p"].double()[:, None]
    keep &= (p >= 1) | (before < p * w.sum(1, keepdim=True)) | (i == 0)
    keep &= w >= st["min_p"].double()[:, None]
    w = torch.where(keep, w, torch.zeros((), device="cuda", dtype=torch.float64))
    total = w.sum(1, keepdim=True)
    by_id = torch.zeros_like(w).scatter_(1, ids, w)
    token = (by_id.cumsum(1) > st["u"].double()[:, None] * total).to(torch.uint8).argmax(1, keepdim=True)
    return token[:, 0].int(), (by_id.gather(1, token) / total).log()[:, 0].float(), keep.sum(1).int()


# ---------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The same outputs from the definitions in 64 bits, pair by pair, head by head and row by row."""
    st = prepare(case, seed)
    return {"rope": _rope64, "shared": _shared64, "sample": _sample64}[case["op"]](st)


def _rope64(st):
    case = st["case"]
    rot, hd = case["rot"], case["hd"]
    angle = st["pos"].double()[:, None] * _theta(case).cuda() * (-1.0 if case["inverse"] else 1.0)
    z = torch.polar(torch.full_like(angle, _rope_numbers(case)[2]), angle)         # one complex number per pair

    def turn(x):
        y = x.double().reshape(x.shape[0], -1, hd).clone()
        for i in range(rot // 2):
            a, b = (i, i + rot // 2) if case["layout"] == "half" else (2 * i, 2 * i + 1)
            t = torch.complex(y[..., a], y[..., b]) * z[:, None, i]
            y[..., a], y[..., b] = t.real, t.imag
        return y.reshape(x.shape[0], -1)

    src = torch.arange(case["rows"], device="cuda") if st["src_row"] is None else st["src_row"].long()
    dst = torch.arange(case["rows"], device="cuda") if st["kv_row"] is None else st["kv_row"].long()
    out = [] if st["q"] is None else [turn(st["q"])]
    for x, y in ((turn(st["k"][src]), st["k_out"]), (st["v"][src].double(), st["v_out"])):
        out.append(y.double().index_copy_(0, dst, x))
    return out


def _shared64(st):
    case = st["case"]
    n, nq, h, hkv, hd = (case[k] for k in ("n_seq", "n_q", "h", "hkv", "hd"))
    g = h // hkv
    o = torch.zeros(n, nq, h, hd, dtype=torch.float64, device="cuda")
    last = st["last"].tolist()
    col = lambda t, kv: t[..., kv * hd:(kv + 1) * hd].double()  # noqa: E731
    for (row0, rows), a, b in zip(_prefixes(case), _seq0(case), _seq0(case)[1:]):
        for kv in range(hkv):
            kp, vp = col(st["k"][row0:row0 + rows], kv), col(st["v"][row0:row0 + rows], kv)
            for s in range(a, b):
                live = [j for j in range(nq) if last[s][j] > -2]
                m = max(last[s]) + 1
                k, v = torch.cat([kp, col(st["own_k"][s, :m], kv)]), torch.cat([vp, col(st["own_v"][s, :m], kv)])
                q = st["q"][s, live, kv * g:(kv + 1) * g].double()                    # [queries, g, hd]
                z = torch.einsum("jgc,ic->jgi", q, k) / math.sqrt(hd)
                i = torch.arange(rows + m, device="cuda")
                z[(i >= rows + 1 + st["last"][s, live, None]).unsqueeze(1).expand_as(z)] = float("-inf")
                o[s, live, kv * g:(kv + 1) * g] = torch.einsum("jgi,ic->jgc", torch.softmax(z, 2), v)
    return o


def _sample64(st):
    tok, lp, kept = [], [], []
    for b in range(st["case"]["rows"]):
        x = st["logits"][b].double().cpu().numpy()
        heat, k, p, m, u = (float(st[a][b]) for a in ("temperature", "top_k", "top_p", "min_p", "u"))
        order = np.argsort(-x, kind="stable")
        order = order[:np.count_nonzero(x > -np.inf)]
        if heat == 0:
            heat, k = 1.0, 1
        if k > 0:
            order = order[:int(k)]
        w = np.exp((x[order] - x[order[0]]) / heat)
        if p < 1:
            order = order[:1 + int(np.searchsorted(np.cumsum(w), p * math.fsum(w)))]
        order = order[:np.count_nonzero(w[:len(order)] >= m)]
        ids = np.sort(order)
        w = np.exp((x[ids] - x.max()) / heat)
        total = math.fsum(w)
        at = min(int(np.searchsorted(np.cumsum(w), u * total, side="right")), len(ids) - 1)
        tok.append(int(ids[at]))
        lp.append((x[ids[at]] - x.max()) / heat - math.log(total))
        kept.append(len(ids))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    return i32(tok), torch.tensor(lp, dtype=torch.float64, device="cuda"), i32(kept)


# ---------------------------------------------------------------------------- work
def work(case):
    """Bytes and operations that one pass cannot do without."""
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rope":
        n, W = case["rows"], (case["h"] + 2 * case["hkv"]) * case["hd"]
        return {"bytes": n * (2 * e * W + 12), "flops": n * 3 * (case["h"] + case["hkv"]) * case["rot"]}
    if case["op"] == "sample":
        n, V = case["rows"], case["vocab"]
        return {"bytes": n * (e * V + 32), "flops": 4 * n * V}
    n, nq, h, hkv, hd = (case[k] for k in ("n_seq", "n_q", "h", "hkv", "hd"))
    held = sum(r for _, r in _prefixes(case)) + sum(_lens(case))
    pairs = 0
    for (_, rows), a, b in zip(_prefixes(case), _seq0(case), _seq0(case)[1:]):
        for s in range(a, b):
            m, l = _queries(case)[s], _lens(case)[s]
            pairs += m * (rows + l) - (m * (m - 1) // 2 if nq > 1 else 0)
    return {"bytes": 2 * e * held * hkv * hd + 2 * e * n * nq * h * hd + 4 * n * nq, "flops": 4 * h * hd * pairs}
