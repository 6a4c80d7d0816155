"""Workloads of the operators behind a blended prefill: the KV cache held in 8 bits with one
scale per block of tokens and head, attention over it (with the attention weight each row
receives), eviction by that weight, and the rules on the logits before the next token.

Each workload has a plain form (elementary torch operations in fp32, rounded once at the end)
and the library's own calls.  `own` chooses between them.

Formulas (s = sequence, h = KV head, b = block of `block` rows, G = query heads per KV head):

  append   a block's scale  sc = max(amax|x| / 127, 1e-8) over its new rows, rounded to fp32; a
           block that already holds rows keeps at least its old scale, and its codes c become
           rne(c * old / sc); new codes  c = rne(x / sc) in [-127, 127].  Which integer is the
           nearest is decided exactly (quotients at a half are common: 64 bits here)
  read     x = c * sc
  attend   o[j] = sum_{i <= last[j]} softmax_i(q[j] . k[i] / sqrt(hd)) v[i]; last = -1: zeros
           weights[s, h, i] += sum over the queries j and the G heads of h of that softmax
  evict    rows kept of [0, len): the first n_sink, the last n_recent and the heaviest others,
           n_keep in all (everything while len <= n_keep), ascending, moved to rows 0, 1, ... of
           another cache and re-coded there as by append into empty blocks
  logits   x > 0 ? x / r : x * r for ids seen; x -= frequency * count + presence * (count > 0)
           over the generated ids; x += biases of the id; -inf where the mask bit is 0;
           token = lowest index of the largest, -1 if none is above -inf
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # a decoding step of four answers: one new row each, inside a block (latency)
        dict(name="append_token_7b", op="append", n_seq=4, rows=1, h=32, hkv=32, hd=128, cap=4096, block=32,
             start="ragged", dtype="bf16"),
        # the blended prompts of four requests, an odd number of rows, moved into 8 bits
        dict(name="append_prompt_yi", op="append", n_seq=4, rows=16001, h=56, hkv=8, hd=128, cap=16384, block=64,
             start="zero", dtype="bf16"),
        # the first tokens of one answer after a 4096-token blend
        dict(name="attend_token_7b", op="attend", n_seq=1, n_q=1, h=32, hkv=32, hd=128, cap=4160, block=32,
             last="tail", weigh=False, dtype="bf16"),
        # a batch of 32 answers of different lengths, grouped heads
        dict(name="attend_token_yi_b32", op="attend", n_seq=32, n_q=1, h=56, hkv=8, hd=128, cap=16384, block=64,
             last="tail", weigh=False, dtype="bf16"),
        # the selected rows of a blend (576 + 256 of 4096) over an 8-bit cache
        dict(name="attend_selected_7b", op="attend", n_seq=1, n_q=832, h=32, hkv=32, hd=128, cap=4096, block=64,
             last="selected", weigh=False, dtype="bf16"),
        # the largest: the selected rows of a 16K request with grouped heads
        dict(name="attend_selected_yi", op="attend", n_seq=1, n_q=3328, h=56, hkv=8, hd=128, cap=16384, block=128,
             last="selected", weigh=False, dtype="bf16"),
        # decoding steps that keep account of the attention each row receives
        dict(name="weigh_token_13b", op="attend", n_seq=8, n_q=1, h=40, hkv=40, hd=128, cap=8192, block=32,
             last="tail", weigh=True, dtype="bf16"),
        # the last 64 prompt rows weigh the whole prompt before it is thinned out
        dict(name="weigh_window_yi", op="attend", n_seq=1, n_q=64, h=56, hkv=8, hd=128, cap=16384, block=64,
             last="tail", weigh=True, dtype="bf16"),
        # one answer's cache halved
        dict(name="evict_7b", op="evict", n_seq=1, h=32, hkv=32, hd=128, cap=4096, keep=2048, sink=4, recent=256,
             block=32, dtype="bf16"),
        # a batch of long caches of different lengths thinned out to a quarter
        dict(name="evict_yi_b16", op="evict", n_seq=16, h=56, hkv=8, hd=128, cap=16384, keep=4100, sink=4,
             recent=1024, block=64, dtype="bf16"),
        # the next token of one answer
        dict(name="logits_7b", op="logits", rows=1, vocab=32000, hist=4352, prompt=4096, bias=16, mask=True,
             dtype="f32"),
        # a batch of answers over a large vocabulary
        dict(name="logits_yi_b64", op="logits", rows=64, vocab=64000, hist=2048, prompt=1800, bias=300, mask=True,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "weigh", "evict", "logits"])
    hkv, g = rng.choice([(32, 1), (40, 1), (8, 7), (4, 1), (8, 4), (2, 4)])
    hd = rng.choice([128, 128, 64])
    block = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    heads = dict(h=hkv * g, hkv=hkv, hd=hd)
    if op == "append":
        n_seq, rows = rng.choice([(_log(rng, 1, 64), _log(rng, 1, 8)), (rng.randint(1, 4), _log(rng, 100, 16000))])
        cap = -(-(rows + rng.randint(0, 1000)) // block) * block + block
        while n_seq > 1 and n_seq * cap * hkv * hd > 4 * 16384 * 1024:
            n_seq -= 1
        return dict(op=op, n_seq=n_seq, rows=rows, **heads, cap=cap, block=block,
                    start=rng.choice(["ragged", "zero"]) if cap > rows else "zero", dtype=dtype)
    if op in ("attend", "weigh"):
        n_kv = _log(rng, 32, 16384)
        cap = -(-n_kv // block) * block
        last = rng.choice(["tail", "selected"])
        if last == "tail":
            n_seq, n_q = _log(rng, 1, 32), rng.choice([1, 1, 1, rng.randint(2, 8), rng.randint(9, 100)])
        else:
            n_seq, n_q = rng.choice([1, 1, 2]), _log(rng, 16, min(3328, n_kv))
        if dtype == "f32":   # exact arithmetic: small work only
            n_seq, n_q = min(n_seq, 4), min(n_q, 100)
        n_q = min(n_q, n_kv)
        # at most the work of the largest listed ones, and a score matrix that fits
        while n_seq > 1 and (n_seq * cap * hkv * hd > 32 * 16384 * 1024 or
                             n_seq * n_q * hkv * g * cap > 3328 * 56 * 16384):
            n_seq -= 1
        return dict(op="attend", n_seq=n_seq, n_q=n_q, **heads, cap=cap, block=block, last=last, weigh=op == "weigh",
                    dtype=dtype)
    if op == "evict":
        n_seq, n_kv = _log(rng, 1, 16), _log(rng, 40, 16384)
        cap = -(-n_kv // block) * block
        while n_seq > 1 and n_seq * cap * hkv * hd > 16 * 16384 * 1024:
            n_seq -= 1
        keep = max(2, int(cap * rng.uniform(0.1, 0.9)))
        sink = min(rng.choice([0, 1, 4]), keep // 2)
        return dict(op=op, n_seq=n_seq, **heads, cap=cap, keep=keep, sink=sink,
                    recent=int((keep - sink) * rng.uniform(0, 0.9)), block=block, dtype="bf16")
    hist = _log(rng, 1, 8000)
    return dict(op=op, rows=_log(rng, 1, 64), vocab=rng.choice([32000, 64000, 1024, 5000, rng.randint(3, 64000)]),
                hist=hist, prompt=int(hist * rng.uniform(0, 1)), bias=rng.choice([0, 1, 16, 300]),
                mask=rng.random() < 0.6, dtype=rng.choice(["f32", "bf16"]))


# ---------------------------------------------------------------------------- inputs
def _lens(case):
    """Rows held by each sequence: spread over 55..100 % of the capacity, the first one whole."""
    n, cap = case["n_seq"], case["cap"]
    return [max(1, cap - (cap * 45 * ((i * 5) % n)) // (100 * n)) for i in range(n)]


def _starts(case):
    n, top = case["n_seq"], case["cap"] - case["rows"]
    if case["start"] == "zero":
        return [0] * n
    return [max(0, top - 7 * i - (top * ((i * 3) % n)) // (2 * n)) for i in range(n)]


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _kv(g, n_seq, rows, hkv, hd, k_like):
    """K and V rows as a model leaves them: keys with a few strong channels, token norms that vary."""
    x = _normal(g, n_seq, rows, hkv, hd)
    if k_like:
        x *= 1 + 3 * (torch.rand(hkv, hd, generator=g, device="cuda") < 0.04)
    x *= 0.5 + torch.rand(n_seq, rows, 1, 1, generator=g, device="cuda")
    return x.reshape(n_seq, rows, hkv * hd)


def _filled(g, case, rows):
    """A cache holding `rows` rows per sequence: codes and block scales, drawn as codes."""
    n, hkv, hd, cap, block = (case[k] for k in ("n_seq", "hkv", "hd", "cap", "block"))
    out = []
    for _ in range(2):
        c = torch.empty(n, hkv, cap, hd, dtype=torch.int8, device="cuda")
        for s in range(n):
            c[s] = (_normal(g, hkv, cap, hd) * 34).round_().clamp_(-127, 127).to(torch.int8)
        out += [c, 0.02 + 0.03 * torch.rand(n, hkv, cap // block, generator=g, device="cuda")]
    return out


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    st = {"case": case}
    if op == "logits":
        B, V, T = case["rows"], case["vocab"], case["hist"]
        st["logits"] = (_normal(g, B, V) * 2.5).to(_DT[case["dtype"]])
        # ids repeat as words do: most from a small part of the vocabulary
        u = torch.rand(B, T, generator=g, device="cuda")
        st["hist"] = (u.pow(4) * V).long().clamp_(max=V - 1).int()
        st["hist_len"] = torch.tensor([T - (T * i) // (3 * B) for i in range(B)], dtype=torch.int32, device="cuda")
        st["prompt_len"] = st["hist_len"].clamp(max=case["prompt"])
        st["rep"] = 1.0 + 0.3 * torch.rand(B, generator=g, device="cuda")
        st["pres"] = 0.5 * torch.rand(B, generator=g, device="cuda")
        st["freq"] = 0.2 * torch.rand(B, generator=g, device="cuda")
        n = case["bias"]
        st["bias_id"] = (torch.rand(B, n, generator=g, device="cuda") * V).long().clamp_(max=V - 1).int()
        st["bias"] = _normal(g, B, n) * 3
        W = (V + 31) // 32
        # a grammar leaves about half of the ids open
        st["mask"] = (torch.randint(-2 ** 31, 2 ** 31, (B, W), generator=g, device="cuda", dtype=torch.int64).int()
                      if case["mask"] else None)
        st["out"] = torch.empty_like(st["logits"])
        st["token"] = torch.empty(B, dtype=torch.int32, device="cuda")
    else:
        n, hkv, hd, cap, block = (case[k] for k in ("n_seq", "hkv", "hd", "cap", "block"))
        dt = _DT[case["dtype"]]
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        st["kc"], st["ks"], st["vc"], st["vs"] = _filled(g, case, cap)
        if op == "append":
            st["k"] = _kv(g, n, case["rows"], hkv, hd, True).to(dt)
            st["v"] = _kv(g, n, case["rows"], hkv, hd, False).to(dt)
            s0 = _starts(case)
            st["start"] = i32(s0)
            # what a reader of the touched blocks asks for: from the first one's first row
            st["r_start"] = i32([s // block * block for s in s0])
            st["r_count"] = i32([s % block + case["rows"] for s in s0])
            st["r_rows"] = block - 1 + case["rows"]
        elif op == "attend":
            nq = case["n_q"]
            # scores of standard deviation 1.4: some rows draw most of the attention
            st["q"] = (_normal(g, n, nq, case["h"], hd) * (1.4 / math.sqrt(0.035 ** 2 * 34 ** 2))).to(dt)
            if case["last"] == "tail":
                # the newest n_q rows of each sequence; the shorter ones bring fewer queries
                rows = []
                for i, l in enumerate(_lens(case)):
                    m = max(1, nq - (nq * i) // (2 * n))
                    rows.append([max(0, l - m + j) for j in range(m)] + [-1] * (nq - m))
                st["last"] = i32(rows)
            else:
                tail = max(1, nq * 4 // 13)
                picks = [torch.randperm(cap - tail, generator=g, device="cuda")[:nq - tail].sort().values
                         for _ in range(n)]
                st["last"] = torch.stack([torch.cat([p, torch.arange(cap - tail, cap, device="cuda")])
                                          for p in picks]).int()
            st["w0"] = (torch.rand(n, hkv, cap, generator=g, device="cuda") * 0.1 if case["weigh"] else None)
            st["o"] = torch.empty_like(st["q"])
        else:
            st["len"] = i32(_lens(case))
            st["w"] = torch.rand(n, hkv, cap, generator=g, device="cuda").pow(8) * 30
            dcap = -(-case["keep"] // block) * block
            st["d_kc"] = torch.zeros(n, hkv, dcap, hd, dtype=torch.int8, device="cuda")
            st["d_vc"] = torch.zeros_like(st["d_kc"])
            st["d_ks"] = torch.zeros(n, hkv, dcap // block, device="cuda")
            st["d_vs"] = torch.zeros_like(st["d_ks"])
            st["d_w"] = torch.zeros(n, hkv, dcap, device="cuda")
            st["d_len"] = torch.zeros(n, dtype=torch.int32, device="cuda")
            st["kept"] = torch.zeros(n, hkv, case["keep"], dtype=torch.int32, device="cuda")
            st["r_start"] = i32([0] * n)
            st["r_count"] = st["d_len"]
            st["r_rows"] = case["keep"]
        if "r_rows" in st:
            st["k_back"] = torch.zeros(n, st["r_rows"], hkv * hd, device="cuda")
            st["v_back"] = torch.zeros_like(st["k_back"])
    if own:   # the handles and the scratch that a decoding program keeps between calls
        st.update(_handles(st))
    return st


def _handles(st):
    from non_prefix_kv_gb300 import binding as B
    case = st["case"]
    if case["op"] == "logits":
        none = lambda t, on: t if on else None  # noqa: E731
        return {"B": B, "rules": B.logit_rules(
            history=st["hist"], history_len=st["hist_len"], prompt_len=st["prompt_len"], repetition=st["rep"],
            presence=st["pres"], frequency=st["freq"], bias_id=none(st["bias_id"], case["bias"]),
            bias=none(st["bias"], case["bias"]), mask=st["mask"])}
    make = lambda dt: B.cb_dims(case["h"] * case["hd"], case["h"], case["hkv"], case["hd"], 1024, 1024, 1e4, 1e-5, dt)  # noqa: E731
    out = {"B": B, "dims": make(B.CB_BF16 if case["dtype"] == "bf16" else B.CB_F32), "dims32": make(B.CB_F32),
           "cache": B.kv8_cache(st["kc"], st["vc"], st["ks"], st["vs"], case["block"])}
    if case["op"] == "attend":
        n = B.cb_kv8_workspace_bytes(out["dims"], case["n_seq"], case["cap"], case["n_q"], case["weigh"])
        out["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    if case["op"] == "evict":
        out["dst"] = B.kv8_cache(st["d_kc"], st["d_vc"], st["d_ks"], st["d_vs"], case["block"])
    return out


# ---------------------------------------------------------------------------- one pass
def run(st):
    return {"append": _append, "attend": _attend, "evict": _evict, "logits": _logits}[st["case"]["op"]](st)


def _append(st):
    case = st["case"]
    if own:
        B = st["B"]
        B.cb_kv8_append(st["k"], st["v"], case["rows"], st["start"], None, st["cache"], st["dims"])
        B.cb_kv8_read(st["cache"], st["r_start"], st["r_count"], st["r_rows"], st["dims32"], st["k_back"], st["v_back"])
        return st["k_back"], st["v_back"]
    return (_append_plain(st, st["k"], st["kc"], st["ks"]), _append_plain(st, st["v"], st["vc"], st["vs"]))


def _scale(amax):
    return (amax.double() / 127).float().clamp(min=1e-8)


def _append_plain(st, x, codes, scale):
    """The blocks that the new rows touch: old rows re-coded, new rows coded, read back as values."""
    case = st["case"]
    n, hkv, hd, cap, block, rows = (case[k] for k in ("n_seq", "hkv", "hd", "cap", "block", "rows"))
    nb = (block - 1 + rows + block - 1) // block
    start = st["start"].long()
    b0 = start // block
    r = b0[:, None] * block + torch.arange(nb * block, device="cuda")            # cache rows of these blocks
    j = r - start[:, None]                                                        # their new row
    is_new = (j >= 0) & (j < rows) & (r < cap)
    kept = j < 0
    si = torch.arange(n, device="cuda")[:, None]
    xn = x.float().reshape(n, rows, hkv, hd)[si, j.clamp(0, rows - 1)]
    xn = torch.where(is_new[..., None, None], xn, torch.zeros((), device="cuda"))
    rc = r.clamp(max=cap - 1)
    old = codes[si, :, rc].float()                                                # [n, rows of blocks, hkv, hd]
    bi = b0[:, None] + torch.arange(nb, device="cuda")
    bc = bi.clamp(max=cap // block - 1)
    old_s = scale[si, :, bc]                                                      # [n, nb, hkv]
    has_old = kept.reshape(n, nb, block).any(2)[..., None]
    has_new = is_new.reshape(n, nb, block).any(2)
    amax = xn.reshape(n, nb, block, hkv, hd).abs().amax((2, 4))
    s = torch.maximum(_scale(amax), torch.where(has_old, old_s, torch.zeros_like(old_s)))
    s = torch.where(has_new[..., None], s, old_s)
    up = lambda t: t.repeat_interleave(block, 1)[..., None]  # noqa: E731
    s64 = up(s.double())
    c = torch.where(kept[..., None, None], old * up(old_s.double()) / s64, xn / s64).round().clamp(-127, 127).float()
    live = (kept | is_new) & up(has_new[..., None])[..., 0, 0]
    where = live.nonzero(as_tuple=True)
    codes[where[0], :, r[where]] = c[where].to(torch.int8)
    hit = has_new.nonzero(as_tuple=True)
    scale[hit[0], :, bi[hit]] = s[hit]
    return torch.where(live[..., None, None], c * up(s), torch.zeros((), device="cuda")).reshape(
        n, nb * block, hkv * hd)[:, :st["r_rows"]].contiguous()


def _values(codes, scale, block):
    return codes.float() * scale.repeat_interleave(block, 2)[..., None]


def _attend(st):
    case = st["case"]
    w = st["w0"].clone() if case["weigh"] else None      # the account so far, carried on by this pass
    if own:
        st["B"].cb_kv8_attention(st["q"], st["last"], case["n_q"], st["cache"], st["dims"], st["o"], w, st["ws"])
        return (st["o"], w) if case["weigh"] else st["o"]
    n, nq, h, hkv, hd, cap, block = (case[k] for k in ("n_seq", "n_q", "h", "hkv", "hd", "cap", "block"))
    g = h // hkv
    q = st["q"].float().reshape(n, nq, hkv, g, hd).permute(0, 2, 1, 3, 4).reshape(n, hkv, nq * g, hd)
    k = _values(st["kc"], st["ks"], block)
    p = q @ k.transpose(2, 3)
    del k
    p *= 1 / math.sqrt(hd)
    last = st["last"].repeat_interleave(g, 1)[:, None, :, None]
    p.masked_fill_(torch.arange(cap, device="cuda") > last, float("-inf"))
    m = p.amax(3, keepdim=True)
    p -= torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p.exp_()
    l = p.sum(3, keepdim=True)
    p /= torch.where(l > 0, l, torch.ones_like(l))
    o = p @ _values(st["vc"], st["vs"], block)
    o = o.reshape(n, hkv, nq, g, hd).permute(0, 2, 1, 3, 4).reshape(n, nq, h, hd).to(st["q"].dtype)
    return (o, w + p.sum(2)) if case["weigh"] else o


def _evict(st):
    case = st["case"]
    if own:
        B = st["B"]
        B.cb_kv8_evict(st["cache"], st["len"], st["w"], case["keep"], case["sink"], case["recent"], st["dst"],
                       st["d_len"], st["d_w"], st["kept"], st["dims"])
        B.cb_kv8_read(st["dst"], st["r_start"], st["r_count"], st["r_rows"], st["dims32"], st["k_back"], st["v_back"])
        return st["kept"], st["d_len"], st["d_w"], st["k_back"], st["v_back"]
    n, hkv, hd, cap, block, keep = (case[k] for k in ("n_seq", "hkv", "hd", "cap", "block", "keep"))
    ln = st["len"].long()[:, None, None]
    i = torch.arange(cap, device="cuda")
    must = (i < case["sink"]) | (i >= ln - case["recent"]) | (ln <= keep)
    score = torch.where(must, torch.full_like(st["w"], float("inf")), st["w"])
    score = torch.where(i < ln, score, torch.full_like(score, float("-inf")))
    order = torch.sort(score, dim=2, descending=True, stable=True).indices[..., :keep]
    n_out = ln.clamp(max=keep)
    j = torch.arange(keep, device="cuda")
    kept = torch.where(j < n_out, order, torch.full_like(order, cap)).sort(2).values    # the unused places last
    held = kept < cap
    src = kept.clamp(max=cap - 1)
    dcap = -(-keep // block) * block
    w = torch.zeros(n, hkv, dcap, device="cuda")
    w[..., :keep] = torch.where(held, st["w"].gather(2, src), torch.zeros((), device="cuda"))
    back = []
    for codes, scale in ((st["kc"], st["ks"]), (st["vc"], st["vs"])):
        x = codes.gather(2, src[..., None].expand(-1, -1, -1, hd)).float() * scale.gather(2, src // block)[..., None]
        full = torch.zeros(n, hkv, dcap, hd, device="cuda")
        full[:, :, :keep] = torch.where(held[..., None], x, torch.zeros((), device="cuda"))
        s = _scale(full.reshape(n, hkv, dcap // block, block, hd).abs().amax((3, 4)))
        s = s.repeat_interleave(block, 2)[..., None]
        y = (full.double() / s).round().clamp(-127, 127).float() * s
        back.append(y[:, :, :keep].transpose(1, 2).reshape(n, keep, hkv * hd))
    return (torch.where(held, kept, torch.full_like(kept, -1)).int(), n_out[:, 0, 0].int(), w, back[0], back[1])


def _logits(st):
    case = st["case"]
    if own:
        st["B"].cb_logits_process(st["logits"], st["rules"], st["out"], st["token"])
        return st["out"], st["token"]
    rows, V = case["rows"], case["vocab"]
    x = st["logits"].float()
    t = torch.arange(case["hist"], device="cuda")
    ids = st["hist"].long()
    held = t < st["hist_len"][:, None]
    made = (held & (t >= st["prompt_len"][:, None])).float()
    zero = torch.zeros(rows, V, device="cuda")
    seen = zero.scatter_add(1, ids, held.float()) > 0
    count = zero.scatter_add(1, ids, made)
    rep = st["rep"][:, None]
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = x - (st["freq"][:, None] * count + st["pres"][:, None] * (count > 0))
    if case["bias"]:
        x = x + zero.scatter_add(1, st["bias_id"].long(), st["bias"])
    if case["mask"]:
        i = torch.arange(V, device="cuda")
        x = torch.where((st["mask"][:, i // 32] >> (i % 32)) & 1 > 0, x, torch.full_like(x, float("-inf")))
    out = x.to(st["logits"].dtype)
    top = out.float().amax(1, keepdim=True)
    i = torch.arange(V, device="cuda").expand(rows, V)
    token = torch.where(out.float() == top, i, torch.full_like(i, V)).amin(1)
    return out, torch.where(top[:, 0] == float("-inf"), torch.full_like(token, -1), token).int()


# ---------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    """The same outputs from the definitions in 64 bits, sequence by sequence and head by head."""
    st = prepare(case, seed)
    return {"append": _append64, "attend": _attend64, "evict": _evict64, "logits": _logits64}[case["op"]](st)


def _code64(x, s):
    return torch.round(x / s).clamp_(-127, 127)


def _append64(st):
    case = st["case"]
    hkv, hd, block, rows = (case[k] for k in ("hkv", "hd", "block", "rows"))
    out = []
    for x, codes, scale in ((st["k"], st["kc"], st["ks"]), (st["v"], st["vc"], st["vs"])):
        back = torch.zeros(case["n_seq"], st["r_rows"], hkv, hd, dtype=torch.float64, device="cuda")
        for s, a in enumerate(st["start"].tolist()):
            lo = a // block * block
            for b in range(lo, a + rows, block):
                f, e = max(a, b), min(a + rows, b + block)
                new = x[s, f - a:e - a].double().reshape(e - f, hkv, hd)
                # a stored scale is a 32-bit value
                sc = (new.abs().amax((0, 2)) / 127).float().double().clamp_(min=float(np.float32(1e-8)))
                if b < a:
                    old_s = scale[s, :, b // block].double()
                    sc = torch.maximum(sc, old_s)
                    old = codes[s, :, b:a].double().transpose(0, 1)
                    back[s, b - lo:a - lo] = _code64(old * old_s[:, None], sc[:, None]) * sc[:, None]
                back[s, f - lo:e - lo] = _code64(new, sc[:, None]) * sc[:, None]
        out.append(back.reshape(case["n_seq"], st["r_rows"], hkv * hd))
    return tuple(out)


def _attend64(st):
    case = st["case"]
    n, nq, h, hkv, hd, cap, block = (case[k] for k in ("n_seq", "n_q", "h", "hkv", "hd", "cap", "block"))
    g = h // hkv
    o = torch.zeros(n, nq, h, hd, dtype=torch.float64, device="cuda")
    w = st["w0"].double() if case["weigh"] else None
    i = torch.arange(cap, device="cuda")
    per = max(1, (1 << 28) // cap)                      # query rows at a time
    for s in range(n):
        for kv in range(hkv):
            k = st["kc"][s, kv].double() * st["ks"][s, kv].double().repeat_interleave(block)[:, None]
            v = st["vc"][s, kv].double() * st["vs"][s, kv].double().repeat_interleave(block)[:, None]
            for a in range(0, nq, per):
                for hh in range(kv * g, kv * g + g):
                    z = st["q"][s, a:a + per, hh].double() @ k.T / math.sqrt(hd)
                    z = z.masked_fill(i > st["last"][s, a:a + per, None], float("-inf"))
                    p = torch.nan_to_num(torch.softmax(z, 1))      # a row that sees nothing: 0
                    o[s, a:a + per, hh] = p @ v
                    if w is not None:
                        w[s, kv] += p.sum(0)
    return (o, w) if case["weigh"] else o


def _evict64(st):
    case = st["case"]
    n, hkv, hd, block, keep = (case[k] for k in ("n_seq", "hkv", "hd", "block", "keep"))
    kept = torch.full((n, hkv, keep), -1, dtype=torch.int32, device="cuda")
    dw = torch.zeros(st["d_w"].shape, dtype=torch.float64, device="cuda")
    dl = torch.zeros(n, dtype=torch.int32, device="cuda")
    back = [torch.zeros(n, keep, hkv, hd, dtype=torch.float64, device="cuda") for _ in range(2)]
    for s, ln in enumerate(st["len"].tolist()):
        m = min(ln, keep)
        dl[s] = m
        for kv in range(hkv):
            if ln <= keep:
                rows = np.arange(ln)
            else:
                lo, hi = case["sink"], ln - case["recent"]
                w = st["w"][s, kv, lo:hi].double().cpu().numpy()
                best = np.argsort(-w, kind="stable")[:keep - case["sink"] - case["recent"]] + lo
                rows = np.sort(np.concatenate([np.arange(lo), best, np.arange(hi, ln)]))
            r = torch.from_numpy(rows).cuda()
            kept[s, kv, :m] = r.int()
            dw[s, kv, :m] = st["w"][s, kv, r].double()
            for b, (codes, scale) in zip(back, ((st["kc"], st["ks"]), (st["vc"], st["vs"]))):
                # the value that is moved is the 32-bit product of code and scale
                x = (codes[s, kv, r].float() * scale[s, kv, r // block][:, None]).double()
                pad = torch.zeros(-(-m // block) * block, hd, dtype=torch.float64, device="cuda")
                pad[:m] = x
                sc = (pad.reshape(-1, block * hd).abs().amax(1) / 127).float().double()
                sc = sc.clamp_(min=float(np.float32(1e-8))).repeat_interleave(block)[:m, None]
                b[s, :m, kv] = _code64(x, sc) * sc
    return kept, dl, dw, back[0].reshape(n, keep, hkv * hd), back[1].reshape(n, keep, hkv * hd)


def _logits64(st):
    case = st["case"]
    V = case["vocab"]
    out = torch.empty(case["rows"], V, dtype=torch.float64, device="cuda")
    tok = []
    for b in range(case["rows"]):
        x = st["logits"][b].double().cpu().numpy()
        ln, pl = int(st["hist_len"][b]), int(st["prompt_len"][b])
        ids = st["hist"][b, :ln].cpu().numpy()
        r, f, p = (float(st[k][b]) for k in ("rep", "freq", "pres"))
        seen = np.unique(ids)
        x[seen] = np.where(x[seen] > 0, x[seen] / r, x[seen] * r)
        made, count = np.unique(ids[pl:], return_counts=True)
        x[made] -= f * count + p
        np.add.at(x, st["bias_id"][b].cpu().numpy(), st["bias"][b].double().cpu().numpy())
        if case["mask"]:
            bits = np.unpackbits(st["mask"][b].cpu().numpy().view(np.uint8), bitorder="little")[:V]
            x[bits == 0] = -np.inf
        out[b] = torch.from_numpy(x).cuda()
        # the token is chosen among the values as they are returned
        y = torch.from_numpy(x).to(st["logits"].dtype).double().numpy()
        tok.append(-1 if y.max() == -np.inf else int(np.argmax(y)))
    return out, torch.tensor(tok, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------- work
def work(case):
    """Bytes and operations that one pass cannot do without."""
    op = case["op"]
    if op == "logits":
        B, V = case["rows"], case["vocab"]
        e = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": B * (2 * e * V + 4 * case["hist"] + 8 * case["bias"] + (V // 8 if case["mask"] else 0) + 28),
                "flops": 8 * B * V}
    n, h, hkv, hd, cap, block = (case[k] for k in ("n_seq", "h", "hkv", "hd", "cap", "block"))
    e = 2 if case["dtype"] == "bf16" else 4
    row = 2 * hkv * hd                                             # K and V codes of one cache row
    if op == "append":
        new, old = n * case["rows"], sum(s % block for s in _starts(case))
        return {"bytes": new * row * (e + 1) + (new + old) * row * (1 + 4) + 8 * hkv * (new + old) // block,
                "flops": 4 * (new + old) * row}
    if op == "attend":
        nq = case["n_q"]
        if case["last"] == "tail":
            lens, pairs = _lens(case), 0
            for i, l in enumerate(lens):
                m = max(1, nq - (nq * i) // (2 * n))
                pairs += sum(max(1, l - m + j + 1) for j in range(m))
            held = sum(lens)
        else:
            tail = max(1, nq * 4 // 13)
            pairs = n * (tail * (cap - tail / 2) + (nq - tail) * (cap - tail) / 2)
            held = n * cap
        return {"bytes": int(held * row + 8 * hkv * held // block + 2 * e * n * nq * h * hd + 4 * n * nq
                             + (8 * hkv * held if case["weigh"] else 0)),
                "flops": int(4 * h * hd * pairs)}
    lens = _lens(case)
    out = sum(min(l, case["keep"]) for l in lens)
    return {"bytes": sum(lens) * hkv * 4 + out * (row * (1 + 1 + 4) + hkv * (4 + 4) + 16 * hkv // block),
            "flops": 4 * out * row}

