"""The 8-bit cache's attention, its account of weights and the logit rules where they are easily
wrong: queries that are not finite, padding, keys split over CTAs, tiny queries, very long
caches, one buffer for calls of different sizes.  Oracle and tolerances as in test_gpu_kv8.py."""
import numpy as np
import pytest

import oracle.kv8_oracle as K8
from tests.gpu_util import dev, dev_i32, ensure_lib, host, tdt, torch_mod
from tests.test_gpu_kv8 import (Dev, attend, check_attention, check_cache, filled, make_dims, rounded, run_logits)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    torch_mod()
    ensure_lib()
    from non_prefix_kv_gb300 import binding
    return binding


# Which kernels take the call: few rows in one tile and in more; one query tile (bf16 converts the
# codes itself), several.  One sequence over 9 key tiles: the keys are split over a cluster.
WAYS = [(2, 2, 64, 3), (4, 2, 64, 7), (2, 2, 64, 30), (2, 2, 128, 60), (4, 2, 64, 90), (2, 2, 128, 140)]   # H, hkv, hd, n_q


# ------------------------------------------------------------------ queries that are not finite
@pytest.mark.parametrize("what", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,hkv,hd,n_q", WAYS)
def test_padding_weighs_nothing_whatever_it_holds(B, H, hkv, hd, n_q, dtype, what):
    """Queries that see nothing (last = -1) may hold anything; the others see whole key tiles."""
    torch = torch_mod()
    g = np.random.default_rng(n_q)
    cap = 1152
    d, o = filled(B, g, 1, hkv, cap, hd, 32, [cap])
    q = rounded(g.standard_normal((1, n_q, H, hd)), dtype)
    last = np.sort(g.integers(cap - 100, cap, (1, n_q)))
    pad = [0, n_q // 2, n_q - 1]
    last[0, pad] = -1
    bad = q.copy()
    bad[0, pad] = what
    w = torch.zeros(1, hkv, cap, device="cuda")
    out = attend(B, d, bad, last, make_dims(B, H, hkv, hd, dtype), dtype, w)
    B.cb_sync(None)
    assert torch.all(out[0, pad] == 0)
    check_attention(out, host(w), K8.attention(o, q.astype(np.float64), last), last, dtype, hd)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,hkv,hd,n_q", WAYS)
def test_a_nan_query_leaves_rows_it_does_not_see_alone_when_the_keys_are_split(B, H, hkv, hd, n_q, dtype):
    """One query with a NaN sees the first 91 rows, all others the first 700 at least: several whole
    key tiles lie in between."""
    torch = torch_mod()
    g = np.random.default_rng(n_q + 1)
    cap = 1152
    d, o = filled(B, g, 1, hkv, cap, hd, 32, [cap])
    q = rounded(g.standard_normal((1, n_q, H, hd)), dtype)
    last = g.integers(700, cap, (1, n_q))
    last[0, 1] = 90
    bad = q.copy()
    bad[0, 1, H - 1, 17] = np.nan                   # a head of the last KV head
    w = torch.zeros(1, hkv, cap, device="cuda")
    out = attend(B, d, bad, last, make_dims(B, H, hkv, hd, dtype), dtype, w)
    B.cb_sync(None)
    assert torch.all(torch.isnan(out[0, 1, H - 1])) and torch.all(torch.isnan(w[0, hkv - 1, :91]))
    out[0, 1, H - 1] = 0
    w[0, hkv - 1, :91] = 0
    q[0, 1, H - 1] = 0
    ref = list(K8.attention(o, q.astype(np.float64), last))
    ref[0][0, 1, H - 1] = 0
    ref[1][0, hkv - 1, :91] = 0
    check_attention(out, host(w), ref, last, dtype, hd)


@pytest.mark.parametrize("what", [np.inf, -np.inf])
@pytest.mark.parametrize("cap", [160, 1152])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,hkv,hd,n_q", WAYS)
def test_an_infinite_query_spoils_only_its_own_rows(B, H, hkv, hd, n_q, dtype, cap, what):
    torch = torch_mod()
    g = np.random.default_rng(n_q + 2)
    d, o = filled(B, g, 1, hkv, cap, hd, 32, [cap])
    q = rounded(g.standard_normal((1, n_q, H, hd)), dtype)
    last = g.integers(cap * 2 // 3, cap, (1, n_q))
    last[0, 1] = 50
    bad = q.copy()
    bad[0, 1, H - 1, 5] = what
    w = torch.zeros(1, hkv, cap, device="cuda")
    out = attend(B, d, bad, last, make_dims(B, H, hkv, hd, dtype), dtype, w)
    B.cb_sync(None)
    out[0, 1, H - 1] = 0
    w[0, hkv - 1, :51] = 0
    q[0, 1, H - 1] = 0
    ref = list(K8.attention(o, q.astype(np.float64), last))
    ref[0][0, 1, H - 1] = 0
    ref[1][0, hkv - 1, :51] = 0
    check_attention(out, host(w), ref, last, dtype, hd)


# ------------------------------------------------------------------ scores next to zero
@pytest.mark.parametrize("weigh", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [2.0 ** -121, 2.0 ** -126, 2.0 ** -133])
@pytest.mark.parametrize("hd,n_q", [(32, 1), (64, 1), (128, 3), (256, 1), (256, 3), (256, 12), (64, 20), (128, 60), (64, 140)])
def test_tiny_queries_over_keys_of_zero(B, hd, n_q, size, dtype, weigh):
    """The score's factor (query's magnitude times the smallest scale) lies below fp32's range; keys
    past `last` share groups of 16 with visible ones.  Every visible row weighs the same."""
    torch = torch_mod()
    g = np.random.default_rng(hd + n_q)
    hkv, cap, dims = 2, 48, make_dims(B, 2, 2, hd, dtype)
    d, o = Dev(B, 1, hkv, cap, hd, 16), K8.empty(1, hkv, cap, hd, 16)
    k, v = np.zeros((1, cap, hkv, hd), np.float32), g.standard_normal((1, cap, hkv, hd)).astype(np.float32)
    B.cb_kv8_append(dev(k), dev(v), cap, dev_i32([0]), None, d.c, make_dims(B, 2, 2, hd, "f32"))
    K8.append(o, k, v, [0])
    q = rounded(g.uniform(-1, 1, (1, n_q, 2, hd)) * size, dtype)
    last = g.integers(0, cap, (1, n_q))
    last[0, 0] = 20
    w = torch.zeros(1, hkv, cap, device="cuda") if weigh else None
    out = attend(B, d, q, last, dims, dtype, w)
    B.cb_sync(None)
    check_attention(out, host(w) if weigh else None, K8.attention(o, q.astype(np.float64), last), last, dtype, hd)


# ------------------------------------------------------------------ sizes
@pytest.mark.parametrize("weigh", [False, True])
def test_many_queries_over_many_rows(B, weigh):
    """The few-row kernels count ceil(n_q G / 8) n_seq Hkv capacity / 16 in 32 bits; this call's 2^31
    are no business of the tensor-core kernels."""
    torch = torch_mod()
    g = np.random.default_rng(0)
    H, hkv, hd, n_q, cap, held = 8, 1, 64, 65536, 1 << 19, 96
    c = [torch.zeros(1, hkv, cap, hd, dtype=torch.int8, device="cuda") for _ in range(2)]
    sc = [torch.full((1, hkv, cap // 128), float("nan"), device="cuda") for _ in range(2)]
    cache = B.kv8_cache(*c, *sc, 128)
    o = K8.empty(1, hkv, 128, hd, 128)
    k, v = (rounded(g.standard_normal((1, held, hkv, hd)), "bf16") for _ in range(2))
    dims = make_dims(B, H, hkv, hd, "bf16")
    B.cb_kv8_append(dev(k, "bf16"), dev(v, "bf16"), held, dev_i32([0]), None, cache, dims)
    K8.append(o, k, v, [0])
    q = torch.randn(1, n_q, H, hd, device="cuda").to(torch.bfloat16)
    last = torch.full((1, n_q), -1, dtype=torch.int32, device="cuda")
    rows = np.array([0, 1, 30000, n_q - 2, n_q - 1])
    at = np.array([0, 50, 95, 31, 95])
    last[0, torch.from_numpy(rows).cuda()] = dev_i32(at)
    out = torch.full_like(q, 7.5)
    w = torch.zeros(1, hkv, cap, device="cuda") if weigh else None
    ws = torch.empty(B.cb_kv8_workspace_bytes(dims, 1, cap, n_q, weigh), dtype=torch.uint8, device="cuda")
    B.cb_kv8_attention(q, last, n_q, cache, dims, out, w, ws)
    B.cb_sync(None)
    ref = K8.attention(o, host(q[:, rows]), at[None])
    check_attention(out[:, rows], None, ref, at[None], "bf16", hd)
    rest = torch.ones(n_q, dtype=torch.bool, device="cuda")
    rest[torch.from_numpy(rows).cuda()] = False
    assert torch.all(out[0, rest] == 0)
    if weigh:
        assert torch.all(w[..., held:] == 0)
        # as in check_attention: exp's argument and ex2 twice, sums over 96 keys and 40 rows
        r = 2 * (ref[3].max() * (hd + 4) * 2.0 ** -24 + 2.0 ** -21) + (held + 5 * H + 8) * 2.0 ** -24
        assert np.all(np.abs(host(w[..., :held]) - ref[1][..., :held]) <= ref[1][..., :held] * r + 1e-30)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_workspace_for_calls_of_different_sizes(B, dtype):
    """Fewer queries may ask for more: a buffer for several n_q is the largest of what each asks for."""
    torch = torch_mod()
    g = np.random.default_rng(1)
    H, hkv, hd, cap = 8, 4, 128, 528
    dims = make_dims(B, H, hkv, hd, dtype)
    d, o = filled(B, g, 1, hkv, cap, hd, 16, [cap])
    counts = [64, 1, 24, 4, 12, 65, 8, 30]
    ask = [B.cb_kv8_workspace_bytes(dims, 1, cap, n, w) for n in counts for w in (False, True)]
    ws = torch.full((max(ask),), 255, dtype=torch.uint8, device="cuda")
    if dtype == "bf16":
        assert B.cb_kv8_workspace_bytes(dims, 1, cap, 64) == 0 < B.cb_kv8_workspace_bytes(dims, 1, cap, 1)
    for n in counts:
        for weigh in (False, True):
            q = rounded(g.standard_normal((1, n, H, hd)), dtype)
            last = g.integers(-1, cap, (1, n))
            qd = dev(q, dtype)
            out = torch.full_like(qd, 7.5)
            w = torch.zeros(1, hkv, cap, device="cuda") if weigh else None
            B.cb_kv8_attention(qd, dev_i32(last), n, d.c, dims, out, w, ws)
            B.cb_sync(None)
            check_attention(out, host(w) if weigh else None, K8.attention(o, q.astype(np.float64), last), last, dtype, hd)


class Long:
    """A cache of 3 sequences x 2 heads x 2^22 rows x 128: the last sequence starts 2^31 bytes into the
    codes.  Its keys are 0 but for a few marked rows near both ends and in the middle, each with a
    channel of its own; its values are distinct there, and elsewhere 50 (first half) or 110 in units
    of 0.01.  A query points at a marked row (its score is 60, the others' 0: they weigh e^-60) or at
    none (every visible row weighs the same)."""
    HKV, HD, CAP, NSEQ, BLOCK = 2, 128, 1 << 22, 3, 128
    MARKED = [0, 5, 127, 128, (1 << 21) + 77, (1 << 22) - 4097, (1 << 22) - 130, (1 << 22) - 2, (1 << 22) - 1]

    def __init__(self, B):
        torch = torch_mod()
        n, h, c, d = self.NSEQ, self.HKV, self.CAP, self.HD
        mk = lambda: torch.empty(n, h, c, d, dtype=torch.int8, device="cuda")  # noqa: E731
        sc = lambda: torch.full((n, h, c // self.BLOCK), float("nan"), device="cuda")  # noqa: E731
        self.k, self.v, self.ks, self.vs = mk(), mk(), sc(), sc()
        self.cache = B.kv8_cache(self.k, self.v, self.ks, self.vs, self.BLOCK)
        self.k[2] = 0
        self.v[2, :, :c // 2] = 50
        self.v[2, :, c // 2:] = 110
        self.ks[2] = 1.0 / 128
        self.vs[2] = 0.01
        self.row = np.random.default_rng(6).integers(-127, 128, (h, len(self.MARKED), d))
        for i, r in enumerate(self.MARKED):
            self.k[2, :, r, 3 * i] = 64                 # 0.5
            self.v[2, :, r] = torch.from_numpy(self.row[:, i].astype(np.int8)).cuda()

    def query(self, i):
        """The query that points at marked row i; None: at none."""
        q = np.zeros(self.HD, np.float32)
        if i is not None:
            q[3 * i] = 2 * 60 * np.sqrt(np.float64(self.HD))
        return q


@pytest.fixture(scope="module")
def long_cache(B):
    x = Long(B)
    yield x


@pytest.mark.parametrize("dtype,n_q", [("bf16", 1), ("f32", 1), ("bf16", 12), ("bf16", 40), ("bf16", 150), ("f32", 60)])
def test_attention_and_weights_over_a_long_cache(B, long_cache, dtype, n_q):
    """Every path past 2^31 bytes of codes: rows near the end told apart by their values, the account
    of each of the 2^22 rows."""
    torch = torch_mod()
    L = long_cache
    h, cap, hd, marks = L.HKV, L.CAP, L.HD, L.MARKED
    dims = make_dims(B, h, h, hd, dtype)
    # per query and head: the marked row it points at; the last row it sees
    point = [[(j + 4 * hh) % (len(marks) + 1) for hh in range(h)] for j in range(n_q)]
    point = [[None if p == len(marks) else p for p in r] for r in point]
    if n_q == 1:
        point = [[len(marks) - 2, None]]
    last = np.full((L.NSEQ, n_q), -1)
    last[2] = cap - 1
    if n_q > 1:
        last[2, 1] = marks[7]              # the last row of all is not seen
        last[2, 2] = cap // 2 - 1          # only values of 50 and marked ones
    q = np.zeros((L.NSEQ, n_q, h, hd), np.float32)
    for j in range(n_q):
        for hh in range(h):
            q[2, j, hh] = L.query(point[j][hh])
    q = rounded(q, dtype)
    w = torch.zeros(L.NSEQ, h, cap, device="cuda")
    qd = dev(q, dtype)
    out = torch.full_like(qd, 7.5)
    ws = torch.empty(B.cb_kv8_workspace_bytes(dims, L.NSEQ, cap, n_q, True), dtype=torch.uint8, device="cuda")
    B.cb_kv8_attention(qd, dev_i32(last), n_q, L.cache, dims, out, w, ws)
    B.cb_sync(None)
    assert torch.all(out[:2] == 0) and torch.all(w[:2] == 0)
    got, acc = host(out[2]), host(w[2])
    eps = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    want = np.zeros((h, cap))
    for hh in range(h):
        v = np.where(np.arange(cap) < cap // 2, 50.0, 110.0)
        for j in range(n_q):
            n, p = last[2, j] + 1, point[j][hh]
            if p is not None and marks[p] < n:
                # one row has all the weight but 2^22 e^-60; its own is rounded once on both sides of
                # the fraction line (fp16: 2^-11, fp32: 2^-21)
                ref = L.row[hh, p] * np.float64(np.float32(0.01))
                tol = np.abs(ref) * (eps * 1.01 + (2.0 ** -11 if dtype == "bf16" else 2.0 ** -21) * 2) + 1e-12
                assert np.all(np.abs(got[j, hh] - ref) <= tol), (j, hh)
                want[hh, marks[p]] += 1
            else:
                # n equal weights, added 16 keys at a time: at most n / 16 sums, each cut to 24 bits
                seen = [m for m in marks if m < n]
                tot = v[:n].sum() - v[seen].sum() + L.row[hh, :len(seen)].sum(0)
                ref = tot / n * np.float64(np.float32(0.01))
                bound = (n / 16) * 2.0 ** -23 + 2.0 ** -10
                assert np.all(np.abs(got[j, hh] - ref) <= np.abs(ref) * (bound + eps)), (j, hh)
                want[hh, :n] += 1.0 / n
    bound = cap / 16 * 2.0 ** -23 + 2.0 ** -18 + n_q * 2.0 ** -23
    assert np.all(np.abs(acc - want) <= want * bound + n_q * np.exp(-59.0))


# ------------------------------------------------------------------ logits
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,V,T,nb", [(3, 5000, 4000, 0), (2, 32000, 9000, 600), (4, 1027, 3000, 64)])
def test_every_step_of_the_logit_rules_is_rounded_to_fp32(B, n, V, T, nb, dtype):
    """The rules one after the other, each operation rounded: the same bits as numpy's fp32."""
    torch = torch_mod()
    g = np.random.default_rng(V)
    f = np.float32
    x = rounded(g.standard_normal((n, V)) * 3, dtype)
    hist = (g.uniform(0, 1, (n, T)) ** 2 * V).astype(np.int32).clip(0, V - 1)
    pl = g.integers(0, T // 2, n)
    rep, pres, freq = (g.uniform(a, b, n).astype(f) for a, b in ((0.5, 2), (-1, 1), (0, 0.5)))
    bid = g.integers(0, V, (n, nb)).astype(np.int32)
    if nb:
        bid[:, nb // 2:] = bid[:, :nb - nb // 2]           # each id twice at least
    bias = g.standard_normal((n, nb)).astype(f)
    rules = dict(history=dev_i32(hist), history_len=dev_i32([T] * n), prompt_len=dev_i32(pl), repetition=dev(rep),
                 presence=dev(pres), frequency=dev(freq))
    if nb:
        rules.update(bias_id=dev_i32(bid), bias=dev(bias))
    y, tok = run_logits(B, x, dtype, **rules)
    B.cb_sync(None)
    for b in range(n):
        v = x[b].astype(f)
        seen = np.bincount(hist[b], minlength=V) > 0
        v = np.where(seen, np.where(v > 0, v / rep[b], v * rep[b]), v).astype(f)
        made = np.bincount(hist[b, pl[b]:], minlength=V)
        take = (freq[b] * made.astype(f)).astype(f) + pres[b]
        v = np.where(made > 0, v - take.astype(f), v).astype(f)
        total = {}
        for i, z in zip(bid[b], bias[b]):
            total[i] = f(total[i] + z) if i in total else z
        for i, z in total.items():
            v[i] = f(v[i] + z)
        ref = rounded(v, dtype)
        np.testing.assert_array_equal(y[b].float().cpu().numpy(), ref)
        assert int(tok[b]) == K8.token(ref.astype(np.float64))


# ------------------------------------------------------------------ from a blend to its answer
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_blends_rows_become_the_cache_that_answers(B, dtype):
    """run_blend's K and V of every layer appended as they are; the next tokens attend over them."""
    from non_prefix_kv_gb300 import engine as E, synth
    torch = torch_mod()
    s = synth.ModelShape(n_layers=2, d_model=256, n_heads=4, n_kv_heads=2, head_dim=64, d_ff=512, vocab=512, dtype=dtype,
                         w_std=0.06)
    g = np.random.default_rng(50)
    pool = [g.integers(0, s.vocab, 96).astype(np.int32) for _ in range(3)]
    tokens = np.concatenate(pool + [g.integers(0, s.vocab, 30).astype(np.int32)])
    n, hkv, hd, H, cap = len(tokens), s.n_kv_heads, s.head_dim, s.n_heads, 384
    dm = E.DeviceModel.from_host(synth.make_model(s, seed=4))
    eng = E.BlendEngine(dm, n, max_pos=512)
    req = E.Request(eng, eng.precompute_pool(pool), [0, 1, 2], tokens)
    E.run_blend(req, E.layer_plan(s, req.N, req.n_cached, [1.0, 0.3]))
    caches = [Dev(B, 1, hkv, cap, hd, 32) for _ in range(s.n_layers)]
    twins = [K8.empty(1, hkv, cap, hd, 32) for _ in range(s.n_layers)]
    for l in range(s.n_layers):
        B.cb_kv8_append(req.K[l], req.V[l], n, dev_i32([0]), None, caches[l].c, dm.dims)
    B.cb_sync(None)
    rows = lambda t: host(t).reshape(1, -1, hkv, hd).astype(np.float32)  # noqa: E731
    for l in range(s.n_layers):
        K8.append(twins[l], rows(req.K[l]), rows(req.V[l]), [0])
        check_cache(caches[l], twins[l], [n])
    x, q, k, v, o = (torch.empty(1, w, dtype=tdt(dtype), device="cuda")
                     for w in (s.d_model, s.q_width, s.kv_width, s.kv_width, s.q_width))
    ws = torch.empty(B.cb_kv8_workspace_bytes(dm.dims, 1, cap, 1, True), dtype=torch.uint8, device="cuda")
    acc = [torch.zeros(1, hkv, cap, device="cuda") for _ in range(s.n_layers)]
    total, rel = [np.zeros((1, hkv, cap)) for _ in range(s.n_layers)], 0.0
    tok, logits = req.token, torch.empty(1, s.vocab, device="cuda")
    hist, rules = list(tokens), None
    for step in range(5):
        at = n + step
        hist.append(int(tok))
        B.cb_gather_rows(x, dm.embed, tok, 1, s.d_model * x.element_size())
        for l in range(s.n_layers):
            B.cb_selective_qkv(x, None, dev_i32([at]), 1, dm.dims, dm.layers_c[l], eng.cos_sin, eng.max_pos, q, k, v, eng.ws)
            B.cb_kv8_append(k, v, 1, dev_i32([at]), None, caches[l].c, dm.dims)
            B.cb_kv8_attention(q, dev_i32([at]), 1, caches[l].c, dm.dims, o, acc[l], ws)
            B.cb_sync(None)
            K8.append(twins[l], rows(k), rows(v), [at])
            check_cache(caches[l], twins[l], [at + 1])
            ref = K8.attention(twins[l], host(q).reshape(1, 1, H, hd), np.array([[at]]))
            check_attention(o.view(1, 1, H, hd), None, ref, np.array([[at]]), dtype, hd)
            total[l] += ref[1]
            # of a weight, as in check_attention; one rounding of each of the account's five sums
            rel = max(rel, 2 * (ref[3].max() * ((hd + 4) * 2.0 ** -24 + (2.0 ** -21 if dtype == "f32" else 0)) + 2.0 ** -21)
                      + (at + 1 + H + 8 + 5) * 2.0 ** -24)
            B.cb_o_proj_ffn(o, x, 1, dm.dims, dm.layers_c[l], x, eng.ws)
        B.cb_lmhead_argmax(x[0], dm.final_norm, dm.w_lm, dm.dims, logits, tok, eng.ws)
        rules = B.logit_rules(history=dev_i32([hist]), history_len=dev_i32([len(hist)]), prompt_len=dev_i32([n]),
                              repetition=dev(np.array([1.2], np.float32)))
        B.cb_logits_process(logits, rules, logits, tok)
        B.cb_sync(None)
        assert int(tok) == K8.token(host(logits)[0])
    for l in range(s.n_layers):
        assert np.all(np.abs(host(acc[l]) - total[l]) <= total[l] * rel + 1e-30)


# ------------------------------------------------------------------ cb_sync
SYNC = """
import sys
import torch
from torch.profiler import ProfilerActivity, profile
from non_prefix_kv_gb300 import binding as B

def copies():
    B.cb_sync(None)
    with profile(activities=[ProfilerActivity.CUDA]) as p:
        B.cb_sync(None)
        torch.cuda.synchronize()
    names = [e.name for e in p.events() if e.name.startswith("Memcpy")]
    return sum("DtoH" in n for n in names), sum("HtoD" in n for n in names)

x = torch.zeros(1, 64, device="cuda")
torch.cuda.synchronize()
copies()          # (the profiler's first session may miss its copies)
print(*copies())
t = torch.zeros(1, dtype=torch.int32, device="cuda")
B.cb_logits_process(x, B.logit_rules(), None, t)
print(*copies())
"""


def test_sync_asks_only_for_what_was_launched(B):
    """cb_sync's blocking copies in a process of its own: none for operators that nobody called, and
    none to clear a word that holds nothing."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", SYNC], capture_output=True, text=True, cwd=root, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
    first, later = (tuple(map(int, line.split())) for line in r.stdout.strip().splitlines()[-2:])
    if first == later == (0, 0):
        pytest.skip("the profiler records no copies here")
    assert (first, later) == ((5, 0), (6, 0))


# ------------------------------------------------------------------ calls at once
@pytest.mark.parametrize("hd,n_q", [(64, 30), (64, 150), (128, 30)])
def test_two_streams_at_once(B, hd, n_q):
    """Attention with the keys split over clusters, and its weights, on two streams at once (a cache
    and a workspace each): the same bits as one after the other."""
    torch = torch_mod()
    g = np.random.default_rng(hd)
    hkv, cap, dims = 2, 2064, make_dims(B, 2, 2, hd, "bf16")
    n = B.cb_kv8_workspace_bytes(dims, 1, cap, n_q, True)
    sets = []
    for _ in range(2):
        d, _ = filled(B, g, 1, hkv, cap, hd, 16, [cap])
        q = dev(rounded(g.standard_normal((1, n_q, 2, hd)), "bf16"), "bf16")
        last = dev_i32(g.integers(0, cap, (1, n_q)))
        sets.append((d, q, last, torch.empty_like(q), torch.zeros(1, hkv, cap, device="cuda"),
                     torch.empty(n, dtype=torch.uint8, device="cuda")))
    call = lambda s: B.cb_kv8_attention(s[1], s[2], n_q, s[0].c, dims, s[3], s[4], s[5])  # noqa: E731
    ref = []
    for s in sets:
        for _ in range(20):
            call(s)
        B.cb_sync(None)
        ref.append((s[3].clone(), s[4].clone()))
        s[3].zero_(), s[4].zero_()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, s in zip(streams, sets):
            with torch.cuda.stream(st):
                call(s)
    for st in streams:
        B.cb_sync(st)
    for s, (o, w) in zip(sets, ref):
        assert torch.equal(s[3], o) and torch.equal(s[4], w)
