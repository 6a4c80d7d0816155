"""Drawing tokens from given numbers, against the fp64 oracle: tokens and counts exactly (unless the oracle
says that a decision is nearer than 2^-28 of the weight, where the weights' own rounding may decide: no input
here is), logprobs within their fp32 rounding and 2^-28 (the token's weight and the sum)."""
import numpy as np
import pytest

import oracle.answers_oracle as A
from tests.gpu_util import dev_i32, ensure_lib, torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    torch_mod()
    ensure_lib()
    from non_prefix_kv_gb300 import binding
    return binding


def f32(a):
    return torch_mod().from_numpy(np.ascontiguousarray(a, np.float32)).cuda()


def draw(B, x, u, T=None, k=None, p=None, m=None, dtype="f32"):
    torch = torch_mod()
    n = len(x)
    logits = f32(x) if dtype == "f32" else f32(x).bfloat16()
    r = B.sample_rules(temperature=None if T is None else f32(T), top_k=None if k is None else dev_i32(k),
                       top_p=None if p is None else f32(p), min_p=None if m is None else f32(m))
    tok, kept = (torch.full((n,), -7, dtype=torch.int32, device="cuda") for _ in range(2))
    lp = torch.full((n,), 7.0, device="cuda")
    B.cb_sample_token(logits, f32(u), r, tok, lp, kept)
    return logits, tok, lp, kept


def check(B, x, u, T=None, k=None, p=None, m=None, dtype="f32", least=2.0 ** -28):
    logits, tok, lp, kept = draw(B, x, u, T, k, p, m, dtype)
    B.cb_sync(None)
    logits, tok, lp, kept = (t.double().cpu().numpy() for t in (logits, tok, lp, kept))
    one = lambda a, b, d: d if a is None else float(np.float32(a[b]))  # noqa: E731
    for b in range(len(x)):
        w_tok, w_lp, w_kept, near = A.sample(logits[b], float(np.float32(u[b])), one(T, b, 1.0), 0 if k is None else int(k[b]),
                                             one(p, b, 1.0), one(m, b, 0.0))
        assert near > least, "an input too close to a border"
        assert tok[b] == w_tok and kept[b] == w_kept, (b, tok[b], w_tok, kept[b], w_kept)
        if w_tok >= 0:
            assert abs(lp[b] - w_lp) <= 2.0 ** -24 * abs(w_lp) + 2.0 ** -28
        else:
            assert lp[b] == -np.inf
    return tok


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 7, 255, 257, 1000, 4099, 32000])
def test_every_rule_and_size(B, dtype, V):
    g = np.random.default_rng(V)
    n = 24
    x = g.standard_normal((n, V)) * 2.5
    x[::3] += g.random((len(x[::3]), V)) ** 50 * 10
    if V > 2:
        x[1::4, : V // 2] = -np.inf
    u = g.random(n)
    T = np.array([0.7, 1.0, 1.4, 0.0])[np.arange(n) % 4]
    k = np.array([0, 1, 5, 50, 100000])[np.arange(n) % 5]
    p = np.array([1.0, 0.9, 0.5, 0.0, 0.97, 0.2, 1.5])[np.arange(n) % 7]
    m = np.array([0.0, 0.0, 0.05, 0.3])[(np.arange(n) // 2) % 4]
    check(B, x, u, T, k, p, m, dtype)
    check(B, x, u, dtype=dtype)
    check(B, x, u, k=k, dtype=dtype)
    check(B, x, u, p=p, dtype=dtype)
    check(B, x, u, T=T, m=m, dtype=dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_equal_logits_go_by_id(B, dtype):
    """Rows of a few values only: the border falls inside a run of equals."""
    g = np.random.default_rng(3)
    V, n = 3001, 16
    x = g.integers(-3, 4, (n, V)).astype(float)
    u = g.random(n)
    k = g.integers(1, 900, n)
    check(B, x, u, k=k, dtype=dtype)
    check(B, x, u, p=g.uniform(0.05, 0.95, n), dtype=dtype)
    check(B, x, u, T=np.full(n, 0.9), k=k, p=g.uniform(0.05, 0.95, n), m=np.full(n, 0.01), dtype=dtype)
    same = np.zeros((n, V))
    tok = check(B, same, u, k=k, dtype=dtype)
    assert np.all(tok < k)
    # halves and quarters: borders met exactly, on both sides the same
    x = np.full((4, 8), -np.inf)
    x[:, 2:6] = 1.25
    for p, kept in ((0.25, 1), (0.5, 2), (0.75, 3), (0.5000001, 3)):
        _, tok, _, got = draw(B, x, [0.0, 0.49, 0.5, 0.99], p=[p] * 4, dtype=dtype)
        assert got.tolist() == [kept] * 4 and tok.tolist()[0] == 2


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_vocabularies_and_many_rows(B, dtype):
    """131072, 150001 and 2^20 ids, and more rows than clusters at once; the same row gives the same answer
    wherever it stands."""
    g = np.random.default_rng(4)
    for n, V in ((3, 131072), (2, 150001), (2, 1 << 20)):
        x = (g.standard_normal((n, V)) * 2).astype(np.float32)
        check(B, x, g.random(n), T=np.full(n, 0.9), k=np.array([0, 900, 0])[:n], p=np.array([0.9, 0.9, 1.0])[:n], dtype=dtype)
    x = np.repeat(g.standard_normal((1, 5003)) * 2, 700, 0)
    u = np.full(700, 0.37)
    a = draw(B, x, u, p=np.full(700, 0.9), dtype=dtype)
    b = draw(B, x[:1], u[:1], p=[0.9], dtype=dtype)
    for s, t in zip(a[1:], b[1:]):
        assert bool((s == t).all())
    B.cb_sync(None)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_flat_rows(B, dtype):
    """All ids equal: one class holds the whole row, of up to 2^17 ids in a block.  Every weight is that
    of the largest, exactly 1 (2^42 of the kernel's units), so that a decision has no error but u's and p's own
    products': below 2^-44."""
    u = [0.0, 0.123456789, 0.87654321, 0.99999994]
    for V in (70000, 131072, 300001, 1 << 20):
        x = np.full((4, V), 1.5)
        for p in (0.3100001, 0.7700003):
            check(B, x, u, p=np.full(4, p), dtype=dtype, least=2.0 ** -44)
        check(B, x, u, k=np.full(4, V // 3), p=np.full(4, 0.56789), dtype=dtype, least=2.0 ** -44)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_lists_of_uneven_values(B, dtype):
    """Ids that no classes of one width tell apart: one far above the others, infinities, most of them equal."""
    g = np.random.default_rng(6)
    n, V = 6, 3000
    x = g.random((n, V))
    x[:, 1234] = 1e6
    x[1, 77] = 2e6
    x[2:4, :1500] = 0.75
    u = g.random(n)
    T = np.full(n, 1e6)
    for k in (1, 300, 900, 1024):
        check(B, x, u, T=T, k=np.full(n, k), dtype=dtype)
        check(B, x, u, T=T, k=np.full(n, k), p=np.linspace(0.2, 0.9, n), dtype=dtype)
    check(B, x[:, :2000], u, T=T, m=np.full(n, 0.3), p=np.linspace(0.2, 0.9, n), dtype=dtype)
    x[0, [5, 9, 2000]] = np.inf
    x[1, 0] = np.inf
    _, tok, lp, kept = draw(B, x[:2], [0.7, 0.2], k=[700, 700], p=[0.9, 0.9], dtype=dtype)
    B.cb_sync(None)
    assert tok.tolist() == [2000, 0] and kept.tolist() == [3, 1]


def test_temperatures_of_no_weight(B):
    """Below the smallest normal number a temperature counts as 0: the first of the largest."""
    x = np.zeros((3, 700))
    x[:, [300, 301]] = 1.0
    for T in (0.0, 1e-45, 1.1e-38):
        for kw in (dict(), dict(k=[5] * 3), dict(p=[0.9] * 3), dict(m=[0.1] * 3)):
            _, tok, lp, kept = draw(B, x, [0.0, 0.6, 0.99], T=[T] * 3, **kw)
            assert tok.tolist() == [300] * 3 and kept.tolist() == [1] * 3 and lp.tolist() == [0.0] * 3
    B.cb_sync(None)
    check(B, x, [0.1, 0.6, 0.9], T=[1.2e-38, 1e-30, 1e30])


def test_extremes(B):
    V = 600
    base = np.linspace(-5, 5, V)
    inf = np.inf
    x = np.stack([base] * 8)
    x[0] = -inf                                 # nothing
    x[1] = -inf
    x[1, 77] = -3e38                            # one id
    x[2, 5] = x[2, 400] = inf                   # infinite ones share the weight
    x[3] = 3.0e38 * np.sign(base)               # differences past fp32's range
    x[4] *= 1e-30                               # all but equal
    x[5] = -1e30 * np.arange(V)                 # only the first counts
    x[6, :] = np.float32(-3.4028235e38)         # the type's lowest value everywhere
    T = [1, 1, 1, 1, 1, 1, 1, 1e-30]
    _, tok, lp, kept = draw(B, x, [0.6] * 8, T=T, p=[0.9875] * 8)
    B.cb_sync(None)
    tok, lp, kept = tok.tolist(), lp.tolist(), kept.tolist()
    assert tok[0] == -1 and lp[0] == -inf and kept[0] == 0
    assert tok[1] == 77 and lp[1] == 0 and kept[1] == 1
    assert tok[2] == 400 and kept[2] == 2 and abs(lp[2] + np.log(2)) < 1e-6
    assert tok[3] == 300 + int(0.6 * 297) and kept[3] == 297     # 300 equal ones, 296.25 hold the share
    assert tok[4] in range(V // 2, V) and kept[4] == 593
    assert tok[5] == 0 and kept[5] == 1
    assert tok[6] == int(0.6 * 593) and kept[6] == 593
    assert tok[7] == V - 1 and kept[7] == 1


def test_what_is_reported(B):
    g = np.random.default_rng(6)
    V, n = 900, 8
    x = g.standard_normal((n, V))
    ok = dict(u=np.full(n, 0.3), T=np.ones(n), p=np.full(n, 0.9), m=np.full(n, 0.01))

    def status(x=x, **kw):
        a = {**ok, **kw}
        out = draw(B, x, a["u"], T=a["T"], p=a["p"], m=a["m"])[1:]
        try:
            B.cb_sync(None)
        except B.CBError as e:
            return e.status, out
        return 0, out

    st, ref = status()
    assert st == 0
    for key, bad, same in (("T", np.nan, 1.0), ("T", -1.0, 1.0), ("T", np.inf, 1.0), ("p", np.nan, 1.0), ("m", np.nan, 0.0),
                           ("u", np.nan, 0.0), ("u", -0.5, 0.0), ("u", 1.0, 0.99999994), ("u", 7.0, 0.99999994)):
        a, b = ok[key].copy(), ok[key].copy()
        a[3], b[3] = bad, same
        st, got = status(**{key: a})
        st2, want = status(**{key: b})
        assert st == 5 and st2 == 0, key
        assert all(bool((s == t).all()) for s, t in zip(got, want)), key
    y = x.copy()
    y[2, 10] = np.nan
    z = x.copy()
    z[2, 10] = -np.inf
    st, got = status(y)
    assert st == 5 and all(bool((s == t).all()) for s, t in zip(got, status(z)[1]))


def test_shares_of_many_draws(B):
    """u over a fine grid: each kept id is drawn as often as its share says, to within one step."""
    torch = torch_mod()
    g = np.random.default_rng(7)
    V, n = 50, 8192
    x = g.standard_normal(V) * 2
    tok = draw(B, np.repeat(x[None], n, 0), (np.arange(n) + 0.5) / n, k=[20] * n)[1]
    B.cb_sync(None)
    order = np.argsort(-x)[:20]
    w = np.exp(x[order].astype(np.float32).astype(float))
    for i, share in zip(order, w / w.sum()):
        assert abs(int((tok == int(i)).sum()) - n * share) <= 1.0
    assert bool((tok >= 0).all()) and torch.unique(tok).numel() <= 20


def test_captured_after_the_logit_rules(B):
    """Rules on the logits, then the draw from what they leave, in a graph that is replayed with new inputs."""
    torch = torch_mod()
    n, V = 5, 3210
    g = torch.Generator(device="cuda").manual_seed(1)
    logits, out = torch.empty(n, V, device="cuda"), torch.empty(n, V, device="cuda")
    hist = torch.zeros(n, 40, dtype=torch.int32, device="cuda")
    rules = B.logit_rules(history=hist, history_len=dev_i32([40] * n), repetition=torch.full((n,), 1.3, device="cuda"),
                          mask=torch.randint(-2 ** 31, 2 ** 31, (n, (V + 31) // 32), generator=g, device="cuda").int())
    s = B.sample_rules(temperature=torch.full((n,), 0.8, device="cuda"), top_p=torch.full((n,), 0.9, device="cuda"))
    u, tok, lp, kept = (torch.zeros(n, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(n, device="cuda"),
                        torch.zeros(n, dtype=torch.int32, device="cuda"))

    def step():
        B.cb_logits_process(logits, rules, out)
        B.cb_sample_token(out, u, s, tok, lp, kept)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        logits.copy_(torch.randn(n, V, generator=g, device="cuda") * 2)
        u.copy_(torch.rand(n, generator=g, device="cuda"))
        hist.copy_(torch.randint(0, V, (n, 40), generator=g, device="cuda"))
        graph.replay()
        B.cb_sync(None)
        for b in range(n):
            w = A.sample(out[b].double().cpu().numpy(), float(u[b]), float(np.float32(0.8)), 0, float(np.float32(0.9)))
            assert (int(tok[b]), int(kept[b])) == (w[0], w[2]) and w[3] > 2.0 ** -28


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [5000, 40000])
def test_a_least_share_that_many_or_few_reach(B, dtype, V):
    """With a share of the weight beside it, from a handful of ids to all of them, by way of about as many as a list takes.
    (Of more ids than these some weight is always too near the least share for the oracle.)"""
    g = np.random.default_rng(V)
    n = 8
    x = g.standard_normal((n, V)) * np.array([0.02, 0.2, 0.5, 0.8, 1.1, 1.4, 2.0, 3.0])[:, None]
    x[::3, ::2] = -np.inf
    u = g.random(n)
    for m in (0.3, 0.05, 0.005):
        check(B, x, u, p=np.full(n, 0.93), m=np.full(n, m), dtype=dtype)
        check(B, x, u, T=np.linspace(0.6, 1.4, n), p=np.linspace(0.3, 0.99, n), m=np.full(n, m), dtype=dtype)
