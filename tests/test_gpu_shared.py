"""Attention over a shared prefix and each sequence's own rows, against the fp64 oracle.

Tolerances, element by element, with A = sum_i p_i |v_i| and S = max_i sum_c |q_c k_ic| / sqrt(hd):
  a score's hd products and sums are fp32, and so are its scaling and the distance from the maximum, at most
  (hd + 8) 2^-24 S in all; the exponential turns that into a relative error of the weight, adds 2^-20 of its
  own, and it counts above and below the fraction line; sums over n keys and pieces add (n + 16) 2^-24;
  bf16: a weight's rounding is 2^-8 of it where the tensor cores take it, the output's 2^-8; fp32: 2^-24."""
import numpy as np
import pytest

import oracle.answers_oracle as A
from tests.gpu_util import dev_i32, ensure_lib, host, tdt, torch_mod

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24


@pytest.fixture(scope="module")
def B():
    torch_mod()
    ensure_lib()
    from non_prefix_kv_gb300 import binding
    return binding


def dims_of(B, H, hkv, hd, dtype):
    return B.cb_dims(H * hd, H, hkv, hd, 256, 64, 1e4, 1e-5, B.CB_BF16 if dtype == "bf16" else B.CB_F32)


class Case:
    """Random inputs whose unused memory holds NaN: gaps between the prefixes, own rows past the last one seen,
    queries that see nothing."""

    def __init__(self, B, seed, dtype, H, hkv, hd, lens, seq0, n_q, cap, last=None, gap=3, std=1.0):
        torch = torch_mod()
        g = np.random.default_rng(seed)
        self.B, self.dtype, self.shape = B, dtype, (H, hkv, hd)
        n_seq = seq0[-1]
        self.n_q, self.lens, self.seq0 = n_q, lens, seq0
        draw = lambda *s: torch.from_numpy(g.standard_normal(s).astype(np.float32) * std).cuda().to(tdt(dtype))  # noqa: E731
        self.row0, at = [], 0
        for n in lens:
            self.row0.append(at)
            at += n + gap
        self.k, self.v = draw(max(at, 1), hkv * hd), draw(max(at, 1), hkv * hd)
        for r, n in zip(self.row0, lens):
            self.k[r + n:r + n + gap] = float("nan")
            self.v[r + n:r + n + gap] = float("inf")
        self.ok, self.ov = draw(n_seq, cap, hkv * hd), draw(n_seq, cap, hkv * hd)
        self.q = draw(n_seq, n_q, H * hd)
        if last is None:
            last = g.integers(-2, cap, (n_seq, n_q)) if cap else g.integers(-2, 0, (n_seq, n_q))
            last[0, 0] = cap - 1
        self.last_np = np.asarray(last).reshape(n_seq, n_q)
        for s in range(n_seq):
            m = max(self.last_np[s].max() + 1, 0)
            self.ok[s, m:] = float("nan")
            self.ov[s, m:] = float("nan")
        self.q[torch.from_numpy(self.last_np == -2).cuda()] = float("nan")
        self.last = dev_i32(self.last_np)
        self.dims = dims_of(B, H, hkv, hd, dtype)
        self.kv = B.shared_kv(self.k, self.v, self.row0, lens, seq0, self.ok if cap else None, self.ov if cap else None)
        self.out = torch.full_like(self.q, 9.0)
        self.ws = torch.full((B.cb_shared_workspace_bytes(self.kv, self.dims, n_q),), 255, dtype=torch.uint8, device="cuda")

    def run(self):
        self.B.cb_shared_attention(self.q, self.last, self.n_q, self.kv, self.dims, self.out, self.ws)
        return self.out

    def check(self, rows=None):
        """rows: sequences to compare (all)."""
        H, hkv, hd = self.shape
        rows = range(self.seq0[-1]) if rows is None else rows
        heads = lambda t: np.nan_to_num(host(t)).reshape(*t.shape[:-1], hkv, hd)  # noqa: E731
        out = host(self.out).reshape(-1, self.n_q, H, hd)
        assert np.all(np.isfinite(out))
        k, v = heads(self.k), heads(self.v)
        for s in rows:
            g = int(np.searchsorted(self.seq0, s, side="right")) - 1
            while self.seq0[g] == self.seq0[g + 1]:
                g += 1
            r = slice(self.row0[g], self.row0[g] + self.lens[g])
            q = np.nan_to_num(host(self.q[s:s + 1])).reshape(1, self.n_q, H, hd)
            ok, ov = heads(self.ok[s:s + 1]), heads(self.ov[s:s + 1])
            ref, mag = A.shared_attention(q, self.last_np[s:s + 1], [(k[r], v[r])], [0, 1], ok, ov)
            keys = np.repeat(np.concatenate([k[r], ok[0]]), H // hkv, axis=1)
            S = np.einsum("jhc,ihc->jhi", np.abs(q[0]), np.abs(keys)).max(2, initial=0) / np.sqrt(hd)
            n = keys.shape[0]
            rel = 2 * ((hd + 8) * EPS * S + 2.0 ** -20) + (n + 16) * EPS + (2.0 ** -8 if self.dtype == "bf16" else 0.0)
            tol = rel[..., None] * mag[0] + (2.0 ** -8 if self.dtype == "bf16" else EPS) * np.abs(ref[0]) * 1.01 + 1e-30
            err = np.abs(out[s] - ref[0])
            assert np.all(err <= tol), (s, float((err / tol).max()))
            assert np.all(out[s][self.last_np[s] == -2] == 0)


SHAPES = [(4, 4, 64), (7, 1, 128), (8, 2, 64), (2, 2, 128), (6, 2, 32), (3, 3, 96), (4, 1, 256), (4, 2, 160)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,hkv,hd", SHAPES)
@pytest.mark.parametrize("lens,seq0,n_q,cap", [([1], [0, 1], 1, 1), ([129], [0, 3], 1, 40), ([300, 17], [0, 2, 5], 2, 70),
                                               ([0, 128, 5], [0, 2, 2, 4], 1, 33), ([255], [0, 1], 1, 0), ([0], [0, 3], 3, 200)])
def test_against_the_oracle(B, dtype, H, hkv, hd, lens, seq0, n_q, cap):
    c = Case(B, hd + sum(lens), dtype, H, hkv, hd, lens, seq0, n_q, cap)
    c.run()
    B.cb_sync(None)
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,hkv,hd,lens,seq0,n_q,cap", [
    (4, 4, 128, [4096], [0, 4], 1, 64),                  # few answers, a prefix cut into many pieces
    (14, 2, 128, [2000], [0, 37], 1, 300),               # more rows than a tile
    (8, 8, 64, [700, 1500, 64], [0, 9, 10, 30], 4, 260),  # several prefixes
    (7, 1, 128, [1000], [0, 5], 61, 130),                # questions of many rows
    (12, 4, 64, [130], [0, 2], 130, 140)])
def test_larger_ones(B, dtype, H, hkv, hd, lens, seq0, n_q, cap):
    c = Case(B, 11, dtype, H, hkv, hd, lens, seq0, n_q, cap)
    c.run()
    B.cb_sync(None)
    c.check(range(0, seq0[-1], max(1, seq0[-1] // 6)))
    first = c.out.clone()
    c.ws.fill_(127)
    c.out.fill_(3.0)
    c.run()
    B.cb_sync(None)
    assert bool((c.out == first).all())                  # the same from run to run, whatever the workspace held


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hd", [64, 128, 256])
def test_strong_scores_late_maxima_and_equal_rows(B, dtype, hd):
    """Scores up to about 60 whose largest comes last (or first), and rows that are all alike."""
    torch = torch_mod()
    for order in (1, -1):
        c = Case(B, 3, dtype, 2, 1, hd, [600], [0, 2], 2, 90, last=[[89, 50], [-1, 3]])
        ramp = torch.linspace(0.1, 8.0, 690, device="cuda")
        ramp = ramp if order == 1 else ramp.flip(0)
        base = torch.randn(hd, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4))
        base /= base.norm()
        c.k[:600] = (ramp[:600, None] * base).to(c.k.dtype)
        c.ok[0] = (ramp[600:, None] * base).to(c.k.dtype)
        c.ok[1, :4] = (ramp[600:604, None] * base).to(c.k.dtype)
        c.q[:] = (8.0 * hd ** 0.5 * base).repeat(2).to(c.q.dtype)
        c.run()
        B.cb_sync(None)
        c.check()
    c = Case(B, 5, dtype, 2, 1, hd, [500], [0, 1], 1, 20, last=[[19]])
    c.k[:500], c.v[:500] = 1.0, 2.0
    c.ok[0], c.ov[0] = 1.0, 2.0
    c.run()
    B.cb_sync(None)
    assert float((c.out.float() - 2).abs().max()) <= (2.0 ** -6 if dtype == "bf16" else 2.0 ** -14)


def test_bad_bounds_are_reported_and_count_as_padding(B):
    for dtype, hd in (("bf16", 128), ("f32", 64)):
        c = Case(B, 6, dtype, 2, 2, hd, [40], [0, 3], 2, 10, last=[[9, -1], [3, 4], [-1, 0]])
        c.run()
        B.cb_sync(None)
        ref = c.out.clone()
        for s, j, bad in ((0, 0, 10), (1, 1, -3), (2, 0, 2 ** 31 - 1), (2, 1, -2 ** 31)):
            l = c.last_np.copy()
            l[s, j] = bad
            c.last = dev_i32(l)
            c.out.fill_(5.0)
            c.run()
            with pytest.raises(B.CBError) as e:
                B.cb_sync(None)
            assert e.value.status == 9
            keep = torch_mod().ones(3, 2, dtype=torch_mod().bool, device="cuda")
            keep[s, j] = False
            assert bool((c.out[keep] == ref[keep]).all()) and bool((c.out[s, j] == 0).all())


def test_a_query_that_is_not_finite_spoils_its_own_row_only(B):
    torch = torch_mod()
    for dtype, hd in (("bf16", 128), ("bf16", 64), ("f32", 64), ("bf16", 96)):
        c = Case(B, 7, dtype, 4, 2, hd, [300], [0, 3], 2, 10, last=[[9, -1], [3, 4], [-1, 0]])
        c.run()
        ref = c.out.clone()
        c.q[1, 1, 3 * hd + 5] = float("nan")
        c.run()
        B.cb_sync(None)
        o, r = c.out.reshape(3, 2, 4, hd), ref.reshape(3, 2, 4, hd)
        assert bool(torch.isnan(o[1, 1, 3]).all())
        o[1, 1, 3] = r[1, 1, 3]
        assert torch.equal(o, r)


def test_another_stream_graphs_that_share_a_workspace(B):
    torch = torch_mod()
    a = Case(B, 8, "bf16", 14, 2, 128, [900], [0, 5], 1, 64, last=[[63], [0], [-1], [12], [40]])
    b = Case(B, 9, "bf16", 14, 2, 128, [333, 100], [0, 2, 5], 1, 64, last=[[5], [0], [-1], [63], [-2]])
    ref = [c.run().clone() for c in (a, b)]
    B.cb_sync(None)
    if b.ws.numel() > a.ws.numel():
        a.ws = b.ws
    b.ws = a.ws
    graphs = []
    s = torch.cuda.Stream()
    for c in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            c.run()
        graphs.append(g)
    for _ in range(3):
        for c in (a, b):
            c.out.fill_(1.0)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.out, ref[0]) and torch.equal(b.out, ref[1])
    with torch.cuda.stream(s):
        a.out.fill_(1.0)
        a.run()
    B.cb_sync(s)
    assert torch.equal(a.out, ref[0])


def test_own_caches_past_2_to_the_31_elements(B):
    """The last sequences of a large batch of caches, and a prefix that starts past 2^31 elements."""
    torch = torch_mod()
    H, hkv, hd, cap, n_seq = 8, 8, 128, 1 << 15, 66
    rows = (1 << 21) + 200
    k, v = (torch.zeros(rows, hkv * hd, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ok, ov = (torch.zeros(n_seq, cap, hkv * hd, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(1)
    for t in (k[-150:], v[-150:], ok[-1, :40], ov[-1, :40], ok[-1, -30:], ov[-1, -30:]):
        t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
    q = torch.randn(n_seq, 1, H * hd, generator=g, device="cuda").bfloat16()
    dims = dims_of(B, H, hkv, hd, "bf16")
    kv = B.shared_kv(k, v, [rows - 150], [150], [0, n_seq], ok, ov)
    out, ws = torch.empty_like(q), torch.empty(B.cb_shared_workspace_bytes(kv, dims, 1), dtype=torch.uint8, device="cuda")
    last = torch.full((n_seq, 1), -1, dtype=torch.int32, device="cuda")
    for l in (39, cap - 1):
        last[-1] = l
        B.cb_shared_attention(q, last, 1, kv, dims, out, ws)
        B.cb_sync(None)
        keys = torch.cat([k[-150:], ok[-1, :l + 1]]).double().reshape(-1, hkv, hd)
        vals = torch.cat([v[-150:], ov[-1, :l + 1]]).double().reshape(-1, hkv, hd)
        p = torch.softmax(torch.einsum("hc,ihc->hi", q[-1, 0].double().reshape(H, hd), keys) / hd ** 0.5, 1)
        ref = torch.einsum("hi,ihc->hc", p, vals).reshape(-1)
        mag = torch.einsum("hi,ihc->hc", p, vals.abs()).reshape(-1)
        assert bool(((out[-1, 0].double() - ref).abs() <= 2.0 ** -7 * 1.1 * mag + (l + 200) * 2 * EPS * mag).all())


@pytest.mark.parametrize("H,hkv,n_seq,n_q", [(2, 2, 1100, 1), (16, 1, 1024, 8), (16, 1, 1025, 8), (14, 2, 300, 1),
                                               (16, 1, 2100, 8), (16, 1, 2100, 3), (2, 2, 2500, 1), (64, 1, 2, 2060)])
def test_many_sequences(B, H, hkv, n_seq, n_q):
    """Row tiles up to as many as a call takes at once, and beyond; more sequences than a block keeps."""
    c = Case(B, n_seq, "bf16", H, hkv, 64, [130, 200], [0, max(n_seq - 7, 1), n_seq], n_q, 21)
    c.run()
    B.cb_sync(None)
    c.check({0, 1, min(2, n_seq - 1), n_seq // 2, max(n_seq - 8, 0), max(n_seq - 7, 0), n_seq - 1})


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("cap", [0, 50, 300])
def test_many_queries_of_several_groups(B, hd, cap):
    """Prefixes and groups that are empty, sequences of padding, of the prefix alone, of the last row alone."""
    lens, seq0, n_q = [300, 64, 0, 129, 0], [0, 2, 2, 5, 6, 7], 36
    g = np.random.default_rng(cap)
    last = g.integers(-2, max(cap, 1), (7, n_q)) if cap else g.integers(-2, 0, (7, n_q))
    last[1] = -2
    last[3] = -1
    last[4, :20] = -2
    last[4, 20:] = cap - 1
    last[6, 18:] = -2
    c = Case(B, 3, "bf16", 14, 2, hd, lens, seq0, n_q, cap, last=last)
    c.run()
    B.cb_sync(None)
    c.check()


def test_absent_prefixes_have_no_address(B):
    """Prefixes of no rows: their buffer may be missing whatever its count of rows says."""
    for dtype in ("bf16", "f32"):
        for n_q in (1, 64):
            c = Case(B, 5, dtype, 4, 2, 64, [0, 0], [0, 2, 3], n_q, 40)
            c.kv.k = c.kv.v = None
            c.run()
            B.cb_sync(None)
            c.check()


def test_two_streams_at_once(B):
    """Calls of three kinds and a draw, on two streams with workspaces of their own, give what they give alone."""
    torch = torch_mod()
    cases = [[Case(B, s, "bf16", 14, 2, 128, [1500], [0, 9], 1, 200), Case(B, s + 1, "bf16", 14, 2, 128, [900], [0, 3], 40, 60),
              Case(B, s + 2, "f32", 4, 4, 64, [500], [0, 3], 2, 40)] for s in (20, 30)]
    logits = [torch.randn(40, 9001, device="cuda") for _ in range(2)]
    u = torch.rand(40, device="cuda")
    rules = B.sample_rules(top_p=torch.full((40,), 0.9, device="cuda"))
    tokens = [torch.zeros(40, dtype=torch.int32, device="cuda") for _ in range(2)]

    def all_of(i, stream=None):
        for c in cases[i]:
            B.cb_shared_attention(c.q, c.last, c.n_q, c.kv, c.dims, c.out, c.ws, stream=stream)
        B.cb_sample_token(logits[i], u, rules, tokens[i], stream=stream)

    alone = []
    for i in range(2):
        all_of(i)
        B.cb_sync(None)
        alone.append([c.out.clone() for c in cases[i]] + [tokens[i].clone()])
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(2):
        for c in cases[i]:
            c.out.fill_(5.0)
        tokens[i].fill_(-9)
    torch.cuda.synchronize()
    for _ in range(30):
        for i, s in enumerate(streams):
            all_of(i, s.cuda_stream)
    torch.cuda.synchronize()
    B.cb_sync(None)
    for i in range(2):
        for got, want in zip([c.out for c in cases[i]] + [tokens[i]], alone[i]):
            assert bool((got == want).all())


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("H,hkv,lens,seq0,n_q,cap", [
    (2, 2, [700], [0, 9], 50, 300),                      # 50 of a tile's 128 rows
    (4, 2, [300, 0, 129], [0, 3, 7, 12], 17, 40),        # a group without a prefix
    (7, 1, [1000, 64], [0, 5, 11], 5, 200),
    (3, 3, [0], [0, 6], 70, 150),                        # no prefix at all
    (32, 1, [513], [0, 20], 1, 33)])
def test_questions_that_share_tiles(B, hd, H, hkv, lens, seq0, n_q, cap):
    """Enough rows of a sequence for its own keys to go with the prefixes, too few to fill tiles."""
    g = np.random.default_rng(n_q)
    n = seq0[-1]
    last = g.integers(-2, cap, (n, n_q))
    last[0] = -2
    last[1] = -1
    last[2, : n_q // 2] = -2
    last[n - 1] = cap - 1
    c = Case(B, 8, "bf16", H, hkv, hd, lens, seq0, n_q, cap, last=last)
    c.run()
    B.cb_sync(None)
    c.check()
    first = c.out.clone()
    c.ws.fill_(129)
    c.run()
    B.cb_sync(None)
    assert bool((c.out == first).all())


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("n_q", [1, 3])
def test_short_and_long_prefixes_by_turns(B, hd, n_q):
    """Runs of work of one key tile each, in which only one of two groups has a share, before longer ones."""
    lens, seq0 = [], [0]
    for i in range(20):
        lens += [60, 400 + 50 * i]
        seq0 += [seq0[-1] + 90, seq0[-1] + 120]
    c = Case(B, 12, "bf16", 8, 8, hd, lens, seq0, n_q, 0)
    c.run()
    B.cb_sync(None)
    c.check([x + d for x in seq0[:-1] for d in (0, 17)])
    first = c.out.clone()
    for _ in range(5):
        c.out.fill_(7.0)
        c.run()
        assert bool((c.out == first).all())
    B.cb_sync(None)


@pytest.mark.parametrize("n_seq,n_q,cap,rows", [(29, 88, 100, [5]), (700, 1, 4, [0, 333, 699])])
def test_a_prefix_larger_than_the_cache(B, n_seq, n_q, cap, rows):
    """Several row tiles over 134 MB of keys and values, a part of the heads at a time."""
    c = Case(B, 14, "bf16", 32, 32, 128, [8204], [0, n_seq], n_q, cap)
    c.run()
    B.cb_sync(None)
    c.check(rows)
    first = c.out.clone()
    c.ws.fill_(130)
    c.run()
    B.cb_sync(None)
    assert bool((c.out == first).all())
