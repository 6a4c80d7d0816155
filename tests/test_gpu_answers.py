"""Several answers sampled from one blended prompt, token by token: the new tokens' rows rotated into their
own caches, attention over the blend's K and V and the own rows, the logit rules, the draw.  Every step's
attention and token are checked against the fp64 oracle fed with the step's own inputs; a captured step gives
what the eager one gives."""
import numpy as np
import pytest

import oracle.answers_oracle as A
from tests.gpu_util import TOL, dev_i32, ensure_lib, host, rel, tdt, torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    torch_mod()
    ensure_lib()
    from non_prefix_kv_gb300 import binding
    return binding


def shape_of(dtype):
    from non_prefix_kv_gb300 import synth
    return synth.ModelShape(n_layers=2, d_model=256, n_heads=4, n_kv_heads=2, head_dim=64, d_ff=512, vocab=512, dtype=dtype,
                            w_std=0.06)


def spec_of(B, s):
    return B.rope_spec(B.CB_ROPE_INTERLEAVED, s.head_dim, 1e4, scaling=B.CB_ROPE_RAMP, factor=4.0, original_len=128,
                       low=1.0, high=32.0, amplitude=0.1 * np.log(4.0) + 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("q8", [False, True])
def test_a_blend_with_scaled_positions(B, dtype, q8):
    """Recomputing every row gives the full prefill, as with plain positions: the first layer's K are the cached
    ones, moved to their places (an amplitude applied twice would show), the second's recomputed."""
    if q8 and dtype == "f32":
        pytest.skip("one store is enough")
    from non_prefix_kv_gb300 import engine as E, synth
    torch = torch_mod()
    s = shape_of(dtype)
    g = np.random.default_rng(3)
    pool = [g.integers(0, s.vocab, 96).astype(np.int32) for _ in range(3)]
    tokens = np.concatenate(pool + [g.integers(0, s.vocab, 30).astype(np.int32)])
    dm = E.DeviceModel.from_host(synth.make_model(s, seed=4))
    eng = E.BlendEngine(dm, len(tokens), max_pos=512, rope=spec_of(B, s))
    p = eng.precompute_pool(pool)
    req = E.Request(eng, E.ChunkPoolQ8.from_pool(p, dm.dims) if q8 else p, [0, 1, 2], tokens)
    E.run_blend(req, E.layer_plan(s, req.N, req.n_cached, [1.0, 1.0]))
    K, V = ([torch.empty_like(t) for t in req.K] for _ in range(2))
    eng.full_prefill(req.tokens, K, V, None)
    B.cb_sync(None)
    for l in range(s.n_layers):
        # (8-bit codes: a step of 1/255 of a channel's range of some six standard deviations, rms 0.29 of it: 0.7 %)
        assert rel(host(req.K[l]), host(K[l])) < (2e-2 if q8 else TOL[dtype]), l
    plain = E.BlendEngine(dm, len(tokens), max_pos=512)
    plain.full_prefill(req.tokens, req.K, req.V, None)
    B.cb_sync(None)
    assert rel(host(req.K[0]), host(K[0])) > 0.1                      # another model's positions
    with pytest.raises(ValueError):
        E.BlendEngine(dm, 64, rope=B.rope_spec(B.CB_ROPE_HALF, s.head_dim, 1e4))


class Answers:
    """n answers to one request; every buffer of a step is made once."""

    def __init__(self, B, dtype, n, cap, seed):
        from non_prefix_kv_gb300 import engine as E, synth
        torch = torch_mod()
        s = self.s = shape_of(dtype)
        g = np.random.default_rng(seed)
        pool = [g.integers(0, s.vocab, 96).astype(np.int32) for _ in range(3)]
        tokens = np.concatenate(pool + [g.integers(0, s.vocab, 30).astype(np.int32)])
        self.B, self.n, self.cap, self.dtype = B, n, cap, dtype
        self.dm = E.DeviceModel.from_host(synth.make_model(s, seed=4))
        self.spec = spec_of(B, s)
        self.eng = E.BlendEngine(self.dm, len(tokens), max_pos=512, rope=self.spec)
        self.req = E.Request(self.eng, self.eng.precompute_pool(pool), [0, 1, 2], tokens)
        E.run_blend(self.req, E.layer_plan(s, self.req.N, self.req.n_cached, [1.0, 0.3]))
        self.N = len(tokens)
        dt = tdt(dtype)
        new = lambda *z, d=dt: torch.zeros(*z, dtype=d, device="cuda")  # noqa: E731
        self.own = [(torch.full((n, cap, s.kv_width), float("nan"), dtype=dt, device="cuda"),
                     torch.full((n, cap, s.kv_width), float("nan"), dtype=dt, device="cuda")) for _ in range(s.n_layers)]
        self.kv = [B.shared_kv(self.req.K[l], self.req.V[l], [0], [self.N], [0, n], *self.own[l]) for l in range(s.n_layers)]
        self.ws = new(max(1, B.cb_shared_workspace_bytes(self.kv[0], self.dm.dims, 1)), d=torch.uint8)
        self.x, self.a, self.qkv = new(n, s.d_model), new(n, s.d_model), new(n, s.qkv_width)
        self.q, self.o = new(n, s.q_width), [new(n, s.q_width) for _ in range(s.n_layers)]
        self.qs = [new(n, s.q_width) for _ in range(s.n_layers)]
        self.logits, self.ruled = new(n, s.vocab), new(n, s.vocab)
        self.token, self.kept = new(n, d=torch.int32), new(n, d=torch.int32)
        self.logprob, self.u = new(n, d=torch.float32), new(n, d=torch.float32)
        self.pos, self.row, self.last = (new(n, d=torch.int32) for _ in range(3))
        self.hist, self.hist_len = new(n, 64, d=torch.int32), new(n, d=torch.int32)
        self.rules = B.logit_rules(history=self.hist, history_len=self.hist_len,
                                   repetition=torch.full((n,), 1.2, device="cuda"))
        self.sample = B.sample_rules(temperature=torch.tensor([0.0, 0.7, 1.0, 1.3, 0.9][:n], device="cuda"),
                                     top_k=dev_i32([0, 40, 0, 100, 0][:n]), top_p=torch.tensor([1.0, 0.9, 0.95, 1.0, 1.0][:n], device="cuda"),
                                     min_p=torch.tensor([0.0, 0.0, 0.02, 0.0, 0.0][:n], device="cuda"))

    def step(self):
        B, s, d = self.B, self.s, self.dm.dims
        n, t = self.n, d.dtype
        B.cb_gather_rows(self.x, self.dm.embed, self.token, n, s.d_model * self.x.element_size())
        for l in range(s.n_layers):
            w = self.dm.layers[l]
            B.cb_rmsnorm(self.a, self.x, None, n, s.d_model, w["attn_norm"], s.rms_eps, t, t)
            B.cb_linear(self.a, w["wqkv"], self.qkv, n, s.qkv_width, s.d_model, t)
            q, k, v = self.qkv.split([s.q_width, s.kv_width, s.kv_width], 1)
            ok, ov = (c.view(n * self.cap, s.kv_width) for c in self.own[l])
            B.cb_rope_rows(q, k, v, self.pos, self.qs[l], ok, ov, d, self.spec, self.eng.cos_sin, self.eng.max_pos, kv_row=self.row)
            B.cb_shared_attention(self.qs[l], self.last, 1, self.kv[l], d, self.o[l], self.ws)
            B.cb_o_proj_ffn(self.o[l], self.x, n, d, self.dm.layers_c[l], self.x, self.eng.ws)
        B.cb_rmsnorm(self.a, self.x, None, n, s.d_model, self.dm.final_norm, s.rms_eps, t, t)
        B.cb_linear(self.a, self.dm.w_lm, self.logits, n, s.vocab, s.d_model, t)
        B.cb_logits_process(self.logits, self.rules, self.ruled)
        B.cb_sample_token(self.ruled, self.u, self.sample, self.token, self.logprob, self.kept)

    def place(self, i, u, done):
        """The inputs of step i: answers that have ended (done) store nothing and see nothing."""
        torch = torch_mod()
        n, r = self.n, torch.arange(self.n, device="cuda", dtype=torch.int32)
        over = torch.tensor(done, device="cuda")
        self.pos.fill_(self.N + i)
        self.row.copy_(torch.where(over, torch.full_like(r, -1), r * self.cap + i))
        self.last.copy_(torch.where(over, torch.full_like(r, -2), torch.full_like(r, i)))
        self.hist[:, i] = self.token
        self.hist_len.fill_(i + 1)
        self.u.copy_(torch.from_numpy(u.astype(np.float32)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_answers_token_by_token(B, dtype):
    """Tolerance of the attention as in its own test, here with one figure a row: a score's error at most
    (hd + 8) 2^-24 max |q||k| / sqrt(hd), doubled, plus bf16's roundings of a weight and of the output."""
    a = Answers(B, dtype, 5, 24, 11)
    s = a.s
    hkv, hd, H = s.n_kv_heads, s.head_dim, s.n_heads
    g = np.random.default_rng(1)
    a.token.copy_(dev_i32(g.integers(0, s.vocab, a.n)))
    drawn = set()
    prefix = [(host(a.req.K[l]).reshape(-1, hkv, hd), host(a.req.V[l]).reshape(-1, hkv, hd)) for l in range(s.n_layers)]
    for i in range(6):
        u, done = g.random(a.n), [i > 3 and j == 2 for j in range(a.n)]
        a.place(i, u, done)
        a.step()
        B.cb_sync(None)
        last = np.array([[-2 if d else i] for d in done])
        for l in range(s.n_layers):
            ok, ov = (np.nan_to_num(host(c)).reshape(a.n, a.cap, hkv, hd) for c in a.own[l])
            q = np.nan_to_num(host(a.qs[l])).reshape(a.n, 1, H, hd)
            ref, mag = A.shared_attention(q, last, [prefix[l]], [0, a.n], ok, ov)
            S = np.linalg.norm(q, axis=3).max() * max(np.linalg.norm(prefix[l][0], axis=2).max(), np.linalg.norm(ok, axis=3).max()) / np.sqrt(hd)
            relative = 2 * ((hd + 8) * 2.0 ** -24 * S + 2.0 ** -20) + (a.N + 40) * 2.0 ** -24 + (2.0 ** -8 if dtype == "bf16" else 0)
            err = np.abs(host(a.o[l]).reshape(ref.shape) - ref)
            assert np.all(err <= relative * mag + (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) * np.abs(ref) * 1.01 + 1e-30)
        x, uu = host(a.ruled), host(a.u)
        T, k, p, m = (host(t) for t in a.sample.tensors)
        for j in range(a.n):
            w = A.sample(x[j], uu[j], T[j], int(k[j]), p[j], m[j])
            assert w[3] > 2.0 ** -28 and (int(a.token[j]), int(a.kept[j])) == (w[0], w[2])
        drawn.update(a.token.tolist())
    assert len(drawn) > 8


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_captured_step_gives_what_an_eager_one_gives(B, dtype):
    torch = torch_mod()
    a, b = Answers(B, dtype, 4, 16, 12), Answers(B, dtype, 4, 16, 12)
    b.place(0, np.full(4, 0.5), [False] * 4)
    b.step()                                              # first calls set kernel attributes
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step()
    for x in b.own:
        for t in x:
            t.fill_(float("nan"))
    g = np.random.default_rng(2)
    start = g.integers(0, a.s.vocab, 4)
    for z in (a, b):
        z.token.copy_(dev_i32(start))
        z.hist.zero_()
    for i in range(8):
        u = g.random(4)
        a.place(i, u, [False] * 4)
        b.place(i, u, [False] * 4)
        a.step()
        graph.replay()
        B.cb_sync(None)
        assert a.token.tolist() == b.token.tolist() and torch.equal(a.logprob, b.logprob) and torch.equal(a.ruled, b.ruled)
