"""What the calls of the rotary forms, the shared-prefix attention and the sampling take and refuse, on the host (no
GPU is touched: every call here is refused before anything is launched)."""
import ctypes as C

import pytest

from non_prefix_kv_gb300 import binding as B
from non_prefix_kv_gb300 import build as nb


@pytest.fixture(scope="module")
def lib():
    nb.build()
    return B.lib()


def _dims(**kw):
    base = dict(d_model=256, n_heads=4, n_kv_heads=2, head_dim=64, d_ff=512, vocab=1024, rope_base=1e4,
                rms_eps=1e-5, dtype=B.CB_BF16)
    base.update(kw)
    return B.cb_dims(**base)


# ---- rotary forms ----------------------------------------------------------------------------
@pytest.mark.parametrize("kw,status", [
    (dict(layout=2), 1), (dict(scaling=5), 1), (dict(scaling=-1), 1), (dict(rot_dim=0), 2), (dict(rot_dim=3), 2),
    (dict(rot_dim=258), 2), (dict(base=1.0), 1), (dict(base=float("inf")), 1), (dict(scaling=1, factor=0.5), 1),
    (dict(scaling=1, factor=float("nan")), 1), (dict(scaling=2, rot_dim=2), 2), (dict(scaling=3), 1),
    (dict(scaling=3, original_len=100.0), 1), (dict(scaling=3, original_len=100.0, low=4.0, high=4.0), 1),
    (dict(scaling=4, original_len=0.0, low=1.0, high=2.0), 1), (dict(amplitude=0.0), 1), (dict(amplitude=float("nan")), 1)])
def test_specs_that_are_none(lib, kw, status):
    a = dict(layout=0, rot_dim=64, base=1e4, scaling=0)
    a.update(kw)
    with pytest.raises(B.CBError) as e:
        B.rope_spec(**a)
    assert e.value.status == status


def test_a_plain_spec_needs_no_scaling_figures(lib):
    s = B.rope_spec(0, 64, 1e4, factor=0.0)
    assert len(B.cb_rope_theta(s)) == 32
    assert lib.cb_rope_theta(C.byref(s), None) == 1 and lib.cb_rope_table_scaled(None, 10, C.byref(s), None) == 1
    assert lib.cb_rope_table_scaled(None, 0, C.byref(s), None) == 0 and lib.cb_rope_table_scaled(8, 10, C.byref(s), None) == 1
    assert lib.cb_rope_table_scaled(1 << 40, -1, C.byref(s), None) == 2 and lib.cb_rope_table_scaled(1 << 40, 1, None, None) == 1


N, QW, W = 10, 256, 128                                     # rows, and elements of theirs
AT = dict(q=1 << 30, q_out=1 << 31, k=1 << 32, v=1 << 33, k_out=1 << 34, v_out=1 << 35, src_row=1 << 36, kv_row=1 << 37)
POS, TAB = 1 << 38, 1 << 39


def rope(lib, n=N, dims=None, spec=None, pos=POS, tab=TAB, max_pos=100, **kw):
    a = dict(AT, q_ld=0, q_out_ld=0, k_ld=0, v_ld=0, n_src_rows=20, kv_out_ld=0, n_out_rows=30)
    a.update(kw)
    io = B.cb_rope_rows_io(**a)
    return lib.cb_rope_rows(C.byref(io), pos, n, 0, C.byref(dims or _dims()), C.byref(spec or B.rope_spec(1, 64, 1e4)), tab,
                            max_pos, None)


def refused(lib, status):
    return status == 1 and b"overlaps" in lib.cb_last_error_message()


def test_rope_rows_refuses_bad_arguments(lib):
    assert rope(lib, n=-1) == 2 and rope(lib, max_pos=0) == 2 and rope(lib, n=0) == 0
    assert rope(lib, dims=_dims(head_dim=32, d_model=128)) == 2              # rot_dim exceeds head_dim
    assert rope(lib, pos=None) == 1 and rope(lib, tab=None) == 1 and rope(lib, pos=POS + 2) == 1 and rope(lib, tab=TAB + 4) == 1
    for k in ("q", "q_out", "k", "k_out", "v", "v_out"):
        assert rope(lib, **{k: None}) == 1
        assert rope(lib, **{k: AT[k] + 1}) == 1
    assert rope(lib, q=None, q_out=None, k=None, k_out=None, v=None, v_out=None) == 1
    assert rope(lib, k=None, k_out=None) == 1                               # v without k
    for k, w in (("q_ld", QW), ("q_out_ld", QW), ("k_ld", W), ("v_ld", W), ("kv_out_ld", W)):
        assert rope(lib, **{k: w - 1}) == 2 and rope(lib, **{k: -1}) == 2 and rope(lib, **{k: 1 << 41}) == 2
    assert rope(lib, src_row=None, n_src_rows=N - 1) == 2 and rope(lib, kv_row=None, n_out_rows=N - 1) == 2
    assert rope(lib, n_src_rows=-1) == 2 and rope(lib, n_out_rows=1 << 31) == 2
    assert rope(lib, src_row=AT["src_row"] + 2) == 1


def test_rope_rows_refuses_outputs_that_overlap(lib):
    size = dict(q=N * QW, q_out=N * QW, k=20 * W, v=20 * W, k_out=30 * W, v_out=30 * W)
    for out in ("q_out", "k_out", "v_out"):
        others = [(AT[k], 2 * size[k]) for k in size if k != out] + [(AT["src_row"], 4 * N), (AT["kv_row"], 4 * N), (POS, 4 * N),
                                                                      (TAB, 100 * 64 * 4)]
        for base, n in others:
            for p in (base, base + n - 2, base - 2 * size[out] + 2):
                if (out, p) == ("q_out", AT["q"]):
                    continue                                # in place, row by row
                assert refused(lib, rope(lib, **{out: p})), (out, p - base)
    # in place only row by row
    assert refused(lib, rope(lib, k_out=AT["k"])) and refused(lib, rope(lib, v_out=AT["v"], kv_row=None))
    assert refused(lib, rope(lib, q_out=AT["q"], q_ld=QW + 8))


# ---- shared prefix ---------------------------------------------------------------------------
def kv(row0=(0,), length=(100,), seq0=(0, 3), n_rows=100, capacity=20, **kw):
    i32 = lambda a: (C.c_int32 * len(a))(*a)  # noqa: E731
    a = dict(k=1 << 40, v=1 << 41, n_rows=n_rows, row0_host=i32(row0), len_host=i32(length), seq0_host=i32(seq0),
             n_groups=len(row0), n_seq=seq0[-1], own_k=1 << 42, own_v=1 << 43, capacity=capacity)
    a.update(kw)
    c = B.cb_shared_kv(**a)
    c.keep = a
    return c


def query(lib, c, n_q=2, dims=None):
    out = C.c_size_t(0)
    st = lib.cb_shared_workspace_bytes(C.byref(c) if c is not None else None, C.byref(dims or _dims()), n_q, C.byref(out))
    return st, out.value


@pytest.mark.parametrize("dtype", [B.CB_BF16, B.CB_F32])
@pytest.mark.parametrize("kw,status", [
    (dict(n_groups=0), 2), (dict(n_groups=65), 2), (dict(n_seq=0, seq0=(0, 0)), 2), (dict(n_seq=65536, seq0=(0, 65536)), 2),
    (dict(row0_host=None), 1), (dict(len_host=None), 1), (dict(seq0_host=None), 1), (dict(n_rows=99), 2), (dict(n_rows=-1), 2),
    (dict(row0=(-1,)), 2), (dict(length=(-1,)), 2), (dict(row0=(1,)), 2), (dict(seq0=(1, 3)), 2), (dict(n_seq=4), 2),
    (dict(row0=(0, 0), length=(1, 1), seq0=(0, 4, 3)), 2), (dict(k=None), 1), (dict(v=None), 1), (dict(own_k=None), 1),
    (dict(own_v=None), 1), (dict(capacity=-1), 2), (dict(capacity=1 << 30), 2), (dict(k=(1 << 40) + 8), 1), (dict(own_v=4), 1)])
def test_the_handle_and_the_workspace_query(lib, kw, status, dtype):
    assert query(lib, kv(**kw), dims=_dims(dtype=dtype))[0] == status


def test_what_a_handle_may_leave_out(lib):
    ok = lambda c, **k: query(lib, c, **k)  # noqa: E731
    assert ok(kv())[0] == 0 and ok(kv())[1] > 0 and ok(kv(), n_q=0) == (0, 0) and ok(kv(), n_q=-1)[0] == 2 and ok(None)[0] == 1
    assert ok(kv(capacity=0, own_k=None, own_v=None))[0] == 0
    assert ok(kv(length=(0,), n_rows=0, k=None, v=None))[0] == 0
    assert ok(kv(seq0=(0, 0, 3), row0=(0, 0), length=(5, 5)))[0] == 0
    assert ok(kv(seq0=(0, 65535), capacity=3), n_q=1 << 15)[0] == 8           # more than 2^30 query rows of a KV head


@pytest.mark.parametrize("dtype,hd", [(B.CB_BF16, 64), (B.CB_BF16, 96), (B.CB_F32, 64)])
@pytest.mark.parametrize("n_q", [1, 2, 70])
def test_shared_attention_refuses_what_it_writes_over_another_argument(lib, dtype, hd, n_q):
    d, c = _dims(dtype=dtype, head_dim=hd, d_model=4 * hd), kv()
    st, need = query(lib, c, n_q, d)
    assert st == 0
    e = 2 if dtype == B.CB_BF16 else 4
    q, last, out, ws = 1 << 30, 1 << 31, 1 << 32, 1 << 33
    rows, w = 3 * n_q, 2 * hd * e

    def call(q=q, last=last, out=out, ws=ws, n=need, c=c, n_q=n_q):
        return lib.cb_shared_attention(q, last, n_q, C.byref(c), C.byref(d), out, ws, n, None)

    assert call(n=need - 1) == 4 and call(ws=None) == 4 and call(n_q=0) == 0 and call(n_q=-1) == 2
    for a in ("q", "last", "out"):
        assert call(**{a: None}) == 1
    assert call(q=q + 2) == 1 and call(out=out + 8) == 1 and call(last=last + 2) == 1 and call(ws=ws + 4) == 1
    big = rows * 4 * hd * e
    for base, n in ((q, big), (last, rows * 4), (c.k, 100 * w), (c.v, 100 * w), (c.own_k, 60 * w), (c.own_v, 60 * w)):
        for p in (base, base + (n - 1) // 16 * 16):
            assert refused(lib, call(out=p)) and refused(lib, call(ws=p))
        assert refused(lib, call(out=base - big + 16))
    assert refused(lib, call(out=ws + (need - 1) // 16 * 16)) and refused(lib, call(ws=out + big - 16))


# ---- sampling ----------------------------------------------------------------------------------
def test_sample_token_refuses_bad_arguments(lib):
    n, V = 3, 100
    at = dict(temperature=1 << 30, top_k=1 << 31, top_p=1 << 32, min_p=1 << 33)
    logits, u, tok, lp, kept = 1 << 34, 1 << 35, 1 << 36, 1 << 37, 1 << 38

    def call(n=n, V=V, dt=B.CB_F32, logits=logits, u=u, tok=tok, lp=lp, kept=kept, rules=True, **kw):
        r = B.cb_sample_rules(**{**at, **kw})
        return lib.cb_sample_token(logits, n, V, dt, u, C.byref(r) if rules else None, tok, lp, kept, None)

    assert call(dt=2) == 3 and call(n=-1) == 2 and call(n=65536) == 2 and call(V=0) == 2 and call(V=(1 << 20) + 1) == 8
    assert call(rules=False) == 1 and call(n=0) == 0 and call(logits=None) == 1 and call(u=None) == 1 and call(tok=None) == 1
    assert call(logits=logits + 4) == 1 and call(u=u + 2) == 1 and call(tok=tok + 1) == 1 and call(top_k=at["top_k"] + 2) == 1
    outs = dict(tok=tok, lp=lp, kept=kept)
    for o in outs:
        for base, size in [(logits, n * V * 4), (u, 12)] + [(v, 12) for v in at.values()] + [(outs[x], 12) for x in outs if x != o]:
            for p in (base, base + size - 4, base - 8):
                assert refused(lib, call(**{o: p})), (o, p - base)


# ---- the binding's checks, with stand-ins for torch's device and tensors -------------------------
class Tensor:
    def __init__(self, dtype, *shape, dev=0, stride=None, at=1 << 20):
        self.dtype, self.shape, self.dev, self.device, self.at = dtype, shape, dev, f"cuda:{dev}", at
        s, st = [], 1
        for x in reversed(shape):
            s.insert(0, st)
            st *= x
        self._stride = tuple(stride or s)
        self.whole = stride is None

    def numel(self):
        n = 1
        for x in self.shape:
            n *= x
        return n

    def element_size(self):
        return self.dtype.itemsize

    def dim(self):
        return len(self.shape)

    def stride(self, i=None):
        return self._stride if i is None else self._stride[i]

    def is_contiguous(self):
        return self.whole

    def get_device(self):
        return self.dev

    def data_ptr(self):
        return self.at


@pytest.fixture
def fake(monkeypatch):
    torch = pytest.importorskip("torch")

    class Fake(B._Torch):
        dev = 0

        def device(self):
            return self.dev

        def stream(self, stream, dev):
            return None

    f = Fake()
    f.t = torch
    monkeypatch.setattr(B, "_TORCH", f)
    return f


def test_the_binding_refuses_tensors_of_another_kind(lib, fake):
    t = fake.t
    bf, f32, i32 = t.bfloat16, t.float32, t.int32
    d, spec = _dims(), B.rope_spec(1, 64, 1e4)
    ok = dict(q=Tensor(bf, N, QW), k=Tensor(bf, N, W), v=Tensor(bf, N, W), pos=Tensor(i32, N), q_out=Tensor(bf, N, QW),
              k_out=Tensor(bf, N, W), v_out=Tensor(bf, N, W), cos_sin=Tensor(f32, 100 * 64))

    def rows(**kw):
        a = {**ok, **kw}
        return B.cb_rope_rows(a["q"], a["k"], a["v"], a["pos"], a["q_out"], a["k_out"], a["v_out"], d, spec, a["cos_sin"], 100,
                              src_row=a.get("src_row"), kv_row=a.get("kv_row"))

    with pytest.raises(B.CBError, match="overlaps"):
        rows()                                                  # all at one address: that far it gets
    for kw in (dict(q=Tensor(f32, N, QW)), dict(q=Tensor(bf, N - 1, QW)), dict(q=Tensor(bf, N, QW + 1)), dict(q=Tensor(bf, N, QW, dev=1)),
               dict(q_out=Tensor(bf, N, QW, stride=(QW * 2, 2))), dict(q=Tensor(bf, N, QW, stride=(0, 1))),
               dict(k_out=Tensor(bf, N, W, stride=(W - 8, 1))), dict(v=Tensor(bf, N + 1, W)), dict(v_out=Tensor(bf, N + 1, W)),
               dict(v_out=Tensor(bf, N, W, stride=(W * 2, 1))), dict(pos=Tensor(t.int64, N)), dict(cos_sin=Tensor(f32, 100 * 64 - 1)),
               dict(src_row=Tensor(i32, N + 1)), dict(kv_row=Tensor(i32, N, dev=1)), dict(k=Tensor(bf, N * W)), dict(k=Tensor(bf, 1, N, W))):
        with pytest.raises((ValueError, IndexError)):
            rows(**kw)
    own = lambda **k: Tensor(bf, 3, 20, W, **k)  # noqa: E731
    pre = Tensor(bf, 100, W)
    make = lambda k=pre, v=pre, r=(0,), n=(100,), s=(0, 3), a=None, b=None: B.shared_kv(k, v, r, n, s, a, b)  # noqa: E731
    c = make(a=own(), b=own())
    for kw in (dict(v=None), dict(k=None, v=None), dict(a=own()), dict(n=(1, 2)), dict(s=(0,)), dict(v=Tensor(bf, 99, W)),
               dict(a=own(), b=Tensor(bf, 3, 19, W)), dict(a=Tensor(bf, 2, 20, W), b=Tensor(bf, 2, 20, W)),
               dict(a=Tensor(bf, 3, 20, W + 2), b=Tensor(bf, 3, 20, W + 2)), dict(a=Tensor(f32, 3, 20, W), b=Tensor(f32, 3, 20, W)),
               dict(k=Tensor(bf, 100, W, dev=1), v=Tensor(bf, 100, W, dev=1))):
        with pytest.raises(ValueError):
            make(**kw)
    q, last, o, ws = Tensor(bf, 3, 1, QW), Tensor(i32, 3, 1), Tensor(bf, 3, 1, QW), Tensor(t.uint8, 1 << 20)
    call = lambda q=q, last=last, o=o, c=c, d=d: B.cb_shared_attention(q, last, 1, c, d, o, ws)  # noqa: E731
    for kw in (dict(q=Tensor(f32, 3, 1, QW)), dict(last=Tensor(i32, 2, 1)), dict(o=Tensor(bf, 3, 2, QW)), dict(d=_dims(dtype=B.CB_F32)),
               dict(d=_dims(head_dim=32, d_model=128))):
        with pytest.raises(ValueError):
            call(**kw)
    r = B.sample_rules(temperature=Tensor(f32, 4), top_k=Tensor(i32, 4))
    x = Tensor(bf, 4, 100)
    for kw in (dict(x=Tensor(bf, 3, 100)), dict(x=Tensor(t.float16, 4, 100)), dict(u=Tensor(f32, 3)), dict(tok=Tensor(t.int64, 4))):
        a = dict(x=x, u=Tensor(f32, 4), tok=Tensor(i32, 4), **{})
        a.update(kw)
        with pytest.raises(ValueError):
            B.cb_sample_token(a["x"], a["u"], r, a["tok"])
    with pytest.raises(ValueError):
        B.sample_rules(temperature=Tensor(f32, 4), top_p=Tensor(f32, 5))
    fake.dev = 1
    for f in (call, lambda: B.cb_sample_token(x, Tensor(f32, 4, dev=1), r, Tensor(i32, 4, dev=1))):
        with pytest.raises(ValueError):
            f()
