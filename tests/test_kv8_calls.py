"""What the calls of the 8-bit cache and the logit rules take and refuse, on the host (no GPU is
touched: every call here is refused before anything is launched)."""
import ctypes

import pytest

from non_prefix_kv_gb300 import binding as B
from non_prefix_kv_gb300 import build as nb

FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    nb.build()
    return B.lib()


def _dims(**kw):
    base = dict(d_model=256, n_heads=4, n_kv_heads=2, head_dim=64, d_ff=512, vocab=1024, rope_base=1e4,
                rms_eps=1e-5, dtype=B.CB_BF16)
    base.update(kw)
    return B.cb_dims(**base)


def _cache(**kw):
    base = dict(k_codes=1 << 40, v_codes=1 << 42, k_scale=1 << 44, v_scale=1 << 45, capacity=256, n_seq=2, block=32)
    base.update(kw)
    return B.cb_kv8_cache(**base)


def attention_status(lib, d, c, n_q, weights=None):
    """Of a call without a workspace: 4 where only that is wrong with it."""
    return lib.cb_kv8_attention(1 << 46, 1 << 47, n_q, ctypes.byref(c), ctypes.byref(d), 1 << 48, weights, None, 0, None)


@pytest.mark.parametrize("kw,n_seq,cap,n_q,weights,ok", [
    # beyond 2^31 steps of the few-row kernels, but on the tensor cores
    (dict(n_heads=32, n_kv_heads=32, head_dim=128), 1, 131072, 131072, False, True),
    (dict(n_heads=56, n_kv_heads=8, head_dim=128), 32, 16384, 16384, False, True),
    (dict(n_heads=56, n_kv_heads=8, head_dim=128), 32, 16384, 16384, True, True),
    (dict(n_heads=56, n_kv_heads=8, head_dim=128, dtype=B.CB_F32), 32, 16384, 16384, True, True),
    # the same on the few-row kernels
    (dict(n_heads=32, n_kv_heads=32, head_dim=256), 1, 131072, 131072, False, False),
    (dict(n_heads=32, n_kv_heads=32, head_dim=32), 1, 131072, 131072, True, False),
    (dict(n_heads=8, n_kv_heads=8, head_dim=128), 65535, 131072, 1, False, False),
    (dict(n_heads=8, n_kv_heads=8, head_dim=128), 65535, 1024, 1, True, True),
    # no kernel at all
    (dict(n_heads=4, n_kv_heads=2, head_dim=96), 1, 256, 1, False, False),
    (dict(n_heads=128, n_kv_heads=1, head_dim=128), 1, 256, (1 << 20) + 1, False, False)])
def test_the_workspace_query_refuses_what_the_call_refuses(lib, kw, n_seq, cap, n_q, weights, ok):
    d, c = _dims(**kw), _cache(n_seq=n_seq, capacity=cap)
    w = 1 << 50 if weights else None
    assert attention_status(lib, d, c, n_q, w) == (4 if ok else 8)
    if ok:
        assert B.cb_kv8_workspace_bytes(d, n_seq, cap, n_q, weights) > 0
    else:
        with pytest.raises(B.CBError) as e:
            B.cb_kv8_workspace_bytes(d, n_seq, cap, n_q, weights)
        assert e.value.status == 8


def test_what_a_workspace_for_several_query_counts_has_to_hold(lib):
    """As the header says: not monotone in n_q (its figures), but in capacity and sequences; with the
    weights at least what it is without."""
    d = _dims(n_heads=32, n_kv_heads=32, head_dim=128)
    ask = lambda n, cap=4096, ns=1, w=False, dd=d: B.cb_kv8_workspace_bytes(dd, ns, cap, n, w)  # noqa: E731
    assert [round(ask(n) / 1e6, 1) for n in (1, 24, 25, 128, 129)] == [2.4, 17.4, 0, 0, 67.1]
    for dt in (B.CB_BF16, B.CB_F32):
        for hd in (32, 64, 128, 256):
            dd = _dims(n_heads=8, n_kv_heads=2, head_dim=hd, dtype=dt)
            for n in (1, 2, 3, 5, 12, 13, 32, 33, 100, 1000):
                assert ask(n, w=True, dd=dd) >= ask(n, dd=dd)
                for w in (False, True):
                    assert ask(n, 4112, 1, w, dd) >= ask(n, 4096, 1, w, dd) and ask(n, 4096, 3, w, dd) >= ask(n, 4096, 2, w, dd)
    # the expanded codes: 2 bytes for each of K's and V's
    assert 0 <= ask(129) - 2 * 2 * 32 * 4096 * 128 < 4096


def test_evict_refuses_outputs_that_overlap(lib):
    """Every output against every input and every other output, by a few bytes or by all."""
    d = _dims()
    src, dst = _cache(), _cache(k_codes=1 << 50, v_codes=1 << 51, k_scale=1 << 52, v_scale=1 << 53, capacity=128)
    heads, n_keep = 2 * 2, 100
    at = dict(len=1 << 30, weights=1 << 31, dst_len=1 << 32, dst_weights=1 << 33, kept=1 << 34)
    size = dict(len=8, weights=heads * 256 * 4, dst_len=8, dst_weights=heads * 128 * 4, kept=heads * n_keep * 4)

    def status(**kw):
        a = {**at, **kw}
        return lib.cb_kv8_evict(ctypes.byref(src), a["len"], a["weights"], n_keep, 1, 2, ctypes.byref(dst), a["dst_len"],
                                a["dst_weights"], a["kept"], ctypes.byref(d), None)

    arrays = [(at[k], size[k], k) for k in at]
    arrays += [(src.k_codes, 2 * 2 * 256 * 64, ""), (src.v_scale, heads * 8 * 4, ""), (dst.v_codes, 2 * 2 * 128 * 64, ""),
               (dst.k_scale, heads * 4 * 4, "")]
    for out in ("dst_len", "dst_weights", "kept"):
        for base, n, name in arrays:
            if name == out:
                continue
            for p in (base, base + (n - 1) // 16 * 16, base - (size[out] - 1) // 16 * 16):
                assert status(**{out: p}) == 1, (out, name, p - base)
                assert b"overlaps" in lib.cb_last_error_message()


def test_append_read_and_attention_refuse_what_they_write_over_another_argument(lib):
    d, c, r = _dims(), _cache(), ctypes.byref
    codes, scales = 2 * 2 * 256 * 64, 2 * 2 * 8 * 4
    cache = [(c.k_codes, codes), (c.v_codes, codes), (c.k_scale, scales), (c.v_scale, scales)]
    k, v, start, count, n = 1 << 30, 1 << 31, 1 << 32, 1 << 33, 5
    rows = 2 * n * 2 * 64 * 2                                  # bytes of k or v
    append = lambda k=k, v=v, start=start, count=count, cc=c: lib.cb_kv8_append(k, v, n, start, count, r(cc), r(d), None)  # noqa: E731
    read = lambda k=k, v=v, start=start, count=count: lib.cb_kv8_read(r(c), start, count, n, r(d), k, v, None)  # noqa: E731

    def refused(status):
        return status == 1 and b"overlaps" in lib.cb_last_error_message()

    for base, size in cache:
        for p in (base, base + size - 16, base - 16):
            assert refused(append(k=p)) and refused(append(v=p)) and refused(read(k=p)) and refused(read(v=p))
        assert refused(append(start=base)) and refused(append(count=base + size - 4))
    assert refused(append(cc=_cache(v_codes=c.k_codes + codes - 16))) and refused(append(cc=_cache(k_scale=c.v_scale)))
    assert refused(read(k=k, v=k + rows - 16)) and refused(read(start=k)) and refused(read(count=v + rows - 4))
    # attention
    q, last, out, w, ws = 1 << 30, 1 << 31, 1 << 32, 1 << 33, 1 << 34
    need = B.cb_kv8_workspace_bytes(d, 2, 256, 4, True)
    row, acc = 2 * 4 * 4 * 64 * 2, 2 * 2 * 256 * 4

    def att(q=q, last=last, out=out, w=w, ws=ws):
        return lib.cb_kv8_attention(q, last, 4, r(c), r(d), out, w, ws, need, None)

    for base, size in cache + [(q, row), (last, 32)]:
        for p in (base, base + (size - 1) // 16 * 16):
            assert refused(att(out=p)) and refused(att(w=p)) and refused(att(ws=p))
    assert refused(att(out=w + acc - 16)) and refused(att(w=ws + need - need % 16 - 16)) and refused(att(ws=out - 16))


# ---- the binding's checks, with stand-ins for torch's device and tensors ----------------------
class Tensor:
    def __init__(self, dtype, *shape, dev=0):
        self.dtype, self.shape, self.dev, self.device = dtype, shape, dev, f"cuda:{dev}"

    def numel(self):
        n = 1
        for x in self.shape:
            n *= x
        return n

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.dev

    def data_ptr(self):
        return FAKE


@pytest.fixture
def fake(monkeypatch):
    """The current device as the binding sees it: fake.dev."""
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


def handle(t, dev=0, **kw):
    a = dict(k=(2, 3, 64, 64), v=(2, 3, 64, 64), ks=(2, 3, 4), vs=(2, 3, 4))
    a.update(kw)
    return B.kv8_cache(Tensor(t.int8, *a["k"], dev=dev), Tensor(t.int8, *a["v"], dev=dev),
                       Tensor(t.float32, *a["ks"], dev=dev), Tensor(t.float32, *a["vs"], dev=dev), 16)


def test_a_cache_is_made_of_tensors_of_the_right_shapes(fake):
    t = fake.t
    c = handle(t)
    assert (c.n_seq, c.capacity, c.block, c.hkv, c.hd) == (2, 64, 16, 3, 64)
    for kw in (dict(ks=(2, 4, 3)), dict(vs=(2, 4, 3)), dict(ks=(24,)), dict(v=(2, 64, 3, 64)), dict(v=(2, 3, 32, 128)),
               dict(ks=(3, 2, 4))):
        with pytest.raises(ValueError, match="shape"):
            handle(t, **kw)
    with pytest.raises(ValueError, match="multiple of block"):
        handle(t, k=(2, 3, 72, 64), v=(2, 3, 72, 64))


def test_a_handle_is_refused_on_another_device(fake):
    """The other arguments may well be on the current device: the handle's memory is not."""
    t, d = fake.t, _dims(n_heads=6, n_kv_heads=3, head_dim=64)
    fake.dev = 1
    c, c2 = handle(t, dev=1), handle(t, dev=1)
    rules = B.logit_rules(mask=Tensor(t.int32, 2, 4, dev=1))
    fake.dev = 0
    row = lambda *shape, dt=t.bfloat16: Tensor(dt, *shape)  # noqa: E731
    i32 = lambda n: Tensor(t.int32, n)  # noqa: E731
    calls = [lambda: B.cb_kv8_append(row(2, 5, 192), row(2, 5, 192), 5, i32(2), None, c, d),
             lambda: B.cb_kv8_read(c, i32(2), None, 5, d, row(2, 5, 192), None),
             lambda: B.cb_kv8_attention(row(2, 1, 384), i32(2), 1, c, d, row(2, 1, 384)),
             lambda: B.cb_kv8_evict(c, i32(2), row(2, 3, 64, dt=t.float32), 8, 0, 0, c2, i32(2), None, i32(48), d),
             lambda: B.cb_logits_process(row(2, 128, dt=t.float32), rules, None, i32(2))]
    for call in calls:
        with pytest.raises(ValueError, match="current CUDA device"):
            call()
