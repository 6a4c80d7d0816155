"""Pins of the fp64 oracle of the 8-bit block-scaled cache, its attention, eviction and the
logit rules, and the host-side checks of their entry points (no GPU is touched)."""
import ctypes

import numpy as np
import pytest

import oracle.kv8_oracle as K8
from non_prefix_kv_gb300 import binding as B
from non_prefix_kv_gb300 import build as nb


def test_scale_one_keeps_integers_and_half_goes_to_even():
    c = K8.empty(1, 1, 16, 4, 16)
    x = np.array([[127.0, 0.5, 1.5, -2.5], [3.0, -4.0, 126.5, -0.5]]).reshape(1, 2, 1, 4)
    K8.append(c, x, x, [0])
    assert c["ks"][0, 0, 0] == 1.0
    np.testing.assert_array_equal(c["k"][0, 0, :2], [[127, 0, 2, -2], [3, -4, 126, 0]])


def test_round_trip_is_within_half_a_step():
    g = np.random.default_rng(0)
    c = K8.empty(2, 3, 64, 32, 16)
    x = g.standard_normal((2, 50, 3, 32)).astype(np.float32)
    K8.append(c, x, 2 * x, [0, 7])
    for s, a in ((0, 0), (1, 7)):
        n = min(50, 64 - a)
        v = K8.values(c["k"], c["ks"], 16)[s, :, a:a + n]
        step = np.repeat(c["ks"][s], 16, axis=1)[:, a:a + n, None]
        assert np.all(np.abs(v - x[s, :n].transpose(1, 0, 2)) <= step * (0.5 + 1e-6))


def test_appending_row_by_row_keeps_older_rows_within_one_and_a_half_steps():
    g = np.random.default_rng(1)
    x = g.standard_normal((1, 32, 1, 16)) * np.linspace(0.1, 3, 32)[None, :, None, None]
    a, b = K8.empty(1, 1, 32, 16, 32), K8.empty(1, 1, 32, 16, 32)
    K8.append(a, x, x, [0])
    for i in range(32):
        K8.append(b, x[:, i:i + 1], x[:, i:i + 1], [i])
    assert a["ks"][0, 0, 0] == b["ks"][0, 0, 0]          # the largest value decides both
    grown = np.abs(a["k"] - b["k"]).max()
    assert grown <= 32                                   # at most half a step per growth
    np.testing.assert_array_equal(a["k"][0, 0, 31], b["k"][0, 0, 31])


def test_attention_of_a_zero_query_is_the_mean_and_of_one_key_its_value():
    g = np.random.default_rng(2)
    c = K8.empty(1, 2, 32, 8, 16)
    x = g.standard_normal((1, 20, 2, 8))
    K8.append(c, x, -x, [0])
    V = K8.values(c["v"], c["vs"], 16)
    out, w, _, _, _ = K8.attention(c, np.zeros((1, 3, 4, 8)), np.array([[19, 0, -1]]))
    for h in range(4):
        np.testing.assert_allclose(out[0, 0, h], V[0, h // 2, :20].mean(0), atol=1e-12)
        np.testing.assert_allclose(out[0, 1, h], V[0, h // 2, 0], atol=1e-12)
        assert np.all(out[0, 2, h] == 0)
    np.testing.assert_allclose(w.sum(), 2 * 4, atol=1e-12)     # one per query that sees a row and head
    np.testing.assert_allclose(w[0, 0, 0], 2 * (1 / 20 + 1))


def test_evict_keeps_the_ends_and_the_heaviest_with_ties_to_the_lower_row():
    c = K8.empty(1, 1, 16, 4, 16)
    x = np.arange(10, dtype=np.float64).reshape(1, 10, 1, 1) * np.ones((1, 1, 1, 4))
    K8.append(c, x, x, [0])
    w = np.zeros((1, 1, 16), np.float32)
    w[0, 0, :10] = [9, 1, 2, 2, 2, 0, 2, 3, 0, 0]
    d, dl, dw, kept = K8.evict(c, [10], w, 6, 1, 2, 16)
    np.testing.assert_array_equal(kept[0, 0], [0, 2, 3, 7, 8, 9])
    np.testing.assert_array_equal(dw[0, 0, :6], [9, 2, 2, 3, 0, 0])
    assert dl[0] == 6
    np.testing.assert_array_equal(d["k"][0, 0, :6, 0], [0, 28, 42, 99, 113, 127])      # rows worth 0, 2, 3, 7, 8, 9
    d, dl, dw, kept = K8.evict(c, [4], w, 6, 1, 2, 16)
    np.testing.assert_array_equal(kept[0, 0], [0, 1, 2, 3, -1, -1])


def test_logit_rules_by_hand():
    x = [2.0, -2.0, 1.0, 0.0, 5.0]
    y = K8.logits(x, history=[0, 1, 2, 2, 0], prompt_len=2, repetition=2.0, presence=0.5, frequency=0.25,
                  bias=[(3, 1.0), (3, 0.5), (-1, 9.0)], mask=np.array([1, 1, 1, 1, 0], bool))
    np.testing.assert_allclose(y, [1 - 0.25 - 0.5, -4.0, 0.5 - 2 * 0.25 - 0.5, 1.5, -np.inf])
    assert K8.token(y) == 3
    assert K8.token(np.array([np.nan, 1.0, 1.0])) == 1
    assert K8.token(np.array([-np.inf, np.nan])) == -1


# ---- refusals (status before any launch) ---------------------------------------------------
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
    base = dict(k_codes=FAKE, v_codes=FAKE << 8, k_scale=FAKE << 16, v_scale=FAKE << 17, capacity=256, n_seq=2, block=32)
    base.update(kw)
    return B.cb_kv8_cache(**base)


BAD_CACHES = [(dict(k_codes=None), 1), (dict(v_scale=None), 1), (dict(k_codes=FAKE + 8), 1), (dict(v_scale=FAKE + 4), 1),
              (dict(block=48), 8), (dict(block=0), 8), (dict(block=256), 8), (dict(n_seq=0), 2), (dict(n_seq=65536), 2),
              (dict(capacity=0), 2), (dict(capacity=250), 2), (dict(capacity=1 << 31), 2)]


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_every_call_refuses_a_bad_cache(lib, bad, status):
    d, c, ok = _dims(), _cache(**bad), _cache(k_codes=FAKE << 9, v_codes=FAKE << 10, k_scale=FAKE << 18, v_scale=FAKE << 19)
    r = ctypes.byref
    assert lib.cb_kv8_append(FAKE, FAKE, 1, FAKE, None, r(c), r(d), None) == status
    assert lib.cb_kv8_read(r(c), FAKE, None, 1, r(d), FAKE, FAKE, None) == status
    assert lib.cb_kv8_attention(FAKE, FAKE, 1, r(c), r(d), FAKE, None, None, 0, None) == status
    assert lib.cb_kv8_evict(r(c), FAKE, FAKE, 8, 0, 0, r(ok), FAKE + 64, None, FAKE, r(d), None) == status
    assert lib.cb_kv8_evict(r(ok), FAKE, FAKE, 8, 0, 0, r(c), FAKE + 64, None, FAKE, r(d), None) == status


def test_kv8_calls_refuse_bad_arguments(lib):
    d, c, r = _dims(), _cache(), ctypes.byref
    assert lib.cb_kv8_append(None, FAKE, 1, FAKE, None, r(c), r(d), None) == 1
    assert lib.cb_kv8_append(FAKE, FAKE, 1, None, None, r(c), r(d), None) == 1
    assert lib.cb_kv8_append(FAKE + 8, FAKE, 1, FAKE, None, r(c), r(d), None) == 1
    assert lib.cb_kv8_append(FAKE, FAKE, -1, FAKE, None, r(c), r(d), None) == 2
    assert lib.cb_kv8_append(FAKE, FAKE, 257, FAKE, None, r(c), r(d), None) == 2
    assert lib.cb_kv8_append(FAKE, FAKE, 0, FAKE, None, r(c), r(d), None) == 0        # nothing to do
    assert lib.cb_kv8_append(FAKE, FAKE, 1, FAKE, None, None, r(d), None) == 1
    assert lib.cb_kv8_append(FAKE, FAKE, 1, FAKE, None, r(c), r(_dims(dtype=5)), None) == 3
    assert lib.cb_kv8_read(r(c), None, None, 1, r(d), FAKE, FAKE, None) == 1
    assert lib.cb_kv8_read(r(c), FAKE, None, -1, r(d), FAKE, FAKE, None) == 2
    assert lib.cb_kv8_read(r(c), FAKE, None, 1, r(d), FAKE + 4, FAKE, None) == 1
    assert lib.cb_kv8_read(r(c), FAKE, None, 1, r(d), None, None, None) == 0
    att = lambda dd=d, n_q=1, w=None, ws=None, n=0, q=FAKE, last=FAKE, out=FAKE: lib.cb_kv8_attention(  # noqa: E731
        q, last, n_q, r(c), r(dd), out, w, ws, n, None)
    assert att(_dims(head_dim=96)) == 8 and att(_dims(head_dim=160)) == 8
    assert att(n_q=-1) == 2 and att(n_q=0) == 0 and att(n_q=1 << 28) == 8
    assert att(q=None) == 1 and att(last=None) == 1 and att(out=None) == 1 and att(q=FAKE + 8) == 1
    need = B.cb_kv8_workspace_bytes(d, 2, 256, 1, True)
    assert need > 0 and B.cb_kv8_workspace_bytes(d, 2, 256, 1, False) <= need
    assert att(w=FAKE) == 4 and att(w=FAKE, ws=FAKE, n=need - 1) == 4 and att(w=FAKE, ws=FAKE + 8, n=need) == 1
    with pytest.raises(B.CBError):
        B.cb_kv8_workspace_bytes(d, 0, 256, 1, True)


def test_attention_refuses_an_output_over_its_queries_and_sizes_past_the_counters(lib):
    d, c, r = _dims(), _cache(), ctypes.byref
    need = B.cb_kv8_workspace_bytes(d, 2, 256, 4, True)
    row = 2 * 4 * d.n_heads * d.head_dim * 2
    for out in (FAKE, FAKE + 16, FAKE + row - 16, FAKE - row + 16):          # two sequences of 4 bf16 rows
        assert lib.cb_kv8_attention(FAKE, FAKE, 4, r(c), r(d), out, None, FAKE, need, None) == 1
        assert b"overlaps" in lib.cb_last_error_message()
    for args in ((65536, 256, 1), (1, (1 << 30) + 1, 1), (1, 256, (1 << 31) - 1)):
        with pytest.raises(B.CBError):
            B.cb_kv8_workspace_bytes(d, *args)


def test_evict_refuses_bad_arguments(lib):
    d, r = _dims(), ctypes.byref
    src = _cache()
    dst = lambda **kw: _cache(**{**dict(k_codes=FAKE << 9, v_codes=FAKE << 10, k_scale=FAKE << 18, v_scale=FAKE << 19), **kw})  # noqa: E731
    ev = lambda t, keep=8, sink=1, rec=2, ln=FAKE, w=FAKE, dl=FAKE + 64, dw=None, kept=FAKE, s=src: lib.cb_kv8_evict(  # noqa: E731
        r(s), ln, w, keep, sink, rec, r(t), dl, dw, kept, r(d), None)
    assert ev(dst(block=64)) == 2 and ev(dst(n_seq=1)) == 2
    assert ev(dst(), keep=0) == 2 and ev(dst(), keep=257) == 2
    assert ev(dst(), sink=-1) == 2 and ev(dst(), rec=-1) == 2 and ev(dst(), sink=5, rec=4) == 2
    assert ev(dst(), sink=2 ** 31 - 1, rec=2 ** 31 - 1) == 2
    assert ev(dst(), ln=None) == 1 and ev(dst(), w=None) == 1 and ev(dst(), dl=None) == 1 and ev(dst(), kept=None) == 1
    assert ev(src) == 1 and b"share memory" in lib.cb_last_error_message()
    # one array of dst inside one of src (the codes of src: 2 x 2 x 256 x 64 bytes)
    assert ev(dst(k_codes=FAKE + 65520)) == 1 and ev(dst(v_scale=FAKE + 1024)) == 1
    assert ev(dst(), dl=FAKE) == 1 and ev(dst(), dw=FAKE) == 1


def test_logits_process_refuses_bad_arguments(lib):
    r = ctypes.byref
    rules = lambda **kw: B.cb_logit_rules(**kw)  # noqa: E731
    lp = lambda ru, n=2, v=100, dt=B.CB_F32, x=FAKE, out=FAKE, tok=FAKE: lib.cb_logits_process(x, n, v, dt, r(ru), out, tok, None)  # noqa: E731
    none = rules()
    assert lp(none, dt=3) == 3 and lp(none, n=-1) == 2 and lp(none, n=65536) == 2 and lp(none, v=0) == 2
    assert lp(none, v=2 ** 31 - 1) == 8
    assert lib.cb_logits_process(FAKE, 2, 100, 0, None, FAKE, FAKE, None) == 1
    assert lp(none, x=None) == 1 and lp(none, x=FAKE + 4) == 1 and lp(none, out=FAKE + 8) == 1
    assert lp(none, n=0) == 0 and lp(none, out=None, tok=None) == 0
    assert lp(none, out=FAKE + 16) == 1                            # overlaps without being the same
    assert lp(rules(history=FAKE, history_ld=5)) == 1              # no lengths
    assert lp(rules(history=FAKE, history_len=FAKE, history_ld=-1)) == 1
    assert lp(rules(history=FAKE, history_len=FAKE, history_ld=1 << 18)) == 8
    assert lp(rules(history_ld=4, repetition=FAKE)) == 1           # ids announced, none given
    assert lp(rules(n_bias=2)) == 1 and lp(rules(n_bias=-1)) == 2 and lp(rules(n_bias=4097, bias=FAKE, bias_id=FAKE)) == 2
    assert lp(rules(mask=FAKE, mask_ld=3)) == 2                    # 100 ids need 4 words


def test_binding_refuses_wrong_tensors():
    torch = pytest.importorskip("torch")
    k = torch.zeros(1, 2, 32, 64, dtype=torch.int8)
    s = torch.zeros(1, 2, 1)
    with pytest.raises(ValueError, match="current CUDA device"):
        B.kv8_cache(k, k.clone(), s, s.clone(), 32)
    with pytest.raises(ValueError, match="expected torch.int8"):
        B.kv8_cache(k.float(), k, s, s, 32)
    with pytest.raises(ValueError, match="not contiguous"):
        B.kv8_cache(k.transpose(1, 2), k, s, s, 32)
    with pytest.raises(ValueError, match="block"):
        B.kv8_cache(k, k, s, s, 48)
    with pytest.raises(ValueError, match="row count"):
        B.logit_rules(bias_id=torch.zeros(2, 1), bias=torch.zeros(3, 1))
    with pytest.raises(ValueError, match="need a history"):
        B.logit_rules(repetition=torch.zeros(2))
    with pytest.raises(ValueError, match="one shape"):
        B.logit_rules(bias=torch.zeros(2, 3))
