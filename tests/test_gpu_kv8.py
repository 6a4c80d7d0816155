"""The 8-bit block-scaled cache, attention over it, eviction and the logit rules against the
fp64 oracle.  Codes, scales, kept rows and tokens are compared exactly.

Tolerances of the attention, element by element, with A = sum_i p_i |v_i|:
  bf16: the output's rounding is 2^-8 of it; a weight is rounded to fp16 (2^-11);
  fp32: the output's rounding is 2^-24, a weight is two fp16 parts (2^-22);
  both: a score's products and sums are fp32, at most (hd + 4) 2^-24 of sum_c |q_c k_c| (plus,
  fp32 only, q as two fp16 parts: 2^-21), and the exponential turns that error of z into a
  relative one of the weight, once above and once below the fraction line; ex2 adds 2^-21;
  sums over n keys add n 2^-24.
  Where a channel's large weights meet codes of 0, fp16's smallest step shows: it is 2^-24
  (half of it per rounding), the weights carry 2^8 at the largest p_i vs_i (vs: the scale of
  v_i) and a code is at most 127, so n keys add at most n 127 2^-33 max_i p_i vs_i.  A weight of the account has the same relative error without
  the rounding to fp16."""
import numpy as np
import pytest

import oracle.kv8_oracle as K8
from tests.gpu_util import dev, dev_i32, ensure_lib, host, tdt, torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    torch_mod()
    ensure_lib()
    from non_prefix_kv_gb300 import binding
    return binding


def make_dims(B, H, hkv, hd, dtype):
    return B.cb_dims(H * hd, H, hkv, hd, 256, 64, 1e4, 1e-5, B.CB_BF16 if dtype == "bf16" else B.CB_F32)


class Dev:
    """A device cache whose unused memory holds what a fresh allocation may: odd codes, NaN scales."""

    def __init__(self, B, n_seq, hkv, cap, hd, block):
        torch = torch_mod()
        mk = lambda: torch.full((n_seq, hkv, cap, hd), -77, dtype=torch.int8, device="cuda")  # noqa: E731
        sc = lambda: torch.full((n_seq, hkv, cap // block), float("nan"), device="cuda")  # noqa: E731
        self.k, self.v, self.ks, self.vs = mk(), mk(), sc(), sc()
        self.c = B.kv8_cache(self.k, self.v, self.ks, self.vs, block)


def rounded(x, dtype):
    """fp32 values as the device sees them."""
    torch = torch_mod()
    x = np.asarray(x, np.float32)
    return torch.from_numpy(x).to(torch.bfloat16).float().numpy() if dtype == "bf16" else x


def rows(g, n_seq, n, hkv, hd, dtype, std=1.0):
    x = g.standard_normal((n_seq, n, hkv, hd)) * std * g.uniform(0.2, 3, (n_seq, n, 1, 1))
    return rounded(x, dtype)


def check_cache(d, o, n):
    """Rows [0, n[s]) of the device cache against the oracle's, exactly; later ones untouched."""
    blk = o["block"]
    for dc, ds, oc, os_ in ((d.k, d.ks, o["k"], o["ks"]), (d.v, d.vs, o["v"], o["vs"])):
        dc, ds = dc.cpu().numpy().astype(np.int64), ds.cpu().numpy()
        for s, m in enumerate(n):
            nb = -(-m // blk)
            np.testing.assert_array_equal(ds[s, :, :nb], os_[s, :, :nb])
            assert np.all(np.isnan(ds[s, :, nb:]))
            np.testing.assert_array_equal(dc[s, :, :m], oc[s, :, :m])
            assert np.all(dc[s, :, m:] == -77)


def filled(B, g, n_seq, hkv, cap, hd, block, lens, dtype="bf16", std=1.0):
    """A device cache and its oracle twin holding lens[s] rows."""
    d, o = Dev(B, n_seq, hkv, cap, hd, block), K8.empty(n_seq, hkv, cap, hd, block)
    n = max(max(lens), 1)
    k, v = rows(g, n_seq, n, hkv, hd, dtype, std), rows(g, n_seq, n, hkv, hd, dtype)
    dims = make_dims(B, hkv, hkv, hd, dtype)
    B.cb_kv8_append(dev(k, dtype), dev(v, dtype), n, dev_i32([0] * n_seq), dev_i32(lens), d.c, dims)
    B.cb_sync(None)
    K8.append(o, k, v, [0] * n_seq, lens)
    return d, o


# ------------------------------------------------------------------------------ append, read
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hkv,hd,block", [(2, 128, 32), (3, 64, 16), (1, 32, 128), (2, 256, 64), (2, 96, 32),
                                          (1, 160, 16), (4, 128, 128)])
def test_append_is_the_oracles_code_for_code(B, dtype, hkv, hd, block):
    g = np.random.default_rng(hd + block)
    cap, n_seq = 3 * block, 5
    d, o = Dev(B, n_seq, hkv, cap, hd, block), K8.empty(n_seq, hkv, cap, hd, block)
    dims = make_dims(B, hkv, hkv, hd, dtype)
    held = np.zeros(n_seq, int)
    # ragged appends, one of them idle, the last one up to the capacity
    for step in range(7):
        n = [1, block + 3, 1, 5, 2, 1, cap][step]
        count = np.minimum(g.integers(0, n + 1, n_seq), cap - held)
        if step in (0, 2, 5):
            count = np.minimum(1, cap - held)
        if step == 6:
            count = cap - held
        start = held.copy()
        start[step % n_seq] = -1 if step != 6 else start[step % n_seq]
        x = rows(g, n_seq, n, hkv, hd, dtype, std=0.3 * (step + 1))
        y = rows(g, n_seq, n, hkv, hd, dtype, std=1e-9 if step == 1 else 2.0)
        B.cb_kv8_append(dev(x, dtype), dev(y, dtype), n, dev_i32(start), dev_i32(count), d.c, dims)
        K8.append(o, x, y, start, count)
        held += np.where(start >= 0, count, 0)
        B.cb_sync(None)
        check_cache(d, o, held)
    assert np.all(held == cap)


def test_append_ties_zeros_and_long_runs(B):
    """Quotients at exactly half a step (scale 1), zero blocks, one row at a time over a block."""
    hd, block = 64, 32
    d, o = Dev(B, 1, 1, 64, hd, block), K8.empty(1, 1, 64, hd, block)
    dims = make_dims(B, 1, 1, hd, "f32")
    x = np.zeros((1, 40, 1, hd), np.float32)
    x[0, 0, 0, :] = np.arange(hd) - 31.5
    x[0, 0, 0, 0] = 127.0
    x[0, 5, 0, :8] = [0.5, 1.5, 2.5, -0.5, -1.5, 63.5, 254.0, 3.0]       # doubles the scale: old halves become ties
    x[0, 6, 0, 0] = 5.0e-9
    for i in range(40):
        B.cb_kv8_append(dev(x[:, i:i + 1]), dev(-x[:, i:i + 1]), 1, dev_i32([i]), None, d.c, dims)
        K8.append(o, x[:, i:i + 1], -x[:, i:i + 1], [i])
    B.cb_sync(None)
    check_cache(d, o, [40])
    # quotients around every half step for odd scales: decided as in 64 bits
    g = np.random.default_rng(5)
    d2, o2 = Dev(B, 8, 1, 64, 256, 64), K8.empty(8, 1, 64, 256, 64)
    y = np.empty((8, 64, 1, 256), np.float32)
    for s in range(8):
        amax = np.float32(g.uniform(0.1, 50))
        sc = np.float64(np.float32(amax / np.float32(127)))
        half = ((g.integers(-126, 126, (64, 256)) + 0.5) * sc).astype(np.float32)
        y[s, :, 0] = np.nextafter(half, np.float32(np.inf) * g.choice([-1, 1], half.shape).astype(np.float32))
        y[s, 1::3, 0] = half[1::3]
        y[s, 0, 0, 0] = amax
    B.cb_kv8_append(dev(y), dev(-y), 64, dev_i32([0] * 8), None, d2.c, make_dims(B, 1, 1, 256, "f32"))
    B.cb_sync(None)
    K8.append(o2, y, -y, [0] * 8)
    check_cache(d2, o2, [64] * 8)


def test_append_reports_bad_rows_and_keeps_the_rest(B):
    g = np.random.default_rng(3)
    hkv, hd, block, cap = 2, 64, 16, 48
    dims = make_dims(B, hkv, hkv, hd, "f32")
    d, o = Dev(B, 4, hkv, cap, hd, block), K8.empty(4, hkv, cap, hd, block)
    x = rows(g, 4, 40, hkv, hd, "f32")
    x[1, 3, 0, 5], x[1, 4, 1, 7], x[2, 0, 0, 0] = np.nan, np.inf, -np.inf
    B.cb_kv8_append(dev(x), dev(x), 40, dev_i32([0, 0, 0, -1]), None, d.c, dims)
    with pytest.raises(B.CBError) as e:
        B.cb_sync(None)
    assert e.value.status == 5
    K8.append(o, x, x, [0, 0, 0, -1])
    check_cache(d, o, [40, 40, 40, 0])
    # past the capacity; a start below -1; counts outside [0, n]
    x = rows(g, 4, 10, hkv, hd, "f32")
    B.cb_kv8_append(dev(x), dev(x), 10, dev_i32([40, -2, 40, 0]), dev_i32([10, 5, -3, 99]), d.c, dims)
    with pytest.raises(B.CBError) as e:
        B.cb_sync(None)
    assert e.value.status == 9
    K8.append(o, x, x, [40, -1, 40, 0], [8, 0, 0, 10])
    check_cache(d, o, [48, 40, 40, 10])
    for start in (48, 2 ** 31 - 1):       # nothing fits
        B.cb_kv8_append(dev(x), dev(x), 10, dev_i32([start, -1, -1, -1]), None, d.c, dims)
        with pytest.raises(B.CBError) as e:
            B.cb_sync(None)
        assert e.value.status == 9
        check_cache(d, o, [48, 40, 40, 10])
    B.cb_sync(None)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hkv,hd", [(3, 64), (2, 160)])
def test_read_returns_the_values_and_leaves_the_rest(B, dtype, hkv, hd):
    torch = torch_mod()
    g = np.random.default_rng(4)
    lens = [64, 33, 0]
    d, o = filled(B, g, 3, hkv, 64, hd, 32, lens)
    dims = make_dims(B, hkv, hkv, hd, dtype)
    for start, count, n in (([0, 0, 0], lens, 64), ([17, 3, -1], [31, 30, 5], 40), ([63, 32, -1], None, 1)):
        outs = [torch.full((3, n, hkv * hd), 7.5, dtype=tdt(dtype), device="cuda") for _ in range(2)]
        B.cb_kv8_read(d.c, dev_i32(start), None if count is None else dev_i32(count), n, dims, *outs)
        only_v = torch.full_like(outs[1], 7.5)
        B.cb_kv8_read(d.c, dev_i32(start), None if count is None else dev_i32(count), n, dims, None, only_v)
        B.cb_sync(None)
        assert torch.equal(only_v, outs[1])
        for out, codes, scale in ((outs[0], o["k"], o["ks"]), (outs[1], o["v"], o["vs"])):
            val = K8.values(codes, scale, 32).astype(np.float32)      # codes times fp32 scales: one rounding
            for s in range(3):
                m = 0 if start[s] < 0 else (n if count is None else count[s])
                ref = val[s, :, start[s]:start[s] + m].transpose(1, 0, 2).reshape(m, hkv * hd) if m else None
                got = out[s].float().cpu().numpy()
                if m:
                    np.testing.assert_array_equal(got[:m], rounded(ref, dtype))
                assert np.all(got[m:] == 7.5)
    out = torch.zeros(3, 10, hkv * hd, dtype=tdt(dtype), device="cuda")
    B.cb_kv8_read(d.c, dev_i32([60, -1, -1]), None, 10, dims, out, None)
    with pytest.raises(B.CBError) as e:
        B.cb_sync(None)
    assert e.value.status == 9
    assert torch.all(out[0, 4:] == 0) and torch.any(out[0, :4] != 0)


# ------------------------------------------------------------------------------ attention
def attend(B, d, q, last, dims, dtype, weights=None, stream=None):
    torch = torch_mod()
    n_seq, nq, H, hd = q.shape
    qd = dev(q, dtype)
    out = torch.full_like(qd, 7.5)
    n = B.cb_kv8_workspace_bytes(dims, n_seq, d.c.capacity, nq, weights is not None)
    ws = torch.full((max(n, 16),), 255, dtype=torch.uint8, device="cuda")     # NaN to a float read of it
    B.cb_kv8_attention(qd, dev_i32(last), nq, d.c, dims, out, weights, ws, stream=stream)
    return out


def check_attention(out, w_gain, ref, last, dtype, hd):
    o, w, mag, zmag, top = ref
    n = np.maximum(np.asarray(last) + 1, 0)[..., None, None]
    dz = (zmag * ((hd + 4) * 2.0 ** -24 + (2.0 ** -21 if dtype == "f32" else 0)))[..., None]
    rel = 2 * (dz + 2.0 ** -21) + n * 2.0 ** -24
    out = host(out)
    tol = ((2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) * np.abs(o)
           + mag * (rel + (2.0 ** -11 if dtype == "bf16" else 2.0 ** -22)) * 1.01
           + n * 127 * 2.0 ** -33 * top[..., None] + 1e-30)
    worst = np.max(np.abs(out - o) / tol)
    assert worst <= 1, worst
    if w_gain is not None:
        seen = w > 0
        # every p of the account carries at most the largest relative error
        assert np.all(np.abs(w_gain - w)[seen] <= w[seen] * (rel.max() + (o.shape[1] * o.shape[2] + 8) * 2.0 ** -24) + 1e-30)
        assert np.all(w_gain[~seen] == 0)
    return worst


CASES = [  # H, hkv, hd, block, cap, n_seq, n_q
    (4, 4, 128, 32, 224, 3, 1), (8, 2, 64, 16, 272, 2, 1), (7, 1, 128, 64, 1024, 2, 1), (56, 8, 128, 64, 512, 2, 1),
    (12, 1, 32, 128, 384, 2, 1), (4, 2, 256, 16, 176, 2, 1), (16, 1, 128, 16, 48, 1, 1), (3, 3, 64, 32, 4096, 1, 1),
    (4, 2, 128, 32, 160, 2, 5), (8, 2, 64, 64, 320, 1, 17), (7, 1, 128, 128, 640, 2, 40), (2, 2, 256, 32, 96, 1, 33),
    (20, 1, 32, 16, 112, 1, 3), (4, 4, 128, 64, 640, 1, 150), (14, 2, 128, 64, 704, 1, 100), (4, 2, 64, 16, 400, 2, 129),
]


@pytest.mark.parametrize("weigh", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,hkv,hd,block,cap,n_seq,n_q", CASES)
def test_attention(B, H, hkv, hd, block, cap, n_seq, n_q, dtype, weigh):
    torch = torch_mod()
    g = np.random.default_rng(H * hd + n_q)
    lens = [cap] + [int(x) for x in g.integers(1, cap + 1, n_seq - 1)]
    d, o = filled(B, g, n_seq, hkv, cap, hd, block, lens)
    q = rounded(g.standard_normal((n_seq, n_q, H, hd)) * 1.5, dtype)
    last = np.stack([g.integers(-1, n, n_q) for n in lens])
    last[0, 0] = lens[0] - 1
    if n_q > 3:
        last[0, 1:3] = [-1, 0]
        last[-1] = np.sort(last[-1])          # the order a blend's rows have
    dims = make_dims(B, H, hkv, hd, dtype)
    w = None
    if weigh:
        w0 = torch.from_numpy(g.uniform(0, 4, (n_seq, hkv, cap)).astype(np.float32)).cuda()
        w = torch.zeros(n_seq, hkv, cap, device="cuda")
        acc = w0.clone()
    out = attend(B, d, q, last, dims, dtype, w)
    if weigh:
        attend(B, d, q, last, dims, dtype, acc)
    B.cb_sync(None)
    check_attention(out, host(w) if weigh else None, K8.attention(o, q.astype(np.float64), last), last, dtype, hd)
    if weigh:       # added to what was there: the same sum, rounded once more
        assert torch.equal(acc, w0 + w)


@pytest.mark.parametrize("weigh", [False, True])
@pytest.mark.parametrize("H,hkv,hd,n_q", [
    (2, 2, 128, 8), (2, 2, 64, 9), (2, 2, 128, 16), (2, 2, 128, 17), (2, 1, 64, 20), (2, 2, 128, 40), (2, 2, 64, 41),
    (2, 2, 128, 41), (8, 1, 128, 5), (16, 1, 64, 1), (17, 1, 128, 1), (40, 1, 128, 1), (41, 1, 64, 1), (128, 1, 128, 1),
    (130, 1, 128, 1), (43, 1, 64, 3), (127, 1, 128, 2)])
def test_attention_where_the_paths_meet(B, H, hkv, hd, n_q, weigh):
    """Query rows per KV head around the counts at which another kernel takes over."""
    torch = torch_mod()
    g = np.random.default_rng(H + 1000 * n_q)
    cap, n_seq = 272, 2
    lens = [cap, 130]
    d, o = filled(B, g, n_seq, hkv, cap, hd, 16, lens)
    q = rounded(g.standard_normal((n_seq, n_q, H, hd)), "bf16")
    last = np.stack([g.integers(-1, n, n_q) for n in lens])
    last[:, -1] = [cap - 1, 127]
    w = torch.zeros(n_seq, hkv, cap, device="cuda") if weigh else None
    dims = make_dims(B, H, hkv, hd, "bf16")
    out = attend(B, d, q, last, dims, "bf16", w)
    B.cb_sync(None)
    check_attention(out, host(w) if weigh else None, K8.attention(o, q.astype(np.float64), last), last, "bf16", hd)
    if weigh:       # what serves a call with the weights serves one without
        n = B.cb_kv8_workspace_bytes(dims, n_seq, cap, n_q, True)
        assert n >= B.cb_kv8_workspace_bytes(dims, n_seq, cap, n_q, False)


@pytest.mark.parametrize("weigh", [False, True])
@pytest.mark.parametrize("H,hkv,hd,n_q", [(2, 2, 128, 16), (2, 2, 64, 17), (2, 2, 128, 17), (4, 1, 128, 12), (2, 2, 128, 49),
                                          (7, 1, 64, 7), (7, 1, 128, 40), (2, 1, 64, 150)])
def test_attention_in_fp32_where_the_paths_meet(B, H, hkv, hd, n_q, weigh):
    """As above; rows of very different magnitudes share a tile."""
    torch = torch_mod()
    g = np.random.default_rng(H + 1000 * n_q + hd)
    cap, n_seq = 272, 2
    lens = [cap, 130]
    d, o = filled(B, g, n_seq, hkv, cap, hd, 16, lens)
    q = (g.standard_normal((n_seq, n_q, H, hd)) * 10.0 ** g.integers(-6, 1, (n_seq, n_q, H, 1))).astype(np.float32)
    q[0, 0, 0] = 0
    last = np.stack([g.integers(-1, n, n_q) for n in lens])
    last[:, -1] = [cap - 1, 127]
    w = torch.zeros(n_seq, hkv, cap, device="cuda") if weigh else None
    out = attend(B, d, q, last, make_dims(B, H, hkv, hd, "f32"), "f32", w)
    B.cb_sync(None)
    check_attention(out, host(w) if weigh else None, K8.attention(o, q.astype(np.float64), last), last, "f32", hd)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_q", [1, 3, 130])
def test_attention_of_unlike_blocks(B, dtype, n_q):
    """Blocks whose V differ by up to 10^10 in size, K by 10^3; sharp and flat rows; large and tiny q."""
    torch = torch_mod()
    g = np.random.default_rng(8)
    H, hkv, hd, block, cap = 8, 2, 64, 16, 320
    d, o = Dev(B, 1, hkv, cap, hd, block), K8.empty(1, hkv, cap, hd, block)
    dims = make_dims(B, H, hkv, hd, dtype)
    k = g.standard_normal((1, cap, hkv, hd)) * np.repeat(10.0 ** g.uniform(-3, 0, cap // block), block)[None, :, None, None]
    v = g.standard_normal((1, cap, hkv, hd)) * np.repeat(10.0 ** g.uniform(-9, 2, cap // block), block)[None, :, None, None]
    v[0, 32:48] = 0
    k, v = rounded(k, "f32"), rounded(v, "f32")
    B.cb_kv8_append(dev(k), dev(v), cap, dev_i32([0]), None, d.c, make_dims(B, hkv, hkv, hd, "f32"))
    K8.append(o, k, v, [0])
    for size in (0.0, 1e-30, 1e-3, 1.0, 40.0):
        q = rounded(g.standard_normal((1, n_q, H, hd)) * size, dtype)
        q[0, 0, 1] *= 0
        last = g.integers(0, cap, (1, n_q))
        last[0, -1] = cap - 1
        w = torch.zeros(1, hkv, cap, device="cuda")
        out = attend(B, d, q, last, dims, dtype, w)
        B.cb_sync(None)
        ref = K8.attention(o, q.astype(np.float64), last)
        # weights of the account may be below fp32's range: an absolute floor of 2^-126
        wg, wr = host(w), ref[1]
        check_attention(out, None, ref, last, dtype, hd)
        dz = ref[3].max() * ((hd + 4) * 2.0 ** -24 + 2.0 ** -21)
        assert np.all(np.abs(wg - wr) <= wr * (2 * (dz + 2.0 ** -21) + (cap + n_q * H + 8) * 2.0 ** -24) + n_q * H * 2.0 ** -125)


def test_attention_is_the_same_from_run_to_run_and_per_sequence(B):
    torch = torch_mod()
    g = np.random.default_rng(9)
    H, hkv, hd, block, cap, n_seq = 8, 2, 128, 32, 512, 6
    lens = [512, 1, 31, 32, 33, 300]
    d, o = filled(B, g, n_seq, hkv, cap, hd, block, lens)
    dims = make_dims(B, H, hkv, hd, "bf16")
    for n_q in (1, 2, 40):
        q = rounded(g.standard_normal((n_seq, n_q, H, hd)), "bf16")
        last = np.array([[max(-1, n - n_q + j) for j in range(n_q)] for n in lens])
        ws = [torch.zeros(n_seq, hkv, cap, device="cuda") for _ in range(2)]
        a, b = (attend(B, d, q, last, dims, "bf16", w) for w in ws)
        B.cb_sync(None)
        assert torch.equal(a, b) and torch.equal(*ws)
        check_attention(a, host(ws[0]), K8.attention(o, q.astype(np.float64), last), last, "bf16", hd)
        # a query that sees nothing has a zero row
        assert torch.all(a[torch.from_numpy(last < 0).cuda()] == 0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_q", [1, 4, 11, 60])
def test_a_query_with_a_nan_spoils_only_its_own_rows(B, n_q, dtype):
    torch = torch_mod()
    g = np.random.default_rng(n_q)
    H, hkv, hd, cap, n_seq = 4, 2, 64, 288, 2
    d, o = filled(B, g, n_seq, hkv, cap, hd, 32, [cap, cap])
    q = rounded(g.standard_normal((n_seq, n_q, H, hd)), dtype)
    last = g.integers(100, cap, (n_seq, n_q))
    last[0, 0] = 90
    bad = q.copy()
    bad[0, 0, 3, 17] = np.nan                       # head 3: KV head 1
    w = torch.zeros(n_seq, hkv, cap, device="cuda")
    dims = make_dims(B, H, hkv, hd, dtype)
    out = attend(B, d, bad, last, dims, dtype, w)
    B.cb_sync(None)
    assert torch.all(torch.isnan(out[0, 0, 3])) and torch.all(torch.isnan(w[0, 1, :91]))
    out[0, 0, 3] = 0
    w[0, 1, :91] = 0
    q[0, 0, 3] = 0
    ref = list(K8.attention(o, q.astype(np.float64), last))
    ref[0][0, 0, 3] = 0
    ref[1][0, 1, :91] = 0
    check_attention(out, host(w), ref, last, dtype, hd)


@pytest.mark.parametrize("n_q", [1, 20, 70])
def test_attention_with_a_workspace_off_any_wider_boundary(B, n_q):
    """The header asks for 16 bytes."""
    torch = torch_mod()
    g = np.random.default_rng(n_q)
    H, hkv, hd, cap = 2, 2, 128, 160
    d, o = filled(B, g, 1, hkv, cap, hd, 16, [cap])
    q = rounded(g.standard_normal((1, n_q, H, hd)), "bf16")
    last = g.integers(0, cap, (1, n_q))
    dims = make_dims(B, H, hkv, hd, "bf16")
    n = B.cb_kv8_workspace_bytes(dims, 1, cap, n_q, True)
    whole = torch.full((n + 256,), 77, dtype=torch.uint8, device="cuda")
    off = -whole.data_ptr() % 256 + 16 if whole.data_ptr() % 256 else 16
    w, qd = torch.zeros(1, hkv, cap, device="cuda"), dev(q, "bf16")
    out = torch.empty_like(qd)
    B.cb_kv8_attention(qd, dev_i32(last), n_q, d.c, dims, out, w, whole[off:off + n])
    B.cb_sync(None)
    check_attention(out, host(w), K8.attention(o, q.astype(np.float64), last), last, "bf16", hd)
    assert torch.all(whole[:off] == 77) and torch.all(whole[off + n:] == 77)


@pytest.mark.parametrize("weigh", [False, True])
@pytest.mark.parametrize("n_seq", [1, 15, 17, 19, 22, 26, 34, 45, 80])
def test_attention_in_any_number_of_parts(B, n_seq, weigh):
    """The keys of a (sequence, KV head) are split over as many CTAs as run at once: 8 down to 1."""
    torch = torch_mod()
    g = np.random.default_rng(n_seq)
    H, hkv, hd, n_q, cap = 2, 1, 64, 13, 2064
    lens = [cap] + [int(x) for x in g.integers(1, cap + 1, n_seq - 1)]
    d, o = filled(B, g, n_seq, hkv, cap, hd, 16, lens)
    q = rounded(g.standard_normal((n_seq, n_q, H, hd)), "bf16")
    last = np.stack([g.integers(-1, n, n_q) for n in lens])
    last[:, 5] = np.array(lens) - 1
    w = torch.zeros(n_seq, hkv, cap, device="cuda") if weigh else None
    out = attend(B, d, q, last, make_dims(B, H, hkv, hd, "bf16"), "bf16", w)
    B.cb_sync(None)
    check_attention(out, host(w) if weigh else None, K8.attention(o, q.astype(np.float64), last), last, "bf16", hd)


def test_attention_without_a_workspace_where_none_is_asked_for(B):
    """One query tile of bf16 rows and no weights need none; a capacity that ends inside a key tile."""
    torch = torch_mod()
    g = np.random.default_rng(77)
    for H, hkv, hd, n_q, cap in ((2, 2, 128, 30, 16), (2, 2, 64, 128, 144), (14, 2, 128, 18, 1040)):
        dims = make_dims(B, H, hkv, hd, "bf16")
        assert B.cb_kv8_workspace_bytes(dims, 2, cap, n_q) == 0
        d, o = filled(B, g, 2, hkv, cap, hd, 16, [cap, cap - 1])
        q = rounded(g.standard_normal((2, n_q, H, hd)), "bf16")
        last = g.integers(-1, cap - 1, (2, n_q))
        last[1] = -1                                # a sequence without a row to see
        out = torch.full((2, n_q, H, hd), 7.5, dtype=torch.bfloat16, device="cuda")
        B.cb_kv8_attention(dev(q, "bf16"), dev_i32(last), n_q, d.c, dims, out)
        B.cb_sync(None)
        check_attention(out, None, K8.attention(o, q.astype(np.float64), last), last, "bf16", hd)
        assert torch.all(out[1] == 0)


def test_attention_reports_a_row_past_the_capacity(B):
    torch = torch_mod()
    g = np.random.default_rng(10)
    d, o = filled(B, g, 2, 2, 64, 64, 16, [64, 64])
    dims = make_dims(B, 4, 2, 64, "bf16")
    for n_q in (1, 20, 200):
        q = rounded(g.standard_normal((2, n_q, 4, 64)), "bf16")
        last = np.full((2, n_q), 63)
        last[0, 0], last[1, -1] = 64, -2
        w = torch.zeros(2, 2, 64, device="cuda")
        out = attend(B, d, q, last, dims, "bf16", w)
        with pytest.raises(B.CBError) as e:
            B.cb_sync(None)
        assert e.value.status == 9
        last[0, 0], last[1, -1] = -1, -1
        check_attention(out, host(w), K8.attention(o, q.astype(np.float64), last), last, "bf16", 64)
        assert torch.all(out[0, 0] == 0) and torch.all(out[1, -1] == 0)


def test_attention_over_a_long_cache(B):
    """Codes past 2^31 bytes from the cache's start, and many key tiles per CTA."""
    torch = torch_mod()
    hkv, hd, block, cap, n_seq = 2, 128, 128, 1 << 22, 3
    mk = lambda: torch.empty(n_seq, hkv, cap, hd, dtype=torch.int8, device="cuda")  # noqa: E731
    sc = lambda: torch.full((n_seq, hkv, cap // block), float("nan"), device="cuda")  # noqa: E731
    k, v, ks, vs = mk(), mk(), sc(), sc()
    c = B.kv8_cache(k, v, ks, vs, block)
    dims = make_dims(B, 2, 2, hd, "f32")
    # the last sequence: uniform keys, so every visible row weighs the same; values 1 except row 5's
    k[2].zero_()
    v[2].fill_(100)
    v[2, :, 5] = 50
    ks[2].fill_(1.0)
    vs[2].fill_(0.01)
    q = torch.randn(n_seq, 1, 2, hd, device="cuda")
    last = dev_i32([[-1], [-1], [cap - 1]])
    out = torch.empty_like(q)
    ws = torch.empty(B.cb_kv8_workspace_bytes(dims, n_seq, cap, 1), dtype=torch.uint8, device="cuda")
    B.cb_kv8_attention(q, last, 1, c, dims, out, None, ws)
    B.cb_sync(None)
    ref = 1.0 - 0.5 / cap
    # sums of 2^22 equal terms in fp32, joined tile by tile: at most 2^22 roundings of 2^-24
    assert torch.all((out[2] - ref).abs() < 0.25) and torch.all(out[:2] == 0)
    x = torch.randn(n_seq, 3, hkv * hd, device="cuda")
    B.cb_kv8_append(x, x, 3, dev_i32([-1, -1, cap - 3]), None, c, dims)
    back = torch.zeros_like(x)
    B.cb_kv8_read(c, dev_i32([-1, -1, cap - 3]), None, 3, dims, back, None)
    B.cb_sync(None)
    # half a step of the block's scale (127 steps to its largest value; 1.0 was there before)
    assert torch.all((back[2] - x[2]).abs() <= 0.51 * torch.maximum(x[2].abs().max() / 127, torch.ones((), device="cuda")))
    w = torch.rand(n_seq, hkv, cap, device="cuda")
    dst = Dev(B, n_seq, hkv, 256, hd, block)
    dl, kept = torch.zeros(n_seq, dtype=torch.int32, device="cuda"), torch.zeros(n_seq, hkv, 200, dtype=torch.int32, device="cuda")
    B.cb_kv8_evict(c, dev_i32([0, 0, cap]), w, 200, 4, 20, dst.c, dl, None, kept, dims)
    B.cb_sync(None)
    for h in range(hkv):
        best = torch.sort(w[2, h, 4:cap - 20], descending=True, stable=True).indices[:176] + 4
        ref = torch.cat([torch.arange(4, device="cuda"), best.sort().values, torch.arange(cap - 20, cap, device="cuda")])
        assert torch.equal(kept[2, h].long(), ref)


# ------------------------------------------------------------------------------ eviction
@pytest.mark.parametrize("kind", ["random", "ties", "equal", "zero", "tiny"])
@pytest.mark.parametrize("hkv,hd,block,cap,keep,sink,recent", [
    (2, 64, 16, 160, 50, 4, 10), (1, 128, 32, 96, 1, 0, 0), (3, 32, 64, 640, 300, 0, 300), (2, 96, 16, 2080, 2000, 1, 7),
    (1, 128, 128, 128, 128, 0, 0), (1, 64, 16, 4096, 77, 77, 0), (1, 256, 32, 4224, 1000, 3, 100)])
def test_evict(B, hkv, hd, block, cap, keep, sink, recent, kind):
    torch = torch_mod()
    g = np.random.default_rng(cap + keep)
    n_seq = 4
    lens = [cap, min(cap, keep + 1), keep, 0]
    d, o = filled(B, g, n_seq, hkv, cap, hd, block, lens)
    w = {"random": lambda s: g.uniform(0, 1, s) ** 8, "ties": lambda s: g.integers(0, 4, s) / 3.0,
         "equal": lambda s: np.full(s, 0.25), "zero": lambda s: np.zeros(s),
         "tiny": lambda s: g.uniform(0, 1, s) * 1e-38}[kind]((n_seq, hkv, cap)).astype(np.float32)
    for s, n in enumerate(lens):
        w[s, :, n:] = np.nan              # never looked at
    dcap = -(-keep // block) * block + block
    t = Dev(B, n_seq, hkv, dcap, hd, block)
    dl = torch.full((n_seq,), -9, dtype=torch.int32, device="cuda")
    dw = torch.full((n_seq, hkv, dcap), 3.0, device="cuda")
    kept = torch.full((n_seq, hkv, keep), -9, dtype=torch.int32, device="cuda")
    dims = make_dims(B, hkv, hkv, hd, "bf16")
    B.cb_kv8_evict(d.c, dev_i32(lens), torch.from_numpy(w).cuda(), keep, sink, recent, t.c, dl, dw, kept, dims)
    B.cb_sync(None)
    rd, rl, rw, rk = K8.evict(o, lens, w, keep, sink, recent, dcap)
    np.testing.assert_array_equal(dl.cpu().numpy(), rl)
    np.testing.assert_array_equal(kept.cpu().numpy(), rk)
    np.testing.assert_array_equal(dw.cpu().numpy(), rw)
    check_cache(t, rd, rl)


@pytest.mark.parametrize("cap", [4096, 4112, 16384, 16400, 32768, 32784])
def test_evict_where_the_kernels_meet(B, cap):
    """Capacities around those at which a thread holds more keys, or none."""
    torch = torch_mod()
    g = np.random.default_rng(cap)
    hkv, hd, block, keep, sink, recent = 2, 32, 16, 1500, 5, 333
    lens = [cap, cap - 7, keep + 1]
    d, o = filled(B, g, 3, hkv, cap, hd, block, lens)
    w = (g.uniform(0, 1, (3, hkv, cap)) ** 6).astype(np.float32)
    w[0, 1] = g.integers(0, 3, cap)                     # ties across threads and warps
    w[1, 0] = 0
    t = Dev(B, 3, hkv, 1504, hd, block)
    dl = torch.zeros(3, dtype=torch.int32, device="cuda")
    dw = torch.full((3, hkv, 1504), 3.0, device="cuda")
    kept = torch.zeros(3, hkv, keep, dtype=torch.int32, device="cuda")
    B.cb_kv8_evict(d.c, dev_i32(lens), torch.from_numpy(w).cuda(), keep, sink, recent, t.c, dl, dw, kept,
                   make_dims(B, hkv, hkv, hd, "bf16"))
    B.cb_sync(None)
    rd, rl, rw, rk = K8.evict(o, lens, w, keep, sink, recent, 1504)
    np.testing.assert_array_equal(kept.cpu().numpy(), rk)
    np.testing.assert_array_equal(dl.cpu().numpy(), rl)
    np.testing.assert_array_equal(dw.cpu().numpy(), rw)
    check_cache(t, rd, rl)


@pytest.mark.parametrize("cap", [16, 112, 1008, 1024, 1040])
def test_evict_of_short_caches(B, cap):
    torch = torch_mod()
    g = np.random.default_rng(cap)
    hkv, hd, block, keep = 3, 64, 16, max(2, cap // 3)
    sink, recent = min(3, keep - 1), keep // 4
    lens = [cap, cap - 1, keep + 1, keep]
    d, o = filled(B, g, 4, hkv, cap, hd, block, lens)
    w = (g.uniform(0, 1, (4, hkv, cap)) ** 8).astype(np.float32)
    w[:, 1] = g.integers(0, 2, (4, cap))
    w[0, 2] = np.exp(-np.arange(cap) % 7 * 11.0)          # many digits of the keys in use
    t = Dev(B, 4, hkv, -(-keep // block) * block, hd, block)
    dl = torch.zeros(4, dtype=torch.int32, device="cuda")
    kept = torch.zeros(4, hkv, keep, dtype=torch.int32, device="cuda")
    B.cb_kv8_evict(d.c, dev_i32(lens), torch.from_numpy(w).cuda(), keep, sink, recent, t.c, dl, None, kept,
                   make_dims(B, hkv, hkv, hd, "bf16"))
    B.cb_sync(None)
    rd, rl, _, rk = K8.evict(o, lens, w, keep, sink, recent, -(-keep // block) * block)
    np.testing.assert_array_equal(kept.cpu().numpy(), rk)
    np.testing.assert_array_equal(dl.cpu().numpy(), rl)
    check_cache(t, rd, rl)


def test_evict_of_a_long_cache_and_bad_weights(B):
    torch = torch_mod()
    g = np.random.default_rng(12)
    hkv, hd, block, cap, keep = 2, 32, 128, 66560, 9000          # past the keys that threads hold
    d, o = filled(B, g, 1, hkv, cap, hd, block, [cap - 3])
    w = (g.uniform(0, 1, (1, hkv, cap)) ** 4).astype(np.float32)
    w[0, 1] = g.integers(0, 9, cap) / 8.0
    t = Dev(B, 1, hkv, 9088, hd, block)
    dl, kept = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, hkv, keep, dtype=torch.int32, device="cuda")
    dims = make_dims(B, hkv, hkv, hd, "bf16")
    call = lambda length: B.cb_kv8_evict(d.c, dev_i32([length]), torch.from_numpy(w).cuda(), keep, 4, 100, t.c, dl, None,  # noqa: E731
                                         kept, dims)
    call(cap - 3)
    B.cb_sync(None)
    rd, rl, _, rk = K8.evict(o, [cap - 3], w, keep, 4, 100, 9088)
    np.testing.assert_array_equal(kept.cpu().numpy(), rk)
    check_cache(t, rd, rl)
    w[0, 0, 50:53] = [np.nan, np.inf, -1.0]
    call(cap - 3)
    with pytest.raises(B.CBError) as e:
        B.cb_sync(None)
    assert e.value.status == 5
    np.testing.assert_array_equal(kept.cpu().numpy(), K8.evict(o, [cap - 3], w, keep, 4, 100, 9088)[3])
    call(-1)
    with pytest.raises(B.CBError) as e:
        B.cb_sync(None)
    assert e.value.status == 9 and int(dl[0]) == 0 and torch.all(kept == -1)


# ------------------------------------------------------------------------------ logits
def run_logits(B, x, dtype, out="new", **rules):
    torch = torch_mod()
    xd = dev(x, dtype)
    y = {"new": torch.empty_like(xd), "in place": xd, "none": None}[out]
    tok = torch.full((x.shape[0],), -9, dtype=torch.int32, device="cuda")
    B.cb_logits_process(xd, B.logit_rules(**rules), y, tok)
    return y, tok


def mask_words(m):
    torch = torch_mod()
    n, V = m.shape
    bits = np.zeros((n, -(-V // 32) * 32 + 32), np.uint8)        # a row longer than it needs to be
    bits[:, :V] = m
    return torch.from_numpy(np.packbits(bits, axis=1, bitorder="little").view(np.int32).copy()).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("out", ["new", "in place", "none"])
@pytest.mark.parametrize("n,V,T,nb", [(1, 1, 3, 1), (3, 7, 40, 5), (2, 1000, 1, 0), (5, 32000, 700, 40), (2, 64000, 3000, 4096),
                                      (1, 150001, 5000, 33), (2, 131072, 100, 300), (17, 4099, 0, 64)])
def test_logits(B, n, V, T, nb, out, dtype):
    g = np.random.default_rng(V + T)
    x = rounded(g.standard_normal((n, V)) * 3, dtype)
    hist = (g.uniform(0, 1, (n, T)) ** 3 * V).astype(np.int32).clip(0, V - 1)
    ln = g.integers(0, T + 1, n)
    ln[0] = T
    pl = g.integers(0, ln + 1)
    rep, pres, freq = (g.uniform(a, b, n).astype(np.float32) for a, b in ((0.5, 2), (-1, 1), (0, 0.5)))
    bid = g.integers(-1, V, (n, nb)).astype(np.int32)
    bid[:, ::3] = bid[:, :1] if nb else 0                          # the same id many times
    bias = g.standard_normal((n, nb)).astype(np.float32)
    mask = g.uniform(0, 1, (n, V)) < 0.5
    mask[-1] = n == 1                                              # one row allows nothing
    rules = dict(history=dev_i32(hist), history_len=dev_i32(ln), prompt_len=dev_i32(pl), repetition=dev(rep),
                 presence=dev(pres), frequency=dev(freq), mask=mask_words(mask))
    if nb:
        rules.update(bias_id=dev_i32(bid), bias=dev(bias))
    y, tok = run_logits(B, x, dtype, out, **rules)
    B.cb_sync(None)
    eps = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    for b in range(n):
        ref = K8.logits(x[b], hist[b, :ln[b]], int(pl[b]), float(rep[b]), float(pres[b]), float(freq[b]),
                        list(zip(bid[b], bias[b].astype(np.float64))), mask[b])
        if out == "none":
            best = K8.token(rounded(ref, dtype))
            t = int(tok[b])
            # a near tie may round the other way: the chosen value is then within two roundings of the best
            assert t == best or abs(ref[t] - ref[best]) <= 4 * eps * abs(ref[best])
            continue
        got = host(y[b])
        # per operation one rounding of the largest magnitude met: the logit, its penalties, each bias
        size = np.abs(x[b]).astype(np.float64) * 2
        cnt = np.bincount(hist[b, :ln[b]], minlength=V)[:V] if T else np.zeros(V)
        size += np.abs(freq[b]) * cnt + np.abs(pres[b])
        ok = bid[b] >= 0
        nbias = np.zeros(V)
        np.add.at(size, bid[b][ok], np.abs(bias[b][ok]))
        np.add.at(nbias, bid[b][ok], 1)
        fin = np.isfinite(ref)
        np.testing.assert_array_equal(np.isneginf(got), ~fin)
        tol = eps * np.abs(ref[fin]) * 1.01 + (6 + nbias[fin]) * 2.0 ** -24 * size[fin]
        assert np.all(np.abs(got[fin] - ref[fin]) <= tol)
        assert int(tok[b]) == K8.token(got)


def test_logits_without_rules_is_the_argmax(B):
    torch = torch_mod()
    x = np.zeros((4, 40000), np.float32)
    x[1, 39999] = x[1, 20000] = 2.0                  # ties: the lower id
    x[2] = -np.inf
    x[3] = -5.0
    x[3, 8191] = -0.0
    x[3, 8192] = 0.0
    y, tok = run_logits(B, x, "f32")
    B.cb_sync(None)
    assert tok.tolist() == [0, 20000, -1, 8191]
    assert torch.equal(y.cpu(), torch.from_numpy(x))
    x[0, 5], x[0, 9] = np.inf, np.nan
    x[2, 3] = np.nan
    y, tok = run_logits(B, x, "f32")
    with pytest.raises(B.CBError) as e:
        B.cb_sync(None)
    assert e.value.status == 5 and tok.tolist() == [5, 20000, -1, 8191]
    # a NaN that the mask hides is none of the call's business; nor is the type's lowest value
    m = np.ones(x.shape, bool)
    m[0, 9] = m[2, 3] = False
    x[2, 17] = np.finfo(np.float32).min
    y, tok = run_logits(B, x, "f32", mask=mask_words(m))
    B.cb_sync(None)
    assert tok.tolist() == [5, 20000, 17, 8191] and float(y[0, 9]) == -np.inf


def test_logits_report_bad_ids_lengths_and_penalties(B):
    x = np.random.default_rng(0).standard_normal((2, 5000)).astype(np.float32)
    base = dict(history_len=dev_i32([3, 3]), repetition=dev(np.array([2.0, 2.0], np.float32)))

    def expect(status, ref, **rules):
        y, tok = run_logits(B, x, "f32", **{**base, **rules})
        with pytest.raises(B.CBError) as e:
            B.cb_sync(None)
        assert e.value.status == status
        for b in range(2):
            np.testing.assert_allclose(host(y[b]), ref[b], rtol=2e-7)
            assert int(tok[b]) == K8.token(host(y[b]))

    h = np.array([[1, 2, 3], [4, 5, 6]])
    bad = h.copy()
    bad[0, 1], bad[1, 2] = 5000, -1
    expect(9, [K8.logits(x[b], bad[b], repetition=2.0) for b in range(2)], history=dev_i32(bad))
    expect(9, [K8.logits(x[b], h[b, :n], repetition=2.0) for b, n in ((0, 3), (1, 0))], history=dev_i32(h),
           history_len=dev_i32([4, -1]))
    expect(9, [K8.logits(x[b], h[b], p, 2.0, 1.0) for b, p in ((0, 3), (1, 0))], history=dev_i32(h),
           prompt_len=dev_i32([4, -1]), presence=dev(np.ones(2, np.float32)))
    for r in (0.0, -1.0, np.nan, np.inf):
        expect(5, [K8.logits(x[b], h[b], repetition=v) for b, v in ((0, 2.0), (1, 1.0))], history=dev_i32(h),
               repetition=dev(np.array([2.0, r], np.float32)))
    expect(9, [K8.logits(x[b], h[b], repetition=2.0, bias=[(7, 1.5)]) for b in range(2)], history=dev_i32(h),
           bias_id=dev_i32([[7, 5000], [7, -2]]), bias=dev(np.full((2, 2), 1.5, np.float32)))
    B.cb_sync(None)


# ------------------------------------------------------------------------------ use
def test_captured_graphs_streams_and_a_shared_workspace(B):
    """Decoding steps captured once and replayed, on a stream of their own, two graphs sharing one
    workspace; the eager calls give the same bits."""
    torch = torch_mod()
    g = np.random.default_rng(20)
    H, hkv, hd, block, cap, n_seq = 8, 2, 64, 16, 128, 3
    dims = make_dims(B, H, hkv, hd, "bf16")
    lens = [100, 17, 64]
    x = dev(rows(g, n_seq, 1, hkv, hd, "bf16"), "bf16")
    q = dev(rounded(g.standard_normal((n_seq, 1, H, hd)), "bf16"), "bf16")
    n = B.cb_kv8_workspace_bytes(dims, n_seq, cap, 1, True)
    shared = torch.empty(n, dtype=torch.uint8, device="cuda")

    def build():
        d, _ = filled(B, np.random.default_rng(21), n_seq, hkv, cap, hd, block, lens)
        return d, dict(start=dev_i32(lens), w=torch.zeros(n_seq, hkv, cap, device="cuda"), out=torch.zeros_like(q))

    def step(d, b):
        B.cb_kv8_append(x, x, 1, b["start"], None, d.c, dims)
        B.cb_kv8_attention(q, b["start"], 1, d.c, dims, b["out"], b["w"], shared)
        b["start"] += 1

    d0, b0 = build()
    for _ in range(4):
        step(d0, b0)
    B.cb_sync(None)
    s = torch.cuda.Stream()
    pairs = [build(), build()]
    graphs = []
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for d, b in pairs:
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=s):
                step(d, b)
            graphs.append(gr)
        for _ in range(4):
            for gr in graphs:
                gr.replay()
    torch.cuda.current_stream().wait_stream(s)
    B.cb_sync(None)
    for d, b in pairs:
        assert torch.equal(d.k, d0.k) and torch.equal(d.v, d0.v)
        assert torch.equal(b["out"], b0["out"]) and torch.equal(b["w"], b0["w"]) and torch.equal(b["start"], b0["start"])


@pytest.mark.parametrize("n_q", [1, 30, 150])
def test_the_first_call_may_be_captured(B, n_q):
    """What the library looks up once per device, it may look up while a graph is captured."""
    torch = torch_mod()
    g = np.random.default_rng(n_q)
    H, hkv, hd, cap = 4, 2, 64, 528
    d, o = filled(B, g, 1, hkv, cap, hd, 16, [cap])
    q = rounded(g.standard_normal((1, n_q, H, hd)), "bf16")
    last = g.integers(0, cap, (1, n_q))
    dims = make_dims(B, H, hkv, hd, "bf16")
    qd, ld, w = dev(q, "bf16"), dev_i32(last), torch.zeros(1, hkv, cap, device="cuda")
    out = torch.zeros_like(qd)
    ws = torch.empty(B.cb_kv8_workspace_bytes(dims, 1, cap, n_q, True), dtype=torch.uint8, device="cuda")
    B.cb_sync(None)
    B.cb_shutdown()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        B.cb_kv8_attention(qd, ld, n_q, d.c, dims, out, w, ws)
    gr.replay()
    B.cb_sync(None)
    check_attention(out, host(w), K8.attention(o, q.astype(np.float64), last), last, "bf16", hd)


class Answer:
    """One request over 8-bit caches: the prompt's rows, then a token per step, all lengths and
    positions on the device; the caches are thinned out in between.  see(cache, layer, q, k, v,
    out, weights before) is called after each attention, said() after each token."""
    KEEP, SINK, RECENT, T = 40, 4, 12, 128

    def __init__(self, B, shape, prompt):
        from non_prefix_kv_gb300 import engine, synth
        torch = torch_mod()
        self.B, self.L, self.s = B, shape.n_layers, shape
        self.dm = engine.DeviceModel.from_host(synth.make_model(shape, seed=3))
        self.eng = engine.BlendEngine(self.dm, len(prompt), max_pos=256)
        self.prompt = dev_i32(prompt)
        n, hkv, hd, dt = len(prompt), shape.n_kv_heads, shape.head_dim, tdt(shape.dtype)
        self.caches = [[Dev(B, 1, hkv, cap, hd, 16) for _ in range(self.L)] for cap in (96, 64)]
        self.acc = [[torch.zeros(1, hkv, cap, device="cuda") for _ in range(self.L)] for cap in (96, 64)]
        self.len = [torch.full((1,), m, dtype=torch.int32, device="cuda") for m in (n, 0)]
        self.kept = torch.empty(1, hkv, self.KEEP, dtype=torch.int32, device="cuda")
        self.pos, self.tok = dev_i32([n]), dev_i32([0])
        self.hist, self.hl = dev_i32(np.pad(prompt, (0, self.T - n))[None]), dev_i32([n])
        mask = np.ones((1, shape.vocab), bool)
        mask[0, ::5] = False
        self.rules = B.logit_rules(history=self.hist, history_len=self.hl, prompt_len=dev_i32([n]),
                                   repetition=dev(np.array([1.3], np.float32)), presence=dev(np.array([0.4], np.float32)),
                                   frequency=dev(np.array([0.2], np.float32)), bias_id=dev_i32([[7, 11, 7]]),
                                   bias=dev(np.array([[0.5, -1.0, 0.25]], np.float32)), mask=mask_words(mask))
        self.mask = mask[0]
        size = max(B.cb_kv8_workspace_bytes(self.dm.dims, 1, 96, m, True) for m in (1, n))
        self.ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        row = lambda w, m=1: torch.empty(m, w, dtype=dt, device="cuda")  # noqa: E731
        self.bufs = {m: [row(shape.d_model, m), row(shape.q_width, m), row(shape.kv_width, m), row(shape.kv_width, m),
                         row(shape.q_width, m)] for m in (1, n)}
        self.logits = torch.empty(1, shape.vocab, device="cuda")
        self.out = torch.empty_like(self.logits)
        self.see = self.said = lambda *a: None

    def rows(self, m, tokens, pos, start, last, which):
        """m rows through the layers; their hidden rows are bufs[m][0]."""
        B, dm, e, s = self.B, self.dm, self.eng, self.s
        x, q, k, v, o = self.bufs[m]
        B.cb_gather_rows(x, dm.embed, tokens, m, s.d_model * x.element_size())
        for l in range(self.L):
            before = self.acc[which][l].clone()
            B.cb_selective_qkv(x, None, pos, m, dm.dims, dm.layers_c[l], e.cos_sin, e.max_pos, q, k, v, e.ws)
            B.cb_kv8_append(k, v, m, start, None, self.caches[which][l].c, dm.dims)
            B.cb_kv8_attention(q, last, m, self.caches[which][l].c, dm.dims, o, self.acc[which][l], self.ws)
            self.see(which, l, q, k, v, o, before)
            B.cb_o_proj_ffn(o, x, m, dm.dims, dm.layers_c[l], x, e.ws)

    def token(self, m):
        B, dm = self.B, self.dm
        B.cb_lmhead_argmax(self.bufs[m][0][m - 1], dm.final_norm, dm.w_lm, dm.dims, self.logits, self.tok, self.eng.ws)
        B.cb_logits_process(self.logits, self.rules, self.out, self.tok)
        self.said()
        self.hist.scatter_(1, self.hl.long()[None], self.tok[None])
        self.hl += 1

    def prefill(self):
        n = len(self.prompt)
        last = torch_mod().arange(n, dtype=torch_mod().int32, device="cuda")
        self.rows(n, self.prompt, last, dev_i32([0]), last, 0)
        self.token(n)

    def step(self, which):
        self.rows(1, self.tok, self.pos, self.len[which], self.len[which], which)
        self.token(1)
        self.pos += 1
        self.len[which] += 1

    def thin(self):
        for l in range(self.L):
            self.B.cb_kv8_evict(self.caches[0][l].c, self.len[0], self.acc[0][l], self.KEEP, self.SINK, self.RECENT,
                                self.caches[1][l].c, self.len[1], self.acc[1][l], self.kept, self.dm.dims)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_an_answer_from_its_prompt_to_its_last_token(B, dtype):
    """The operators as they are used: a prompt's rows appended and attended (their weights
    accounted), eight tokens one by one, the caches thinned out, eight more.  Every operator's
    result is checked against the oracle's from the same inputs; then the same answer with each
    token's step captured once and replayed gives the same bits."""
    from non_prefix_kv_gb300 import synth
    torch = torch_mod()
    shape = synth.ModelShape(n_layers=2, d_model=512, n_heads=8, n_kv_heads=2, head_dim=64, d_ff=1024, vocab=512,
                             dtype=dtype, w_std=0.05)
    prompt = np.random.default_rng(40).integers(0, shape.vocab, 60).astype(np.int32)
    hkv, hd, H = shape.n_kv_heads, shape.head_dim, shape.n_heads

    a = Answer(B, shape, prompt)
    twins = [[K8.empty(1, hkv, cap, hd, 16) for _ in range(a.L)] for cap in (96, 64)]
    used = [0]

    def see(which, l, q, k, v, o, before):
        m = q.shape[0]
        n0 = used[0]
        kv = lambda t: host(t).reshape(1, m, hkv, hd).astype(np.float32)  # noqa: E731
        K8.append(twins[which][l], kv(k), kv(v), [n0])
        last = np.arange(n0, n0 + m)[None]
        ref = K8.attention(twins[which][l], host(q).reshape(1, m, H, hd), last)
        after = a.acc[which][l]
        check_attention(o.view(1, m, H, hd), None, ref, last, dtype, hd)
        # the account: the oracle's weights with the relative error of a weight (above), and one
        # rounding of the sum
        w, zmag = ref[1], ref[3]
        rel = (2 * (zmag.max() * ((hd + 4) * 2.0 ** -24 + (2.0 ** -21 if dtype == "f32" else 0)) + 2.0 ** -21)
               + (n0 + m) * 2.0 ** -24 + (m * H + 8) * 2.0 ** -24)
        assert np.all(np.abs(host(after) - (host(before) + w)) <= w * rel + host(after) * 2.0 ** -23 + 1e-30)
        if l == a.L - 1:
            used[0] += m

    def said():
        h = a.hist[0, :int(a.hl[0])].cpu().numpy()
        ref = K8.logits(host(a.logits)[0], h, len(prompt), float(np.float32(1.3)), float(np.float32(0.4)),
                        float(np.float32(0.2)), [(7, 0.5), (11, -1.0), (7, 0.25)], a.mask)
        got, fin = host(a.out)[0], np.isfinite(ref)
        np.testing.assert_array_equal(np.isneginf(got), ~fin)
        # at most 8 roundings of the largest magnitude met
        size = 2 * np.abs(host(a.logits)[0]) + 0.2 * len(h) + 0.4 + 1.75
        assert np.all(np.abs(got[fin] - ref[fin]) <= 8 * 2.0 ** -24 * size[fin])
        assert int(a.tok[0]) == K8.token(got)

    a.see, a.said = see, said
    a.prefill()
    for _ in range(8):
        a.step(0)
    a.thin()
    B.cb_sync(None)
    for l in range(a.L):
        check_cache(a.caches[0][l], twins[0][l], [used[0]])
        twins[1][l], dl, dw, _ = K8.evict(twins[0][l], [used[0]], a.acc[0][l].cpu().numpy(), a.KEEP, a.SINK, a.RECENT, 64)
        check_cache(a.caches[1][l], twins[1][l], dl)
        np.testing.assert_array_equal(a.acc[1][l].cpu().numpy(), dw)
    used[0] = a.KEEP
    for _ in range(8):
        a.step(1)
    B.cb_sync(None)
    for l in range(a.L):
        check_cache(a.caches[1][l], twins[1][l], [a.KEEP + 8])

    b = Answer(B, shape, prompt)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b.prefill()
        for which in (0, 1):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                b.step(which)
            for _ in range(8):
                g.replay()
            if which == 0:
                b.thin()
    torch.cuda.current_stream().wait_stream(s)
    B.cb_sync(None)
    assert torch.equal(a.hist, b.hist) and torch.equal(a.hl, b.hl) and torch.equal(a.pos, b.pos)
    for which in (0, 1):
        for l in range(a.L):
            x, y = a.caches[which][l], b.caches[which][l]
            assert torch.equal(x.k, y.k) and torch.equal(x.v, y.v)
            assert torch.equal(a.acc[which][l], b.acc[which][l])
