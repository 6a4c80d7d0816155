"""Rotary positions in their usual forms, as a table and over rows, against the fp64 oracle.

Tolerances, element by element: cos and sin are rounded once (2^-24 of a value at most the amplitude a);
an output is two products and a sum in fp32, each rounded at most once (a product may be kept exact by a
fused operation), so it is off by at most 3 x 2^-24 a (|x1| + |x2|), and by its own rounding:
2^-24 of itself in fp32, 2^-8 in bf16.  What is only copied is equal bit by bit."""
import numpy as np
import pytest

import oracle.answers_oracle as A
from tests.gpu_util import dev_i32, ensure_lib, host, tdt, torch_mod

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24
STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def B():
    torch_mod()
    ensure_lib()
    from non_prefix_kv_gb300 import binding
    return binding


def dims_of(B, H, hkv, hd, dtype):
    return B.cb_dims(H * hd, H, hkv, hd, 256, 64, 1e4, 1e-5, B.CB_BF16 if dtype == "bf16" else B.CB_F32)


def normal(g, dtype, *shape):
    torch = torch_mod()
    return torch.from_numpy(g.standard_normal(shape).astype(np.float32)).cuda().to(tdt(dtype))


def table(B, spec, max_pos):
    t = torch_mod().empty(max_pos * spec.rot_dim, device="cuda")
    B.cb_rope_table_scaled(t, max_pos, spec)
    return t


SPECS = [dict(), dict(scaling=1, factor=4.0), dict(scaling=2, factor=8.0), dict(scaling=3, factor=8.0, original_len=64.0, low=1.0, high=4.0),
         dict(scaling=4, factor=8.0, original_len=64.0, low=1.0, high=32.0, amplitude=1.2079441541679836)]


def spec_of(B, layout, rot, base=1e4, **kw):
    return B.rope_spec(layout, rot, base, **kw)


def theta_of(rot, base=1e4, **kw):
    return A.theta(rot, base, kw.get("scaling", 0), kw.get("factor", 1.0), kw.get("original_len", 0.0), kw.get("low", 0.0),
                   kw.get("high", 0.0))


@pytest.mark.parametrize("kw", SPECS)
@pytest.mark.parametrize("rot,max_pos", [(128, 300), (2, 5), (20, 77)])
def test_table(B, kw, rot, max_pos):
    """The angle in fp64 is off by 2^-52 of itself a few times (here below 300 rad): far below the
    rounding to fp32."""
    if kw.get("scaling") == 2 and rot == 2:
        kw = dict(kw, scaling=1)
    t = host(table(B, spec_of(B, 1, rot, **kw), max_pos)).reshape(max_pos, rot // 2, 2)
    a = kw.get("amplitude", 1.0)
    ang = np.arange(max_pos)[:, None] * theta_of(rot, **kw)
    for i, f in enumerate((np.cos, np.sin)):
        assert np.all(np.abs(t[..., i] - a * f(ang)) <= EPS * np.abs(a * f(ang)) + 1e-12)


def test_plain_table_is_the_blends(B):
    torch = torch_mod()
    a = torch.empty(1000 * 64, device="cuda")
    B.cb_rope_table(a, 1000, 64, 5e6)
    b = table(B, B.rope_spec(0, 64, 5e6), 1000)
    # theta by pow on the device and on the host: the angles may differ by a few 2^-52 of themselves
    assert float((a - b).abs().max()) <= 2 * EPS


def check(y, x, pos, th, half, dtype, amp=1.0):
    """y, x [n, heads, hd] on the device."""
    ref = A.rotate(host(x), pos, th, half, amp)
    m = len(th)
    xs = np.abs(host(x))
    a, b = (np.arange(m), np.arange(m) + m) if half else (2 * np.arange(m), 2 * np.arange(m) + 1)
    both = np.zeros_like(xs)
    both[..., a] = both[..., b] = xs[..., a] + xs[..., b]
    got = host(y)
    tol = 3 * EPS * amp * both + STEP[dtype] * np.abs(ref) * 1.01 + 1e-30
    np.testing.assert_array_equal(got[..., 2 * m:], host(x)[..., 2 * m:])
    assert np.all(np.abs(got - ref)[..., :2 * m] <= tol[..., :2 * m])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("n,H,hkv,hd,rot", [(1, 1, 1, 32, 32), (3, 4, 2, 64, 32), (65, 56, 8, 128, 128), (2, 8, 8, 256, 256),
                                            (7, 5, 1, 128, 20), (33, 3, 3, 96, 48), (1100, 4, 2, 64, 64), (2, 2, 2, 256, 2),
                                            (5, 40, 40, 160, 16)])
def test_rows_as_one_projection_leaves_them_into_caches(B, dtype, layout, n, H, hkv, hd, rot):
    torch = torch_mod()
    g = np.random.default_rng(n + hd + rot)
    kw = SPECS[(n + layout) % 5] if rot > 2 else SPECS[0]
    spec, th, amp, max_pos = spec_of(B, layout, rot, **kw), theta_of(rot, **kw), kw.get("amplitude", 1.0), 500
    qw, w = H * hd, hkv * hd
    x = normal(g, dtype, n, qw + 2 * w)
    q, k, v = x.split([qw, w, w], 1)
    pos = g.integers(-max_pos + 1, max_pos, n)
    rows = n + 9
    dst = g.permutation(rows)[:n]
    if n > 2:
        dst[1] = -1                               # an idle row
    qo = torch.full((n, qw), 7.0, dtype=x.dtype, device="cuda")
    ko, vo = (torch.full((rows, w), 5.0, dtype=x.dtype, device="cuda") for _ in range(2))
    before = x.clone()
    tab = table(B, spec, max_pos)
    for inverse in (False, True):
        B.cb_rope_rows(q, k, v, dev_i32(pos), qo, ko, vo, dims_of(B, H, hkv, hd, dtype), spec, tab, max_pos,
                       kv_row=dev_i32(dst), inverse=inverse)
        B.cb_sync(None)
        p = -pos if inverse else pos
        check(qo.reshape(n, H, hd), q.reshape(n, H, hd), p, th, layout == 1, dtype, amp)
        live = dst >= 0
        at = torch.from_numpy(dst[live]).cuda()
        lv = torch.from_numpy(live).cuda()
        check(ko[at].reshape(-1, hkv, hd), k[lv].reshape(-1, hkv, hd), p[live], th, layout == 1, dtype, amp)
        assert torch.equal(vo[at], v[lv])
        rest = torch.ones(rows, dtype=torch.bool, device="cuda")
        rest[at] = False
        assert bool((ko[rest] == 5).all()) and bool((vo[rest] == 5).all())
    assert torch.equal(x, before)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_listed_source_rows_match_rope_shift(B, dtype):
    """With offsets for positions and the plain form the rows are cb_rope_shift's, bit for bit (both one
    fused product and sum after a rounded product, whichever way)."""
    torch = torch_mod()
    g = np.random.default_rng(5)
    n, n_src, hkv, hd = 200, 90, 3, 64
    k, v = normal(g, dtype, n_src, hkv * hd), normal(g, dtype, n_src, hkv * hd)
    src, delta = dev_i32(g.integers(0, n_src, n)), dev_i32(g.integers(-399, 400, n))
    spec, dims = B.rope_spec(0, hd, 1e4), dims_of(B, hkv, hkv, hd, dtype)
    tab = torch.empty(400 * hd, device="cuda")
    B.cb_rope_table(tab, 400, hd, 1e4)
    a, b, c, d = (torch.empty(n, hkv * hd, dtype=k.dtype, device="cuda") for _ in range(4))
    B.cb_rope_rows(None, k, v, delta, None, a, b, dims, spec, tab, 400, src_row=src)
    B.cb_rope_shift(c, d, k, v, src, delta, n, dims, tab, 400)
    B.cb_sync(None)
    assert torch.equal(b, d)
    assert float((a.double() - c.double()).abs().max()) <= (4 * EPS if dtype == "f32" else 2.0 ** -8) * 2 * float(k.abs().max())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", [0, 1])
def test_odd_strides_and_alignments(B, dtype, layout):
    """Rows of odd length that start at odd elements; keys only; queries only."""
    torch = torch_mod()
    g = np.random.default_rng(6)
    n, H, hkv, hd, rot, max_pos = 6, 4, 2, 64, 32, 50
    spec, th = B.rope_spec(layout, rot, 1e4), theta_of(rot)
    tab, dims = table(B, spec, max_pos), dims_of(B, H, hkv, hd, dtype)
    pos = g.integers(0, max_pos, n)
    x = normal(g, dtype, n, 1001)
    y = torch.zeros(n, 777, dtype=x.dtype, device="cuda")
    q, k = x[:, 1:1 + H * hd], x[:, 500:500 + hkv * hd]
    qo, ko = y[:, 3:3 + H * hd], y[:, 301:301 + hkv * hd]
    B.cb_rope_rows(q, k, None, dev_i32(pos), qo, ko, None, dims, spec, tab, max_pos)
    B.cb_sync(None)
    check(qo.reshape(n, H, hd), q.reshape(n, H, hd), pos, th, layout == 1, dtype)
    check(ko.reshape(n, hkv, hd), k.reshape(n, hkv, hd), pos, th, layout == 1, dtype)
    keep = torch.ones(777, dtype=torch.bool, device="cuda")
    keep[3:3 + H * hd] = keep[301:301 + hkv * hd] = False
    assert not y[:, keep].any()
    z = torch.zeros(n, H * hd, dtype=x.dtype, device="cuda")
    B.cb_rope_rows(q, None, None, dev_i32(pos), z, None, None, dims, spec, tab, max_pos)
    B.cb_sync(None)
    assert torch.equal(z, qo.contiguous())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("packed", [False, True])
def test_in_place(B, dtype, layout, packed):
    torch = torch_mod()
    g = np.random.default_rng(7)
    n, H, hkv, hd, rot, max_pos = 37, 4, 2, 128, 64, 90
    spec, dims = B.rope_spec(layout, rot, 1e4), dims_of(B, H, hkv, hd, dtype)
    tab, pos = table(B, spec, max_pos), dev_i32(g.integers(0, max_pos, n))
    x = normal(g, dtype, n, (H + 2 * hkv) * hd)
    parts = [H * hd, hkv * hd, hkv * hd]
    if packed:
        q, k, v = x.clone().split(parts, 1)
    else:
        q, k, v = (t.contiguous() for t in x.split(parts, 1))
    a, b, c = (torch.empty(n, m, dtype=x.dtype, device="cuda") for m in parts)
    B.cb_rope_rows(q, k, v, pos, a, b, c, dims, spec, tab, max_pos)
    B.cb_rope_rows(q, k, v, pos, q, k, v, dims, spec, tab, max_pos)
    B.cb_sync(None)
    for s, t in ((q, a), (k, b), (v, c)):
        assert torch.equal(s, t)


def test_gradient_is_the_inverse_and_agrees_with_differences(B):
    """<R x, y> = <x, R^T y> in fp32 sums of 2^15 products, and the slope of <R(x + e d), y> along d."""
    torch = torch_mod()
    g = np.random.default_rng(8)
    n, H, hd, rot, max_pos = 64, 8, 64, 32, 1000
    for layout in (0, 1):
        spec = B.rope_spec(layout, rot, 1e4, amplitude=1.25)
        tab, dims, pos = table(B, spec, max_pos), dims_of(B, H, H, hd, "f32"), dev_i32(g.integers(0, max_pos, n))
        x, y, d = (normal(g, "f32", n, H * hd) for _ in range(3))

        def turn(t, inverse=False):
            o = torch.empty_like(t)
            B.cb_rope_rows(t, None, None, pos, o, None, None, dims, spec, tab, max_pos, inverse=inverse)
            return o.double()

        grad = turn(y, True)
        size = float((turn(x).abs() * y.double().abs()).sum())
        assert abs(float((turn(x) * y.double()).sum() - (x.double() * grad).sum())) <= 8 * EPS * size
        slope = float(((turn(x + d) - turn(x - d)) * y.double()).sum()) / 2
        assert abs(slope - float((grad * d.double()).sum())) <= 16 * EPS * 2 * size
    B.cb_sync(None)


def test_bad_positions_and_rows_are_skipped_and_reported(B):
    torch = torch_mod()
    g = np.random.default_rng(9)
    H, hd, max_pos, n = 2, 64, 40, 8
    spec, dims = B.rope_spec(1, hd, 1e4), dims_of(B, H, H, hd, "bf16")
    tab = table(B, spec, max_pos)
    x = normal(g, "bf16", n, 3 * H * hd)
    q, k, v = x.split([H * hd] * 3, 1)
    good = np.array([0, 39, -39, 5, 6, 7, 8, 9])
    src, dst = np.arange(n), np.arange(n)[::-1].copy()
    want = None
    for what, i, val in (("", 0, 0), ("pos", 1, 40), ("pos", 2, -40), ("pos", 3, -2 ** 31), ("pos", 4, 2 ** 31 - 1), ("src", 5, n), ("src", 6, -1),
                         ("dst", 7, n), ("dst", 0, -2)):
        p, s, t = good.copy(), src.copy(), dst.copy()
        if what:
            {"pos": p, "src": s, "dst": t}[what][i] = val
        qo, ko, vo = (torch.full((n, H * hd), 3.0, dtype=x.dtype, device="cuda") for _ in range(3))
        B.cb_rope_rows(q, k, v, dev_i32(p), qo, ko, vo, dims, spec, tab, max_pos, src_row=dev_i32(s), kv_row=dev_i32(t))
        if not what:
            B.cb_sync(None)
            want = qo, ko, vo
            continue
        with pytest.raises(B.CBError) as e:
            B.cb_sync(None)
        assert e.value.status == 9
        kv_gone = int(dst[i])
        for o, w, gone in ((qo, want[0], i if what == "pos" else None), (ko, want[1], kv_gone), (vo, want[2], kv_gone)):
            keep = torch.ones(n, dtype=torch.bool, device="cuda")
            if gone is not None:
                keep[gone] = False
                assert bool((o[gone] == 3).all())
            assert torch.equal(o[keep], w[keep])


def test_on_another_stream_captured_and_replayed(B):
    torch = torch_mod()
    g = np.random.default_rng(10)
    n, H, hkv, hd, max_pos = 16, 8, 2, 128, 64
    spec, dims = B.rope_spec(1, hd, 1e4), dims_of(B, H, hkv, hd, "bf16")
    tab = table(B, spec, max_pos)
    x, pos = normal(g, "bf16", n, (H + 2 * hkv) * hd), dev_i32(g.integers(0, max_pos, n))
    q, k, v = x.split([H * hd, hkv * hd, hkv * hd], 1)
    o = [torch.empty(n, m, dtype=x.dtype, device="cuda") for m in (H * hd, hkv * hd, hkv * hd)]
    torch.cuda.synchronize()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        B.cb_rope_rows(q, k, v, pos, *o, dims, spec, tab, max_pos)
    for _ in range(3):
        x.copy_(normal(g, "bf16", *x.shape))
        pos.copy_(dev_i32(g.integers(0, max_pos, n)))
        graph.replay()
        torch.cuda.synchronize()
        ref = [torch.empty_like(t) for t in o]
        with torch.cuda.stream(s):
            B.cb_rope_rows(q, k, v, pos, *ref, dims, spec, tab, max_pos)
        B.cb_sync(s)
        assert all(torch.equal(a, b) for a, b in zip(o, ref))


def test_rows_past_2_to_the_31_elements(B):
    """The last row of a cache of more than 2^31 elements."""
    torch = torch_mod()
    hkv, hd, rows = 8, 256, (1 << 20) + 3
    spec, dims = B.rope_spec(1, hd, 1e4), dims_of(B, hkv, hkv, hd, "bf16")
    tab = table(B, spec, 8)
    cache = [torch.zeros(rows, hkv * hd, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    k = torch.randn(2, hkv * hd, device="cuda").bfloat16()
    B.cb_rope_rows(None, k, k, dev_i32([3, 5]), None, *cache, dims, spec, tab, 8, kv_row=dev_i32([rows - 1, 0]))
    back = torch.empty_like(k)
    B.cb_rope_rows(None, cache[1], None, dev_i32([3, 5]), None, back, None, dims, spec, tab, 8, src_row=dev_i32([rows - 1, 0]))
    B.cb_sync(None)
    assert torch.equal(cache[1][-1], k[0]) and torch.equal(cache[1][0], k[1]) and torch.equal(cache[0][-1], back[0])
    assert int(cache[1].any(1).sum()) == 2
