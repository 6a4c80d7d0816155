"""The fp64 restatement of rotary forms, shared-prefix attention and sampling against closed forms,
and the host's own angles against it (no GPU)."""
import math

import numpy as np
import pytest

import oracle.answers_oracle as A
import oracle.cacheblend_oracle as O
from non_prefix_kv_gb300 import binding as B
from non_prefix_kv_gb300 import build as nb


@pytest.fixture(scope="module")
def lib():
    nb.build()
    return B.lib()


def test_interleaved_unscaled_is_the_blends_rotation():
    g = np.random.default_rng(0)
    x, pos = g.standard_normal((5, 3, 64)), np.array([0, 1, 7, 900, 16383])
    y = A.rotate(x, pos, A.theta(64, 1e4), False)
    np.testing.assert_allclose(y, O.rope_rotate(x, pos, 1e4), atol=1e-11)
    z = (x[..., 0::2] + 1j * x[..., 1::2]) * np.exp(1j * pos[:, None, None] * 1e4 ** (-np.arange(32) / 32))
    np.testing.assert_allclose(y[..., 0::2], z.real, atol=1e-11)
    np.testing.assert_allclose(y[..., 1::2], z.imag, atol=1e-11)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("rot", [2, 20, 64])
def test_rotation_keeps_norms_composes_and_leaves_the_rest(half, rot):
    g = np.random.default_rng(rot)
    x, t = g.standard_normal((6, 2, 64)), A.theta(rot, 5e6)
    p = g.integers(-5000, 5000, 6)
    y = A.rotate(x, p, t, half)
    np.testing.assert_array_equal(y[..., rot:], x[..., rot:])
    np.testing.assert_allclose(np.linalg.norm(y, axis=2), np.linalg.norm(x, axis=2))
    np.testing.assert_allclose(A.rotate(y, -p, t, half), x, atol=1e-9)
    np.testing.assert_allclose(A.rotate(A.rotate(x, p, t, half), 3 * p, t, half), A.rotate(x, 4 * p, t, half), atol=1e-9)


def test_the_layouts_are_one_another_permuted():
    g = np.random.default_rng(1)
    x, t, p = g.standard_normal((4, 1, 32)), A.theta(32, 1e4), np.arange(4)
    perm = np.arange(32).reshape(16, 2).T.reshape(-1)          # interleaved -> half
    np.testing.assert_allclose(A.rotate(x[..., perm], p, t, True), A.rotate(x, p, t, False)[..., perm])


def test_scaled_frequencies_by_hand():
    t = A.theta(128, 1e4)
    np.testing.assert_allclose(A.theta(128, 1e4, A.LINEAR, 4.0), t / 4)
    # with the base scaled the slowest pair turns f times slower, the fastest as before
    b = A.theta(128, 1e4, A.BASE, 8.0)
    assert b[0] == 1.0 and abs(b[-1] / (t[-1] / 8) - 1) < 1e-12
    # by wavelength: fast pairs as they were, slow ones divided, monotone between
    w = A.theta(128, 5e5, A.WAVES, 8.0, 8192, 1.0, 4.0)
    t5 = A.theta(128, 5e5)
    wave = 2 * math.pi / t5
    np.testing.assert_allclose(w[wave < 2048], t5[wave < 2048])
    np.testing.assert_allclose(w[wave > 8192], t5[wave > 8192] / 8)
    assert np.all(np.diff(w) < 0)
    mid = (wave > 2048) & (wave < 8192)
    assert mid.any() and np.all(w[mid] < t5[mid]) and np.all(w[mid] > t5[mid] / 8)
    # by index: the same at the ends, a straight line of weights between
    r = A.theta(128, 1e4, A.RAMP, 16.0, 4096, 1.0, 32.0)
    weight = (t - r) / (t - t / 16)
    inner = (weight > 1e-9) & (weight < 1 - 1e-9)
    assert weight[0] < 1e-9 and abs(weight[-1] - 1) < 1e-9 and inner.sum() > 10
    np.testing.assert_allclose(np.diff(weight[inner], 2), 0, atol=1e-9)


@pytest.mark.parametrize("scaling", range(5))
@pytest.mark.parametrize("rot,base,f,L,low,high", [(128, 1e4, 8.0, 4096, 1.0, 32.0), (64, 5e6, 1.0, 16384, 1.0, 4.0),
                                                   (4, 1e4, 3.5, 100, 0.5, 1.5), (256, 5e5, 32.0, 8192, 1.0, 4.0)])
def test_the_librarys_angles(lib, scaling, rot, base, f, L, low, high):
    """64 bits on both sides: pow and log are off by a few units in the last place, the exponent
    -2 i / rot ln base (at most 16) carries its error into the angle: 64 eps is enough."""
    for layout in (0, 1):
        s = B.rope_spec(layout, rot, base, scaling, f, L, low, high)
        np.testing.assert_allclose(B.cb_rope_theta(s), A.theta(rot, base, scaling, f, L, low, high), rtol=64 * 2 ** -52)


def test_shared_attention_pins():
    g = np.random.default_rng(2)
    k, v = g.standard_normal((7, 2, 8)), g.standard_normal((7, 2, 8))
    ok, ov = g.standard_normal((3, 4, 2, 8)), g.standard_normal((3, 4, 2, 8))
    q = np.zeros((3, 2, 4, 8))
    out, _ = A.shared_attention(q, np.array([[-1, 0], [3, -2], [1, 2]]), [(k, v)], [0, 3], ok, ov)
    np.testing.assert_allclose(out[0, 0, 3], v[:, 1].mean(0))                                  # a zero query: the mean
    np.testing.assert_allclose(out[0, 1, 0], np.concatenate([v[:, 0], ov[0, :1, 0]]).mean(0))
    assert np.all(out[1, 1] == 0)
    # the same rows as one cache
    q = g.standard_normal((1, 1, 4, 8))
    a, _ = A.shared_attention(q, np.array([[3]]), [(k, v)], [0, 1], ok[:1], ov[:1])
    b, _ = A.shared_attention(q, np.array([[-1]]), [(np.concatenate([k, ok[0]]), np.concatenate([v, ov[0]]))], [0, 1],
                              ok[:1], ov[:1])
    np.testing.assert_allclose(a, b)


def test_sampling_by_hand():
    x = np.log([0.1, 0.4, 0.2, 0.3])
    s = lambda u, **kw: A.sample(x, u, **kw)[0]  # noqa: E731
    assert [s(u) for u in (0.0, 0.05, 0.15, 0.49, 0.55, 0.65, 0.75, 0.999)] == [0, 0, 1, 1, 2, 2, 3, 3]
    assert [s(u, top_k=2) for u in (0.0, 0.57, 0.58)] == [1, 1, 3]
    assert A.sample(x, 0.3, top_p=0.69)[2] == 2 and A.sample(x, 0.3, top_p=0.71)[2] == 3 and A.sample(x, 0.3, top_p=0.0)[2] == 1
    assert A.sample(x, 0.3, min_p=0.45)[2] == 3 and A.sample(x, 0.3, min_p=2.0)[2] == 1
    assert s(0.9, temperature=0) == 1 and A.sample(x, 0.9, temperature=0)[1:3] == (0.0, 1)
    assert abs(A.sample(x, 0.2)[1] - math.log(0.4)) < 1e-12
    # ties go to the lower id; ids at -inf do not exist
    assert A.sample([1, 3, 3, 3], 0.99, top_k=2)[0] == 2
    assert A.sample([-np.inf, -np.inf], 0.5)[:3] == (-1, -np.inf, 0) and A.sample([-np.inf, -900.0], 0.99)[0] == 1
    # a temperature flattens: shares follow x / T
    assert abs(math.exp(A.sample(x, 0.999, temperature=2.0)[1]) - 0.3 ** 0.5 / np.sqrt([0.1, 0.4, 0.2, 0.3]).sum()) < 1e-12
