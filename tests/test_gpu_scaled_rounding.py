"""GPU attention over block-scaled 8-bit caches: what an output loses besides its own
rounding to binary16 is float32's, in every route."""
import numpy as np
import pytest

from tests import refs
from tests import step_refs as R
from tests.test_gpu_scaled_attention import Decode, Prefill

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def attend(q, kc, vc, ks, vs, scale):
    """One KV head in 64 bits: (out, tolerance).

    Tolerance: half of binary16's step at the result, and the float32 errors that
    step_refs.attend derives, without a rounding of the weights to 11 bits: the score's 2^-19 S in numerator and denominator, the exponent's 2^-24
    |y|, exponential and logarithm 2^-21, joins and division 2^-20, and 2^-22 for
    weights of 22 bits (2^-31 of the largest where the second half is a subnormal)."""
    x = scale * (q @ kc.T) * ks
    w = np.exp(x - x.max(1, keepdims=True))
    w /= w.sum(1, keepdims=True)
    out, mag = (w * vs) @ vc, (w * vs) @ np.abs(vc)
    S = (scale * (np.abs(q) @ np.abs(kc).T) * ks).max(1, keepdims=True)
    bits = (np.abs(x).max(1, keepdims=True) + np.abs(np.log(np.maximum(vs, 2.0 ** -80))).max()) * 1.45
    rel = 2.0 ** -22 + 2 * (2.0 ** -19 * S + 2.0 ** -24 * bits + 2.0 ** -21) + 2.0 ** -20
    f32 = mag * rel + 2.0 ** -31 * (w * vs).max(1, keepdims=True) * np.abs(vc).sum(0)
    e = np.floor(np.log2(np.maximum(np.abs(out) + f32, 2.0 ** -14)))
    return out, 2.0 ** (e - 11) + f32


def _positive(c, seed):
    """Value codes of one sign and small scores, so that the float32 part of the tolerance is far
    below binary16's step."""
    rng = np.random.default_rng(seed)
    c.c.codes[1] = rng.integers(1, 120, c.c.codes[1].shape)              # E4M3 codes below NaN, too
    c.c.scales[0] *= 0.25
    return c


def _check(got, want, tol):
    off = np.abs(got - want) > tol
    assert not off.any(), f"{off.mean():.4f} of the outputs, by up to {(np.abs(got - want) / tol).max():.3f}"


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("kw", [dict(), dict(workspace=False), dict(force_splits=7)])
def test_decode(kind, kw):
    c = _positive(Decode([1, 2, 3, 5, 17, 64, 300, 700], kind=kind, spread=0.3, seed=30), 30)
    got, _ = c.run(**kw)
    for b, n in enumerate(c.lens):
        rows = [R.gather(c.c.codes[i], c.c.scales[i], c.table[b], np.arange(n), 16, 16, kind,
                         c.c.codes.shape[1]) for i in (0, 1)]
        for j in range(c.c.Hkv):
            h = slice(j * c.G, (j + 1) * c.G)
            want, tol = attend(c.q[b, h].astype(np.float64), rows[0][0][:, j], rows[1][0][:, j],
                               rows[0][1][:, j], rows[1][1][:, j], 1 / 16)
            _check(got[b, h], want, tol)


@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("rows", [3, 50, 400])
def test_prefill(rows, kind):
    """With and without clusters."""
    c = _positive(Prefill(rows, 40, 900, kind=kind, seed=31), 31)
    got, _ = c.run()
    for r in range(0, rows, max(1, rows // 8)):
        t = refs.prefill_tokens(c.sel[r], c.q_pos[r], c.kv_len)
        kc, ks = R.gather(c.c.codes[0], c.c.scales[0], c.table, t, 16, 16, kind, c.c.codes.shape[1])
        vc, vs = R.gather(c.c.codes[1], c.c.scales[1], c.table, t, 16, 16, kind, c.c.codes.shape[1])
        want, tol = attend(c.q[r].astype(np.float64), kc[:, 0], vc[:, 0], ks[:, 0], vs[:, 0], 1 / 16)
        _check(got[r], want, tol)
