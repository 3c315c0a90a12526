"""GPU quantising append into blocks whose stored scales were not written by it: every
code and scale against the 64-bit definition."""
import numpy as np
import pytest

from tests import step_refs as R
from tests.test_gpu_append import Case, D

pytestmark = pytest.mark.gpu

TYPES = ["float16", "bfloat16", "float32"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _begun(scales, kind="e4m3", dtype="float32", step=False, page=16, **kw):
    """One sequence for each value of `scales` ([B] or [B, Hkv]), its begun first block holding 5 rows of
    that scale; one new row each, or three."""
    import torch
    scales = np.asarray(scales, np.float32)
    B = scales.shape[0]
    c = Case([5] * B, [1 if step else 3] * B, kind=kind, dtype=dtype, page=page, block=16, **kw)
    for s in c.sc:
        s[torch.from_numpy(c.table[:, 0]).long().cuda(), 0] = torch.from_numpy(scales.reshape(B, -1)).cuda()
    return c


def _check(c, step):
    want, flags = c.want()
    assert c.run(plain=step) == flags
    c.same(want)


@pytest.mark.parametrize("step", [True, False])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_tiny_stored_scales(kind, dtype, step):
    """Scales down to the smallest subnormal, under rows of zeros (which keep them) and under small rows."""
    import torch
    tiny = [2.0 ** -e for e in (120, 125, 126, 127, 128, 129, 140, 149)] + [3e-39, 1.1e-38, 9e-45, 1e-37]
    c = _begun(tiny * 3, kind, dtype, step, Hkv=3)
    n = len(tiny) * (1 if step else 3)
    for x in c.rows:
        x[:n] = 0
        x[:n, 1] = -0.0
        # in units of the scales where the type has such numbers, else its smallest
        x[n:2 * n] = (x[n:2 * n].double() * 2.0 ** -126).to(x.dtype)
        x[2 * n:, 0] = 0
        x[2 * n:, 1] = torch.finfo(x.dtype).smallest_normal * torch.finfo(x.dtype).eps
    _check(c, step)
    if kind == "e4m3":
        for t in c.kv:
            new = t[torch.from_numpy(c.table[:, 0]).long().cuda(), 5:6 if step else 8]
            assert not bool(((new & 127) == 127).any())


def _midpoints(kind):
    """The midpoints of neighbouring codes and the float32 numbers next to them, of both signs."""
    values = R._E4M3 if kind == "e4m3" else np.arange(128.0)
    mid = (values[1:] + values[:-1]) / 2
    return np.concatenate([mid, -mid])


@pytest.mark.parametrize("step", [True, False])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_stored_scales_that_are_no_powers_of_two(kind, dtype, step):
    """Quotients at and next to every midpoint of the codes, under scales such as amax / 448."""
    import torch
    scales = np.concatenate([[0.1, 1 / 3, 0.7, 1.1, 3.0 / 448, 2.0 ** -6 * 1.5, np.nextafter(np.float32(0.25), np.float32(1)),
                              np.nextafter(np.float32(0.25), np.float32(0))],
                             np.random.default_rng(1).uniform(0.001, 2, 24)]).astype(np.float32)
    c = _begun(scales, kind, dtype, step, Hkv=1)
    t = getattr(torch, dtype)
    mid = _midpoints(kind)
    n = 1 if step else 3
    for x in c.rows:
        for b, s in enumerate(scales):
            v = torch.from_numpy(mid * float(s)).to(t)           # the nearest, or the one before or after it
            if dtype == "float32":
                v = torch.cat([v, torch.nextafter(v, torch.zeros_like(v)), torch.nextafter(v, 2 * v)])
            v = v[torch.randperm(v.numel(), generator=torch.Generator().manual_seed(b))][:n * D]
            x.view(-1)[b * n * D:b * n * D + v.numel()] = v.cuda()
    for i in (0, 1):                                             # no row's largest outgrows its stored scale
        top = 448 if kind == "e4m3" else 127
        limit = torch.from_numpy(np.repeat(scales, n) * np.float32(top) * 0.999).cuda()[:, None, None]
        c.rows[i].copy_(torch.minimum(torch.maximum(c.rows[i].float(), -limit), limit).to(t))
    _check(c, step)


@pytest.mark.parametrize("route", ["step", "ragged", "single"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_infinities_in_blocks_of_zeros(kind, dtype, route):
    """Nothing finite but zeros: the scale is 0, and so is every code but those of NaN; flagged."""
    import torch
    block = 1 if route == "single" else 16
    c = Case([0] * 6, [1] * 6 if route == "step" else [5] * 6, kind=kind, dtype=dtype, block=block, seed=40)
    n = 1 if route == "step" else 5
    inf, nan = float("inf"), float("nan")
    for x in c.rows:
        x.zero_()
        x[0::n, 0, 3], x[0::n, 1, 255], x[0::n, 1, 254] = inf, -inf, -0.0
        x[2 * n, 1, 9] = nan
        x[3 * n:4 * n] = 0
        x[4 * n, 0, 8], x[4 * n, 1, 8] = 3.0, -2.0               # a block with a scale: infinities saturate
    assert c.run(plain=route == "step") == R.BAD_VALUE
    for t, s, x in zip(c.kv, c.sc, c.rows):
        t, s, x = t.cpu().numpy(), s.cpu().numpy(), x.double().cpu().numpy()
        for b in range(6):
            p = c.table[b, 0]
            got, new = t[p, :n], x[b * n:(b + 1) * n]
            scale = s[p, :n] if block == 1 else np.broadcast_to(s[p, 0], (n, 2))
            zero = scale == 0
            m = np.abs(np.where(np.isfinite(new), new, 0)).max(-1)
            assert np.array_equal(zero, (m if block == 1 else np.broadcast_to(m.max(0), m.shape)) == 0)
            if kind == "int8":
                want = R.encode(np.where(zero[..., None], np.where(np.isnan(new), np.nan, 0),
                                         new / np.where(zero, 1, scale)[..., None].astype(np.float64)), kind)
                assert np.array_equal(got, want)
            else:
                assert np.array_equal((got & 127) == 127, np.isnan(new))
                assert np.all((got & 127)[zero[..., None] & ~np.isnan(new)] == 0)
                assert np.all((got & 127)[~zero[..., None] & np.isinf(new)] == 126)


@pytest.mark.parametrize("route", ["step", "ragged"])
def test_e4m3_rows_of_subnormal_scales_coded_again(route):
    """code * s_old at and next to every midpoint of the new codes, below float32's normal numbers."""
    import torch
    values, rng = R._E4M3, np.random.default_rng(2)
    mid = (values[1:] + values[:-1]) / 2
    olds, codes = [], []
    for m in mid:                                                # code * k 2^-149 / 2^-126 next to the midpoint
        for i in rng.choice(np.arange(1, 127), 12, replace=False):
            k = int(round(m / values[i] * 2.0 ** 23)) + int(rng.integers(-1, 2))
            if 0 < k < 1 << 23:
                olds.append(k * 2.0 ** -149)
                codes.append(i)
    olds += [2.0 ** -e for e in (60, 61, 100, 118, 126, 149)] + [1.3 * 2.0 ** -59, 1e-30, 3e-36]
    codes += [7] * 9
    step = route == "step"
    c = _begun(olds, "e4m3", "float32", step, Hkv=1)
    n = 1 if step else 3
    for x, t in zip(c.rows, c.kv):
        x[:] = (x.double() * 2.0 ** -127).float()                # the new scale: 2^-126
        x[-9 * n:] = 1.0                                         # and 2^-8
        pages = torch.from_numpy(c.table[:, 0]).long().cuda()
        held = t[pages, :5]
        held[..., ::2] = torch.tensor(codes, dtype=torch.uint8, device="cuda")[:, None, None, None]
        held[..., 1::2] = held[..., ::2] | 128
        t[pages, :5] = held
    _check(c, step)


@pytest.mark.parametrize("step", [True, False])
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
def test_scales_that_grow_from_zero(kind, step):
    """Rows stored under a scale of 0 are code * 0 / s: zeros of their signs, and NaN stays NaN."""
    import torch
    c = _begun(np.zeros(20, np.float32), kind, "float16", step, Hkv=2)
    if kind == "e4m3":
        for t in c.kv:
            t[torch.from_numpy(c.table[::2, 0]).long().cuda(), 3, 1, ::9] = 0x7F
    _check(c, step)
    if kind == "e4m3":
        for t, s in zip(c.kv, c.sc):
            got = t.cpu().numpy()[c.table[::2, 0], 3, 1]
            assert np.all((got & 127)[:, ::9] == 127) and np.all(s.cpu().numpy()[c.table[:, 0], 0] > 0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["e4m3", "int8"])
@pytest.mark.parametrize("block,B,rows", [(16, 3300, 1), (1, 40, 90), (3, 20, 7), (8, 20, 11), (32, 12, 40),
                                          (64, 12, 70), (392, 6, 500)])
def test_every_route(block, B, rows, kind, dtype):
    """Odd stored scales, zeros and infinities where warps take one unit or several, and where one, two or
    more warps share a unit of few or many rows."""
    import torch
    page = 784 if block == 392 else 48 if block == 3 else 64 if block > 16 else 16
    start = min(2, block - 1)
    c = Case([start] * B, [rows] * B, Hkv=3, kind=kind, dtype=dtype, page=page, block=block, seed=block)
    odd = np.float32([0.1, 2.0 ** -140, 1.1, 0.0, 2.0 ** -6, 3e-39, 1 / 3, 2.0 ** -126])
    pages = torch.from_numpy(c.table[:, 0]).long().cuda()
    for s in c.sc:
        s[pages, 0] = torch.from_numpy(np.resize(odd, (B, 3))).cuda()
    given = []
    for x in c.rows:
        v = x.view(B, rows, 3, D)
        v[::3, :, 0], v[1::3, :, 1], v[2::3, :, 2] = 0, 0, -0.0
        v[::5] *= 40
        v[0, 0, 0, 7] = v[B - 1, rows - 1, 0, 7] = 0
        given.append(x.clone())
        for b, r in ((0, 0), (B - 1, rows - 1)):
            given[-1].view(B, rows, 3, D)[b, r, 0, 7] = float("inf")
    # an infinity does not count for the scale, and under a scale of 0 it is coded as 0
    for x, (_, scales) in zip(c.rows, c.want()[0]):
        for b, r in ((0, 0), (B - 1, rows - 1)):
            at = start + r
            if scales[c.table[b, at // page], at % page // block, 0] > 0:
                x.view(B, rows, 3, D)[b, r, 0, 7] = float("inf")
    want, flags = c.want()
    c.rows = given
    assert c.run(plain=rows == 1) == flags | R.BAD_VALUE
    c.same(want)
