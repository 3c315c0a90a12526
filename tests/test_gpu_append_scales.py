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
