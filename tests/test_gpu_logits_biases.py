"""GPU logits: long bias lists whose tokens have many entries each."""
import numpy as np
import pytest

from tests.test_gpu_logits import _check, _logits, _rules

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _repeated(B, V, n, seed, each):
    """n entries in rising order of their token, `each` of them to a token."""
    k = _rules(B, V, 100, n, seed)
    k["bias_tokens"] = np.tile((np.arange(n) // each % V).astype(np.int32), (B, 1))
    return k


@pytest.mark.parametrize("dtype", ["float32", "float16"])
@pytest.mark.parametrize("B,V,n,each", [(2, 2048, 5000, 7), (1, 70000, 3000, 2), (3, 33, 1000, 30), (2, 4099, 600, 600)])
def test_tokens_with_many_biases(B, V, n, each, dtype):
    k = _repeated(B, V, n, n, each)
    rng = np.random.default_rng(n)
    k["bias_tokens"][-1] = rng.permutation(k["bias_tokens"][-1])
    k["bias_tokens"][:, ::11] = -1
    x = _logits(B, V, dtype, n)
    a = _check(x, k)
    if dtype == "float32":
        assert bool((_check(x.clone(), k, out=x) == a).all())


def test_time_of_long_lists():
    """The work grows with the number of entries, not with its square: with 262,144 entries of 2048
    tokens every thread sweeps the list four times (seconds when every entry looked for its token's
    first one)."""
    import torch
    import fp8_kv_cache_gb300 as P
    n = 1 << 18
    x, k = _logits(1, 2048), _repeated(1, 2048, n, 1, 128)
    _check(x, k)
    tokens, values = torch.from_numpy(k["bias_tokens"]).cuda(), torch.from_numpy(k["bias_values"]).cuda()
    times = []
    for _ in range(3):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        P.paged_gqa_logits_process(x, bias_tokens=tokens, bias_values=values)
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    assert min(times) < 100, f"{times} ms"
