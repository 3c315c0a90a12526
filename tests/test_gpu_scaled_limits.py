"""GPU attention over block-scaled 8-bit caches at the ends of its arguments' ranges."""
import pytest

pytestmark = pytest.mark.gpu

D = 256


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("length", [2 ** 31 - 1, 2 ** 31 - 16])
def test_the_longest_sequence(length):
    """2^31 - 1 tokens, of which two pages are in the pool, the first and the last: the weighted mean over
    them.  The tolerance is half a step of binary16 and 820 sums in a row of a warp's tiles."""
    import torch
    import fp8_kv_cache_gb300 as P
    page, G = 1 << 16, 3
    g = torch.Generator(device="cuda").manual_seed(0)
    codes = [torch.randint(lo, 128, (1, page, 1, D), device="cuda", generator=g).to(torch.int8) for lo in (-127, 1)]
    sc = [torch.full((1, page // 16, 1), s, device="cuda") for s in (2e-4, 0.01)]
    table = torch.full((1, 1 << 15), -1, dtype=torch.int32, device="cuda")
    table[0, 0] = table[0, -1] = 0
    q = torch.randn(1, G, D, device="cuda", generator=g).half()
    lens = torch.tensor([length], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = P.paged_gqa_decode_scaled(q, *codes, *sc, table, lens, page, 1 / 16, err_flag=err,
                                    max_seq_len=2 ** 31 - 1)
    last = length - (2 ** 31 - page)                             # tokens of the last page
    k, v = (torch.cat([c[0, :, 0], c[0, :last, 0]]).double() * float(s[0, 0, 0]) for c, s in zip(codes, sc))
    want = torch.softmax(q[0].double() @ k.T / 16, -1) @ v
    assert int(err.item()) == 1
    assert bool(((out[0].double() - want).abs() <= want * (2.0 ** -11 + 2.0 ** -13)).all())


@pytest.mark.parametrize("B", [3, 4096, 4097])
def test_forced_splits_where_there_is_no_split(B):
    """Without a workspace, or for more than 4096 sequences, force_splits changes nothing, not a bit."""
    import torch
    import fp8_kv_cache_gb300 as P
    g = torch.Generator(device="cuda").manual_seed(B)
    codes = [torch.randint(-127, 128, (64, 16, 1, D), device="cuda", generator=g).to(torch.int8) for _ in (0, 1)]
    sc = [torch.full((64, 1, 1), 0.01, device="cuda") for _ in (0, 1)]
    table = torch.randint(0, 64, (B, 4), device="cuda", generator=g).int()
    lens = torch.randint(0, 65, (B,), device="cuda", generator=g).int()
    q = torch.randn(B, 2, D, device="cuda", generator=g).half()

    def call(**kw):
        return P.paged_gqa_decode_scaled(q, *codes, *sc, table, lens, 16, 1 / 16, **kw)

    plain = call(workspace=False)
    assert torch.equal(call(workspace=False, force_splits=5), plain)
    forced = call(force_splits=5)
    assert torch.equal(forced, plain) or B <= 4096
    assert bool(((forced.double() - plain.double()).abs() <= 2.0 ** -10 * plain.double().abs() + 2.0 ** -24).all())
