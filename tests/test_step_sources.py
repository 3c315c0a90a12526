"""What the step kernels' sources have to keep to, checked without a GPU."""
import os
import re

import pytest

from fp8_kv_cache_gb300 import build as B

STEP = ["append.cu", "decode_scaled.cu", "logits.cu", "prefill_scaled.cu", "rope.cu", "scaled_core.cuh"]


def _code(name):
    text = open(os.path.join(B.CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))


@pytest.mark.parametrize("name", STEP)
def test_no_reads_by_the_read_only_path(name):
    """A step kernel may start while the kernel before it still writes what it reads; the read-only path
    is for data that does not change while a kernel lives, and its loads may pass the wait."""
    code = _code(name)
    assert not re.findall(r"__ldg|ldg_stream|\bld\.global\.nc|\.nc\b|__restrict__|__ldcs|tex1D", code)
    for helper in ("table_page", "prefill_entry"):
        assert not re.findall(rf"\b{helper}\s*\(", code), f"{helper} by its default, the read-only path"
    assert "token_row_offset" not in code and "WarpRing" not in code    # shared helpers that read that way


def test_shared_helpers_have_an_ordinary_form():
    code = _code("pgqa_device.cuh")
    for helper in ("table_page", "prefill_entry"):
        body = re.search(rf"template <bool kStable = true>\s*__device__ __forceinline__ \w+ {helper}\(.*?\n}}", code,
                         flags=re.S).group(0)
        assert "__ldg" not in body and "<kStable>" in body


def test_every_step_kernel_waits_for_the_kernel_before_it():
    for name in STEP[:-1]:
        code = _code(name)
        kernels = re.findall(r"__global__.*?\n}", code, flags=re.S)
        assert kernels and all("enter();" in k for k in kernels), name
