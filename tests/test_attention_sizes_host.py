"""CPU checks of the sizes that the attention calls refuse before anything is enqueued."""
import ctypes

import pytest

import paged_fp8_kv_attn_b200 as pkv
from paged_fp8_kv_attn_b200 import build as pkv_build

A = ctypes.c_void_p(256)     # a non-null, aligned address; no call here reaches the device


@pytest.fixture(scope="module")
def lib():
    pkv_build.build()
    return pkv.library()


@pytest.mark.parametrize("kind", ["fp8", "bf16", "int4", "fp8_window", "int4_window", "fp8_prefix"])
def test_chunk_counts_beyond_32_bits(lib, kind):
    """A batch whose page tables hold 2^31 chunks of 64 tokens or more; one fewer request
    is refused for its missing workspace only."""
    pools = [A] * (4 if kind.startswith("int4") else 2)
    scales = [1.0, 1.0] if kind.startswith("fp8") else []
    window = [100, 4] if kind.endswith("window") else []
    more = [None] if kind == "fp8_prefix" else []

    def call(batch, max_pages, page):
        return getattr(lib, f"paged_decode_attn_{kind}")(
            A, *pools, *scales, A, max_pages, A, batch, 8, 4, 128, page, 8, 0.1, *window, None, A, A,
            None, 0, 0, *more, None)

    assert call(64, 1 << 24, 128) == 3 and b"2^31" in lib.pkv_last_error()
    assert call(63, 1 << 24, 128) == 2
    assert call(1, 2**31 - 1, 128) == 3
    assert call(4, 2**31 - 1, 16) == 3
    assert call(3, 2**31 - 1, 16) == 2


@pytest.mark.parametrize("kind", [pkv.PKV_KV_FP8, pkv.PKV_KV_BF16, pkv.PKV_KV_INT4])
def test_plan_refuses_what_the_call_refuses(lib, kind):
    out = [ctypes.c_int32(0) for _ in range(3)]
    plan = lambda batch, pages: lib.paged_decode_attn_plan(  # noqa: E731
        kind, batch, 8, 4, 128, pages, 128, 0, *[ctypes.byref(o) for o in out])
    assert plan(64, 1 << 24) == 3 and b"2^31" in lib.pkv_last_error()
    assert plan(1, 2**31 - 1) == 3
