"""CPU-only checks of the paged KV cache's borders: what the C entry points refuse before any launch."""
import os

import pytest

import qad_nvfp4_quantize_b200 as nv
from tests.test_kv_cache_host import APPEND, ATTN


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_tables_of_nearly_2_31_tokens(page):
    # token indexes, up to two tiles of 128 behind the last one, are 32-bit numbers
    most = (1 << 31) // page - 256 // page
    L = nv.lib()
    for width, status in ((most, 4), (most + 1, 1), ((1 << 31) // page - 1, 1), ((1 << 31) // page, 1)):
        # (without a workspace: what is not refused for its sizes ends there)
        assert L.nvfp4_paged_attention(*dict(ATTN, page=page, width=width, ws=None).values(), None) == status
    for width in (most + 1, (1 << 31) // page - 1):
        assert L.nvfp4_kv_append(*dict(APPEND, page=page, width=width).values(), None) == 1


def test_attention_timeout_self_test_refuses_its_limits():
    # (no limit, more than 10 s; a workspace that is missing ends what is not refused for its limit)
    for limit, status in ((0, 1), (10_000_000_001, 1), (1_000_000, 4)):
        assert nv.lib().nvfp4_selftest_attention_timeout(*dict(ATTN, ws=None).values(), limit, None) == status


def test_every_kernel_of_the_cache_checks_its_computed_indexes():
    # the bounds-checking build is worth what its sources check: table entries, pages, moves, rows of results
    csrc = os.path.join(os.path.dirname(nv.__file__), "csrc")
    for name, least in (("kv_append.cu", 3), ("kv_attention.cu", 3), ("kv_prefill.cu", 4), ("kv_pages.cu", 12)):
        with open(os.path.join(csrc, name)) as f:
            text = f.read()
        assert text.count("NVFP4_IN_BOUNDS(") >= least, name
