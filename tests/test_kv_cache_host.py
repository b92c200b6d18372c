"""CPU-only checks of the paged KV cache: refusals of the C entry points (before any launch) and of the binding, the
oracle's layout against hand-placed bytes and its attention against a closed form."""
import ctypes
import math

import numpy as np
import pytest
import torch

import qad_nvfp4_quantize_b200 as nv
from oracle import kv_oracle as kv
from oracle import nvfp4_oracle as o

P16 = ctypes.c_void_p(256)   # never dereferenced: the checks come first
ODD = ctypes.c_void_p(264)


def test_page_bytes_and_workspaces():
    L = nv.lib()
    assert L.nvfp4_kv_page_bytes(16, 128) == 2304 and L.nvfp4_kv_page_bytes(64, 64) == 4 * 1152
    for page, dim in ((8, 128), (24, 128), (256, 128), (16, 96), (16, 256), (0, 64), (-16, 64)):
        assert L.nvfp4_kv_page_bytes(page, dim) == 0
    # 4.5 bits a value: 2 * 16 tokens * D values of a granule
    assert L.nvfp4_kv_page_bytes(16, 128) * 8 == 4.5 * 2 * 16 * 128
    assert L.nvfp4_paged_attention_workspace_bytes() > 0
    assert L.nvfp4_kv_compact_workspace_bytes(100) >= 400 and L.nvfp4_kv_compact_workspace_bytes(-1) == 0


APPEND = dict(k=P16, v=P16, stride=1024, total=4, heads=8, dim=128, cu=P16, kv_len=P16, batch=2, table=P16, width=4,
              pages=P16, num_pages=9, page=64, k_g=P16, v_g=P16, mode=0)


@pytest.mark.parametrize("change", [
    dict(dim=96), dict(dim=256), dict(page=48), dict(page=256), dict(heads=0), dict(total=-1), dict(batch=-1),
    dict(width=-1), dict(num_pages=-1), dict(stride=1020), dict(stride=512), dict(mode=2), dict(mode=7), dict(k=None),
    dict(v=None), dict(cu=None), dict(kv_len=None), dict(table=None), dict(pages=None), dict(k_g=None), dict(v_g=None),
    dict(k=ODD), dict(v=ODD), dict(pages=ODD), dict(width=1 << 26)])
def test_append_refusals(change):
    a = dict(APPEND, **change)
    assert nv.lib().nvfp4_kv_append(*a.values(), None) == 1


ATTN = dict(q=P16, stride=4096, total=4, hq=32, heads=8, dim=128, cu=P16, kv_len=P16, batch=2, table=P16, width=4,
            pages=P16, num_pages=9, page=64, k_g=P16, v_g=P16, scale=0.1, causal=1, window=0, max_q=0,
            out=ctypes.c_void_p(512), lse=None, ws=P16, nbytes=1 << 30)


@pytest.mark.parametrize("change,status", [
    (dict(dim=192), 1), (dict(page=8), 1), (dict(hq=20), 1), (dict(hq=0), 1), (dict(hq=8 * 129, stride=8 * 129 * 128), 1),
    (dict(heads=-8), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=math.inf), 1), (dict(scale=math.nan), 1),
    (dict(window=-1), 1), (dict(max_q=-1), 1), (dict(stride=4088), 1), (dict(stride=4100), 1), (dict(q=None), 1),
    (dict(q=ODD), 1), (dict(out=None), 1), (dict(out=P16), 1), (dict(out=ODD), 1), (dict(cu=None), 1),
    (dict(pages=None), 1), (dict(table=None), 1), (dict(k_g=None), 1), (dict(total=1 << 31), 1), (dict(ws=None), 4),
    (dict(nbytes=16), 4), (dict(ws=ODD), 4)])
def test_attention_refusals(change, status):
    a = dict(ATTN, **change)
    assert nv.lib().nvfp4_paged_attention(*a.values(), None) == status


def test_pool_refusals():
    L = nv.lib()
    pool = (P16, 10, P16, 4, 8, P16, 16)
    assert L.nvfp4_kv_fork(None, *pool[1:], P16, P16, 2, P16, ODD, None) == 1
    assert L.nvfp4_kv_fork(*pool, P16, P16, -1, P16, ODD, None) == 1
    assert L.nvfp4_kv_fork(*pool, P16, P16, 2, P16, P16, None) == 1                 # src and dst the same
    assert L.nvfp4_kv_fork(*pool[:6], 0, P16, P16, 2, P16, ODD, None) == 1          # page size 0
    assert L.nvfp4_kv_fork(*pool, P16, P16, (1 << 20) + 1, P16, ODD, None) == 1
    assert L.nvfp4_kv_free(*pool, None, 2, None) == 1
    assert L.nvfp4_kv_free(*pool, P16, -2, None) == 1
    assert L.nvfp4_kv_free(P16, -1, *pool[2:], P16, 2, None) == 1
    outs = (P16, P16, P16, ODD, P16)
    assert L.nvfp4_kv_compact(P16, 0, *pool[2:], *outs, P16, 1 << 20, None) == 1    # an empty pool
    assert L.nvfp4_kv_compact(*pool, *outs, None, 1 << 20, None) == 4
    assert L.nvfp4_kv_compact(*pool, *outs, P16, 8, None) == 4
    assert L.nvfp4_kv_compact(*pool, P16, None, P16, ODD, P16, P16, 1 << 20, None) == 1
    assert L.nvfp4_kv_copy_pages(P16, 10, 24, P16, P16, 1, None) == 1               # not whole 16-byte vectors
    assert L.nvfp4_kv_copy_pages(P16, 10, 0, P16, P16, 1, None) == 1
    assert L.nvfp4_kv_copy_pages(ODD, 10, 32, P16, P16, 1, None) == 1
    assert L.nvfp4_kv_copy_pages(P16, 10, 32, None, P16, 1, None) == 1
    assert L.nvfp4_kv_copy_pages(P16, 10, 32, P16, P16, -1, None) == 1


def test_binding_refuses_host_tensors_and_odd_sizes():
    g = torch.ones(1)
    with pytest.raises(ValueError):
        nv.kv_cache(4, 2, 96, 16, g, g)
    with pytest.raises(ValueError):
        nv.kv_cache(4, 2, 64, 24, g, g)
    cache = nv.kv_cache(4, 2, 64, 16, g, g)               # on the host: made, but no kernel takes it
    assert cache.pages.shape == (4, 2, 1152) and not cache.pages.any()
    x = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    ints = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        nv.kv_append(cache, x, x, ints[None], ints, ints[:1])
    with pytest.raises(ValueError):
        nv.paged_attention(x, cache, ints[None], ints, ints[:1])
    with pytest.raises(ValueError):
        nv.kv_free(ints, ints[None], ints[:1], ints, 16)


def test_status_strings():
    L = nv.lib()
    assert L.nvfp4_status_string(9).startswith(b"KV cache") and L.nvfp4_status_string(10).endswith(b"free pages")


# ------------------------------------------------------------- the oracle itself
def test_oracle_layout_by_hand():
    D, page = 64, 32
    pages = np.zeros((2, 1, page // 16 * 18 * D), np.uint8)
    x = np.zeros((1, 1, D), np.float32)
    x[0, 0, :2] = [6.0, -1.5]
    # token 17 of sequence 0 lies in page 1, slot ... position 17 -> page table entry 0, granule 1, row 1
    kv.append(pages, x, 2 * x, [[1]], [0, 1], [18], 1.0, 1.0, page, "max")
    gr = pages[1, 0].reshape(2, 18 * D)[1]
    assert gr[1 * 32] == 0xB7                       # -1.5 -> 0xB in the high nibble, 6 -> 7 in the low one
    assert gr[8 * D + 4] == 0x38                    # scale 1.0 = E4M3 0x38
    assert gr[9 * D + 32] == 0xB7 and gr[17 * D + 4] == 0x40   # V: the same codes, scale 2.0
    assert not pages[0].any()
    K, V = kv.gather(pages, [1], 18, page, D, 1.0, 0.5)
    assert K[0, 17, 0] == 6.0 and K[0, 17, 1] == -1.5 and V[0, 17, 0] == 6.0 and not K[0, :17].any()


def test_oracle_attention_closed_form():
    # equal keys: the softmax is uniform over the visible tokens, out is their mean
    D, page = 64, 16
    rng = np.random.default_rng(0)
    pages = np.zeros((3, 1, 18 * D), np.uint8)
    k = np.ones((40, 1, D), np.float32)
    v = o.bf16_round(rng.standard_normal((40, 1, D)).astype(np.float32))
    table = [[2, 0, 1]]
    kv.append(pages, k, v, table, [0, 40], [40], 0.01, 0.002, page, "max")
    K, V = kv.gather(pages, table[0], 40, page, D, 0.01, 0.002)
    q = np.ones((3, 2, D), np.float32)
    r = kv.attention(q, pages, table, [0, 3], [40], 0.01, 0.002, page, 0.25, True, 5)
    for i, pos in enumerate((37, 38, 39)):
        np.testing.assert_allclose(r["out"][i, 1], V[0, pos - 4:pos + 1].mean(0), rtol=1e-12)
        np.testing.assert_allclose(r["lse"][i, 0], 0.25 * K[0, 0].sum() + math.log(5), rtol=1e-12)
    # more new tokens than cached ones: the first positions do not exist and see nothing
    r = kv.attention(np.ones((4, 2, D), np.float32), pages, table, [0, 4], [2], 0.01, 0.002, page, 0.25, True, 0)
    assert not r["out"][:2].any() and np.isneginf(r["lse"][:2]).all() and np.isfinite(r["lse"][2:]).all()


def test_oracle_pool_round_trip():
    refs, table = np.array([1, 0, 1, 0, 1, 0, 0]), np.array([[2, 4, 0, -1], [-1] * 4, [-1] * 4])
    lens = [40, 0, 0]
    src, dst, st = kv.fork(refs, table, lens, [0, 0], [2, 1], 16)
    assert (src, dst, st) == ([0, 0], [1, 3], 0)
    assert refs.tolist() == [1, 1, 3, 1, 3, 0, 0] and table[2].tolist() == [2, 4, 1, -1]
    kv.free(refs, table, lens, [0, 2], 16)
    assert refs.tolist() == [0, 0, 1, 1, 1, 0, 0]
    r, t, s, d, live = kv.compact(refs, table, lens, 16)
    assert (s, d, live) == ([3, 4], [0, 1], 3) and r.tolist() == [1, 1, 1, 0, 0, 0, 0] and t[1].tolist() == [2, 1, 0, -1]
    assert kv.fork(refs, table, lens, [1] * 5, [0, 2, 0, 1, 7], 16)[2] == 9
