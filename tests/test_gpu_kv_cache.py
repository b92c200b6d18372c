"""Paged NVFP4 KV cache on the GPU against the CPU oracle (oracle/kv_oracle.py): appending bit for bit, attention within
bounds derived from its roundings, the page pool's state exactly."""
import numpy as np
import pytest
import torch

from oracle import kv_oracle as kv
from tests.util import bf16_np, require_gpu, to_np

pytestmark = pytest.mark.gpu

KG, VG = 0.11, 0.07          # global scales of the attention tests' random pages


@pytest.fixture(scope="module")
def nv():
    return require_gpu()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def scalars(*g):
    return [torch.tensor([x], dtype=torch.float32, device="cuda") for x in g]


def tables(rng, lens, page, spare=2, extra=1):
    """Random distinct pages for each sequence, -1 behind them; (table, pool size)."""
    need = [-(-int(x) // page) for x in lens]
    P = sum(need) + spare
    ids = rng.permutation(P)
    table = np.full((len(lens), max(need) + extra), -1, np.int64)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, P


def random_pages(rng, P, heads, page, D):
    """Random codes; E4M3 scales of 0.5 to 2 (keys and values of about 1 under KG, VG)."""
    pages = rng.integers(0, 256, (P, heads, page // 16, 18 * D), dtype=np.uint8)
    for base in (8 * D, 17 * D):
        pages[..., base:base + D] = rng.integers(48, 65, pages.shape[:3] + (D,), dtype=np.uint8)
    return pages.reshape(P, heads, -1)


def queries(rng, T, hq, D, pad=0):
    """BF16 queries; pad > 0: as the first part of wider rows (a projection's output)."""
    x = torch.from_numpy(rng.standard_normal((T, hq + pad, D)).astype(np.float32)).to(torch.bfloat16)
    return x.cuda()[:, :hq], bf16_np(x[:, :hq])


def cumulative(new):
    return [0] + np.cumsum(new).tolist()


# ------------------------------------------------------------------ appending
@pytest.mark.parametrize("D,page,heads,new,before,mode", [
    (128, 16, 8, [1], [0], "max"),
    (128, 64, 2, [1, 0, 1, 1], [63, 5, 64, 1000], "max"),
    (64, 32, 3, [7, 33, 0, 1], [0, 31, 9, 16], "four_over_six"),
    (128, 128, 1, [300, 17], [100, 0], "four_over_six"),
    (64, 16, 5, [1] * 70, list(range(70)), "max"),
])
def test_append_matches_the_oracle(nv, D, page, heads, new, before, mode):
    rng = np.random.default_rng(D + page + len(new))
    T, lens = sum(new), [a + b for a, b in zip(new, before)]
    table, P = tables(rng, lens, page)
    # K and V inside one wider row, heavy tails: many blocks beyond the static scale's range
    qkv = torch.from_numpy((rng.standard_t(3, (T + 3, 2 * heads + 1, D))).astype(np.float32)).to(torch.bfloat16)
    dev = qkv.cuda()
    k, v = dev[:, 1:1 + heads], dev[:, 1 + heads:]
    pages = rng.integers(0, 256, (P, heads, nv.kv_page_bytes(page, D)), dtype=np.uint8)
    kg, vg = scalars(0.003, 0.0007)
    cache = nv.KVCache(torch.from_numpy(pages).cuda(), kg, vg, page, D)
    nv.kv_append(cache, k, v, ints(table), ints(cumulative(new)), ints(lens), mode=mode)
    ref = pages.copy()
    kn, vn = bf16_np(qkv[:, 1:1 + heads]), bf16_np(qkv[:, 1 + heads:])
    kv.append(ref, kn, vn, table, cumulative(new), lens, 0.003, 0.0007, page, mode)   # rows behind the last: left out
    assert np.array_equal(to_np(cache.pages), ref)
    assert nv.device_status() == 0


def test_append_equals_quantize_with_the_same_scale(nv):
    rng = np.random.default_rng(3)
    T, H, D, page = 128, 4, 128, 64
    x = torch.from_numpy(rng.standard_normal((T, H, D)).astype(np.float32)).to(torch.bfloat16).cuda()
    kg, vg = scalars(0.002, 0.001)
    cache = nv.kv_cache(2, H, D, page, kg, vg)
    nv.kv_append(cache, x, x, ints([[1, 0]]), ints([0, T]), ints([T]), mode="four_over_six")
    kc, _, vc, _ = kv.granule_views(to_np(cache.pages), page, D)
    for c, g in ((kc, kg), (vc, vg)):
        q = nv.quantize(x.reshape(T * H, D), "four_over_six", g=g)
        got = np.concatenate([c[1], c[0]], 1).transpose(1, 0, 2).reshape(T * H, D // 2)
        assert np.array_equal(got, to_np(q.codes))


def test_append_non_finite_values_and_bad_positions(nv):
    D, page = 64, 16
    kg, vg = scalars(0.01, 0.01)
    cache = nv.kv_cache(3, 1, D, page, kg, vg)
    x = torch.ones((3, 1, D), dtype=torch.bfloat16, device="cuda")
    x[1, 0, 20] = float("inf")
    x[2, 0, 40] = float("nan")
    nv.kv_append(cache, x, torch.ones_like(x), ints([[2]]), ints([0, 3]), ints([3]))
    assert nv.device_status() == 5
    kc, ks, vc, vs = kv.granule_views(to_np(cache.pages), page, D)
    assert not kc[2, 0, 1, 8:16].any() and ks[2, 0, 1, 1] == 1 and kc[2, 0, 1, :8].all()    # that block only
    assert not kc[2, 0, 2, 16:24].any() and ks[2, 0, 2, 2] == 1 and vs[2, 0, :3].min() > 1
    # a page outside the pool, a table too short, more new tokens than cached ones, offsets beyond the rows
    one = torch.ones((2, 1, D), dtype=torch.bfloat16, device="cuda")
    for table, cu, lens in (([[3]], [0, 2], [2]), ([[-1]], [0, 2], [2]), ([[0]], [0, 2], [17]), ([[0]], [0, 2], [1]),
                            ([[0]], [0, 3], [3]), ([[0]], [2, 1], [3]), ([[0]], [0, 2], [-4])):
        cache.pages.zero_()
        nv.kv_append(cache, one, one, ints(table), ints(cu), ints(lens))
        assert nv.device_status() == 9, (table, cu, lens)
        kept = to_np(cache.pages)
        if lens == [1]:      # the token that has a position is there
            assert kept[0].any()
        elif lens != [17]:   # a length beyond the table is cut to it
            assert not kept.any(), (table, cu, lens)


# ------------------------------------------------------------------ attention
def check(nv, rng, D, page, hq, heads, new, lens, causal=True, window=0, scale=None, pad=0, max_q=None, spread=1.0):
    T = sum(new)
    table, P = tables(rng, lens, page)
    pages = random_pages(rng, P, heads, page, D)
    q, qn = queries(rng, T, hq, D, pad)
    if spread != 1.0:
        q, qn = (q * spread).to(torch.bfloat16), None
        qn = bf16_np(q)
    kg, vg = scalars(KG, VG)
    cache = nv.KVCache(torch.from_numpy(pages).cuda(), kg, vg, page, D)
    out, lse = nv.paged_attention(q, cache, ints(table), ints(cumulative(new)), ints(lens), scale=scale, causal=causal,
                                  window=window, max_q=max_q, want_lse=True)
    ref = kv.attention(qn, pages, table, cumulative(new), lens, KG, VG, page, D ** -0.5 if scale is None else scale,
                       causal, window)
    compare(out, lse, ref, D)
    assert nv.device_status() == 0


def compare(out, lse, ref, D):
    tol_o, tol_l = kv.attention_tolerance(ref, D)
    err = np.abs(bf16_np(out).astype(np.float64) - ref["out"])
    assert np.isfinite(err).all() and (err <= tol_o).all(), float((err / np.maximum(tol_o, 1e-300)).max())
    if lse is not None:
        got, want = to_np(lse).astype(np.float64), ref["lse"]
        assert np.array_equal(np.isneginf(got), np.isneginf(want))
        some = np.isfinite(want)
        err = np.abs(got[some] - want[some])
        assert (err <= tol_l[some]).all(), float((err / tol_l[some]).max())


SHAPES = [
    # D, page, q heads, kv heads, new tokens, cached tokens
    (128, 16, 8, 2, [1], [1]),
    (128, 16, 4, 4, [1, 1, 1], [15, 16, 17]),
    (64, 64, 6, 2, [1, 1], [200, 63]),                     # three query heads a KV head
    (128, 32, 5, 1, [3, 1, 0, 2], [100, 1, 77, 2]),        # five; a sequence without new tokens
    (64, 16, 16, 2, [5, 2], [40, 333]),
    (128, 128, 16, 1, [2, 1], [129, 700]),                 # sixteen rows of one token
    (64, 128, 1, 1, [20], [64]),
    (128, 64, 40, 8, [37, 1, 64], [37, 500, 130]),         # a prompt from its start, a decode, a chunk
    (64, 32, 7, 7, [130], [257]),
    (128, 16, 24, 8, [4, 4], [5, 4]),
]


@pytest.mark.parametrize("D,page,hq,heads,new,lens", SHAPES)
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 19), (False, 33)])
def test_attention_matches_the_oracle(nv, D, page, hq, heads, new, lens, causal, window):
    for max_q in (None, 1, max(new)):        # the kernel's choice changes no result beyond the bounds
        check(nv, np.random.default_rng(hq * 1000 + sum(lens)), D, page, hq, heads, new, lens, causal, window,
              max_q=max_q)


def test_attention_rows_that_see_nothing(nv):
    # no cached tokens; more new tokens than positions; both with and without the causal mask
    for causal in (True, False):
        check(nv, np.random.default_rng(1), 64, 16, 4, 2, [2, 5, 1], [0, 3, 9], causal=causal)
        check(nv, np.random.default_rng(1), 128, 16, 4, 2, [40, 3], [0, 1], causal=causal)


@pytest.mark.parametrize("max_q", [1, 64])
def test_attention_peaked_and_flat_scores(nv, max_q):
    check(nv, np.random.default_rng(2), 128, 16, 8, 2, [3, 9], [300, 90], spread=30.0, max_q=max_q)   # nearly one-hot
    check(nv, np.random.default_rng(3), 64, 16, 8, 2, [3, 9], [300, 90], spread=1e-3, max_q=max_q)
    check(nv, np.random.default_rng(4), 64, 16, 8, 2, [3], [300], scale=3.0, max_q=max_q)
    # queries over the whole range of BF16: the row's power of two is taken out before FP16
    check(nv, np.random.default_rng(5), 128, 16, 4, 2, [2, 20], [70, 50], spread=2.0 ** 100, scale=2.0 ** -103, max_q=max_q)
    check(nv, np.random.default_rng(6), 128, 16, 4, 2, [2, 20], [70, 50], spread=2.0 ** -100, scale=2.0 ** 97, max_q=max_q)


@pytest.mark.parametrize("max_q", [1, 200])
def test_attention_strided_queries_long_context_many_sequences(nv, max_q):
    rng = np.random.default_rng(7)
    check(nv, rng, 128, 64, 8, 1, [1], [5000], pad=2, max_q=max_q)                 # one context over many blocks
    lens = rng.integers(1, 60, 300).tolist()                                       # more sequences than threads
    check(nv, rng, 64, 16, 2, 2, [1] * 300, lens, pad=1, max_q=max_q)
    new = rng.integers(0, 3, 280).tolist()
    check(nv, rng, 64, 16, 4, 1, new, [x + 5 for x in new], max_q=max_q)


@pytest.mark.parametrize("D,hq,heads,lens,window", [
    (128, 8, 1, [41003], 0),             # one work over every block of the launch: runs of parts, then the runs
    (64, 8, 2, [30001, 17], 29000),      # long and short works side by side
    (128, 16, 1, [9000, 1, 12345], 0),   # 16 rows a KV head
    (64, 5, 1, [70000], 700),            # a window far behind the start
])
def test_attention_joins_many_parts(nv, D, hq, heads, lens, window):
    # a fresh workspace from memory that is not zero: only what the interface names is zero-filled
    size = nv.lib().nvfp4_paged_attention_workspace_bytes()
    nv._attn_ws.clear()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    dirt = [torch.full((size,), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(4)]
    del dirt
    check(nv, np.random.default_rng(11), D, 64, hq, heads, [1] * len(lens), lens, window=window, max_q=1)


@pytest.mark.parametrize("max_q", [1, 64])
def test_attention_more_new_tokens_than_cached_ones(nv, max_q):
    # tokens before position 0 see nothing of a causal mask; without one they see all, or what their window reaches
    for causal, window in ((True, 0), (True, 2), (False, 0), (False, 3)):
        check(nv, np.random.default_rng(3), 64, 16, 4, 2, [5, 3, 40], [2, 0, 21], causal, window, max_q=max_q)


def setup(nv, rng, D=128, page=16, hq=8, heads=2, new=(2, 1), lens=(90, 35)):
    table, P = tables(rng, lens, page)
    pages = random_pages(rng, P, heads, page, D)
    q, qn = queries(rng, sum(new), hq, D)
    return dict(q=q, qn=qn, table=table, pages=pages, P=P, new=list(new), lens=list(lens),
                cache=nv.KVCache(torch.from_numpy(pages).cuda(), *scalars(KG, VG), page, D))


@pytest.mark.parametrize("max_q", [1, 64])
def test_attention_ignores_what_is_masked(nv, max_q):
    # pages and slots that no row sees may hold anything: the result is the same bit for bit
    s = setup(nv, np.random.default_rng(8))
    args = (ints(s["table"]), ints(cumulative(s["new"])), ints(s["lens"]))
    want, lse = nv.paged_attention(s["q"], s["cache"], *args, want_lse=True, max_q=max_q)
    pages = s["pages"].copy()
    owned = set(s["table"][s["table"] >= 0].tolist())
    for p in range(s["P"]):
        if p not in owned:
            pages[p] = 0xFF
    kc, ks, vc, vs = [x.copy() for x in kv.granule_views(pages, 16, 128)]
    for b, L in enumerate(s["lens"]):
        p = s["table"][b][(L - 1) // 16]
        gr = pages[p].reshape(2, -1, 18 * 128)
        for r in range((L - 1) % 16 + 1, 16):
            for base in (0, 9 * 128):
                gr[:, 0, base + r * 64:base + (r + 1) * 64] = 0xFF
                gr[:, 0, base + 1024 + r * 8:base + 1024 + (r + 1) * 8] = 0xFF   # the NaN code with a sign
    cache = s["cache"]._replace(pages=torch.from_numpy(pages).cuda())
    got, lse2 = nv.paged_attention(s["q"], cache, *args, want_lse=True, max_q=max_q)
    assert torch.equal(got, want) and torch.equal(lse, lse2)
    assert nv.device_status() == 0


@pytest.mark.parametrize("max_q", [1, 64])
def test_attention_with_pages_outside_the_pool(nv, max_q):
    s = setup(nv, np.random.default_rng(9))
    table = s["table"].copy()
    table[0, 2], table[1, 0] = s["P"], -1
    cu = cumulative(s["new"])
    out, lse = nv.paged_attention(s["q"], s["cache"], ints(table), ints(cu), ints(s["lens"]), want_lse=True, max_q=max_q)
    assert nv.device_status() == 9
    ref = kv.attention(s["qn"], s["pages"], table, cu, s["lens"], KG, VG, 16, 128 ** -0.5, True, 0,
                       drop=[(0, 2), (1, 0)])
    compare(out, lse, ref, 128)
    # lengths beyond the table are cut to it, offsets beyond the rows belong to nobody
    out.fill_(7.0)
    nv.paged_attention(s["q"], s["cache"], ints(s["table"]), ints([0, 2, 9]), ints([16 * s["table"].shape[1] + 50, 35]),
                       out=out, max_q=max_q)
    assert nv.device_status() == 9
    assert (out[2] == 7.0).all() and torch.isfinite(out.float()).all()


@pytest.mark.parametrize("max_q", [1, 64])
def test_attention_leaves_rows_behind_the_last_sequence(nv, max_q):
    s = setup(nv, np.random.default_rng(10))
    q = torch.cat([s["q"], torch.full_like(s["q"], float("nan"))])
    out, lse = torch.full_like(q, 5.0), torch.full(q.shape[:2], 6.0, device="cuda")
    nv.paged_attention(q, s["cache"], ints(s["table"]), ints(cumulative(s["new"])), ints(s["lens"]), out=out, lse_out=lse,
                       max_q=max_q)
    assert (out[3:] == 5.0).all() and (lse[3:] == 6.0).all() and torch.isfinite(out[:3].float()).all()
    none = torch.empty((0, 8, 128), dtype=torch.bfloat16, device="cuda")
    got, _ = nv.paged_attention(none, s["cache"], ints(s["table"]), ints([0, 0, 0]), ints(s["lens"]))
    assert got.shape == (0, 8, 128)
    assert nv.device_status() == 0


@pytest.mark.parametrize("max_q", [1, 64])
def test_attention_non_finite_queries_stay_in_their_rows(nv, max_q):
    s = setup(nv, np.random.default_rng(11), new=(3, 1))
    args = (ints(s["table"]), ints(cumulative(s["new"])), ints(s["lens"]))
    want, _ = nv.paged_attention(s["q"], s["cache"], *args, max_q=max_q)
    q = s["q"].clone()
    q[1, 3, 5] = float("nan")
    q[3, 0, 0] = float("inf")
    got, _ = nv.paged_attention(q, s["cache"], *args, max_q=max_q)
    assert torch.isnan(got[1, 3]).all() and torch.isnan(got[3, 0]).all()
    got[1, 3], got[3, 0] = want[1, 3], want[3, 0]
    assert torch.equal(got, want)


@pytest.mark.parametrize("max_q", [1, 64])
def test_attention_is_deterministic_and_streams_do_not_meet(nv, max_q):
    s = setup(nv, np.random.default_rng(12), page=64, heads=2, new=(2, 1), lens=(6000, 9000))
    args = (ints(s["table"]), ints(cumulative(s["new"])), ints(s["lens"]))
    want, _ = nv.paged_attention(s["q"], s["cache"], *args, max_q=max_q)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(5):
        for st in side:
            with torch.cuda.stream(st):
                got.append(nv.paged_attention(s["q"], s["cache"], *args, max_q=max_q)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got)


@pytest.mark.parametrize("max_q", [1, 64])
def test_attention_in_graphs_with_other_lengths(nv, max_q):
    s = setup(nv, np.random.default_rng(13), page=32, new=(2, 1), lens=(3000, 4000))
    table, cu, lens = ints(s["table"]), ints(cumulative(s["new"])), ints(s["lens"])
    nv.paged_attention(s["q"], s["cache"], table, cu, lens, max_q=max_q)
    st = torch.cuda.Stream()
    graphs, outs = [], []
    with torch.cuda.stream(st):
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                outs.append(nv.paged_attention(s["q"], s["cache"], table, cu, lens, max_q=max_q)[0])
            graphs.append(g)
    for lengths in ((3000, 4000), (17, 3999), (0, 1)):
        lens.copy_(ints(lengths))
        torch.cuda.synchronize()
        want, _ = nv.paged_attention(s["q"], s["cache"], table, cu, lens, max_q=max_q)
        torch.cuda.synchronize()
        both = [torch.cuda.Stream() for _ in range(2)]
        for _ in range(3):                       # the two graphs at the same time, and an eager call beside them
            for g, x in zip(graphs, both):
                with torch.cuda.stream(x):
                    g.replay()
            eager, _ = nv.paged_attention(s["q"], s["cache"], table, cu, lens, max_q=max_q)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want) and torch.equal(eager, want), lengths


@pytest.mark.parametrize("max_q", [1, 64])
def test_attention_and_append_beyond_32_bit_offsets(nv, max_q):
    # a pool of 4.8 GB: the pages in use lie at its end
    D, page, heads = 128, 128, 8
    P = (5 << 30) // (heads * nv.kv_page_bytes(page, D))
    rng = np.random.default_rng(14)
    kg, vg = scalars(0.002, 0.002)
    big = nv.kv_cache(P, heads, D, page, kg, vg)
    small = nv.kv_cache(2, heads, D, page, kg, vg)
    assert big.pages.numel() > 1 << 32
    x = [torch.from_numpy(rng.standard_normal((150, heads, D)).astype(np.float32)).to(torch.bfloat16).cuda() for _ in "kv"]
    q, _ = queries(rng, 3, 16, D)
    got = []
    for cache, ids in ((big, [P - 1, P - 2]), (small, [0, 1])):
        nv.kv_append(cache, *x, ints([ids]), ints([0, 150]), ints([150]))
        got.append(nv.paged_attention(q, cache, ints([ids]), ints([0, 3]), ints([150]), max_q=max_q)[0])
    assert torch.equal(big.pages[[P - 1, P - 2]], small.pages) and torch.equal(*got)
    nv.kv_copy_pages(big, ints([P - 1]), ints([P - 3]))
    assert torch.equal(big.pages[P - 3], small.pages[0])
    assert nv.device_status() == 0


def test_binding_refuses(nv):
    s = setup(nv, np.random.default_rng(15))
    q, c = s["q"], s["cache"]
    table, cu, lens = ints(s["table"]), ints(cumulative(s["new"])), ints(s["lens"])
    bad = [
        (q.float(), c, table, cu, lens), (q[:, :, :64], c, table, cu, lens), (q.transpose(0, 1), c, table, cu, lens),
        (q.cpu(), c, table, cu, lens), (q, c._replace(pages=c.pages[:, :, :-16]), table, cu, lens),
        (q, c._replace(page_size=32), table, cu, lens), (q, c._replace(k_g=c.k_g.double()), table, cu, lens),
        (q, c, table.long(), cu, lens), (q, c, table[:1], cu, lens), (q, c, table, cu[:2], lens),
        (q, c, table.cpu(), cu, lens), (q, c, table[:, ::2], cu, lens),
    ]
    for args in bad:
        with pytest.raises(ValueError):
            nv.paged_attention(*args)
    for kw in (dict(out=q.float()), dict(out=torch.empty_like(q)[:1]), dict(lse_out=torch.empty(3, 7, device="cuda"))):
        with pytest.raises(ValueError):
            nv.paged_attention(q, c, table, cu, lens, **kw)
    for kw in (dict(out=q), dict(scale=0.0), dict(window=-3), dict(max_q=-1)):
        with pytest.raises(nv.NVFP4Error):
            nv.paged_attention(q, c, table, cu, lens, **kw)
    with pytest.raises(nv.NVFP4Error):                      # seven query heads for two KV heads
        nv.paged_attention(q[:, :7].contiguous(), c, table, cu, lens)
    k = q[:, :2].contiguous()
    with pytest.raises(ValueError):
        nv.kv_append(c, k, k[:2], table, cu, lens)
    with pytest.raises(ValueError):
        nv.kv_append(c, q, q, table, cu, lens)
    with pytest.raises(nv.NVFP4Error):
        nv.kv_append(c, k, k, table, cu, lens, mode="mse")
    with pytest.raises(ValueError):
        nv.kv_copy_pages(c, lens, cu)
    refs = ints([0] * 4)
    with pytest.raises(ValueError):
        nv.kv_fork(refs, table, cu, lens, lens, 16)
    with pytest.raises(ValueError):
        nv.kv_compact(refs, table, lens, 16, refs_out=refs[:2])


# ------------------------------------------------------------------ page pool
def pool(rng, P, slots, width, page, fill=0.6, share=True):
    lens, table, refs = np.zeros(slots, np.int64), np.full((slots, width), -1, np.int64), np.zeros(P, np.int64)
    ids, at = rng.permutation(P), 0
    for s in range(slots):
        n = int(rng.integers(0, width * page + 1))
        m = kv.held(n, page)
        if at + m > fill * P:
            continue
        lens[s] = n
        table[s, :m] = ids[at:at + m]
        at += m
        if share and s and lens[s - 1]:
            both = min(m, kv.held(lens[s - 1], page)) // 2
            table[s, :both] = table[s - 1, :both]
        for p in table[s, :m]:
            refs[p] += 1
    return refs, table, lens


@pytest.mark.parametrize("P,slots,width,page", [(40, 6, 4, 16), (9000, 300, 40, 128), (70000, 64, 700, 16), (5, 3, 2, 64)])
def test_fork_free_compact_match_the_oracle(nv, P, slots, width, page):
    rng = np.random.default_rng(P)
    refs, table, lens = pool(rng, P, slots, width, page)
    dr, dt, dl = ints(refs), ints(table), ints(lens)
    for step in range(4):
        empty = np.flatnonzero(lens == 0)
        named = rng.permutation(empty)[:max(1, len(empty) // 2)].tolist()
        par = rng.integers(0, slots, len(named)).tolist()
        par = [a if a != c else (a + 1) % slots for a, c in zip(par, named)]
        if named:
            src, dst = nv.kv_fork(dr, dt, dl, ints(par), ints(named), page)
            s, d, st = kv.fork(refs, table, lens, par, named, page)
            assert nv.device_status() == st
            assert to_np(src).tolist() == s and to_np(dst).tolist() == d
        gone = rng.integers(0, slots, max(1, slots // 3)).tolist()      # the same slot may be named twice
        nv.kv_free(dr, dt, dl, ints(gone), page)
        kv.free(refs, table, lens, gone, page)
        assert to_np(dr).tolist() == refs.tolist() and to_np(dl).tolist() == lens.tolist()
        assert np.array_equal(to_np(dt), table)
        r, t, src, dst, live = nv.kv_compact(dr, dt, dl, page)
        r2, t2, s2, d2, live2 = kv.compact(refs, table, lens, page)
        assert int(live) == live2 and to_np(r).tolist() == r2.tolist() and np.array_equal(to_np(t), t2)
        rest = [-1] * (max(1, P // 2) - len(s2))
        assert to_np(src).tolist() == s2 + rest and to_np(dst).tolist() == d2 + rest
        if step == 1:                                                    # and in place
            nv.kv_compact(dr, dt, dl, page, refs_out=dr, table_out=dt)
            refs, table = r2, t2
    assert nv.device_status() == 0


def test_fork_refusals_on_the_device(nv):
    page = 16
    refs, table = np.array([1, 1, 0, 0, 0]), np.array([[0, 1, -1], [-1, -1, -1], [-1] * 3, [-1] * 3])
    lens = np.array([20, 0, 0, 0])
    # out of range, a child that holds tokens, parent == child, the same child twice
    par, child = [0, 0, 0, 2, 0, -1, 4], [2, 0, 2, 2, 1, 3, 3]
    dr, dt, dl = ints(refs), ints(table), ints(lens)
    src, dst = nv.kv_fork(dr, dt, dl, ints(par), ints(child), page)
    s, d, st = kv.fork(refs, table, lens, par, child, page)
    assert st == 9 and nv.device_status() == 9
    assert to_np(src).tolist() == s == [1, -2, -2, -2, 1, -2, -2] and to_np(dst).tolist() == d
    assert to_np(dr).tolist() == refs.tolist() and np.array_equal(to_np(dt), table) and to_np(dl).tolist() == lens.tolist()
    # two part pages wanted, one page free: nothing changes
    refs, lens = np.array([1, 1, 0, 1, 1]), np.array([20, 0, 0, 0])
    dr, dl, before = ints(refs), ints(lens), dt.clone()
    src, dst = nv.kv_fork(dr, dt, dl, ints([0, 0]), ints([1, 2]), page)
    assert nv.device_status() == 10
    assert to_np(src).tolist() == [-2, -2] and to_np(dst).tolist() == [-2, -2]
    assert to_np(dr).tolist() == refs.tolist() and to_np(dl).tolist() == lens.tolist() and torch.equal(dt, before)
    # freeing what is not there
    nv.kv_free(dr, dt, dl, ints([9, -1, 3]), page)
    assert nv.device_status() == 9 and to_np(dr).tolist() == refs.tolist()


def test_copy_pages_skips_and_refuses(nv):
    rng = np.random.default_rng(20)
    pages = rng.integers(0, 256, (9, 3, 18 * 64), dtype=np.uint8)
    cache = nv.KVCache(torch.from_numpy(pages).cuda(), *scalars(1.0, 1.0), 16, 64)
    nv.kv_copy_pages(cache, ints([0, -1, 4, 2]), ints([8, 3, -2, 5]))
    pages[8], pages[5] = pages[0], pages[2]
    assert np.array_equal(to_np(cache.pages), pages) and nv.device_status() == 0
    nv.kv_copy_pages(cache, ints([9, 1]), ints([3, 9]))
    assert np.array_equal(to_np(cache.pages), pages) and nv.device_status() == 9
    nv.kv_copy_pages(cache, ints([]), ints([]))


# ------------------------------------------------------- all of them together
def test_a_sequence_of_serving_steps(nv):
    """Prompt, fork, decode on both branches, free, compact, decode on: attention agrees with the oracle over the keys
    and values as nv.quantize stores them, and does not change under fork and compaction."""
    rng = np.random.default_rng(30)
    D, page, heads, hq, slots, width, P = 128, 16, 2, 8, 4, 6, 20
    kg, vg = 0.002, 0.0025
    cache = nv.kv_cache(P, heads, D, page, *scalars(kg, vg))
    refs, table, lens = ints([0] * P), ints([[-1] * width] * slots), ints([0] * slots)
    history = {s: [] for s in range(slots)}          # what each slot's tokens are, on the host

    def grow(slot, n):
        """The caller's part: pages for n more tokens of a slot, taken from the top of the pool."""
        old, new = int(lens[slot]), int(lens[slot]) + n
        for j in range(kv.held(old, page), kv.held(new, page)):
            p = max(i for i in range(P) if int(refs[i]) == 0)
            refs[p] = 1
            table[slot, j] = p
        lens[slot] = new

    def step(new):
        """One forward step: append the new tokens of slots {slot: n}, then attend with them."""
        which = sorted(new)
        for s in which:
            grow(s, new[s])
        T = sum(new.values())
        qkv = torch.from_numpy(rng.standard_normal((T, hq + 2 * heads, D)).astype(np.float32)).to(torch.bfloat16).cuda()
        cu, rows = cumulative([new[s] for s in which]), table[which].contiguous()
        nv.kv_append(cache, qkv[:, hq:hq + heads], qkv[:, hq + heads:], rows, ints(cu), lens[which].contiguous(),
                     mode="four_over_six")
        for i, s in enumerate(which):
            history[s] = history[s] + list(qkv[cu[i]:cu[i + 1], hq:])
        return which, cu, rows, qkv[:, :hq]

    def attend(which, cu, rows, q):
        out, lse = nv.paged_attention(q, cache, rows, ints(cu), lens[which].contiguous(), want_lse=True)
        # the oracle's pages: every slot's history quantized and laid out one after another
        own = np.zeros((slots * width, heads, nv.kv_page_bytes(page, D)), np.uint8)
        flat = np.arange(slots * width).reshape(slots, width)
        for s in which:
            x = bf16_np(torch.stack(history[s]))
            kv.append(own, x[:, :heads], x[:, heads:], [flat[s]], [0, len(x)], [len(x)], kg, vg, page, "four_over_six")
        ref = kv.attention(bf16_np(q), own, flat[which], cu, [len(history[s]) for s in which], kg, vg, page, D ** -0.5,
                           True, 0)
        compare(out, lse, ref, D)
        return out

    attend(*step({0: 37, 1: 16}))                                         # two prompts
    src, dst = nv.kv_fork(refs, table, lens, ints([0, 0, 1]), ints([2, 3, 3]), page)
    assert to_np(src)[2] == -2 and nv.device_status() == 9                # slot 3 is taken by then
    nv.kv_copy_pages(cache, src, dst)
    history[2], history[3] = list(history[0]), list(history[0])
    for _ in range(12):                                                   # every branch goes on by itself
        last = step({0: 1, 1: 1, 2: 2, 3: 1})
        before = attend(*last)
    nv.kv_free(refs, table, lens, ints([1, 0]), page)
    new_refs, new_table, src, dst, live = nv.kv_compact(refs, table, lens, page)
    nv.kv_copy_pages(cache, src, dst)
    refs, table = new_refs, new_table
    assert int(live) == int((refs > 0).sum()) and not refs[int(live):].any() and int(live) < P // 2
    which, cu, rows, q = last
    after, _ = nv.paged_attention(q[2:].contiguous(), cache, table[2:].contiguous(), ints([0, 2, 3]), lens[2:].contiguous())
    assert torch.equal(after, before[2:])                                 # moved pages, the same result
    attend(*step({2: 1, 3: 5}))
    assert nv.device_status() == 0
