"""Paged NVFP4 KV cache on the GPU at the borders of what its interface allows."""
import numpy as np
import pytest
import torch

from oracle import kv_oracle as kv
from tests.test_gpu_kv_cache import compare, cumulative, ints, queries, random_pages, scalars, tables
from tests.util import bf16_np, require_gpu, to_np

pytestmark = pytest.mark.gpu

KG = 0.11                    # global scale of the random keys: values of about 1


@pytest.fixture(scope="module")
def nv():
    return require_gpu()


def problem(nv, rng, D, page, hq, heads, new, lens, vg):
    """Random pages and queries under the value scale vg: what attention takes, and what the oracle takes."""
    table, P = tables(rng, lens, page)
    pages = random_pages(rng, P, heads, page, D)
    q, qn = queries(rng, sum(new), hq, D)
    cache = nv.KVCache(torch.from_numpy(pages).cuda(), *scalars(KG, vg), page, D)
    return q, qn, cache, pages, table


# ---------------------------------------------------- rows that see nothing
@pytest.mark.parametrize("vg", [0.07, 0.3, 1.0, 4.0, 2.0 ** 100])
@pytest.mark.parametrize("max_q", [1, 64])
def test_rows_that_see_nothing_are_zero_under_every_value_scale(nv, max_q, vg):
    # no cached tokens; more new tokens than positions, before rows that see some; a window in front of what is there
    for D, page, hq, heads, new, lens, causal, window in (
            (64, 16, 4, 2, [2, 5, 1], [0, 3, 9], True, 0), (128, 16, 4, 2, [40, 3], [0, 1], True, 0),
            (128, 16, 8, 2, [300, 1], [140, 0], True, 0), (64, 32, 6, 3, [70, 2], [64, 0], True, 5),
            (128, 64, 2, 1, [1, 1], [0, 0], False, 0)):
        q, qn, cache, pages, table = problem(nv, np.random.default_rng(sum(new)), D, page, hq, heads, new, lens, vg)
        cu = cumulative(new)
        out, lse = nv.paged_attention(q, cache, ints(table), ints(cu), ints(lens), causal=causal, window=window,
                                      max_q=max_q, want_lse=True)
        ref = kv.attention(qn, pages, table, cu, lens, KG, vg, page, D ** -0.5, causal, window)
        none = ref["seen"] == 0
        assert none.any() and not bf16_np(out)[none].any() and np.isneginf(to_np(lse)[none]).all()
        compare(out, lse, ref, D)
        assert nv.device_status() == 0


@pytest.mark.parametrize("vg", [0.07, 4.0])
@pytest.mark.parametrize("max_q", [1, 64])
def test_rows_without_a_page_are_zero(nv, max_q, vg):
    # every page outside the pool: nothing to see, in short works and in one that is cut into parts
    for lens in ([35, 1], [30000, 5]):
        q, _, cache, _, table = problem(nv, np.random.default_rng(3), 128, 64, 8, 2, [2, 1], lens, vg)
        for page in (-1, cache.pages.shape[0]):
            out, lse = nv.paged_attention(q, cache, ints(np.full_like(table, page)), ints([0, 2, 3]), ints(lens),
                                          max_q=max_q, want_lse=True)
            assert not out.any() and torch.isneginf(lse).all()
            assert nv.device_status() == 9


# ------------------------------------------------------- non-finite queries
@pytest.mark.parametrize("lens", [(90, 35), (9000, 700), (100000, 60000)])
@pytest.mark.parametrize("max_q", [1, 64])
def test_non_finite_queries_give_nan_whether_their_work_is_cut_or_not(nv, max_q, lens):
    q, _, cache, _, table = problem(nv, np.random.default_rng(lens[0]), 128, 64, 8, 2, [3, 1], lens, 0.07)
    args = (ints(table), ints([0, 3, 4]), ints(lens))
    want, lse0 = nv.paged_attention(q, cache, *args, max_q=max_q, want_lse=True)
    assert torch.isfinite(want.float()).all() and torch.isfinite(lse0).all()
    rows = [(0, 1), (1, 3), (3, 0), (2, 7)]
    for value in (float("nan"), float("inf"), -float("inf")):
        bad = q.clone()
        for t, h in rows:
            bad[t, h, 5 * h % 128] = value       # (among so many keys one has the value's sign there: its score is +Inf)
        out, lse = nv.paged_attention(bad, cache, *args, max_q=max_q, want_lse=True)
        for t, h in rows:
            assert torch.isnan(out[t, h]).all() and torch.isnan(lse[t, h]), (value, t, h)
            out[t, h], lse[t, h] = want[t, h], lse0[t, h]
        assert torch.equal(out, want) and torch.equal(lse, lse0)      # the other rows: bit for bit
    assert nv.device_status() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("max_q", [1, 64])
def test_nan_queries_that_see_one_or_two_tokens(nv, max_q, D):
    # each place of a 64-token step by itself, under windows of one and two tokens
    lens = list(range(1, 81))
    q, _, cache, _, table = problem(nv, np.random.default_rng(D), D, 32, 2, 2, [1] * 80, lens, 0.07)
    bad = q.clone()
    bad[:, 0] = float("nan")
    for window in (1, 2):
        args = (ints(table), ints(range(81)), ints(lens))
        want, _ = nv.paged_attention(q, cache, *args, window=window, max_q=max_q)
        out, lse = nv.paged_attention(bad, cache, *args, window=window, max_q=max_q, want_lse=True)
        assert torch.isnan(out[:, 0]).all() and torch.isnan(lse[:, 0]).all()
        assert torch.equal(out[:, 1], want[:, 1])


@pytest.mark.parametrize("max_q", [1, 64])
def test_scores_of_minus_infinity_weigh_nothing(nv, max_q):
    # A query of -Inf in one dimension, keys that are positive there: every score is -Inf, the sum of their weights 0.
    D, page, n = 64, 16, 50
    k = torch.ones((n, 1, D), dtype=torch.bfloat16, device="cuda")
    cache = nv.kv_cache(4, 1, D, page, *scalars(0.001, 0.001))
    table = ints([[0, 1, 2, 3]])
    nv.kv_append(cache, k, k, table, ints([0, n]), ints([n]))
    q = torch.ones((1, 2, D), dtype=torch.bfloat16, device="cuda")
    q[0, 1, 7] = -float("inf")
    out, lse = nv.paged_attention(q, cache, table, ints([0, 1]), ints([n]), max_q=max_q, want_lse=True)
    assert not out[0, 1].any() and torch.isneginf(lse[0, 1])
    assert torch.isfinite(lse[0, 0]) and out[0, 0].all()


# ------------------------------------------------------------ attention sinks
@pytest.mark.parametrize("nats", [12.0, 14.0, 16.0, 18.0])
@pytest.mark.parametrize("max_q", [1, 64])
def test_tokens_behind_an_attention_sink_keep_their_weights(nv, max_q, nats):
    """The first token far above all others, with values of zero: the output is what the others' small weights bring. As
    many works as the card holds CTAs, so that a row's tokens are not divided and its state has the sink in it."""
    D, page, heads, hq, L, seqs = 128, 64, 8, 16, 4096, 37
    rng = np.random.default_rng(int(nats))
    sign = np.where(rng.random((heads, D)) < 0.5, -1.0, 1.0)
    k = rng.standard_normal((L, heads, D)) * 0.05
    k[0] = sign * nats / D ** 0.5                      # scale * q . k = nats, for a query of the signs
    v = rng.uniform(0.5, 1.0, (L, heads, D))
    v[0] = 0.0
    k, v = (torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).cuda() for x in (k, v))
    kg, vg = 0.001, 0.0005                              # keys to 2.6, values to 1.3
    cache = nv.kv_cache(L // page, heads, D, page, *scalars(kg, vg))
    row = rng.permutation(L // page)
    nv.kv_append(cache, k, v, ints(row[None]), ints([0, L]), ints([L]))
    q = torch.from_numpy(np.repeat(sign, hq // heads, 0)[None].astype(np.float32)).to(torch.bfloat16)
    ref = kv.attention(bf16_np(q), to_np(cache.pages), row[None], [0, 1], [L], kg, vg, page, D ** -0.5, True, 0)
    # (the sink's key is a multiple of its block scale, which rounds by at most 2^-4 of itself)
    assert (ref["out"] > 0).all() and (ref["out"] < np.exp(0.5 - nats * (1 - 2.0 ** -4)) * L).all()
    out, _ = nv.paged_attention(q.cuda().repeat(seqs, 1, 1), cache, ints(np.repeat(row[None], seqs, 0)),
                                ints(range(seqs + 1)), ints([L] * seqs), max_q=max_q)
    err = np.abs(bf16_np(out).astype(np.float64) - ref["out"])
    tol, _ = kv.attention_tolerance(ref, D)
    assert (err <= tol).all(), float((err / tol).max())


# -------------------------------------------- a batch that begins behind row 0
@pytest.mark.parametrize("mode", ["max", "four_over_six"])
def test_append_of_the_last_sequences_of_a_batch(nv, mode):
    """Offsets that begin above 0 (the last sequences of a larger batch over the same rows): the rows before them belong
    to nobody, which is no error."""
    rng = np.random.default_rng(5)
    D, page, heads, new, lens = 64, 16, 2, [40, 7, 1, 20], [40, 30, 16, 21]
    table, P = tables(rng, lens, page)
    x = torch.from_numpy(rng.standard_normal((2, sum(new), heads, D)).astype(np.float32)).to(torch.bfloat16)
    pages = rng.integers(0, 256, (P, heads, nv.kv_page_bytes(page, D)), dtype=np.uint8)
    for first in range(4):
        cache = nv.KVCache(torch.from_numpy(pages).cuda(), *scalars(0.002, 0.003), page, D)
        cu = cumulative(new)[first:]
        nv.kv_append(cache, x[0].cuda(), x[1].cuda(), ints(table[first:]), ints(cu), ints(lens[first:]), mode=mode)
        assert nv.device_status() == 0, first
        ref = pages.copy()
        kv.append(ref, bf16_np(x[0]), bf16_np(x[1]), table[first:], cu, lens[first:], 0.002, 0.003, page, mode)
        assert np.array_equal(to_np(cache.pages), ref)


def test_append_reports_every_malformed_offset_and_length(nv):
    """Offsets that decrease and lengths outside the table are reported however the rows are divided over the card, also
    those of a sequence that no row leads to."""
    D, page, n = 64, 16, 8
    one = torch.ones((n, 1, D), dtype=torch.bfloat16, device="cuda")
    cache = nv.kv_cache(4, 1, D, page, *scalars(0.01, 0.01))
    table = ints([[0], [1], [2]])
    for cu, lens, status in (([0, 5, 5, 8], [5, 0, 3], 0), ([0, 5, 5, 8], [16, 16, 16], 0), ([0, 5, 3, 8], [5, 9, 9], 9),
                             ([0, 5, 5, 8], [5, 17, 3], 9), ([0, 5, 5, 8], [5, -1, 3], 9), ([-1, 0, 5, 8], [1, 5, 3], 9),
                             ([0, 5, 8, 9], [5, 3, 1], 9)):
        nv.kv_append(cache, one, one, table, ints(cu), ints(lens))
        assert nv.device_status() == status, (cu, lens)


@pytest.mark.parametrize("max_q", [1, 64])
def test_a_window_of_any_size(nv, max_q):
    # windows up to the type's largest value, with tokens before position 0: what no window gives, bit for bit
    new, lens = [200, 40, 1], [100, 0, 77]
    q, _, cache, _, table = problem(nv, np.random.default_rng(21), 128, 16, 4, 2, new, lens, 0.07)
    args = (ints(table), ints(cumulative(new)), ints(lens))
    for causal in (True, False):
        want, lse0 = nv.paged_attention(q, cache, *args, causal=causal, max_q=max_q, want_lse=True)
        for window in (1 << 20, (1 << 31) - 1, 1 << 31, (1 << 63) - (1 << 31), (1 << 63) - 1):
            out, lse = nv.paged_attention(q, cache, *args, causal=causal, window=window, max_q=max_q, want_lse=True)
            assert torch.equal(out, want) and torch.equal(lse, lse0), window
    assert nv.device_status() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("max_q", [1, 4, 64])
def test_attention_waits_that_run_out(nv, max_q, D):
    """Copies that are awaited but never issued: the waits give up and are reported, what is in flight lands before the
    blocks leave, calls beside it and behind it are right."""
    new, lens = [2, 1], [30000, 700]
    q, _, cache, _, table = problem(nv, np.random.default_rng(22), D, 32, 8, 2, new, lens, 0.07)
    args = (ints(table), ints(cumulative(new)), ints(lens))
    want, lse0 = nv.paged_attention(q, cache, *args, max_q=max_q, want_lse=True)
    assert nv.device_status() == 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(side):
            nv.selftest_attention_timeout(q, cache, *args, timeout_ns=1_000_000, max_q=max_q)
        beside = [nv.paged_attention(q, cache, *args, max_q=max_q, want_lse=True) for _ in range(20)]
        torch.cuda.synchronize()
        assert nv.device_status() == 6
        out, lse = nv.paged_attention(q, cache, *args, max_q=max_q, want_lse=True)
        for x, y in beside + [(out, lse)]:
            assert torch.equal(x, want) and torch.equal(y, lse0)
        assert nv.device_status() == 0
    # nothing cached: nothing is awaited
    nv.selftest_attention_timeout(q, cache, args[0], args[1], ints([0, 0]), timeout_ns=1_000_000, max_q=max_q)
    torch.cuda.synchronize()
    assert nv.device_status() == 0
    with pytest.raises(nv.NVFP4Error):
        nv.selftest_attention_timeout(q, cache, *args, timeout_ns=0)


@pytest.mark.parametrize("max_q", [1, 64])
def test_attention_of_thousands_of_sequences_with_prompts_among_them(nv, max_q):
    # prompts of many tiles in front of the 256th sequence and behind it, and far behind
    rng = np.random.default_rng(23)
    n, D, page = 3000, 64, 16
    new = np.ones(n, int)
    new[[3, 290, 2500]] = [700, 900, 400]
    new[rng.integers(0, n, 200)] = 0
    lens = new + rng.integers(0, 20, n)
    q, qn, cache, pages, table = problem(nv, rng, D, page, 2, 1, new.tolist(), lens.tolist(), 0.07)
    cu = cumulative(new.tolist())
    out, lse = nv.paged_attention(q, cache, ints(table), ints(cu), ints(lens.tolist()), max_q=max_q, want_lse=True)
    assert nv.device_status() == 0
    ref = kv.attention(qn, pages, table, cu, lens.tolist(), KG, 0.07, page, D ** -0.5, True, 0)
    compare(out, lse, ref, D)


@pytest.mark.parametrize("max_q", [None, 1, 64])
def test_a_batch_without_new_tokens_leaves_everything(nv, max_q):
    # every row behind the last sequence (a padded batch that has run empty), a few sequences and many
    for n in (3, 70):
        q, _, cache, pages, table = problem(nv, np.random.default_rng(24), 64, 16, 4, 2, [1] * n, [40] * n, 0.07)
        args = (ints(table), ints([0] * (n + 1)), ints([40] * n))
        out, lse = torch.full_like(q, 5.0), torch.full(q.shape[:2], 6.0, device="cuda")
        nv.paged_attention(q, cache, *args, out=out, lse_out=lse, max_q=max_q)
        nv.kv_append(cache, q[:, :2], q[:, 2:], *args)
        assert (out == 5.0).all() and (lse == 6.0).all() and np.array_equal(to_np(cache.pages), pages)
        assert nv.device_status() == 0


@pytest.mark.parametrize("max_q", [1, 64])
def test_zero_and_subnormal_queries(nv, max_q):
    # a row's power of two is taken out before FP16 down to BF16's smallest numbers; a query of zeros weighs all alike
    D, page, new, lens = 128, 16, [2, 20], [70, 50]
    for value in (2.0 ** -130, 2.0 ** -126, 0.0):
        q, _, cache, pages, table = problem(nv, np.random.default_rng(25), D, page, 4, 2, new, lens, 0.07)
        q = (q.float() * value).to(torch.bfloat16)
        out, lse = nv.paged_attention(q, cache, ints(table), ints(cumulative(new)), ints(lens), scale=2.0 ** 126,
                                      max_q=max_q, want_lse=True)
        ref = kv.attention(bf16_np(q), pages, table, cumulative(new), lens, KG, 0.07, page, 2.0 ** 126, True, 0)
        assert value == 0.0 or np.ptp(ref["lse"]) > 0.1
        compare(out, lse, ref, D)
        assert nv.device_status() == 0


# -------------------------------------------------------------- huge scores
@pytest.mark.parametrize("power", [0, 10, 18, 20, 21, 22, 23, 24, 26, 30, 60, 110])
@pytest.mark.parametrize("max_q", [1, 64])
def test_scores_of_any_size_pick_the_largest(nv, max_q, power):
    """Queries up to 2^110: the softmax of scores that lie far apart is one at the largest, whatever their size."""
    D, page, heads = 128, 64, 2
    rng = np.random.default_rng(power)
    for new, L in ((1, 200), (3, 60000)):
        sign = np.where(rng.random((1, heads, D)) < 0.5, -1.0, 1.0)
        size = rng.choice([0.25, 0.5, 1.0, 1.25], (L, heads, 1))
        best = rng.integers(0, L - new, heads)
        size[best, np.arange(heads)] = 2.0
        k = torch.from_numpy((sign * size).astype(np.float32)).to(torch.bfloat16).cuda()
        v = torch.from_numpy(rng.uniform(0.5, 1.0, (L, heads, D)).astype(np.float32)).to(torch.bfloat16).cuda()
        kg, vg = 0.001, 0.0005
        cache = nv.kv_cache(-(-L // page), heads, D, page, *scalars(kg, vg))
        row = rng.permutation(cache.pages.shape[0])[None]
        nv.kv_append(cache, k, v, ints(row), ints([0, L]), ints([L]))
        K, V = kv.gather(to_np(cache.pages), row[0], L, page, D, kg, vg)
        q = torch.from_numpy(np.repeat(sign * 2.0 ** power, new, 0).astype(np.float32)).to(torch.bfloat16).cuda()
        for flip in (1.0, -1.0):
            # the opposite query: all scores are negative, the smallest keys win (many of them, all alike)
            out, lse = nv.paged_attention(q * flip, cache, ints(row), ints([0, new]), ints([L]), max_q=max_q, want_lse=True)
            for h in range(heads):
                s = D ** -0.5 * 2.0 ** power * flip * (K[h] @ sign[0, h])
                top = s.max()
                for t in range(new):
                    see = s[:L - new + t + 1]
                    p = np.exp(see - top)
                    want, mass = p @ V[h, :len(see)] / p.sum(), top + np.log(p.sum())
                    # A score is off by at most e_s (kv.attention_tolerance). From queries of 2^10 on two different ones lie
                    # 0.25 * 2^10 * sqrt(D) nats or more apart, far beyond e_s: all but the largest vanish, and those of
                    # equal keys are equal. Weights are rounded to FP16 (2^-11), the sums add (n + 64) * 2^-24 each, the
                    # output is rounded to BF16; its values lie below 1.
                    e_s = (D + 16) * 2.0 ** -24 * np.abs(see).max() + 2.0 ** -21
                    rel = (2 * e_s if power < 10 else 0.0) + 2.0 ** -11 + 2 * (len(see) + 64) * 2.0 ** -24
                    err = np.abs(bf16_np(out)[t, h] - want)
                    assert (err <= 2.0 ** -8 * np.abs(want) + rel * (1 + 2.0 ** -8)).all(), (power, flip, err.max())
                    got = float(lse[t, h])
                    assert abs(got - mass) <= e_s + (len(see) + 64) * 2.0 ** -24 + 2.0 ** -21 * (abs(mass) + 1), (got, mass)
    assert nv.device_status() == 0


@pytest.mark.parametrize("vg", [2.0 ** -120, 2.0 ** -100, 2.0 ** 100, 2.0 ** 120])
@pytest.mark.parametrize("max_q", [1, 64])
def test_value_scales_near_the_ends_of_fp32(nv, max_q, vg):
    # outputs that BF16 holds come out whatever the global scale, from whole works and from parts
    for new, lens in (([3, 20], [70, 50]), ([1, 2], [40000, 9])):
        D, page = 128, 64
        q, qn, cache, pages, table = problem(nv, np.random.default_rng(26), D, page, 4, 2, new, lens, vg)
        cu = cumulative(new)
        out, lse = nv.paged_attention(q, cache, ints(table), ints(cu), ints(lens), max_q=max_q, want_lse=True)
        ref = kv.attention(qn, pages, table, cu, lens, KG, vg, page, D ** -0.5, True, 0)
        compare(out, lse, ref, D)
        assert nv.device_status() == 0
