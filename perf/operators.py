"""Workloads of the paged NVFP4 KV cache: appending new tokens to its pages,
attention of new tokens over it, forking sequences and compacting the pool.

``own`` False computes every operator in plain torch (FP32 arithmetic, no fused
library call); ``own`` True calls the package's kernels on the same state.

Cache of one layer: ``pages`` uint8 [pages][kv heads][page/16 granules][18*D].
A granule holds 16 consecutive tokens of one head: K codes [16][D/2], K block
scales [16][D/16], V codes, V block scales. Value = g * E4M3 scale * E2M1 code.
"""
import functools
import math
import random

import torch

own = False

_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_K_G, _V_G = 0.002, 0.0025  # static global scales, amax / 2688 of calibration data of a few sigma


# ---------------------------------------------------------------------- cases
def listed():
    return [
        # one user's next token over a short context: latency
        dict(name="attn_decode_1x1k", op="attention", batch=1, new=1, ctx=1000, ragged=False, hq=32, hkv=8, dim=128,
             page=16, causal=True, window=0),
        # a serving batch, one token each, contexts of different lengths
        dict(name="attn_decode_64x16k", op="attention", batch=64, new=1, ctx=16384, ragged=True, hq=32, hkv=8, dim=128,
             page=64, causal=True, window=0),
        # two long documents: the split of one context over the whole card
        dict(name="attn_decode_2x131k", op="attention", batch=2, new=1, ctx=131075, ragged=False, hq=16, hkv=2, dim=128,
             page=128, causal=True, window=0),
        # checking a few drafted tokens per sequence, sliding-window layer, head size 64, three query heads a key head
        dict(name="attn_draft_32x4_win", op="attention", batch=32, new=4, ctx=8191, ragged=True, hq=24, hkv=8, dim=64,
             page=32, causal=True, window=2048),
        # chunked prefill: ragged chunks behind long prefixes
        dict(name="attn_chunk_4x512_16k", op="attention", batch=4, new=512, ctx=16384, ragged=True, hq=32, hkv=8,
             dim=128, page=64, causal=True, window=0),
        # one long prompt's second part
        dict(name="attn_prefill_4096_12k", op="attention", batch=1, new=4096, ctx=12288, ragged=False, hq=32, hkv=4,
             dim=128, page=64, causal=True, window=0),
        # the batch's new tokens written to their pages, one token a sequence
        dict(name="append_decode_64", op="append", batch=64, new=1, ctx=4096, ragged=True, hq=32, hkv=8, dim=128,
             page=64, mode="max"),
        # a prompt written with the four_over_six recipe
        dict(name="append_prefill_32k_fos", op="append", batch=5, new=8192, ctx=8192, ragged=True, hq=32, hkv=8,
             dim=128, page=64, mode="four_over_six"),
        # four continuations of two prompts
        dict(name="fork_2x4", op="fork", parents=2, ways=4, ctx=1500, hkv=8, dim=128, page=16),
        # many samples of long prompts
        dict(name="fork_64x16", op="fork", parents=64, ways=16, ctx=20000, hkv=8, dim=128, page=128),
        # a small pool, tidied between two requests
        dict(name="compact_512_pages", op="compact", pages=512, slots=16, width=24, hkv=8, dim=128, page=16),
        # a pool with holes after requests have left it
        dict(name="compact_16k_pages", op="compact", pages=16384, slots=128, width=96, hkv=8, dim=128, page=64),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5))))))


def draw(rng):
    op = rng.choice(("attention",) * 4 + ("append",) * 2 + ("fork", "compact"))
    dim, page = rng.choice((64, 128, 128)), rng.choice((16, 32, 64, 128))
    if op in ("attention", "append"):
        hkv = rng.choice((1, 2, 4, 8))
        hq = hkv * rng.choice((1, 2, 3, 4, 5, 8, 16))
        if op == "append":
            new = _log(rng, 1, 4096)
            batch = _log(rng, 1, max(1, min(64, 32768 // new)))
            return dict(op=op, batch=batch, new=new, ctx=new + rng.randrange(0, 3000), ragged=rng.random() < 0.7, hq=hq,
                        hkv=hkv, dim=dim, page=page, mode=rng.choice(("max", "four_over_six")))
        new = rng.choice((1, 1, rng.randrange(2, 9), _log(rng, 9, 2048)))
        batch = _log(rng, 1, 64 if new < 64 else 4)
        most = min(100000, 600000 * 8 // (batch * hkv), 1200000000 // (batch * new * hq))
        ctx = _log(rng, max(16, min(new, most)), max(16, most))
        return dict(op=op, batch=batch, new=new, ctx=ctx, ragged=rng.random() < 0.6, hq=hq, hkv=hkv, dim=dim, page=page,
                    causal=rng.random() < 0.8, window=rng.choice((0, 0, 0, _log(rng, 16, 8192))))
    if op == "fork":
        return dict(op=op, parents=_log(rng, 1, 64), ways=rng.randrange(1, 17), ctx=_log(rng, 1, 16000),
                    hkv=rng.choice((1, 2, 4, 8)), dim=dim, page=page)
    width = rng.randrange(4, 97)
    return dict(op=op, pages=_log(rng, 96, 12000), slots=rng.randrange(2, 129), width=width, hkv=rng.choice((1, 2, 4)),
                dim=dim, page=page)


def _lengths(case):
    """(new tokens, cached tokens with the new ones) of each sequence, from the case alone."""
    b, new, ctx = case["batch"], case["new"], case["ctx"]
    if not case["ragged"]:
        return [new] * b, [ctx] * b
    r = random.Random("%d %d %d" % (b, new, ctx))
    n = [new] + [r.randint(max(1, new // 2), new) for _ in range(b - 1)]
    kv = [ctx] + [max(m, r.randint(max(1, ctx // 4), ctx)) for m in n[1:]]
    return n, kv


def _fork_lengths(case):
    r = random.Random("%d %d" % (case["parents"], case["ctx"]))
    return [case["ctx"]] + [r.randint(max(1, case["ctx"] // 2), case["ctx"]) for _ in range(case["parents"] - 1)]


def _compact_lengths(case):
    """Tokens of each slot: about half of the pool's pages in all, some slots empty."""
    r = random.Random("%d %d %d" % (case["pages"], case["slots"], case["width"]))
    most = case["width"] * case["page"]
    got, left = [], int(0.55 * case["pages"])
    for _ in range(case["slots"]):
        n = 0 if r.random() < 0.1 else r.randint(1, most)
        n = min(n, left * case["page"])
        left -= -(-n // case["page"])
        got.append(n)
    return got


# ------------------------------------------------------------------- encoding
def _e2m1_codes(v):
    a = v.abs()
    c = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return c | (torch.signbit(v).to(torch.uint8) << 3)


def _grid(device, dtype=torch.float32):
    return torch.tensor(_GRID + tuple(-x for x in _GRID), dtype=dtype, device=device)


def _encode(x, g, mode):
    """NVFP4 of BF16 values [..., D] under the static global scale g: (packed codes, block scale bytes)."""
    x = x.float().unflatten(-1, (-1, 16))
    bmax = x.abs().amax(-1)

    def under(target):
        s = (bmax / (target * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
        s = s.view(torch.uint8).clamp(min=1).view(torch.float8_e4m3fn)
        d = g * s.float()
        c = _e2m1_codes(x * (1.0 / d)[..., None])
        return s.view(torch.uint8), d, c

    s, d, c = under(6.0)
    if mode == "four_over_six":
        s4, d4, c4 = under(4.0)
        grid = _grid(x.device)

        def error(d, c):  # the squares summed in element order
            e = x - d[..., None] * grid[c.long()]
            return functools.reduce(torch.add, (e * e).unbind(-1))

        four = error(d4, c4) < error(d, c)
        s, c = torch.where(four, s4, s), torch.where(four[..., None], c4, c)
    c = c.flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), s


def _granules(k, v, k_g, v_g, mode):
    """Granules [..., 18*D] of K and V [..., 16, D]."""
    return torch.cat([p.flatten(-2) for x, g in ((k, k_g), (v, v_g)) for p in _encode(x, g, mode)], -1)


# -------------------------------------------------------------------- prepare
def _pool(gen, n, case, k_g, v_g):
    """A pool of n pages with quantized N(0, 1) keys and values, made a part at a time."""
    hkv, dim, page = case["hkv"], case["dim"], case["page"]
    pages = torch.empty((n, hkv, page // 16 * 18 * dim), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (hkv * page * dim))
    for a in range(0, n, step):
        m = min(step, n - a)
        kv = torch.randn((2, m, hkv, page // 16, 16, dim), device="cuda", generator=gen).to(torch.bfloat16)
        pages[a:a + m] = _granules(kv[0], kv[1], k_g, v_g, "max").flatten(2)
    return pages


def _int(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = random.Random(seed)
    page, op = case["page"], case["op"]
    s = dict(case, k_g=torch.tensor([_K_G], device="cuda"), v_g=torch.tensor([_V_G], device="cuda"))
    if op in ("attention", "append"):
        new, kv = _lengths(case)
        need = [-(-x // page) for x in kv]
        n = sum(need) + 3
        ids = rng.sample(range(n), sum(need))
        width = max(need) + 1
        table, at = [], 0
        for m in need:
            table.append(ids[at:at + m] + [-1] * (width - m))
            at += m
        total = sum(new)
        s.update(table=_int(table), cu=_int([sum(new[:i]) for i in range(len(new) + 1)]), kv_len=_int(kv), total=total,
                 max_new=max(new), max_kv=max(kv))
        # queries, keys and values of the new tokens lie side by side, as a fused projection leaves them
        qkv = torch.randn((total, case["hq"] + 2 * case["hkv"], case["dim"]), device="cuda", generator=gen)
        qkv = qkv.to(torch.bfloat16)
        s.update(q=qkv[:, :case["hq"]], k=qkv[:, case["hq"]:case["hq"] + case["hkv"]], v=qkv[:, case["hq"] + case["hkv"]:])
        s["pages"] = _pool(gen, n, case, s["k_g"], s["v_g"])
    elif op == "fork":
        lens, kids = _fork_lengths(case), case["parents"] * case["ways"]
        need = [-(-x // page) for x in lens]
        n = sum(need) + kids + 5
        ids = rng.sample(range(n), sum(need))
        width = max(need) + 2
        table, refs, at = [], [0] * n, 0
        for m in need:
            table.append(ids[at:at + m] + [-1] * (width - m))
            at += m
        for p in ids:
            refs[p] = 1
        table += [[-1] * width for _ in range(kids)]
        s.update(table=_int(table), refs=_int(refs), seq_len=_int(lens + [0] * kids), count=kids,
                 parent=_int([i // case["ways"] for i in range(kids)]),
                 child=_int([case["parents"] + i for i in range(kids)]), pages=_pool(gen, n, case, s["k_g"], s["v_g"]))
    else:
        lens = _compact_lengths(case)
        need = [-(-x // page) for x in lens]
        ids = rng.sample(range(case["pages"]), sum(need))
        refs, table, at = [0] * case["pages"], [], 0
        for i, m in enumerate(need):
            row = ids[at:at + m]
            at += m
            if i % 3 == 2:  # a fork: the first pages are its neighbour's
                both = min(m, need[i - 1]) // 2
                row[:both] = table[i - 1][:both]
            for p in row:
                refs[p] += 1
            table.append(row + [-1] * (case["width"] - m))
        s.update(table=_int(table), refs=_int(refs), seq_len=_int(lens), pages=_pool(gen, case["pages"], case, s["k_g"], s["v_g"]))
    return s


# ---------------------------------------------------------------- plain forms
def _places(s):
    """(sequence, place among its new tokens, position) of every new token."""
    t = torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    i = t - s["cu"][b]
    return b, i, s["kv_len"][b] - (s["cu"][b + 1] - s["cu"][b]) + i


def _plain_append(s):
    page, dim = s["page"], s["dim"]
    b, _, pos = _places(s)
    gran = s["pages"].view(s["pages"].shape[0], s["hkv"], page // 16, 18 * dim)
    at_page = s["table"][b, pos // page].long()[:, None]
    at_gran, row = (pos % page // 16)[:, None], (pos % 16)[:, None, None]
    head = torch.arange(s["hkv"], device="cuda")[None]
    base = 0
    for x, g in ((s["k"], s["k_g"]), (s["v"], s["v_g"])):
        codes, scales = _encode(x, g, s["mode"])
        for part in (codes, scales):
            w = part.shape[-1]
            byte = base + row * w + torch.arange(w, device="cuda")
            gran[at_page[..., None], head[..., None], at_gran[..., None], byte] = part
            base += 16 * w
    return s["pages"]


def _cached(s):
    """K and V of every sequence in FP32, [B, kv heads, tokens, D], padded with what the table's next pages hold."""
    dim, page = s["dim"], s["page"]
    w = -(-s["max_kv"] // page)
    got = s["pages"][s["table"][:, :w].clamp(min=0).long()]  # [B, w, heads, bytes]
    got = got.transpose(1, 2).unflatten(-1, (page // 16, 18 * dim)).flatten(2, 3)  # [B, heads, granules, 18*D]
    pair = torch.stack([_grid("cuda").repeat(16), _grid("cuda").repeat_interleave(16)], -1)

    def half(at, g):
        codes = got[..., at:at + 8 * dim].unflatten(-1, (16, dim // 2))
        scales = got[..., at + 8 * dim:at + 9 * dim].unflatten(-1, (16, dim // 16))
        x = pair[codes.long()].flatten(-2).unflatten(-1, (-1, 16))
        x *= (g * scales.contiguous().view(torch.float8_e4m3fn).float())[..., None]
        return x.flatten(-2).flatten(2, 3)

    return half(0, s["k_g"]), half(9 * dim, s["v_g"])


def _plain_attention(s):
    hkv, dim, group = s["hkv"], s["dim"], s["hq"] // s["hkv"]
    k, v = _cached(s)
    bsz, n, length = k.shape[0], s["max_new"], k.shape[2]
    i = torch.arange(n, device="cuda")
    at = (s["cu"][:-1, None] + i).clamp(max=s["total"] - 1)
    q = s["q"][at].float().unflatten(2, (hkv, group)).permute(0, 2, 3, 1, 4).reshape(bsz, hkv, group * n, dim)
    x = (q @ k.transpose(-1, -2)).view(bsz, hkv, group, n, length).mul_(1.0 / math.sqrt(dim))
    pos = (s["kv_len"] - (s["cu"][1:] - s["cu"][:-1]))[:, None] + i
    j = torch.arange(length, device="cuda")
    see = (j < s["kv_len"][:, None, None]).expand(bsz, n, length)
    if s["causal"]:
        see = see & (j <= pos[..., None])
    if s["window"]:
        see = see & (pos[..., None] - j < s["window"])
    x.masked_fill_(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(m.clamp(min=-3e38)).exp_()
    total = x.sum(-1, keepdim=True)
    out = (x.view(bsz, hkv, group * n, length) @ v).view(bsz, hkv, group, n, dim) / torch.where(total > 0, total, 1.0)
    b, i, _ = _places(s)
    out = out.permute(0, 3, 1, 2, 4).flatten(2, 3)[b, i].to(torch.bfloat16)
    lse = (m + total.log())[..., 0].permute(0, 3, 1, 2).flatten(2, 3)[b, i]
    return dict(out=out, lse=lse)


def _pages_of(lens, page):
    return (lens + page - 1) // page


def _plain_fork(s):
    table, refs, lens, page = s["table"], s["refs"], s["seq_len"], s["page"]
    parent, child = s["parent"].long(), s["child"].long()
    j = torch.arange(table.shape[1], device="cuda")
    # the children of the last pass go
    old = j < _pages_of(lens[child], page)[:, None]
    gone = table[child]
    refs.index_add_(0, torch.where(old, gone, 0).flatten().long(), -old.flatten().int())
    table[child] = torch.where(old, -1, gone)
    # full pages are shared, a part page is copied to the lowest free pages in the children's order
    length = lens[parent]
    full, part = length // page, length % page > 0
    rank = part.cumsum(0)
    free = torch.searchsorted((refs == 0).cumsum(0), rank)
    dst = torch.where(part, free, -1).int()
    row = table[parent]
    src = torch.where(part, row.gather(1, full[:, None].long())[:, 0], -1)
    share = j < full[:, None]
    refs.index_add_(0, torch.where(share, row, 0).flatten().long(), share.flatten().int())
    refs.index_add_(0, torch.where(part, dst, 0).long(), part.int())
    mine = torch.where(share, row, table[child])
    table[child] = torch.where((j == full[:, None]) & part[:, None], dst[:, None], mine)
    lens[child] = length
    # a child without a part page repeats the first copy that there is
    i = torch.where(part, torch.arange(s["count"], device="cuda"), part.int().argmax())
    s["pages"][dst[i].clamp(min=0).long()] = s["pages"][src[i].clamp(min=0).long()]
    return dict(refs=refs, table=table, seq_len=lens, src=src, dst=dst, pages=s["pages"])


def _plain_compact(s):
    refs, page, n = s["refs"], s["page"], s["refs"].shape[0]
    p = torch.arange(n, device="cuda")
    used = refs > 0
    live = used.sum()
    high, low = used & (p >= live), ~used & (p < live)
    most = max(1, n // 2)
    r = torch.arange(1, most + 1, device="cuda")
    moves = r <= high.sum()
    src = torch.where(moves, torch.searchsorted(high.cumsum(0), r), -1).int()
    dst = torch.where(moves, torch.searchsorted(low.cumsum(0), r), -1).int()
    here = torch.where(high, dst[(high.cumsum(0) - 1).clamp(0, most - 1)], p.int())
    new_refs = torch.zeros_like(refs).index_add_(0, torch.where(used, here, 0).long(), torch.where(used, refs, 0))
    held = torch.arange(s["table"].shape[1], device="cuda") < _pages_of(s["seq_len"], page)[:, None]
    table = torch.where(held, here[torch.where(held, s["table"], 0).long()], s["table"])
    # the rows behind the last move repeat the first one
    s["pages"][torch.where(moves, dst, dst[0]).clamp(min=0).long()] = s["pages"][torch.where(moves, src, src[0]).clamp(min=0).long()]
    return dict(refs=new_refs, table=table, src=src, dst=dst, live=live.int()[None], pages=s["pages"])


# ------------------------------------------------------------------------ run
def _own(s):
    import qad_nvfp4_quantize_b200 as nv
    cache = nv.KVCache(s["pages"], s["k_g"], s["v_g"], s["page"], s["dim"])
    if s["op"] == "attention":
        out, lse = nv.paged_attention(s["q"], cache, s["table"], s["cu"], s["kv_len"], causal=s["causal"],
                                      window=s["window"], max_q=s["max_new"], want_lse=True)
        return dict(out=out, lse=lse)
    if s["op"] == "append":
        nv.kv_append(cache, s["k"], s["v"], s["table"], s["cu"], s["kv_len"], mode=s["mode"])
        return s["pages"]
    if s["op"] == "fork":
        nv.kv_free(s["refs"], s["table"], s["seq_len"], s["child"], s["page"])
        src, dst = nv.kv_fork(s["refs"], s["table"], s["seq_len"], s["parent"], s["child"], s["page"])
        nv.kv_copy_pages(cache, src, dst)
        return dict(refs=s["refs"], table=s["table"], seq_len=s["seq_len"], src=src, dst=dst, pages=s["pages"])
    refs, table, src, dst, live = nv.kv_compact(s["refs"], s["table"], s["seq_len"], s["page"])
    nv.kv_copy_pages(cache, src, dst)
    return dict(refs=refs, table=table, src=src, dst=dst, live=live, pages=s["pages"])


def run(state):
    if own:
        return _own(state)
    plain = {"attention": _plain_attention, "append": _plain_append, "fork": _plain_fork, "compact": _plain_compact}
    return plain[state["op"]](state)


# ----------------------------------------------------------------------- work
def _seen(case):
    """Per sequence: (new tokens, pairs that the mask leaves, cached tokens that any new token sees)."""
    got = []
    for n, kv in zip(*_lengths(case)):
        pairs, first, last = 0, kv, 0
        for i in range(n):
            pos = kv - n + i
            hi = min(kv, pos + 1) if case["causal"] else kv
            lo = max(0, pos - case["window"] + 1) if case["window"] else 0
            if hi > lo:
                pairs += hi - lo
                first, last = min(first, lo), max(last, hi)
        got.append((n, pairs, max(0, last - first)))
    return got


def work(case):
    dim, hkv, page = case["dim"], case["hkv"], case["page"]
    token = hkv * dim * 18 // 16  # bytes of a token's K and V
    if case["op"] == "attention":
        seen = _seen(case)
        rows = sum(n for n, _, _ in seen) * case["hq"]
        data = sum(t for _, _, t in seen) * token
        tables = sum(-(-t // page) + 2 for _, _, t in seen) * 4
        return dict(bytes=data + rows * (4 * dim + 4) + tables, flops=4 * dim * case["hq"] * sum(p for _, p, _ in seen))
    if case["op"] == "append":
        n = sum(_lengths(case)[0])
        values = 2 * n * hkv * dim
        return dict(bytes=2 * values + n * token + 12 * case["batch"], flops=(20 if case["mode"] == "max" else 45) * values)
    if case["op"] == "fork":
        lens = _fork_lengths(case)
        ways, parts = case["ways"], sum(x % page > 0 for x in lens)
        full = sum(x // page for x in lens)
        meta = 4 * (full * (1 + 4 * ways) + full + 3 * len(lens) * ways + sum(-(-x // page) for x in lens))
        return dict(bytes=meta + (1 + ways) * parts * page * token, flops=0)
    need = [-(-x // page) for x in _compact_lengths(case)]
    # a share of the live pages as large as the free share lies above the live count
    shared = sum(min(m, need[i - 1]) // 2 for i, m in enumerate(need) if i % 3 == 2)
    live = sum(need) - shared
    moves = round(live * (case["pages"] - live) / case["pages"])
    meta = 4 * (2 * case["pages"] + 2 * sum(need) + case["slots"] + case["pages"])
    return dict(bytes=meta + 2 * moves * page * token, flops=0)


# ---------------------------------------------------------------------- exact
def exact(case, seed):
    """Attention from its definition in 64 bits, one sequence and head at a time; the other operators give whole numbers."""
    if case["op"] != "attention":
        return None
    s = prepare(case, seed)
    new, kv = _lengths(case)
    dim, page, hkv = case["dim"], case["page"], case["hkv"]
    group = case["hq"] // hkv
    out = torch.zeros((sum(new), case["hq"], dim), dtype=torch.float64, device="cuda")
    lse = torch.full((sum(new), case["hq"]), -math.inf, dtype=torch.float64, device="cuda")

    def value(c):  # sign, two exponent bits of bias 1, one mantissa bit
        e, m = (c >> 1 & 3).double(), (c & 1).double()
        mag = torch.where(e > 0, (1 + m / 2) * 2.0 ** (e - 1), m / 2)
        return torch.where(c >= 8, -mag, mag)

    def scale(c):  # four exponent bits of bias 7, three mantissa bits
        e, m = (c >> 3).double(), (c & 7).double()
        return torch.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7), m / 8 * 2.0 ** -6)

    at = 0
    for b, (n, length) in enumerate(zip(new, kv)):
        i = torch.arange(n, device="cuda")[:, None] + length - n
        j = torch.arange(length, device="cuda")[None]
        hidden = torch.zeros((n, length), dtype=torch.bool, device="cuda")
        if case["causal"]:
            hidden |= j > i
        if case["window"]:
            hidden |= i - j >= case["window"]
        ids = s["table"][b, :-(-length // page)].long()
        for h in range(hkv):
            raw = s["pages"][ids, h].reshape(-1, 18 * dim).int()
            both = []
            for start, g in ((0, _K_G), (9 * dim, _V_G)):
                c = raw[:, start:start + 8 * dim].reshape(-1, dim // 2)
                c = torch.stack([c & 15, c >> 4], -1).reshape(-1, dim)[:length]
                t = raw[:, start + 8 * dim:start + 9 * dim].reshape(-1, dim // 16)[:length]
                g = float(torch.tensor(g, dtype=torch.float32))
                both.append(value(c) * scale(t).repeat_interleave(16, -1) * g)
            for r in range(group):
                x = s["q"][at:at + n, h * group + r].double() @ both[0].T / math.sqrt(dim)
                x = x.masked_fill(hidden, -math.inf)
                top = torch.logsumexp(x, -1)
                lse[at:at + n, h * group + r] = top
                p = torch.exp(x - torch.where(top.isinf(), torch.zeros_like(top), top)[:, None])
                out[at:at + n, h * group + r] = p @ both[1]
        at += n
    return dict(out=out, lse=lse)
