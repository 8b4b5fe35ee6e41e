"""Measured cases of the 8-bit K/V cache operators: appending quantised tokens
(`kv_append_fp8`), sparse attention over the cache (`sparse_attention_fp8`),
adding its attention weights up per cached token (`accumulate_weights`) and
dropping the lightest pages (`evict_pages`).

Heads are 256 wide (the core attention's head dimension).  Block selections
follow the rule of the repository's own workloads: the k blocks of a row are
drawn uniformly without replacement from the 4-token blocks it can see.
"""
import math

import torch

own = False

D = 256          # head dimension
UNIT = 2.0 ** 32  # token weights are counted in units of 2^-32


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of a serving batch: 16 requests, one new token each, somewhere in a scale block
        dict(name="append_b16_q1", op="append", reqs=16, rows=1, lo=1, hi=2000, Hkv=2, ps=64, bt=16, f16=False),
        # a ragged prefill batch in fp16 over 196-token pages with 49-token scale blocks, 4 KV heads
        dict(name="append_ragged_f16", op="append", reqs=17, rows=131, lo=3, hi=1500, Hkv=4, ps=196, bt=49, f16=True),
        # one prefill chunk: 8,192 new tokens after 50,144 cached ones
        dict(name="append_prefill_8192", op="append", reqs=1, rows=8192, lo=50144, hi=50144, Hkv=2, ps=64, bt=16,
             f16=False),
        # one request decoding at 2,048 tokens: every block is selected, latency counts
        dict(name="attn_b1_q1_ctx2048", op="attn", reqs=1, rows=1, lo=2048, hi=2048, Hq=24, Hkv=2, ps=16, bt=16,
             k=512, f16=False, weights=False, gate=False),
        # 16 requests decoding in fp16, whose weights are wanted for eviction
        dict(name="attn_b16_q1_f16_weights", op="attn", reqs=16, rows=1, lo=1536, hi=43876, Hq=24, Hkv=2, ps=64,
             bt=64, k=512, f16=True, weights=True, gate=False),
        # the speculative step of the repository's own core-attention workload: 16 requests x 4 rows, top-512
        dict(name="attn_b16_q4_top512", op="attn", reqs=16, rows=4, lo=3508, hi=102400, Hq=24, Hkv=2, ps=64, bt=16,
             k=512, f16=False, weights=False, gate=False),
        # odd sizes: one KV head for 10 query heads, 49-token scale blocks in 196-token pages, gate and weights
        dict(name="attn_odd_gate_weights", op="attn", reqs=7, rows=3, lo=9, hi=5003, Hq=10, Hkv=1, ps=196, bt=49,
             k=77, f16=False, weights=True, gate=True),
        # prefill rows: two chunks of 512 rows each after long prefixes, top-512
        dict(name="attn_prefill_1024", op="attn", reqs=2, rows=512, lo=20000, hi=30000, Hq=24, Hkv=2, ps=64, bt=32,
             k=512, f16=False, weights=False, gate=False),
        # the weights of the speculative step
        dict(name="accumulate_b16_q4", op="accumulate", reqs=16, rows=4, lo=3508, hi=102400, ps=64, k=512),
        # the weights of a prefill chunk of two requests
        dict(name="accumulate_prefill_2048", op="accumulate", reqs=2, rows=1024, lo=20000, hi=30000, ps=64, k=512),
        # 16 long requests give up half of their pages
        dict(name="evict_b16_ps64", op="evict", reqs=16, lo=3508, hi=102400, ps=64, keep=0.5),
        # a large batch over small pages gives up a tenth
        dict(name="evict_b256_ps16", op="evict", reqs=256, lo=500, hi=40000, ps=16, keep=0.9),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "accumulate", "evict"])
    ps, bt = rng.choice([(16, 16), (16, 4), (64, 16), (64, 64), (64, 1), (196, 49), (100, 20), (32, 8)])
    if op == "append":
        reqs = _log_int(rng, 1, 64)
        rows = _log_int(rng, 1, max(1, 8000 // reqs))
        Hkv = rng.choice([1, 2, 4])
        lo = _log_int(rng, 1, 3000)
        return dict(op=op, reqs=reqs, rows=rows, lo=lo, hi=lo + _log_int(rng, 1, 3000), Hkv=Hkv, ps=ps, bt=bt,
                    f16=rng.random() < 0.5)
    if op == "evict":
        reqs = _log_int(rng, 1, 128)
        lo = _log_int(rng, 100, 10000)
        return dict(op=op, reqs=reqs, lo=lo, hi=lo + _log_int(rng, 100, 30000), ps=ps,
                    keep=round(rng.uniform(0.1, 1.0), 3))
    reqs = _log_int(rng, 1, 24)
    rows = rng.choice([1, 2, 3, 4]) if rng.random() < 0.7 else _log_int(rng, 5, max(6, 600 // reqs))
    lo = _log_int(rng, 5, 20000)
    hi = lo + _log_int(rng, 1, 40000)
    k = _log_int(rng, 1, 512)
    if op == "accumulate":
        return dict(op=op, reqs=reqs, rows=rows, lo=lo, hi=hi, ps=ps, k=k)
    Hq, Hkv = rng.choice([(24, 2), (12, 1), (16, 1), (10, 1), (8, 4), (32, 4), (5, 5)])
    return dict(op=op, reqs=reqs, rows=rows, lo=lo, hi=hi, Hq=Hq, Hkv=Hkv, ps=ps, bt=bt, k=k,
                f16=rng.random() < 0.3, weights=rng.random() < 0.5, gate=rng.random() < 0.3)


def _contexts(case):
    """Cached tokens of each request before its new rows: log-spaced between lo and hi, in a fixed order."""
    n, lo, hi = case["reqs"], case["lo"], case["hi"]
    if n == 1:
        return [hi]
    return [int(round(math.exp(math.log(lo) + (math.log(hi) - math.log(lo)) * ((i * 7) % n) / (n - 1))))
            for i in range(n)]


def _query_lens(case):
    """New rows of each request: `rows` each for decode shapes, ragged around it for larger ones."""
    n, rows = case["reqs"], case.get("rows", 1)
    if rows <= 4 or n <= 2:
        return [rows] * n
    return [max(1, rows + (i * 37) % 41 - 20) for i in range(n)]


# ------------------------------------------------------------------ inputs

def _layout(case, dev, g):
    """Page table (pages handed out by a random permutation), lengths and row offsets."""
    ctx, qlens = _contexts(case), _query_lens(case)
    lens = [c + n for c, n in zip(ctx, qlens)]
    ps = case["ps"]
    per = [-(-n // ps) for n in lens]
    pages = sum(per) + 1
    perm = torch.randperm(pages, device=dev, generator=g).to(torch.int32)
    width = max(per)
    cols = torch.arange(width, device=dev)[None]
    per_t = torch.tensor(per, device=dev)
    first = torch.cumsum(per_t, 0) - per_t
    table = torch.where(cols < per_t[:, None], perm[(first[:, None] + cols).clamp(max=pages - 1)],
                        torch.full((), -1, dtype=torch.int32, device=dev)).contiguous()
    seq_lens = torch.tensor(lens, dtype=torch.int32, device=dev)
    cu = torch.zeros(len(lens) + 1, dtype=torch.int32, device=dev)
    cu[1:] = torch.cumsum(torch.tensor(qlens, device=dev), 0).to(torch.int32)
    return table, seq_lens, cu, pages, sum(qlens)


def _row_positions(cu, seq_lens, T):
    """Request and logical position of every query row (row i of request r sits at seq_len - qlen + i)."""
    t = torch.arange(T, device=cu.device)
    req = torch.searchsorted(cu[1:].long(), t, right=True)
    qlen = (cu[1:] - cu[:-1]).long()
    return req, seq_lens.long()[req] - qlen[req] + t - cu.long()[req]


def _token_lists(cu, seq_lens, T, k, g):
    """k visible blocks per row, ascending, expanded to tokens and followed by the row's open group and -1."""
    dev = cu.device
    req, pos = _row_positions(cu, seq_lens, T)
    vis = (pos + 1) // 4
    most = max(k, int(vis.max()))
    tok = torch.full((T, 4 * k + 3), -1, dtype=torch.int32, device=dev)
    for a in range(0, T, 256):
        n = min(256, T - a)
        key = torch.rand((n, most), device=dev, generator=g)
        key.masked_fill_(torch.arange(most, device=dev)[None] >= vis[a:a + n, None], -1.0)
        val, blk = key.topk(k, dim=1)
        blk = torch.where(val >= 0, blk, torch.full_like(blk, 1 << 40)).sort(dim=1).values
        four = blk[:, :, None] * 4 + torch.arange(4, device=dev)
        four = torch.where(blk[:, :, None] < (1 << 40), four, torch.full_like(four, -1)).reshape(n, 4 * k)
        m = torch.clamp(vis[a:a + n], max=k) * 4
        open_tok = 4 * vis[a:a + n, None] + torch.arange(3, device=dev)
        open_tok = torch.where(open_tok <= pos[a:a + n, None], open_tok, torch.full_like(open_tok, -1))
        part = torch.cat([four, torch.full((n, 3), -1, device=dev)], 1)
        part.scatter_(1, m[:, None] + torch.arange(3, device=dev), open_tok)
        tok[a:a + n] = part.to(torch.int32)
    return tok


def _quantised(shape, bt, dev, g):
    """A pool [pages, page_size, Hkv, D] of codes with a power-of-two scale per block of bt tokens and head; rows
    are normal, and blocks differ in size."""
    pages, ps, H, _ = shape
    nb = ps // bt
    codes = torch.empty((pages, nb, bt, H, D), dtype=torch.float8_e4m3fn, device=dev)
    scales = torch.empty((pages, nb, H), dtype=torch.float32, device=dev)
    step = max(1, (1 << 26) // (ps * H * D))
    for a in range(0, pages, step):
        n = min(step, pages - a)
        x = torch.randn((n, nb, bt, H, D), device=dev, generator=g)
        x *= torch.exp(0.5 * torch.randn((n, nb, 1, H, 1), device=dev, generator=g))
        s = _pow2_scale(x.abs().amax(dim=(2, 4)))
        codes[a:a + n] = (x / s[:, :, None, :, None]).to(torch.float8_e4m3fn)
        scales[a:a + n] = s
    return codes.view(pages, ps, H, D), scales


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    table, seq_lens, cu, pages, T = _layout(case, dev, g)
    s = dict(op=case["op"], table=table, seq_lens=seq_lens, cu=cu, T=T)
    ps = case["ps"]
    if case["op"] == "evict":
        w = torch.exp(2.0 * torch.randn((pages, ps), device=dev, generator=g) +
                      torch.randn((pages, 1), device=dev, generator=g)) * 0.01
        s["token_weight"] = (w.double() * UNIT).round().to(torch.int64)
        live = (seq_lens + ps - 1) // ps
        s["keep"] = torch.ceil(live.float() * case["keep"]).to(torch.int32)
        return s
    if case["op"] == "accumulate":
        s["token_weight"] = torch.randint(0, 1 << 34, (pages, ps), device=dev, generator=g)
        tok = _token_lists(cu, seq_lens, T, case["k"], g)
        x = torch.exp(1.5 * torch.randn(tok.shape, device=dev, generator=g)) * (tok >= 0)
        s["tok"], s["weights"] = tok, 24.0 * x / x.sum(1, keepdim=True)
        return s
    dt = torch.float16 if case["f16"] else torch.bfloat16
    H = case["Hkv"]
    s["k_cache"], s["k_scale"] = _quantised((pages, ps, H, D), case["bt"], dev, g)
    s["v_cache"], s["v_scale"] = _quantised((pages, ps, H, D), case["bt"], dev, g)
    if case["op"] == "append":
        x = torch.randn((2, T, H, D), device=dev, generator=g)
        x *= torch.exp(0.7 * torch.randn((2, T, H, 1), device=dev, generator=g))
        s["k"], s["v"] = x[0].to(dt), x[1].to(dt)
        return s
    s["q"] = torch.randn((T, case["Hq"], D), device=dev, generator=g).to(dt)
    s["tok"] = _token_lists(cu, seq_lens, T, case["k"], g)
    s["gate"] = 2.0 * torch.randn((T, case["Hq"]), device=dev, generator=g) if case["gate"] else None
    s["weights"] = torch.empty(s["tok"].shape, dtype=torch.float32, device=dev) if case["weights"] else None
    return s


# ------------------------------------------------------------------ plain forms

def _pow2_scale(amax):
    """The smallest power of two s >= 2^-64 with amax <= 448 s (448 is E4M3's largest finite value)."""
    m, e = torch.frexp(amax.float())                                 # 448 is 0.875 * 2^9
    return torch.ldexp(torch.ones_like(m), torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-64))


def _plain_append(s):
    k_cache = s["k_cache"]
    pages, ps, H, _ = k_cache.shape
    nb = s["k_scale"].shape[1]
    bt = ps // nb
    req, pos = _row_positions(s["cu"], s["seq_lens"], s["T"])
    row = s["table"].long()[req, pos // ps] * ps + pos % ps          # pool row of every new token
    blk = row // bt                                                  # pool block of every new token
    # only the block that holds a request's first new token can hold older tokens
    p0 = s["seq_lens"].long() - (s["cu"][1:] - s["cu"][:-1]).long()
    page0 = torch.gather(s["table"].long(), 1, (p0 // ps)[:, None])[:, 0]
    old = p0 % ps % bt                                               # its tokens from before
    blk0 = (page0 * ps + p0 % ps) // bt
    for x, cache, scale in ((s["k"], k_cache, s["k_scale"]), (s["v"], s["v_cache"], s["v_scale"])):
        x = x.float()
        sc = scale.view(-1, H)
        codes = cache.view(torch.uint8).view(-1, H, D)
        amax = torch.zeros_like(sc).scatter_reduce_(0, blk[:, None].expand(-1, H), x.abs().amax(-1), "amax")
        need = _pow2_scale(amax)
        before = sc[blk0].clone()
        s0 = torch.where((old > 0)[:, None], torch.maximum(before, need[blk0]), need[blk0])
        sc[blk] = need[blk]
        sc[blk0] = s0
        rows0 = blk0[:, None] * bt + torch.arange(bt, device=x.device)
        was = codes[rows0]
        again = (was.view(torch.float8_e4m3fn).float() * (before / s0)[:, None, :, None]).to(torch.float8_e4m3fn)
        keep = (torch.arange(bt, device=x.device) < old[:, None])[:, :, None, None]
        codes[rows0] = torch.where(keep, again.view(torch.uint8), was)
        codes[row] = (x / sc[blk][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)


def _gathered(s, cache, scale, wide):
    """K or V rows of every list entry, [T, width, Hkv, D], as the values they stand for."""
    pages, ps, H, _ = cache.shape
    bt = ps // scale.shape[1]
    row, _ = _entries(s, ps)
    x = cache.view(torch.uint8).view(-1, H, D)[row].view(torch.float8_e4m3fn).to(wide)
    return x * scale.view(-1, H)[row // bt].to(wide)[..., None]


def _entries(s, ps):
    """Pool row and visibility of every list entry."""
    tok = s["tok"].long()
    req, pos = _row_positions(s["cu"], s["seq_lens"], s["T"])
    seen = (tok >= 0) & (tok <= pos[:, None]) & (tok < s["seq_lens"].long()[req][:, None])
    j = torch.where(seen, tok, torch.zeros_like(tok))
    page = s["table"].long()[req[:, None], j // ps]
    seen &= page >= 0
    return page.clamp(min=0) * ps + j % ps, seen


def _plain_attention(s):
    q = s["q"].float()
    T, Hq, _ = q.shape
    ps, H = s["k_cache"].shape[1:3]
    _, seen = _entries(s, ps)
    k = _gathered(s, s["k_cache"], s["k_scale"], torch.float32)
    sc = torch.einsum("thgd,twhd->thgw", q.view(T, H, Hq // H, D), k) / 16.0
    del k
    sc.masked_fill_(~seen[:, None, None, :], -math.inf)
    top = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + torch.log(total)).view(T, Hq)
    out = torch.einsum("thgw,twhd->thgd", p, _gathered(s, s["v_cache"], s["v_scale"], torch.float32)).reshape(T, Hq, D)
    if s["gate"] is not None:
        out = out / (1.0 + torch.exp(-s["gate"]))[..., None]
    out = out.to(s["q"].dtype)
    return (out, lse) if s["weights"] is None else (out, lse, p.sum((1, 2)))


def _plain_accumulate(s):
    row, seen = _entries(s, s["token_weight"].shape[1])
    add = torch.where(seen, (s["weights"].double() * UNIT).round().to(torch.int64), 0)
    s["token_weight"].view(-1).scatter_add_(0, row.reshape(-1), add.reshape(-1))


def _plain_evict(s):
    table, keep = s["table"], s["keep"].long()
    R, width = table.shape
    pages, ps = s["token_weight"].shape
    lp = torch.arange(width, device=table.device)[None]
    n = ((s["seq_lens"].long() + ps - 1) // ps)[:, None]
    live = (lp < n) & (table >= 0)
    held = live & ((lp < 1) | (lp >= n - 1))                         # the first and the last page always stay
    w = s["token_weight"].sum(1)[table.clamp(min=0).long()]
    free = live & ~held
    # heaviest first, the earlier page among equals; what may not go sorts behind
    order = torch.where(free, w, torch.full_like(w, -1)).sort(dim=1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, lp.expand(R, -1).contiguous())
    gone = free & (rank >= (keep - held.sum(1))[:, None])
    out = torch.where(gone, torch.full_like(table, -1), table)
    at = torch.where(gone, torch.cumsum(gone, 1) - 1, torch.full_like(order, width))
    freed = torch.full((R, width + 1), -1, dtype=torch.int32, device=table.device)
    freed.scatter_(1, at, torch.where(gone, table, torch.full_like(table, -1)))
    return out, freed[:, :width].contiguous(), gone.sum(1).to(torch.int32)


def run(s):
    if s["op"] == "append":
        if own:
            import sparse_attention_block_qsa_b200 as qsa
            qsa.kv_append_fp8(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"],
                              s["cu"], s["seq_lens"])
        else:
            _plain_append(s)
        return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    if s["op"] == "attn":
        if own:
            import sparse_attention_block_qsa_b200 as qsa
            out, lse = qsa.sparse_attention_fp8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                                s["table"], s["cu"], s["seq_lens"], s["tok"], 1.0 / 16.0,
                                                gate=s["gate"], weights=s["weights"])
            return (out, lse) if s["weights"] is None else (out, lse, s["weights"])
        return _plain_attention(s)
    if s["op"] == "accumulate":
        if own:
            import sparse_attention_block_qsa_b200 as qsa
            qsa.accumulate_weights(s["weights"], s["tok"], s["table"], s["cu"], s["seq_lens"], s["token_weight"])
        else:
            _plain_accumulate(s)
        return s["token_weight"]
    if own:
        import sparse_attention_block_qsa_b200 as qsa
        return qsa.evict_pages(s["token_weight"], s["table"], s["seq_lens"], s["keep"], keep_first=1, keep_last=1)
    return _plain_evict(s)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    ctx, qlens = _contexts(case), _query_lens(case)
    T, ps = sum(qlens), case["ps"]
    tables = 4 * sum(-(-(c + n) // ps) for c, n in zip(ctx, qlens))
    if case["op"] == "append":
        rows = T * case["Hkv"] * D * 2                               # K and V elements
        scales = 8 * case["Hkv"] * (T // case["bt"] + case["reqs"])
        return {"bytes": rows * 3 + scales, "flops": 2 * rows}
    if case["op"] == "evict":
        tokens = sum(c + n for c, n in zip(ctx, qlens))
        return {"bytes": 8 * tokens + 3 * tables, "flops": tokens}
    k = case["k"]
    entries, distinct = 0.0, 0.0
    for c, n in zip(ctx, qlens):
        vis = [(c + i + 1) // 4 for i in range(n)]
        take = [min(k, v) for v in vis]
        entries += sum(4 * a + 2 for a in take)
        missed = 1.0
        for a, v in zip(take, vis):
            missed *= 1.0 - a / max(v, 1)
        distinct += (c + n) * (1.0 - missed) if max(vis) > 0 else c + n
    lists = T * (4 * k + 3) * 4
    if case["op"] == "accumulate":
        return {"bytes": 2 * lists + 16 * distinct, "flops": entries}
    Hq, H = case["Hq"], case["Hkv"]
    scales = 8 * H * distinct / case["bt"]
    moved = distinct * H * D * 2 + scales + T * Hq * (4 * D + 4) + lists
    if case["weights"]:
        moved += lists
    return {"bytes": moved, "flops": entries * Hq * D * 4}


# ------------------------------------------------------------------ the definition in 64 bits

def _e4m3(x):
    """x rounded to E4M3 (3 fraction bits, smallest normal 2^-6, ties to even), values up to 448."""
    a = x.abs().clamp(min=2.0 ** -6)
    step = torch.exp2(torch.floor(torch.log2(a)) - 3.0)
    step = torch.where(a < 8.0 * step, step / 2, torch.where(a >= 16.0 * step, step * 2, step))   # log2's rounding
    return torch.round(x / step) * step


def _exact_append(s):
    ps, H = s["k_cache"].shape[1:3]
    nb = s["k_scale"].shape[1]
    bt = ps // nb
    lens, cu, table = s["seq_lens"].tolist(), s["cu"].tolist(), s["table"].tolist()
    res = []
    for x, cache, scale in ((s["k"], s["k_cache"], s["k_scale"]), (s["v"], s["v_cache"], s["v_scale"])):
        c, sc, x = cache.double().view(-1, bt, H, D), scale.double().view(-1, H), x.double()
        for r, L in enumerate(lens):
            first = L - (cu[r + 1] - cu[r])
            a = first
            while a < L:                                             # one scale block at a time
                b = min((a // ps) * ps + (a % ps // bt + 1) * bt, L)
                at = table[r][a // ps] * nb + a % ps // bt
                lo = a % ps % bt
                new = x[cu[r] + a - first:cu[r] + b - first]
                top = new.abs().amax(dim=(0, 2))
                want = torch.exp2(torch.floor(torch.log2(top)).clamp(min=-56.0) - 8.0)
                want = torch.where((top <= 224.0 * want) & (want > 2.0 ** -64), want / 2, want)  # log2's rounding
                want = torch.where(top > 448.0 * want, want * 2, want)
                if lo:
                    want = torch.maximum(want, sc[at])
                    c[at, :lo] = _e4m3(c[at, :lo] * (sc[at] / want)[None, :, None])
                c[at, lo:lo + b - a] = _e4m3(new / want[None, :, None])
                sc[at] = want
                a = b
        res.append((c.view(cache.shape), sc.view(scale.shape)))
    return res[0][0], res[1][0], res[0][1], res[1][1]


def _exact_attention(s):
    q = s["q"].double()
    T, Hq, _ = q.shape
    ps, H = s["k_cache"].shape[1:3]
    bt = ps // s["k_scale"].shape[1]
    lens, cu = s["seq_lens"].tolist(), s["cu"].tolist()
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=q.device)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=q.device)
    wts = torch.zeros(s["tok"].shape, dtype=torch.float64, device=q.device)
    for r, L in enumerate(lens):
        for t in range(cu[r], cu[r + 1]):
            pos = L - (cu[r + 1] - t)
            at = torch.nonzero((s["tok"][t] >= 0) & (s["tok"][t] <= pos) & (s["tok"][t] < L))[:, 0]
            j = s["tok"][t, at].long()
            pg = s["table"][r, j // ps].long()
            ok = pg >= 0
            at, j, pg = at[ok], j[ok], pg[ok]
            if at.numel() == 0:
                continue
            b = j % ps // bt
            K = s["k_cache"].view(torch.uint8)[pg, j % ps].view(torch.float8_e4m3fn).double()
            V = s["v_cache"].view(torch.uint8)[pg, j % ps].view(torch.float8_e4m3fn).double()
            K, V = K * s["k_scale"].double()[pg, b][..., None], V * s["v_scale"].double()[pg, b][..., None]
            for h in range(H):
                heads = slice(h * (Hq // H), (h + 1) * (Hq // H))
                x = q[t, heads] @ K[:, h].T / 16.0
                lse[t, heads] = torch.logsumexp(x, 1)
                p = torch.softmax(x, 1)
                out[t, heads] = p @ V[:, h]
                wts[t, at] += p.sum(0)
    if s["gate"] is not None:
        out = out * torch.sigmoid(s["gate"].double())[..., None]
    return (out, lse) if s["weights"] is None else (out, lse, wts)


def exact(case, seed):
    if case["op"] in ("accumulate", "evict"):
        return None                                                  # whole numbers only
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attention(s)
