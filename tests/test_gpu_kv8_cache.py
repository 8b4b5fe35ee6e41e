"""Filling the 8-bit K/V cache, adding attention weights up and evicting pages (B200 only) against the 64-bit
reference.  Codes, scales, token weights, tables and page lists are exact."""
import numpy as np
import pytest
import torch

import kv8_reference as ref

pytestmark = pytest.mark.gpu

qsa = pytest.importorskip("sparse_attention_block_qsa_b200")
DEV = torch.device("cuda")


# ------------------------------------------------------------------ append

def append_inputs(seq_lens, qlens, H, ps, bt, seed, dtype=torch.bfloat16, spread=1.0):
    table, sl, cu, pages = ref.layout(seq_lens, qlens, ps, seed)
    kc, ks = ref.cache(pages, ps, H, bt, seed + 1)
    vc, vs = ref.cache(pages, ps, H, bt, seed + 2)
    g = torch.Generator().manual_seed(seed + 3)
    x = torch.randn((2, sum(qlens), H, 256), generator=g) * torch.exp(spread * torch.randn((2, sum(qlens), H, 1), generator=g))
    return dict(k=x[0].to(dtype), v=x[1].to(dtype), kc=kc, vc=vc, ks=ks, vs=vs, table=table, sl=sl, cu=cu)


def gpu_append(d, tw=None, **kw):
    c = {n: d[n].clone().to(DEV) for n in ("kc", "vc", "ks", "vs")}
    qsa.kv_append_fp8(d["k"].to(DEV), d["v"].to(DEV), c["kc"], c["vc"], c["ks"], c["vs"], d["table"].to(DEV),
                      d["cu"].to(DEV), d["sl"].to(DEV), token_weight=tw, **kw)
    torch.cuda.synchronize()
    return {n: c[n].cpu() for n in c}


def check_append(d, got, tw=None, got_tw=None):
    tw = None if tw is None else tw.clone().numpy()
    for x, c, s in (("k", "kc", "ks"), ("v", "vc", "vs")):
        codes, scales = d[c].clone().numpy(), d[s].double().numpy().copy()
        ref.append(d[x].double().numpy(), codes, scales, d["table"].numpy(), d["cu"].numpy(), d["sl"].numpy(), tw)
        assert np.array_equal(got[s].double().numpy(), scales)
        a, b = got[c].numpy(), codes
        nan = np.isnan(ref.VALUE[b])
        assert np.array_equal(a[~nan], b[~nan]) and np.all(np.isnan(ref.VALUE[a[nan]]))
    if tw is not None:
        assert np.array_equal(got_tw.cpu().numpy(), tw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("seq_lens,qlens,H,ps,bt", [
    ([1], [1], 1, 1, 1), ([1, 17, 16, 64, 33], [1, 1, 1, 1, 1], 2, 16, 16), ([70, 5, 200], [4, 3, 2], 2, 64, 16),
    ([300, 131, 77], [300, 130, 1], 2, 64, 64), ([500, 198], [333, 3], 4, 196, 49), ([90, 41], [37, 41], 5, 8, 1),
    ([700], [650], 1, 256, 256),
])
def test_append_matches_reference(seq_lens, qlens, H, ps, bt, dtype):
    d = append_inputs(seq_lens, qlens, H, ps, bt, seed=ps + bt, dtype=dtype)
    check_append(d, gpu_append(d))


def test_append_token_by_token_is_read_back():
    """One token at a time with growing magnitude: the scale grows, older codes follow, and what attention reads is
    within half an E4M3 step (2^-4 relative, 2^-10 of the scale for subnormals) of what was written, twice for
    tokens that were rescaled below the normal range."""
    ps, bt, n = 16, 8, 21
    table, _, _, pages = ref.layout([n], [1], ps, 1)
    c = [torch.zeros((pages, ps, 2, 256), dtype=torch.uint8, device=DEV) for _ in range(2)]
    s = [torch.zeros((pages, ps // bt, 2), device=DEV) for _ in range(2)]
    g = torch.Generator().manual_seed(5)
    x = (torch.randn((2, n, 2, 256), generator=g) * torch.exp2(torch.arange(n) % 7 - 3.0)[None, :, None, None]).to(torch.bfloat16)
    for i in range(n):
        qsa.kv_append_fp8(x[0, i:i + 1].to(DEV), x[1, i:i + 1].to(DEV), *c, *s, table.to(DEV),
                          torch.tensor([0, 1], dtype=torch.int32, device=DEV),
                          torch.tensor([i + 1], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    for w in range(2):
        for j in range(n):
            page, row = int(table[0, j // ps]), j % ps
            sc = s[w][page, row // bt].cpu().double().numpy()[:, None]
            got = ref.VALUE[c[w][page, row].cpu().numpy()] * sc
            want = x[w, j].double().numpy()
            assert np.all(np.abs(got - want) <= 2.0 ** -4 * np.abs(want) + 2 * 2.0 ** -10 * sc)


def test_append_overwrites_rejected_tokens():
    d = append_inputs([70, 30], [4, 4], 2, 64, 16, seed=4)
    c = gpu_append(d)
    d2 = dict(append_inputs([70, 30], [4, 4], 2, 64, 16, seed=14), table=d["table"], cu=d["cu"], **{n: c[n] for n in c})
    d2["sl"] = d["sl"] - 3                           # three of the four were rejected, four new ones follow
    check_append(d2, gpu_append(d2))


def test_append_special_values_missing_pages_and_weights():
    d = append_inputs([70, 40, 90], [20, 3, 50], 2, 16, 8, seed=6)
    d["k"][3, 0, 5], d["k"][4, 1, 9], d["v"][30, 0, 2] = float("nan"), float("inf"), float("-inf")
    d["k"][21] = 0                                   # request 1's rows: nothing but zeros in K
    d["k"][20], d["k"][22] = 0, 0
    d["v"][60:70] = float("nan")
    d["table"][2, 3] = -1
    d["table"][0, 3] = d["kc"].shape[0]
    tw = torch.arange(d["kc"].shape[0] * 16, dtype=torch.int64).view(-1, 16) + 1
    got_tw = tw.to(DEV)
    check_append(d, gpu_append(d, got_tw), tw, got_tw)


def test_append_extreme_magnitudes():
    d = append_inputs([40, 9], [40, 3], 2, 16, 16, seed=7)
    d["k"][:16] *= 2.0 ** 100
    d["k"][16:32] *= 2.0 ** -100
    d["v"][40:, 1] = 0
    check_append(d, gpu_append(d))


def test_append_padded_batch_and_short_requests():
    d = append_inputs([40, 5, 2, 30], [3, 0, 2, 4], 2, 16, 4, seed=8)
    d["k"], d["v"] = (torch.cat([d[n], d[n][:2]]) for n in "kv")   # two rows behind the last request's
    check_append(d, gpu_append(d))
    d["sl"][2] = 1                                   # two rows for a request of one token: the first has no position
    check_append(d, gpu_append(d))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("ps,bt", [(8, 2), (12, 3), (16, 4), (10, 5), (14, 7), (16, 8), (18, 9), (51, 17)])
def test_append_many_small_blocks(ps, bt, dtype):
    """Blocks that a warp takes, some with tokens in front, in requests of all alignments and in large numbers."""
    seq_lens, qlens = [450, 333, 5, 40, 9, 21], [450, 331, 2, 1, 4, 3]
    d = append_inputs(seq_lens, qlens, 4, ps, bt, seed=ps, dtype=dtype, spread=2.0)
    tw = torch.ones((d["kc"].shape[0], ps), dtype=torch.int64)
    got_tw = tw.to(DEV)
    check_append(d, gpu_append(d, got_tw), tw, got_tw)
    few = append_inputs(seq_lens[2:], qlens[2:], 1, ps, bt, seed=ps + 1, dtype=dtype, spread=2.0)
    check_append(few, gpu_append(few))


def test_append_behind_scales_that_are_no_powers_of_two(monkeypatch):
    """A block begun with another writer's scale keeps it while it is large enough.  What becomes a code is rounded to
    fp32 on the way: x / s once, an older value times s / s' twice (the ratio and the product), 2^-24 relative each.
    So a code is that of a value within 2^-23 of the exact one.  (With s = 1.3 * 2^n this does happen: 2.03125 / 1.3 =
    25 / 16 lies in the middle of two codes, and the fp32 value of 1.3 is 4e-8 below it.)"""
    exact = ref.encode
    for ps, bt in ((16, 16), (64, 64), (16, 4), (16, 8)):
        d = append_inputs([70, 40, 90, 31], [2, 1, 3, 2], 2, ps, bt, seed=15, spread=0.2)
        d["ks"], d["vs"] = d["ks"] * 1.3, d["vs"] * 37.7
        got = gpu_append(d)
        for x, c, n in (("k", "kc", "ks"), ("v", "vc", "vs")):
            either = []
            for off in (1 - 2.0 ** -23, 1 + 2.0 ** -23):
                monkeypatch.setattr(ref, "encode", lambda v: exact(np.asarray(v) * off))
                codes, scales = d[c].clone().numpy(), d[n].double().numpy().copy()
                ref.append(d[x].double().numpy(), codes, scales, d["table"].numpy(), d["cu"].numpy(), d["sl"].numpy())
                either.append(codes)
            assert np.array_equal(got[n].double().numpy(), scales)
            assert np.any(scales != 2.0 ** np.round(np.log2(scales)))
            assert np.all((got[c].numpy() == either[0]) | (got[c].numpy() == either[1]))


@pytest.mark.parametrize("bt", [1, 4, 16])
def test_append_rows_in_front_of_the_first_request(bt):
    """The requests of a batch's tail with the whole batch's rows: the head's are written nowhere."""
    d = append_inputs([40, 3, 90, 31], [20, 2, 33, 31], 2, 16, bt, seed=8)
    for n in (1, 2, 3):
        tail = dict(d, cu=d["cu"][n:], sl=d["sl"][n:], table=d["table"][n:])
        tail["ks"] = torch.zeros_like(d["ks"])       # (old scales of 0: a write to a wrong block would show)
        tw = torch.ones((d["kc"].shape[0], 16), dtype=torch.int64)
        got_tw = tw.to(DEV)
        check_append(tail, gpu_append(tail, got_tw), tw, got_tw)


def test_append_layouts():
    d = append_inputs([70, 5, 200], [4, 3, 2], 2, 64, 16, seed=9)
    want = gpu_append(d)
    pages = d["kc"].shape[0]
    pool = torch.zeros((pages, 2, 2, 64, 256), dtype=torch.uint8, device=DEV)
    pool[:, 0], pool[:, 1] = d["kc"].transpose(1, 2).to(DEV), d["vc"].transpose(1, 2).to(DEV)
    sc = torch.zeros((pages, 2, 4, 5), device=DEV)
    sc[:, 0, :, :2], sc[:, 1, :, :2] = d["ks"].to(DEV), d["vs"].to(DEV)
    qkv = torch.zeros((9, 7, 264), dtype=torch.bfloat16, device=DEV)
    qkv[:, 1:3, :256], qkv[:, 4:6, :256] = d["k"].to(DEV), d["v"].to(DEV)
    k = qkv[:, 1:3, :256].clone()                    # rotated keys are often a tensor of their own
    qsa.kv_append_fp8(k, qkv[:, 4:6, :256], pool[:, 0].transpose(1, 2), pool[:, 1].transpose(1, 2), sc[:, 0, :, :2],
                      sc[:, 1, :, :2], d["table"].to(DEV), d["cu"].to(DEV), d["sl"].to(DEV))
    torch.cuda.synchronize()
    assert torch.equal(pool[:, 0].transpose(1, 2).cpu(), want["kc"])
    assert torch.equal(pool[:, 1].transpose(1, 2).cpu(), want["vc"])
    assert torch.equal(sc[:, 0, :, :2].cpu(), want["ks"]) and torch.equal(sc[:, 1, :, :2].cpu(), want["vs"])
    assert torch.all(sc[:, :, :, 2:] == 0)


def test_append_behind_4_gib_and_on_another_stream():
    d = append_inputs([70, 40], [20, 3], 2, 64, 16, seed=19)
    want = gpu_append(d)
    pages, n = 140000, d["kc"].shape[0]
    pools = {k: torch.zeros((pages, *d[k].shape[1:]), dtype=d[k].dtype, device=DEV) for k in ("kc", "vc", "ks", "vs")}
    assert pools["kc"].numel() > 1 << 32
    at = torch.arange(n) + pages - n
    for k in pools:
        pools[k][at.to(DEV)] = d[k].to(DEV)
    table = torch.where(d["table"] >= 0, d["table"] + (pages - n), d["table"])
    x = [d[k].to(DEV) for k in "kv"]
    rest = [table.to(DEV), d["cu"].to(DEV), d["sl"].to(DEV)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    qsa.kv_append_fp8(*x, *pools.values(), *rest, stream=side)
    torch.cuda.synchronize()
    for k in pools:
        assert torch.equal(pools[k][pages - n:].cpu(), want[k])
        assert not torch.any(pools[k][:1000].view(torch.uint8))


def test_append_captured_into_a_graph():
    d = append_inputs([70, 5, 200], [4, 3, 2], 2, 64, 16, seed=9)
    want = gpu_append(d)
    c = {n: d[n].clone().to(DEV) for n in ("kc", "vc", "ks", "vs")}
    args = [d["k"].to(DEV), d["v"].to(DEV), *c.values(), d["table"].to(DEV), d["cu"].to(DEV), d["sl"].to(DEV)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qsa.kv_append_fp8(*args)
    for n in c:
        c[n].copy_(d[n])
    g.replay()
    g.replay()                                       # the same rows again: nothing more to grow
    torch.cuda.synchronize()
    assert all(torch.equal(c[n].cpu(), want[n]) for n in c)


# ------------------------------------------------------------------ accumulate

@pytest.mark.parametrize("ps,width", [(16, 1), (64, 130), (196, 700), (1, 33)])
def test_accumulate_is_exact(ps, width):
    seq_lens, qlens = [1, 300, 64, 1003, 1003], [1, 4, 3, 2, 30]
    table, sl, cu, pages = ref.layout(seq_lens, qlens, ps, 3)
    if pages > 8:
        table[4, :5] = table[3, :5]                  # a shared prefix
        table[1, 2] = -1
        table[3, 1] = pages
    tok = ref.token_lists(seq_lens, qlens, width, 4)
    g = torch.Generator().manual_seed(width)
    w = torch.exp(3 * torch.randn(tok.shape, generator=g)) * 1e-3
    w[0, 0] = float("nan")
    w[2, 0] = -1.0
    w[3, 0] = 1e30
    w[-1, -1] = float("inf")
    tw = torch.randint(0, 1 << 40, (pages, ps), generator=g)
    want = tw.clone().numpy()
    ref.accumulate(w.double().numpy(), tok.numpy(), table.numpy(), cu.numpy(), sl.numpy(), want)
    for _ in range(2):                               # the order of the additions does not matter
        got = tw.to(DEV)
        assert qsa.accumulate_weights(w.to(DEV), tok.to(DEV), table.to(DEV), cu.to(DEV), sl.to(DEV), got) is got
        torch.cuda.synchronize()
        assert np.array_equal(got.cpu().numpy(), want)


def test_accumulate_strides_padding_and_empty():
    table, sl, cu, pages = ref.layout([90, 50], [3, 2], 16, 5)
    tok = ref.token_lists([90, 50], [3, 2], 40, 6)
    tok = torch.cat([tok, tok[:2]])                  # rows behind the last request's add nothing
    w = torch.rand((7, 40))
    want = np.zeros((pages, 16), np.int64)
    ref.accumulate(w.double().numpy(), tok.numpy(), table.numpy(), cu.numpy(), sl.numpy(), want)
    got = torch.zeros((pages, 16), dtype=torch.int64, device=DEV)
    W, K = torch.ones((7, 47), device=DEV), torch.zeros((7, 45), dtype=torch.int32, device=DEV)
    W[:, :40], K[:, :40] = w.to(DEV), tok.to(DEV)
    args = table.to(DEV), cu.to(DEV), sl.to(DEV)
    qsa.accumulate_weights(W[:, :40], K[:, :40], *args, got)
    qsa.accumulate_weights(W[:, :0], K[:, :0], *args, got)
    qsa.accumulate_weights(W[:0, :40], K[:0, :40], args[0], args[1] * 0, args[2], got)
    torch.cuda.synchronize()
    assert np.array_equal(got.cpu().numpy(), want)


def test_accumulate_rows_in_front_of_the_first_request():
    table, sl, cu, pages = ref.layout([90, 50, 33], [3, 2, 4], 16, 6)
    tok = ref.token_lists([90, 50, 33], [3, 2, 4], 40, 7)
    w = torch.rand((9, 40))
    for n in (1, 2):
        want = np.zeros((pages, 16), np.int64)
        ref.accumulate(w.double().numpy(), tok.numpy(), table[n:].numpy(), cu[n:].numpy(), sl[n:].numpy(), want)
        got = torch.zeros((pages, 16), dtype=torch.int64, device=DEV)
        qsa.accumulate_weights(w.to(DEV), tok.to(DEV), table[n:].to(DEV), cu[n:].to(DEV), sl[n:].to(DEV), got)
        torch.cuda.synchronize()
        assert np.array_equal(got.cpu().numpy(), want)


# ------------------------------------------------------------------ eviction

def gpu_evict(tw, table, sl, keep, first, last, **kw):
    got = qsa.evict_pages(tw.to(DEV), table.to(DEV), sl.to(DEV), keep.to(DEV), first, last, **kw)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in got]


@pytest.mark.parametrize("ps,first,last", [(16, 0, 0), (16, 1, 1), (5, 2, 3), (64, 0, 1), (1, 1, 1)])
def test_evict_matches_reference(ps, first, last):
    seq_lens = [1, 2500, 64, 1003, 17, 0, 999]
    table, sl, cu, pages = ref.layout(seq_lens, [1] * 7, ps, ps)
    g = torch.Generator().manual_seed(ps)
    table[1, 3:9] = -1
    table[3, 2] = pages + 5
    tw = torch.randint(0, 4, (pages, ps), generator=g) << torch.randint(0, 40, (pages, 1), generator=g)
    for frac in (0.0, 0.3, 0.9, 2.0):
        keep = (torch.tensor([max(1, -(-n // ps)) for n in seq_lens]) * frac).to(torch.int32)
        keep[4] = -3
        want = ref.evict(tw.numpy(), table.numpy(), sl.numpy(), keep.numpy(), first, last)
        got = gpu_evict(tw, table, sl, keep, first, last)
        assert all(np.array_equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("tokens", [400, 90000])
def test_evict_extreme_counts(tokens):
    table, sl, cu, pages = ref.layout([tokens, tokens - 5, 30], [1, 1, 1], 16, 9)
    tw = torch.randint(0, 1 << 30, (pages, 16), generator=torch.Generator().manual_seed(2))
    for keep in (-2 ** 31, -1, 2 ** 31 - 1):
        k = torch.full((3,), keep, dtype=torch.int32)
        for first, last in ((2, 1), (2 ** 31 - 1, 0), (0, 2 ** 31 - 1)):
            want = ref.evict(tw.numpy(), table.numpy(), sl.numpy(), k.numpy(), first, last)
            got = gpu_evict(tw, table, sl, k, first, last)
            assert all(np.array_equal(a, b) for a, b in zip(got, want))


def test_evict_ties_keep_the_earlier_pages():
    table, sl, cu, pages = ref.layout([5000, 160], [1, 1], 16, 2)
    tw = torch.full((pages, 16), 3, dtype=torch.int64)
    keep = torch.tensor([100, 4], dtype=torch.int32)
    out, freed, counts = gpu_evict(tw, table, sl, keep, 1, 1)
    want = ref.evict(tw.numpy(), table.numpy(), sl.numpy(), keep.numpy(), 1, 1)
    assert all(np.array_equal(a, b) for a, b in zip((out, freed, counts), want))
    assert np.all(out[0, :99] >= 0) and np.all(out[0, 99:312] == -1) and out[0, 312] >= 0


def test_evict_large_and_negative_weights_and_strides():
    seq_lens = [40000, 33000]                        # more pages than one pass over the CTA takes
    table, sl, cu, pages = ref.layout(seq_lens, [1, 1], 8, 7)
    g = torch.Generator().manual_seed(1)
    tw = torch.randint(-(1 << 59), 1 << 59, (pages, 8), generator=g)
    keep = torch.tensor([2345, 0], dtype=torch.int32)
    want = ref.evict(tw.numpy(), table.numpy(), sl.numpy(), keep.numpy(), 1, 2)
    R, width = table.shape
    wide = torch.full((3, R, width + 9), -5, dtype=torch.int32, device=DEV)
    wide[0, :, :width] = table.to(DEV)
    t = wide[0, :, :width]
    ws = torch.empty(qsa.evict_pages_workspace_size(R, width, 8), dtype=torch.uint8, device=DEV)
    out, freed, counts = qsa.evict_pages(tw.to(DEV), t, sl.to(DEV), keep.to(DEV), 1, 2, table_out=t,
                                         freed=wide[1, :, :width], workspace=ws)
    torch.cuda.synchronize()
    assert out is t
    assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip((out, freed, counts), want))
    assert torch.all(wide[:2, :, width:] == -5)


@pytest.mark.parametrize("R,tokens,ps", [(2, 4000, 4), (3, 210000, 64), (150, 700, 1), (150, 9000, 4), (1, 90000, 16)])
def test_evict_forms(R, tokens, ps):
    """Tables of up to 1,024, 4,096 and more pages, few and many requests, short and long."""
    seq_lens = [max(1, tokens - 137 * i * tokens // 30000) for i in range(R)]
    table, sl, cu, pages = ref.layout(seq_lens, [1] * R, ps, R)
    g = torch.Generator().manual_seed(R)
    tw = torch.randint(0, 1 << 20, (pages, ps), generator=g) << torch.randint(0, 20, (pages, 1), generator=g)
    tw[: pages // 3] = 5                             # many equal pages
    keep = torch.tensor([-(-n // ps) * (1 + i % 5) // 6 for i, n in enumerate(seq_lens)], dtype=torch.int32)
    want = ref.evict(tw.numpy(), table.numpy(), sl.numpy(), keep.numpy(), 1, 1)
    got = gpu_evict(tw, table, sl, keep, 1, 1)
    assert all(np.array_equal(a, b) for a, b in zip(got, want))


def test_evict_captured_in_place():
    table, sl, cu, pages = ref.layout([5000, 160], [1, 1], 16, 2)
    tw = torch.randint(0, 1 << 40, (pages, 16), generator=torch.Generator().manual_seed(4))
    keep = torch.tensor([100, 4], dtype=torch.int32)
    want = ref.evict(tw.numpy(), table.numpy(), sl.numpy(), keep.numpy(), 1, 1)
    t, args = table.to(DEV), (tw.to(DEV), sl.to(DEV), keep.to(DEV))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _, freed, counts = qsa.evict_pages(args[0], t, args[1], args[2], 1, 1, table_out=t)
    for _ in range(2):
        t.copy_(table)
        g.replay()
        torch.cuda.synchronize()
        assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip((t, freed, counts), want))
    g.replay()                                       # the pages are gone already
    torch.cuda.synchronize()
    assert counts.tolist() == [0, 0] and torch.all(freed == -1) and np.array_equal(t.cpu().numpy(), want[0])


def test_evict_empty():
    z = torch.zeros(0, dtype=torch.int32, device=DEV)
    tw = torch.zeros((4, 16), dtype=torch.int64, device=DEV)
    out, freed, counts = qsa.evict_pages(tw, torch.zeros((0, 3), dtype=torch.int32, device=DEV), z, z)
    assert out.shape == (0, 3) and counts.shape == (0,)
    one = torch.ones(2, dtype=torch.int32, device=DEV)
    out, freed, counts = qsa.evict_pages(tw, torch.zeros((2, 0), dtype=torch.int32, device=DEV), one, one)
    torch.cuda.synchronize()
    assert out.shape == (2, 0) and counts.tolist() == [0, 0]


# ------------------------------------------------------------------ together

def test_decode_loop_with_eviction():
    """The operators as a serving loop uses them: prompts are appended, each step scores the compressed keys,
    selects blocks, attends over the 8-bit cache, adds the weights up; pages are evicted twice and the steps after
    run on the smaller table, which the compressed key cache shares."""
    ps, bt, H, Hq, k, steps = 32, 8, 2, 24, 12, 6
    lens, new = [400, 150], 2
    g = torch.Generator().manual_seed(3)
    total = [n + new * steps for n in lens]
    table, _, _, pages = ref.layout(total, [1, 1], ps, 11)
    kc, vc = (torch.zeros((pages, ps, H, 256), dtype=torch.float8_e4m3fn, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros((pages, ps // bt, H), device=DEV) for _ in range(2))
    index = torch.randn((pages, ps // 4, 1, 128), generator=g).to(torch.bfloat16)
    tw = torch.zeros((pages, ps), dtype=torch.int64, device=DEV)
    ref_tw = np.zeros((pages, ps), np.int64)
    rc = [np.zeros((pages, ps, H, 256), np.uint8) for _ in range(2)]
    rs = [np.zeros((pages, ps // bt, H)) for _ in range(2)]
    table_d = table.to(DEV)
    cur = list(lens)
    for step in range(-1, steps):
        q_lens = lens if step < 0 else [new, new]
        if step >= 0:
            cur = [c + new for c in cur]
        T = sum(q_lens)
        cu = torch.tensor([0, q_lens[0], T], dtype=torch.int32)
        sl = torch.tensor(cur, dtype=torch.int32)
        x = (torch.randn((2, T, H, 256), generator=g) * 2).to(torch.bfloat16)
        qsa.kv_append_fp8(x[0].to(DEV), x[1].to(DEV), kc, vc, ks, vs, table_d, cu.to(DEV), sl.to(DEV), token_weight=tw)
        for i in range(2):
            ref.append(x[i].double().numpy(), rc[i], rs[i], table.numpy(), cu.numpy(), sl.numpy(), ref_tw)
        if step < 0:
            continue
        qi = torch.randn((2, new, 4, 128), generator=g).to(torch.bfloat16)
        scores = qsa.mqa_decode(qi.to(DEV), index.to(DEV), table_d, sl.to(DEV), max(cur) // 4)
        blocks = qsa.topk(scores.view(T, -1), k)
        tok = qsa.expand_block_indices(blocks, cu.to(DEV), sl.to(DEV))
        q = torch.randn((T, Hq, 256), generator=g).to(torch.bfloat16)
        w = torch.empty(tok.shape, device=DEV)
        out, lse = qsa.sparse_attention_fp8(q.to(DEV), kc, vc, ks, vs, table_d, cu.to(DEV), sl.to(DEV), tok, 1 / 16, weights=w)
        qsa.accumulate_weights(w, tok, table_d, cu.to(DEV), sl.to(DEV), tw)
        torch.cuda.synchronize()
        want, wlse, ww, t_out, t_lse, t_w = ref.attention(
            q.double().numpy(), *rc, *rs, table.numpy(), cu.numpy(), sl.numpy(), tok.cpu().numpy(), 1 / 16)
        assert np.all(np.abs(out.cpu().double().numpy() - want) <= t_out)
        assert np.all(np.abs(lse.cpu().double().numpy() - wlse) <= t_lse)
        assert np.all(np.abs(w.cpu().double().numpy() - ww) <= t_w)
        ref.accumulate(w.cpu().double().numpy(), tok.cpu().numpy(), table.numpy(), cu.numpy(), sl.numpy(), ref_tw)
        assert np.array_equal(tw.cpu().numpy(), ref_tw)
        if step in (1, 3):
            keep = torch.tensor([8 - step, 4], dtype=torch.int32)
            got = qsa.evict_pages(tw, table_d, sl.to(DEV), keep.to(DEV), 1, 1, table_out=table_d)
            torch.cuda.synchronize()
            want = ref.evict(ref_tw, table.numpy(), sl.numpy(), keep.numpy(), 1, 1)
            assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(got, want)) and want[2].sum() > 0
            table = torch.from_numpy(want[0])
    assert np.array_equal(kc.view(torch.uint8).cpu().numpy(), rc[0])
    assert qsa.device_error() == 0
