"""Sparse attention over the 8-bit K/V cache (B200 only) against the 64-bit reference, whose docstring derives the
tolerances."""
import numpy as np
import pytest
import torch

import kv8_reference as ref

pytestmark = pytest.mark.gpu

qsa = pytest.importorskip("sparse_attention_block_qsa_b200")
DEV = torch.device("cuda")
SCALE = 1.0 / 16.0


def make(seq_lens, qlens, Hq, H, ps, bt, width, seed, dtype=torch.bfloat16, pow2=True):
    table, sl, cu, pages = ref.layout(seq_lens, qlens, ps, seed)
    kc, ks = ref.cache(pages, ps, H, bt, seed + 1, pow2)
    vc, vs = ref.cache(pages, ps, H, bt, seed + 2, pow2)
    g = torch.Generator().manual_seed(seed + 3)
    q = torch.randn((sum(qlens), Hq, 256), generator=g).to(dtype)
    tok = ref.token_lists(seq_lens, qlens, width, seed + 4)
    return dict(q=q, kc=kc, vc=vc, ks=ks, vs=vs, table=table, cu=cu, sl=sl, tok=tok)


def gpu(d, gate=None, weights=True, **kw):
    w = torch.full(d["tok"].shape, 7.0, device=DEV) if weights else None
    out, lse = qsa.sparse_attention_fp8(d["q"].to(DEV), d["kc"].to(DEV), d["vc"].to(DEV), d["ks"].to(DEV),
                                        d["vs"].to(DEV), d["table"].to(DEV), d["cu"].to(DEV), d["sl"].to(DEV),
                                        d["tok"].to(DEV), SCALE, gate=None if gate is None else gate.to(DEV), weights=w,
                                        **kw)
    torch.cuda.synchronize()
    assert qsa.device_error() == 0
    return out.cpu().double().numpy(), lse.cpu().double().numpy(), None if w is None else w.cpu().double().numpy()


def check(d, got, gate=None):
    out, lse, w = got
    step = 2.0 ** -11 if d["q"].dtype == torch.float16 else 2.0 ** -8
    want, wlse, ww, t_out, t_lse, t_w = ref.attention(
        d["q"].double().numpy(), d["kc"].numpy(), d["vc"].numpy(), d["ks"].double().numpy(), d["vs"].double().numpy(),
        d["table"].numpy(), d["cu"].numpy(), d["sl"].numpy(), d["tok"].numpy(), SCALE,
        None if gate is None else gate.double().numpy(), step)
    empty = np.isneginf(wlse)
    assert np.array_equal(np.isneginf(lse), empty)
    assert np.all(out[empty] == 0)
    live = ~empty
    assert np.all(np.abs(out - want)[live] <= t_out[live]), np.max(np.abs(out - want)[live] / t_out[live])
    assert np.all(np.abs(lse[live] - wlse[live]) <= t_lse[live])
    if w is not None:
        assert np.all(np.abs(w - ww) <= t_w), np.max(np.abs(w - ww) / np.maximum(t_w, 1e-30))
        assert np.all(w[t_w == 0] == 0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("Hq,H,ps,bt,width", [
    (24, 2, 16, 16, 163), (16, 1, 64, 16, 128), (4, 1, 196, 49, 129), (5, 5, 8, 1, 77), (1, 1, 1, 1, 5),
    (12, 1, 64, 64, 700), (30, 2, 100, 20, 1),
])
def test_matches_reference(Hq, H, ps, bt, width, dtype):
    d = make([1, 300, 64, 1003], [1, 4, 3, 2], Hq, H, ps, bt, width, seed=Hq + ps, dtype=dtype)
    check(d, gpu(d))


def test_no_weights_gives_the_same_output():
    d = make([700, 31], [2, 3], 24, 2, 64, 16, 300, seed=3)
    a, b = gpu(d), gpu(d, weights=False)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_gate_missing_pages_and_empty_rows():
    d = make([600, 1500, 40], [4, 3, 2], 24, 2, 16, 8, 250, seed=11)
    d["table"][1, 3] = -1
    d["table"][0, 1] = d["kc"].shape[0]              # one past the pool
    d["table"][1, 5:40] = -7
    d["tok"][2, :] = -1
    d["tok"][5, :] = 1500                            # past the request
    gate = torch.randn((9, 24), generator=torch.Generator().manual_seed(3)) * 3
    check(d, gpu(d, gate), gate)


def test_scales_that_are_no_powers_of_two_and_differ_widely():
    d = make([500, 90], [3, 2], 24, 2, 64, 4, 200, seed=5, pow2=False)
    f = torch.exp2(torch.randint(-12, 13, d["vs"].shape, generator=torch.Generator().manual_seed(1)).float())
    d["vs"] = d["vs"] * f
    d["ks"] = d["ks"] * torch.exp2(torch.randint(-3, 2, d["ks"].shape, generator=torch.Generator().manual_seed(2)).float())
    check(d, gpu(d))


def test_zero_scores_give_exact_means():
    """All keys zero: equal probabilities, so the output is the mean of the visible values up to its rounding."""
    d = make([900, 2000], [3, 2], 24, 2, 64, 16, 600, seed=7)
    d["kc"] = torch.zeros_like(d["kc"])
    d["vc"] = torch.from_numpy(ref.encode(np.random.default_rng(1).integers(-4, 5, d["vc"].shape)))
    d["vs"] = torch.ones_like(d["vs"])
    out, lse, w = gpu(d)
    want, wlse, ww, *_ = ref.attention(d["q"].double().numpy(), d["kc"].numpy(), d["vc"].numpy(), d["ks"].double().numpy(),
                                       d["vs"].double().numpy(), d["table"].numpy(), d["cu"].numpy(), d["sl"].numpy(),
                                       d["tok"].numpy(), SCALE)
    # values up to 4 times probabilities that are exact before one division: half a bf16 step of the result
    assert np.all(np.abs(out - want) <= 2.0 ** -8 * np.abs(want) + 1e-6)
    assert np.allclose(lse, wlse, rtol=1e-6, atol=1e-6)
    assert np.allclose(w, ww, rtol=1e-5, atol=0)


def test_one_token_gives_its_value_exactly():
    d = make([300], [1], 24, 2, 64, 16, 9, seed=8)
    d["tok"][:] = -1
    d["tok"][0, 4] = 217
    out, lse, w = gpu(d)
    page = int(d["table"][0, 217 // 64])
    for h in range(24):
        g = h // 12
        v = ref.VALUE[d["vc"][page, 217 % 64, g].numpy()] * float(d["vs"][page, 217 % 64 // 16, g])
        assert np.array_equal(out[0, h], v)          # 4 significant bits and a power of two: a bf16 value
    assert w[0, 4] == pytest.approx(24.0, abs=1e-5) and np.count_nonzero(w) == 1


def test_nan_in_masked_tokens_does_not_show():
    d = make([300, 200], [2, 2], 24, 2, 16, 16, 60, seed=9)
    want = gpu(d)
    listed = set()
    for t, (r, pos) in enumerate(ref.rows_of(d["cu"].numpy(), d["sl"].numpy(), 4)):
        listed |= {(p, w) for _, p, w in ref.visible(d["tok"][t].numpy(), r, pos, d["sl"].numpy(), d["table"].numpy(),
                                                     d["kc"].shape[0], 16)}
    used = {(p, 0) for p, _ in listed}
    for p in range(d["kc"].shape[0]):
        for w in range(16):
            if (p, w) not in listed:
                d["kc"][p, w] = 127
                d["vc"][p, w] = 255
        if (p, 0) not in used:
            d["ks"][p] = float("nan")
            d["vs"][p] = float("inf")
    got = gpu(d)
    assert all(np.array_equal(a, b) for a, b in zip(want, got))


def test_nan_query_head_gives_nan_there_only():
    d = make([300], [2], 24, 2, 16, 16, 60, seed=10)
    want = gpu(d, weights=False)
    d["q"][1, 3, 17] = float("nan")
    d["q"][0, 20, 200] = float("inf")
    got = gpu(d, weights=False)
    bad = np.zeros((2, 24), bool)
    bad[1, 3] = bad[0, 20] = True
    assert np.all(np.isnan(got[0][bad])) and np.all(np.isnan(got[1][bad]))
    assert np.array_equal(got[0][~bad], want[0][~bad]) and np.array_equal(got[1][~bad], want[1][~bad])


def test_extreme_queries():
    d = make([300], [2], 24, 2, 16, 16, 60, seed=12)
    d["q"][0] = 0
    d["q"][1, :6] *= 2.0 ** -100
    d["q"][1, 6:12] *= 8.0
    check(d, gpu(d))


def test_padded_rows_belong_to_no_request():
    d = make([300, 65], [2, 1], 24, 2, 16, 16, 60, seed=13)
    want = gpu(d)
    d["q"] = torch.cat([d["q"], d["q"][:2]])
    d["tok"] = torch.cat([d["tok"], d["tok"][:2]])
    got = gpu(d)
    assert all(np.array_equal(a, b[:3]) for a, b in zip(want, got))
    assert np.all(got[0][3:] == 0) and np.all(np.isneginf(got[1][3:])) and np.all(got[2][3:] == 0)


def test_layouts_give_the_same_bits():
    """Heads outermost inside a page, K and V interleaved in one pool, strided q, out and lists."""
    d = make([500, 90], [3, 2], 24, 2, 64, 16, 200, seed=14)
    want = gpu(d)
    pages, ps, H, _ = d["kc"].shape
    pool = torch.zeros((pages, 2, H, ps, 256), dtype=torch.uint8, device=DEV)
    pool[:, 0] = d["kc"].transpose(1, 2).to(DEV)
    pool[:, 1] = d["vc"].transpose(1, 2).to(DEV)
    sc = torch.zeros((pages, 2, ps // 16, H + 3), device=DEV)
    sc[:, 0, :, :H], sc[:, 1, :, :H] = d["ks"].to(DEV), d["vs"].to(DEV)
    q = torch.zeros((5, 3, 24, 264), dtype=torch.bfloat16, device=DEV)
    q[:, 1, :, :256] = d["q"].to(DEV)
    tok = torch.full((5, 205), 3, dtype=torch.int32, device=DEV)
    tok[:, :200] = d["tok"].to(DEV)
    out = torch.zeros((5, 26, 256), dtype=torch.bfloat16, device=DEV)
    w = torch.full((5, 210), -1.0, device=DEV)
    _, lse = qsa.sparse_attention_fp8(q[:, 1, :, :256], pool[:, 0].transpose(1, 2).view(torch.float8_e4m3fn),
                                      pool[:, 1].transpose(1, 2).view(torch.float8_e4m3fn), sc[:, 0, :, :H],
                                      sc[:, 1, :, :H], d["table"].to(DEV), d["cu"].to(DEV), d["sl"].to(DEV),
                                      tok[:, :200], SCALE, out=out[:, :24], weights=w[:, :200])
    torch.cuda.synchronize()
    assert np.array_equal(out[:, :24].cpu().double().numpy(), want[0]) and torch.all(out[:, 24:] == 0)
    assert np.array_equal(lse.cpu().double().numpy(), want[1])
    assert np.array_equal(w[:, :200].cpu().double().numpy(), want[2]) and torch.all(w[:, 200:] == -1)


def test_split_counts_agree():
    """Rows alone (many splits) and in a large batch (one split) agree within the sum of their tolerances."""
    d = make([2100] * 40, [8] * 40, 24, 2, 64, 16, 900, seed=15)
    big = gpu(d)
    one = dict(d, q=d["q"][:8], table=d["table"][:1], cu=d["cu"][:2], sl=d["sl"][:1], tok=d["tok"][:8])
    small = gpu(one)
    check(one, small)
    check(one, tuple(x[:8] for x in big))


@pytest.mark.parametrize("Hq,H,width,rows", [(24, 2, 5000, 1), (4, 1, 2400, 2), (24, 2, 2310, 1), (8, 4, 9000, 3)])
def test_lists_cut_into_many_pieces(Hq, H, width, rows):
    """More pieces a row (up to 40) than the merge loads in one round, with and without weights."""
    d = make([width + 300], [rows], Hq, H, 64, 16, width, seed=22)
    got = gpu(d)
    check(d, got)
    bare = gpu(d, weights=False)
    assert np.array_equal(got[0], bare[0]) and np.array_equal(got[1], bare[1])


def test_another_stream_and_a_captured_replay():
    d = {k: v.to(DEV) for k, v in make([700, 31], [2, 3], 24, 2, 64, 16, 300, seed=16).items()}
    args = [d[k] for k in ("q", "kc", "vc", "ks", "vs", "table", "cu", "sl", "tok")]
    want, want_lse = qsa.sparse_attention_fp8(*args, SCALE)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream, 0):
        out, lse = qsa.sparse_attention_fp8(*args, SCALE, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    # two graphs that share a workspace, replayed in turn
    ws = torch.empty(qsa.sparse_attention_fp8_workspace_size(5, 24, 2, 300), dtype=torch.uint8, device=DEV)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(qsa.sparse_attention_fp8(*args, SCALE, workspace=ws)[0])
        graphs.append(g)
    for n in (0, 1, 0):
        ws.fill_(255)
        outs[n].zero_()
        graphs[n].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[n], want)


def test_empty_calls():
    d = {k: v.to(DEV) for k, v in make([70], [2], 24, 2, 16, 16, 8, seed=17).items()}
    out, lse = qsa.sparse_attention_fp8(d["q"][:0], d["kc"], d["vc"], d["ks"], d["vs"], d["table"], d["cu"] * 0, d["sl"],
                                        d["tok"][:0], SCALE)
    assert out.shape == (0, 24, 256) and lse.shape == (0, 24)
    w = torch.empty((2, 0), device=DEV)
    out, lse = qsa.sparse_attention_fp8(d["q"], d["kc"], d["vc"], d["ks"], d["vs"], d["table"], d["cu"], d["sl"],
                                        d["tok"][:, :0], SCALE, weights=w)
    torch.cuda.synchronize()
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse))


def test_blocks_that_hold_nothing_are_not_seen():
    """A k_scale of 0: the block's tokens are masked for that head, whatever its codes and v_scale are."""
    for Hq, dtype in ((24, torch.bfloat16), (32, torch.bfloat16), (24, torch.float16)):
        d = make([300, 64], [2, 3], Hq, 2, 16, 8, 60, seed=18, dtype=dtype)
        d["ks"][:, 0, 1] = 0
        d["ks"][3] = 0
        d["vs"][:, 0, 1] = float("nan")
        d["ks"][d["table"][1, :4].long()] = 0            # nothing is left for the second request
        check(d, gpu(d))


def test_nan_codes_of_blocks_that_hold_nothing_do_not_show():
    """Pools whose scales alone were zeroed: the codes of blocks never written may be NaN."""
    for Hq, dtype in ((24, torch.bfloat16), (32, torch.bfloat16), (24, torch.float16), (32, torch.float16)):
        d = make([300, 400], [2, 3], Hq, 2, 16, 8, 300, seed=20, dtype=dtype)
        d["ks"][d["table"][:, 1].long(), 1] = 0
        d["ks"][d["table"][:, 3].long(), :, 0] = 0
        want = gpu(d)
        for c in ("kc", "vc"):
            b = d[c].view(-1, 2, 8, 2, 256)
            b[(d["ks"] == 0)[:, :, None, :].expand(-1, -1, 8, -1)] = 255
        got = gpu(d)
        check(d, got)
        assert all(np.array_equal(a, b) for a, b in zip(want, got))


def test_rows_in_front_of_the_first_request_belong_to_none():
    """The requests of a batch's tail with the whole batch's rows."""
    d = make([300, 65, 90], [2, 5, 1], 24, 2, 16, 16, 60, seed=21)
    tail = dict(d, cu=d["cu"][1:], sl=d["sl"][1:], table=d["table"][1:])
    got = gpu(tail)
    check(tail, got)
    assert np.all(np.isneginf(got[1][:2])) and np.all(got[0][:2] == 0) and np.all(got[2][:2] == 0)
    assert all(np.array_equal(a[2:], b[2:]) for a, b in zip(gpu(d), got))
    for n in (1, 2, 5):                              # and one request alone
        last = dict(d, cu=d["cu"][2:], sl=d["sl"][2:], table=d["table"][2:], q=d["q"][:n], tok=d["tok"][:n])
        assert np.all(np.isneginf(gpu(last)[1]))


@pytest.mark.parametrize("rows,width", [(600, 300), (90, 1500)])
def test_many_rows(rows, width):
    """Runs of whole lists (600 rows of 3 tiles) and runs that cut lists (90 rows of 12 tiles)."""
    d = make([width + 500] * (rows // 30), [30] * (rows // 30), 4, 1, 64, 32, width, seed=19)
    check(d, gpu(d))


def test_rows_behind_4_gib():
    """A pool whose last pages lie more than 2^32 bytes from its start."""
    ps, H, pages = 64, 2, 140000
    pool = torch.empty((pages, ps, H, 256), dtype=torch.uint8, device=DEV)
    assert pool.numel() > 1 << 32
    ks = torch.ones((pages, 4, H), device=DEV)
    small = make([200], [2], 24, H, ps, 16, 150, seed=20)
    want = gpu(small)
    n = small["kc"].shape[0]
    at = torch.randperm(1000)[:n] + pages - 1000
    table = small["table"].clone()
    table[table >= 0] = at[small["table"][table >= 0].long()].to(torch.int32)
    vp, vs = torch.empty_like(pool), ks.clone()
    for dst, src in ((pool, "kc"), (vp, "vc"), (ks, "ks"), (vs, "vs")):
        dst[at.to(DEV)] = small[src].to(DEV)
    d = dict(small, kc=pool, vc=vp, ks=ks, vs=vs, table=table)
    got = gpu(d)
    assert all(np.array_equal(a, b) for a, b in zip(want, got))


def test_two_calls_at_once_on_two_streams():
    a = {k: v.to(DEV) for k, v in make([3000] * 20, [8] * 20, 24, 2, 64, 16, 900, seed=21).items()}
    b = {k: v.to(DEV) for k, v in make([700, 31], [2, 3], 24, 2, 64, 16, 300, seed=22).items()}
    names = ("q", "kc", "vc", "ks", "vs", "table", "cu", "sl", "tok")
    want = [qsa.sparse_attention_fp8(*[d[k] for k in names], SCALE) for d in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [qsa.sparse_attention_fp8(*[d[k] for k in names], SCALE, stream=s) for d, s in zip((a, b), streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for g, w in zip(got, want) for x, y in zip(g, w))
    assert qsa.device_error() == 0
