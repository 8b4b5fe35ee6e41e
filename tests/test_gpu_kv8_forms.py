"""Every form that the 8-bit cache calls choose by size is reached and right (B200 only): attention whose thread blocks
take several lists each, in every instance of the kernel; blocks of 8 tokens that a warp appends; accumulation with 8
entries a lane; eviction of 1,025 to 4,096 pages in one launch, two tokens a load."""
import numpy as np
import pytest
import torch

import kv8_reference as ref
from test_gpu_kv8_attention import DEV, SCALE, make
from test_gpu_kv8_cache import append_inputs, check_append, gpu_append, gpu_evict

pytestmark = pytest.mark.gpu

qsa = pytest.importorskip("sparse_attention_block_qsa_b200")


def check_all_rows(d, out, lse, w):
    """kv8_reference.attention and its tolerances, all rows at once in fp64 on the GPU."""
    T, Hq, _ = d["q"].shape
    pages, ps, H, _ = d["kc"].shape
    G, bt = Hq // H, ps // d["ks"].shape[1]
    value = torch.from_numpy(ref.VALUE).to(DEV)
    step = 2.0 ** -11 if d["q"].dtype == torch.float16 else 2.0 ** -8
    cu, sl, table = d["cu"].long(), d["sl"].long(), d["table"].long()
    for a in range(0, T, 50):
        t = torch.arange(a, min(a + 50, T), device=DEV)
        r = torch.searchsorted(cu[1:], t, right=True)
        pos = sl[r] - (cu[r + 1] - t)
        j = d["tok"][t].long()
        lp = (j.clamp(min=0) // ps).clamp(max=table.shape[1] - 1)
        pg = table[r[:, None], lp]
        seen = (j >= 0) & (j <= pos[:, None]) & (pg >= 0) & (pg < pages)
        pg, row = pg.clamp(0, pages - 1), j.clamp(min=0) % ps
        want_w, tol_w = torch.zeros(j.shape, dtype=torch.float64, device=DEV), 0
        for g in range(H):
            K = value[d["kc"][pg, row, g].long()] * d["ks"].double()[pg, row // bt, g][..., None]
            V = value[d["vc"][pg, row, g].long()] * d["vs"].double()[pg, row // bt, g][..., None]
            q = d["q"][t, g * G:(g + 1) * G].double()
            s = (SCALE * torch.einsum("thd,twd->thw", q, K)).masked_fill(~seen[:, None], -torch.inf)
            p = torch.softmax(s, -1)
            want, want_lse = torch.einsum("thw,twd->thd", p, V), torch.logsumexp(s, -1)
            ds = SCALE * (2.0 ** -16 * torch.einsum("thd,twd->thw", q.abs(), K.abs()) + 2.0 ** -22 *
                          q.abs().amax(-1)[..., None] * K.abs().sum(-1)[:, None]).masked_fill(~seen[:, None], 0).amax(-1)
            n, vmax = seen.sum(-1), (V.abs() * seen[..., None]).amax((1, 2))
            tol = ((2.0 ** -12 + 2.0 ** -14 + 4 * ds)[..., None] * torch.einsum("thw,twd->thd", p, V.abs()) +
                   (n * 2.0 ** -26 * vmax)[:, None, None] + step * want.abs() + 1e-6)
            assert torch.all((out[t, g * G:(g + 1) * G].double() - want).abs() <= tol)
            assert torch.all((lse[t, g * G:(g + 1) * G] - want_lse).abs() <= 2 * ds + 4e-6 * (want_lse.abs() + 1))
            want_w += p.sum(1)
            tol_w = tol_w + (p * (4 * ds + 8e-6 * (want_lse.abs() + 1))[..., None] + 1e-12).sum(1)
        if w is not None:
            assert torch.all((w[t] - want_w).abs() <= tol_w)


@pytest.mark.parametrize("rows,width", [(600, 300), (90, 1500)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("Hq,H", [(4, 1), (12, 1), (16, 1), (32, 2)])
def test_runs_of_several_lists(Hq, H, dtype, rows, width):
    """600 lists of 3 tiles: several whole ones a run.  90 lists of 12 tiles: runs that end inside a list and go on with
    the next.  Some rows see nothing, some little."""
    d = make([width + 500] * (rows // 30), [30] * (rows // 30), Hq, H, 64, 32, width, seed=Hq + rows, dtype=dtype)
    d["tok"][7::30, 5:] = -1
    d = {k: v.to(DEV) for k, v in d.items()}
    args = [d[k] for k in ("q", "kc", "vc", "ks", "vs", "table", "cu", "sl", "tok")]
    w = torch.full(d["tok"].shape, 7.0, device=DEV)
    out, lse = qsa.sparse_attention_fp8(*args, SCALE, weights=w)
    bare, bare_lse = qsa.sparse_attention_fp8(*args, SCALE)
    torch.cuda.synchronize()
    assert qsa.device_error() == 0
    assert torch.equal(out, bare) and torch.equal(lse, bare_lse)
    check_all_rows(d, out, lse, w)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("ps,bt", [(16, 8), (14, 7), (20, 5)])
def test_append_blocks_of_up_to_8_tokens_a_warp(ps, bt, dtype):
    """So many that a warp takes each, full ones among them."""
    seq_lens, qlens = [900, 700, 5, 41, 650], [900, 695, 2, 9, 650]
    d = append_inputs(seq_lens, qlens, 4, ps, bt, seed=ps, dtype=dtype, spread=2.0)
    tw = torch.ones((d["kc"].shape[0], ps), dtype=torch.int64)
    got_tw = tw.to(DEV)
    check_append(d, gpu_append(d, got_tw), tw, got_tw)


@pytest.mark.parametrize("T,width", [(2000, 1291), (20000, 3)])
def test_accumulate_many_entries(T, width):
    ps, requests = 64, 5
    seq_lens, qlens = [3 * T // requests + 70 * i for i in range(requests)], [T // requests] * requests
    table, sl, cu, pages = ref.layout(seq_lens, qlens, ps, 3)
    table[1, 2] = -1
    rng = np.random.default_rng(T)
    tok = rng.integers(-3, max(seq_lens) + 5, (T, width)).astype(np.int32)
    w = np.exp(3 * rng.standard_normal((T, width))).astype(np.float32) * np.float32(1e-3)
    w[::7, ::3] = np.nan
    r = np.repeat(np.arange(requests), T // requests)
    pos = sl.numpy()[r] - (cu.numpy()[r + 1] - np.arange(T))
    page = table.numpy()[r[:, None], np.clip(tok // ps, 0, table.shape[1] - 1)]
    adds = (tok >= 0) & (tok <= pos[:, None]) & (page >= 0) & (w > 0)
    want = np.zeros((pages, ps), np.int64)
    np.add.at(want, (page[adds], tok[adds] % ps), np.rint(w[adds].astype(np.float64) * 2.0 ** 32).astype(np.int64))
    got = torch.zeros((pages, ps), dtype=torch.int64, device=DEV)
    qsa.accumulate_weights(torch.from_numpy(w).to(DEV), torch.from_numpy(tok).to(DEV), table.to(DEV), cu.to(DEV),
                           sl.to(DEV), got)
    torch.cuda.synchronize()
    assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("R,tokens,ps", [(2, 5000, 2), (3, 32000, 8), (5, 6000, 4), (2, 9000, 3)])
def test_evict_in_one_launch_with_several_pages_a_thread(R, tokens, ps):
    seq_lens = [tokens - 501 * i for i in range(R)]
    table, sl, cu, pages = ref.layout(seq_lens, [1] * R, ps, R)
    assert 1024 < table.shape[1] <= 4096 and qsa.evict_pages_workspace_size(R, table.shape[1], ps) == 0
    table[0, 5:900:7] = -1
    g = torch.Generator().manual_seed(R)
    tw = torch.randint(0, 1 << 20, (pages, ps), generator=g) << torch.randint(0, 20, (pages, 1), generator=g)
    tw[: pages // 3] = 5                             # many equal pages
    for part in (1, 3, 5):
        keep = torch.tensor([-(-n // ps) * part // 6 for n in seq_lens], dtype=torch.int32)
        want = ref.evict(tw.numpy(), table.numpy(), sl.numpy(), keep.numpy(), 1, 1)
        got = gpu_evict(tw, table, sl, keep, 1, 1)
        assert all(np.array_equal(a, b) for a, b in zip(got, want))
