"""Attention over the 8-bit cache where v_scales differ by many powers of two: the entries that carry the probability
keep their values, whatever the scales of entries that carry none (B200 only).

Tolerance.  A product p v_scale is held to 2^-16 relative and to 2^-22 of the head's largest product; its exponent, a
sum of magnitude up to 2^8, to 2^-16 (0.69 * 2 roundings of 2^-17); up to 1,200 fp32 additions to 2^-24 each (2^-13.8);
scores to ds, twice in p and twice in its sum; then one rounding to the output's type.  Nothing is added for values that
nothing attends to."""
import numpy as np
import pytest
import torch

import kv8_reference as ref
from test_gpu_kv8_attention import SCALE, gpu, make

pytestmark = pytest.mark.gpu


def loud_and_quiet(n, rows, Hq, H, order, far, down, dtype, seed):
    """n tokens in blocks of one: quiet ones and loud ones, whose v_scales are 2^far above.  Feature 0 of q and K puts
    the loud tokens' probability 2^-down below for even query heads and as far above for odd ones."""
    d = make([n + 3], [rows], Hq, H, 8, 1, n, seed=seed, dtype=dtype)
    rng = np.random.default_rng(seed)
    L = n + 3
    pages, _, _, _ = d["kc"].shape
    loud = np.zeros(L, bool)
    half = rng.permutation(L)[:max(1, L // 2)]
    loud[half] = True
    # log2 of the quiet scales: fp16 has to hold the loud values too (448 * 2^(12 - 6) < 65504)
    low = 12 - far if dtype == torch.float16 else -far // 2
    table = d["table"].numpy()
    K = rng.standard_normal((L, H, 256)) * 0.25
    kc, ks = d["kc"].numpy(), torch.ones_like(d["ks"]).numpy()
    vs = torch.ones_like(d["vs"]).numpy()
    step = down * np.log(2.0) / SCALE / 8.0          # what feature 0 has to add to K: q's is +-8
    for j in range(L):
        page, row = table[0, j // 8], j % 8
        K[j, :, 0] = -step if loud[j] else 0.0
        s = 2.0 ** np.ceil(np.log2(max(1.0, np.abs(K[j]).max()) / 448.0))
        ks[page, row] = s
        kc[page, row] = ref.encode(K[j] / s)
        vs[page, row] = 2.0 ** (low + (far if loud[j] else 0) - rng.integers(6, 9))
    d["ks"], d["vs"] = torch.from_numpy(ks), torch.from_numpy(vs)
    q = torch.randn((rows, Hq, 256), generator=torch.Generator().manual_seed(seed)).mul_(0.5)
    q[:, 0::2, 0], q[:, 1::2, 0] = 8.0, -8.0
    d["q"] = q.to(dtype)
    for t in range(rows):
        see = rng.permutation(L - rows + t + 1)[:n]
        key = {"quiet first": loud[see], "loud first": ~loud[see], "mixed": np.zeros(len(see), bool)}[order]
        see = see[np.argsort(key, kind="stable")]
        d["tok"][t] = torch.from_numpy(np.concatenate([see, np.full(n - len(see), -1)]).astype(np.int32))
    return d


def check(d, got, every=1):
    out, lse, w = got
    q, K8, V8 = d["q"].double().numpy(), d["kc"].numpy(), d["vc"].numpy()
    ks, vs = d["ks"].double().numpy(), d["vs"].double().numpy()
    fp16 = d["q"].dtype == torch.float16
    T, Hq, _ = q.shape
    G = Hq // K8.shape[2]
    rows = ref.rows_of(d["cu"].numpy(), d["sl"].numpy(), T)
    want_w, tol_w = np.zeros(w.shape), np.zeros(w.shape)
    for t, (r, pos) in list(enumerate(rows))[::every]:
        e, pg, rw = (np.array(c) for c in zip(*ref.visible(d["tok"][t].numpy(), r, pos, d["sl"].numpy(),
                                                           d["table"].numpy(), K8.shape[0], 8)))
        for h in range(Hq):
            g = h // G
            K = ref.VALUE[K8[pg, rw, g]] * ks[pg, rw, g][:, None]
            C, sc = np.abs(ref.VALUE[V8[pg, rw, g]]), vs[pg, rw, g]
            s = SCALE * (K @ q[t, h])
            ds = SCALE * float(np.max(2.0 ** -16 * (np.abs(K) @ np.abs(q[t, h])) +
                                      2.0 ** -22 * np.abs(q[t, h]).max() * np.abs(K).sum(1)))
            p = np.exp(s - s.max())
            want_lse = s.max() + np.log(p.sum())
            p /= p.sum()
            want = (p * sc) @ ref.VALUE[V8[pg, rw, g]]
            tol = (2.0 ** -16 + 2.0 ** -16 + 2.0 ** -13.8 + 4 * ds) * ((p * sc) @ C)
            tol += 2.0 ** -22 * (p * sc).max() * C.sum(0)
            tol += (2.0 ** -11 if fp16 else 2.0 ** -8) * np.abs(want) + (2.0 ** -25 if fp16 else 2.0 ** -134)
            err = np.abs(out[t, h] - want)
            assert np.all(err <= tol), (t, h, float(np.max(err / tol)), float(np.max(err / np.abs(want))))
            assert abs(lse[t, h] - want_lse) <= 2 * ds + 4e-6 * (abs(want_lse) + 1)
            np.add.at(want_w[t], e, p)
            np.add.at(tol_w[t], e, p * (4 * ds + 8e-6 * (abs(want_lse) + 1)) + 1e-12)
    assert np.all((np.abs(w - want_w) <= tol_w)[::every])


@pytest.mark.parametrize("order", ["quiet first", "loud first", "mixed"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,rows,Hq,H", [(2, 1, 24, 2), (130, 3, 24, 2), (300, 2, 32, 2), (300, 1, 8, 1), (1100, 1, 24, 2)])
@pytest.mark.parametrize("far,down", [(10, 60), (16, 20), (24, 30), (40, 60), (40, 42)])
def test_v_scales_of_unattended_entries_do_not_matter(n, rows, Hq, H, order, dtype, far, down):
    """Short lists (whole) and 9 tiles for one row (cut), every head count the kernel is built for."""
    if dtype == torch.float16:
        far = min(far, 26)
    check(*(lambda d: (d, gpu(d)))(loud_and_quiet(n, rows, Hq, H, order, far, down, dtype, seed=n + far)))


@pytest.mark.parametrize("order", ["quiet first", "loud first", "mixed"])
@pytest.mark.parametrize("n", [60, 1100])
def test_v_scales_over_the_whole_range(n, order):
    """2^-97 beside 2^83, about as far apart as the scales that appending writes (2^-64 to 2^120): a probability of 2^-170
    beside one of 1 is no number of fp32's."""
    d = loud_and_quiet(n, 1, 24, 2, order, 180, 170, torch.bfloat16, seed=n)
    check(d, gpu(d))


@pytest.mark.parametrize("Hq,H", [(8, 1), (24, 2), (32, 2)])
@pytest.mark.parametrize("dtype,first,later", [(t, *v) for t in (torch.bfloat16, torch.float16)
                                               for v in ((5, -25), (5, -90), (-90, 5), (60, -110), (-110, 60))
                                               if t == torch.bfloat16 or max(v) < 8])   # (fp16 ends at 65504)
def test_references_that_move_with_every_tile(Hq, H, dtype, first, later):
    """Scores that rise from tile to tile (2^5 each, for even heads; odd heads' fall) over the first tile's v_scales and
    the others': the references move with every tile, the units of the products must not drift, and v_scales come to
    lie far apart in the middle of a list, in either direction.  200 rows: runs of several tiles."""
    rows, n = 200, 1100
    d = loud_and_quiet(n, rows, Hq, H, "mixed", 12, 0, dtype, seed=5)
    see = np.random.default_rng(1).permutation(n + 3 - rows)
    d["tok"][:] = -1
    d["tok"][:, :len(see)] = torch.from_numpy(see.astype(np.int32))
    table = d["table"].numpy()
    for i, j in enumerate(see):
        page, row = table[0, j // 8], j % 8
        K = ref.VALUE[d["kc"][page, row].numpy()] * d["ks"][page, row].double().numpy()[:, None]
        K[:, 0] = 5.0 * (i // 128) * np.log(2.0) / SCALE / 8.0
        s = 2.0 ** np.ceil(np.log2(max(1.0, np.abs(K).max()) / 448.0))
        d["ks"][page, row] = float(s)
        d["kc"][page, row] = torch.from_numpy(ref.encode(K / s))
        d["vs"][page, row] = 2.0 ** (first if i < 128 else later)
    check(d, gpu(d), every=27)
