"""What include/qsa.h promises of the 8-bit cache calls' arguments, seen from C (no GPU needed)."""
import random

import pytest

import sparse_attention_block_qsa_b200 as qsa
from test_kv8_refusals import A, ALIGN, INVALID, OK, S, UNSUP, WS, append, attn

REFUSALS = (INVALID, ALIGN, UNSUP, WS)


@pytest.mark.parametrize("name", ["qsa_sparse_attention_fp8", "qsa_sparse_attention_fp8_f16"])
@pytest.mark.parametrize("weights", [None, A + 11 * S])
def test_a_call_with_empty_lists_takes_the_workspace_that_its_size_says(name, weights):
    """Without lists the size is 0, and the call takes that: without a GPU it gets as far as CUDA's error."""
    assert qsa.lib().qsa_sparse_attention_fp8_workspace_size(8, 24, 2, 0, 1 if weights else 0) == 0
    st, detail = attn(name, width=0, tok=None, w=weights, ws=None, nbytes=0)
    assert st not in REFUSALS, (st, detail)


@pytest.mark.parametrize("kw", [
    dict(sps=1), dict(sps=6), dict(sps=4, sbs=8), dict(sps=10, sbs=3),             # pages or blocks that share scales
    dict(krs=256), dict(khs=512), dict(kps=64 * 512 - 256), dict(kps=256, krs=512), dict(khs=16384, krs=512),
    dict(vs=A + 3 * S + 4), dict(vs=A + 3 * S + 32), dict(ks=A + 4 * S + 99 * 32), dict(vc=A + S + 128),
    dict(vc=A + S + 256), dict(vc=A + S + 64 * 512), dict(kc=A + 2 * S + 99 * 64 * 512 + 63 * 512),
    dict(kps=64 * 1024, krs=1024, vc=A + S + 256), dict(Hkv=1, khs=0, krs=512, vc=A + S + 128),
])
@pytest.mark.parametrize("name", ["qsa_kv_append_fp8", "qsa_kv_append_fp8_f16"])
def test_append_refuses_rows_and_scales_that_overlap(name, kw):
    """They are written concurrently."""
    st, detail = append(name, **kw)
    assert st == INVALID and detail, (st, detail)


@pytest.mark.parametrize("kw", [
    dict(), dict(khs=64 * 256, krs=256), dict(kps=64 * 1024, krs=1024, vc=A + S + 512),      # heads outermost, K | V a row
    dict(kps=2 * 64 * 512, vc=A + S + 64 * 512), dict(kps=64 * 1024, krs=1024, khs=512, vc=A + S + 256),
    dict(kps=512, krs=51200), dict(kps=256, krs=51200, khs=25600), dict(sps=2, sbs=200), dict(sps=300, sbs=3), dict(sps=16, vs=A + 3 * S + 32),
    dict(sps=16, sbs=4, vs=A + 3 * S + 8), dict(sps=4, sbs=400, vs=A + 3 * S + 8), dict(vs=A + 3 * S + 100 * 32),
    dict(pages=1, kps=0, sps=0), dict(pages=1, ps=1, bt=1, kps=0, krs=0, sps=0, sbs=0), dict(bt=64, sbs=0, sps=2),
    dict(Hkv=1, khs=0, krs=512, vc=A + S + 256), dict(vc=A + S - 100 * 64 * 512), dict(vs=A + 3 * S - 100 * 32),
])
def test_append_takes_every_layout_without_overlap(kw):
    """Without a GPU an accepted call gets as far as CUDA's error."""
    st, detail = append(**dict(dict(kc=A + S, ksh=256, vsh=256), **kw))
    assert st not in REFUSALS, (st, detail)


def test_append_refuses_exactly_the_overlaps_of_nested_strides():
    """Against every pair of rows and of scales, for random small layouts."""
    rng = random.Random(1)
    refused = 0
    for _ in range(400):
        pages, ps, H = rng.choice([1, 2, 3]), rng.choice([1, 2, 4]), rng.choice([1, 2, 3])
        bt = rng.choice([n for n in (1, 2, 4) if ps % n == 0])
        nb = ps // bt
        dims, order = dict(kps=pages, krs=ps, khs=H), ["kps", "krs", "khs"]
        rng.shuffle(order)
        at, kw = 256, {}
        for n in order:                              # nested, the first innermost, with gaps
            kw[n] = at + rng.choice([0, 0, 128, 256, 512])
            at = kw[n] * dims[n] + (at - kw[n] if dims[n] == 1 else 0)
            at += -at % 16
        sdims, sorder = dict(sps=pages, sbs=nb), rng.sample(["sps", "sbs"], 2)
        sat = H
        for n in sorder:
            kw[n] = sat + rng.choice([0, 0, 1, H, 2 * H])
            sat = kw[n] * sdims[n]
        v, s = rng.randrange(-40, 40) * 128, rng.randrange(-24, 24)
        rows = [a * kw["kps"] + b * kw["krs"] + c * kw["khs"] for a in range(pages) for b in range(ps) for c in range(H)]
        sc = [a * kw["sps"] + b * kw["sbs"] for a in range(pages) for b in range(nb)]
        meet = any(abs(v + b - a) < 256 for a in rows for b in rows) or any(abs(s + b - a) < H for a in sc for b in sc)
        st, detail = append(pages=pages, ps=ps, bt=bt, Hkv=H, kst=1024, vst=1024, vc=A + S + v, vs=A + 3 * S + 4 * s, **kw)
        refused += meet
        assert (st == INVALID) == meet and (meet or st not in REFUSALS), (kw, v, s, st, detail)
    assert 100 < refused < 300, refused


def test_scales_that_pages_share_are_refused_by_attention_too():
    st, detail = attn(sps=1)
    assert st == INVALID and detail, (st, detail)
    st, detail = attn(vc=A + S, vs=A + 3 * S)        # (reading may share: K for V)
    assert st not in REFUSALS, (st, detail)
