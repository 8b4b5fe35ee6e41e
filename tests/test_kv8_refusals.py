"""The 8-bit K/V cache calls refuse bad arguments on the host, before any CUDA call (no GPU needed)."""
import pytest
import torch

import sparse_attention_block_qsa_b200 as qsa

OK, INVALID, ALIGN, UNSUP, WS = 0, 1, 2, 3, 4
A = 0x7f0000000000      # fake device addresses: validation never dereferences them
S = 1 << 28             # distance between fake buffers
CACHE = dict(kc=A + S, vc=A + 2 * S, ks=A + 3 * S, vs=A + 4 * S, pages=100, ps=64, bt=16, kps=64 * 512, krs=512, khs=256,
             sps=8, sbs=2, Hkv=2, pt=A + 5 * S, pts=10, maxp=10, cu=A + 6 * S, sl=A + 7 * S, R=4)


def cache_args(a):
    return [a[n] for n in ("kc", "vc", "ks", "vs", "pages", "ps", "bt", "kps", "krs", "khs", "sps", "sbs", "Hkv", "pt",
                           "pts", "maxp", "cu", "sl", "R")]


def call(name, *args):
    L = qsa.lib()
    return getattr(L, name)(*args), L.qsa_last_error_detail().decode()


def append(name="qsa_kv_append_fp8", **kw):
    a = dict(CACHE, k=A, kst=512, ksh=256, v=A + S // 2, vst=512, vsh=256, T=8, tw=None)
    a.update(kw)
    return call(name, a["k"], a["kst"], a["ksh"], a["v"], a["vst"], a["vsh"], *cache_args(a), a["T"], a["tw"], None)


def attn(name="qsa_sparse_attention_fp8", **kw):
    a = dict(CACHE, q=A, qst=6144, qsh=256, Hq=24, tok=A + 8 * S, tst=67, width=67, T=8, gate=None, scale=0.0625,
             out=A + 9 * S, ost=6144, lse=A + 10 * S, w=A + 11 * S, wst=67, ws=A + 12 * S, nbytes=1 << 27)
    a.update(kw)
    return call(name, a["q"], a["qst"], a["qsh"], a["Hq"], *cache_args(a), a["tok"], a["tst"], a["width"], a["T"],
                a["gate"], a["scale"], a["out"], a["ost"], a["lse"], a["w"], a["wst"], a["ws"], a["nbytes"], None)


def accumulate(**kw):
    a = dict(w=A, wst=67, tok=A + S, tst=67, width=67, T=8, pt=A + 2 * S, pts=10, maxp=10, cu=A + 3 * S, sl=A + 4 * S,
             R=4, tw=A + 5 * S, pages=100, ps=64)
    a.update(kw)
    return call("qsa_accumulate_weights", *[a[n] for n in ("w", "wst", "tok", "tst", "width", "T", "pt", "pts", "maxp",
                                                            "cu", "sl", "R", "tw", "pages", "ps")], None)


def evict(**kw):
    a = dict(tw=A, pages=100, ps=64, pt=A + S, pts=10, maxp=10, sl=A + 2 * S, keep=A + 3 * S, R=4, first=1, last=1,
             out=A + 4 * S, ost=10, freed=A + 5 * S, fst=10, counts=A + 6 * S, ws=A + 7 * S, nbytes=1 << 20)
    a.update(kw)
    return call("qsa_evict_pages", *[a[n] for n in ("tw", "pages", "ps", "pt", "pts", "maxp", "sl", "keep", "R", "first",
                                                     "last", "out", "ost", "freed", "fst", "counts", "ws", "nbytes")],
                None)


CACHE_CASES = [
    (dict(kc=0), INVALID), (dict(vs=0), INVALID), (dict(kc=A + S + 8), ALIGN), (dict(ks=A + 3 * S + 2), ALIGN),
    (dict(ps=0), INVALID), (dict(bt=0), INVALID), (dict(bt=24), INVALID), (dict(bt=128), INVALID),
    (dict(pages=0), INVALID), (dict(pages=1 << 31), INVALID), (dict(Hkv=0), UNSUP), (dict(kps=64 * 512 + 8), ALIGN),
    (dict(krs=-512), ALIGN), (dict(krs=240), INVALID), (dict(khs=128), INVALID), (dict(kps=128), INVALID),
    (dict(sbs=1), INVALID), (dict(sps=0), INVALID), (dict(R=-1), INVALID), (dict(R=0), INVALID), (dict(T=-1), INVALID),
    (dict(T=1 << 31), UNSUP), (dict(maxp=-1), INVALID), (dict(pt=0), INVALID), (dict(pts=9), INVALID),
    (dict(cu=0), INVALID), (dict(cu=A + 6 * S + 2), ALIGN),
]


@pytest.mark.parametrize("name", ["qsa_kv_append_fp8", "qsa_kv_append_fp8_f16"])
@pytest.mark.parametrize("kw,code", CACHE_CASES + [
    (dict(k=0), INVALID), (dict(v=A + S // 2 + 8), ALIGN), (dict(kst=516), ALIGN), (dict(vsh=-256), ALIGN),
    (dict(tw=A + 4), ALIGN), (dict(k=A + S + 512), INVALID), (dict(v=A + 2 * S), INVALID), (dict(vc=A + S), INVALID),
    (dict(vs=A + 3 * S), INVALID),
])
def test_append_refuses(name, kw, code):
    st, detail = append(name, **kw)
    assert st == code and detail, (st, detail)


@pytest.mark.parametrize("name", ["qsa_sparse_attention_fp8", "qsa_sparse_attention_fp8_f16"])
@pytest.mark.parametrize("kw,code", CACHE_CASES + [
    (dict(Hq=23), UNSUP), (dict(Hq=34), UNSUP), (dict(Hq=0), UNSUP), (dict(width=-1), INVALID), (dict(q=0), INVALID),
    (dict(tok=0), INVALID), (dict(out=0), INVALID), (dict(q=A + 8), ALIGN), (dict(out=A + 9 * S + 4), ALIGN),
    (dict(w=A + 11 * S + 2), ALIGN), (dict(qst=6140), ALIGN), (dict(qsh=248), INVALID), (dict(ost=6136), INVALID),
    (dict(tst=66), INVALID), (dict(wst=66), INVALID), (dict(scale=float("inf")), INVALID), (dict(out=A + 64), INVALID),
    (dict(out=A + 2 * S), INVALID), (dict(lse=A + 9 * S), INVALID), (dict(w=A + 8 * S), INVALID),
    (dict(w=A + 9 * S), INVALID), (dict(ws=0), WS), (dict(nbytes=1000), WS), (dict(ws=A + 12 * S + 8), ALIGN),
])
def test_attention_refuses(name, kw, code):
    st, detail = attn(name, **kw)
    assert st == code and detail, (st, detail)


@pytest.mark.parametrize("kw,code", [
    (dict(w=0), INVALID), (dict(tok=0), INVALID), (dict(tw=0), INVALID), (dict(cu=0), INVALID), (dict(pt=0), INVALID),
    (dict(w=A + 1), ALIGN), (dict(tw=A + 5 * S + 4), ALIGN), (dict(wst=66), INVALID), (dict(tst=5), INVALID),
    (dict(pts=3), INVALID), (dict(width=-1), INVALID), (dict(T=-1), INVALID), (dict(R=0), INVALID),
    (dict(pages=0), INVALID), (dict(ps=0), INVALID), (dict(tw=A), INVALID), (dict(tw=A + S), INVALID),
])
def test_accumulate_refuses(kw, code):
    st, detail = accumulate(**kw)
    assert st == code and detail, (st, detail)


LONG = dict(maxp=5000, pts=5000, ost=5000, fst=5000)   # a table that needs a workspace


@pytest.mark.parametrize("kw,code", [
    (dict(tw=0), INVALID), (dict(keep=0), INVALID), (dict(counts=0), INVALID), (dict(out=0), INVALID),
    (dict(freed=0), INVALID), (dict(tw=A + 4), ALIGN), (dict(keep=A + 3 * S + 1), ALIGN), (dict(first=-1), INVALID),
    (dict(last=-1), INVALID), (dict(R=-1), INVALID), (dict(maxp=-1), INVALID), (dict(pts=9), INVALID),
    (dict(ost=9), INVALID), (dict(fst=9), INVALID), (dict(out=A + S + 4), INVALID), (dict(out=A + S, ost=11), INVALID),
    (dict(freed=A + S), INVALID), (dict(freed=A + 4 * S + 40), INVALID), (dict(LONG, ws=0), WS),
    (dict(LONG, nbytes=5000 * 32 - 1), WS), (dict(LONG, ws=A + 7 * S + 8), ALIGN), (dict(ps=0), INVALID),
    (dict(pages=0), INVALID),
])
def test_evict_refuses(kw, code):
    st, detail = evict(**kw)
    assert st == code and detail, (st, detail)


def test_empty_calls_do_nothing():
    assert append(T=0)[0] == attn(T=0)[0] == accumulate(T=0)[0] == accumulate(width=0)[0] == evict(R=0)[0] == OK


def test_workspace_sizes():
    L = qsa.lib()
    size = L.qsa_sparse_attention_fp8_workspace_size
    assert size(0, 24, 2, 67, 0) == size(8, 23, 2, 67, 0) == size(8, 24, 2, 0, 1) == 0
    assert size(8, 24, 2, 67, 1) >= size(8, 24, 2, 67, 0) > 0
    evict_size = L.qsa_evict_pages_workspace_size
    assert evict_size(4, 512, 64) == evict_size(148, 4096, 8) == evict_size(0, 5000, 16) == 0
    assert evict_size(4, 513, 64) >= 4 * 513 * 8 and evict_size(1, 4097, 1) >= 4097 * 8
    assert evict_size(149, 10, 1) >= 149 * 80


def test_binding_refuses_tensors_that_are_not_on_a_gpu():
    z = torch.zeros
    with pytest.raises(TypeError):
        qsa.kv_append_fp8(z(1, 2, 256, dtype=torch.bfloat16), z(1, 2, 256, dtype=torch.bfloat16), z(1), z(1), z(1), z(1),
                          z(1), z(1), z(1))
    with pytest.raises(TypeError):
        qsa.sparse_attention_fp8(z(1, 24, 256), z(1), z(1), z(1), z(1), z(1), z(1), z(1), z(1), 1.0)
    with pytest.raises(TypeError):
        qsa.accumulate_weights(z(1, 4), z(1, 4, dtype=torch.int32), z(1), z(1), z(1), z(1))
    with pytest.raises(TypeError):
        qsa.evict_pages(z(1, 4, dtype=torch.int64), z(1), z(1), z(1))
