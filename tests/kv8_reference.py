"""The 8-bit K/V cache operators in 64 bits, plain and slow, from their definitions (include/qsa.h): what the GPU
tests of those operators compare with.  Arrays are numpy; codes are uint8."""
import math

import numpy as np
import torch


def _e4m3_values():
    """All 256 codes by the format's definition: bias 7, 3 fraction bits, subnormals m * 2^-9, NaN at 0x7f / 0xff."""
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if e == 15 and m == 7:
            x = math.nan
        v[c] = -x if c & 128 else x
    return v


VALUE = _e4m3_values()
_POS = VALUE[:127]                                   # 0 .. 448, ascending


def encode(x):
    """E4M3 codes of float64 values: nearest, ties to the even code, +-448 for what is larger, NaN -> 0x7f."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(_POS, a), 0, 126)   # first code with value >= a
    lo = np.maximum(hi - 1, 0)
    up, down = _POS[hi] - a, a - _POS[lo]
    code = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    code = np.where(np.isnan(x), 127, code)
    return np.where(np.signbit(x) & ~np.isnan(x), code + 128, code).astype(np.uint8)


def pow2_scale(amax):
    """The smallest power of two s >= 2^-64 with amax <= 448 s."""
    s = 2.0 ** -64
    while amax > 448.0 * s:
        s *= 2
    return s


def rows_of(cu, seq_lens, T):
    """(request, position) of every row; (-1, -1) for rows behind the last request's."""
    out = [(-1, -1)] * T
    for r in range(len(seq_lens)):
        for t in range(int(cu[r]), min(int(cu[r + 1]), T)):
            out[t] = (r, int(seq_lens[r]) - (int(cu[r + 1]) - t))
    return out


def page_of(table, r, lp, pages):
    if not 0 <= lp < table.shape[1]:
        return -1
    p = int(table[r, lp])
    return p if 0 <= p < pages else -1


def append(x, codes, scales, table, cu, seq_lens, token_weight=None):
    """One of K or V: x float64 [T, H, 256], codes uint8 [pages, ps, H, 256], scales float64 [pages, nb, H], in place."""
    pages, ps, H, _ = codes.shape
    bt = ps // scales.shape[1]
    for r in range(len(seq_lens)):
        first, end, L = int(cu[r]), int(cu[r + 1]), int(seq_lens[r])
        p0 = L - (end - first)
        for b in range(max(p0, 0) // bt, -(-L // bt) if L > 0 else 0):
            new = [j for j in range(b * bt, min((b + 1) * bt, L)) if j >= max(p0, 0)]
            page = page_of(table, r, b * bt // ps, pages)
            if not new or page < 0:
                continue
            r0 = b * bt % ps
            for h in range(H):
                rows = np.stack([x[first + j - p0, h] for j in new])
                fin = np.abs(rows[np.isfinite(rows)])
                need = pow2_scale(fin.max() if fin.size else 0.0)
                was = scales[page, r0 // bt, h]
                s = need if new[0] == b * bt else max(was, need)
                n_old = new[0] - b * bt
                if n_old and s != was:
                    codes[page, r0:r0 + n_old, h] = encode(VALUE[codes[page, r0:r0 + n_old, h]] * (was / s))
                codes[page, r0 + n_old:r0 + n_old + len(new), h] = encode(rows / s)
                scales[page, r0 // bt, h] = s
            if token_weight is not None:
                token_weight[page, r0 + new[0] - b * bt:r0 + new[-1] + 1 - b * bt] = 0


def visible(tok_row, r, pos, seq_lens, table, pages, ps):
    """[(entry, page, row in page)] of what a row sees."""
    out = []
    for e, j in enumerate(tok_row):
        j = int(j)
        if r < 0 or j < 0 or j > pos or j >= int(seq_lens[r]):
            continue
        page = page_of(table, r, j // ps, pages)
        if page >= 0:
            out.append((e, page, j % ps))
    return out


def attention(q, kc, vc, ks, vs, table, cu, seq_lens, tok, scale, gate=None, half_step=2.0 ** -8):
    """out, lse, weights, and how far each may be off (see below), all float64.  q [T, Hq, 256].

    Tolerances: scores are 256 products added in fp32 (256 * 2^-24 of sum |q k|) of queries held to 2^-22 of the
    head's largest element; probabilities at least to 2^-12 relative and, as errors of n entries of 2^-22 of the
    largest with signs of their own, n * 2^-26 of it in all; sums and exponentials in fp32 (2^-14 relative covers
    width-2^10 sums); the output one rounding of half_step relative.  A k_scale of 0 hides a block's tokens."""
    T, Hq, _ = q.shape
    pages, ps, H, _ = kc.shape
    bt = ps // ks.shape[1]
    G = Hq // H
    out, lse, w = np.zeros((T, Hq, 256)), np.full((T, Hq), -np.inf), np.zeros(tok.shape)
    t_out, t_lse, t_w = np.zeros((T, Hq, 256)), np.zeros((T, Hq)), np.zeros(tok.shape)
    for t, (r, pos) in enumerate(rows_of(cu, seq_lens, T)):
        seen = visible(tok[t], r, pos, seq_lens, table, pages, ps)
        if not seen:
            continue
        every = [np.array(c) for c in zip(*seen)]
        for g in range(H):
            e, pg, rw = every
            held = ks[pg, rw // bt, g] != 0
            e, pg, rw = e[held], pg[held], rw[held]
            if len(e) == 0:
                continue
            K = VALUE[kc[pg, rw, g]] * ks[pg, rw // bt, g][:, None]
            V = VALUE[vc[pg, rw, g]] * vs[pg, rw // bt, g][:, None]
            for h in range(g * G, (g + 1) * G):
                s = scale * (K @ q[t, h])
                top = s.max()
                p = np.exp(s - top)
                lse[t, h] = top + math.log(p.sum())
                p /= p.sum()
                m = 1.0 if gate is None else 1.0 / (1.0 + math.exp(-gate[t, h]))
                out[t, h] = m * (p @ V)
                np.add.at(w[t], e, p)
                ds = scale * float(np.max(2.0 ** -16 * (np.abs(K) @ np.abs(q[t, h])) +
                                          2.0 ** -22 * np.abs(q[t, h]).max() * np.abs(K).sum(1)))
                t_out[t, h] = (m * ((2.0 ** -12 + 2.0 ** -14 + 4 * ds) * (p @ np.abs(V)) +
                                    len(e) * 2.0 ** -26 * np.abs(V).max()) +
                               half_step * np.abs(out[t, h]) + 1e-6)
                t_lse[t, h] = 2 * ds + 4e-6 * (abs(lse[t, h]) + 1)
                np.add.at(t_w[t], e, p * (4 * ds + 8e-6 * (abs(lse[t, h]) + 1)) + 1e-12)
    return out, lse, w, t_out, t_lse, t_w


def accumulate(weights, tok, table, cu, seq_lens, token_weight):
    """weights float64 holding fp32 values; token_weight int64, in place."""
    pages, ps = token_weight.shape
    for t, (r, pos) in enumerate(rows_of(cu, seq_lens, len(tok))):
        for e, page, row in visible(tok[t], r, pos, seq_lens, table, pages, ps):
            w = float(weights[t, e])
            if w > 0:
                token_weight[page, row] += int(np.rint(min(w, 2.0 ** 20) * 2.0 ** 32))


def evict(token_weight, table, seq_lens, keep, keep_first, keep_last):
    pages, ps = token_weight.shape
    R, width = table.shape
    out, freed, counts = table.copy(), np.full((R, width), -1, np.int32), np.zeros(R, np.int32)
    for r in range(R):
        n = min(-(-max(int(seq_lens[r]), 0) // ps), width)
        live = [lp for lp in range(n) if page_of(table, r, lp, pages) >= 0]
        held = [lp for lp in live if lp < keep_first or lp >= n - keep_last]
        other = [lp for lp in live if lp not in held]
        weight = {lp: int(token_weight[int(table[r, lp])].sum()) for lp in other}
        stay = sorted(other, key=lambda lp: (-weight[lp], lp))[:max(0, int(keep[r]) - len(held))]
        gone = [lp for lp in other if lp not in stay]
        for i, lp in enumerate(gone):
            freed[r, i] = table[r, lp]
            out[r, lp] = -1
        counts[r] = len(gone)
    return out, freed, counts


# ------------------------------------------------------------------ inputs

def layout(seq_lens, qlens, ps, seed, spare=2, pad=1):
    """(page table int32 [R, max_pages + pad], seq_lens, cu int32, pages): random pages, -1 behind a request's."""
    g = torch.Generator().manual_seed(seed)
    per = [max(1, -(-n // ps)) for n in seq_lens]
    pages = sum(per) + spare
    perm = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(per), max(per) + pad), -1, dtype=torch.int32)
    at = 0
    for r, n in enumerate(per):
        table[r, :n] = perm[at:at + n]
        at += n
    cu = torch.zeros(len(per) + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor(qlens), 0)
    return table, torch.tensor(seq_lens, dtype=torch.int32), cu, pages


def cache(pages, ps, H, bt, seed, pow2=True):
    """Random codes (no NaN) and scales that differ by block."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((pages, ps // bt, bt, H, 256), generator=g) * torch.exp(torch.randn((pages, ps // bt, 1, H, 1), generator=g))
    s = x.abs().amax(dim=(2, 4)).double() / 448.0
    s = torch.exp2(torch.ceil(torch.log2(s))) if pow2 else s * 1.1
    s = s.float()
    codes = encode((x.double() / s.double()[:, :, None, :, None]).numpy()).reshape(pages, ps, H, 256)
    return torch.from_numpy(codes), s


def token_lists(seq_lens, qlens, width, seed, extra=True):
    """Lists of `width` entries in random order: visible tokens, and (extra) future ones, -1 and repeats."""
    rng = np.random.default_rng(seed)
    out = []
    for L, n in zip(seq_lens, qlens):
        for i in range(n):
            pos = L - n + i
            row = rng.permutation(max(pos + 1, 0))[:width]
            row = np.concatenate([row, np.full(width - len(row), -1)])
            if extra and width > 6:
                row[rng.integers(width)] = pos + 1 + rng.integers(3)
                row[rng.integers(width)] = -1 - rng.integers(5)
                row[rng.integers(width)] = row[rng.integers(width)]
            out.append(row)
    return torch.from_numpy(np.stack(out).astype(np.int32))
