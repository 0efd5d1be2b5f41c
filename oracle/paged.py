"""fp64 oracle of serving over an 8-bit paged KV cache and of rotary positions -- TEST INFRASTRUCTURE ONLY.

Plain definitions in numpy loops, sharing no code with the library:

* ``round_e4m3``    -- round to nearest even onto the e4m3 (fn) grid from the format's definition
  (3 mantissa bits, exponents -6..8, steps of 2^-9 below 2^-6, largest 448), and ``e4m3_codes``,
  its bytes by a search in the table of the 256 values.
* ``append``        -- the write of new tokens into pages: one power-of-two scale per page and head.
* ``page_tables``   -- a free list and a loop over the requests.
* ``rope``          -- rotation of pairs as complex numbers.
* ``decode_paged``  -- attention of each query row over the visible tokens of its request's pages,
  with the bounds that the tolerances use.
"""
from __future__ import annotations

import math

import numpy as np


def _e4m3_table():
    t = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        if e == 15 and m == 7:
            v = math.nan
        t[c] = -v if c & 128 else v
    return t


E4M3 = _e4m3_table()
_POS = E4M3[:127]                                   # 0 .. 448, increasing


def e4m3_codes(x):
    """Bytes of x rounded to nearest even, saturating; not finite -> NaN (0x7f)."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.where(np.isfinite(x), x, 0.0)), 448.0)
    hi = np.searchsorted(_POS, a)                   # first value >= a
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    c = np.where(up, hi, lo) | np.where(np.signbit(x), 128, 0)
    return np.where(np.isfinite(x), c, 0x7F).astype(np.uint8)


def round_e4m3(x):
    return E4M3[e4m3_codes(x)]


def scale_for(amax):
    """2^e with the smallest e in [-60, 60] such that amax <= 448 * 2^e."""
    e = -60
    while e < 60 and amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(k, v, slots, k_codes, v_codes, k_scale, v_scale, page):
    """In place on codes uint8 [pages, Hkv, page, d] and scales fp64 [pages, Hkv]; k, v [B, Hkv, N, d] fp64."""
    B, Hkv, N, _ = k.shape
    pages = k_codes.shape[0]
    for b in range(B):
        n = 0
        while n < N:
            p = slots[b, n] // page if 0 <= slots[b, n] < pages * page else -1
            run = {}
            m = n
            while m < N and 0 <= slots[b, m] < pages * page and slots[b, m] // page == p:
                run[int(slots[b, m]) % page] = m     # a later token of the same slot replaces an earlier one
                m += 1
            n = max(m, n + 1)
            if not run:
                continue
            rows, toks = list(run), list(run.values())
            rest = [r for r in range(page) if r not in run]
            for h in range(Hkv):
                for x, codes, scale in ((k, k_codes, k_scale), (v, v_codes, v_scale)):
                    y = x[b, h, toks]
                    fin = np.abs(y[np.isfinite(y)])
                    want = scale_for(fin.max() if fin.size else 0.0)
                    if 0 in run:
                        now = want
                    else:
                        was = scale[p, h]
                        ok = np.isfinite(was) and was > 0
                        now = max(was, want) if ok else want
                        if now != was or not ok:
                            old = E4M3[codes[p, h, rest]]
                            codes[p, h, rest] = e4m3_codes(old * (was / now)) if ok else 0
                    codes[p, h, rows] = e4m3_codes(y / now)
                    scale[p, h] = now


def page_tables(ctx, new, free, head, table, N, page, held=None):
    """(table, free, slots, positions, lens, head) after the step; nothing of the inputs is changed but `held`, the
    number of each request's pages where lengths may have been lowered."""
    table, free, head = table.copy(), free.copy(), int(head)
    B, per_row = table.shape
    slots, pos, lens = np.full((B, N), -1), np.zeros((B, N), int), ctx.copy()
    has = [-(-int(n) // page) for n in ctx]
    if held is not None:
        has = [min(max(int(held[b]), has[b]), per_row) for b in range(B)]
        held[:] = [0 if new[b] < 0 else has[b] for b in range(B)]
    back = [p for b in range(B) if new[b] < 0 for p in table[b, : has[b]]]
    if len(back) <= head:
        head -= len(back)
        free[head:head + len(back)] = back
    avail, asked, taken = len(free) - head, 0, 0
    for b in range(B):
        if new[b] < 0:
            lens[b] = 0
            continue
        if new[b] > N or ctx[b] + new[b] > per_row * page:
            continue
        need = max(-(-int(ctx[b] + new[b]) // page) - has[b], 0)
        asked += need
        if need and asked > avail:
            continue
        for i in range(need):
            table[b, has[b] + i] = free[head + asked - need + i]
        if held is not None:
            held[b] += need
        taken += need
        for t in range(int(new[b])):
            at = int(ctx[b]) + t
            slots[b, t], pos[b, t] = table[b, at // page] * page + at % page, at
        lens[b] = ctx[b] + new[b]
    return table, free, slots, pos, lens, head + taken


def rope(x, positions, inv_freq, factor=1.0, interleaved=False, transpose=False):
    """Rotation of x [B, H, N, d] fp64; positions [B, N]."""
    r = 2 * len(inv_freq)
    a = np.asarray(positions, np.float64)[:, None, :, None] * np.asarray(inv_freq) * (-1.0 if transpose else 1.0)
    t = factor * np.exp(1j * a)
    y = x.copy()
    u, w = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    z = (x[..., u] + 1j * x[..., w]) * t
    y[..., u], y[..., w] = z.real, z.imag
    return y


def decode_paged(q, k_codes, v_codes, k_scale, v_scale, table, lens, scale, causal):
    """O [B,H,Nq,d], LSE [B,H,Nq], and per row A = sum_j p_j |V_j| and the largest
    sum_c |q_c K_jc| * scale among the visible keys (what the tolerances are made of)."""
    B, H, Nq, d = q.shape
    pages, Hkv, page, _ = k_codes.shape
    o, lse = np.zeros(q.shape), np.full((B, H, Nq), -np.inf)
    mag, big = np.zeros(q.shape), np.zeros((B, H, Nq))
    for b in range(B):
        n = min(max(int(lens[b]), 0), table.shape[1] * page)
        j = np.arange(n)
        p = table[b, j // page]
        ok = (p >= 0) & (p < pages)
        p = np.where(ok, p, 0)
        for hk in range(Hkv):
            K = E4M3[k_codes[p, hk, j % page]] * k_scale[p, hk][:, None]
            V = E4M3[v_codes[p, hk, j % page]] * v_scale[p, hk][:, None]
            for h in range(hk * (H // Hkv), (hk + 1) * (H // Hkv)):
                for i in range(Nq):
                    see = ok & (j <= n - Nq + i if causal else j >= 0)
                    if not see.any():
                        continue
                    s = scale * (K[see] @ q[b, h, i])
                    m = s.max()
                    e = np.exp(s - m)
                    e_sum = e.sum()
                    lse[b, h, i] = m + math.log(e_sum)
                    o[b, h, i] = e @ V[see] / e_sum
                    mag[b, h, i] = e @ np.abs(V[see]) / e_sum
                    big[b, h, i] = scale * (np.abs(K[see]) @ np.abs(q[b, h, i])).max()
    return o, lse, mag, big
