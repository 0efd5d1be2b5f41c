"""GPU parity of the calls around a decode step over the 8-bit paged cache -- rotary positions, page tables,
the cache write, attention over the pages -- against the fp64 oracle, alone and run together.

Tolerances, from the arithmetic:
  rope    y is rounded once to bf16 (half a step, 2^-8 |y|); before that the angle's remainder is rounded to
          fp32 (2^-25 turns, 2^-22 rad) and sine, cosine and the two products to fp32: below 2^-20 factor (|u| + |w|).
  append  exact: codes, scales (powers of two) and what is not written are compared byte for byte.
  tables  exact.
  decode  a score is an fp32 sum of d products of e4m3 and bf16 values and three factors: its error is at most
          e = (d + 8) 2^-23 S with S = scale sum |q_c K_c| (and 2^-20 for exponent and logarithm), which is LSE's
          tolerance.  p then is off by 2e relative, and its rounding for the product with V (fp16's half step,
          2^-11; 2^-14 for the fp32 sums and the merge) adds up to A = sum p |V|: O is off by at most
          2^-8 |O| + (2^-11 + 2^-14 + 2 e) A.
"""
import math

import numpy as np
import pytest
import torch

import synth
from oracle import paged
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

fa = pytest.importorskip("exact_io_aware_55_b200")


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def bf16(x):
    """fp array -> (its bf16 values in fp64, the CUDA tensor)."""
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(torch.bfloat16)
    return t.double().numpy(), t.cuda()


@pytest.fixture(autouse=True)
def no_status():
    fa.fa_device_status()
    yield
    torch.cuda.synchronize()
    assert fa.fa_device_status() == (0, 0)


# ------------------------------------------------------------------------------------------------------ rope
ROPE = [  # B, H, N, d, rot, interleaved, transpose, strided
    (1, 1, 1, 64, 16, False, False, False), (3, 5, 1, 128, 128, False, False, True), (2, 3, 77, 64, 64, True, True, False),
    (1, 40, 33, 128, 96, True, False, True), (2, 7, 130, 128, 48, False, True, True), (1, 2, 1025, 64, 32, True, False, True),
    (260, 9, 1, 64, 48, False, False, False), (1, 16, 3000, 128, 128, False, True, False)]


@pytest.mark.parametrize("B,H,N,d,rot,inter,tr,strided", ROPE)
def test_rope_parity(B, H, N, d, rot, inter, tr, strided):
    rng = np.random.default_rng(B * 7 + N)
    x64, x = bf16(rng.standard_normal((B, N, H + 3, d) if strided else (B, H, N, d)))
    if strided:
        x64, x = x64[:, :, 1:H + 1].transpose(0, 2, 1, 3), x[:, :, 1:H + 1].transpose(1, 2)
    pos = rng.integers(0, 1 << 20, (B, 1)) + np.arange(N)
    pos[0, -1] = 2 ** 31 - 1 if N > 1 else -3
    freq, factor = fa.rope_frequencies(rot, 10000.0, "yarn", 8.0, 4096.0, 1.0, 32.0)
    out = gu.Guarded((B, H, N, d), torch.bfloat16)
    fa.fa_rope(x, out.view, i32(pos), freq, factor, inter, tr)
    torch.cuda.synchronize()
    ref = paged.rope(x64, pos, freq.cpu().numpy(), factor, inter, tr)
    y = gu.to_f64(out.view)
    assert out.intact()
    r = rot // 2
    pair = np.zeros_like(x64)
    a = np.abs(x64)
    if inter:
        pair[..., :rot] = np.repeat(a[..., 0:rot:2] + a[..., 1:rot:2], 2, -1)
    else:
        pair[..., :rot] = np.tile(a[..., :r] + a[..., r:rot], 2)
    assert np.all(np.abs(y - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * factor * pair)
    assert np.array_equal(y[..., rot:], x64[..., rot:])
    # in place, and the strides of a token-major output
    z = x.clone() if not strided else x.transpose(1, 2).contiguous().transpose(1, 2)
    fa.fa_rope(z, z, i32(pos), freq, factor, inter, tr)
    assert torch.equal(z, out.view)


def test_rope_default_positions_and_repeated_rows():
    rng = np.random.default_rng(8)
    x64, x = bf16(rng.standard_normal((1, 1, 50, 64)))
    freq, _ = fa.rope_frequencies(64)
    y = fa.rope_forward(x.expand(3, 4, 50, 64), None, freq)
    ref = paged.rope(x64, np.arange(50)[None], freq.cpu().numpy())
    assert torch.equal(y, fa.rope_forward(x, i32(np.arange(50)[None]), freq).expand(3, 4, 50, 64))
    assert np.max(np.abs(gu.to_f64(y[0, :1]) - ref[0])) <= 2.0 ** -8 * np.abs(ref).max() + 1e-5


def test_rope_backward_is_the_gradient():
    """<dy, R x> = <R^T dy, x> with the outputs' rounding, and a round trip returns x."""
    rng = np.random.default_rng(9)
    (x64, x), (g64, g) = bf16(rng.standard_normal((2, 3, 40, 128))), bf16(rng.standard_normal((2, 3, 40, 128)))
    freq, _ = fa.rope_frequencies(96)
    pos = i32(rng.integers(0, 100000, (2, 40)))
    y, dx = fa.rope_forward(x, pos, freq), fa.rope_backward(g, pos, freq)
    a, b = np.sum(g64 * gu.to_f64(y)), np.sum(x64 * gu.to_f64(dx))
    bound = 2.0 ** -8 * (np.sum(np.abs(g64 * gu.to_f64(y))) + np.sum(np.abs(x64 * gu.to_f64(dx))))
    assert abs(a - b) <= bound
    back = gu.to_f64(fa.rope_backward(y, pos, freq))
    size = np.sqrt(x64 ** 2 + 0) + np.roll(np.abs(x64), 48, -1) + np.roll(np.abs(x64), -48, -1)
    assert np.all(np.abs(back - x64) <= 2.0 ** -8 * np.abs(x64) * 1.01 + 2.0 ** -7 * size)


# ---------------------------------------------------------------------------------------------------- append
def cache(rng, pages, Hkv, page, d, spread=4):
    """Random codes and power-of-two scales: (codes uint8, scale fp64) and their CUDA tensors."""
    x = rng.standard_normal((pages, Hkv, page, d)) * 100.0
    codes = paged.e4m3_codes(x)
    scale = 2.0 ** rng.integers(-8 - spread, -8 + spread + 1, (pages, Hkv))
    return codes, scale, torch.from_numpy(codes).cuda(), torch.from_numpy(scale.astype(np.float32)).cuda()


def check_append(k64, v64, k, v, slots, kc, vc, ks, vs, page, Hkv, d):
    pages = kc[0].shape[0]
    bufs = [gu.Guarded((pages, Hkv, page, d), torch.uint8) for _ in range(2)]
    scales = [gu.Guarded((pages, Hkv), torch.float32) for _ in range(2)]
    for g, t in zip(bufs + scales, (kc[1], vc[1], ks[1], vs[1])):
        g.view.copy_(t)
    fa.fa_cache_append_fp8(k, v, i32(slots), bufs[0].view, bufs[1].view, scales[0].view, scales[1].view)
    torch.cuda.synchronize()
    want = [kc[0].copy(), vc[0].copy(), ks[0].astype(np.float64).copy(), vs[0].astype(np.float64).copy()]
    paged.append(k64, v64, slots, *want, page)
    for g in bufs + scales:
        assert g.intact()
    for g, w, name in zip(bufs, want, "kv"):
        got = g.view.cpu().numpy()
        nan = (got & 0x7F) == 0x7F
        assert np.array_equal(nan, (w & 0x7F) == 0x7F) and np.array_equal(got[~nan], w[~nan]), name
    for g, w in zip(scales, want[2:]):
        assert np.array_equal(g.view.cpu().numpy().astype(np.float64), w.astype(np.float32).astype(np.float64), equal_nan=True)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("B,Hkv,N", [(1, 1, 1), (3, 5, 1), (2, 3, 7), (2, 2, 300), (1, 9, 131)])
def test_append_parity(B, Hkv, N, page, d):
    rng = np.random.default_rng(page + N + d)
    per_row = -(-(N + 200) // page)
    pages = B * per_row + 2
    table = rng.permutation(pages)[: B * per_row].reshape(B, per_row)
    ctx = rng.integers(0, 200, B)
    at = ctx[:, None] + np.arange(N)
    slots = np.take_along_axis(table, at // page, 1) * page + at % page
    slots[-1, (N + 1) // 2:] = -1                      # a shorter request: its tail is left alone
    kc, ks, kct, kst = cache(rng, pages, Hkv, page, d)
    vc, vs, vct, vst = cache(rng, pages, Hkv, page, d)
    size = np.exp(rng.standard_normal((B, Hkv, N, 1)) * 1.5)
    (k64, k), (v64, v) = (bf16(rng.standard_normal((B, Hkv, N, d)) * size) for _ in range(2))
    check_append(k64, v64, k, v, slots, (kc, kct), (vc, vct), (ks, kst), (vs, vst), page, Hkv, d)


def test_append_special_values():
    """NaN and infinities, values beyond the largest scale, zeros, subnormal codes, -0, old scales that are no scale."""
    rng = np.random.default_rng(11)
    page, d, Hkv, pages = 16, 64, 2, 12
    kc, ks, kct, kst = cache(rng, pages, Hkv, page, d)
    vc, vs, vct, vst = cache(rng, pages, Hkv, page, d, spread=8)
    bad = np.array([np.nan, np.inf, -1.0, 0.0, 1e-40, 2.0 ** 70])
    ks[:6, 0], kst[:6, 0] = bad.astype(np.float32), torch.from_numpy(bad.astype(np.float32)).cuda()
    x = rng.standard_normal((12, Hkv, 3, d)) * 2.0 ** rng.integers(-12, 12, (12, Hkv, 3, 1))
    x[0, 0, 1, 5], x[1, 0, 0, :3], x[2, 1, 2, 9] = np.nan, [np.inf, -np.inf, 3.0], -np.inf
    x[3], x[4, 0, 0, 0], x[5, 0, 0, 1] = 0.0, 3e38, -3e38
    x[6, 0, 1] = -0.0
    x[7, 0] = np.nan
    slots = np.arange(12)[:, None] * page + np.array([[0, 1, 2]]) + (np.arange(12) % 2)[:, None] * 4
    (k64, k), (v64, v) = bf16(x), bf16(x[::-1].copy())
    check_append(k64, v64, k, v, slots, (kc, kct), (vc, vct), (ks.astype(np.float32), kst), (vs, vst), page, Hkv, d)


def test_append_every_value_and_scale_step():
    """Every finite bf16 magnitude of a range of exponents under scales that just hold, or just do not hold, it."""
    page, d = 16, 128
    bits = np.arange(0x2000, 0x5F00, 3, dtype=np.uint16)
    x = synth.bf16_bits_to_f64(bits)
    n = len(x) // d
    x = x[: n * d].reshape(1, 1, n, d)
    k64, k = bf16(x)
    slots = np.arange(n)[None] * page + 3               # one page each, continued
    rng = np.random.default_rng(12)
    kc, _, kct, _ = cache(rng, n, 1, page, d)
    top = np.abs(x).max(-1).reshape(-1)
    ks = np.array([paged.scale_for(t) for t in top])[:, None] * 2.0 ** rng.integers(-2, 3, (n, 1))
    kst = torch.from_numpy(ks.astype(np.float32)).cuda()
    check_append(k64, -k64, k, -k, slots, (kc, kct), (kc.copy(), kct.clone()), (ks, kst), (ks.copy(), kst.clone()), page, 1, d)


def test_append_same_slot_twice_keeps_the_later():
    rng = np.random.default_rng(13)
    page, d = 32, 64
    kc, ks, kct, kst = cache(rng, 4, 1, page, d)
    k64, k = bf16(rng.standard_normal((1, 1, 200, d)))
    slots = np.full((1, 200), 32 + 5)
    slots[0, 150:] = 64 + rng.integers(0, 32, 50)
    check_append(k64, k64, k, k, slots, (kc, kct), (kc.copy(), kct.clone()), (ks, kst), (ks.copy(), kst.clone()), page, 1, d)


def test_append_skips_slots_outside_the_cache():
    rng = np.random.default_rng(14)
    kc, ks, kct, kst = cache(rng, 3, 2, 16, 64)
    k64, k = bf16(rng.standard_normal((1, 2, 6, 64)))
    slots = np.array([[16, 17, 48, 2 ** 31 - 1, -(2 ** 31), 40]])
    check_append(k64, k64, k, k, slots, (kc, kct), (kc.copy(), kct.clone()), (ks, kst), (ks.copy(), kst.clone()), 16, 2, 64)
    assert fa.fa_device_status() == (9, 80)


# ---------------------------------------------------------------------------------------------------- tables
def check_tables(ctx, new, free, head, table, N, page, alias):
    B = len(ctx)
    c, n, f, h, t = i32(ctx), i32(new), i32(free), i32([head]), i32(table)
    slots, pos = gu.Guarded((B, N), torch.int32), gu.Guarded((B, N), torch.int32)
    seq = c if alias else torch.full_like(c, -7)
    out = h if alias else torch.full_like(h, -7)
    fa.fa_page_tables(c, n, f, h, t, slots.view, pos.view, seq, out, page)
    torch.cuda.synchronize()
    wt, wf, wslots, wpos, wlens, whead = paged.page_tables(ctx, new, free, head, table, N, page)
    assert slots.intact() and pos.intact()
    for got, want, name in ((slots.view, wslots, "slots"), (pos.view, wpos, "positions"), (seq, wlens, "lens"),
                            (out, [whead], "head"), (t, wt, "table"), (f, wf, "free")):
        assert np.array_equal(got.cpu().numpy(), np.asarray(want)), name
    if not alias:
        assert np.array_equal(c.cpu().numpy(), ctx) and int(h) == head
    return wt, wf, wlens, whead


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("B,N,page,pages", [(1, 1, 16, 4), (5, 40, 16, 30), (33, 3, 32, 25), (700, 9, 64, 900), (2500, 1, 16, 4000),
                                            (3, 2000, 128, 90)])
def test_page_tables_steps(B, N, page, pages, alias):
    rng = np.random.default_rng(B + N)
    per_row = max(2, -(-4 * N // page))
    table, free, head, ctx = rng.integers(-5, 10 ** 9, (B, per_row)), rng.permutation(pages), 0, np.zeros(B, int)
    for step in range(6):
        new = rng.integers(0, N + 1, B)
        new[rng.random(B) < 0.15] = -1
        new[rng.random(B) < 0.05] = N + 1 + step          # refused: more than there is room for in slots
        table, free, ctx, head = check_tables(ctx, new, free, head, table, N, page, alias)


def test_page_tables_edges():
    table = np.arange(6).reshape(2, 3)
    # exactly full, one page too few, row of the table full, nothing asked, only giving back (N = 0)
    check_tables(np.array([16, 0]), np.array([16, 16]), np.array([0, 7, 8]), 1, table, 16, 16, False)
    check_tables(np.array([16, 0]), np.array([16, 16]), np.array([0, 7]), 1, table, 16, 16, False)
    check_tables(np.array([47, 40]), np.array([1, 9]), np.array([0, 7, 8]), 0, table, 16, 16, False)
    check_tables(np.array([48, 0]), np.array([0, 0]), np.zeros(0, int), 0, table, 4, 16, False)
    check_tables(np.array([48, 5]), np.array([-1, -9]), np.arange(10, 16), 5, table, 0, 16, True)
    # a refused request does not stop one behind it that needs no page
    check_tables(np.array([16, 3]), np.array([16, 2]), np.zeros(0, int), 0, table, 16, 16, False)


def test_page_tables_contradicting_lists_take_nothing_back():
    check_tables(np.array([48, 3]), np.array([-1, 2]), np.arange(4), 2, np.arange(6).reshape(2, 3), 4, 16, False)
    assert fa.fa_device_status() == (9, 81)


# ---------------------------------------------------------------------------------------------------- decode
def check_decode(q, kc, vc, ks, vs, table, lens, scale, causal, d, want=None):
    """kc.. (numpy, CUDA) pairs; returns O, LSE after comparing every row."""
    q64, qt = q
    B, H, Nq, _ = q64.shape
    Hkv = kc[0].shape[1]
    og, lg = gu.Guarded(q64.shape, torch.bfloat16), gu.Guarded((B, H, Nq), torch.float32)
    wg = gu.Guarded((max(16, fa.fa_fwd_decode_paged_fp8_workspace_size(B, H, Hkv, Nq, d)),), torch.uint8)
    fa.fa_fwd_decode_paged_fp8(qt, kc[1], vc[1], ks[1], vs[1], i32(table), i32(lens), og.view, lg.view, scale, causal, wg.view)
    torch.cuda.synchronize()
    assert og.intact() and lg.intact() and wg.intact()
    o, lse = gu.to_f64(og.view), gu.to_f64(lg.view)
    ro, rl, mag, big = want or paged.decode_paged(q64, kc[0], vc[0], ks[0], vs[0], table, lens, scale, causal)
    none = np.isneginf(rl)
    assert np.array_equal(np.isneginf(lse), none) and np.all(o[none] == 0)
    assert np.array_equal(np.isnan(o), np.isnan(ro)) and np.array_equal(np.isnan(lse), np.isnan(rl))
    fin = np.isfinite(rl)
    e = (d + 8) * 2.0 ** -23 * big + 2.0 ** -20
    worst = np.max(np.abs(lse - rl)[fin] / (e + 2.0 ** -23 * np.abs(rl))[fin], initial=0)
    assert worst <= 1, f"LSE off by {worst:.3g} of its bound"
    tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -11 + 2.0 ** -14 + 2 * e[..., None]) * mag + 1e-38
    with np.errstate(invalid="ignore"):
        worst = np.max((np.abs(o - ro) / tol)[np.isfinite(ro)], initial=0)
    assert worst <= 1, f"O off by {worst:.3g} of its bound"
    return og.view.clone(), lg.view.clone()


def decode_case(B, H, Hkv, Nq, d, page, lens, seed, q_mult=1.0, stale=True):
    rng = np.random.default_rng(seed)
    per_row = max(1, -(-int(max(lens)) // page))
    pages = B * per_row + 1
    table = rng.permutation(pages)[: B * per_row].reshape(B, per_row)
    kc, ks, kct, kst = cache(rng, pages, Hkv, page, d, spread=1)
    vc, vs, vct, vst = cache(rng, pages, Hkv, page, d, spread=2)
    if stale:                                           # bytes behind a length: NaN codes, NaN scales of unused pages
        for b in range(B):
            for j in range(int(lens[b]), per_row * page):
                kc[table[b, j // page], :, j % page] = 0x7F
                vc[table[b, j // page], :, j % page] = 0xFF
            for i in range(-(-int(lens[b]) // page), per_row):
                ks[table[b, i]] = vs[table[b, i]] = np.nan
                table[b, i] = (-1, 2 ** 31 - 1)[i % 2]
        kct, vct = torch.from_numpy(kc).cuda(), torch.from_numpy(vc).cuda()
        kst, vst = (torch.from_numpy(s.astype(np.float32)).cuda() for s in (ks, vs))
    q = bf16(rng.standard_normal((B, H, Nq, d)) * q_mult)
    return q, (kc, kct), (vc, vct), (ks, kst), (vs, vst), table, np.asarray(lens)


DECODE = [  # B, H, Hkv, Nq, page, lens
    (1, 1, 1, 1, 16, [1]), (2, 2, 2, 1, 16, [15, 16]), (4, 8, 2, 1, 32, [0, 127, 128, 129]), (3, 4, 4, 3, 64, [2, 0, 300]),
    (2, 16, 1, 1, 128, [1000, 257]), (1, 32, 2, 2, 16, [777]), (2, 7, 1, 16, 32, [130, 16]), (1, 24, 2, 5, 16, [2049]),
    (5, 3, 3, 16, 128, [500, 1, 16, 17, 0]), (1, 2, 1, 1, 16, [20000]), (40, 4, 2, 1, 16, list(range(0, 400, 10))),
    (3, 64, 4, 4, 64, [5000, 4999, 1])]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,Hkv,Nq,page,lens", DECODE)
def test_decode_parity(B, H, Hkv, Nq, page, lens, d, causal):
    case = decode_case(B, H, Hkv, Nq, d, page, lens, seed=B + H + Nq + d)
    check_decode(*case, d ** -0.5, causal, d)


WIDE = [  # B, H, Hkv, Nq, page, lens: tables that could hold far more than the requests have
    (3, 8, 2, 1, 16, [900, 0, 5000]), (2, 32, 2, 1, 16, [4000, 17]), (2, 16, 2, 3, 16, [2100, 1300]), (1, 4, 2, 1, 32, [3001])]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,H,Hkv,Nq,page,lens", WIDE)
def test_decode_wide_tables(B, H, Hkv, Nq, page, lens, d, causal):
    q, kc, vc, ks, vs, table, n = decode_case(B, H, Hkv, Nq, d, page, lens, seed=B + H + d)
    wide = np.full((B, 400_000 // (B * Hkv)), -1)
    wide[:, : table.shape[1]] = table
    a = check_decode(q, kc, vc, ks, vs, wide, n, d ** -0.5, causal, d)
    b = check_decode(q, kc, vc, ks, vs, table, n, d ** -0.5, causal, d)
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("d", [64, 128])
def test_decode_requests_that_share_pages(d):
    """A common prompt: the first pages of every request are the same ones."""
    q, kc, vc, ks, vs, table, n = decode_case(6, 8, 2, 2, d, 32, [700, 640, 641, 33, 699, 700], seed=88, stale=False)
    table[:, :20] = table[0, :20]
    check_decode(q, kc, vc, ks, vs, table, n, d ** -0.5, True, d)


@pytest.mark.parametrize("seed", range(8))
def test_decode_drawn_shapes_in_one_workspace(seed):
    """Shapes drawn at random, one after the other in a workspace that the calls before have left as it is."""
    rng = np.random.default_rng(100 + seed)
    work = torch.empty(1 << 25, dtype=torch.uint8, device="cuda").random_()
    for _ in range(4):
        d, page = int(rng.choice([64, 128])), int(rng.choice([16, 32, 64, 128]))
        Hkv, group, Nq, B = int(rng.integers(1, 6)), int(rng.choice([1, 2, 3, 4, 7, 8, 12])), int(rng.integers(1, 17)), int(rng.integers(1, 9))
        lens = [int(2 ** rng.uniform(0, 12)) if rng.random() < 0.9 else 0 for _ in range(B)]
        q, kc, vc, ks, vs, table, n = decode_case(B, group * Hkv, Hkv, Nq, d, page, lens, seed=int(rng.integers(2 ** 31)))
        causal = bool(rng.integers(2))
        o, lse = fa.attention_decode_paged_fp8(q[1], kc[1], vc[1], ks[1], vs[1], i32(table), i32(n), d ** -0.5, causal, work)
        want = check_decode(q, kc, vc, ks, vs, table, n, d ** -0.5, causal, d)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("mult", [8.0, 64.0, 2.0 ** -40, 2.0 ** 30])
def test_decode_score_ranges(mult, d):
    case = decode_case(2, 8, 2, 2, d, 32, [900, 450], seed=77, q_mult=mult)
    check_decode(*case, d ** -0.5 * (1.0 if mult < 100 else 2.0 ** -28), True, d)


@pytest.mark.parametrize("d", [64, 128])
def test_decode_scale_zero(d):
    check_decode(*decode_case(2, 4, 2, 3, d, 16, [700, 2], seed=78), 0.0, True, d)


@pytest.mark.parametrize("d", [64, 128])
def test_decode_unlike_value_scales_and_a_heavy_first_token(d):
    """Value scales over a factor of 2^40, zero scales, and one key that outweighs each other by e^14 while
    the others together outweigh it."""
    q, kc, vc, ks, vs, table, lens = decode_case(2, 4, 2, 1, d, 16, [6000, 900], seed=79)
    rng = np.random.default_rng(80)
    live = vs[0][table[0]]
    vs[0][table[0]] = live * 2.0 ** rng.integers(-40, 1, live.shape)
    vs[0][table[0, 3]] = 0.0
    ks[0][table[0, 5]] = 0.0
    for x in (ks, vs):
        x[1].copy_(torch.from_numpy(x[0].astype(np.float32)))
    check_decode(q, kc, vc, ks, vs, table, lens, d ** -0.5, False, d)
    # keys orthogonal to the query but for the first one
    q64, _ = q
    q64 = np.zeros_like(q64)
    q64[..., 0] = 1.0
    kc[0][..., 0] = 0
    first = table[:, 0]
    kc[0][first, :, 0, 0] = paged.e4m3_codes(448.0)
    ks[0][first] = 14.0 / 448.0 * d ** 0.5
    vs[0][table[0]], vs[0][table[1, :57]] = 2.0 ** -8, 2.0 ** -8
    kc[1].copy_(torch.from_numpy(kc[0]))
    for x in (ks, vs):
        x[0][:] = x[0].astype(np.float32)
        x[1].copy_(torch.from_numpy(x[0].astype(np.float32)))
    check_decode(bf16(q64), kc, vc, ks, vs, table, lens, d ** -0.5, False, d)


@pytest.mark.parametrize("d", [64, 128])
def test_decode_nan_reaches_only_the_rows_that_see_it(d):
    q, kc, vc, ks, vs, table, lens = decode_case(3, 4, 2, 2, d, 16, [300, 300, 300], seed=81, stale=False)
    kc[0][table[1, 4], 1, 3, 7] = 0x7F                  # a key: request 1, KV head 1
    q[0][2, 3, 1, 5] = np.nan                           # a query: request 2, head 3, second token
    q[1][2, 3, 1, 5] = math.nan
    kc[1].copy_(torch.from_numpy(kc[0]))
    o, lse = check_decode(q, kc, vc, ks, vs, table, lens, d ** -0.5, False, d,
                          want=nan_rows(paged.decode_paged(np.nan_to_num(q[0]), np.where(kc[0] == 0x7F, 0, kc[0]), vc[0], ks[0],
                                                           vs[0], table, lens, d ** -0.5, False),
                                        [(1, 2, slice(None)), (1, 3, slice(None)), (2, 3, 1)]))
    assert bool(torch.isnan(lse[1, 2:]).all()) and bool(torch.isnan(o[2, 3, 1]).all())


def nan_rows(ref, rows):
    for r in rows:
        for x in ref:
            x[r] = np.nan
    return ref


@pytest.mark.parametrize("lens", [[300, 3, 130], [128, 257, 1500]])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_nan_value_of_a_newer_token(d, lens):
    """NaN codes in the values of the newest tokens: only the queries that see those tokens become NaN, in
    those columns alone, over many requests per CTA and over a tile's and a CTA's border."""
    B, Nq = 3 * 60, 4
    q, kc, vc, ks, vs, table, n = decode_case(B, 4, 2, Nq, d, 16, lens * 60, seed=86, stale=False)
    rng = np.random.default_rng(87)
    clean = vc[0].copy()
    hits = []
    for b in range(B):
        for back in rng.choice(Nq, 2, replace=False) if b % 4 else []:
            j = int(n[b]) - 1 - back
            if j < 0:
                continue
            hk, col = int(rng.integers(2)), int(rng.integers(d))
            vc[0][table[b, j // 16], hk, j % 16, col] = (0x7F, 0xFF)[b % 2]
            clean[table[b, j // 16], hk, j % 16, col] = 0
            hits.append((b, hk, j, col))
    vc[1].copy_(torch.from_numpy(vc[0]))
    ref = paged.decode_paged(q[0], kc[0], clean, ks[0], vs[0], table, n, d ** -0.5, True)
    for b, hk, j, col in hits:
        for i in range(Nq):
            if j <= n[b] - Nq + i:
                ref[0][b, 2 * hk:2 * hk + 2, i, col] = np.nan
    assert np.isnan(ref[0]).any() and len(hits) > 100
    check_decode(q, kc, vc, ks, vs, table, n, d ** -0.5, True, d, want=ref)


@pytest.mark.parametrize("d", [64, 128])
def test_decode_skips_pages_outside_the_cache(d):
    case = list(decode_case(2, 4, 2, 1, d, 16, [900, 40], seed=82, stale=False))
    case[5][0, 7], case[5][0, 30], case[5][1, 0] = -1, 10 ** 6, len(case[1][0])
    check_decode(*case, d ** -0.5, False, d)
    assert fa.fa_device_status()[0] == 9


def test_decode_lengths_outside_the_table():
    case = list(decode_case(2, 4, 2, 1, 64, 16, [160, 160], seed=83, stale=False))
    case[6] = np.array([10 ** 9, -5])
    check_decode(*case, 0.125, False, 64)


def test_a_timeout_is_reported_over_a_skipped_page():
    k = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16, device="cuda")
    cache, scales = torch.zeros(3, 1, 16, 64, dtype=torch.uint8, device="cuda"), torch.ones(3, 1, device="cuda")
    slots = torch.tensor([[3 * 16, 1, 2, 3]], dtype=torch.int32, device="cuda")
    fa.fa_cache_append_fp8(k, k, slots, cache, cache.clone(), scales, scales.clone())
    fa.fa_watchdog_selftest(2000)
    assert fa.fa_device_status() == (fa.STATUS_CODES["FA_ERR_DEVICE_TIMEOUT"], 99)


def test_decode_repeat_is_identical():
    q, kc, vc, ks, vs, table, lens = decode_case(7, 16, 2, 2, 128, 16, [3000, 5, 800, 0, 129, 4000, 64], seed=84)
    args = (q[1], kc[1], vc[1], ks[1], vs[1], i32(table), i32(lens))
    a, b = (fa.attention_decode_paged_fp8(*args, causal=True) for _ in range(2))
    torch.cuda.synchronize()
    assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def test_decode_offsets_beyond_32_bits():
    """A cache of more than 4 GiB whose last pages are the ones in use."""
    d, Hkv, page = 128, 4, 128
    pages = (2 ** 32 + 2 ** 28) // (Hkv * page * d)
    q, kc, vc, ks, vs, table, lens = decode_case(2, 8, Hkv, 1, d, page, [1000, 700], seed=85, stale=False)
    n = kc[0].shape[0]
    big = [torch.zeros((pages, Hkv, page, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    sc = [torch.zeros((pages, Hkv), device="cuda") for _ in range(2)]
    for t, s in zip(big + sc, (kc[1], vc[1], ks[1], vs[1])):
        t[-n:] = s
    ref = paged.decode_paged(q[0], kc[0], vc[0], ks[0], vs[0], table, lens, d ** -0.5, False)
    check_decode(q, (kc[0], big[0]), (vc[0], big[1]), (ks[0], sc[0]), (vs[0], sc[1]), table + pages - n, lens, d ** -0.5, False, d,
                 want=ref)
    k64, k = bf16(np.random.default_rng(1).standard_normal((1, Hkv, 3, d)))
    slots = (pages - 2) * page + np.array([[0, 1, 2]])
    want = [x[0].copy() for x in (kc, vc, ks, vs)]
    fa.fa_cache_append_fp8(k, k, i32(slots), *big, *sc)
    paged.append(k64, k64, slots - (pages - n) * page, *want, page)
    assert np.array_equal(big[0][-n:].cpu().numpy(), want[0]) and np.array_equal(sc[1][-n:].cpu().numpy(), want[3])
    assert int(big[0][:-n].max()) == 0


# ---------------------------------------------------------------------------------------------- run together
class Loop:
    """A decode loop's state on the GPU: what one step reads and writes, and the same state in the oracle."""

    def __init__(self, B, H, Hkv, N, d, page, pages, per_row, seed):
        self.shape = (B, H, Hkv, N, d, page)
        self.rng = np.random.default_rng(seed)
        self.n_table, self.n_free = np.full((B, per_row), -1), self.rng.permutation(pages)
        self.n_ctx, self.n_head = np.zeros(B, int), 0
        self.n_kc, self.n_vc = (np.full((pages, Hkv, page, d), 0x7F, np.uint8) for _ in range(2))
        self.n_ks, self.n_vs = (np.full((pages, Hkv), np.nan) for _ in range(2))
        self.table, self.free, self.ctx, self.head = i32(self.n_table), i32(self.n_free), i32(self.n_ctx), i32([0])
        self.kc, self.vc = (torch.full((pages, Hkv, page, d), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
        self.ks, self.vs = (torch.full((pages, Hkv), math.nan, device="cuda") for _ in range(2))
        self.freq, self.factor = fa.rope_frequencies(d, 10000.0, "bands", 8.0, 64.0)
        # a fused projection, token-major, and the step's buffers
        self.qkv = torch.zeros(B, N, H + 2 * Hkv, d, dtype=torch.bfloat16, device="cuda")
        self.new = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.slots, self.pos = (torch.zeros(B, N, dtype=torch.int32, device="cuda") for _ in range(2))
        self.qk = torch.zeros(B, H + Hkv, N, d, dtype=torch.bfloat16, device="cuda")
        self.o = torch.zeros(B, H, N, d, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.zeros(B, H, N, device="cuda")
        self.work = torch.empty(max(16, fa.fa_fwd_decode_paged_fp8_workspace_size(B, H, Hkv, N, d)), dtype=torch.uint8, device="cuda")

    def load(self, new):
        B, H, Hkv, N, d, _ = self.shape
        self.x64, x = bf16(self.rng.standard_normal((B, N, H + 2 * Hkv, d)))
        self.qkv.copy_(x)
        self.n_new = np.asarray(new)
        self.new.copy_(i32(new))

    def step(self):
        B, H, Hkv, N, d, page = self.shape
        fa.fa_page_tables(self.ctx, self.new, self.free, self.head, self.table, self.slots, self.pos, self.ctx, self.head, page)
        x = self.qkv.transpose(1, 2)
        fa.fa_rope(x[:, :H + Hkv], self.qk, self.pos, self.freq, self.factor)
        fa.fa_cache_append_fp8(self.qk[:, H:].contiguous(), x[:, H + Hkv:].contiguous(), self.slots, self.kc, self.vc, self.ks, self.vs)
        fa.fa_fwd_decode_paged_fp8(self.qk[:, :H].contiguous(), self.kc, self.vc, self.ks, self.vs, self.table, self.ctx,
                                   self.o, self.lse, d ** -0.5, True, self.work)

    def check(self):
        B, H, Hkv, N, d, page = self.shape
        torch.cuda.synchronize()
        self.n_table, self.n_free, slots, pos, self.n_ctx, self.n_head = paged.page_tables(
            self.n_ctx, self.n_new, self.n_free, self.n_head, self.n_table, N, page)
        for got, want in ((self.table, self.n_table), (self.free, self.n_free), (self.slots, slots), (self.pos, pos),
                          (self.ctx, self.n_ctx), (self.head, [self.n_head])):
            assert np.array_equal(got.cpu().numpy(), want)
        x = self.x64.transpose(0, 2, 1, 3)
        rot = paged.rope(x[:, :H + Hkv], pos, self.freq.cpu().numpy(), self.factor)
        qk = gu.to_f64(self.qk)
        assert np.max(np.abs(qk - rot) - 2.0 ** -8 * np.abs(rot)) <= 2.0 ** -20 * 2 * np.abs(x).max()
        paged.append(qk[:, H:], x[:, H + Hkv:], slots, self.n_kc, self.n_vc, self.n_ks, self.n_vs, page)
        assert np.array_equal(self.kc.cpu().numpy(), self.n_kc) and np.array_equal(self.vc.cpu().numpy(), self.n_vc)
        assert np.array_equal(self.ks.cpu().numpy().astype(float), self.n_ks, equal_nan=True)
        o, lse = self.o, self.lse
        self_o, self_l = gu.to_f64(o), gu.to_f64(lse)
        ro, rl, mag, big = paged.decode_paged(qk[:, :H], self.n_kc, self.n_vc, self.n_ks, self.n_vs, self.n_table, self.n_ctx, d ** -0.5, True)
        none = np.isneginf(rl)
        e = (d + 8) * 2.0 ** -23 * big + 2.0 ** -20
        assert np.array_equal(np.isneginf(self_l), none) and np.all(self_o[none] == 0)
        assert np.all(np.abs(self_l - rl)[~none] <= (e + 2.0 ** -23 * np.abs(rl))[~none])
        assert np.all(np.abs(self_o - ro) <= 2.0 ** -8 * np.abs(ro) + (2.0 ** -11 + 2.0 ** -14 + 2 * e[..., None]) * mag)


SCRIPT = [[5, 5, 0, 3, 1], [1, 1, 4, 1, 0], [5, -1, 5, 5, 5], [1, 5, 1, -1, 1], [5, 5, 5, 0, 5], [-1, -1, 1, 5, 1], [5, 2, 5, 5, -1]]


@pytest.mark.parametrize("d,page", [(64, 16), (128, 32)])
def test_decode_loop(d, page):
    loop = Loop(5, 8, 2, 5, d, page, pages=12, per_row=3, seed=d)
    for new in SCRIPT * 3:
        loop.load(new)
        loop.step()
        loop.check()


@pytest.mark.parametrize("two", [False, True])
def test_decode_loop_captured(two):
    """The whole step in a CUDA graph, replayed as the lengths grow; with `two`, two captured loops that share
    one workspace and are replayed one after the other."""
    loops = [Loop(5, 8, 2, 5, 128, 16, pages=14, per_row=3, seed=90 + i) for i in range(2 if two else 1)]
    graphs = []
    for lp in loops:
        lp.work = loops[0].work
        lp.load([0] * 5)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            lp.step()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lp.step()
        graphs.append(g)
    for new in SCRIPT:
        for lp in loops:
            lp.load(new)
        for g in graphs:
            g.replay()
        for lp in loops:
            lp.check()


def test_decode_on_two_streams():
    """Two calls at once on streams of their own, each with its workspace."""
    cases = [decode_case(3, 16, 2, 2, 128, 16, [4000, 1, 900], seed=95 + i) for i in range(2)]
    alone = []
    for c in cases:
        q, kc, vc, ks, vs, table, lens = c
        alone.append(fa.attention_decode_paged_fp8(q[1], kc[1], vc[1], ks[1], vs[1], i32(table), i32(lens), causal=True))
    args = [(c[0][1], c[1][1], c[2][1], c[3][1], c[4][1], i32(c[5]), i32(c[6])) for c in cases]
    work = [torch.empty(max(16, fa.fa_fwd_decode_paged_fp8_workspace_size(3, 16, 2, 2, 128)), dtype=torch.uint8, device="cuda")
            for _ in cases]
    outs = [(torch.empty_like(a[0]), torch.empty(a[0].shape[:3], device="cuda")) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for rep in range(20):
        for s, a, w, (o, lse) in zip(streams, args, work, outs):
            fa.fa_fwd_decode_paged_fp8(*a, o, lse, 128 ** -0.5, True, w, stream=s)
    torch.cuda.synchronize()
    for (o, lse), (ro, rl) in zip(outs, alone):
        assert torch.equal(o, ro) and torch.equal(lse, rl)


def test_allocating_calls_on_another_stream():
    """What a call allocates for another stream is not handed to the current stream while it runs."""
    q, kc, vc, ks, vs, table, lens = decode_case(16, 16, 2, 2, 128, 16, [4000 + i for i in range(16)], seed=97)
    args = (q[1], kc[1], vc[1], ks[1], vs[1], i32(table), i32(lens))
    x = torch.randn(4, 16, 4096, 128, device="cuda").to(torch.bfloat16)
    freq = fa.rope_frequencies(128)[0]
    ro, rl = fa.attention_decode_paged_fp8(*args, causal=True)
    ry = fa.rope_backward(fa.rope_forward(x, None, freq), None, freq)
    torch.cuda.synchronize()
    n = fa.fa_fwd_decode_paged_fp8_workspace_size(16, 16, 2, 2, 128)
    side, outs = torch.cuda.Stream(), []
    for _ in range(20):
        outs.append(fa.attention_decode_paged_fp8(*args, causal=True, stream=side))
        y = fa.rope_backward(fa.rope_forward(x, None, freq, stream=side), None, freq, stream=side)
        for size in (n, 2 * x.numel()):
            torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert all(torch.equal(o, ro) and torch.equal(lse, rl) for o, lse in outs)
    assert torch.equal(y, ry)


def test_python_calls_refuse_tensors_that_do_not_fit():
    """Each tensor of a call in turn with another type, another shape or not contiguous: refused before any launch."""
    bf, i4, f4, u1 = torch.bfloat16, torch.int32, torch.float32, torch.uint8
    t = lambda dtype, *shape: torch.zeros(*shape, dtype=dtype, device="cuda")
    q, kv, slots, cache, scale = t(bf, 2, 4, 3, 64), t(bf, 2, 2, 3, 64), t(i4, 2, 3), t(u1, 5, 2, 16, 64), t(f4, 5, 2)
    table, two, one, free, lse = t(i4, 2, 2), t(i4, 2), t(i4, 1), t(i4, 5), t(f4, 2, 4, 3)
    work = t(u1, fa.fa_fwd_decode_paged_fp8_workspace_size(2, 4, 2, 3, 64))
    calls = [(fa.fa_cache_append_fp8, (kv, kv, slots, cache, cache, scale, scale), ()),
             (fa.fa_page_tables, (two, two, free, one, table, slots, slots, two, one), (16,)),
             (lambda *a: fa.fa_fwd_decode_paged_fp8(*a, 0.1, False, work), (q, cache, cache, scale, scale, table, two, q, lse), ()),
             (lambda q, *a: fa.fa_rope(q, q, *a), (q, slots, t(torch.float64, 32)), ())]
    for fn, args, rest in calls:
        fn(*(a.clone() for a in args), *rest)
        for n, a in enumerate(args):
            apart = torch.zeros(*a.shape[:-1], 2 * a.shape[-1], dtype=a.dtype, device="cuda")[..., ::2]
            bads = [a.to(torch.int64), a.cpu(), a[None]]
            if not apart.is_contiguous():              # one element is, whatever its stride
                bads.append(apart)
            for bad in bads:
                with pytest.raises(ValueError):
                    fn(*args[:n], bad, *args[n + 1:], *rest)
    torch.cuda.synchronize()


def test_empty_calls():
    z = torch.zeros
    bf, c = torch.bfloat16, "cuda"
    q = z(0, 4, 1, 64, dtype=bf, device=c)
    kc = z(3, 2, 16, 64, dtype=torch.uint8, device=c)
    ks = z(3, 2, device=c)
    o, lse = fa.attention_decode_paged_fp8(q, kc, kc, ks, ks, z(0, 2, dtype=torch.int32, device=c), z(0, dtype=torch.int32, device=c))
    assert o.numel() == lse.numel() == 0
    # a cache without pages, a table without columns: every row is empty
    q = z(2, 4, 3, 64, dtype=bf, device=c)
    for pages, cols in ((0, 3), (3, 0)):
        o, lse = fa.attention_decode_paged_fp8(q, kc[:pages], kc[:pages], ks[:pages], ks[:pages],
                                               z(2, cols, dtype=torch.int32, device=c), i32([7, 9]))
        assert bool((o == 0).all()) and bool(torch.isneginf(lse).all())
    assert fa.rope_forward(z(2, 3, 0, 64, dtype=bf, device=c), None, fa.rope_frequencies(64)[0]).numel() == 0
