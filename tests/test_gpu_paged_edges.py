"""GPU tests of edges of the calls on the 8-bit paged cache.  Tolerances as in tests/test_gpu_paged.py, whose
helpers these tests use; what they add to them is derived beside each."""
import numpy as np
import pytest
import torch

from oracle import paged
from tests import gpu_util as gu
from tests.test_gpu_paged import SCRIPT, Loop, bf16, cache, check_append, check_decode, decode_case, fa, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def no_status():
    fa.fa_device_status()
    yield
    torch.cuda.synchronize()
    assert fa.fa_device_status() == (0, 0)


def upload(*pairs):
    for host, dev in pairs:
        dev.copy_(torch.from_numpy(host if host.dtype == np.uint8 else host.astype(np.float32)))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("what", ["query", "keys"])
def test_decode_rows_that_see_only_nan_behind_skipped_pages(what, d):
    """A row whose every visible score is NaN is NaN also where the first page of each tile lies outside the cache."""
    q, kc, vc, ks, vs, table, lens = decode_case(2, 4, 2, 2, d, 16, [300, 100], seed=201, stale=False)
    table[0, ::8] = -1                                  # a tile is 128 or 256 keys, 8 or 16 pages
    if what == "query":
        q[0][0, 1, 0, 3] = np.nan
        q[1][0, 1, 0, 3] = float("nan")
        rows = [(0, 1, 0)]
    else:
        for p in table[0][table[0] >= 0]:
            kc[0][p, 1, :, 5] = 0x7F
        upload((kc[0], kc[1]))
        rows = [(0, 2), (0, 3)]
    ref = paged.decode_paged(np.nan_to_num(q[0]), np.where(kc[0] == 0x7F, 0, kc[0]), vc[0], ks[0], vs[0], table, lens, d ** -0.5, False)
    for r in rows:
        for x in ref:
            x[r] = np.nan
    check_decode(q, kc, vc, ks, vs, table, lens, d ** -0.5, False, d, want=ref)
    assert fa.fa_device_status()[0] == fa.STATUS_CODES["FA_ERR_BAD_PAGE"]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("bad", [np.nan, -1.0])
@pytest.mark.parametrize("at", [0, 7])
def test_decode_value_scale_that_is_no_scale(at, bad, d):
    """A V scale that is NaN or negative shows as NaN in the rows that see its page, and in no others."""
    q, kc, vc, ks, vs, table, lens = decode_case(2, 4, 2, 3, d, 16, [113, 400], seed=202, stale=False)
    vs[0][table[0, at], 1] = bad                        # page 7 holds key 112, which the last query alone sees
    vs[1][int(table[0, at]), 1] = bad
    fine = np.where(np.isnan(vs[0]) | (vs[0] < 0), 1.0, vs[0])
    ref = paged.decode_paged(q[0], kc[0], vc[0], ks[0], fine, table, lens, d ** -0.5, True)
    for x in ref:
        x[0, 2:, 2 if at == 7 else slice(None)] = np.nan
    check_decode(q, kc, vc, ks, vs, table, lens, d ** -0.5, True, d, want=ref)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("below", [0, 10, 20, 26, 30, 44])
@pytest.mark.parametrize("Nq", [1, 4])
def test_decode_columns_that_only_light_keys_fill(Nq, below, d):
    """Half of the columns are zero in the pages of a large V scale, so that the others, 2^-below of it, alone count
    there.  A weight times its V scale is rounded to 11 bits (in the usual tolerance), and by at most 2^-23 + 2^-25 where
    the maximum in use is 2^11: 1.25 * 2^-34 of the largest product of the row, times the key's code."""
    q, kc, vc, ks, vs, table, lens = decode_case(2, 8, 2, Nq, d, 16, [900, 300], seed=203, q_mult=0.25, stale=False)
    heavy = np.zeros(vs[0].shape[0], bool)
    heavy[table[:, ::2]] = True                         # every tile has pages of both kinds
    vs[0][:] = np.where(heavy[:, None], 1.0, 2.0 ** -below)
    vc[0][heavy, :, :, : d // 2] = 0
    upload((vs[0], vs[1]), (vc[0], vc[1]))
    scale = d ** -0.5
    ref = paged.decode_paged(q[0], kc[0], vc[0], ks[0], vs[0], table, lens, scale, False)
    o, _ = (gu.to_f64(t) for t in check_decode_floor(q, kc, vc, ks, vs, table, lens, scale, d, ref))
    light = np.abs(ref[0][..., : d // 2])
    if below == 44:
        assert np.all(o[..., : d // 2] == 0)            # below half of the last step, 2^-34: gone, and documented as such
    if below <= 20:                                     # 11 bits, but for rounding errors of sums that cancel
        assert np.median(np.abs(o[..., : d // 2] - ref[0][..., : d // 2]) / light) <= 2.0 ** -8


def check_decode_floor(q, kc, vc, ks, vs, table, lens, scale, d, ref):
    o, lse, mag, big = ref
    B, H, Nq, _ = q[0].shape
    page, Hkv = kc[0].shape[2], kc[0].shape[1]
    floor = np.zeros_like(o)
    for b in range(B):
        j = np.arange(lens[b])
        p, r = table[b, j // page], j % page
        for h in range(H):
            hk = h // (H // Hkv)
            K, C, w = paged.E4M3[kc[0][p, hk, r]] * ks[0][p, hk][:, None], paged.E4M3[vc[0][p, hk, r]], vs[0][p, hk]
            s = scale * (K @ q[0][b, h].T)
            top = (np.exp(s - lse[b, h]) * w[:, None]).max(0)
            floor[b, h] = 1.25 * 2.0 ** -34 * top[:, None] * np.abs(C).sum(0)
    got = fa.attention_decode_paged_fp8(q[1], kc[1], vc[1], ks[1], vs[1], i32(table), i32(lens), scale)
    e = (d + 8) * 2.0 ** -23 * big + 2.0 ** -20
    assert np.all(np.abs(gu.to_f64(got[1]) - lse) <= e + 2.0 ** -23 * np.abs(lse))
    tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -11 + 2.0 ** -14 + 2 * e[..., None]) * mag + floor + 1e-38
    worst = np.max(np.abs(gu.to_f64(got[0]) - o) / tol)
    assert worst <= 1, f"O off by {worst:.3g} of its bound"
    return got


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 128])
def test_append_to_pages_whose_scale_is_no_power_of_two(page, d):
    """A cache that was quantised elsewhere, with any positive scale: code = e4m3(x / scale) where the scale stays, ties to
    even included (values are scale times numbers of six bits, exact in bf16), and codes moved to a power of two where it grows."""
    rng = np.random.default_rng(204)
    pages = 24
    kc, ks, kct, kst = cache(rng, pages, 1, page, d)
    vc, vs, vct, vst = cache(rng, pages, 1, page, d)
    for s in (ks, vs):
        s[:] = rng.choice([0.75, 1.25, 0.625, 0.875], s.shape) * 2.0 ** rng.integers(-6, 3, s.shape)
    upload((ks, kst), (vs, vst))

    def values(scale):
        m = rng.integers(16, 32, (pages, 1, 2, d)) * 2.0 ** rng.integers(-8, 4, (pages, 1, 2, d)) * rng.choice([-1, 1], (pages, 1, 2, d))
        m[::3] *= 64.0                                  # these pages grow
        return m * scale[:, :, None, None]

    (k64, k), (v64, v) = bf16(values(ks)), bf16(values(vs))
    slots = np.arange(pages)[:, None] * page + np.array([[3, 4]])
    check_append(k64, v64, k, v, slots, (kc, kct), (vc, vct), (ks, kst), (vs, vst), page, 1, d)


@pytest.mark.parametrize("B,N,page,pages", [(1, 5, 16, 6), (5, 40, 16, 30), (33, 3, 32, 25), (2500, 2, 16, 4000), (3, 700, 128, 40)])
def test_page_tables_of_requests_that_shrink(B, N, page, pages):
    """Lengths lowered between calls (rejected drafts), across pages' borders too: every call as the oracle's, and no page
    is lost or in two places."""
    rng = np.random.default_rng(B + N)
    per_row = max(3, -(-4 * N // page))
    table, free, head, ctx = np.full((B, per_row), -1), rng.permutation(pages), 0, np.zeros(B, int)
    held, held_t = np.zeros(B, int), torch.zeros(B, dtype=torch.int32, device="cuda")
    for _ in range(8):
        new = rng.integers(0, N + 1, B)
        new[rng.random(B) < 0.1] = -1
        new[rng.random(B) < 0.05] = N + 1
        c, f, h, t = i32(ctx), i32(free), i32([head]), i32(table)
        slots, pos = (torch.empty(B, N, dtype=torch.int32, device="cuda") for _ in range(2))
        fa.fa_page_tables(c, i32(new), f, h, t, slots, pos, c, h, page, held_pages=held_t)
        table, free, wslots, wpos, ctx, head = paged.page_tables(ctx, new, free, head, table, N, page, held)
        for got, want in ((slots, wslots), (pos, wpos), (c, ctx), (h, [head]), (t, table), (f, free), (held_t, held)):
            assert np.array_equal(got.cpu().numpy(), np.asarray(want))
        own = [p for b in range(B) for p in table[b, :held[b]]] + list(free[head:])
        assert sorted(own) == list(range(pages))
        ctx = np.maximum(ctx - rng.integers(0, 2 * N, B), 0)


def test_page_tables_held_counts_out_of_range():
    """A count below the length's pages, or beyond the row, is the nearest possible one; other tensors are refused."""
    table, free = np.arange(8).reshape(2, 4), np.arange(8, 16)
    ctx, new, held = np.array([20, 5]), np.array([30, 3]), np.array([-7, 10 ** 6])
    held_t, t, f, h = i32(held), i32(table), i32(free), i32([4])
    slots, pos, seq = (torch.empty(*s, dtype=torch.int32, device="cuda") for s in ((2, 32), (2, 32), (2,)))
    args = (i32(ctx), i32(new), f, h, t, slots, pos, seq, h, 16)
    fa.fa_page_tables(*args, held_pages=held_t)
    table, free, wslots, _, lens, head = paged.page_tables(ctx, new, free, 4, table, 32, 16, held)
    assert list(held) == [4, 4] and head == 6
    for got, want in ((slots, wslots), (seq, lens), (h, [head]), (t, table), (held_t, held)):
        assert np.array_equal(got.cpu().numpy(), np.asarray(want))
    for bad in (held_t.long(), held_t[:1], held_t.cpu(), held_t[None]):
        with pytest.raises(ValueError):
            fa.fa_page_tables(*args, held_pages=bad)


def test_batches_of_more_heads_than_a_grid_dimension():
    """1030 requests of 64 heads (65920) through rope, the cache write and the paged decode."""
    rng = np.random.default_rng(205)
    B, H, d, page = 1030, 64, 64, 16
    x64, x = bf16(rng.standard_normal((B, H, 1, d)))
    freq, _ = fa.rope_frequencies(d)
    pos = rng.integers(0, 5000, (B, 1))
    ref = paged.rope(x64, pos, freq.cpu().numpy())
    y = gu.to_f64(fa.rope_forward(x, i32(pos), freq))
    pair = np.tile(np.abs(x64[..., : d // 2]) + np.abs(x64[..., d // 2:]), 2)
    assert np.all(np.abs(y - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * pair)
    kc, ks, kct, kst = cache(rng, B, H, page, d)
    slots = rng.permutation(B)[:, None] * page + rng.integers(0, page, (B, 1))
    check_append(x64, x64, x, x, slots, (kc, kct), (kc, kct), (ks, kst), (ks, kst), page, H, d)
    lens = rng.integers(0, 40, B)
    case = decode_case(B, H, 8, 1, d, page, lens, seed=206)
    check_decode(*case, d ** -0.5, False, d)


def test_decode_loop_captured_over_two_streams():
    """A captured step whose rope calls run on a stream each, behind a memset and before a copy, and which joins them again."""
    loop = Loop(5, 8, 2, 5, 128, 16, pages=14, per_row=3, seed=207)
    side = torch.cuda.Stream()

    def step():
        B, H, Hkv, N, d, page = loop.shape
        main = torch.cuda.current_stream()
        loop.o.zero_()
        fa.fa_page_tables(loop.ctx, loop.new, loop.free, loop.head, loop.table, loop.slots, loop.pos, loop.ctx, loop.head, page)
        x = loop.qkv.transpose(1, 2)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            fa.fa_rope(x[:, H:H + Hkv], loop.qk[:, H:], loop.pos, loop.freq, loop.factor)
            k = loop.qk[:, H:].contiguous()
        fa.fa_rope(x[:, :H], loop.qk[:, :H], loop.pos, loop.freq, loop.factor)
        q = loop.qk[:, :H].contiguous()
        main.wait_stream(side)
        fa.fa_cache_append_fp8(k, x[:, H + Hkv:].contiguous(), loop.slots, loop.kc, loop.vc, loop.ks, loop.vs)
        fa.fa_fwd_decode_paged_fp8(q, loop.kc, loop.vc, loop.ks, loop.vs, loop.table, loop.ctx, loop.o, loop.lse, d ** -0.5, True, loop.work)

    loop.load([0] * 5)
    first = torch.cuda.Stream()
    first.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(first):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for new in SCRIPT:
        loop.load(new)
        graph.replay()
        loop.check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H", [2, 8, 32])
def test_decode_nan_value_of_a_key_far_below_the_others(H, d):
    """The first tile's scores lie 300 below the second's, so that its weights are 0 in fp32: a NaN among its values shows all
    the same (0 times NaN), whichever way the two tiles are joined."""
    B, tile = 60, 128 if d == 128 else 256
    q, kc, vc, ks, vs, table, lens = decode_case(B, H, 2, 1, d, 16, [2 * tile] * B, seed=208, stale=False)
    q[0][:] = 0.0
    q[0][..., 0] = 1.0
    kc[0][..., 0] = 0x7E                                # 448, and -448 in the first tile
    kc[0][table[:, : tile // 16], :, :, 0] = 0xFE
    ks[0][:] = 2.0 ** -3
    vc[0][table[::3, 1], 1, 5, 7] = 0x7F
    upload((kc[0], kc[1]), (vc[0], vc[1]), (ks[0], ks[1]))
    q[1].copy_(torch.from_numpy(q[0]))
    scale = 300.0 / 112.0
    ref = paged.decode_paged(q[0], kc[0], vc[0], ks[0], vs[0], table, lens, scale, False)
    assert np.isnan(ref[0][::3, H // 2:, :, 7]).all() and np.isnan(ref[0]).sum() == 20 * (H // 2)
    check_decode(q, kc, vc, ks, vs, table, lens, scale, False, d, want=ref)


@pytest.mark.parametrize("seed", range(12))
def test_decode_drawn_nan_and_skipped_pages(seed):
    """NaN in queries, keys and values and pages outside the cache, drawn at random together: NaN where the definition has it."""
    rng = np.random.default_rng(300 + seed)
    d, page, causal = int(rng.choice([64, 128])), int(rng.choice([16, 32, 64])), bool(rng.integers(2))
    Hkv, group, Nq, B = int(rng.integers(1, 4)), int(rng.choice([1, 3, 4, 8])), int(rng.integers(1, 9)), int(rng.integers(1, 30))
    lens = [int(2 ** rng.uniform(0, 10)) for _ in range(B)]
    q, kc, vc, ks, vs, table, n = decode_case(B, group * Hkv, Hkv, Nq, d, page, lens, seed=int(rng.integers(2 ** 31)), stale=False)
    skipped = rng.random(table.shape) < 0.1
    kc[0][rng.random(kc[0].shape) < 2e-5] = 0x7F
    vc[0][rng.random(vc[0].shape) < 1e-4] = 0xFF
    table[skipped] = rng.choice([-1, 10 ** 8], skipped.sum())
    bad = rng.random(q[0].shape) < 1e-3
    q[0][bad] = np.nan
    q[1][torch.from_numpy(bad).cuda()] = float("nan")
    upload((kc[0], kc[1]), (vc[0], vc[1]))
    with np.errstate(invalid="ignore"):
        ref = paged.decode_paged(q[0], kc[0], vc[0], ks[0], vs[0], table, n, d ** -0.5, causal)
    check_decode(q, kc, vc, ks, vs, table, n, d ** -0.5, causal, d, want=ref)
    fa.fa_device_status()
