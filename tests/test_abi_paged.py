"""The calls on the 8-bit paged cache and fa_rope without a GPU: argument errors come back as status codes
before anything touches a device, empty calls succeed, and the host-side frequencies follow their formulas."""
import ctypes
import math

import numpy as np
import pytest
import torch

import exact_io_aware_55_b200 as fa

F, C = ctypes.c_float, fa.STATUS_CODES
P = 4096
NO_GPU = (C["FA_ERR_ARCH"], C["FA_ERR_LAUNCH"])     # got past every argument check
gpu = fa.lib.fa_get_device_status(None) != C["FA_ERR_ARCH"]


def rope(x=P, y=2 * P, pos=P, freq=P, factor=1.0, B=1, H=2, N=8, d=64, rot=64, inter=0, tr=0, xs=(1024, 512, 64),
         ys=(1024, 512, 64)):
    return fa.lib.fa_rope(x, y, pos, freq, F(factor), B, H, N, d, rot, inter, tr, *xs, *ys, None)


def test_rope_argument_errors():
    assert rope(d=96) == C["FA_ERR_UNSUPPORTED"]
    assert rope(rot=8) == rope(rot=24) == rope(rot=128) == C["FA_ERR_UNSUPPORTED"]
    assert rope(B=-1) == rope(inter=2) == rope(tr=-1) == rope(factor=math.inf) == C["FA_ERR_INVALID_ARG"]
    assert rope(x=None) == rope(y=None) == rope(freq=None) == C["FA_ERR_INVALID_ARG"]
    assert rope(xs=(-8, 512, 64)) == C["FA_ERR_INVALID_ARG"]
    assert rope(B=2, ys=(0, 512, 64)) == C["FA_ERR_INVALID_ARG"]          # output rows on one another
    assert rope(ys=(0, 512, 32)) == C["FA_ERR_INVALID_ARG"]
    assert rope(y=P, ys=(1024, 64, 128)) == C["FA_ERR_INVALID_ARG"]       # in place needs equal strides
    assert rope(xs=(1024, 516, 64)) == C["FA_ERR_ALIGNMENT"]
    assert rope(x=P + 8) == rope(pos=P + 2) == rope(freq=P + 4) == C["FA_ERR_ALIGNMENT"]
    assert rope(B=40000, H=2) == rope(B=40000, N=1 << 20, H=1) == C["FA_ERR_UNSUPPORTED"]
    assert rope(N=0, x=None) == C["FA_OK"]


def test_rope_refuses_output_rows_on_one_another():
    bad = C["FA_ERR_INVALID_ARG"]
    assert rope(B=2, H=2, N=8, ys=(512, 512, 64)) == bad                  # two batches in the same place
    assert rope(B=1, H=2, N=8, ys=(0, 448, 64)) == bad                    # a head on the last token of the one before
    assert rope(B=1, H=2, N=8, ys=(0, 64, 64)) == bad
    assert rope(B=3, H=2, N=8, ys=(960, 512, 64)) == bad
    assert rope(B=2, H=2, N=8, ys=(1 << 62, 512, 64)) == bad              # extents beyond 64 bits
    assert rope(y=P, xs=(512, 512, 64), B=2, ys=(512, 512, 64)) == bad    # in place on repeated rows


@pytest.mark.skipif(gpu, reason="the pointers are not memory")
def test_valid_calls_reach_the_device_check():
    assert rope(pos=None, xs=(0, 0, 0)) in NO_GPU                         # repeated input rows are fine
    assert append(hkv=3, page=128) in NO_GPU
    assert tables(N=0, slots=None, pos=None) in NO_GPU
    need = fa.fa_fwd_decode_paged_fp8_workspace_size(2, 8, 2, 3, 64)
    assert decode(ws=P, wbytes=need) in NO_GPU


def append(k=P, v=P, slots=P, kc=P, vc=P, ks=P, vs=P, B=2, hkv=2, N=4, d=64, pages=9, page=16):
    return fa.lib.fa_cache_append_fp8(k, v, slots, kc, vc, ks, vs, B, hkv, N, d, pages, page, None)


def test_append_argument_errors():
    assert append(d=32) == append(page=48) == append(page=256) == C["FA_ERR_UNSUPPORTED"]
    assert append(B=-1) == append(pages=-1) == C["FA_ERR_INVALID_ARG"]
    for name in ("k", "v", "slots", "kc", "vc", "ks", "vs"):
        assert append(**{name: None}) == C["FA_ERR_INVALID_ARG"], name
        assert append(**{name: P + 2}) == C["FA_ERR_ALIGNMENT"], name
    assert append(B=30000, hkv=3) == append(pages=1 << 30, hkv=4) == append(pages=1 << 27) == C["FA_ERR_UNSUPPORTED"]
    assert append(B=0, k=None) == append(N=0, k=None) == C["FA_OK"]


def tables(ctx=P, new=P, free=P, head=P, table=P, slots=P, pos=P, seq=P, out=P, B=3, N=2, nf=10, mp=4, page=16):
    return fa.lib.fa_page_tables(ctx, new, free, head, table, slots, pos, seq, out, B, N, nf, mp, page, None)


def test_page_tables_argument_errors():
    assert tables(page=20) == tables(B=70000) == tables(mp=1 << 28) == C["FA_ERR_UNSUPPORTED"]
    assert tables(B=-1) == tables(N=-1) == tables(nf=-1) == tables(mp=-1) == C["FA_ERR_INVALID_ARG"]
    for name in ("ctx", "new", "free", "head", "table", "slots", "pos", "seq", "out"):
        assert tables(**{name: None}) == C["FA_ERR_INVALID_ARG"], name
        assert tables(**{name: P + 1}) == C["FA_ERR_ALIGNMENT"], name
    assert tables(B=0, ctx=None) == C["FA_OK"]


def decode(q=P, kc=P, vc=P, ks=P, vs=P, table=P, lens=P, o=P, lse=P, B=2, H=8, hkv=2, Nq=3, d=64, pages=9, page=16,
           mp=4, scale=0.1, causal=0, ws=None, wbytes=0):
    return fa.lib.fa_fwd_decode_paged_fp8(q, kc, vc, ks, vs, table, lens, o, lse, B, H, hkv, Nq, d, pages, page, mp,
                                          F(scale), causal, ws, wbytes, None)


def test_decode_argument_errors():
    assert decode(d=96) == decode(page=17) == decode(Nq=17) == decode(B=9000) == C["FA_ERR_UNSUPPORTED"]
    assert decode(H=7) == decode(hkv=0) == decode(scale=-1.0) == decode(scale=math.nan) == C["FA_ERR_INVALID_ARG"]
    assert decode(causal=2) == decode(B=-1) == decode(mp=-1) == decode(pages=-1) == C["FA_ERR_INVALID_ARG"]
    assert decode(pages=1 << 30, hkv=4) == decode(mp=1 << 27, page=16) == C["FA_ERR_UNSUPPORTED"]
    need = fa.fa_fwd_decode_paged_fp8_workspace_size(2, 8, 2, 3, 64)
    for name in ("q", "kc", "vc", "ks", "vs", "table", "lens", "o", "lse"):
        assert decode(ws=P, wbytes=need, **{name: None}) == C["FA_ERR_INVALID_ARG"], name
        assert decode(ws=P, wbytes=need, **{name: P + 2}) == C["FA_ERR_ALIGNMENT"], name
    if need:
        assert decode(ws=P, wbytes=need - 1) == decode(ws=None, wbytes=need) == C["FA_ERR_WORKSPACE"]
        assert decode(ws=P + 8, wbytes=need) == C["FA_ERR_ALIGNMENT"]
    assert decode(B=0, q=None) == decode(Nq=0, q=None) == decode(H=0, hkv=0, q=None) == C["FA_OK"]
    with pytest.raises(fa.FAError):
        fa.fa_fwd_decode_paged_fp8_workspace_size(1, 7, 2, 1, 64)


def test_decode_refuses_more_tiles_than_a_share_counts():
    big = dict(H=256, hkv=256, Nq=1, page=128, mp=(1 << 22) + (1 << 20), d=128, pages=9)
    assert decode(B=255, **big) == C["FA_ERR_UNSUPPORTED"]      # 1.25 * 2^22 * 256 * 255 / 148 > 2^31
    assert decode(B=100, **big) == C["FA_ERR_WORKSPACE"]        # counted; the next check is the workspace's


def test_python_wrappers_refuse():
    t = torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16)
    f = torch.zeros(8, dtype=torch.float64)
    i = torch.zeros(1, 1, dtype=torch.int32)
    for call in (lambda: fa.rope_forward(t, None, f), lambda: fa.fa_cache_append_fp8(t, t, i, t, t, f, f),
                 lambda: fa.attention_decode_paged_fp8(t, t, t, f, f, i, i),
                 lambda: fa.fa_page_tables(i[0], i[0], i[0], i[0], i, i, i, i[0], i[0], 16)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError):
        fa.rope_frequencies(64, scaling="other", device="cpu")


def test_rope_frequencies_follow_the_formulas():
    r, base, s, orig = 64, 10000.0, 8.0, 4096.0
    i = np.arange(r // 2)
    f = base ** (-2.0 * i / r)

    def got(scaling, **kw):
        t, a = fa.rope_frequencies(r, base, scaling, device="cpu", **kw)
        return t.numpy(), a

    for name, want in (("none", f), ("linear", f / s), ("ntk", (base * s ** (r / (r - 2))) ** (-2.0 * i / r))):
        g, a = got(name, factor=s)
        assert np.allclose(g, want, rtol=1e-14) and a == 1.0
    g, a = got("bands", factor=s, original_length=orig, low=1.0, high=4.0)
    wave = 2 * np.pi / f
    keep = np.clip((orig / wave - 1) / 3, 0, 1)
    assert a == 1.0 and np.allclose(g, f / s * (1 - keep) + f * keep, rtol=1e-14)
    assert g[0] == f[0] and np.isclose(g[-1], f[-1] / s)
    g, a = got("yarn", factor=s, original_length=orig, low=1.0, high=32.0)
    dim = lambda t: r * math.log(orig / (t * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    lo, hi = math.floor(dim(32.0)), math.ceil(dim(1.0))
    assert np.isclose(a, 0.1 * math.log(s) + 1)
    assert np.allclose(g[: lo + 1], f[: lo + 1]) and np.allclose(g[hi:], f[hi:] / s)
    mid = (lo + hi) // 2
    t = (mid - lo) / (hi - lo)
    assert np.isclose(g[mid], f[mid] / s * t + f[mid] * (1 - t))
    assert got("yarn", factor=1.0, original_length=orig, low=1.0, high=32.0)[1] == 1.0


def test_rope_frequencies_argument_errors():
    buf, att = (ctypes.c_double * 64)(), ctypes.c_double()

    def call(rot=64, base=1e4, scaling=0, factor=1.0, orig=4096.0, low=1.0, high=4.0, out=buf):
        return fa.lib.fa_rope_frequencies(out, ctypes.byref(att), rot, base, scaling, factor, orig, low, high)

    bad = [dict(rot=63), dict(rot=0), dict(base=1.0), dict(base=math.nan), dict(scaling=5), dict(scaling=-1),
           dict(scaling=1, factor=0.5), dict(scaling=2, rot=2, factor=2.0), dict(scaling=3, low=4.0), dict(scaling=4, low=0.0),
           dict(scaling=4, orig=0.0), dict(scaling=4, high=math.inf), dict(out=None)]
    for kw in bad:
        assert call(**kw) == C["FA_ERR_INVALID_ARG"], kw
    assert call() == C["FA_OK"]


def test_bad_page_status_text():
    assert C["FA_ERR_BAD_PAGE"] == 9 and "page" in fa.strerror(9)
