"""Pins of the paged-cache oracle (oracle/paged.py): the e4m3 grid against torch's cast, the cache write
against its definition, the page tables against invariants, the rotation against brute force, and decode
against the rectangular oracle on the same tokens laid out contiguously."""
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import paged


def test_e4m3_rounding_matches_torch():
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.standard_normal(20000) * 10.0 ** rng.uniform(-4, 3, 20000), paged.E4M3[np.isfinite(paged.E4M3)],
                        np.arange(0, 900) * 2.0 ** -11, [0.0, -0.0, 448.0, -448.0]])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(paged.e4m3_codes(x), want)
    assert np.array_equal(paged.e4m3_codes([500.0, -1e9, math.nan, math.inf]), [0x7E, 0xFE, 0x7F, 0x7F])


def test_scale_is_the_smallest_power_of_two():
    for a in (1.0, 448.0, 449.0, 447.9, 1e-3, 7.0, 7.0001, 2.0 ** 40):
        s = paged.scale_for(a)
        assert a <= 448 * s and a > 224 * s and math.log2(s) == int(math.log2(s))
    assert paged.scale_for(0.0) == 2.0 ** -60 and paged.scale_for(1e38) == 2.0 ** 60


def test_append_grows_the_scale_and_keeps_the_codes():
    rng = np.random.default_rng(2)
    page, d = 16, 64
    kc, vc = (np.full((3, 1, page, d), 0x7F, np.uint8) for _ in range(2))
    ks, vs = np.full((3, 1), 99.0), np.full((3, 1), np.nan)
    x = rng.standard_normal((1, 1, 5, d))
    slots = np.array([[16, 17, 18, -1, 19]])
    paged.append(x, x, slots, kc, vc, ks, vs, page)
    s = paged.scale_for(np.abs(x[0, 0, [0, 1, 2]]).max())     # token 4's run starts anew behind the gap
    s2 = max(s, paged.scale_for(np.abs(x[0, 0, 4]).max()))
    assert ks[1, 0] == vs[1, 0] == s2 and ks[0, 0] == 99.0
    got = paged.E4M3[kc[1, 0, :4]] * ks[1, 0]
    assert np.max(np.abs(got - x[0, 0, [0, 1, 2, 4]])) <= 2.0 ** -4 * np.abs(x).max()
    paged.append(x * 64, x * 64, np.array([[20, -1, -1, -1, -1]]), kc, vc, ks, vs, page)
    assert ks[1, 0] == paged.scale_for(64 * np.abs(x[0, 0, 0]).max()) > s2
    moved = paged.E4M3[kc[1, 0, :4]] * ks[1, 0]
    assert np.max(np.abs(moved - got)) <= ks[1, 0] * 2.0 ** -10      # only subnormals move
    assert np.all(kc[[0, 2]] == 0x7F)


def test_page_tables_never_share_a_page():
    rng = np.random.default_rng(3)
    page, B, N, per_row, pages = 16, 7, 40, 8, 40
    table = np.full((B, per_row), -1)
    free, head, ctx = rng.permutation(pages), 0, np.zeros(B, int)
    for step in range(60):
        new = rng.integers(-1, N + 2, B)
        table, free, slots, pos, ctx2, head = paged.page_tables(ctx, new, free, head, table, N, page)
        held = [p for b in range(B) for p in table[b, : -(-int(ctx2[b]) // page)]]
        assert len(set(held)) == len(held) and set(held) | set(free[head:]) == set(range(pages))
        live = slots[slots >= 0]
        assert len(set(live)) == len(live)
        for b in range(B):
            grew = ctx2[b] - ctx[b] if new[b] >= 0 else 0
            assert (slots[b] >= 0).sum() == grew
            assert np.array_equal(pos[b, :grew], np.arange(ctx[b], ctx[b] + grew))
        ctx = ctx2


def test_rope_is_a_rotation_and_depends_on_distance():
    rng = np.random.default_rng(4)
    f = 10000.0 ** (-np.arange(0, 32, 2) / 32)
    for inter in (False, True):
        q, k = rng.standard_normal((2, 1, 1, 1, 64))
        rot = lambda x, p: paged.rope(x, np.array([[p]]), f, 1.0, inter)  # noqa: E731
        a = float(np.sum(rot(q, 1000007) * rot(k, 1000000)))
        b = float(np.sum(rot(q, 7) * rot(k, 0)))
        assert abs(a - b) < 1e-7
        y = rot(q, 12345)
        assert np.allclose(paged.rope(y, np.array([[12345]]), f, 1.0, inter, True), q, atol=1e-12)
        assert np.array_equal(y[..., 32:], q[..., 32:])
        i, j = (0, 1) if inter else (0, 16)
        assert np.isclose(y[..., i], q[..., i] * math.cos(12345) - q[..., j] * math.sin(12345)).all()


def test_rope_gradient_by_differences():
    rng = np.random.default_rng(5)
    f = 100.0 ** (-np.arange(0, 16, 2) / 16)
    x, w = rng.standard_normal((2, 1, 1, 2, 64))
    pos = np.array([[3, 9]])
    g = paged.rope(w, pos, f, 1.3, True, transpose=True)
    for _ in range(10):
        t = rng.standard_normal(x.shape)
        d = (np.sum(w * paged.rope(x + 1e-6 * t, pos, f, 1.3, True)) - np.sum(w * paged.rope(x - 1e-6 * t, pos, f, 1.3, True))) / 2e-6
        assert abs(d - np.sum(g * t)) < 1e-6


@pytest.mark.parametrize("causal", [False, True])
def test_decode_matches_the_rectangular_oracle(causal):
    rng = np.random.default_rng(6)
    B, H, Hkv, Nq, d, page, pages = 3, 4, 2, 3, 64, 16, 20
    kc, vc = (paged.e4m3_codes(rng.standard_normal((pages, Hkv, page, d)) * 50) for _ in range(2))
    ks, vs = (2.0 ** rng.integers(-8, -4, (pages, Hkv)) for _ in range(2))
    table = rng.permutation(pages)[:18].reshape(3, 6)
    lens = np.array([70, 2, 0])
    q = rng.standard_normal((B, H, Nq, d))
    o, lse, mag, big = paged.decode_paged(q, kc, vc, ks, vs, table, lens, 0.125, causal)
    for h in range(H):
        at = table[0]
        K = (paged.E4M3[kc[at, h // 2]] * ks[at, h // 2][:, None, None]).reshape(-1, d)[:70]
        V = (paged.E4M3[vc[at, h // 2]] * vs[at, h // 2][:, None, None]).reshape(-1, d)[:70]
        ro, rl = oracle.head_forward_rect(q[0, h], K, V, 0.125, causal)
        assert np.allclose(o[0, h], ro, atol=1e-12) and np.allclose(lse[0, h], rl, atol=1e-12)
    assert np.all(o[2] == 0) and np.all(lse[2] == -np.inf)
    assert (lse[1, 0, 0] == -np.inf) == causal            # two tokens, three queries
    assert np.all(mag >= np.abs(o) - 1e-12) and np.all(big >= 0)
