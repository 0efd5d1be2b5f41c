"""Edges of the calls on the 8-bit paged cache and of the rotary frequencies that need no GPU."""
import math

import numpy as np
import pytest

import exact_io_aware_55_b200 as fa
from oracle import paged


@pytest.mark.parametrize("scaling,high", [("yarn", 32.0), ("bands", 4.0)])
def test_rope_frequencies_default_edges_are_the_scaling_s_own(scaling, high):
    """Without low and high: 1 and 32 turns for the ramp over pairs, 1 and 4 for the bands."""
    rot, base, factor, length = 128, 10000.0, 8.0, 4096.0
    i = np.arange(rot // 2)
    f = base ** (-2.0 * i / rot)
    if scaling == "yarn":
        pair = lambda t: rot * math.log(length / (t * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        first, last = math.floor(pair(high)), math.ceil(pair(1.0))
        keep = 1 - np.clip((i - first) / (last - first), 0, 1)
    else:
        keep = np.clip((length * f / (2 * math.pi) - 1) / (high - 1), 0, 1)
    got, _ = fa.rope_frequencies(rot, base, scaling, factor, length, device="cpu")
    assert np.allclose(got.numpy(), f / factor * (1 - keep) + f * keep, rtol=1e-13)
    same, _ = fa.rope_frequencies(rot, base, scaling, factor, length, 1.0, high, device="cpu")
    assert np.array_equal(got.numpy(), same.numpy())


def test_page_tables_held_argument_errors():
    C, P = fa.STATUS_CODES, 4096

    def call(held=P, B=3, page=16, ctx=P):
        return fa.lib.fa_page_tables_held(ctx, P, P, P, P, P, P, P, P, held, B, 2, 10, 4, page, None)

    assert call(held=P + 2) == C["FA_ERR_ALIGNMENT"] and call(ctx=None) == C["FA_ERR_INVALID_ARG"]
    assert call(page=20) == C["FA_ERR_UNSUPPORTED"] and call(B=-1) == C["FA_ERR_INVALID_ARG"] and call(B=0) == C["FA_OK"]


def owned(table, held, free, head):
    return sorted([p for b, n in enumerate(held) for p in table[b, :n]] + list(free[head:]))


def test_lowered_lengths_lose_no_page():
    """A draft of 5 tokens rejected and drafted again: with the number of held pages the page behind the length is used again."""
    table, free, new = np.full((1, 4), -1), np.array([5, 1, 2, 3, 4, 0]), np.array([5])
    table[0, 0], held = 5, np.array([1])
    ctx, head = np.array([16]), 1
    for _ in range(3):
        table, free, slots, _, lens, head = paged.page_tables(ctx, new, free, head, table, 5, 16, held)
        assert lens[0] == 21 and held[0] == 2 and head == 2 and slots[0, 0] == table[0, 1] * 16
        assert len(set(owned(table, held, free, head))) == 6
    _, free, _, _, _, head = paged.page_tables(ctx, np.array([-1]), free, head, table, 5, 16, held)
    assert held[0] == 0 and head == 0 and sorted(free) == sorted(set(free))
    rng = np.random.default_rng(6)
    B, N, page, per_row, pages = 7, 40, 16, 8, 40
    table, free, head, ctx, held = np.full((B, per_row), -1), rng.permutation(pages), 0, np.zeros(B, int), np.zeros(B, int)
    for _ in range(80):
        table, free, slots, _, lens, head = paged.page_tables(ctx, rng.integers(-1, N + 2, B), free, head, table, N, page, held)
        assert owned(table, held, free, head) == list(range(pages))
        live = slots[slots >= 0]
        assert len(set(live)) == len(live)
        ctx = np.maximum(lens - rng.integers(0, 2 * N, B), 0)


def test_batches_of_many_heads_are_not_refused():
    """1024 requests of 64 heads (and 8192 of any number that the other limits allow) pass the host's checks of shapes."""
    C, P = fa.STATUS_CODES, 4096
    bad = C["FA_ERR_ALIGNMENT"]                          # q, x, k at an odd address: the check behind those of shapes

    def decode(B, H, Hkv):
        need = fa.fa_fwd_decode_paged_fp8_workspace_size(B, H, Hkv, 1, 64)
        return fa.lib.fa_fwd_decode_paged_fp8(P + 2, P, P, P, P, P, P, P, P, B, H, Hkv, 1, 64, 9, 16, 4, 0.1, 0, P, need, None)

    def rope(B, H):
        return fa.lib.fa_rope(P + 2, 2 * P, P, P, 1.0, B, H, 1, 64, 64, 0, 0, H * 64, 64, 64, H * 64, 64, 64, None)

    def append(B, Hkv):
        return fa.lib.fa_cache_append_fp8(P + 2, P, P, P, P, P, P, B, Hkv, 1, 64, 9, 16, None)

    for B, H in ((1024, 64), (1024, 256), (8192, 128), (1, 65535), (65535, 1)):
        assert decode(B, H, H // 4 if H % 4 == 0 else H) == rope(B, H) == append(B, H) == bad, (B, H)
    for B, H in ((8193, 8), (65536, 1), (1, 65536)):
        assert rope(B, H) == append(B, H) == C["FA_ERR_UNSUPPORTED"], (B, H)
        with pytest.raises(fa.FAError, match="unsupported"):
            decode(B, H, H)
