"""CPU model of how the paged decode kernel splits a weight times its V scale for the product with V, over every fp16
value, and the accuracy that include/fa.h states for it."""
import os
import re

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = open(os.path.join(ROOT, "exact_io_aware_55_b200", "csrc", "fa_decode_paged.cu")).read()
HEADER = re.sub(r"\n \* ", " ", open(os.path.join(ROOT, "include", "fa.h")).read())


def f16(bits):
    return np.asarray(bits, np.uint16).view(np.float16)


def parts(h):
    """The value of hi + mid/8 + lo/64 for fp16 values h, each part the upper byte of an fp16 number."""
    up = lambda x: f16((x.view(np.uint16) + np.uint16(0x80)) & np.uint16(0xFF00))  # noqa: E731
    hi = up(h)
    d1 = ((h - hi) * np.float16(8)).astype(np.float16)
    mid = up(d1)
    lo = up(((d1 - mid) * np.float16(8)).astype(np.float16))
    return hi.astype(np.float64) + mid.astype(np.float64) / 8 + lo.astype(np.float64) / 64


def test_the_split_has_the_accuracy_that_the_header_states():
    base = float(re.search(r"kBase = ([\d.]+)f;", SRC).group(1))
    bits_down_to = 2.0 ** -int(re.search(r"has 11 bits down to 2\^-(\d+) of the largest", HEADER).group(1))
    step = 2.0 ** -int(re.search(r"multiples of 2\^-(\d+) of it at the coarsest", HEADER).group(1))
    gone = 2.0 ** -int(re.search(r"under 2\^-(\d+) of it a key may be gone", HEADER).group(1))
    h = f16(np.arange(1, 0x7800 + 1))                   # every value up to 2^15, the largest that P takes
    x, got = h.astype(np.float64), parts(h)
    exact = x >= base * bits_down_to
    assert np.array_equal(got[exact], x[exact]) and not np.array_equal(got[x < base * bits_down_to], x[x < base * bits_down_to])
    off = np.abs(got - x)
    assert np.all(off <= base * step / 2) and np.any(off == base * step / 2)
    assert np.all(got[x < base * gone] == 0) and np.all(got[x >= base * gone] > 0)


def test_negative_parts_do_not_carry_into_the_other_half():
    """Two rows are packed in a word and rounded by one addition: only a value whose magnitude is all ones would carry."""
    h = f16(np.arange(1, 0x7800 + 1))
    for r in (h, ((h - f16((h.view(np.uint16) + np.uint16(0x80)) & np.uint16(0xFF00))) * np.float16(8)).astype(np.float16)):
        assert np.all(r.view(np.uint16).astype(np.uint32) + 0x80 <= 0xFFFF)
