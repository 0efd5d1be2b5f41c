"""GPU tests of edges of the calls on the 8-bit paged cache.  Tolerances as in tests/test_gpu_paged.py, whose
helpers these tests use; what they add to them is derived beside each."""
import numpy as np
import pytest
import torch

from oracle import paged
from tests import gpu_util as gu
from tests.test_gpu_paged import bf16, cache, check_append, check_decode, decode_case, fa, i32

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
