"""dsa_dense_attn's prompt tiles where few inputs take them: maxima that rise
from tile to tile, pages outside the pool, keys that are not finite, the
interleaved cache.  Every call reads enough to be given tiles; the bounds are
test_dense_attn's."""
import numpy as np
import pytest
import torch

from oracle import dsa_oracle as O
from tests.test_dense_attn import HEADS, ONE_TERM, TWO_TERMS, _bf16, _Call, _check, _check_row, _problem

pytestmark = pytest.mark.gpu

NAMES = dict(ids=lambda h: "q%d_kv%d_d%d_p%d" % h)


def _set_keys(pr, b, g, dim, values, first=0):
    """Element `dim` of KV head g's keys of request b, positions first on, on the host and in the cache."""
    bits, exact = _bf16(np.asarray(values, np.float32))
    for i, t in enumerate(range(first, first + len(bits))):
        pr["kb"][pr["table"][b, t // pr["page"]], t % pr["page"], g, dim] = bits[i]
    pr["keys"][b][0][first:first + len(bits), g, dim] = exact


def _set_queries(pr, rows, heads, dim, values):
    bits, exact = _bf16(np.broadcast_to(np.asarray(values, np.float32), pr["q"][rows, heads, dim].shape))
    pr["qb"][rows, heads, dim], pr["q"][rows, heads, dim] = bits, exact


def _rows_of(pr, step):
    """Every step-th row, and each request's first and last."""
    n = len(pr["row_len"])
    ends = np.flatnonzero(np.diff(pr["row_req"]) != 0)
    return sorted({*range(0, n, step), *ends, *(ends + 1), n - 1})


@pytest.mark.parametrize("heads", [HEADS[4], HEADS[9], HEADS[10], HEADS[7]], **NAMES)
def test_maxima_that_rise(heads, dsa_lib, cuda_ok):
    """Keys whose scores rise by 12 and more (log2) at five positions that are no tile's end: the running maximum
    moves and what was summed before is scaled down, inside a CTA's share and across shares."""
    reqs = [(3000, 700), (900, 1), (1025, 1025)]
    pr = _problem(41, *heads, reqs, pad=3, block_rows=4, left=False)
    _set_queries(pr, slice(None), slice(None), 0, 8.0)
    for b, (n, _) in enumerate(reqs):
        stair = np.searchsorted(np.array([0.046, 0.17, 0.37, 0.57, 0.87]) * n, np.arange(n)) * 12.0
        for g in range(pr["hkv"]):
            _set_keys(pr, b, g, 0, stair)
    call = _Call(dsa_lib, pr)
    call.run()
    _check(pr, *call.got(), rows=_rows_of(pr, 29))
    assert call.status() == 0


@pytest.mark.parametrize("heads", [HEADS[4], HEADS[8]], **NAMES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (700, 9)])
def test_sharp_scores(heads, window, sinks, dsa_lib, cuda_ok):
    """Scores in the hundreds: a few keys have all the weight, and maxima move often."""
    pr = _problem(42, *heads, [(2500, 900), (77, 77)], pad=2, window=window, sinks=sinks, block_rows=4, scale_q=30.0,
                  left=False)
    call = _Call(dsa_lib, pr)
    call.run()
    _check(pr, *call.got(), rows=_rows_of(pr, 23))
    assert call.status() == 0


@pytest.mark.parametrize("heads", [(16, 2, 128, 16), (64, 8, 128, 64), (12, 4, 64, 128), (18, 3, 64, 32)], **NAMES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (500, 20)])
def test_bad_pages_in_tiles(heads, window, sinks, dsa_lib, cuda_ok):
    """Pages outside the pool, missing ones, first, last and side by side: flagged, left out by the rows that see
    them, and no other row's concern."""
    page = heads[3]
    pr = _problem(43, *heads, [(2000, 900), (600, 1)], pad=4, window=window, sinks=sinks, block_rows=4, left=False)
    bad = {0: pr["pool"], 900 // page: -1, 1500 // page: -7, 1500 // page + 1: 2 ** 31 - 1, 1999 // page: pr["pool"] + 5}
    call = _Call(dsa_lib, pr)
    for i, pg in bad.items():
        call.t["page_table"][0, i] = pg
    call.run()
    out, lse = call.got()
    assert call.status() == dsa_lib.DSA_DEV_BAD_PAGE
    gone = np.concatenate([np.arange(i * page, (i + 1) * page) for i in bad])
    for r in [*range(0, 900, 17), 399, 400, 401, 899]:
        n = int(pr["row_len"][r])
        k, v = pr["keys"][0]
        t = np.setdiff1d(O.visible_positions(n, window, sinks), gone)
        _check_row(out[r], lse[r], *O.dense_row(pr["q"][r], k[t], v[t], pr["d"] ** -0.5, pr["hkv"]), n, ONE_TERM, (r, n))
    _check(pr, out, lse, rows=range(900, 905), terms=TWO_TERMS)


@pytest.mark.parametrize("heads", [(16, 2, 128, 32), (12, 2, 64, 64)], **NAMES)
def test_keys_that_are_not_finite_in_tiles(heads, dsa_lib, cuda_ok):
    """An infinite key makes the heads that score it +inf NaN, from the row that sees it on, and has no weight where
    its score is -inf; a NaN key makes every head of its KV head NaN; rows all of whose scores are -inf are empty."""
    hq, G, d = heads[0], heads[0] // 2, heads[2]
    pr = _problem(44, *heads, [(1400, 900), (700, 700)], pad=3, block_rows=4, left=False)
    plus, minus, other = list(range(G // 2)), list(range(G // 2, G)), list(range(G, hq))
    _set_queries(pr, slice(None), slice(0, G // 2), 0, 1.0)
    _set_queries(pr, slice(None), slice(G // 2, G), 0, -1.0)
    _set_keys(pr, 0, 0, 0, [np.inf], 950)
    _set_keys(pr, 0, 1, 3, [np.nan], 1100)
    _set_queries(pr, slice(900, 1600), slice(0, G), 5, 1.0)
    _set_keys(pr, 1, 0, 5, np.full(700, -np.inf))
    call = _Call(dsa_lib, pr)
    call.run()
    out, lse = call.got()

    def check(r, some, k, v):
        # the heads `some` on their own: the oracle over their KV head alone
        g = some[0] // G
        want = O.dense_row(pr["q"][r, some], k[:, g:g + 1], v[:, g:g + 1], d ** -0.5, 1)
        _check_row(out[r, some], lse[r, some], *want, len(k), ONE_TERM, (r, some))

    k, v = pr["keys"][0]
    for r in [*range(0, 900, 31), 450, 451, 600, 601, 899]:
        n = int(pr["row_len"][r])
        fine = np.setdiff1d(np.arange(n), [950])
        check(r, minus, k[fine], v[fine])
        if n > 950:
            assert np.isnan(out[r, plus]).all() and not np.isfinite(lse[r, plus]).any(), r
        else:
            check(r, plus, k[:n], v[:n])
        if n > 1100:
            assert np.isnan(out[r, other]).all() and np.isnan(lse[r, other]).all(), r
        else:
            check(r, other, k[:n], v[:n])
    k, v = pr["keys"][1]
    for r in [*range(900, 1600, 37), 1599]:
        n = int(pr["row_len"][r])
        assert not out[r, :G].any() and np.all(lse[r, :G] == -np.inf), r
        check(r, other, k[:n], v[:n])
    assert not out[1600:].any() and np.all(lse[1600:] == -np.inf)
    assert call.status() == 0


@pytest.mark.parametrize("heads", [HEADS[2], HEADS[3], HEADS[4], HEADS[9]], **NAMES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (500, 20), (100, 300)])
def test_tiles_on_the_interleaved_cache(heads, window, sinks, dsa_lib, cuda_ok):
    """Prompts of many tiles beside single tokens, K and V of a token side by side in one cache: the bits that the
    separate caches give."""
    pr = _problem(45, *heads, [(2600, 800), (3000, 1), (700, 700)], pad=5, window=window, sinks=sinks, block_rows=4,
                  left=False)
    apart, call = _Call(dsa_lib, pr), _Call(dsa_lib, pr, interleaved=True)
    call.run()
    apart.run()
    out, lse = call.got()
    _check(pr, out, lse, rows=_rows_of(pr, 41))
    assert torch.equal(call.t["out"].view(torch.int16), apart.t["out"].view(torch.int16))
    assert torch.equal(call.t["lse"], apart.t["lse"])
    assert call.status() == apart.status() == 0
