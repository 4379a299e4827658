"""mtp_heads_attn with a window over a table whose hidden pages are gone: entries that no visible
position needs are not read, whatever they hold (-1, as the page calls leave what is given back, or
the number of a page that is now another row's)."""
import pytest
import torch

import verify_spec_greedy_gb300 as lib
from heads_reference import Batch

pytestmark = pytest.mark.gpu
BF, F16 = torch.bfloat16, torch.float16

# rows whose windows start inside a key tile and inside a page, with one query and with several,
# with units that start at different keys, and a row without queries (which needs no page at all)
ROWS = [(1, 1000), (3, 1301), (1, 64), (200, 900), (0, 300), (5, 517), (1, 2049)]


def hidden_entries(x, window, sinks):
    """(row, entry) of the pages below the rows' lengths of which no query sees a position."""
    gone = []
    for b, (n, length) in enumerate(x.rows):
        first = max(0, length - n - window + 1)  # the first query's window
        for e in range(-(-length // x.P)):
            lo, hi = e * x.P, min((e + 1) * x.P, length)
            if n == 0 or (lo >= sinks and hi <= first):
                gone.append((b, e))
    return gone


@pytest.mark.parametrize("entry", ["given back", "another's"])
@pytest.mark.parametrize("window,sinks", [(100, 4), (37, 0), (128, 130), (300, 1), (1, 77), (257, 16)])
@pytest.mark.parametrize("Hq,Hkv,D,P,dtype,tokens", [
    (8, 2, 64, 16, F16, 3), (4, 4, 48, 8, BF, 3), (16, 2, 64, 48, BF, 3),             # units of 32 rows
    (8, 2, 64, 16, BF, 200), (8, 2, 128, 16, BF, 200), (6, 1, 128, 48, F16, 200),     # of 128 rows
    (8, 2, 256, 8, F16, 200), (5, 1, 144, 40, BF, 200), (4, 2, 128, 256, BF, 200)])
def test_pages_that_no_query_sees_are_not_read(Hq, Hkv, D, P, dtype, tokens, window, sinks, entry):
    rows = [r for r in ROWS if r[0] <= tokens]
    x = Batch(rows, Hq, Hkv, D, P, dtype, seed=window + D, spare=3)
    gone = hidden_entries(x, window, sinks)
    assert len(gone) > 3
    nan_page = sorted(set(range(x.k.shape[0])) - set(x.table[x.table >= 0].tolist()))[0]
    assert x.k[nan_page].isnan().all() and x.v[nan_page].isnan().all()
    for b, e in gone:
        x.table[b, e] = -1 if entry == "given back" else nan_page
    x.run(lib, window, sinks)
    x.check(window, sinks, heads=sorted({0, Hq - 1}))
