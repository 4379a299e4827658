"""Page ids out of range in a block table: mtp_pages_resize passes them over and reports them, both
where a page is given back and where a row goes on in a partly filled one."""
import pytest
import torch

import verify_spec_greedy_gb300 as lib
from pages_reference import Pages
from test_gpu_pages import I32, Device, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [3, 1500])
@pytest.mark.parametrize("bad", [-1, 40_000, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("entry,keep", [(1, 12), (2, 16), (2, 3), (1, 9)])
def test_resize_reports_a_page_id_out_of_range(B, bad, entry, keep):
    m = Pages(B, 5, 4 * B + 4, 8)
    m.take(0, 3)
    m.take(B - 1, 3)
    d = Device(m)
    d.table[B - 1, entry] = bad
    lens = [20] + [0] * (B - 2) + [keep]
    d.status.zero_()
    lib.mtp_pages_resize(dev([20] + [0] * (B - 2) + [keep]), dev(lens), d.table, d.held, d.refs, 8, d.copies,
                         status=d.status)
    assert int(d.status) == lib.STATUS_BAD_PARAM
    # the pages of good ids follow as ever, the one that the table lost stays, and nothing is copied
    kept = -(-keep // 8)
    refs = torch.zeros(4 * B + 4, dtype=I32, device="cuda")
    refs[:3] = refs[3 + entry] = 1
    for i in range(kept):
        if i != entry:
            refs[3 + i] = 1
    assert torch.equal(d.refs, refs) and int(d.held[B - 1]) == kept and (d.copies == -1).all()
    want = [3 + i if i != entry else bad for i in range(kept)] + [-1] * (5 - kept)
    assert d.table[B - 1].tolist() == want


def test_a_partly_filled_page_that_is_not_written_into_is_not_looked_at():
    m = Pages(2, 4, 10, 8)
    m.take(0, 2)
    d = Device(m)
    d.table[0, 1] = -1
    for keep, copies in ((16, d.copies), (12, None), (-1, d.copies)):
        d.status.zero_()
        lib.mtp_pages_resize(dev([keep, 0]), dev([max(keep, 0), 0]), d.table, d.held, d.refs, 8, copies,
                             status=d.status)
        assert int(d.status) == 0 and d.table[0].tolist() == [0, -1, -1, -1]
