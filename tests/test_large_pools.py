"""dsa_update_pages and dsa_compact_pages on page tables and pools larger than
what a plan's threads load ahead (32768 table entries, 32768 pages), and on
more slots than its shared memory holds, bit for bit against the list model."""
import numpy as np
import pytest

from tests.test_pages import Device, Pool

pytestmark = pytest.mark.gpu


# slots, table width, pages; the last page of the pool is no whole group of 32
@pytest.mark.parametrize("slots,width,pages", [(300, 200, 20011), (40, 1500, 50003), (1300, 30, 33007)])
def test_steps_on_large_pools(slots, width, pages, dsa_lib, cuda_ok):
    rng = np.random.default_rng(slots)
    page = 16
    pool = Pool(slots, width, pages, page)
    dev = Device(dsa_lib, pool, words=(4,))
    share = min(width, pages // slots) * page
    moved = 0
    for step in range(6):
        before = [c.clone() for c in dev.caches]
        if step % 3 == 2:
            moves = pool.compact()
            dev.compact()
            moved += len(moves)
            dev.check(pool, before, moves, live_only=True)
            continue
        if step % 3 == 0:  # half stay, the others start anew, move or fork; long and short ones beside one another
            frm = [b if rng.random() < 0.5 else int(rng.integers(-1, slots)) for b in range(slots)]
            grow = rng.integers(0, share, slots) * (rng.random(slots) < 0.9)
        else:  # a third leave
            frm = [b if rng.random() < 0.67 else -1 for b in range(slots)]
            grow = rng.integers(0, 3, slots)
        have = [pool.len[f] if f >= 0 else 0 for f in frm]
        add = [int(min(a, max(0, share - n))) for a, n in zip(grow, have)]
        moves = pool.update(frm, add)
        dev.update(frm, add)
        assert moves is not None
        dev.check(pool, before, moves)
    assert dev.status() == 0
    assert moved > 1000 and sum(c > 0 for c in pool.refs) > pages // 5
