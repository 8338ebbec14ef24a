"""harness.PagePool and harness.DeviceStep's calls beside the step: on which
stream their copies and fills run, what they refuse, their status, and their
results on a stream of the caller's."""
import contextlib

import numpy as np
import pytest
import torch

from tests.test_pages import Pool, make_cfg


def _fake_streams(monkeypatch):
    """Records the streams that torch works on, without a GPU: the list of those entered and not left."""
    active = []

    @contextlib.contextmanager
    def stream(s):
        active.append(s)
        yield
        active.pop()

    monkeypatch.setattr(torch.cuda, "stream", stream)
    return active


class _Buffer:
    """Stands for a device buffer: what was copied into it, on which stream."""

    def __init__(self, name, log, active):
        self.name, self.log, self.active = name, log, active
        self.shape = (4,)

    def copy_(self, new):
        self.log.append((self.name, new.tolist(), list(self.active)))


@pytest.fixture
def cpu_pool(dsa_lib, monkeypatch):
    """A PagePool without a GPU: (pool, log of copies and launches)."""
    from sparse_attention_decode_paged_gb300 import harness

    active, log = _fake_streams(monkeypatch), []
    monkeypatch.setattr(dsa_lib, "make_pages_args", lambda cfg, t, caches: None)
    monkeypatch.setattr(dsa_lib, "dsa_update_pages", lambda cfg, args, ws, stream=None: log.append(("update", stream)))
    pool = harness.PagePool(make_cfg(dsa_lib, Pool(4, 4, 12, 16)), [], device="cpu")
    pool.req_from, pool.req_add = _Buffer("from", log, active), _Buffer("add", log, active)
    return pool, log


class _Stream:
    cuda_stream = 1234


def test_update_copies_on_its_stream(cpu_pool):
    """The new values go to the stream that the update runs on, so they come after an update queued there."""
    pool, log = cpu_pool
    s = _Stream()
    pool.update([0, 1, 2, -1], [1, 1, 1, 0], stream=s)
    assert log == [("from", [0, 1, 2, -1], [s]), ("add", [1, 1, 1, 0], [s]), ("update", s)]
    log.clear()
    pool.update([0, 1, 2, 3])  # the current stream, the other buffer as it is
    assert log == [("from", [0, 1, 2, 3], []), ("update", None)]


@pytest.mark.gpu
@pytest.mark.parametrize("handle", [False, True], ids=["stream", "raw handle"])
def test_updates_in_a_row_on_a_busy_stream(handle, dsa_lib, cuda_ok):
    """Updates that follow one another on a stream with work before them, nothing waited for in between."""
    from sparse_attention_decode_paged_gb300 import harness

    want = Pool(8, 6, 60, 16)
    caches = [torch.randint(-2 ** 31, 2 ** 31 - 1, (60, 64), dtype=torch.int32, device="cuda")]
    pool = harness.PagePool(make_cfg(dsa_lib, want), caches)
    expect = caches[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    rng = np.random.default_rng(3)
    for _ in range(12):
        frm = [int(f) for f in rng.integers(-1, 8, 8)]
        add = [min(int(a), 96 - (want.len[f] if f >= 0 else 0)) for a, f in zip(rng.integers(0, 20, 8), frm)]
        with torch.cuda.stream(side):
            torch.cuda._sleep(200000)
        pool.update(frm, add, stream=side.cuda_stream if handle else side)
        for a, b in want.update(frm, add):
            expect[b] = expect[a]
    torch.cuda.synchronize()
    assert np.array_equal(pool.page_table.cpu().numpy(), want.rows())
    assert pool.req_len.tolist() == want.len and pool.page_refs.tolist() == want.refs
    live = torch.tensor(want.refs, device="cuda") > 0
    assert torch.equal(caches[0][live], expect[live]) and pool.status() == 0
