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


@pytest.mark.parametrize("bad", [[1], [[0, 0, 0, 0]], 0, [0] * 5, [0.5] * 4, [True] * 4,
                                 np.array([0, 0, 0, 2 ** 32])], ids=repr)
@pytest.mark.parametrize("name", ["req_from", "req_add"])
def test_update_refuses_what_is_not_an_int_a_slot(name, bad, cpu_pool):
    """One value would be spread over all slots, a fraction or a long int cut: nothing is copied or launched."""
    pool, log = cpu_pool
    with pytest.raises(ValueError, match=name):
        pool.update(**{"req_from": [0, 1, 2, 3], "req_add": [0, 0, 0, 0], name: bad})
    assert log == []


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


# ----------------------------------------------------------------------------
# DeviceStep.dense and DeviceStep.append
# ----------------------------------------------------------------------------
@pytest.fixture
def cpu_step(dsa_lib, monkeypatch):
    """A DeviceStep without a GPU: (step, log of dense calls)."""
    from sparse_attention_decode_paged_gb300 import harness, workloads

    log = []
    monkeypatch.setattr(dsa_lib, "make_step_args", lambda cfg, t: None)
    monkeypatch.setattr(dsa_lib, "dsa_dense_attn", lambda cfg, args, ws, stream=None, window=0, sinks=0:
                        log.append((ws, stream, window, sinks)))
    return harness.DeviceStep(workloads.generate(1), device="cpu"), log


def test_dense_workspace_is_there_before_the_call(cpu_step, dsa_lib, monkeypatch):
    """Nothing is allocated or filled while dense() runs: a fill would be on another stream than the call."""
    step, log = cpu_step

    def refuse(*a, **kw):
        raise AssertionError("a fill inside the call")

    monkeypatch.setattr(torch, "zeros", refuse)
    s = _Stream()
    step.dense(7, 2, stream=s)
    (ws, stream, window, sinks), = log
    assert ws.numel() == dsa_lib.dsa_dense_workspace_size(step.cfg) and not ws.any()
    assert stream is s and (window, sinks) == (7, 2)


def test_status_holds_what_dense_flagged(cpu_step, dsa_lib, monkeypatch):
    step, _ = cpu_step
    monkeypatch.setattr(dsa_lib, "dsa_read_device_status", lambda ws, stream=None: int(ws[:4].view(torch.int32)))
    assert step.status() == 0
    step.dense_workspace[0] = dsa_lib.DSA_DEV_BAD_PAGE
    assert step.status() == dsa_lib.DSA_DEV_BAD_PAGE
    step.workspace[0] = dsa_lib.DSA_DEV_BAD_ROW
    assert step.status() == dsa_lib.DSA_DEV_BAD_PAGE | dsa_lib.DSA_DEV_BAD_ROW


def test_dense_of_a_config_that_outgrew_its_workspace_is_refused(cpu_step, dsa_lib):
    step, log = cpu_step
    step.cfg.flags |= dsa_lib.DSA_FLAG_NO_PREFILL_GROUPS
    step.dense()
    step.cfg.flags &= ~dsa_lib.DSA_FLAG_NO_PREFILL_GROUPS
    step.cfg.block_rows = 4  # prompt tiles from now on
    with pytest.raises(ValueError, match="dense workspace"):
        step.dense()
    assert len(log) == 1


def _dense_rows_match(step, window, sinks, rows=None):
    """step.t's outputs against the oracle on the workload's caches, at test_dense_attn's bound."""
    from oracle import dsa_oracle as O
    from tests.test_dense_attn import ONE_TERM, _check_row

    torch.cuda.synchronize()
    cfg, t = step.cfg, step.t
    out, lse = t["out"].double().cpu().numpy(), t["lse"].double().cpu().numpy()
    q, k, v = (t[n].double().cpu().numpy() for n in ("q", "k_cache", "v_cache"))
    table = t["page_table"].cpu().numpy()
    for r in rows if rows is not None else range(step.rows["num_rows"]):
        n, b = int(step.rows["row_len"][r]), int(step.rows["row_req"][r])
        pages = table[b, :-(-n // cfg.page_size)]
        kr, vr = (c[pages].reshape(-1, *c.shape[2:])[:n] for c in (k, v))
        _check_row(out[r], lse[r], *O.dense_row(q[r], kr, vr, cfg.sm_scale, cfg.num_kv_heads, window, sinks), n,
                   ONE_TERM, r)
    pad = step.rows["num_rows"]
    assert not out[pad:].any() and np.all(lse[pad:] == -np.inf)


@pytest.mark.gpu
def test_dense_on_a_side_stream(dsa_lib, cuda_ok):
    """The first call of a step's dense layer on a stream of the caller's, while the current stream is busy."""
    from sparse_attention_decode_paged_gb300 import harness, workloads

    step = harness.DeviceStep(workloads.generate(1))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(20000000)  # about 10 ms: what the call put on the current stream would come late
    step.dense(100, 3, stream=side)
    side.synchronize()
    _dense_rows_match(step, 100, 3)
    step.dense()
    _dense_rows_match(step, 0, 0)
    assert step.status() == 0
    step.t["page_table"][0, 0] = step.cfg.num_pages
    step.dense()
    assert step.status() == dsa_lib.DSA_DEV_BAD_PAGE


@pytest.mark.gpu
def test_append_of_a_step(dsa_lib, cuda_ok):
    """A step's own rows appended: the caches hold the new tokens at the rows' positions, and dense() reads them."""
    from sparse_attention_decode_paged_gb300 import harness, workloads

    step = harness.DeviceStep(workloads.generate(1))
    cfg, t = step.cfg, step.t
    gen = torch.Generator(device="cuda").manual_seed(5)
    k, v, key = (torch.randn(cfg.max_rows, *s, generator=gen, dtype=torch.bfloat16, device="cuda")
                 for s in ((cfg.num_kv_heads, cfg.head_dim), (cfg.num_kv_heads, cfg.head_dim), (cfg.idx_dim,)))
    was = t["idx_cache"].clone()
    step.append(k, v, None)
    torch.cuda.synchronize()
    assert torch.equal(t["idx_cache"].view(torch.int16), was.view(torch.int16))  # index keys left alone
    step.append(k, v, key)
    step.dense()
    n = step.rows["num_rows"]
    at = torch.from_numpy(step.rows["row_len"][:n].astype(np.int64)).cuda() - 1
    req = torch.from_numpy(step.rows["row_req"][:n].astype(np.int64)).cuda()
    pg = t["page_table"][req, at // cfg.page_size].long()
    for cache, new in (("k_cache", k), ("v_cache", v), ("idx_cache", key)):
        assert torch.equal(t[cache][pg, at % cfg.page_size].view(torch.int16), new[:n].view(torch.int16)), cache
    _dense_rows_match(step, 0, 0)
    assert step.status() == 0


@pytest.mark.parametrize("kw", [dict(window=5), dict(sinks=2)], ids=repr)
def test_packed_dense_args_fix_the_window(kw, dsa_lib):
    """A window beside packed arguments would be passed over."""
    with pytest.raises(ValueError, match="make_dense_args"):
        dsa_lib.dsa_dense_attn(make_cfg(dsa_lib, Pool(4, 4, 12, 16)), dsa_lib.dsa_dense_args_t(), None, **kw)


class _OnGpu(torch.Tensor):
    """Passes for a CUDA tensor where only that and its size are asked for."""

    is_cuda = True


@pytest.mark.parametrize("short", [0, 1, 16], ids=lambda n: f"{n} short")
@pytest.mark.parametrize("call", ["dsa_dense_attn", "dsa_update_pages", "dsa_compact_pages"])
def test_workspace_too_small_is_refused(call, short, dsa_lib):
    """A workspace of another call (or config) is smaller than what the kernels write."""
    cfg = make_cfg(dsa_lib, Pool(40, 40, 120, 16), rows=64, block_rows=4)
    dense = call == "dsa_dense_attn"
    need = (dsa_lib.dsa_dense_workspace_size if dense else dsa_lib.dsa_pages_workspace_size)(cfg)
    args = dsa_lib.dsa_dense_args_t() if dense else dsa_lib.dsa_pages_args_t()
    ws = torch.zeros(need - short, dtype=torch.uint8).as_subclass(_OnGpu)
    # the arguments are empty: what is refused first tells how far the call came
    with pytest.raises(ValueError if short else dsa_lib.DsaError, match="workspace" if short else "page_table"):
        getattr(dsa_lib, call)(cfg, args, ws, stream=0)
