"""The step's single calls right behind dsa_update_pages and
dsa_compact_pages, with nothing waited for in between: they see the page table
and lengths that those write."""
import numpy as np
import pytest
import torch

from tests.test_pages import Pool, make_cfg

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")
PAGE, D = 16, 128


class _State:
    """A device page state as a Pool's, and its update and compaction by device buffers."""

    def __init__(self, dsa, pool, cfg, caches):
        self.dsa, self.cfg, self.caches = dsa, cfg, caches
        self.t = dict(page_table=torch.tensor(pool.rows(), **I32), req_len=torch.tensor(pool.len, **I32),
                      page_refs=torch.tensor(pool.refs, **I32))
        self.ws = torch.zeros(dsa.dsa_pages_workspace_size(cfg), dtype=torch.uint8, device="cuda")
        self.keep = []

    def args(self, frm, add):
        t = dict(self.t, req_from=torch.tensor(frm, **I32), req_add=torch.tensor(add, **I32))
        self.keep.append(t)
        return self.dsa.make_pages_args(self.cfg, t, self.caches)

    def update(self, args):
        self.dsa.dsa_update_pages(self.cfg, args, self.ws)

    def compact(self, args):
        self.dsa.dsa_compact_pages(self.cfg, args, self.ws)


def _kv(pages, hkv, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(pages, PAGE, hkv, D, generator=g, dtype=torch.bfloat16, device="cuda") for _ in range(2)]


def _parts(cfg):
    shape = (cfg.max_rows, cfg.num_q_heads, cfg.num_splits)
    return [torch.full(s, 7.0, device="cuda") for s in (shape, shape, (*shape, D))]


@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
@pytest.mark.parametrize("groups", [True, False], ids=["groups", "rows"])
def test_attention_of_a_request_that_moved(groups, graph, dsa_lib, cuda_ok):
    """A request goes back and forth between two slots, whose table rows are -1 while it is away; each time its 16
    rows attend over one and the same selection, to the same bits."""
    pool = Pool(3, 8, 64, PAGE)
    pool.update([-1] * 3, [0, 0, 128])
    pool.update([-1, -1, 2], [100, 0, 0])
    cfg = make_cfg(dsa_lib, pool, rows=16, num_q_heads=8, num_kv_heads=1, head_dim=D, topk=32, num_splits=2,
                   block_rows=4, flags=0 if groups else dsa_lib.DSA_FLAG_NO_PREFILL_GROUPS)
    k, v = _kv(64, 1, 1)
    st = _State(dsa_lib, pool, cfg, [k, v])
    q = torch.randn(16, 8, D, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(2)
    idx = torch.tensor(np.array([np.sort(rng.permutation(85)[:32]) for _ in range(16)]), **I32)
    row_len = torch.arange(85, 101, **I32)
    row_req = [torch.full((16,), b, **I32) for b in range(2)]
    ws = dsa_lib.alloc_workspace(cfg)

    def attend(b, parts):
        dsa_lib.dsa_sparse_attn(cfg, q, k, v, st.t["page_table"], row_req[b], row_len, idx, *parts, ws)

    want = _parts(cfg)
    attend(0, want)
    torch.cuda.synchronize()
    there, back = st.args([-1, 0, 2], [0] * 3), st.args([1, -1, 2], [0] * 3)
    parts = [_parts(cfg) for _ in range(21)]

    def sequence():
        for i in range(20):
            st.update(back if i % 2 else there)
            attend((i + 1) % 2, parts[i])
        st.update(st.args_drop)  # slot 2 leaves, its pages are taken by slot 0's
        st.compact(there)
        attend(0, parts[20])

    st.args_drop = st.args([0, -1, -1], [0] * 3)
    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sequence()
        g.replay()
    else:
        sequence()
    torch.cuda.synchronize()
    for got in parts:
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert dsa_lib.dsa_read_device_status(ws) == dsa_lib.dsa_read_device_status(st.ws) == 0
    assert st.t["page_table"][0, :7].tolist() == list(range(7))


def test_calls_on_lengths_that_just_grew(dsa_lib, cuda_ok):
    """One row a request whose length is the pool's own: each update adds a token, the top-k selects it and the
    attention takes it in."""
    n, steps = 8, 40
    pool = Pool(n, 8, 96, PAGE)
    start = [3 + 11 * b for b in range(n)]
    pool.update([-1] * n, start)
    cfg = make_cfg(dsa_lib, pool, rows=n, num_q_heads=8, num_kv_heads=1, head_dim=D, topk=128, num_splits=2)
    k, v = _kv(96, 1, 3)
    st = _State(dsa_lib, pool, cfg, [k, v])
    grow = st.args(list(range(n)), [1] * n)
    rows = torch.arange(n, **I32)
    q = torch.randn(n, 8, D, dtype=torch.bfloat16, device="cuda")
    scores = torch.randn(n, 128, device="cuda")
    idx = [torch.full((n, 128), -7, **I32) for _ in range(steps)]
    given = [torch.tensor([[*range(s + i + 1)] + [-1] * (127 - s - i) for s in start], **I32) for i in range(steps)]
    parts = [_parts(cfg) for _ in range(2)]
    ws = dsa_lib.alloc_workspace(cfg)

    def attend(sel, to):
        dsa_lib.dsa_sparse_attn(cfg, q, k, v, st.t["page_table"], rows, st.t["req_len"], sel, *to, ws)

    for i in range(steps):
        st.update(grow)
        if i % 2:  # a selection from before: the attention follows the update itself
            attend(given[i], parts[0])
            dsa_lib.dsa_topk(cfg, scores, st.t["req_len"], idx[i], ws)
        else:
            dsa_lib.dsa_topk(cfg, scores, st.t["req_len"], idx[i], ws)
            attend(idx[i], parts[0])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(idx, given))
    attend(given[-1], parts[1])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*parts))
    assert dsa_lib.dsa_read_device_status(ws) == dsa_lib.dsa_read_device_status(st.ws) == 0
    assert st.t["req_len"].tolist() == [s + steps for s in start]
