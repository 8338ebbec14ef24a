"""Device-side plumbing around the C-ABI: upload one step's inputs, build the
rows through the library, hold the outputs and workspace, run or capture a
step.  PyTorch is used here only for device memory, streams and CUDA graphs.
"""
from __future__ import annotations

import contextlib

import numpy as np
import torch

from . import dsa


def to_device(a: np.ndarray | None, device="cuda", kind: str = "raw"):
    """numpy -> CUDA tensor; kind 'bf16' reinterprets uint16 bits as bfloat16."""
    if a is None:
        return None
    a = np.ascontiguousarray(a)
    if kind == "bf16":
        t = torch.from_numpy(a.view(np.int16)).to(device).view(torch.bfloat16)
    else:
        t = torch.from_numpy(a).to(device)
    return t


def on_stream(stream):
    """Context in which torch works on `stream` as the calls here take it: a
    torch stream, a raw handle, or None for the current stream."""
    if stream is None:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream))
    return torch.cuda.stream(stream)


DEVICE_ROW_KEYS = ("row_req", "row_len", "block_first", "block_nrows")


def _arena(parts, device):
    """One byte buffer holding several tensors, each at a 256-byte aligned
    offset: parts = [(name, dtype, shape)] -> (buffer, {name: view})."""
    off, spans = 0, []
    for name, dtype, shape in parts:
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        spans.append((name, dtype, shape, off, n))
        off = (off + n + 255) // 256 * 256
    buf = torch.zeros(max(off, 256), dtype=torch.uint8, device=device)
    return buf, {name: buf[o:o + n].view(dtype).view(*shape) for name, dtype, shape, o, n in spans}


class DeviceStep:
    """All device buffers of one DSA layer-step for a generated workload.

    The per-step inputs that change from step to step (row maps, page table,
    q_idx, w, q) live in one device arena, `inputs`, and the outputs (out,
    lse) in another, `outputs`, so a serving loop moves them with one copy
    each way; t[...] are views into them."""

    def __init__(self, inp: dict, device="cuda", **cfg_override):
        wl = inp["workload"]
        self.inp = inp
        self.cfg = dsa.config_from_workload(wl, inp["num_pages"], **cfg_override)
        dsa.dsa_validate_config(self.cfg)
        self.rows = dsa.dsa_build_rows(self.cfg, inp["cache_len"], inp["new_tokens"])
        R, Hq, D = wl.max_rows, wl.num_q_heads, wl.head_dim
        pt = np.ascontiguousarray(inp["page_table"])
        self.inputs, t = _arena(
            [(k, torch.int32, (R,)) for k in DEVICE_ROW_KEYS]
            + [("page_table", torch.int32, pt.shape),
               ("q_idx", torch.bfloat16, inp["q_idx"].shape),
               ("w", torch.float32, inp["w"].shape),
               ("q", torch.bfloat16, inp["q"].shape)], device)
        for k in DEVICE_ROW_KEYS:
            t[k].copy_(torch.from_numpy(self.rows[k]))
        t["page_table"].copy_(torch.from_numpy(pt))
        for k, kind in (("q_idx", "bf16"), ("w", "raw"), ("q", "bf16")):
            t[k].copy_(to_device(inp[k], device, kind))
        if inp["idx_scale"] is None:
            t["idx_cache"] = to_device(inp["idx_cache"], device, "bf16")
            t["idx_scale"] = None
        else:
            t["idx_cache"] = to_device(inp["idx_cache"], device)
            t["idx_scale"] = to_device(inp["idx_scale"], device)
        t["k_cache"] = to_device(inp["k_cache"], device, "bf16")
        t["v_cache"] = to_device(inp["v_cache"], device, "bf16")
        if self.cfg.flags & dsa.DSA_FLAG_KV_INTERLEAVED:
            # one cache [NP, P, 2, Hkv, D]: each token's K row, then its V row
            kv = torch.stack((t["k_cache"], t["v_cache"]), dim=2).contiguous()
            t["k_cache"], t["v_cache"] = kv, kv[:, :, 1]
        self.outputs, outs = _arena([("out", torch.bfloat16, (R, Hq, D)), ("lse", torch.float32, (R, Hq))], device)
        t.update(outs)
        self.t = t
        self.workspace = dsa.alloc_workspace(self.cfg, device)
        self.views = dsa.workspace_views(self.cfg, self.workspace)
        self.args = dsa.make_step_args(self.cfg, t)
        # filled here, like every other buffer, so that no call's stream has to wait for it
        self.dense_workspace = torch.zeros(dsa.dsa_dense_workspace_size(self.cfg), dtype=torch.uint8,
                                           device=self.workspace.device)

    def step(self, stream=None):
        dsa.dsa_step(self.cfg, self.args, self.workspace, stream)

    def dense(self, window: int = 0, sinks: int = 0, stream=None):
        """The same rows over their whole prefix, or a sliding window with
        sinks, into t["out"] and t["lse"]: a layer that selects no keys."""
        need, have = dsa.dsa_dense_workspace_size(self.cfg), self.dense_workspace.numel()
        if need > have:  # cfg was changed since
            raise ValueError(f"the config needs {need} bytes of dense workspace, the step was made with {have}")
        dsa.dsa_dense_attn(self.cfg, self.t, self.dense_workspace, stream, window=window, sinks=sinks)

    def append(self, k_new, v_new, key_new, stream=None):
        """The step's new K and V [max_rows, Hkv, D] and index keys [max_rows,
        idx_dim] (bf16 tensors; either part may be None) into their pages."""
        dsa.dsa_append(self.cfg, dict(self.t, k_new=k_new, v_new=v_new, key_new=key_new), self.workspace, stream)

    def status(self) -> int:
        """The status bits of step(), append() and dense()."""
        return dsa.dsa_read_device_status(self.workspace) | dsa.dsa_read_device_status(self.dense_workspace)

    def capture(self, stream: torch.cuda.Stream | None = None) -> torch.cuda.CUDAGraph:
        """Warm up once eagerly, then capture one step into a CUDA graph."""
        stream = stream or torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            self.step(stream)
        torch.cuda.current_stream().wait_stream(stream)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            self.step(torch.cuda.current_stream())
        torch.cuda.synchronize()
        return g

    def set_rows(self, cache_len, new_tokens, page_table=None):
        """Rebuild rows on the host and copy them into the static buffers."""
        self.rows = dsa.dsa_build_rows(self.cfg, cache_len, new_tokens)
        for k in ("row_req", "row_len", "block_first", "block_nrows"):
            self.t[k].copy_(torch.from_numpy(self.rows[k]))
        if page_table is not None:
            self.t["page_table"].copy_(torch.from_numpy(np.ascontiguousarray(page_table)))


class PagePool:
    """The page state of a pool (page table, lengths, reference counts) over
    caches [num_pages, ...], and its two changes.  Starts empty; page_table is
    the tensor that a step's calls read."""

    def __init__(self, cfg, caches, device="cuda"):
        self.cfg, self.caches = cfg, list(caches)
        i32 = dict(dtype=torch.int32, device=device)
        B = cfg.max_reqs
        self.page_table = torch.full((B, cfg.max_pages_per_req), -1, **i32)
        self.req_len = torch.zeros(B, **i32)
        self.page_refs = torch.zeros(cfg.num_pages, **i32)
        self.req_from = torch.full((B,), -1, **i32)
        self.req_add = torch.zeros(B, **i32)
        self.num_used = torch.zeros(1, **i32)
        self.workspace = torch.zeros(dsa.dsa_pages_workspace_size(cfg), dtype=torch.uint8, device=device)
        self.args = dsa.make_pages_args(
            cfg, dict(page_table=self.page_table, req_len=self.req_len, page_refs=self.page_refs,
                      req_from=self.req_from, req_add=self.req_add, num_used=self.num_used), self.caches)

    def update(self, req_from=None, req_add=None, stream=None):
        """New slot b continues old slot req_from[b] (-1: none) with room for
        req_add[b] more tokens; int sequences, or None for what the device
        buffers hold.  Everything runs on `stream`: the buffers' new values
        arrive behind the updates queued there, which read the old ones."""
        new = [(buf, self._slots(name, a)) for name, buf, a in
               (("req_from", self.req_from, req_from), ("req_add", self.req_add, req_add)) if a is not None]
        with on_stream(stream):
            for buf, a in new:
                buf.copy_(a)
        dsa.dsa_update_pages(self.cfg, self.args, self.workspace, stream)

    def _slots(self, name, a):
        """One int32 a request slot, from an int sequence."""
        a = np.asarray(a)
        if a.shape != (self.cfg.max_reqs,) or a.dtype.kind not in "iu":
            raise ValueError(f"{name}: expected {self.cfg.max_reqs} ints, one a slot, not {a.dtype} {a.shape}")
        a32 = np.ascontiguousarray(a, dtype=np.int32)
        if not np.array_equal(a32, a):
            raise ValueError(f"{name}: values outside 32 bits")
        return torch.from_numpy(a32)

    def compact(self, stream=None):
        """Moves the live pages to the front of the pool."""
        dsa.dsa_compact_pages(self.cfg, self.args, self.workspace, stream)

    def status(self) -> int:
        return dsa.dsa_read_device_status(self.workspace)
