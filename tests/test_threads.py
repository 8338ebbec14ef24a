"""Calls from host threads of the caller's own."""
import ctypes
import dataclasses
import threading

import pytest
import torch

from sparse_attention_decode_paged_gb300 import workloads as W

pytestmark = pytest.mark.gpu


def _in_thread(f):
    """f()'s result in a host thread of its own; what it raises is raised here."""
    got = []

    def run():
        try:
            got.append((f(), None))
        except Exception as e:  # raised by the test's own thread
            got.append((None, e))

    t = threading.Thread(target=run)
    t.start()
    t.join()
    result, error = got[0]
    if error is not None:
        raise error
    return result


@pytest.mark.parametrize("block_rows", [1, 4])
@pytest.mark.parametrize("call", ["step", "dense"])
def test_first_call_of_a_thread(call, block_rows, dsa_lib, cuda_ok):
    """A host thread whose first work on the GPU is a call of this library, with prompt rows (row groups, tiles) and
    without."""
    from sparse_attention_decode_paged_gb300.harness import DeviceStep

    wl = dataclasses.replace(W.workload(1), block_rows=block_rows, max_rows=64 if block_rows > 1 else 8)
    inp = W.generate(wl)
    if block_rows > 1:
        inp["new_tokens"] = inp["new_tokens"].copy()
        inp["new_tokens"][-1] = 40
    step = DeviceStep(inp)
    run = step.step if call == "step" else step.dense
    run()
    torch.cuda.synchronize()
    want = step.outputs.clone()
    step.outputs.zero_()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    _in_thread(lambda: run(stream=stream))
    stream.synchronize()
    assert torch.equal(step.outputs, want) and step.status() == 0


def test_calls_of_two_configs_at_once(dsa_lib, cuda_ok):
    """Two threads, each with a config, a stream and buffers of its own: the kernels they share are launched with
    different amounts of shared memory, and every call gives what it gives alone."""
    from sparse_attention_decode_paged_gb300.harness import DeviceStep

    wide = W.workload(1)
    narrow = dataclasses.replace(wide, num_q_heads=8, num_kv_heads=1, idx_heads=16)
    steps = [DeviceStep(W.generate(wl)) for wl in (wide, narrow)]
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()

    def outputs(step, stream):
        got = []
        for call in (step.step, lambda stream: step.dense(300, 5, stream=stream)):
            call(stream=stream)
            with torch.cuda.stream(stream):
                got.append(step.outputs.clone())
        return got

    want = [outputs(*x) for x in zip(steps, streams)]
    torch.cuda.synchronize()
    ready, failed = threading.Barrier(2), []

    def many(step, stream, want):
        handle = ctypes.c_void_p(stream.cuda_stream)
        cfg, args, ws = ctypes.byref(step.cfg), ctypes.byref(step.args), ctypes.c_void_p(step.workspace.data_ptr())
        try:
            ready.wait()
            for i in range(40):
                # one launch behind the other, with as little as can be between them
                refused = sum(dsa_lib._lib.dsa_step(cfg, args, ws, handle) != 0 for _ in range(200))
                assert refused == 0, (i, refused, dsa_lib._lib.dsa_last_error())
                got = outputs(step, stream)
                stream.synchronize()
                assert all(torch.equal(a, b) for a, b in zip(got, want)), i
        except Exception as e:  # reported by the test's own thread
            failed.append(e)

    threads = [threading.Thread(target=many, args=x) for x in zip(steps, streams, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    assert all(step.status() == 0 for step in steps)
