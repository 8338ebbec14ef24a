"""Calls from host threads of the caller's own."""
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
