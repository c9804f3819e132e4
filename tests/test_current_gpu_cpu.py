"""Calls on tensors of a GPU that is not the current one, on the CPU: a default stream's handle is 0 on every GPU, and
the library launches on the current one, so each call has to make the tensors' GPU current for as long as it lasts.
The tensors and the library are stand-ins; nothing is launched."""
import os

import pytest
import torch

from moe_routed_expert_amd import binding, routed
from tests.test_routed_abi_cpu import TENSORS, Tensor

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
EPILOGUES = {
    "swiglu_clamped_fwd": ([((6, 16), BF16), ((6,), F32), ((6, 8), BF16)], {3: 7.0}),
    "swiglu_clamped_bwd": ([((6, 16), BF16), ((6,), F32), ((6, 8), BF16), ((6, 16), BF16), ((6,), F32)], {5: 7.0}),
    "router_weight_mul_fwd": ([((6, 16), BF16), ((6,), F32), ((6, 16), BF16)], {}),
    "router_weight_mul_bwd": ([((6, 16), BF16), ((6, 16), BF16), ((6,), F32), ((6, 16), BF16), ((6,), F32)], {}),
    "grouped_gate_up_swiglu_fwd": ([((6, 16), BF16), ((2, 8, 16), BF16), ((2, 8, 16), BF16), ((2,), I32), ((6,), F32),
                                    ((6, 8), BF16), ((6, 16), BF16)], {7: 7.0}),
    "grouped_down_router_fwd": ([((6, 16), BF16), ((2, 8, 16), BF16), ((2,), I32), ((6,), F32), ((6, 8), BF16)], {}),
    "moe_combine_fwd": ([((6, 16), BF16), ((3, 2), I32), ((3, 16), F32)], {}),
}
CALLS = {name: (binding, *spec) for name, spec in EPILOGUES.items()}
CALLS |= {name: (routed, *spec) for name, spec in TENSORS.items()}
# the older calls have a form for each set of types
CALLS["swiglu_clamped_fwd, float32"] = (binding, [(s, F32) for s, _ in EPILOGUES["swiglu_clamped_fwd"][0]], {3: 7.0})
CALLS["router_weight_mul_fwd, float32"] = (binding, [(s, F32) for s, _ in EPILOGUES["router_weight_mul_fwd"][0]], {})
CALLS["swiglu_clamped_bwd, float32"] = (binding, [(s, F32) for s, _ in EPILOGUES["swiglu_clamped_bwd"][0]], {5: 7.0})
CALLS["router_weight_mul_bwd, float32"] = (binding, [(s, F32) for s, _ in EPILOGUES["router_weight_mul_bwd"][0]], {})


class Stream:
    """A torch stream; a default one has handle 0 whichever GPU it is on."""

    def __init__(self, device_index, handle=0):
        self.device_index, self.cuda_stream = device_index, handle


@pytest.fixture
def gpus(monkeypatch):
    """Two GPUs, of which 0 is current; .calls lists the current GPU and the stream's handle of each call."""
    class Gpus:
        def __init__(self):
            self.current, self.calls, self.status = 0, [], 0

    g = Gpus()

    class device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, g.current = g.current, self.index

        def __exit__(self, *exc):
            g.current = self.before

    class Library:
        def __getattr__(self, call):
            return lambda *args: g.calls.append((g.current, args[-1])) or g.status

        def moe_epi_status_string(self, status):
            return b"refused"

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: g.current)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: Stream(getattr(d, "index", d)))
    monkeypatch.setattr(binding, "_lib", Library())
    monkeypatch.setattr(binding, "_several_gpus", True, raising=False)
    monkeypatch.setattr(routed, "_fns", Library())
    monkeypatch.setattr(routed, "_raw_stream", lambda index: 0)
    return g


def call(name, index, **kw):
    module, specs, others = CALLS[name]
    args = [Tensor(*s, device=index) for s in specs]
    for at in sorted(others):
        args.insert(at, others[at])
    getattr(module, name.split(",")[0])(*args, **kw)


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("index", [0, 1])
def test_the_tensors_gpu_is_current_during_the_call(gpus, name, index):
    call(name, index)
    assert gpus.calls == [(index, 0)] and gpus.current == 0
    gpus.status = 5                                # the current GPU is put back after an error too
    with pytest.raises(binding.MoeEpiError):
        call(name, index)
    assert gpus.current == 0 and gpus.calls[-1] == (index, 0)


@pytest.mark.parametrize("name", sorted(CALLS))
def test_a_stream_of_another_gpu_is_refused(gpus, name):
    with pytest.raises(ValueError, match="GPU 0.*GPU 1"):
        call(name, 1, stream=Stream(0, 64))
    assert gpus.calls == []
    call(name, 1, stream=Stream(1, 64))
    call(name, 1, stream=128)                      # a handle is taken as it is
    assert gpus.calls == [(1, 64), (1, 128)]


@pytest.mark.parametrize("count", [0, 1, 2, 8])
def test_the_library_is_loaded_with_the_number_of_gpus_seen(count, monkeypatch):
    if not os.path.exists(binding.LIB_PATH):
        pytest.skip("the library is not built")
    monkeypatch.setattr(torch.cuda, "device_count", lambda: count)
    monkeypatch.setattr(binding, "_lib", None)
    monkeypatch.setattr(binding, "_several_gpus", None)
    binding.lib()
    assert binding._several_gpus is (count > 1)
