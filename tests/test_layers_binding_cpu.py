"""The binding of the layers (layers.py, build.py) without a GPU: which arguments it lets
through to the C ABI, and what it does with the compiled calls' answers."""
import pytest
import torch

import chunkwise_gated_delta_gdr_gb300 as gdr
from chunkwise_gated_delta_gdr_gb300 import build as gbuild


@pytest.fixture(scope="module")
def layers():
    gbuild.build()
    from chunkwise_gated_delta_gdr_gb300 import layers as mod
    mod._lib()
    return mod


class Recorder:
    """Stands in for the C library: counts its calls, answers sizes and GDR_OK."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 1024 if name.endswith("_size") else gdr.GDR_OK
        return call


@pytest.fixture
def recorded(layers, monkeypatch):
    """The Python calls on host tensors, up to a C library that only records."""
    lib = Recorder()
    monkeypatch.setattr(layers, "_host", None)
    monkeypatch.setattr(layers, "_lib", lambda: lib)
    monkeypatch.setattr(layers, "_stream", lambda device, stream: 0)
    return lib


# ------------------------------------------------------------------ workspaces
def attn_args():
    k = torch.zeros(5, 16, 2, 64)
    return (torch.zeros(3, 4, 64), k, k, torch.zeros(3, 4, dtype=torch.int32),
            torch.ones(3, dtype=torch.int32))


def test_workspaces_are_checked(layers, recorded):
    """A workspace on another device, or a strided one, never reaches the C ABI."""
    q, k = torch.zeros(2, 3, 4, 64), torch.zeros(2, 3, 2, 64)
    calls = (lambda ws: gdr.paged_decode_attn(*attn_args(), workspace=ws),
             lambda ws: gdr.qk_norm_rope_bwd(q, k, q, k, workspace=ws))
    for call in calls:
        for ws in (torch.empty(4096, dtype=torch.uint8, device="meta"),
                   torch.empty(8192, dtype=torch.uint8)[::2]):
            with pytest.raises(ValueError, match="workspace"):
                call(ws)
        assert not [n for n, _ in recorded.calls if not n.endswith("_size")]
        ws = torch.empty(512, dtype=torch.float32)
        call(ws)
        name, args = recorded.calls.pop()
        assert ws.data_ptr() in args and ws.numel() * 4 in args, name
