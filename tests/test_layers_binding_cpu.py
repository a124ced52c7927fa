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


# ------------------------------------------------------------------ the compiled calls' answers
class Compiled:
    """Stands in for the compiled module: every call answers `value`."""

    def __init__(self, value):
        self.value, self.count = value, 0

    def __getattr__(self, name):
        def call(*args):
            self.count += 1
            return self.value
        return call


def every_call():
    x, q = torch.zeros(1, 4, 8), torch.zeros(2, 3, 4, 64)
    k = torch.zeros(5, 16, 4, 64)
    pos, table = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32)
    return {"linear_scan_fwd": lambda: gdr.linear_scan_fwd(x, x),
            "linear_scan_bwd": lambda: gdr.linear_scan_bwd(x, x, x, gdr.linear_scan_checkpoints(x)),
            "qk_norm_rope": lambda: gdr.qk_norm_rope(q, q),
            "qk_norm_rope_bwd": lambda: gdr.qk_norm_rope_bwd(q, q, q, q),
            "qk_norm_rope_append": lambda: gdr.qk_norm_rope_append(
                q, q, q, None, None, None, None, pos, k, k, table),
            "paged_decode_attn": lambda: gdr.paged_decode_attn(*attn_args())}


@pytest.mark.parametrize("name", list(every_call()))
def test_a_call_that_was_made_is_not_made_again(layers, recorded, monkeypatch, name):
    """The compiled call answers a status: an error, and no second call. It answers None:
    the Python call is made, once."""
    call = every_call()[name]
    for status in (gdr.GDR_ERR_CUDA, gdr.GDR_ERR_INVALID_ARG):
        host = Compiled(status)
        monkeypatch.setattr(layers, "_host", host)
        with pytest.raises(gdr.GdrError, match="gdr_" + name) as error:
            call()
        assert error.value.status == status
        assert host.count == 1 and not recorded.calls
    monkeypatch.setattr(layers, "_host", Compiled(None))
    call()
    assert [n for n, _ in recorded.calls if not n.endswith("_size")] == ["gdr_" + name]


# ------------------------------------------------------------------ the compiled module and torch
def test_compiled_module_is_named_after_its_torch(layers):
    assert gbuild._host_target() == gbuild.host_path(torch.__version__)
    assert gbuild.host_path("1.2.3") != gbuild.host_path("1.2.4")
    assert layers._host is None or layers._host.__file__ == gbuild.host_path(torch.__version__)


def test_another_torch_is_not_up_to_date(layers, monkeypatch, tmp_path):
    (tmp_path / "version.py").write_text("__version__ = '0.0.1'\n")
    monkeypatch.setattr(gbuild, "_torch_dir", lambda: str(tmp_path))
    assert gbuild._host_target() == gbuild.host_path("0.0.1")
    assert not gbuild.up_to_date()


def test_module_that_is_missing_or_broken_leaves_the_python_calls(layers, tmp_path):
    with pytest.warns(UserWarning, match="not built"):
        assert layers._load_host(gbuild.host_path("0.0.1")) is None
    broken = tmp_path / "_layers_host.so"
    broken.write_bytes(b"no module")
    with pytest.warns(UserWarning, match="from Python"):
        assert layers._load_host(str(broken)) is None


@pytest.mark.parametrize("error", [FileNotFoundError("g++"), RuntimeError("g++ failed")])
def test_library_builds_without_the_compiled_module(layers, monkeypatch, tmp_path, error):
    """No compiler for it, no torch headers: build() still gives the library."""
    def fail():
        raise error
    monkeypatch.setattr(gbuild, "_compile_host", fail)
    monkeypatch.setattr(gbuild, "_host_target", lambda: str(tmp_path / "none.so"))
    with pytest.warns(UserWarning, match="no compiled calls"):
        assert gbuild.build() == gbuild.LIB
    monkeypatch.undo()
    monkeypatch.setattr(gbuild, "_torch_dir", lambda: None)
    assert gbuild._host_target() is None and gbuild.up_to_date()
