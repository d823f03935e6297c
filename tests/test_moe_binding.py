"""CPU checks of the mixture-of-experts binding around its calls: where outputs are allocated, and what the
package does without the parts that are not everywhere."""
import contextlib
import os
import subprocess
import sys
import sysconfig

import pytest
import torch

from blockwise_scaled_fp8_act_amd import binding, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class _Like:
    """Stands for a GPU tensor; notes the stream that is current when memory is asked for."""
    is_cuda = True
    device = "cuda:0"

    def __init__(self, current):
        self.current = current

    def new_empty(self, shape, dtype):
        return self.current[-1], shape, dtype


@pytest.mark.parametrize("handle,want", [(0, "default"), (7, "external 7")])
def test_outputs_belong_to_the_stream_whose_handle_is_given(monkeypatch, handle, want):
    """The handle 0 names the default stream and no new one: the memory of a call's outputs is handed on in
    the order of the work that uses it."""
    current = ["current"]

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    def external(handle, device=None):
        return f"external {handle}" if handle else "a new stream"
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", external)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    assert binding._empty(_Like(current), (2, 3), torch.int32, handle) == (want, (2, 3), torch.int32)
    assert binding._empty(_Like(current), 5, torch.uint8, None) == ("current", 5, torch.uint8)


def test_checks_work_where_torch_lacks_its_shortcuts():
    """A torch without the private functions that the binding prefers: every check of a GPU tensor, the older entry
    points' among them, goes by the public ones."""
    code = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
torch.cuda.current_device = lambda: 1
from blockwise_scaled_fp8_act_amd import binding
class T:
    device, is_cuda = "cuda", True
    def __init__(self, at): self.at = at
    def get_device(self): return self.at
assert binding._gpu(x=T(1), y=None) == 1 and binding._current(T(1), None, T(1)) == 1 and binding._current(T(0)) is None
try:
    binding._gpu(x=T(0))
except ValueError as e:
    assert "current device" in str(e)
else:
    raise SystemExit("accepted a tensor of another device")
binding.lib()
assert binding._calls is None
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_library_works_without_the_c_part(monkeypatch):
    """_calls not built, or for another interpreter: the library loads, and the long way of a call answers."""
    import blockwise_scaled_fp8_act_amd as bf
    monkeypatch.delattr(bf, "_calls", raising=False)
    monkeypatch.setitem(sys.modules, bf.__name__ + "._calls", None)
    monkeypatch.setattr(binding, "_lib", None)
    monkeypatch.setattr(binding, "_calls", None)
    assert binding.lib().bsfp8_status_string(0) and binding._calls is None
    with pytest.raises(ValueError, match="k = 17"):
        bf.moe_route(torch.zeros(4, 16), 17)
    with pytest.raises(ValueError, match="GPU tensor"):
        bf.moe_route(torch.zeros(4, 16), 2)


def test_c_part_is_built_for_this_interpreter_or_left_out(monkeypatch, tmp_path):
    """Its name carries the interpreter's tag; without Python's headers or a C compiler the build goes on, and
    nothing that an earlier build made stays behind."""
    assert build.CALLS_PATH.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    here = str(tmp_path)
    old = tmp_path / "_calls.so"
    monkeypatch.setattr(build, "PKG", here)
    monkeypatch.setattr(build, "CALLS_PATH", os.path.join(here, os.path.basename(build.CALLS_PATH)))
    old.write_bytes(b"of another interpreter")
    assert build._build_calls() and os.listdir(here) == [os.path.basename(build.CALLS_PATH)]
    for name, value in (("CC", "no-such-compiler"), ("sysconfig", type("S", (), {"get_paths": staticmethod(lambda: {"include": here})}))):
        old.write_bytes(b"of another interpreter")
        with monkeypatch.context() as m:
            m.setattr(build, name, value)
            assert not build._build_calls() and os.listdir(here) == []
        assert build._build_calls()
