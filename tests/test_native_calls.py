"""The compiled calls of the sequence operators (_native.so) on the host: what works
without them, and when they are built again."""
import subprocess
import sys

import pytest

from conftest import ROOT


@pytest.fixture(scope="module", autouse=True)
def built():
    from protein_structure_models_b200 import build
    build.build()


def run(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)


def test_the_library_loads_without_them():
    """What needs libfipa.so only, the core, the layer and the kNN features, does not need them; the sequence operators say how to build them."""
    res = run("""
import sys
class Gone:
    def find_spec(self, name, path=None, target=None):
        if name.endswith("._native"):
            raise ImportError("undefined symbol")
sys.meta_path.insert(0, Gone())
import torch, protein_structure_models_b200 as fw
lib = fw.load_library()
assert lib.fipa_status_string(0) and fw.embedding_backward_workspace_size(5, 4, 8) > 0
try:
    fw.Fipa("f32", 0)
except fw.FipaError:
    pass                                   # no GPU here: the library itself answered
idx, x = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 8)
for call in (lambda: fw.embedding(idx, x), lambda: fw.embedding_backward(idx, x, 2), lambda: fw.norm_residual(x, x),
             lambda: fw.norm_residual_backward(x, x, x, x, x)):
    try:
        call()
    except RuntimeError as e:
        assert "undefined symbol" in str(e) and "protein_structure_models_b200.build" in str(e), e
    else:
        raise AssertionError
print("fine")
""")
    assert res.stdout.strip() == "fine", res.stdout + res.stderr


def test_they_refuse_tensors_of_the_host():
    import torch

    import protein_structure_models_b200 as fw
    with pytest.raises(ValueError):
        fw.embedding(torch.zeros(2, dtype=torch.int32), torch.zeros(2, 8))
    with pytest.raises(ValueError):
        fw.norm_residual(torch.zeros(2, 8), torch.zeros(2, 8))


def test_they_are_built_again_for_another_python_or_pytorch(monkeypatch):
    import sysconfig

    import torch

    from protein_structure_models_b200 import build, fipa
    assert not build.native_needs_build() and fipa.load_native().__doc__ == build.built_for()
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", torch.__version__ + "1")
        assert build.native_needs_build()
    with monkeypatch.context() as m:
        m.setattr(sysconfig, "get_config_var", lambda name: "cpython-313-x86_64-linux-gnu")
        assert build.native_needs_build()
    with monkeypatch.context() as m:
        m.setattr(build, "NATIVE", build.NATIVE + ".none")
        assert build.native_needs_build()
    assert not build.native_needs_build()


def test_what_is_asked_for_needs_a_buffer():
    """want_lse and want_stats beside `out` without such a buffer are refused, not dropped."""
    import torch

    import protein_structure_models_b200 as fw
    t, x = torch.zeros(1, 4, 2, 8), torch.zeros(2, 8)
    h = object.__new__(fw.Fipa)
    for out in ({"out": t}, {"lse": t}):
        with pytest.raises(ValueError, match="buffer out or lse missing"):
            h.window_attention(t, t, t, (1, 1), want_lse=True, out=out)
    with pytest.raises(ValueError, match="buffer r, x or stats missing"):
        fw.norm_residual(x, x, out={"r": x}, want_stats=True)
