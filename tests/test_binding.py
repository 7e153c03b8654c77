"""The native part of the Python binding: what it is built for."""

import sys

import pytest

import block_scaled_fp8_w8a16_amd as w8
from block_scaled_fp8_w8a16_amd import attention

torch = pytest.importorskip("torch")


@pytest.fixture
def unset(monkeypatch):
    """As before the first call."""
    monkeypatch.setattr(attention, "_state", None)
    monkeypatch.setattr(attention, "_fast", None)
    return monkeypatch


def test_built_for_this_torch(unset):
    attention._setup()
    binding = attention._fast[0]
    assert binding.torch_version == str(torch.__version__)
    assert binding.python_version == "%d.%d" % sys.version_info[:2]


def test_another_torch_is_refused(unset):
    """Tensors' layout is that of the torch it was built against."""
    unset.setattr(torch, "__version__", "1.0.0")
    t = torch.zeros(1, 1, 16)
    with pytest.raises(ImportError, match="built for torch .*, this is 1.0.0.*build"):
        w8.rope(t, t, t)
    with pytest.raises(ImportError, match="build"):       # again, not a half-set-up module
        w8.rope(t, t, t)


def test_the_build_step_loads_it(unset):
    """A binding that does not load fails the build."""
    import inspect

    import __graft_entry__ as entry
    assert "_binding" in inspect.getsource(entry.build) or "_setup" in inspect.getsource(entry.build)
