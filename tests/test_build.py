"""When the native parts are built anew (CPU)."""
import sys
import sysconfig

import pytest
import torch

from mixed_sliding_global_gb300 import _build, binding
from mixed_sliding_global_gb300.binding import library


@pytest.mark.parametrize("what", ["torch", "path", "suffix", "python"])
def test_another_torch_or_python_needs_another_bind(what, monkeypatch, tmp_path):
    """_bind.so was compiled against one PyTorch and one interpreter: with others it is stale."""
    library()
    assert _build.up_to_date()
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", torch.__version__ + ".post1")
    elif what == "path":
        monkeypatch.setattr(torch, "__file__", str(tmp_path / "torch" / "__init__.py"))
    elif what == "suffix":
        var = sysconfig.get_config_var
        monkeypatch.setattr(sysconfig, "get_config_var",
                            lambda n: ".cpython-399.so" if n == "EXT_SUFFIX" else var(n))
    else:
        monkeypatch.setattr(sys, "version", "3.99")
    assert not _build.up_to_date()


def test_library_does_not_need_the_bind(monkeypatch, tmp_path):
    """Without a compiler for _bind.so (or PyTorch's or Python's headers) the library builds and
    loads; the calls that need _bind.so, and a build of everything, say why they cannot."""
    library()

    def fail():
        raise RuntimeError("no headers")

    monkeypatch.setattr(_build, "BIND", str(tmp_path / "_bind.so"))
    monkeypatch.setattr(_build, "_compile_bind", fail)
    monkeypatch.setattr(binding, "_lib", None)
    monkeypatch.setattr(binding, "_bind", None)
    assert library().gemma_abi_version() == binding.gemma_abi_version()
    x = torch.zeros(1, 8)
    with pytest.raises(RuntimeError, match="no headers"):
        binding.gemma_logit_sample(x, x, x)
    built = []
    monkeypatch.setattr(_build, "build_library", lambda *a: built.append(a))
    with pytest.raises(RuntimeError, match="no headers"):
        _build.build()
    assert built
