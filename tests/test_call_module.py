"""The CPython module of the serving calls belongs to the Python and torch that it
was built against: with another torch it is built again and never loaded."""
import os
import subprocess

import pytest
import torch

from paged_kv_decode_rope_gb300 import _binding, build


def test_every_torch_has_its_own_file(monkeypatch):
    here = build.call_module()
    assert os.path.exists(here), "built by build()"
    seen = {here}
    for module, name, value in ((torch, "__version__", "99.1.0+cu1"), (torch.version, "git_version", "0123456789abcdef"),
                                (torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)):
        with monkeypatch.context() as m:
            m.setattr(module, name, value)
            seen.add(build.call_module())
    assert len(seen) == 4 and all(os.path.dirname(p) == os.path.dirname(here) for p in seen)


def test_a_module_of_another_torch_is_not_loaded(monkeypatch):
    monkeypatch.setattr(_binding, "_call_module", None)
    monkeypatch.setattr(torch, "__version__", "99.1.0+cu1")
    with pytest.raises(RuntimeError, match="not built for this Python and torch"):
        _binding._native()


def test_a_module_of_another_torch_is_built_again(monkeypatch):
    class Compiled(Exception):
        pass

    def run(cmd, **kw):
        raise Compiled(cmd)

    monkeypatch.setattr(subprocess, "run", run)
    assert build.build_call() == build.call_module()  # up to date: nothing is compiled
    monkeypatch.setattr(torch, "__version__", "99.1.0+cu1")
    with pytest.raises(Compiled):
        build.build_call()
