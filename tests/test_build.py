"""When the extension module is built again: it is compiled against torch's C++
interfaces, so that file times alone do not tell."""
import os
import shutil

import pytest
import torch

import rotated_w4a4_quantized_b200 as cr
from rotated_w4a4_quantized_b200 import build


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def test_a_fresh_build_is_not_stale():
    assert not build.stale()


def test_another_torch_makes_the_extension_stale(monkeypatch):
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    assert build.stale()
    built = []
    monkeypatch.setattr(build, "_build_binding", lambda verbose: built.append(verbose))
    monkeypatch.setattr(build, "_build_one", lambda *a: pytest.fail("a library was built"))
    build.build()
    assert built == [False]


@pytest.mark.parametrize("left", ["", "torch 0.0.1 abi 1 python 3.0.0", None])
def test_an_extension_of_unknown_origin_is_stale(monkeypatch, tmp_path, left):
    lib = str(tmp_path / os.path.basename(build.LIB_BINDING))
    shutil.copy(build.LIB_BINDING, lib)
    monkeypatch.setattr(build, "LIB_BINDING", lib)
    if left is not None:
        with open(lib + ".built", "w") as f:
            f.write(left)
    assert build._binding_stale()
    with open(lib + ".built", "w") as f:
        f.write(build._built_against())
    assert not build._binding_stale()


def test_an_extension_that_does_not_load_says_what_to_do(monkeypatch):
    import sys
    monkeypatch.setattr(cr, "_extension", None)
    monkeypatch.delattr(cr, "_decoding", raising=False)
    monkeypatch.setitem(sys.modules, cr.__name__ + "._decoding", None)
    with pytest.raises(RuntimeError, match="does not fit this torch: build it"):
        cr._native()
