"""When the Python binding of the 8-bit activation calls is built, and what
happens where it cannot be."""
import os

import pytest

from bit_quantized_shampoo_b200 import build as B


@pytest.fixture
def place(monkeypatch, tmp_path):
    """An empty build folder; returns the list of commands that were run."""
    monkeypatch.setattr(B, "BUILD", str(tmp_path))
    monkeypatch.setattr(B, "BINDING", str(tmp_path / "_act8.so"))
    monkeypatch.delenv("CXX", raising=False)
    ran = []

    def run(cmd):
        ran.append(cmd)
        with open(B.BINDING, "w") as f:
            f.write("x")
    return run, ran


def test_built_once_for_one_torch(place, monkeypatch):
    import torch
    run, ran = place
    B._build_binding(run, False)
    B._build_binding(run, False)
    assert len(ran) == 1 and f'-DACT8_BUILT_FOR="{torch.__version__}"' in ran[0]
    monkeypatch.setattr(torch, "__version__", "99.0")
    B._build_binding(run, False)
    assert len(ran) == 2 and '-DACT8_BUILT_FOR="99.0"' in ran[1]
    B._build_binding(run, True)
    assert len(ran) == 3
    os.remove(B.BINDING)
    B._build_binding(run, False)
    assert len(ran) == 4


def test_a_failed_build_is_tried_again(place):
    def fail(cmd):
        raise RuntimeError("no")
    with pytest.raises(RuntimeError):
        B._build_binding(fail, False)
    run, ran = place
    B._build_binding(run, False)
    assert len(ran) == 1


def test_the_library_is_built_without_what_the_binding_needs(place, monkeypatch, capsys):
    run, ran = place
    B._build_binding(run, False)
    monkeypatch.setenv("CXX", "no-such-compiler")
    B._build_binding(run, False)
    assert len(ran) == 1 and not os.path.exists(B.BINDING)
    assert "no compiler no-such-compiler" in capsys.readouterr().err


def test_a_binding_for_another_torch_is_not_used(monkeypatch):
    import torch
    from bit_quantized_shampoo_b200 import api
    monkeypatch.setattr(api, "_act8_module", None)
    monkeypatch.setattr(torch, "__version__", "99.0")
    with pytest.raises(RuntimeError, match="is for torch"):
        api._act8()
