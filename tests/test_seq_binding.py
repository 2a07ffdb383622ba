"""The package with and without the C++ checks of the operators between a block's projections (_binding.so).  No kernel is
launched."""
import importlib.util
import os
import shutil
import subprocess
import sys

import pytest
import torch

PACKAGE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_quantized_matvec_amd")

USE = """
import warnings
with warnings.catch_warnings(record=True) as said:
    warnings.simplefilter("always")
    import bit_quantized_matvec_amd as tq
assert tq.seq._binding is None and len(said) == 1 and "_binding.so is not used" in str(said[0].message), said
import torch
assert tq.check_shape("pq2_0", 64, 256, 1) == 0
x = torch.zeros(1, 1, 64)
c = torch.zeros(1, 1, 16, 64)
for call in (lambda: tq.rope_append(x, x, x, None, x, None, c, c, out=x), lambda: tq.paged_attn(x, c, c, x, x, out=x),
             lambda: tq.gdn(x, x, x, x, x, c, out=x)):
    try:
        call()
    except ValueError as e:
        assert "CUDA tensor" in str(e), e
    else:
        raise AssertionError("host tensors were taken")
"""


def package(tmp_path):
    """A copy of the package without the module."""
    to = tmp_path / "bit_quantized_matvec_amd"
    to.mkdir()
    for f in os.listdir(PACKAGE):
        if f.endswith(".py") or f == "libtq.so":
            shutil.copy(os.path.join(PACKAGE, f), to)
    return to


def use(tmp_path):
    r = subprocess.run([sys.executable, "-c", USE], cwd=tmp_path, capture_output=True, text=True, env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert r.returncode == 0, r.stderr


def test_the_package_works_without_the_module(tmp_path):
    package(tmp_path)
    use(tmp_path)


def test_a_module_of_another_torch_is_not_used(tmp_path):
    (package(tmp_path) / "_binding.py").write_text("torch_version = '1.0'\n")
    use(tmp_path)


def test_the_built_module_is_used():
    import bit_quantized_matvec_amd as tq

    if not os.path.exists(os.path.join(PACKAGE, "_binding.so")):
        pytest.skip("_binding.so is not built")
    assert tq.seq._binding is not None and tq.seq._binding.torch_version == torch.__version__


def test_the_build_goes_on_without_a_compiler(tmp_path, monkeypatch, capsys):
    spec = importlib.util.spec_from_file_location("tq_build", os.path.join(PACKAGE, "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    old = tmp_path / "_binding.so"
    old.write_text("of other sources")
    monkeypatch.setattr(build, "BINDING", str(old))
    monkeypatch.setattr(build, "CXX", "no-such-compiler")
    build._build_binding()
    assert not old.exists() and "no no-such-compiler" in capsys.readouterr().err
