"""The build without what only the Python extension needs (no GPU needed)."""

import os
import subprocess
import sys

import pytest

from chunkwise_delta_rule_gb300 import build as kbuild


@pytest.mark.parametrize("how", ["no compiler", "no headers"])
def test_libkda_is_built_where_the_extension_can_not_be(how, monkeypatch, tmp_path, capsys):
    lib, binding = tmp_path / "libkda.so", tmp_path / "_binding.so"
    binding.write_bytes(b"of other sources")
    monkeypatch.setattr(kbuild, "LIB", str(lib))
    monkeypatch.setattr(kbuild, "BINDING", str(binding))
    if how == "no compiler":
        os.utime(binding, (0, 0))
        monkeypatch.setenv("CXX", str(tmp_path / "none"))
    else:
        def fail():
            raise RuntimeError("the host compiler failed")
        monkeypatch.setattr(kbuild, "_compile_binding", fail)
    assert kbuild.build() == str(lib) and lib.exists()
    assert not binding.exists()
    assert "_binding.so was not built" in capsys.readouterr().err


def test_a_missing_extension_is_named_at_its_first_use(tmp_path):
    code = ("import sys; sys.modules['chunkwise_delta_rule_gb300._binding'] = None\n"
            "import torch, chunkwise_delta_rule_gb300 as kda\n"
            "kda.make_norm_problem(torch.zeros(1, 8), torch.zeros(8))")
    r = subprocess.run([sys.executable, "-c", code], cwd=kbuild.ROOT, capture_output=True, text=True)
    assert r.returncode != 0 and "ImportError: _binding.so is not built" in r.stderr
