"""When the extension module is compiled anew (no compiler is run here)."""
import os
import subprocess
import sysconfig

import torch

from compressed_sparse_attention_window_gb300 import build as ds41_build


def test_extension_module_follows_torch_and_python(monkeypatch, tmp_path):
    """It is compiled against both: another version of either makes it stale, and
    nothing else does."""
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(ds41_build.subprocess, "run", run)
    monkeypatch.setattr(ds41_build, "BUILD", str(tmp_path))
    monkeypatch.setattr(ds41_build, "BINDING", str(tmp_path / "module.so"))

    def compiled():
        n = len(ran)
        ds41_build._build_binding(False, False)
        assert os.path.exists(ds41_build.BINDING)
        return len(ran) - n
    assert compiled() == 1 and compiled() == 0
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "0.0.0")
        assert compiled() == 1 and compiled() == 0
    assert compiled() == 1 and compiled() == 0
    soabi = sysconfig.get_config_var

    with monkeypatch.context() as m:
        m.setattr(sysconfig, "get_config_var",
                  lambda name: "cpython-000" if name == "SOABI" else soabi(name))
        assert compiled() == 1 and compiled() == 0
    with monkeypatch.context() as m:
        m.setattr(torch, "compiled_with_cxx11_abi", lambda: not True)
        assert compiled() == 1 and compiled() == 0
