"""The extension module behind the calls around the experts: a build without torch, and a package whose
module is missing or was built for another torch, keep everything else."""
import glob
import importlib.util
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "routed_expert_ffn_02_amd")

BROKEN = {"missing": "sys.modules['routed_expert_ffn_02_amd._marshal'] = None",
          "another torch": "import types; m = types.ModuleType('routed_expert_ffn_02_amd._marshal'); m.torch_version = '1.0.0'; "
                           "sys.modules[m.__name__] = m",
          "an earlier module": "import types; m = types.ModuleType('routed_expert_ffn_02_amd._marshal'); "
                               "sys.modules[m.__name__] = m"}


@pytest.mark.parametrize("why", BROKEN)
def test_calls_on_a_context_need_no_module(why):
    code = f"""
import sys, torch
{BROKEN[why]}
import routed_expert_ffn_02_amd as R
cfg = R.make_config(1, 8, 2, 64, 128, R.MOE_WFMT_F32, R.MOE_AFMT_F32, 1, R.MOE_MODE_OFFLOAD)
assert R.moe_record_bytes(cfg) > 0 and R.qstar_split(4, 1, 4, R.MOE_MODE_HYBRID, 3) >= 0
assert R.moe_dispatch_workspace(4096, 8, 256) > 0
try:
    R.moe_combine(torch.zeros(2, 4), torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, 2), torch.zeros(1, 4))
except ImportError as e:
    assert "_build.py" in str(e), e
    print("refused", e)
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert "refused" in r.stdout and ("1.0.0" in r.stdout) == (why == "another torch")


def builder():
    spec = importlib.util.spec_from_file_location("routed_expert_ffn_02_amd_build_test", os.path.join(PKG, "_build.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_the_module_carries_its_abi():
    import sysconfig

    import torch

    import routed_expert_ffn_02_amd as R
    assert [os.path.basename(f) for f in glob.glob(os.path.join(PKG, "_marshal*.so"))] == [
        "_marshal" + sysconfig.get_config_var("EXT_SUFFIX")]
    assert torch.__version__.startswith(R._marshal.torch_version)


@pytest.mark.parametrize("lacks", ["torch", "headers"])
def test_the_library_is_built_without_torch(lacks, tmp_path, monkeypatch, capsys):
    """Compiling and linking stubbed: which objects are made and what is linked."""
    b = builder()
    made, linked = [], []
    monkeypatch.setattr(b, "BUILD", str(tmp_path))
    monkeypatch.setattr(b, "HERE", str(tmp_path))
    monkeypatch.setattr(b, "_compile", lambda src, flags=(): made.append(src) or src + ".o")
    monkeypatch.setattr(b, "_link", lambda cmd, out, libs: linked.append(out))
    if lacks == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)
    else:
        monkeypatch.setattr(b.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    b.build(verbose=False)
    assert sorted(made) == sorted(b.HIP_SOURCES + b.CPP_SOURCES) and linked == [b.LIB]
    assert "without their Python module" in capsys.readouterr().err


def test_the_library_is_linked_where_the_module_fails(tmp_path, monkeypatch):
    b = builder()
    linked = []

    def compile_(src, flags=()):
        if src == b.MARSHAL_SOURCE:
            raise RuntimeError("compile failed")
        return src + ".o"

    monkeypatch.setattr(b, "BUILD", str(tmp_path))
    monkeypatch.setattr(b, "HERE", str(tmp_path))
    monkeypatch.setattr(b, "_compile", compile_)
    monkeypatch.setattr(b, "_link", lambda cmd, out, libs: linked.append(out))
    with pytest.raises(RuntimeError, match="compile failed"):
        b.build(verbose=False)
    assert linked == [b.LIB]
