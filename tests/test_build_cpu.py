"""The build of the binding's extension module: its file belongs to one Python, its
failure leaves no compiler running, and what does not use it does without it."""
import importlib.util
import os
import subprocess
import sys
import sysconfig

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "vision_transformer_encoder_layernorm_b200")


def build_module(tmp_path):
    """build.py, writing to tmp_path."""
    spec = importlib.util.spec_from_file_location("_build_under_test", os.path.join(PKG, "build.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    name = os.path.basename(m.MARSHAL)
    m.HERE, m.LIB, m.MARSHAL = str(tmp_path), str(tmp_path / "libvit.so"), str(tmp_path / name)
    return m


def script(path, text):
    path.write_text("#!/bin/sh\n" + text)
    path.chmod(0o755)
    return str(path)


@pytest.fixture
def nvcc(tmp_path, monkeypatch):
    """A stand-in that notes its start and its end and leaves an empty output."""
    log = tmp_path / "log"
    monkeypatch.setenv("NVCC", script(tmp_path / "nvcc", f'''
echo start >> {log}
sleep 0.5
while [ $# -gt 1 ]; do [ "$1" = -o ] && : > "$2"; shift; done
echo end >> {log}
'''))
    return lambda word: log.read_text().split().count(word) if log.exists() else 0


def test_module_is_named_for_its_python(tmp_path):
    assert build_module(tmp_path).MARSHAL.endswith("_marshal" + sysconfig.get_config_var("EXT_SUFFIX"))


def test_failed_module_leaves_no_compiler_running(tmp_path, monkeypatch, nvcc):
    monkeypatch.setenv("CC", "false")
    m = build_module(tmp_path)
    with pytest.raises(Exception):
        m.build()
    assert nvcc("end") == nvcc("start") > 0
    # and the library is there: what does not need the module works
    assert os.path.exists(m.LIB) and not os.path.exists(m.MARSHAL)


def test_each_part_is_built_when_it_is_stale(tmp_path, monkeypatch, nvcc):
    m = build_module(tmp_path)
    m.build()
    n = nvcc("start")
    assert n > 0 and os.path.exists(m.LIB) and os.path.exists(m.MARSHAL)
    os.remove(m.MARSHAL)
    m.build()
    assert os.path.exists(m.MARSHAL) and nvcc("start") == n  # the library was not
    monkeypatch.setenv("CC", "false")  # nothing is stale: nothing runs
    m.build()


def test_package_without_the_module(tmp_path):
    """Imports; a checked call says what is missing, another does not miss it."""
    pkg = tmp_path / os.path.basename(PKG)
    pkg.mkdir()
    os.symlink(os.path.join(PKG, "libvit.so"), pkg / "libvit.so")
    (pkg / "__init__.py").write_bytes(open(os.path.join(PKG, "__init__.py"), "rb").read())
    code = '''
import torch
import vision_transformer_encoder_layernorm_b200 as vit
c = vit.Context.__new__(vit.Context)
c.cfg, c._h, c._device = vit.VitConfig(1152, 16, 72, 64, 1e-6, 1e4, vit.BF16, 0), None, -1
x = torch.zeros(4, 64, dtype=torch.bfloat16)
try:
    c.layernorm(x, x, x, x, stream=0)
except vit.VitError as e:
    print("refused", e.code)
try:
    c.rmsnorm(x, x[0], x, stream=0)
except ImportError as e:
    print("missing", "_marshal" in str(e))
'''
    out = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True,
                         env={k: v for k, v in os.environ.items() if k != "PYTHONPATH"})
    assert out.stdout.split("\n")[:2] == ["refused 1", "missing True"], out
