"""The marshalling module _marshal: what works without it, and that one built against another torch is noticed (CPU)."""

import os
import shutil
import subprocess
import sys

import pytest

from conftest import ROOT, _build_module

PKG = os.path.join(ROOT, "paged_kv_cache_126_gb300")


def run(code, cwd):
    return subprocess.run([sys.executable, "-c", code], cwd=cwd, capture_output=True, text=True, timeout=300)


def test_package_works_without_it_until_its_calls(pa, tmp_path):
    to = tmp_path / "paged_kv_cache_126_gb300"
    shutil.copytree(PKG, to, ignore=shutil.ignore_patterns("_build", "csrc", "__pycache__", "_marshal.so"))
    res = run("import paged_kv_cache_126_gb300 as pa\n"
              "bm = pa.BlockManager(4, 8)\n"
              "assert len(bm.add_seq(1, 9)) == 9\n"
              "try:\n"
              "    pa.pa_cache_read_q4(None, None, None, None, None)\n"
              "except ImportError as e:\n"
              "    assert '_marshal.so not found' in str(e), e\n"
              "else:\n"
              "    raise SystemExit('no error')\n", tmp_path)
    assert res.returncode == 0, res.stdout + res.stderr


def test_another_torch_is_refused(pa):
    res = run("import torch\n"
              "import paged_kv_cache_126_gb300 as pa\n"
              "torch.__version__ = '1.0.0+cu1'\n"
              "try:\n"
              "    pa.pa_cache_read_q4(None, None, None, None, None)\n"
              "except ImportError as e:\n"
              "    assert 'built against torch' in str(e), e\n"
              "else:\n"
              "    raise SystemExit('no error')\n", ROOT)
    assert res.returncode == 0, res.stdout + res.stderr


@pytest.mark.parametrize("suffix", ["", "+cu130", "a0+gitabc123", ".dev20260101+cu130", "rc2"])
def test_the_same_release_under_other_names_is_taken(pa, monkeypatch, suffix):
    import torch

    import paged_kv_cache_126_gb300._binding as b

    release = b._load_marshal().torch_version
    monkeypatch.setattr(torch, "__version__", release + suffix)
    assert b._load_marshal().torch_version == release


def test_another_torch_is_rebuilt_for(pa, tmp_path, monkeypatch):
    mod = _build_module()
    assert not mod.is_stale()
    stamp = tmp_path / "torch"
    monkeypatch.setattr(mod, "MARSHAL_TORCH", str(stamp))
    assert mod.is_stale()
    stamp.write_text("1.0.0")
    assert mod.is_stale()
    stamp.write_text(mod._torch_version())
    assert not mod.is_stale()


def test_loaded_once(pa):
    import paged_kv_cache_126_gb300._binding as b

    with pytest.raises(TypeError):
        pa.pa_cache_read_q4(None, None, None, None, None)
    assert type(b._marshal).__name__ == "module"
