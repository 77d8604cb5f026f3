"""What the package needs where the native binding of the cache-filling calls
cannot be built: the other calls work, these say what is missing (no GPU)."""
import os
import shutil
import subprocess
import sys
import sysconfig

import pytest

from tests.conftest import ensure_lib

CODE = """
import torch
from self_speculative_sparse_vg_gb300 import vg
assert vg.version() and vg.verify_workspace_bytes(1, 1, 8, 2, 64, 1000) >= 0
assert vg.status_string(0)
i = torch.zeros(1, dtype=torch.int32)
p = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
kv = vg.PagedKV(p, p, i[None])
for name, call in (("step_tables", lambda: vg.step_tables(i[None], 2, i, i, i, i, i, i)),
                   ("rope_append", lambda: vg.rope_append(kv, None, p, p, i)),
                   ("chunk_attention", lambda: vg.chunk_attention(kv, p, i, i, 1.0, p, workspace=i))):
    try:
        call()
    except ImportError as e:
        assert name in str(e) and "vg_binding.so" in str(e), e
    else:
        raise AssertionError(name)
print("fine")
"""


@pytest.mark.parametrize("binding", [None, b"not a library"])
def test_the_older_calls_need_libvg_alone(tmp_path, binding):
    ensure_lib()
    from self_speculative_sparse_vg_gb300 import build
    pkg = tmp_path / "self_speculative_sparse_vg_gb300"
    pkg.mkdir()
    for name in os.listdir(build.PKG):
        if name.endswith(".py") or name == "libvg.so":
            shutil.copy(os.path.join(build.PKG, name), pkg / name)
    if binding is not None:
        (pkg / "vg_binding.so").write_bytes(binding)
    r = subprocess.run([sys.executable, "-c", CODE], cwd=tmp_path, capture_output=True, text=True,
                       env={k: v for k, v in os.environ.items() if k != "PYTHONPATH"})
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr


def test_what_the_binding_lacks(monkeypatch, tmp_path):
    from self_speculative_sparse_vg_gb300 import build
    assert build.binding_lacks() == ""
    monkeypatch.setattr(build, "CXX", "no-such-compiler")
    assert "no-such-compiler" in build.binding_lacks()
    monkeypatch.undo()
    monkeypatch.setattr(sysconfig, "get_paths", lambda *a, **k: {"include": str(tmp_path)})
    assert build.binding_lacks().endswith("Python.h")
    monkeypatch.undo()
    monkeypatch.setattr(build, "_torch_dir", lambda: str(tmp_path))
    assert build.binding_lacks().endswith("CUDAGuard.h")


def test_the_build_goes_on_without_the_binding(monkeypatch, tmp_path):
    """libvg.so is built, a binding of another one is taken away, and a warning
    says why; where nothing is missing, a failure of the binding is an error."""
    from self_speculative_sparse_vg_gb300 import build
    lib, binding = tmp_path / "libvg.so", tmp_path / "vg_binding.so"
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "obj"))
    monkeypatch.setattr(build, "LIB", str(lib))
    monkeypatch.setattr(build, "BINDING", str(binding))
    monkeypatch.setattr(build, "_compile", lambda src, verbose: src)

    def run(cmd, what):
        if "binding" in what:
            raise RuntimeError(what)
        open(cmd[cmd.index("-o") + 1], "w").close()
    monkeypatch.setattr(build, "_run", run)
    with pytest.raises(RuntimeError, match="vg_binding"):
        build.build()
    binding.write_bytes(b"old")
    monkeypatch.setattr(build, "binding_lacks", lambda: "Python.h")
    with pytest.warns(UserWarning, match="Python.h is missing"):
        assert build.build() == str(lib)
    assert lib.exists() and not binding.exists()


def test_the_build_command_without_the_binding(monkeypatch):
    """build() of the entry module, where the binding is left out, ends well."""
    ensure_lib()
    import __graft_entry__ as entry
    from self_speculative_sparse_vg_gb300 import build
    monkeypatch.setattr(build, "build", lambda: build.LIB)
    monkeypatch.setattr(build, "binding_lacks", lambda: "Python.h")
    monkeypatch.setitem(sys.modules, "self_speculative_sparse_vg_gb300.vg_binding", None)   # an import raises
    entry.build()
    monkeypatch.setattr(build, "binding_lacks", lambda: "")
    with pytest.raises(ImportError):
        entry.build()
