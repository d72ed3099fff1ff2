"""The key-value cache operators' compiled binding is theirs alone: without it,
or with one for another torch, the rest of the package works."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def built():
    import __graft_entry__

    b = __graft_entry__._load_build_module()
    b.build()
    return b


def run(root, code, **env):
    return subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=root, timeout=300,
                          env=dict(os.environ, PYTHONPATH=str(root), **env))


@pytest.fixture
def copy(built, tmp_path):
    """The package as it was built, without the binding."""
    shutil.copytree(os.path.join(ROOT, "topk_selection_gb300"), tmp_path / "topk_selection_gb300",
                    ignore=shutil.ignore_patterns("*.o", "__pycache__", "csrc", "kv_binding*.so"))
    return tmp_path


CODE = """
import torch, topk_selection_gb300 as tk
assert tk.status_string(0) == "ok" and tk.launch_count() == 0
assert tk.topk_i32_ptr(0, 0, 0, 0) == 1
half, i32 = torch.zeros(4, 16, 2, 64, dtype=torch.float16), torch.zeros(2, dtype=torch.int32)
try:
    tk.kv_attend(half[:2, 0], half, half, i32[:, None], i32)
except ImportError as e:
    print("missing", "kv_binding" in str(e))
"""


def test_the_package_without_the_binding(copy):
    r = run(copy, CODE)
    assert r.returncode == 0, r.stderr
    assert r.stdout.split() == ["missing", "True"]


def test_a_binding_of_another_torch_is_not_taken(copy, built):
    """Neither as up to date nor at a call."""
    import torch

    path = built.binding_path()
    assert torch.__version__ in os.path.basename(path) and os.path.exists(path)
    other = os.path.basename(path).replace(torch.__version__, "1.0.0")
    (copy / "topk_selection_gb300" / "_lib" / other).write_bytes(b"not a module")
    (copy / "topk_selection_gb300" / "_lib" / "kv_binding.so").write_bytes(b"not a module")
    r = run(copy, CODE + "assert not tk._build.up_to_date()\n")
    assert r.returncode == 0, r.stderr
    assert r.stdout.split() == ["missing", "True"]


def test_the_library_is_built_without_torch(built, monkeypatch):
    """build() asks for torch only to compile the binding."""
    monkeypatch.setattr(built.importlib.util, "find_spec", lambda name: None)
    assert built.binding_path() is None
    assert built.up_to_date()


def test_first_call_loads_it_once(built):
    r = run(ROOT, """
import torch, topk_selection_gb300 as tk
half, i32 = torch.zeros(4, 16, 2, 64, dtype=torch.float16), torch.zeros(2, dtype=torch.int32)
assert "attend" not in vars(tk._kv)
for _ in range(2):
    try:
        tk.kv_attend(half[:2, 0], half, half, i32[:, None], i32)
    except ValueError as e:
        assert "CUDA" in str(e)
    first = vars(tk._kv)["attend"]
assert vars(tk._kv)["attend"] is first
print("ok")
""")
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr
