"""The binding's argument check belongs to one torch and one Python: one of another is not loaded, and
without one the binding checks in Python."""
import os
import shutil
import subprocess
import sys
import sysconfig

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "hybrid_packed_tree_b200")

REFUSALS = """
import torch
from hybrid_packed_tree_b200 import stree
bf = dict(dtype=torch.bfloat16)
q, k, cu = torch.zeros(5, 4, 128, **bf), torch.zeros(5, 2, 128, **bf), torch.zeros(3, dtype=torch.int32)
gates, S = torch.zeros(5, 4), torch.zeros(5, 4, 128, 128)
for call, kind, text in (
        (lambda: stree.stree_prompt_attention(q, k, k, cu, q, 0.1), ValueError, "q must be a CUDA tensor"),
        (lambda: stree.stree_linear_prompt(k[:4], k, q, gates, None, cu, q), ValueError, "q has shape (4, 2, 128)"),
        (lambda: stree.stree_linear_step(k.float(), k, q, gates, None, S, q, S), TypeError, "q has dtype torch.float32"),
        (lambda: stree.stree_linear_prompt(None, k, q, gates, None, cu, q), TypeError, "q must be a torch.Tensor")):
    try:
        call()
    except kind as e:
        assert text in str(e), str(e)
    else:
        raise AssertionError(text)
print("checked", stree._bind is not None)
"""


@pytest.fixture
def package(tmp_path):
    """A copy of the package with its library and without a check."""
    from hybrid_packed_tree_b200.build import build
    build()
    at = tmp_path / "hybrid_packed_tree_b200"
    at.mkdir()
    for f in ("__init__.py", "build.py", "stree.py", "libstree.so"):
        shutil.copy(os.path.join(PKG, f), at)
    return at


def _run(package, code):
    env = {k: v for k, v in os.environ.items() if k != "PYTHONPATH"}
    return subprocess.run([sys.executable, "-c", code], cwd=package.parent, env=env, capture_output=True, text=True)


def test_a_check_built_for_something_else_is_not_loaded(package):
    for name in ("_bind.so", f"_bind.torch-0.0.1-abi1{sysconfig.get_config_var('EXT_SUFFIX')}"):
        (package / name).write_bytes(b"not a library of this torch")
    r = _run(package, REFUSALS)
    assert r.returncode == 0 and "checked False" in r.stdout, r.stderr


def test_a_check_that_does_not_load_is_reported_and_left(package):
    from hybrid_packed_tree_b200.build import bind_path
    (package / os.path.basename(bind_path())).write_bytes(b"broken")
    r = _run(package, REFUSALS)
    assert r.returncode == 0 and "checked False" in r.stdout and "does not load" in r.stderr, r.stderr


def test_the_check_of_this_torch_is_loaded():
    from hybrid_packed_tree_b200.build import bind_path, build
    build()
    assert torch.__version__ in bind_path() and bind_path().endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    r = subprocess.run([sys.executable, "-c", REFUSALS], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and "checked True" in r.stdout, r.stderr


def test_the_library_builds_without_a_compiler_for_the_check(tmp_path, monkeypatch):
    from hybrid_packed_tree_b200 import build
    lib = build.build()
    monkeypatch.setattr(build, "bind_path", lambda: str(tmp_path / "_bind.so"))
    monkeypatch.setenv("CXX", "/nonexistent/g++")
    with pytest.warns(UserWarning, match="checked in Python"):
        assert build.build() == lib


def test_the_python_check_asks_what_the_compiled_one_asks():
    """Both accept and refuse the same arguments (on no device: the pointers are not reached)."""
    from hybrid_packed_tree_b200 import stree
    code = (
        "import torch\n"
        "from hybrid_packed_tree_b200 import stree\n"
        "t = torch.zeros(2, 4)\n"
        "for args in ((t, 'x', (2, 4), torch.float32, 0), (t.T, 'x', (4, 2), torch.float32, 0), (3, 'x', (), torch.float32, 0),\n"
        "             (t, 'x', (2, 5), torch.float32, 0), (t, 'x', (2, 4, 1), torch.float32, 0), (t, 'x', (2, 4), torch.int32, 0),\n"
        "             (t, 'x', (2, 4), torch.float32, -1), (t.to_sparse(), 'x', (2, 4), torch.float32, 0)):\n"
        "    for f in (stree._arg, stree._opt):\n"
        "        try:\n"
        "            f(*args)\n"
        "            print('accepted')\n"
        "        except (TypeError, ValueError) as e:\n"
        "            print(type(e).__name__, e)\n"
        "print(stree._opt(None, 'x', (2,), torch.float32, 0))\n")
    outs = []
    for pre in ("", "import hybrid_packed_tree_b200.build as b; b.bind_path = lambda: '/nonexistent'\n"):
        r = subprocess.run([sys.executable, "-c", pre + code], cwd=ROOT, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        outs.append(r.stdout)
    assert outs[0] == outs[1] and "accepted" not in outs[0] and stree._arg is not None
