"""The calls with their arguments checked in Python, as on a machine where the compiled check was not built."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def test_calls_and_refusals_without_the_compiled_check():
    tests = [os.path.join(HERE, "test_gpu_serving_run.py"), os.path.join(HERE, "test_gpu_paged.py") + "::test_binding_refuses_each_tensor"]
    code = ("import sys, pytest\n"
            "import hybrid_packed_tree_b200.build as b\n"
            "b.bind_path = lambda: '/nonexistent'\n"
            "from hybrid_packed_tree_b200 import stree\n"
            "assert stree._bind is None\n"
            f"sys.exit(pytest.main(['-q', '-x', '-p', 'no:cacheprovider', *{tests!r}]))\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=os.path.dirname(HERE), capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
