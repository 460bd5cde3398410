"""The bounded waits of k_tree_mma, made to run out on purpose by a hand-over that a test-only setting leaves out.  The kernel gives up
after about a second, lets its copies and products land, gives its tensor memory back and leaves; the call is reported once, and the
context stays usable.  In a child process: the test build of the library (libar_test.so) reads the setting once per process, and the
product library (libar.so) ignores it."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("args,said", [([], "tree timeout ok"), (["product"], "product library ignores")])
def test_bounded_waits_run_out_and_the_next_calls_are_right(args, said):
    env = dict(os.environ, AR_TEST_TREE_STALL="3")
    res = subprocess.run([sys.executable, "-m", "tests.tree_timeout_child", *args], cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0 and said in res.stdout, res.stdout[-3000:] + res.stderr[-3000:]
