"""`python __graft_entry__.py smoke` runs what importing the module and calling smoke() runs."""
import ast
import os
import subprocess
import sys

import pytest

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "__graft_entry__.py")


def test_everything_is_defined_before_the_script_runs():
    body = ast.parse(open(PATH).read()).body
    guards = [i for i, s in enumerate(body) if isinstance(s, ast.If) and "__name__" in ast.dump(s.test)]
    assert guards == [len(body) - 1]


@pytest.mark.gpu
def test_the_script_runs_to_its_end():
    r = subprocess.run([sys.executable, PATH, "smoke"], cwd=os.path.dirname(PATH), capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "smoke decode after eviction ok" in r.stdout
