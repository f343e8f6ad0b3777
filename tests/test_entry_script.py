"""__graft_entry__.py as a script."""
import ast
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SCRIPT = os.path.join(ROOT, "__graft_entry__.py")


def test_nothing_is_defined_after_the_scripts_calls():
    """What smoke() calls has to be there when the script's last block calls smoke()."""
    with open(SCRIPT) as f:
        body = ast.parse(f.read()).body
    runs = [k for k, node in enumerate(body)
            if isinstance(node, ast.If) and "__name__" in ast.unparse(node.test)]
    assert runs == [len(body) - 1]


@pytest.mark.gpu
def test_smoke_from_the_command_line():
    run = subprocess.run([sys.executable, SCRIPT, "--smoke"], cwd=ROOT, capture_output=True,
                         text=True, timeout=600)
    assert run.returncode == 0, run.stderr[-2000:]
    assert "smoke ok" in run.stdout
