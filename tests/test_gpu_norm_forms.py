"""Group norm in the forms that its planner would not take by itself: every
shape as a slab where it fits one, and every shape by parts (ACP_NORM_FORM,
read once per process, so each runs in one child process)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.parametrize("form", ["slab", "parts"])
def test_every_shape_in_one_form(form):
    print(f"[gpu] child process: group norms with ACP_NORM_FORM={form}", flush=True)
    r = subprocess.run([sys.executable, "-u", os.path.join(HERE, "norm_form_child.py")],
                       env=dict(os.environ, ACP_NORM_FORM=form), capture_output=True, text=True, timeout=110)
    print(r.stdout[-3000:], flush=True)
    assert r.returncode == 0, r.stderr[-3000:]
    assert "all ok" in r.stdout
