"""The dropout and grouped layers in the bounds-checking build: their GPU tests
run once more in a process that loads it, and no check fails."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

INNER = """
import sys, pytest
rc = pytest.main(["-x", "-q", "-p", "no:cacheprovider", "-m", "gpu", *sys.argv[1:]])
import nf4_base_lora_b200 as nf
assert nf.lib.nf4lora_debug_build() == 1
site = nf.debug_site()
print("site %d line %d" % (site >> 16, site & 0xFFFF))
sys.exit(rc or site != 0)
"""


def test_no_access_check_fails():
    from nf4_base_lora_b200 import build
    build.build(debug=True)
    env = dict(os.environ, NF4LORA_DEBUG="1", PYTHONPATH=os.pathsep.join([ROOT, os.path.join(ROOT, "tests")]))
    out = subprocess.run([sys.executable, "-c", INNER, "tests/test_gpu_grouped.py", "tests/test_gpu_dropout.py",
                          "tests/test_gpu_adapter_edges.py"], cwd=ROOT, env=env, capture_output=True, text=True,
                         timeout=900)
    assert out.returncode == 0 and "site 0 line 0" in out.stdout, out.stdout[-3000:] + out.stderr[-3000:]
