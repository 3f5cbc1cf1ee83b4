"""Importing the package maps no library, so that a build in the same process is the one that is loaded after it."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import block_scaled_fp8_grouped_amd as bs
maps = lambda: [l.split()[-1] for l in open("/proc/self/maps") if "libbsfp8" in l or "_native" in l]
assert not maps(), maps()
assert bs._native is not None and bs._native is bs._native
assert any(m.endswith("_native.so") for m in maps()) and any(m.endswith("libbsfp8.so") for m in maps())
assert bs._native.residual_norm() is None
try:
    bs.no_such_name
except AttributeError:
    pass
else:
    raise SystemExit("an unknown name")
"""


def test_import_maps_no_library():
    r = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
