"""The library and its host-only calls where torch cannot be imported (ctypes users, size planning)."""

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import sys

class Blocked:
    def find_spec(self, name, path=None, target=None):
        if name == "torch" or name.startswith("torch."):
            raise ImportError("torch is blocked")

sys.meta_path.insert(0, Blocked())
import decoupled_momentum_optimizer_gb300 as dm

L = dm.lib()
assert all(size > 0 for size in dm.payload_bytes("demo", 65536, 4))
assert L.demo_fp8_bytes(5, 129, None) == 1280 and L.demo_fp8_linear_workspace(1, 8, 8) == 0
assert L.demo_dropout.argtypes is not None
assert "torch" not in sys.modules
try:
    dm.dropout
except ImportError:
    print("loaded")
"""


def test_the_library_loads_and_answers():
    from decoupled_momentum_optimizer_gb300 import build

    build.build()
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "loaded", r.stderr
