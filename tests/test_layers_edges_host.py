"""Calls of layer norm, the dense layer and AdamW at the edge of what they allow, without a
GPU: sizes of zero, strides of zero, arrays that are not where they seem."""
import os
import subprocess
import sys

import pytest

import momentum_compression_gb300 as ob



@pytest.fixture(scope="module", autouse=True)
def _built():
    from momentum_compression_gb300 import _build
    _build.build()


SIZES = """
import momentum_compression_gb300 as ob
for M in (0, 1, 5, 300):
    for N in (0, 1, 5, 4096):
        for K in (0, 7, 64):
            for act in (0, 2):
                for kn in (0, 1):
                    for off in (0, 1):
                        for backward in (0, 1):
                            b = ob.ob_linear_workspace_bytes(1, act, kn, off, M, N, K, backward)
                            assert 0 <= b < 1 << 26, (M, N, K, b)
print("fine")
"""


def test_workspaces_of_sizes_of_zero():
    """In a process of its own, which a division by zero would end."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", SIZES], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "fine", (r.returncode, r.stderr[-2000:])
