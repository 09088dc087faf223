"""The extension module that marshals the per-layer calls, as far as no GPU is
needed."""

import os
import subprocess
import sys

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from speculative_decoding_verification_07_gb300 import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(binding.LIB_PATH):
        from speculative_decoding_verification_07_gb300 import build
        build.build()


def test_the_library_loads_without_the_extension_module():
    """The verification and the cache calls need the C library alone; the
    per-layer calls fail loudly."""
    code = """
import sys
from speculative_decoding_verification_07_gb300 import binding
sys.modules["speculative_decoding_verification_07_gb300._calls"] = None
lib = binding.load_library()
a = binding.SvVerifyArgs()
a.B, a.kmax = 64, 4
assert binding.sv_workspace_size(a) > 0
try:
    binding._calls()
except ImportError:
    print("loud")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.split() == ["loud"], r.stderr


class Refusing(TorchDispatchMode):
    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        raise torch.OutOfMemoryError("no room")


def test_an_exception_of_an_allocation_keeps_its_type():
    q = torch.zeros(1, 1, 2, 64)
    call = binding._calls().attention
    args = (None, None, 0, q, None, None, None, None, None, None, None, None, 0)
    for _ in range(3):
        with Refusing(), pytest.raises(torch.OutOfMemoryError, match="no room"):
            call(*args)


def test_refusals_without_a_gpu():
    c = binding._calls()
    x = torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="parent"):
        c.tree_mask(None, x.long(), None, None, None, 0)
    with pytest.raises(TypeError):
        c.tree_mask(None, x)
    for mask, depth in ((x, None), (None, x)):  # one of the two would be ignored or missed
        with pytest.raises(ValueError, match="mask and depth"):
            c.tree_mask(None, x, None, mask, depth, 0)
