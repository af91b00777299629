"""The cache's binding on a torch that lacks the library functions which only make small calls
faster."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("name", ["_dynamo", "_dynamo.guards", "_dynamo.guards._empty_strided_cuda",
                                  "_cuda_cudaCachingAllocator_raw_alloc",
                                  "_cuda_cudaCachingAllocator_raw_delete"])
def test_the_package_is_imported_without(name):
    code = f"""
import operator, torch
*path, last = "{name}".split(".")
owner = operator.attrgetter(".".join(path))(torch._C) if path else torch._C
if hasattr(owner, last):
    delattr(owner, last)
from gated_delta_rule_kaczmarz_gb300 import cache
gone = cache._empty if "{name}".startswith("_dynamo") else cache._free if "delete" in "{name}" else cache._alloc
assert gone is None
"""
    subprocess.run([sys.executable, "-c", code], cwd=ROOT, check=True)
