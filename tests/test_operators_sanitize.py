"""The host code of the router's and the adapters' entry points under
AddressSanitizer and UndefinedBehaviorSanitizer: their sizes over a wide grid
and next to the limits of what they accept (tests/sanitize/operators_host_sanitize.cpp).
The sanitizers are on the host pass only; nothing here touches a GPU."""
import glob
import os
import tempfile
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_abi_sanitize import B, CSRC, HERE, _compile, _link_and_run

DRIVER = os.path.join(HERE, "sanitize", "operators_host_sanitize.cpp")


@pytest.fixture(scope="module")
def objects():
    if not os.path.exists(B.HIPCC):
        pytest.skip("hipcc is not available")
    with tempfile.TemporaryDirectory() as d:
        srcs = sorted(glob.glob(os.path.join(CSRC, "*.hip"))) + [DRIVER]
        objs = [os.path.join(d, os.path.basename(src) + ".o") for src in srcs]
        with ThreadPoolExecutor(4) as pool:
            list(pool.map(_compile, srcs, objs))
        yield d, objs


def test_sizes_and_checks_at_their_limits_run_clean(objects):
    d, objs = objects
    r = _link_and_run(objs, os.path.join(d, "operators"))
    assert r.returncode == 0, r.stderr[-3000:]
    assert "run clean" in r.stdout
