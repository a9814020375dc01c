"""The host code of the router's and the adapters' entry points under
AddressSanitizer and UndefinedBehaviorSanitizer: their sizes over a wide grid
and next to the limits of what they accept (tests/sanitize/operators_host_sanitize.cpp).
The sanitizers are on the host pass only; nothing here touches a GPU."""
import glob
import os
import subprocess
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
    r = _link_and_run(objs, os.path.join(d, "clean"))
    assert r.returncode == 0, r.stderr[-3000:]
    assert "run clean" in r.stdout


def test_the_gpu_tests_reach_every_form_of_the_adapters_projection(objects):
    """The rule that picks a tile goes by costs, so that a change of it can move a
    shape to another form: the shapes of test_gpu_adapter_tiles.py take the ones
    they stand for, and together all that there are."""
    from test_gpu_adapter_tiles import FORMS
    d, objs = objects
    exe = os.path.join(d, "forms")
    _link_and_run(objs, exe)
    got = subprocess.run([exe] + [",".join(map(str, s)) for s in FORMS], capture_output=True, text=True, check=True,
                         env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0")).stdout.split()
    assert [tuple(map(int, g.split(","))) for g in got] == list(FORMS.values())
    assert {f[:2] for f in FORMS.values()} == {(64, 64), (64, 96), (64, 128), (128, 128), (256, 256)}
    assert {(f[0], f[2]) for f in FORMS.values()} == {(64, 64), (64, 128), (128, 128), (256, 256)}
