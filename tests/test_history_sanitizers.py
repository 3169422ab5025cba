"""The host-side tests of the event-history calls on a library whose host code is built with the address and
undefined-behaviour sanitizers, in a child interpreter with the sanitizer runtime loaded first."""
import os
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CHILD = """
import sys
sys.path[:0] = [{root!r}, {here!r}]
import pytest
import dlrm_embedding_interaction_amd as dl
dl.LIBRARY = {lib!r}
sys.exit(int(pytest.main(["-q", "-s", "-p", "no:cacheprovider", *{tests!r}])))
"""


def test_history_abi_under_address_and_undefined_behaviour_sanitizers():
    import test_sanitizers as ts
    from dlrm_embedding_interaction_amd import _build
    try:
        cc = _build.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not found")
    rt = ts._clang_asan_runtime(cc)
    if not rt:
        pytest.skip("clang AddressSanitizer runtime not found next to hipcc")
    tests = [os.path.join(HERE, f) for f in ("test_history_abi.py", "test_history_limits.py")]
    code = CHILD.format(root=ROOT, here=HERE, lib=ts._sanitized_library(), tests=tests)
    r = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, LD_PRELOAD=rt, **ts.SAN_ENV),
                       capture_output=True, text=True, timeout=600)
    if r.returncode != 0:
        pytest.fail(f"sanitized run exited {r.returncode}\n{r.stdout[-3000:]}\n{r.stderr[-6000:]}")
    assert "passed" in r.stdout
