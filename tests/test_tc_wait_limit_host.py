"""Every kernel on tcgen05 gets the limit of waits that outlasts its copies in flight."""
import re

from tests.test_source_rules import _sources


def test_tensor_core_kernels_take_their_own_limit():
    found = 0
    for name, src in _sources().items():
        if name.endswith(".cu") and "tcgen05.mma" in src:
            found += 1
            assert re.search(r"\btc_wait_timeout_ns\(\)", src), name
            assert not re.search(r"(?<!tc_)\bwait_timeout_ns\(\)", src), name
    assert found == 2
