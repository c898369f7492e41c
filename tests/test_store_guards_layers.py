"""Every global store of the scored router, the norm and the epilogue's gradient is
guarded by the addresses that it writes (CPU only, on the sources)."""
import os

import pytest

from tests.test_store_guards import CSRC, unguarded


@pytest.mark.parametrize("name,least", [("gate_group.cu", 5), ("norm.cu", 6), ("epilogue_grad.cu", 6)])
def test_stores_are_guarded_by_address(name, least):
    with open(os.path.join(CSRC, name)) as f:
        found, bad = unguarded(f.read())
    assert found >= least and not bad, (found, bad)
