"""A CTA that gives up a wait must not leave while its own copies are in flight: they would land
in shared memory that is another CTA's by then. The exits cannot be run without a copy that never
comes, so the sources are looked at."""

import os
import re

import pytest

from sparse_mla_attention_gb300 import build


@pytest.mark.parametrize("name", ["k_cache_write.cu", "k_cache_pages.cu"])
def test_a_timed_out_wait_is_followed_by_one_for_the_copies(name):
    with open(os.path.join(build.CSRC, name)) as f:
        text = f.read()
    assert "bulk_load(" in text
    flags = [m.end() for m in re.finditer(r"flag_status\(status, SMLA_ERR_TIMEOUT\);", text)]
    assert flags
    for at in flags:
        left = re.search(r"\b(return|break);", text[at:])
        assert left and "mbar_wait(" in text[at:at + left.start()], \
            f"{name}: the CTA leaves with a copy in flight: {text[at:at + left.end()]!r}"
