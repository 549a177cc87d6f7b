"""What the decode calls' kernels must do where it cannot be run: a look at another CTA's shared memory before that CTA
has started would fault, and a copy that never comes is not to be had. The sources are looked at."""

import os
import re

import pytest

from sparse_mla_attention_gb300 import build


def _source(name):
    with open(os.path.join(build.CSRC, name)) as f:
        return f.read()


def _depth(text):
    """How many braces are open at the end of text."""
    return text.count("{") - text.count("}")


def test_evictions_clusters_meet_before_they_write_to_each_other():
    text = _source("k_cache_evict.cu")
    body = text[text.index("__device__ void choose("):]
    body = body[body.index("{"):body.index("\n}\n")]
    # the lambda that joins a CTA or a cluster is no barrier yet
    remote = re.search(r"map_shared_rank\(", body).start()
    meet = [m.start() for m in re.finditer(r"\n    if \(kParts > 1\) cl\.sync\(\);", body)]
    assert meet and meet[0] < remote, "a CTA looks at another's shared memory that may not have started"
    # in every sequence: not within a branch or a loop
    assert _depth(body[:meet[0]]) == 1


def test_a_weights_cta_that_gave_up_leaves_after_its_loads():
    # any warp may give up, also when the loading ones are done: they wait once all warps are out of their loops
    text = _source("k_cache_weights.cu")
    for kernel, bars in (("weights_kernel", ("full", "q_full", "f_full")), ("weights_resident_kernel", ("full", "q_full"))):
        body = text[re.search(r"\n%s\(" % kernel, text).start():]
        body = body[:body.index("\n}\n")]
        out = body.rindex("__syncthreads();")
        for bar in bars:
            waits = [m.start() for m in re.finditer(r"mbar_wait\(&sh\.%s\[" % bar, body)]
            assert waits and min(waits) > out, f"{kernel}: a copy of {bar} may be in flight when the CTA leaves"
        assert "sh.abort_flag" in body[out:]


@pytest.mark.parametrize("name", ["k_fwd_paged.cu", "k_fwd_tc.cu", "k_attn_tc.cu"])
def test_a_loading_warp_waits_for_its_loads_whoever_gives_up(name):
    # not only where a wait has run out already: another warp's may, once this one has left its loop
    text = _source(name)
    waits = [m.start() for m in re.finditer(r"mbar_wait\(&sh\.(full|q_full)\[", text)]
    assert waits
    for at in waits:
        before = text[max(0, at - 600):at]
        guard = before.rfind("if (sh.abort_flag)")
        assert guard < 0 or _depth(before[guard:]) < 0, f"{name}: {text[at - 200:at + 60]!r}"
