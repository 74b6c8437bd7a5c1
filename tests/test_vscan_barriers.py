"""Order of the vector-state scan's barrier set-up, read from its source (a
race there shows on no machine, so no run can test it): every mbarrier that a
block's first, relaxed cluster barrier publishes is initialised before the
fence that releases initialisations."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "discrete_selective_ssm_b200", "csrc")
FENCE = "fence.mbarrier_init.release.cluster"


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", ["naju_vscan.cu", "naju_vscan_bwd.cu"])
def test_every_initialisation_is_released(name):
    head = source("naju_vscan.cuh")
    assert head.count(FENCE) == 1  # in mbar_init_release alone
    assert FENCE in re.search(r"void mbar_init_release\(\) \{(.*?)\n\}", head, re.S).group(1)
    text = source(name)
    assert FENCE not in text and text.count("mbar_init_release()") == 1
    release = text.index("mbar_init_release()")
    inits = [m.start() for m in re.finditer(r"\bmbar_init\(|\bex\.init\(", text)]
    declared = re.findall(r"uint64_t (\w+(?:, \w+)*);", text)
    names = [n for d in declared for n in d.split(", ")]
    assert names == ["full", "empty"] and len(inits) == len(names) + 1
    first_sync = text.index("cluster_sync()")
    assert max(inits) < release < first_sync


@pytest.mark.parametrize("name", ["naju_vscan.cu", "naju_vscan_bwd.cu", "naju_vscan.cuh"])
def test_the_status_word_changes_by_atomics_alone(name):
    """A plain store of one block could undo the timeout that another, which
    nothing orders after it, has recorded."""
    text = source(name)
    for m in re.finditer(r"\bp\.status\b", text):
        assert re.search(r"(status_timeout_of\(|atomicOr\(|reinterpret_cast<StatusWord\*>\()$",
                         text[:m.start()]), text[m.start() - 40:m.end() + 20]
