"""What the attention kernels' sources have to hold where no run shows it: a
missing order between two CTAs' accesses, or a warp that is not converged, goes
well until it does not.  Read from the sources, without a GPU."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mla_attention_prolog_gb300", "csrc")


def code(name, start=None, end=None):
    """A source, or what lies between two of its role headings, without comments."""
    src = open(os.path.join(CSRC, name)).read()
    if start:
        a = src.index(start)
        src = src[a:src.index(end, a)]
    return " ".join(re.sub(r"//[^\n]*", "", src).split())


@pytest.mark.parametrize("name", ["attend_cache8_pair.cu", "attend_cache.cu"])
def test_copies_come_before_the_other_ctas_clears(name):
    """Rows behind a sequence's end are cleared by each CTA of a pair over rows that
    a copy brought, which the even CTA's barrier counted: its arrival at the odd one
    releases, and both looks acquire, at the scope of the cluster."""
    src = code(name)
    at = [m.start() for m in re.finditer(r"map_shared_rank\(smem_u32\(&sh->v_seen\), 1\)", src)]
    assert at
    for a in at:
        assert src[:a].endswith("mbar_arrive_cluster(")
        before = src[:a]
        seen = before.rindex("mbar_acquire_cluster(smem_u32(&sh->v_full[")
        assert seen > before.rindex("look(&sh->v_full[")
    waits = [m.end() for m in re.finditer(r"wait\(&sh->v_seen, tails\)", src)]
    assert waits
    for a in waits:
        behind = src[a:]
        assert behind.index("mbar_acquire_cluster(smem_u32(&sh->v_seen), tails & 1)") < behind.index("st_shared_v4(")
