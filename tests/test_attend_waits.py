"""Bounded waits of the attention kernels, read from their sources: no GPU waits
in vain for this, and none is made to."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mla_attention_prolog_gb300", "csrc")


def statements(name, start, end):
    """The code between two of a kernel's role headings, without comments, split
    at semicolons and braces."""
    src = open(os.path.join(CSRC, name)).read()
    a = src.index(start)
    code = re.sub(r"//[^\n]*", "", src[a:src.index(end, a)])
    return [" ".join(s.split()) for s in re.split(r"[;{}]", code) if s.strip()]


LEAVES = re.compile(r"if \(!ok\) (continue|break)|if \(named_bar_or\(1, 128, (grow \|\| )?!ok\)\)|if \(!__all_sync\(~0u, ok\)\)|"
                    r"if \(ok && rows\)|if \(kSplit\)|const bool all = named_bar_and|ok = __all_sync\(~0u, ok")
EFFECT = re.compile(r"\b(tmem_st16(_raw)?|st_shared_v4|arrive|mbar_arrive|clean_v)\(")


@pytest.mark.parametrize("name,start,end", [
    ("attend_cache.cu", "- softmax\n", " MMA (the even CTA's"), ("attend_prompt.cu", "- softmax\n", "- MMA\n")])
def test_a_failed_wait_of_the_softmax_warps_stays_failed(name, start, end):
    """A wait that gave up is not forgotten when a later one succeeds, and what
    depends on it (O rescaled, P overwritten, rows cleared, the arrival that
    hands them over) is not done."""
    code = statements(name, start, end)
    waits = [i for i, s in enumerate(code) if re.search(r"\bok = ", s) and "wait(" in s]
    assert len(waits) >= 4
    for i in waits:
        leaves = next(j for j in range(i + 1, len(code)) if LEAVES.search(code[j]))
        done = [s for s in code[i + 1:leaves] if EFFECT.search(s)]
        assert not done, f"after `{code[i]}`: {done}"
        kept = re.search(r"\bok &&", code[i]) or not LEAVES.search(code[leaves]).group(0).startswith("if (named_bar_or(1, 128, grow")
        assert kept, f"`{code[i]}` forgets an earlier wait"
