"""Selection's use of shared memory across threads, checked on the source: what one
thread writes behind the last barrier of `cut` (csrc/beam.cu) no other touches
before the next one.  `finish` and `settle` go on from there."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_flashattention_gb300", "csrc")
BARRIER = "__syncthreads();"


def body(name):
    """The text of a member function of Chooser, without comments."""
    s = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "beam.cu")).read())
    s = s[s.index("struct Chooser {"):]
    s = s[s.index("{", re.search(r"\b%s\([^)]*\) \{" % name, s).start()):]
    depth = 0
    for i, c in enumerate(s):
        depth += (c == "{") - (c == "}")
        if depth == 0:
            return s[:i + 1]


def words(text):
    return set(re.findall(r"\bsh\.(\w+)", text))


@pytest.mark.parametrize("after", ["finish", "settle"])
def test_no_word_is_written_and_used_without_a_barrier(after):
    tail = body("cut").rsplit(BARRIER, 1)[1]
    written = set(re.findall(r"\bsh\.(\w+)(?:\[[^]]*\])? [-+]?= ", tail))
    assert "dropped" in written                      # (else this test looks at the wrong place)
    follows = body(after)
    follows = follows[follows.index("cut("):].split(BARRIER, 1)[0]
    # thread 0's own accesses are in order
    follows = re.sub(r"if \(threadIdx\.x == 0\)[^;]*;", "", follows)
    assert not written & words(follows)
