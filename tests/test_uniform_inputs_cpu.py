"""Device values that barriers depend on: a caller who rewrites them on another stream while the
kernel runs must not make a block's threads disagree about a barrier.  (Shown by the sources: a
kernel in which they disagree may never end.)"""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "linear_attention_08_b200", "csrc")


def source(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def test_multi_token_decode_decides_together():
    text = source("kda_decode_multi_tc.cu")
    loop = text[text.index("for (; u < units; u += G)"):]
    assert "const bool keep = __syncthreads_or(a >= 0);" in loop
    assert not re.search(r"if \(a [<>=]+ 0\)", loop)      # (selects of values are fine)


def test_commit_decides_together():
    text = source("kda_tree_commit.cu")
    loop = text[text.index("for (; item < items; item += G)"):]
    assert loop.count("more = __syncthreads_or(__popcll(path) > kGroup);") == 2
    steps = loop[loop.index("for (;;) {"):loop.index("float4 *dst")]
    assert steps.count("__syncthreads") == 2 and re.search(r"if \(!more\) break;", steps)
    assert "if (active)" in steps and "if (active)" not in steps[:steps.rindex("__syncthreads_or")]
