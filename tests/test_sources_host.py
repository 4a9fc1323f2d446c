"""What the CUDA sources must not contain. Every kernel of the library is launched while the one before it may still run
(programmatic dependent launch), so nothing that it reads is constant for as long as its grid lives."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "decode_attention_mfa_gb300", "csrc")
SOURCES = sorted(f for f in glob.glob(os.path.join(CSRC, "*")) if f.endswith((".cu", ".cuh", ".h", ".hpp")))


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_loads_through_the_non_coherent_path(path):
    """__ldg and ld.global.nc may return what a line held before an earlier kernel of the stream wrote it."""
    code = re.sub(r"//[^\n]*", "", open(path).read())
    assert not re.search(r"__ldg\s*\(|ld\.global(\.\w+)*\.nc\b", code)
