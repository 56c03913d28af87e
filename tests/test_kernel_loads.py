"""Every kernel of the library may start before the kernel ahead of it on the
stream has ended, so none may read memory through the read-only path: that is
defined only for memory nobody writes while the reading kernel lives."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "nvfp4_w4a4_quantized_10_b200", "csrc")
FILES = sorted(glob.glob(os.path.join(CSRC, "*")))


@pytest.mark.parametrize("path", FILES, ids=[os.path.basename(f) for f in FILES])
def test_no_load_goes_through_the_read_only_path(path):
    with open(path, encoding="utf-8") as f:
        code = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
    assert not re.search(r"__ldg\b|ld\.global(\.\w+)*\.nc\b", code)
    # a const __restrict__ pointer lets the compiler choose that path for a plain load; the quantizers, which have
    # one, read it by streaming loads alone
    for name in re.findall(r"const \w+\*\s*__restrict__\s+(\w+)", code):
        assert os.path.basename(path) in ("quantize.cu", "mxfp4.cu"), name
