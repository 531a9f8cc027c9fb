"""Every kernel launch's own error code is read before anything follows it: a
launch that was refused must not let the kernels after it run on what it should
have written, nor leave its error to a later, unrelated call."""
import glob
import os
import re

import pytest

from quantized_recurrent_state_lq_b200 import build

FILES = sorted(glob.glob(os.path.join(build.CSRC, "*.cu")) + glob.glob(os.path.join(build.CSRC, "*.cuh")))


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_every_launch_is_followed_by_its_error(path):
    text = re.sub(r"//[^\n]*", "", open(path).read())
    for m in re.finditer(r"<<<", text):
        end = text.index(";", text.index(">>>", m.end()))
        after = text[end + 1:].lstrip()
        line = text.count("\n", 0, m.start()) + 1
        # the next statement (the else branch's launch is a match of its own)
        assert re.match(r"(else\s+[^;]*<<<|return cudaGetLastError\(\);|e = cudaGetLastError\(\);[\s}]*(if \()?"
                        r"(const cudaError_t f = [^;]*;\s*return )?e [!=]= cudaSuccess)",
                        after), \
            f"{os.path.basename(path)}:{line}: launch not checked: {after[:60]!r}"
