"""Which forms of the tensor-core prefill the library holds (CPU): at head_dim 512 there is none that
walks sinks, so no call can reach one. Form numbers: enum Form of attn_tc.cu."""
import os
import re
import shutil
import subprocess

import pytest

from paged_sliding_window_qkv_gb300 import build

PLAIN, SUMS, SINKS, PART = range(4)


def test_forms_in_the_library():
    if not shutil.which("nm") or not os.path.exists(build.LIB):
        pytest.skip("no nm, or no library built")
    names = subprocess.run(["nm", "-C", build.LIB], capture_output=True, text=True, check=True).stdout
    found = {(int(d), int(f)) for d, f in re.findall(r"attn_tc_kernel<(\d+), \([^)]*\(anonymous namespace\)::Form\)(\d+)>",
                                                     names)}
    assert found == {(256, PLAIN), (256, SINKS), (256, PART), (512, PLAIN), (512, SUMS), (512, PART)}


def test_form_numbers():
    src = open(os.path.join(build.CSRC, "attn_tc.cu")).read()
    assert "enum Form { kPlain, kSums, kSinks, kPart };" in src
