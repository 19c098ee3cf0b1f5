"""A kernel that divides its registers among its warps is not launched when it was compiled to others than it counts on, and the
error says so: host code, linked from the library's own objects."""
import os
import shutil
import subprocess

import pytest

from backward_adapter_gb300 import build as fbuild

MAIN = """
#include <cstdio>
#include "fa_check.h"
int main() {
  for (int got : {96, 88, 104}) {
    fa::clear_error();
    const fa_status st = fa::check_split("some launch", got, 96);
    std::printf("%d %s\\n", (int)st, fa_last_error());
  }
}
"""


def test_another_register_count_is_refused_with_its_reason(tmp_path):
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    fbuild.build()
    (tmp_path / "main.cu").write_text(MAIN)
    objects = [os.path.join(fbuild.BUILD, os.path.basename(s)[:-3] + ".o") for s in fbuild.sources()]
    exe = str(tmp_path / "main")
    subprocess.run([fbuild._nvcc(), "-std=c++17", "-I", fbuild.CSRC, "-I", os.path.join(fbuild.ROOT, "include"), str(tmp_path / "main.cu"),
                    *objects, "-o", exe], check=True)
    lines = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.splitlines()
    assert lines[0].strip() == "0"
    for line, got in zip(lines[1:], (88, 104)):
        status, text = line.split(" ", 1)
        assert status == "2" and text.startswith("some launch") and f"{got} registers" in text and "divide 96" in text
