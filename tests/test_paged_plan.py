"""The attention's plan on the host against the one that its workgroups work out, and the pools' comparison, under AddressSanitizer
and UndefinedBehaviorSanitizer: tests/sanitize/paged_plan_host.cpp takes the place of the launches."""
import os

from gated_delta_rule_45_amd import build as kbuild
from test_sanitizers import ROCM, SAN, SAN_FLAGS, _build, _need, _run, pytestmark  # noqa: F401

import gated_delta_rule_45_amd as kda


def test_paged_plans_under_asan_ubsan(tmp_path):
    _need("g++")
    kda.library()
    exe = str(tmp_path / "paged_plan_host")
    _build(["g++", "-std=c++17", *SAN_FLAGS, "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include", f"-I{kbuild.INCLUDE}",
            f"-I{kbuild.CSRC}", "-Wno-format-truncation", os.path.join(SAN, "paged_plan_host.cpp"),
            os.path.join(kbuild.CSRC, "kda_api.cpp"), os.path.join(kbuild.CSRC, "kda_paged_api.cpp"), f"-L{kbuild.HERE}",
            f"-Wl,-rpath,{kbuild.HERE}", "-l:libkda.so", f"-L{ROCM}/lib", f"-Wl,-rpath,{ROCM}/lib", "-lamdhip64", "-o", exe])
    _run(exe, "4000")
