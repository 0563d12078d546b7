"""Host code of rotary positions and of the paged cache under AddressSanitizer and UndefinedBehaviorSanitizer:
tests/sanitize/paged_host.cpp drives their entry points (refusals, empty problems, a seeded fuzz over edge-valued problem
fields) and the quotients that the kernels take by multiplication; the kernel side comes from libkda.so and is never reached."""
import os

from gated_delta_rule_45_amd import build as kbuild
from test_sanitizers import ROCM, SAN, SAN_FLAGS, _build, _need, _run, pytestmark  # noqa: F401

import gated_delta_rule_45_amd as kda


def test_paged_host_code_under_asan_ubsan(tmp_path):
    _need("g++")
    kda.library()
    exe = str(tmp_path / "paged_host")
    _build(["g++", "-std=c++17", *SAN_FLAGS, "-D__HIP_PLATFORM_AMD__", f"-I{ROCM}/include", f"-I{kbuild.INCLUDE}",
            f"-I{kbuild.CSRC}", "-Wno-format-truncation", os.path.join(SAN, "paged_host.cpp"),
            os.path.join(kbuild.CSRC, "kda_api.cpp"), os.path.join(kbuild.CSRC, "kda_paged_api.cpp"), f"-L{kbuild.HERE}",
            f"-Wl,-rpath,{kbuild.HERE}", "-l:libkda.so", f"-L{ROCM}/lib", f"-Wl,-rpath,{ROCM}/lib", "-lamdhip64", "-o", exe])
    _run(exe, "20000")
