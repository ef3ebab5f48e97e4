"""AddressSanitizer and UndefinedBehaviorSanitizer build of the attention layer's host code, on the CPU: attn_api.cpp
rebuilt with both (g++), linked with the objects of the last build and run under a driver that sends every entry point
arguments that fail validation, the empty calls, and sizes up to the limits (tests/sanitize/attn_abi_driver.cpp).  No call
reaches a kernel."""
import os
import shutil

import pytest

from test_sanitizers import ENV, ROCM, ROOT, SAN, _run

pytestmark = pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists(os.path.join(ROCM, "lib", "libamdhip64.so")),
                                reason="g++ or the HIP runtime not found")


def test_attn_abi_layer_under_asan_ubsan(tmp_path):
    from linear_attention_sequence_gated_amd import build as gbuild
    objs = [os.path.join(gbuild.OBJDIR, os.path.splitext(s)[0] + ".o") for s in gbuild.SOURCES if s != "attn_api.cpp"]
    if not all(os.path.exists(o) for o in objs):
        gbuild.build()
    api, drv, exe = (str(tmp_path / n) for n in ("attn_api.o", "driver.o", "attn_asan"))
    inc = ["-I", os.path.join(ROOT, "include")]
    _run(["g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROCM, "include")] + inc + SAN +
         ["-c", os.path.join(ROOT, "linear_attention_sequence_gated_amd", "csrc", "attn_api.cpp"), "-o", api])
    _run(["g++", "-std=c++17"] + inc + SAN + ["-c", os.path.join(ROOT, "tests", "sanitize", "attn_abi_driver.cpp"), "-o", drv])
    _run(["g++"] + SAN + [drv, api] + objs +
         ["-L", os.path.join(ROCM, "lib"), "-lamdhip64", "-Wl,-rpath," + os.path.join(ROCM, "lib"), "-o", exe])
    assert "all checks passed" in _run([exe], env=ENV).stdout
