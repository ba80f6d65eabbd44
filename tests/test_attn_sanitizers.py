"""AddressSanitizer and UndefinedBehaviorSanitizer build of the attention layers' host
code (argument checks, tile planner, workspace sizes), driven on the CPU with stub
kernel launchers (tests/asan/attn_driver.cpp).  Only the host side is instrumented:
device code is never built with a sanitizer."""
import os

import pytest

from test_sanitizers import ASAN_DIR, CLANG, ENV, HIPCC, ROOT, _run


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)), reason="ROCm toolchain not found")
def test_attn_host_code_under_asan(tmp_path):
    csrc = os.path.join(ROOT, "chunked_gated_delta_14_amd", "csrc")
    inc = ["-I", os.path.join(ROOT, "include"), "-I", csrc]
    host_only = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
                 "-Xarch_host", "-fno-omit-frame-pointer"]
    objs = []
    for src in (os.path.join(csrc, "gdr_api.cpp"), os.path.join(csrc, "gdr_attn_api.cpp"),
                os.path.join(ASAN_DIR, "attn_driver.cpp")):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        _run([HIPCC, "--offload-arch=gfx950", "-std=c++17", "-O1", "-g", *host_only, *inc, "-c", src, "-o", obj])
        objs.append(obj)
    exe = str(tmp_path / "attn_asan")
    _run([CLANG, "-fsanitize=address,undefined", *objs, "-L/opt/rocm/lib", "-Wl,-rpath,/opt/rocm/lib", "-lamdhip64", "-o", exe])
    out = _run([exe], env=ENV, timeout=300).stdout
    assert "0 failures, 0 launches" in out
