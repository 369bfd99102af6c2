"""The validation of include/fp8q_ops.h under AddressSanitizer and
UndefinedBehaviorSanitizer on the host (no GPU): the host code of ops_api.hip
linked with launcher stand-ins that abort if reached, and a driver whose
every call must be refused."""
import os

import pytest

from test_sanitize_cpu import ENV, HIPCC, ROOT, SAN, _run


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not found")
def test_ops_validation_under_asan_and_ubsan(tmp_path):
    san = ["-Xarch_host", "-fsanitize=address,undefined", "-Xarch_host", "-fno-sanitize-recover=all",
           "-Xarch_host", "-fno-omit-frame-pointer"]
    flags = ["-O1", "-g", "-std=c++17", "-Wno-unused-command-line-argument"]
    objs = []
    for src in (os.path.join(ROOT, "fp8_precision_quant_amd", "csrc", "ops_api.hip"),
                os.path.join(SAN, "ops_stubs.cpp"), os.path.join(SAN, "ops_driver.cpp")):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        _run([HIPCC, "--cuda-host-only", *flags, *san, "-c", src, "-o", obj], cwd=str(tmp_path))
        objs.append(obj)
    exe = str(tmp_path / "ops_driver")
    _run([HIPCC, *san, *objs, "-o", exe], cwd=str(tmp_path))
    r = _run([exe], cwd=str(tmp_path), env=ENV, timeout=120)
    assert "all validation cases passed" in r.stdout
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr
