"""The host side of a tensor list (tiles, launches, offsets, workspace) under
AddressSanitizer and UndefinedBehaviorSanitizer on the CPU: the driver in
tests/sanitize/list_driver.cpp checks the invariants its kernels rely on."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SAN = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer"]
ENV = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:verify_asan_link_order=0:abort_on_error=0",
           UBSAN_OPTIONS="print_stacktrace=1")


def test_list_plans_under_sanitizers(tmp_path):
    src = os.path.join(ROOT, "sharded_mixed_precision_amd", "csrc")
    exe = str(tmp_path / "list_driver")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-g", *SAN, "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"),
                        "-I", src, "-I", "/opt/rocm/include", os.path.join(src, "mapper.cpp"), os.path.join(src, "list.cpp"),
                        os.path.join(ROOT, "tests", "sanitize", "list_driver.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, env=ENV, timeout=600)
    assert r.returncode == 0, (r.stdout[-500:], r.stderr[-3000:])
    assert "AddressSanitizer" not in r.stderr and "runtime error" not in r.stderr, r.stderr[-3000:]
    lines = r.stdout.splitlines()
    assert lines[-1] == "ok" and len(lines) > 100
