"""A kernel's set-up per device, when several host threads make its first call
at the same time (no GPU: device_setup_host.cpp compiles the header alone)."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "long_context_mask_gb300", "csrc")


def build(tmp_path, *flags):
    exe = str(tmp_path / "setup")
    r = subprocess.run(["g++", "-O1", "-std=c++17", "-pthread", *flags, "-I", CSRC,
                        os.path.join(ROOT, "tests", "device_setup_host.cpp"), "-o", exe], capture_output=True, text=True)
    return exe, r


@pytest.mark.parametrize("flags", [(), ("-fsanitize=thread", "-g")])
def test_first_calls_of_many_threads(tmp_path, flags):
    exe, r = build(tmp_path, *flags)
    if flags and r.returncode:
        pytest.skip("no thread sanitizer")
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    if flags and "unexpected memory mapping" in r.stderr:
        pytest.skip("the thread sanitizer does not run here")
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout + r.stderr


@pytest.mark.parametrize("name", ["bsa_paged.cu", "bsa_paged_attn.cu", "bsa_paged_select.cu"])
def test_paged_launches_set_up_through_it(name):
    """A plain static flag beside plain static values has no order between threads."""
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        src = f.read()
    assert not re.findall(r"static int (?:done|ready)\b", src)
    inside = "".join(re.findall(r"\.once\(dev, \[&\] \{(.*?)\n    \}\)", src, flags=re.S))
    for call in ("cudaFuncSetAttribute(", "cudaDeviceGetAttribute("):
        assert src.count(call) == inside.count(call)
