"""The launches of the 8-bit integer layers cover their call's output exactly
(tests/host_launch/int8_cover.cpp), and the check fails where one does not.  Needs no GPU."""
import concurrent.futures as cf
import os
import re
import subprocess

import pytest

from test_host_int8_sweep import SOURCES
from test_host_sanitize import CSRC, ROOT, _tools


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    hipcc, clang = _tools()
    tmp = tmp_path_factory.mktemp("int8_cover")
    srcs = [os.path.join(CSRC, f) for f in SOURCES] + [os.path.join(ROOT, "tests", "host_launch", "int8_cover.cpp")]
    objs = [str(tmp / (os.path.basename(s) + ".o")) for s in srcs]
    flags = ["-x", "hip", "--cuda-host-only", "--offload-arch=gfx950", "-O1", "-std=c++17",
             "-I", os.path.join(ROOT, "include"), "-I", CSRC]
    with cf.ThreadPoolExecutor(4) as ex:
        for src, r in zip(srcs, ex.map(lambda p: subprocess.run([hipcc, "-c", p[0], "-o", p[1]] + flags, capture_output=True, text=True),
                                       zip(srcs, objs))):
            assert r.returncode == 0, f"{src}:\n{r.stderr[-3000:]}"
    # no device code was built: the images that the launchers would register are empty
    undefined = subprocess.run(["nm", "-u"] + objs, capture_output=True, text=True).stdout
    images = tmp / "images.c"
    images.write_text("".join(f"const char {name}[16] = {{0}};\n" for name in sorted(set(re.findall(r"__hip_fatbin_\w+", undefined)))))
    out = str(tmp / "int8_cover")
    r = subprocess.run([clang, "-o", out] + objs + ["-x", "c", str(images), "-x", "none", "-lstdc++"], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    return out


def test_launches_cover_the_output(exe):
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "int8 cover ok" in r.stdout, (r.stdout + r.stderr)[-2000:]


@pytest.mark.parametrize("kernel", ["k_i8_few", "k_i8_few_dx", "k_i8_tile", "k_i8_finish", "k_i8_big", "k_i8_copies", "k_i8_quant_rows"])
def test_a_short_launch_is_seen(exe, kernel):
    r = subprocess.run([exe, kernel], capture_output=True, text=True, timeout=300)
    assert r.returncode == 1 and "check failed" in r.stdout, (r.stdout + r.stderr)[-2000:]
