"""The host code of the 8-bit integer layers (argument checks, planning,
workspace layout, launch shapes), built for the host alone, plainly and with
AddressSanitizer and UndefinedBehaviorSanitizer, and swept over their whole range of sizes
(tests/host_launch/int8_sweep.cpp).  Needs no GPU."""
import concurrent.futures as cf
import os
import re
import subprocess

import pytest

from test_host_sanitize import CSRC, HOST_SAN, ROOT, _tools

SOURCES = ["hm_api_i8.cpp", "k_i8_rows.hip", "k_i8_tile.hip", "k_i8_big.hip", "k_i8_few.hip", "k_i8_few_dx.hip"]


@pytest.mark.parametrize("san", [False, True])
def test_every_accepted_size_is_a_launch_that_can_run(tmp_path, san):
    hipcc, clang = _tools()
    srcs = [os.path.join(CSRC, f) for f in SOURCES] + [os.path.join(ROOT, "tests", "host_launch", "int8_sweep.cpp")]
    objs = [str(tmp_path / (os.path.basename(s) + ".o")) for s in srcs]
    flags = ["-x", "hip", "--cuda-host-only", "--offload-arch=gfx950", "-O1", "-std=c++17",
             "-I", os.path.join(ROOT, "include"), "-I", CSRC]
    # (kernels are launched through pointers, which are handles on the host: no check of function types)
    ubsan = ["-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize=function", "-Xarch_host", "-fno-sanitize-recover=all"]

    def compile_one(pair):
        more = [] if not san else ubsan if pair[0].endswith(".hip") else HOST_SAN
        return pair[0], subprocess.run([hipcc, "-c", pair[0], "-o", pair[1]] + flags + more, capture_output=True, text=True)

    with cf.ThreadPoolExecutor(4) as ex:
        for src, r in ex.map(compile_one, zip(srcs, objs)):
            assert r.returncode == 0, f"{src}:\n{r.stderr[-3000:]}"
    # no device code was built: the images that the launchers would register are empty
    undefined = subprocess.run(["nm", "-u"] + objs, capture_output=True, text=True).stdout
    images = sorted(set(re.findall(r"__hip_fatbin_\w+", undefined)))
    images_c = tmp_path / "images.c"
    images_c.write_text("".join(f"const char {name}[16] = {{0}};\n" for name in images))
    exe = str(tmp_path / "int8_sweep")
    r = subprocess.run([clang] + (["-fsanitize=address,undefined"] if san else []) + ["-o", exe] + objs + ["-x", "c", str(images_c), "-x", "none", "-lstdc++"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:halt_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600, env=env)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "int8 sweep ok" in r.stdout
    assert "runtime error" not in out and "AddressSanitizer" not in out, out[-4000:]
