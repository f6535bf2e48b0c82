"""Launch shapes of the expert-order row operators and the low-rank adapters
over their whole range of sizes, from the library's own launchers built for the
host alone (tests/host_launch/launch_dims.cpp).  Needs no GPU."""
import concurrent.futures as cf
import os
import re
import subprocess

from test_host_sanitize import CSRC, ROOT, _tools

SOURCES = ["hm_api_rows.cpp", "hm_api_lora.cpp", "plan_host.cpp", "k_rows.hip", "k_lora.hip", "k_lora_grad.hip", "k_moe.hip"]


def test_every_accepted_size_is_a_launch_that_can_run(tmp_path):
    hipcc, clang = _tools()
    srcs = [os.path.join(CSRC, f) for f in SOURCES] + [os.path.join(ROOT, "tests", "host_launch", "launch_dims.cpp")]
    objs = [str(tmp_path / (os.path.basename(s) + ".o")) for s in srcs]
    flags = ["-x", "hip", "--cuda-host-only", "--offload-arch=gfx950", "-O1", "-std=c++17",
             "-I", os.path.join(ROOT, "include"), "-I", CSRC]

    def compile_one(pair):
        return pair[0], subprocess.run([hipcc, "-c", pair[0], "-o", pair[1]] + flags, capture_output=True, text=True)

    with cf.ThreadPoolExecutor(4) as ex:
        for src, r in ex.map(compile_one, zip(srcs, objs)):
            assert r.returncode == 0, f"{src}:\n{r.stderr[-3000:]}"
    # no device code was built: the images that the launchers would register are empty
    undefined = subprocess.run(["nm", "-u"] + objs, capture_output=True, text=True).stdout
    images = sorted(set(re.findall(r"__hip_fatbin_\w+", undefined)))
    images_c = tmp_path / "images.c"
    images_c.write_text("".join(f"const char {name}[16] = {{0}};\n" for name in images))
    exe = str(tmp_path / "launch_dims")
    r = subprocess.run([clang, "-o", exe] + objs + ["-x", "c", str(images_c), "-x", "none", "-lstdc++"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "launch shapes ok" in r.stdout
