"""The host code of the expert-order row operators and the low-rank adapters
(argument checks, planning, workspace layout) built with AddressSanitizer and
UndefinedBehaviorSanitizer for the host side only and swept over 200000 drawn
calls with checking stand-ins of the kernel launchers
(tests/host_sanitize/rows_lora_sweep.cpp).  Needs no GPU."""
import concurrent.futures as cf
import os
import subprocess

from test_host_sanitize import CSRC, HERE, HOST_SAN, ROCM, ROOT, _tools


def test_rows_and_lora_host_code_under_asan_ubsan(tmp_path):
    hipcc, clang = _tools()
    srcs = [os.path.join(CSRC, f) for f in ("hm_api_rows.cpp", "hm_api_lora.cpp", "plan_host.cpp")]
    srcs.append(os.path.join(HERE, "rows_lora_sweep.cpp"))
    objs = [str(tmp_path / (os.path.basename(s) + ".o")) for s in srcs]
    flags = ["-x", "hip", "--offload-arch=gfx950", "-O1", "-g", "-std=c++17",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-I", os.path.join(ROOT, "include"), "-I", CSRC] + HOST_SAN

    def compile_one(pair):
        return pair[0], subprocess.run([hipcc, "-c", pair[0], "-o", pair[1]] + flags, capture_output=True, text=True)

    with cf.ThreadPoolExecutor(4) as ex:
        for src, r in ex.map(compile_one, zip(srcs, objs)):
            assert r.returncode == 0, f"{src}:\n{r.stderr[-3000:]}"
    exe = str(tmp_path / "rows_lora_sweep")
    link = [clang, "-fsanitize=address,undefined", "-o", exe] + objs + [
        "-L", os.path.join(ROCM, "lib"), "-lamdhip64", f"-Wl,-rpath,{os.path.join(ROCM, 'lib')}"]
    r = subprocess.run(link, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=0:halt_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-6000:]
    assert "sweep ok" in r.stdout
    assert "runtime error" not in out and "AddressSanitizer" not in out, out[-6000:]
