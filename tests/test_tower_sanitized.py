"""The tower operators' host-side checks under AddressSanitizer and UndefinedBehaviorSanitizer (CPU
only), as tests/test_abi_sanitized.py does for the core's: the library's sources compiled with the
sanitizers on their host code, linked with tests/native/tower_sanitized.cpp."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
SAN = ["-Xarch_host", "-fsanitize=address",
       "-Xarch_host", "-fsanitize=undefined",
       "-Xarch_host", "-fno-sanitize-recover=all",
       "-Xarch_host", "-fno-omit-frame-pointer"]
SOURCES = ("abi", "act_dropout", "dense_epi", "group_norm")  # the entry points and what they call
NEEDED_BY_ABI = ("calib", "cat_interact", "dot_interact", "emb_bag_fwd", "emb_dot_fwd", "grad_sort", "grad_update")


def test_tower_checks_run_clean_under_sanitizers(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    csrc = os.path.join(ROOT, "embedding_lookup_feature_amd", "csrc")
    inc = ["-I", os.path.join(ROOT, "include"), "-I", csrc]
    common = ["-O1", "-g", "-std=c++17", "-fPIC", "--offload-arch=gfx950",
              "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"] + inc
    procs, objs = [], []
    for name in SOURCES + NEEDED_BY_ABI:
        obj = str(tmp_path / (name + ".o"))
        objs.append(obj)
        cmd = [HIPCC, *common, *SAN, "-c", os.path.join(csrc, name + ".hip"), "-o", obj]
        procs.append(subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT))
    for p in procs:
        out, _ = p.communicate()
        assert p.returncode == 0, out.decode(errors="replace")[-3000:]
    drv = str(tmp_path / "drv.o")
    subprocess.run([HIPCC, "-O1", "-g", "-std=c++17", *SAN, *inc, "-c", os.path.join(HERE, "native", "tower_sanitized.cpp"),
                    "-o", drv], check=True)
    exe = str(tmp_path / "tower_sanitized")
    subprocess.run([HIPCC, "--offload-arch=gfx950", *SAN, *objs, drv, "-o", exe], check=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0")  # the HIP runtime's own allocations
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout[-3000:] + r.stderr[-3000:]
    assert "runtime error" not in r.stderr and "Sanitizer" not in r.stderr, r.stderr[-3000:]
