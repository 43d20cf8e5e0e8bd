"""The residual block's host-side checks under AddressSanitizer and UndefinedBehaviorSanitizer (CPU
only), as tests/test_tower_sanitized.py does for the tower's: the library's sources compiled with the
sanitizers on their host code, linked with tests/native/block_sanitized.cpp."""
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from tests.test_tower_sanitized import HERE, HIPCC, NEEDED_BY_ABI, ROOT, SAN, SOURCES

BLOCK = ("block_norm", "ckpt", "dense_ckpt", "dense_fp4")  # the entry points
# kernels and their launches, many: linked as the library's build left them where it did
KERNELS = ("block_norm_fwd_f32", "block_norm_fwd_f16", "block_norm_fwd_bf16", "block_norm_bwd_f32", "block_norm_bwd_f16",
           "block_norm_bwd_bf16")


def test_block_checks_run_clean_under_sanitizers(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    csrc = os.path.join(ROOT, "embedding_lookup_feature_amd", "csrc")
    inc = ["-I", os.path.join(ROOT, "include"), "-I", csrc]
    common = ["-O1", "-g", "-std=c++17", "-fPIC", "--offload-arch=gfx950",
              "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"] + inc

    def compile_one(name):
        built = os.path.join(ROOT, "embedding_lookup_feature_amd", "_build", name + ".o")
        if name in KERNELS and os.path.exists(built):
            return built
        obj = str(tmp_path / (name + ".o"))
        r = subprocess.run([HIPCC, *common, *SAN, "-c", os.path.join(csrc, name + ".hip"), "-o", obj], stdout=subprocess.PIPE,
                           stderr=subprocess.STDOUT)
        assert r.returncode == 0, r.stdout.decode(errors="replace")[-3000:]
        return obj

    with ThreadPoolExecutor(8) as pool:
        objs = list(pool.map(compile_one, BLOCK + KERNELS + SOURCES + NEEDED_BY_ABI))
    drv = str(tmp_path / "drv.o")
    subprocess.run([HIPCC, "-O1", "-g", "-std=c++17", *SAN, *inc, "-c", os.path.join(HERE, "native", "block_sanitized.cpp"),
                    "-o", drv], check=True)
    exe = str(tmp_path / "block_sanitized")
    subprocess.run([HIPCC, "--offload-arch=gfx950", *SAN, *objs, drv, "-o", exe], check=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0")  # the HIP runtime's own allocations
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout[-3000:] + r.stderr[-3000:]
    assert "runtime error" not in r.stderr and "Sanitizer" not in r.stderr, r.stderr[-3000:]
