"""The host side of the key/value-cache entry points under AddressSanitizer
and UndefinedBehaviorSanitizer, with the stand-ins of test_sanitizers.py:
tests/sanitize/kv_driver.c drives validation and launch shapes with valid,
invalid and extreme arguments.  No GPU."""
import os
import re

import pytest

from test_sanitizers import (CLANG, CLANGXX, CSRC, ENV, HIPCC, ROCM, ROOT, SAN_DIR, SAN_FLAGS,
                             _have, _run)


@pytest.mark.skipif(not _have(HIPCC, CLANG, CLANGXX), reason="ROCm compilers not found")
def test_kv_host_side_under_asan_ubsan(tmp_path):
    objs = []
    for f in ("api.hip", "kv_api.hip", "kv_plan.hip", "qk_rope.hip", "kv_cache.hip", "kv_attention.hip",
              "amax.hip", "quantize.hip", "dequantize.hip", "fakequant.hip", "requant.hip", "rht.hip"):
        o = str(tmp_path / (f[:-4] + ".o"))
        cmd = [HIPCC, "--offload-host-only", "-std=c++17", "-fPIC", "-c", os.path.join(CSRC, f),
               "-o", o, "-fno-omit-frame-pointer", "-g", "-O1"]
        if f.startswith(("kv_", "qk_")) or f == "api.hip":
            for flag in SAN_FLAGS[:3]:
                cmd += ["-Xarch_host", flag]
        _run(cmd)
        objs.append(o)
    nm = _run(["nm", "-u"] + objs).stdout
    fatbins = sorted(set(re.findall(r"__hip_fatbin_[0-9a-f]+", nm)))
    fb_c = tmp_path / "fatbins.c"
    fb_c.write_text("".join(f"const unsigned char {s}[16] = {{0}};\n" for s in fatbins))
    inc = ["-std=c11", "-D__HIP_PLATFORM_AMD__", "-I" + os.path.join(ROOT, "include"),
           "-I" + os.path.join(ROCM, "include")]
    extra = []
    for src, flags in ((str(fb_c), []), (os.path.join(SAN_DIR, "hip_runtime_stubs.c"), ["-std=c11"]),
                       (os.path.join(SAN_DIR, "kv_driver.c"), inc)):
        o = str(tmp_path / (os.path.basename(src)[:-2] + ".o"))
        _run([CLANG] + SAN_FLAGS + flags + ["-c", src, "-o", o])
        extra.append(o)
    exe = str(tmp_path / "kv_driver")
    _run([CLANGXX] + SAN_FLAGS + ["-o", exe] + extra + objs)
    r = _run([exe], env=ENV, timeout=600)
    assert "every status as expected" in r.stdout
