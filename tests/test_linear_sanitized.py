"""Host side of linear attention and the state pool under AddressSanitizer and
UBSan: the C entry points' checks, with the host code instrumented."""
import glob
import os

import pytest

from test_sanitized import OUT, PKG, REPORT_MARKERS, ROOT, _cached, _run


def test_checks_under_asan_ubsan():
    from gated_deltanet_recurrence_delta_amd import build as hip_build

    rt = glob.glob("/opt/rocm/lib/llvm/lib/clang/*/lib/linux/libclang_rt.asan-x86_64.so")
    if not rt or not os.path.exists(hip_build.HIPCC):
        pytest.skip("no hipcc / clang sanitizer runtime in this image")
    os.makedirs(OUT, exist_ok=True)
    sources = hip_build.SRCS + glob.glob(os.path.join(PKG, "csrc", "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))
    lib = _cached(os.path.join(OUT, "libgdn_linear_san.so"), sources, lambda t: hip_build.build(out=t, sanitize=True))
    rc, text = _run(["tests/test_linear_host.py", "-k", "not python and not bookkeeping"],
                    {"GDN_LIB_PATH": lib, "LD_PRELOAD": rt[0]})
    assert not any(m in text for m in REPORT_MARKERS), text[-4000:]
    assert rc == 0, text[-4000:]
