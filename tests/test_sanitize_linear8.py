"""The host code of the 8-bit linear layer's six calls (argument checks, plans,
workspace arithmetic) under AddressSanitizer and UndefinedBehaviorSanitizer.

api.hip, quant8.hip and linear8.hip are compiled for the host only, with every
sanitizer flag on the host side only, and linked ahead of libsg.so with the
driver tests/abi_sanitize_linear8.cpp, in which no call reaches a launch.
"""

import os
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIBDIR = os.path.join(ROOT, "post_pruning_amd")
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"

pytestmark = pytest.mark.skipif(
    not (os.path.exists(HIPCC) and os.path.exists(os.path.join(LIBDIR, "libsg.so"))),
    reason="hipcc or libsg.so missing")

SAN = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
       "-Xarch_host", "-fno-sanitize-recover=undefined", "-Xarch_host", "-fno-omit-frame-pointer"]


def _run(cmd, **kw):
    res = subprocess.run(cmd, capture_output=True, text=True, **kw)
    assert res.returncode == 0, f"{' '.join(cmd)}\n{res.stdout}\n{res.stderr}"
    return res


def test_linear8_host_layer_sanitized(tmp_path):
    inc = "-I" + os.path.join(ROOT, "include")

    def compile_(src):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        lang = ["--offload-arch=gfx950", "--offload-host-only"] if src.endswith(".hip") else ["-x", "c++"]
        _run([HIPCC, "-std=c++17", "-O1", "-g", *lang, "-fPIC", *SAN, inc, src, "-c", "-o", obj])
        return obj

    srcs = [os.path.join(LIBDIR, "csrc", f) for f in ("api.hip", "quant8.hip", "linear8.hip")]
    with ThreadPoolExecutor(4) as ex:
        objs = list(ex.map(compile_, [*srcs, os.path.join(ROOT, "tests", "abi_sanitize_linear8.cpp")]))
    exe = str(tmp_path / "drv")
    _run([HIPCC, *SAN, "-rdynamic", "-Wl,--unresolved-symbols=ignore-in-object-files", *objs, "-L" + LIBDIR, "-lsg", "-Wl,-rpath," + LIBDIR, "-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1", HIP_VISIBLE_DEVICES="")
    assert "linear8 host checks passed" in _run([exe], env=env, timeout=120).stdout
