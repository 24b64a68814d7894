"""Host replay of the launches of dropout and of the linear layer in 8-bit
floating point: tests/f8_launches.cpp, linked ahead of the HIP runtime, takes
the library's kernel launches and replays the addresses of their threads
against the operands' extents.  No GPU is needed and no kernel runs."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIBDIR = os.path.join(ROOT, "post_pruning_amd")
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"

pytestmark = pytest.mark.skipif(
    not (os.path.exists(HIPCC) and os.path.exists(os.path.join(LIBDIR, "libsg.so"))),
    reason="hipcc or libsg.so missing")


def _run(cmd, **kw):
    res = subprocess.run(cmd, capture_output=True, text=True, **kw)
    assert res.returncode == 0, f"{' '.join(cmd)}\n{res.stdout}\n{res.stderr}"
    return res


@pytest.fixture(scope="module")
def replay(tmp_path_factory):
    d = tmp_path_factory.mktemp("replay")
    obj, exe = str(d / "replay.o"), str(d / "replay")
    _run([HIPCC, "-std=c++17", "-O2", "--offload-arch=gfx950", "--offload-host-only", "-x", "hip",
          "-I" + os.path.join(ROOT, "include"), "-c", os.path.join(ROOT, "tests", "f8_launches.cpp"), "-o", obj])
    _run([HIPCC, "-rdynamic", obj, "-L" + LIBDIR, "-lsg", "-Wl,-rpath," + LIBDIR, "-o", exe])
    return lambda test: _run([exe, test], timeout=300).stdout


def test_every_address_of_many_shapes(replay):
    out = replay("shapes")
    # every tile of the library, whole and split, and every kernel is among them
    for wide, tiles in (("false", ("256, 256, 2, 4, 2", "256, 128, 4, 2, 3", "128, 128, 2, 4, 4", "64, 64, 1, 4, 4")),
                        ("true", ("256, 128, 4, 2, 3", "128, 128, 2, 4, 4", "64, 64, 1, 4, 4"))):
        for tile in tiles:
            for e5 in ("false", "true"):
                name = f"F8Tile<{wide}, {e5}, {tile}>"
                for split in ("false", "true"):
                    assert f"f8_tiles_kernel<sg::{name}, {split}>" in out, f"{name}, {split} is not reached\n{out}"
                assert f"f8_join_kernel<sg::{name}" in out
        for cf, tf, waves in ((2, 1, 4), (1, 1, 4), (1, 1, 8), (1, 2, 8), (1, 4, 8)):
            assert f"f8_stream_kernel<{wide}, false, {cf}, {tf}, {waves}" in out or \
                f"f8_stream_kernel<{wide}, true, {cf}, {tf}, {waves}" in out, f"{cf} {tf} {waves}\n{out}"
    for kernel in ("f8_rows_kernel", "f8_tile_kernel", "f8_values_kernel", "dropout_kernel"):
        for kind in ("float", "unsigned short"):
            assert f"::{kernel}<{kind}" in out


def test_rows_far_apart(replay):
    replay("pitches")


def test_the_largest_sizes(replay):
    # a launch holds less than 2^32 threads: whatever is launched fits, and
    # every row is in some launch
    replay("many")
