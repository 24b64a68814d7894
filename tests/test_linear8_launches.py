"""Host replay of the 8-bit linear layer's launches: tests/linear8_launches.cpp,
linked ahead of the HIP runtime, takes the library's kernel launches and
replays the addresses of their threads against the operands' extents.  No GPU
is needed and no kernel runs."""

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
          "-I" + os.path.join(ROOT, "include"), "-c", os.path.join(ROOT, "tests", "linear8_launches.cpp"), "-o", obj])
    _run([HIPCC, "-rdynamic", obj, "-L" + LIBDIR, "-lsg", "-Wl,-rpath," + LIBDIR, "-o", exe])
    return lambda test: _run([exe, test], timeout=300).stdout


def test_every_address_of_many_shapes(replay):
    out = replay("shapes")
    # every tile of the library is among them
    for tile in ("NtTile<true, 256, 256", "NtTile<true, 256, 128", "NtTile<true, 128, 64", "NtTile<true, 64, 64",
                 "NtTile<false, 256, 256", "NtTile<false, 256, 128", "NtTile<false, 128, 64", "NtTile<false, 64, 64",
                 "CodeTile<128, 128", "CodeTile<128, 64", "CodeTile<64, 64", "nt_stream_kernel", "nt_join_kernel",
                 "operands_kernel", "::quantize_kernel", "::dequantize_kernel"):
        assert tile in out, f"{tile} is not reached\n{out}"


def test_rows_far_apart(replay):
    replay("pitches")


def test_weight_gradient_of_many_tokens(replay):
    # the pitch of the bf16 copy grows with the tokens; a row's offset stays
    # within the 32 bits it is kept in
    replay("weight_gradient_of_many_tokens")


def test_more_tokens_than_a_launch_takes(replay):
    # a launch holds less than 2^32 threads: up to the largest sizes of the
    # interface, whatever is launched fits, and every row is in some launch
    replay("many_tokens")
