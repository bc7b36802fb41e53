"""What the workgroups of cider_kv4_attention_shared's launches are, on the host (tests/shared_launches.cpp): in grids of
more than 2^22, which are rounded up, and where the parts over shared pages are a launch of their own."""
import os
import subprocess

import pytest

from w4a8_quantized_linear_amd import build

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    if not os.path.exists(build.HIPCC):
        pytest.skip("no compiler")
    out = tmp_path_factory.mktemp("launches")
    sources = [os.path.join(build.CSRC, f) for f in ("kv4_attention.hip", "kv4_few_rows.hip", "kv4_many_rows.hip")]
    sources.append(os.path.join(HERE, "shared_launches.cpp"))
    objects = [str(out / (os.path.basename(f) + ".o")) for f in sources]
    running = [subprocess.Popen([build.HIPCC, "-x", "hip", "--offload-host-only", "-O1", "-std=c++17", "-I" + build.CSRC, "-c",
                                 f, "-o", o]) for f, o in zip(sources, objects)]
    assert [p.wait() for p in running] == [0] * len(running)
    # no runtime: what it would load, the device code, is not there
    subprocess.run(["g++", "-no-pie", "-o", str(out / "launches"), *objects, "-Wl,--unresolved-symbols=ignore-all"], check=True)
    return str(out / "launches")


@pytest.mark.parametrize("sizes", [
    # batch rows max_rows max_kv_len kv_heads q_heads head_dim groups run_rows max_shared_len tiles
    (5, 600, 512, 300000, 8, 32, 64, 1100, 16, 262144, 0),      # shared pages alone, 4505600 workgroups of 16 columns
    (1100, 600, 512, 300000, 8, 32, 64, 1100, 16, 262144, 0),
    (8, 600, 512, 300000, 32, 128, 128, 257, 16, 262144, 0),
    (600, 600, 1, 300000, 8, 32, 64, 1100, 16, 262144, 0),      # both in one
    (600, 600, 1, 300000, 8, 32, 64, 1100, 16, 262144, 128),
    (64, 64, 1, 9216, 8, 32, 128, 1, 64, 8192, 0),
    (30, 120, 4, 6700, 4, 28, 64, 3, 40, 6000, 0),
    (16, 1024, 64, 65664, 8, 32, 128, 1, 1024, 65536, 0),       # tiles of 256 columns, and of 128
    (3, 300, 200, 900, 2, 14, 64, 2, 250, 512, 256),
    (70000, 70000, 1, 640, 64, 64, 64, 70000, 1, 320, 0),
])
def test_each_workgroup_has_its_own_part_or_none(program, sizes):
    done = subprocess.run([program, *map(str, sizes)], capture_output=True, text=True)
    assert done.returncode == 0, done.stdout + done.stderr
    print(done.stdout)
