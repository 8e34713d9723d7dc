"""The paged cache's host code, compiled for the CPU with the driver and the kernels stood in for
(host_pages_main.cpp): what the attention's plans cover, and that a call which fails leaves the host's books
and the device's tables alike, no GPU needed."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    from causal_dit_kv_b200 import build
    out = str(tmp_path_factory.mktemp("host_pages") / "host_pages_main")
    cuda = os.path.join(os.path.dirname(os.path.dirname(build.nvcc())), "include")
    cmd = [shutil.which("g++") or "g++", "-O1", "-std=c++17", f"-I{os.path.join(ROOT, 'include')}", f"-I{build.CSRC}",
           f"-I{cuda}", "-Wno-subobject-linkage", "-o", out, os.path.join(HERE, "host_pages_main.cpp")]
    subprocess.run(cmd, check=True)
    return out


def _run(program, *args):
    got = subprocess.run([program, *map(str, args)], capture_output=True, text=True, timeout=300)
    assert got.returncode == 0, got.stdout + got.stderr


def test_plans_of_few_and_many_rows_in_one_call(program):
    """Few or many query rows in the groups' common part and in the streams' own: the plan is the one of
    the kernel that is launched, every key of every query is in it once, now and after growth."""
    _run(program, "mixed")


@pytest.mark.parametrize("seed", range(8))
def test_plans_of_random_sessions(program, seed):
    """Extends, forks, forks of forks, frees and compactions in any order, any mix of queries."""
    _run(program, "plan", seed, 150)


def test_the_sharing_rule_on_both_sides_of_its_borders(program):
    """Automatic, always and never; up to 16 rows to a key head and more; idle members."""
    _run(program, "share")


def test_failed_allocations_and_launches(program):
    """Every allocation and every launch of extend, fork, free and compact failing in turn: the call changes
    nothing and succeeds when made again; after edits that were launched in part the pool is refused."""
    _run(program, "failures")
