"""The division of the attention calls of gdn_attn.h over workgroups at its ends: sizes of nothing and the largest."""
import os
import shutil
import subprocess
import sys

import pytest

import gated_deltanet_tree_gdn_amd as gdn
from gated_deltanet_tree_gdn_amd import attn
from test_attn_cpu import cache, call, dims, need

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(gdn.LIB_PATH):
        pytest.fail("libgdn_tree.so is not built: run __graft_entry__.build()")
    return attn.attn_library()


@pytest.mark.parametrize("kind", ["prefill", "verify"])
def test_sequences_without_queries(kind):
    """nothing is launched where no seq_status is asked for; in a process of its own, which a division by zero would end"""
    code = f"""
import sys
sys.path.insert(0, {os.path.join(ROOT, 'tests')!r})
from test_attn_cpu import *
lib = attn.attn_library()
for H_q in (2, 8, 600):
    assert need(lib, {kind!r}, dims(T=0, H_q=H_q), cache()) == 0
    assert call(lib, {kind!r}, dims(T=0, H_q=H_q), cache(), q=None, o=None, anc=None, seq_status=None, workspace=None) == "GDN_OK"
"""
    code = code.replace(", anc=None", "") if kind == "prefill" else code
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert r.returncode == 0, f"{r.returncode}: {r.stderr[-600:]}"


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    """The host layer with its own sizing, under sanitizers."""
    if shutil.which("g++") is None:
        pytest.skip("g++ not installed")
    exe = str(tmp_path_factory.mktemp("sizes") / "attn_sizes_driver")
    csrc = os.path.join(ROOT, "gated_deltanet_tree_gdn_amd", "csrc")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                        "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I", os.path.join(ROOT, "include"), "-I", csrc,
                        os.path.join(csrc, "gdn_attn_api.cpp"), os.path.join(csrc, "gdn_attn_shape.cpp"),
                        os.path.join(ROOT, "tests", "sanitize", "attn_sizes_driver.cpp"), "-o", exe],
                       capture_output=True, text=True)
    if r.returncode != 0 and "cannot find" in r.stderr and "asan" in r.stderr.lower():
        pytest.skip("sanitizer runtime not installed")
    assert r.returncode == 0, r.stderr
    return exe


def run(exe, *args):
    r = subprocess.run([exe, *args], capture_output=True, text=True, timeout=120,
                       env=dict(os.environ, UBSAN_OPTIONS="print_stacktrace=1"))
    assert r.returncode == 0, r.stdout + r.stderr
    assert "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr, r.stderr


def test_the_workspace_of_a_tree_serves_smaller_ones(driver):
    run(driver, "trees")


def test_the_workspace_of_a_call_serves_smaller_ones(driver):
    run(driver, "calls")


def test_the_largest_sizes_that_pass_the_checks(driver):
    run(driver, "largest")


def test_workgroups_are_spread_evenly(driver):
    run(driver, "numbers")


def test_a_cache_that_is_listed_twice_moves_once(driver):
    run(driver, "shared")
