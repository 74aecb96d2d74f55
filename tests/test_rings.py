"""The rules by which kernels wait for ring slots, checked on the host for every
delay of the barriers' arrivals (tests/c/rings_check.cc)."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "nf4_base_lora_b200", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_decode_slot_waits_are_sound(tmp_path):
    exe = str(tmp_path / "rings_check")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I", CSRC,
                    os.path.join(ROOT, "tests", "c", "rings_check.cc"), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, timeout=60, check=True).stdout.split()
    # the rule holds everywhere, and the check does find the decode ring's own barriers wanting
    assert out == ["0", "1"]


def test_the_copying_thread_follows_the_rule():
    """Its role (from the copies' loop to the issuing warp's) waits on the load
    ring's barriers alone."""
    text = open(os.path.join(CSRC, "gemm.cuh")).read()
    role = text[text.index("- producer"):text.index("TMEM + MMA issuer")]
    waits = re.findall(r"mbar_wait\(&(\w+)\[([^\]]*)\]", role)
    assert waits == [("bar_empty", "it % LS"), ("bar_empty", "w.slot")]


def test_no_warp_waits_for_others_where_one_may_have_left():
    """The clearing warps of the rank-r products leave their loop when a bounded
    wait runs out; a barrier among them there would have no bound."""
    text = open(os.path.join(CSRC, "rank.cuh")).read()
    loop = text[text.index("- clearing"):text.index("- epilogue")]
    assert not re.search(r"bar(rier)?\.sync|__syncthreads|named_barrier", loop)


@pytest.mark.parametrize("name", ["rank.cuh", "grouped.cuh", "gemm.cuh"])
def test_tensor_memory_is_read_by_converged_warps(name):
    """A loop whose lanes store under conditions of their own brings the warp
    together before it reads tensor memory again."""
    text = open(os.path.join(CSRC, name)).read()
    for m in re.finditer(r"for \(int (?:cc|tt) = \w+; [^\n]*\{\n(.*?)tmem_ld_32x32b", text, flags=re.S):
        loop = text[m.start():]
        depth, end = 0, 0
        for end, c in enumerate(loop):
            depth += (c == "{") - (c == "}")
            if c == "}" and depth == 0:
                break
        if re.search(r"dst\[|\*reinterpret_cast<\w+\*>\(dst", loop[:end]):
            assert "__syncwarp()" in m.group(1), m.group(0)
