"""Kernels whose last workgroup reads what the others stored: one wave's
release publishes the whole workgroup's stores, so every wave has to have
waited for its own ahead of the barrier before it. The compiler does not add
that wait; the test reads the gfx950 assembly of this repository's sources."""
import os
import re
import subprocess

import pytest

from moe_expert_load_ue_amd import build as B


def device_assembly(source, tmp_path):
    out = str(tmp_path / (source + ".s.txt"))
    flags = [f for f in B.HIPCC_FLAGS if f not in ("-shared", "-fPIC")]
    subprocess.run([B.hipcc(), *flags, "-I", B.INCLUDE, "-S", "--cuda-device-only",
                    "-o", out, os.path.join(B.CSRC, source)], check=True,
                   stderr=subprocess.DEVNULL)
    with open(out) as f:
        return f.read().split("\n")


def unwaited(lines):
    """(releases behind a barrier, those whose barrier lacks the wait): walking
    up from a release to the barrier before it, then up from the barrier, a
    wait for all loads and stores has to come before any store."""
    found, bad = 0, []
    for i, line in enumerate(lines):
        if "buffer_wbl2" not in line:
            continue
        j = i - 1
        while "s_barrier" not in lines[j]:
            assert not re.match(r"\s+global_store|\s+flat_store|\s+buffer_store", lines[j])
            j -= 1
        found += 1
        for k in range(j - 1, max(j - 60, 0), -1):
            if re.match(r"\s+s_waitcnt\b.*vmcnt\(0\)", lines[k]):
                break
            if re.match(r"\s+(global|flat|buffer)_(store|atomic)|\s+s_endpgm", lines[k]):
                bad.append(i + 1)
                break
        else:
            bad.append(i + 1)
    return found, bad


@pytest.mark.parametrize("source", ["k_moe.hip", "k_plan.hip"])
def test_stores_are_waited_for_before_they_are_published(source, tmp_path):
    found, bad = unwaited(device_assembly(source, tmp_path))
    assert found > 0 and bad == []


def test_the_reader_of_assembly_sees_a_missing_wait():
    good = ["\tglobal_store_dword v1", "\ts_waitcnt vmcnt(0)", "\ts_barrier", "\tbuffer_wbl2 sc1"]
    assert unwaited(good) == (1, [])
    assert unwaited([good[0], "\ts_waitcnt lgkmcnt(0)"] + good[2:]) == (1, [4])
