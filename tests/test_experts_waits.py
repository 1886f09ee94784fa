"""The gradient's product with its row operand in memory waits for all loads but
the newest four, which have to be the next step's codes: in the code that is
built, plain loads stand neither between a step's direct loads nor, other than
those four, between them and the wait."""
import os
import re
import subprocess

import pytest

from bit_weight_only_int4_amd import build

pytestmark = pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="no hipcc")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """Per kernel its vector memory operations, waits and barriers in order."""
    out = str(tmp_path_factory.mktemp("asm") / "k.s")
    src = os.path.join(build.CSRC, "q4_experts_back_direct.hip")
    subprocess.run([build.HIPCC, *build.CFLAGS, "--cuda-device-only", "-S", src, "-o", out], check=True,
                   capture_output=True)
    found, name = {}, None
    for line in open(out):
        m = re.match(r"(\w*back_direct_kernel\w*):", line)
        if m:
            name = m.group(1)
            found[name] = []
        op = re.match(r"\s+(global_load_lds_dwordx4|global_load_dword|global_store_dword|s_barrier|s_waitcnt vmcnt\(\d+\))", line)
        if name and op:
            found[name].append(op.group(1))
    return found


def test_order_of_loads(kernels):
    assert len(kernels) == 2  # tiles of 64 and of 128 rows
    for name, ops in kernels.items():
        rows = 128 if "128" in name else 64
        direct = 2 * rows // 32  # of a step: two parts
        # the loop's waits: a count, then the barrier
        waits = [i for i, op in enumerate(ops) if op == "s_waitcnt vmcnt(4)" and ops[i + 1] == "s_barrier"]
        assert len(waits) >= 2, name
        runs = re.findall(r"L+", "".join("L" if op == "global_load_lds_dwordx4" else "." for op in ops))
        assert all(len(r) == direct for r in runs) and len(runs) >= 3, (name, runs)
        for i in waits:
            before = [op for op in ops[:i] if op.startswith("global_load")]
            assert before[-4:] == ["global_load_dword"] * 4 and before[-5] == "global_load_lds_dwordx4", name
