"""CPU: where lanes of one wave exchange values through LDS with no workgroup
barrier, the compiler is told the order: seen from one lane the stores and the
loads go to different places and could change theirs.  In the gfx950 assembly
the order shows as a wave barrier (no instruction) in front of each store of a
turned line and behind it, and no read of the exchange lies between the two."""
import os
import re
import subprocess
import tempfile

import pytest

from dora_adapter_amd import build as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.HIPCC), reason="hipcc not available")


def kernels(asm, name):
    """{mangled name: its LDS instructions and wave barriers, in order}."""
    out, now = {}, None
    for line in asm.splitlines():
        m = re.match(r"^(_Z\S+):", line)
        if m:
            now = out.setdefault(m.group(1), []) if name in m.group(1) else None
        if now is None:
            continue
        text = line.strip()
        if text.startswith("; wave barrier"):
            now.append("order")
        elif text.startswith(("ds_write", "ds_read", "s_barrier")):
            now.append(text.split()[0])
    return {k: v for k, v in out.items() if v}


@pytest.mark.parametrize("source,name,least", [("gemm_fourbit.hip", "linear_fourbit", 40),
                                               ("newton_schulz.hip", "ns_poly_kernel", 4)])
def test_exchanges_within_a_wave_are_ordered(source, name, least):
    with tempfile.TemporaryDirectory() as d:
        asm = os.path.join(d, "a.s")
        res = subprocess.run([B.HIPCC, *B.COMMON, "-x", "hip", "--cuda-device-only", "-S",
                              os.path.join(B.CSRC, source), "-o", asm], capture_output=True, text=True)
        assert res.returncode == 0, res.stderr[-2000:]
        with open(asm) as fh:
            found = kernels(fh.read(), name)
    assert len(found) >= least
    for kernel, steps in found.items():
        at = [i for i, s in enumerate(steps) if s == "order"]
        # a pair at least: one on each side of the stores (ns_poly: of the reads)
        assert len(at) >= 2 and len(at) % 2 == 0, kernel
        for a, b in zip(at[::2], at[1::2]):
            between = steps[a + 1:b]
            assert between and len({s[:7] for s in between}) == 1, (kernel, between)
