"""The 8-bit 256-tile kernels keep their accumulators in fixed AGPRs and schedule their own waits; both rest on what the
compiler emits, so this test compiles scaled.hip for gfx950 to assembly (with the library's own flags) and checks every
scaled_quad_kernel: no scratch, the AGPRs written only by zeroing and read only at the end, no register moves between
AGPRs, and in the main loop no wait for loads but the schedule's own and those of the scale words.

No GPU is needed (hipcc cross-compiles)."""

import os
import re
import subprocess

import pytest

from newton_schulz_quintic_amd import build as nsq_build

SRC = os.path.join(nsq_build.CSRC, "scaled.hip")


def _kernels(asm: str):
    starts = [(m.start(), m.group(1)) for m in re.finditer(r"^(_ZN\w+):", asm, re.M)]
    for k, (pos, name) in enumerate(starts):
        end = starts[k + 1][0] if k + 1 < len(starts) else len(asm)
        if "scaled_quad_kernel" in name:
            yield name, asm[pos:end].splitlines()


@pytest.mark.skipif(not os.path.exists(nsq_build._hipcc()), reason="hipcc not found")
def test_scaled_quad_kernels_isa(tmp_path):
    out = str(tmp_path / "scaled.s")
    cmd = ([nsq_build._hipcc()] + nsq_build.COMMON + nsq_build.DEVICE + ["--cuda-device-only", "-S", SRC, "-o", out])
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    found = 0
    for name, lines in _kernels(open(out).read()):
        found += 1
        text = "\n".join(lines)
        count = lambda pat: len(re.findall(pat, text))  # noqa: E731
        assert count(r"scratch_(load|store)") == 0, name
        assert count(r"\bv_accvgpr_mov") == 0 and count(r"\bv_accvgpr_read") == 256, name
        assert count(r"\bv_accvgpr_write") == 256 * (2 if "ILi2E" in name else 1), name
        assert int(re.search(r"; NumAgprs: (\d+)", text).group(1)) == 256, name
        loops = [i for i, line in enumerate(lines) if re.match(r"^\.LBB\w+:.*Loop Header", line)]
        main = [i for i in loops if sum("v_mfma" in x for x in lines[i:i + 700]) >= 128]
        assert main, name
        # two stages: the MFMAs, the loads into LDS, one counted wait each before a barrier
        body = lines[main[0]:]
        last = [i for i, x in enumerate(body) if "v_mfma" in x][127]
        body = body[:last + 6]   # the last load follows the last MFMA
        assert sum(" lds" in x and "buffer_load" in x for x in body) == 32, name
        assert [x.split()[-1] for x in body if "s_waitcnt vmcnt" in x] == ["vmcnt(16)"] * 2, name
        assert not any("v_readfirstlane" in x and "v_cmp" in y for x, y in zip(body, body[1:])), name
    assert found == 5
