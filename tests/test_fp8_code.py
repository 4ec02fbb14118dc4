"""What the compiler makes of the block-scaled product's kernels for few rows (their
gfx950 assembly, compiled on the CPU): which waits stand between their loads."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """{mangled name: instructions} of rq_gemm_fp8.hip, compiled as the library is."""
    if not (os.path.exists(HIPCC) or shutil.which("hipcc")):
        pytest.skip("hipcc not available")
    from gemm_rwkv_decode_amd import build
    out = str(tmp_path_factory.mktemp("fp8") / "rq_gemm_fp8.s")
    r = subprocess.run([HIPCC, *build.FLAGS, "-S", "--cuda-device-only",
                        os.path.join(build.CSRC, "rq_gemm_fp8.hip"), "-o", out],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    found, name = {}, None
    for line in open(out):
        label = re.match(r"(_Z\S+):", line)
        if label:
            name = found.setdefault(label.group(1), [])
        elif name is not None and re.match(r"\.LBB\S+:", line):
            name.append(line.split()[0])
        elif name is not None and line.startswith("\t") and not line.startswith("\t."):
            name.append(line.split(";")[0].split("//")[0].strip())
    return found


def rings(kernels):
    """((outputs, rows in 16s, stages), instructions) of every ring."""
    for name, code in kernels.items():
        m = re.search(r"k_ringILi(\d+)ELi(\d+)ELi(\d+)ELb", name)
        if m:
            yield tuple(map(int, m.groups())), code


def test_every_ring_is_there(kernels):
    assert len(list(rings(kernels))) >= 12


def test_a_ring_waits_for_its_oldest_stage_only(kernels):
    """Between a ring's first product and its last, the only loads that are waited for
    are those ahead of the copies of the later stages: 2 (outputs + rows) copies of
    each stay in flight."""
    for (tn, tm, stages), code in rings(kernels):
        mfma = [i for i, c in enumerate(code) if c.startswith("v_mfma")]
        loop = code[mfma[0]:mfma[-1]]
        waits = [int(n) for c in loop for n in re.findall(r"vmcnt\((\d+)\)", c)]
        assert set(waits) <= {(stages - 1) * 2 * (tn + tm)}, (tn, tm, stages, waits)
        assert waits or stages == 1  # the wait of a ring of one stage is ahead of all products


def test_a_ring_asks_for_scales_before_copies(kernels):
    """Where a wait leaves later stages in flight, a stage's copies stand together and
    its scales before them, so that nothing but the copies of later stages has to be
    counted on behind a stage's own: a wait by their number holds whichever scales the
    compiler loads by vector instructions."""
    for (tn, tm, stages), code in rings(kernels):
        if stages == 1:
            continue
        kinds = "".join("c" if c.split()[-1] == "lds" else "s" for c in code
                        if re.match(r"(buffer|global|flat)_load", c))
        kinds = kinds[:kinds.rindex("c") + 1]
        assert re.fullmatch(f"(s+c{{{2 * (tn + tm)}}})+", kinds), (tn, tm, stages, kinds)


def loops(code):
    """Instructions of the innermost loops: from a label to a branch back to it."""
    for i, c in enumerate(code):
        m = re.match(r"s_cbranch_\w+ (\S+)", c)
        if m and m.group(1) + ":" in code[:i]:
            body = code[code.index(m.group(1) + ":"):i]
            if not any(x.endswith(":") for x in body[1:]):
                yield body


def test_rows_keep_the_next_block_in_flight(kernels):
    """k_rows of two blocks: no wait in its loop is for every load, so one block's are on
    their way while the other is multiplied."""
    found = 0
    for name, code in kernels.items():
        if "k_rowsILi1ELi2E" not in name:
            continue
        for body in loops(code):
            if any(c.startswith("v_mfma") for c in body):
                waits = [int(n) for c in body for n in re.findall(r"vmcnt\((\d+)\)", c)]
                assert waits and min(waits) >= 6, waits  # 2 of w, 2 of x, 2 scales
                found += 1
    assert found == 2
