"""Static checks, on the AMD assembly hipcc produces for gfx950, of the products that pass an operand through LDS of a
wave's own (built here, no GPU needed): a block's values are written, then come the order point of the source and the
reads of other lanes' values."""
import os
import re
import shutil
import subprocess

import pytest

from bit_nf4_quantized_15_amd import build

pytestmark = pytest.mark.skipif(not os.path.exists(build.HIPCC) and shutil.which("hipcc") is None,
                                reason="hipcc not available")
SOURCES = {"fp8_prep": ("fp8_prep_stream_kernelI", 48), "lora_dropout": ("down_stream_kernelI", 16)}


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    d = tmp_path_factory.mktemp("isaprep")
    procs = {}
    for name in SOURCES:
        cmd = [build.HIPCC, *[f for f in build.CFLAGS if f != "-fPIC"], "--cuda-device-only", "-S",
               os.path.join(build.CSRC, f"{name}.hip"), "-o", str(d / f"{name}.s")]
        procs[name] = subprocess.Popen(cmd, stdout=subprocess.DEVNULL, stderr=subprocess.PIPE)
    out = {}
    for name, p in procs.items():
        _, err = p.communicate()
        assert p.returncode == 0, err.decode()[-2000:]
        out[name] = (d / f"{name}.s").read_text()
    return out


def kernels(asm, pattern):
    """(name, lines) of each kernel whose name holds the pattern."""
    for m in re.finditer(r"^(_Z\w+):\s*(?:;.*)?$", asm, re.M):
        if pattern in m.group(1):
            yield m.group(1), [l.strip() for l in asm[m.start():asm.find(".Lfunc_end", m.start())].split("\n")]


def args(name):
    """Groups of 32 ranks, and whether Y is [C, r]."""
    v = [int(v) for v in re.findall(r"L[ibj](\d+)E", name.split("_kernelI", 1)[1])]
    return v[0], name.find("down_stream") >= 0 or bool(v[2])


@pytest.mark.parametrize("source", sorted(SOURCES))
def test_reads_of_other_lanes_values_follow_the_order_point(asm, source):
    pattern, count = SOURCES[source]
    n = 0
    for name, body in kernels(asm[source], pattern):
        points = [i for i, l in enumerate(body) if l.startswith("; wave barrier")]
        assert len(points) == 2, (name, len(points))                      # the two blocks of a turn
        groups, ynat = args(name)
        for w in points:
            b = max(i for i in range(w) if body[i] == "s_barrier")
            e = min([i for i in range(w, len(body)) if body[i] == "s_barrier"] + [len(body)])
            # 8 rows of 16 bytes a lane, whatever the stores' width
            stored = sum({"ds_write_b128": 16, "ds_write2_b64": 16, "ds_write_b64": 8, "ds_write2st64_b64": 16}
                         .get(l.split()[0], 0) for l in body[b:w] if l.startswith("ds_write"))
            assert stored >= 128, (name, stored)
            reads = lambda part: sum(l.startswith("ds_read_b128") for l in part)
            if ynat:         # (Y's operands are transposed reads)
                assert (reads(body[b:w]), reads(body[w:e])) == (0, 8), name
            else:            # (Y's are of this width too: the first of each group of ranks may lie in front)
                assert reads(body[b:w]) <= groups and reads(body[b:e]) == 8 * (1 + groups), name
        n += 1
    assert n == count
