"""Static checks of the fp8 and dropout kernels on the AMD assembly hipcc produces for gfx950 (built here, no GPU
needed).

The tiled products wait at barriers that leave a counted number of loads in flight.  Loads complete in order, so the
tile that is read next has landed if the loads issued since are exactly that many: the direct HBM->LDS loads of whole
later tiles, and nothing else.  Every step of every instantiation is counted, and its products have to lie between the
barriers where the source has them.  Kernels that hand partial results to another workgroup must have waited for their
payload stores before the tag that publishes them.  No kernel writes through the scalar data cache, and those that keep
anything in scratch memory are named here."""
import os
import re
import shutil
import subprocess

import pytest

from bit_nf4_quantized_15_amd import build

from test_isa_waits import _descriptor, _kernels

pytestmark = pytest.mark.skipif(not os.path.exists(build.HIPCC) and shutil.which("hipcc") is None,
                                reason="hipcc not available")
SOURCES = ("fp8_gemm", "fp8_gemv", "fp8_prep", "fp8_quant", "lora_dropout", "lora_grads_dropout", "gemm_dx_dropout", "int8_gemm_dx_dropout")


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    d = tmp_path_factory.mktemp("isaf8")
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


def _args(name):
    return [int(v) for v in re.findall(r"L[ibj](\d+)E", name.split("_kernelI", 1)[1])]


def _steps(body):
    """What lies before each barrier that the source places itself: (direct loads, loads to registers, f8 products,
    vmcnt)."""
    out, direct, regs, mfma, in_asm, wait = [], 0, 0, 0, False, None
    for l in body:
        if l.startswith(";;#ASMSTART"):
            in_asm = True
        elif l.startswith(";;#ASMEND"):
            in_asm = False
        elif in_asm and l.startswith("s_waitcnt"):
            wait = int(re.search(r"vmcnt\((\d+)\)", l).group(1))
        elif in_asm and l == "s_barrier":
            out.append((direct, regs, mfma, wait))
            direct = regs = mfma = 0
        elif l.startswith("buffer_load") and " lds" in l:
            direct += 1
        elif l.startswith(("global_load", "buffer_load", "flat_load")):
            regs += 1
        elif l.startswith("v_mfma_scale_f32_32x32x64_f8f6f4"):
            mfma += 1
    return out


def test_steps_leave_whole_tiles_in_flight(asm):
    n = 0
    for name, body in _kernels(asm["fp8_gemm"], "fp8_gemm_kernelI"):
        NWM, NWN, MT, NT, RING = _args(name)[:5]
        tile = (32 * MT * NWM + 32 * NT * NWN) * 128 // 1024 // (NWM * NWN) + 2   # loads of a wave: tiles, two of scales
        steps = _steps(body)
        first = steps.pop(0)
        assert first == ((2 if RING == 2 else 3) * tile, first[1], 0, tile), (name, first)
        depth = MT * NT
        if RING == 2:      # one barrier a step, in its middle, that waits for everything: a depth on either side
            assert steps == [(0, 0, depth, 0), (tile, 0, 2 * depth, 0)], (name, steps)
        else:
            assert len(steps) == RING and set(steps) == {(tile, 0, 2 * depth, tile)}, (name, steps)
        n += 1
    assert n == 4 * 18     # three tiles and the split x (forward: branch x 16-byte rows, gradient: 5) x dtype


def test_publication_waits_for_the_payload(asm):
    counts = {}
    for src in SOURCES:
        n = 0
        for name, body in _kernels(asm[src], ""):
            tags = [i for i, l in enumerate(body) if l.startswith("global_store_dwordx2") and " sc1" in l]
            for t in tags:
                b = max(i for i in range(t) if body[i] == "s_barrier")
                p = max(i for i in range(b) if body[i].startswith(("buffer_store", "global_store")) and " sc1" in body[i])
                assert any(body[i].startswith("s_waitcnt") and "vmcnt(0)" in body[i] for i in range(p, b)), \
                    f"{name}: the tag may overtake the payload"
            if tags:
                text = "\n".join(body)
                assert re.search(r"global_load_dwordx2 .* sc1", text) and "s_sleep" in text, f"{name}: polls"
                assert re.search(r"buffer_load_dword(x4)? .* sc1", text), f"{name}: payload loads"
                n += 1
            assert not any(l.startswith("buffer_wbl2") for l in body), f"{name}: L2 write-back"
        counts[src] = n
    assert counts["fp8_gemm"] == 18 and counts["fp8_gemv"] == 4 and counts["lora_grads_dropout"] == 20
    assert counts["fp8_prep"] == counts["lora_dropout"] == counts["fp8_quant"] == counts["gemm_dx_dropout"] == 0


# bytes of scratch a lane, at most, by kernel and first template arguments: masks in the epilogue of the 256 x 256 input
# gradient; a few values in the split forms; rows that are no whole 16-byte chunks in the products with x
SCRATCH = {("fp8_gemm_kernel", (2, 2, 4, 4)): 280, ("fp8_gemm_kernel", (2, 2, 2, 2)): 24,
           ("fp8_prep_stream_kernel", (1, 0)): 112, ("fp8_prep_stream_kernel", (2, 0)): 128,
           ("down_stream_kernel", (1, 0)): 112, ("down_stream_kernel", (2, 0)): 224, ("down_stream_kernel", (2, 1)): 16,
           ("fp8_prep_stream_kernel", (2, 1)): 16}


def test_registers_and_scratch(asm):
    found = {}
    for src in SOURCES:
        for m in re.finditer(r"\.amdhsa_kernel (\S+)", asm[src]):
            name = m.group(1)
            d = _descriptor(asm[src], name)
            assert d["amdhsa_group_segment_fixed_size"] <= 160 * 1024, name
            used = d["amdhsa_private_segment_fixed_size"]
            if used:
                kernel = re.search(r"\d+((?:fp8|down|grads|nf4|int8|prep)_\w+?_kernel)", name).group(1)
                found[name] = (used, max([v for (k, a), v in SCRATCH.items()
                                          if k == kernel and tuple(_args(name)[:len(a)]) == a], default=0))
    bad = {k: v for k, v in found.items() if v[0] > v[1]}
    assert not bad, bad


def test_no_scalar_memory_writes(asm):
    for src in SOURCES:
        for l in asm[src].split("\n"):
            t = l.strip()
            assert not t.startswith(("s_store", "s_buffer_store", "s_atomic", "s_buffer_atomic", "s_dcache_wb",
                                     "s_dcache_discard")), f"{src}: {t}"
            assert not t.startswith(("v_pk_add_f32", "v_pk_mul_f32", "v_pk_fma_f32")), f"{src}: {t}"
