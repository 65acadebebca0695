"""Static checks of the int8 kernels on the AMD assembly hipcc produces for gfx950 (built here, no GPU needed).

The tiled products end each step with a barrier that leaves a counted number of loads in flight.  Loads complete in
order, so the tile that the next step reads has landed if the loads issued since are exactly that many: the direct
HBM->LDS loads of whole later tiles, and nothing else.  A load that the compiler placed among them would turn the
barrier into a race, so every step of every instantiation is counted.  Kernels that hand partial results to another
workgroup must have waited for their payload stores before the tag that publishes them, and write and read both at the
device-coherent level.  No kernel writes through the scalar data cache, and those that keep anything in scratch memory
are named here."""
import re
import shutil
import subprocess

import os

import pytest

from bit_nf4_quantized_15_amd import build

from test_isa_waits import _descriptor, _kernels

pytestmark = pytest.mark.skipif(not os.path.exists(build.HIPCC) and shutil.which("hipcc") is None,
                                reason="hipcc not available")
SOURCES = ("int8_gemm_fwd", "int8_gemm_dx", "int8_gemv", "int8_grads", "int8_prep", "int8_quant")


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    """Device assembly of the int8 sources, compiled side by side with the library's flags."""
    d = tmp_path_factory.mktemp("isa8")
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
    """Template arguments of a kernel, in order."""
    return [int(v) for v in re.findall(r"L[ibj](\d+)E", name.split("_kernelI", 1)[1])]


def _steps(body):
    """What lies before each barrier that the source places itself: (direct loads, loads to registers, vmcnt)."""
    out, direct, regs, in_asm, wait = [], 0, 0, False, None
    for l in body:
        if l.startswith(";;#ASMSTART"):
            in_asm = True
        elif l.startswith(";;#ASMEND"):
            in_asm = False
        elif in_asm and l.startswith("s_waitcnt"):
            wait = int(re.search(r"vmcnt\((\d+)\)", l).group(1))
        elif in_asm and l == "s_barrier":
            out.append((direct, regs, wait))
            direct = regs = 0
        elif l.startswith("buffer_load") and " lds" in l:
            direct += 1
        elif l.startswith(("global_load", "buffer_load", "flat_load")):
            regs += 1
    return out


def test_forward_steps_leave_whole_tiles_in_flight(asm):
    n = 0
    for name, body in _kernels(asm["int8_gemm_fwd"], "int8_gemm_fwd_kernelI"):
        NWM, NWN, MT, NT, S, RING = _args(name)[:6]
        waves = NWM * NWN
        tile = (32 * MT * NWM + 32 * NT * NWN) * S // 1024 // waves        # loads of a wave per tile
        steps = _steps(body)
        flight = tile if RING == 2 else (RING - 3) * tile
        # before the loop: the ring but one tile; the last of them stay in flight
        first = steps.pop(0)
        assert first[0] == (2 if RING == 2 else RING - 1) * tile and first[2] == flight, name
        if RING == 2:          # one barrier a step, in its middle, that waits for everything
            assert steps == [(0, 0, 0), (tile, 0, 0)], (name, steps)
        else:
            assert len(steps) == RING and set(steps) == {(tile, 0, flight)}, (name, steps)
        n += 1
    assert n == 40             # tiles and split x LoRA x 16-byte rows x dtype


def test_input_gradient_steps_leave_whole_tiles_in_flight(asm):
    n = 0
    for name, body in _kernels(asm["int8_gemm_dx"], "int8_gemm_dx_kernelI"):
        MT, NT, RING, split, dyv, av, dt = _args(name)
        w = 64 * 32 * NT * 4 // 1024 // 4 + 1                              # codes, and their scales
        tile = w + (32 * MT * 128 // 1024 // 4 if dyv else 0)              # dy: direct, or through registers
        steps = _steps(body)
        first = steps.pop(0)
        assert first[0] == (2 if RING == 2 else 3) * tile and first[2] == tile, name
        if RING == 2:
            assert steps == [(0, 0, 0), (tile, 0, 0)], (name, steps)
        else:
            assert len(steps) == 4 and {(d, v) for d, _, v in steps} == {(tile, tile)}, (name, steps)
            if dyv:
                assert all(g == 0 for _, g, _ in steps), (name, steps)
        n += 1
    assert n == 28


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
    assert counts == {"int8_gemm_fwd": 8, "int8_gemm_dx": 4, "int8_gemv": 4, "int8_grads": 20, "int8_prep": 0,
                      "int8_quant": 0}


# bytes of scratch a lane: ranks above 64 that are no multiple of 8 in the preparation; ranks 33 to 64 over a dy whose
# columns are no multiple of 4 in the gradients
SCRATCH = {("int8_prep_kernel", (8, 1, 0)): 328, ("int8_grads_kernel", (2, 0, 0)): 112, ("int8_grads_kernel", (2, 1, 0)): 20}


def test_registers_and_scratch(asm):
    n, found = 0, {}
    for src in SOURCES:
        for m in re.finditer(r"\.amdhsa_kernel (\S+)", asm[src]):
            name = m.group(1)
            d = _descriptor(asm[src], name)
            assert d["amdhsa_group_segment_fixed_size"] <= 160 * 1024, name
            used = d["amdhsa_private_segment_fixed_size"]
            if used:
                key = (re.search(r"int8_\w+?_kernel", name).group(0), tuple(_args(name)[:3]))
                found[key] = max(used, found.get(key, 0))
            n += 1
    assert set(found) <= set(SCRATCH) and all(v <= SCRATCH[k] for k, v in found.items()), found
    assert n == 40 + 28 + 4 + 20 + 28 + 8 + 16


def test_no_scalar_memory_writes(asm):
    for src in SOURCES:
        for l in asm[src].split("\n"):
            t = l.strip()
            assert not t.startswith(("s_store", "s_buffer_store", "s_atomic", "s_buffer_atomic", "s_dcache_wb",
                                     "s_dcache_discard")), f"{src}: {t}"
            assert not t.startswith(("v_pk_add_f32", "v_pk_mul_f32", "v_pk_fma_f32")), f"{src}: {t}"
