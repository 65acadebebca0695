"""Which kernel each size of the fp8 GPU tests takes, by the library's own choices (csrc/fp8_plan.h and prep_plan.h,
compiled for the host), and that every kernel has its sizes."""
import ctypes
import shutil
import subprocess

import pytest

from bit_nf4_quantized_15_amd import build

import fp8_sizes

TILES = ["256x256", "128x128", "64x64"]
SOURCE = """
#include "fp8_plan.h"
#include "prep_plan.h"
using namespace qlora;
extern "C" {
int choice(int64_t M, int64_t O, int64_t C, int64_t may_split) {
    const Fp8Choice c = fp8_choice(M, O, C, may_split);
    return 16 * c.tile + c.splits;
}
int gemv(int64_t M, int64_t K, int64_t, int64_t) { return fp8_gemv_supported(M, K); }
int quantizes(int64_t M, int64_t K, int64_t, int64_t) { return fp8_gemv_quantizes(M, K); }
int prep(int64_t M, int64_t C, int64_t, int64_t) { return plan_stream(M, C, 1, C).splits; }
int64_t down_ws(int64_t M, int64_t C, int64_t r, int64_t items) {   // what the sums of t take, and have
    const SplitPlan p = plan_down(M, C, (int)r, (int)items);
    if ((int64_t)p.splits * p.chunk < C || (p.splits - 1) * (int64_t)p.chunk >= C || p.chunk % 128) return -1;
    const int64_t need = p.splits > 1 ? (int64_t)p.splits * M * ((r + 3) / 4 * 4) * 4 : 0;
    return (int64_t)nt_ws_bytes(M, C, (int)r) - need;
}
int64_t prep_ws(int64_t M, int64_t C, int64_t r, int64_t) {
    const SplitPlan p = plan_stream(M, C, 1, C);
    if ((int64_t)p.splits * p.chunk < C || (p.splits - 1) * (int64_t)p.chunk >= C || p.chunk % 128) return -1;
    return (int64_t)stream_ws_bytes(M, C, (int)r) - (p.splits > 1 ? (int64_t)p.splits * M * ((r + 3) / 4 * 4) * 4 : 0);
}
}
"""

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", build.CSRC, str(d / "plan.cpp"), "-o",
                    str(d / "plan.so")], check=True)
    lib = ctypes.CDLL(str(d / "plan.so"))
    for f in ("choice", "gemv", "quantizes", "prep", "down_ws", "prep_ws"):
        getattr(lib, f).argtypes = [ctypes.c_int64] * 4
        getattr(lib, f).restype = ctypes.c_int64 if f.endswith("ws") else ctypes.c_int
    return lib


def _choice(f, *a):
    c = f(*a)
    return TILES[c // 16], c % 16


def test_forward_sizes_take_their_tiles(plan):
    have = {}
    for tile, splits, fmt, M, N, K, r in fp8_sizes.FWD:
        assert not plan.gemv(M, K, 0, 0)
        assert _choice(plan.choice, M, N, K, 1) == (tile, splits), (M, N, K)
        have.setdefault((tile, splits > 1), set()).add((fmt, r > 0, N % 8 == 0 and r % 8 == 0))
    assert set(have) == {(t, False) for t in TILES} | {("128x128", True)}
    assert {s for _, s, *_ in fp8_sizes.FWD} == {1, 2, 3, 4, 5}
    for k, v in have.items():      # with the branch or without, in 16 bytes or by the element; both types
        assert {(lora, vec) for _, lora, vec in v} == {(a, b) for a in (False, True) for b in (False, True)}, k
        assert {f for f, *_ in v} == {"bf16", "f16"}, k
    for tile in TILES:             # ranks past the 64 that are staged; the last step half empty
        assert any(c[0] == tile and c[6] > 64 for c in fp8_sizes.FWD)
        assert any(c[0] == tile and c[5] % 128 == 64 for c in fp8_sizes.FWD)


def test_input_gradient_sizes_take_their_tiles(plan):
    have = {}
    for tile, splits, fmt, M, N, K, r, p in fp8_sizes.DX:
        assert _choice(plan.choice, M, K, N, 1) == (tile, splits), (M, N, K)
        have.setdefault((tile, splits > 1), set()).add(("none" if not r else "drop" if p else "lora", r % 8 == 0))
    assert set(have) == {(t, False) for t in TILES} | {("128x128", True)}
    for k, v in have.items():
        assert v == {("none", True)} | {(a, b) for a in ("lora", "drop") for b in (False, True)}, (k, v)
    for tile in TILES:
        assert any(c[0] == tile and c[6] > 64 for c in fp8_sizes.DX) and any(c[0] == tile and c[4] % 8 for c in fp8_sizes.DX)


def test_decode_sizes(plan):
    for own, turns, fmt, M, N, K, r in fp8_sizes.DECODE:
        assert plan.gemv(M, K, 0, 0) and bool(plan.quantizes(M, K, 0, 0)) == own, (M, K)
        assert -(-((N + 15) // 16) // (256 if M > 4 else 512)) == turns, (M, N)
    have = {(own, turns > 1, fmt) for own, turns, fmt, *_ in fp8_sizes.DECODE}
    assert {(a, True, f) for a in (True, False) for f in ("bf16", "f16")} <= have
    assert not plan.gemv(17, 64, 0, 0) and not plan.gemv(1, (1 << 18) + 64, 0, 0)


def test_preparation_sizes(plan):
    for splits, fmt, M, C, r in fp8_sizes.PREP:
        assert plan.prep(M, C, 0, 0) == splits, (M, C)
    have = {((r + 31) // 32, splits > 1, r % 8 == 0) for splits, _, _, _, r in fp8_sizes.PREP}
    assert {t for t, *_ in have} == {1, 2, 3, 4} and {s for _, s, _ in have} == {False, True} == {v for *_, v in have}


def test_split_sums_fit_their_workspace(plan):
    """The sums of dropped t go where the queries of the call without dropout leave room for its own."""
    for M in (1, 2, 16, 17, 127, 128, 129, 500, 1000, 1025, 4096, 4097, 8192, 16385, 70000, 1 << 20):
        for C in (64, 128, 192, 448, 512, 576, 1088, 4096, 4160, 11008, 28672, 65536, 1 << 20):
            for r in (1, 7, 8, 16, 33, 64, 65, 96, 97, 100, 128):
                assert plan.prep_ws(M, C, r, 0) >= 0, (M, C, r)
                for items in (1, 2, 3, 7, 8):
                    assert plan.down_ws(M, C, r, items) >= 0, (M, C, r, items)
