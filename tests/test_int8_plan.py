"""Which kernel each size of the int8 GPU tests takes, by the library's own choices (csrc/int8_plan.h, compiled for
the host), and that every kernel has its sizes."""
import ctypes
import shutil
import subprocess

import pytest

from bit_nf4_quantized_15_amd import build

import int8_sizes

FWD_TILES = ["256x256", "256x192", "128x128", "64x64"]
DX_TILES = ["256x256", "128x256", "128x128", "64x128"]
SOURCE = """
#include "int8_plan.h"
using namespace qlora;
extern "C" {
static int pack(Int8Choice c) { return 16 * c.tile + c.splits; }
int fwd(int64_t M, int64_t N, int64_t K, int may_split) { return pack(int8_fwd_choice(M, N, K, may_split)); }
int dx(int64_t M, int64_t N, int64_t K, int may_split) { return pack(int8_dx_choice(M, N, K, may_split)); }
int gemv(int64_t M, int64_t N, int64_t K, int64_t r) { return int8_gemv_supported(M, N, K, (int)r); }
int quantizes(int64_t M, int64_t K, int64_t, int64_t) { return int8_gemv_quantizes(M, K); }
int prep(int64_t M, int64_t r, int64_t, int64_t) { return int8_prep_rows(M, (int)r); }
int u_rows(int64_t M, int64_t N, int64_t r, int64_t) { return int8_u_supported(M, N, (int)r) ? int8_rows_per_wg(M) : 0; }
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
    for f in ("fwd", "dx", "gemv", "quantizes", "prep", "u_rows"):
        getattr(lib, f).argtypes = [ctypes.c_int64] * 4
    return lib


def _choice(f, tiles, *a):
    c = f(*a)
    return tiles[c // 16], c % 16


def _variants(cases):
    """What the kernels' template arguments depend on: (tile, split or not) -> {(dtype, LoRA, 16-byte rows)}."""
    out = {}
    for tile, splits, fmt, M, N, K, r in cases:
        out.setdefault((tile, splits > 1), set()).add((fmt, r > 0, N % 8 == 0, r % 8 == 0))
    return out


def test_forward_sizes_take_their_tiles(plan):
    for tile, splits, fmt, M, N, K, r in int8_sizes.FWD:
        assert not plan.gemv(M, N, K, r)
        assert _choice(plan.fwd, FWD_TILES, M, N, K, 1) == (tile, splits), (M, N, K)
    v = _variants(int8_sizes.FWD)
    assert set(v) == {(t, False) for t in FWD_TILES} | {("128x128", True)}
    assert {s for _, s, *_ in int8_sizes.FWD} == {1, 2, 3, 4}
    for k, have in v.items():
        # vec: t, B and y in 16 bytes (r and N whole), or not; with LoRA or without; both types
        assert {(lora, n8 and r8) for _, lora, n8, r8 in have} == {(a, b) for a in (False, True) for b in (False, True)}, k
        assert {f for f, *_ in have} == {"bf16", "f16"}, k
    for tile in FWD_TILES:      # ranks past the 64 held in registers; the last step half empty
        assert any(c[0] == tile and c[6] > 64 for c in int8_sizes.FWD)
        assert tile == "64x64" or any(c[0] == tile and c[5] % 128 == 64 for c in int8_sizes.FWD)
    # without a workspace every size takes one workgroup per tile: the tiles that sizes of a split then take
    got = {_choice(plan.fwd, FWD_TILES, *c[3:6], 0) for c in int8_sizes.FWD}
    assert {s for _, s in got} == {1} and {t for t, _ in got} == set(FWD_TILES)


def test_input_gradient_sizes_take_their_tiles(plan):
    for tile, splits, fmt, M, N, K, r in int8_sizes.DX:
        assert _choice(plan.dx, DX_TILES, M, N, K, 1) == (tile, splits), (M, N, K)
    v = _variants(int8_sizes.DX)
    assert set(v) == {(t, False) for t in DX_TILES} | {("128x256", True)}
    assert {s for _, s, *_ in int8_sizes.DX} == set(range(1, 9))
    for (tile, split), have in v.items():
        dyv = {(n8, r8) for _, _, n8, r8 in have}
        want = {(True, True), (True, False)} | (set() if tile.endswith("x256") else {(False, True), (False, False)})
        assert dyv == want, tile
        assert {f for f, *_ in have} == {"bf16", "f16"} and {l for _, l, *_ in have} == {False, True}, tile
    for tile in DX_TILES:
        assert any(c[0] == tile and c[6] > 64 for c in int8_sizes.DX)


def test_decode_sizes(plan):
    for own, turns, fmt, M, N, K, r in int8_sizes.DECODE:
        assert plan.gemv(M, N, K, r) and bool(plan.quantizes(M, K, 0, 0)) == own
        assert -(-((N + 15) // 16) // 512) == turns                        # 512 workgroups of 16 rows
    have = {(own, turns > 1, fmt, r > 0) for own, turns, fmt, M, N, K, r in int8_sizes.DECODE}
    assert {(a, True, f, l) for a in (True, False) for f in ("bf16", "f16") for l in (True,)} <= have
    assert {(a, f) for a, _, f, l in have if not l} >= {(True, "f16"), (False, "f16"), (False, "bf16")}


def test_preparation_sizes(plan):
    for per, fmt, M, K, r in int8_sizes.PREP:
        assert plan.prep(M, r, 0, 0) == per, (M, r)
    ranks = lambda r: 16 if r <= 16 else 32 if r <= 32 else 64 if r <= 64 else 128
    have = {(ranks(r), per == 32, r % 8 == 0) for per, _, _, _, r in int8_sizes.PREP}
    assert have == {(t, big, v) for t in (16, 32, 64, 128) for big in (False, True) for v in (True, False)} - \
        {(128, True, v) for v in (True, False)}
    assert {per for per, *_ in int8_sizes.PREP} == {2, 4, 8, 16, 32}
    for per, fmt, M, N, r in int8_sizes.U:
        assert plan.u_rows(M, N, r, 0) == per, (M, N, r)
    assert {ranks(c[4]) for c in int8_sizes.U if c[0]} == {16, 32, 64, 128}
