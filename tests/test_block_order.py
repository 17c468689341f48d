"""Which tile of a block-scaled product comes when, on the CPU: csrc/block_order.h
compiled by the host compiler, where an operation that leaves 32 bits ends the
run, against the same order in Python's integers."""
import ctypes
import random
import subprocess

import pytest
import torch

from oracle import cbuild
from routing_grouped_expert_router_gb300 import binding as mb
from routing_grouped_expert_router_gb300 import build as mbuild

MOST_ROWS = 2 ** 31 - 512
SOURCE = r"""
#include "block_order.h"
extern "C" {
void order_of(long long a, long long b, long long sa, long long sb, long long MT, long long NT, int* o) {
  const moe::TileOrder t = moe::tile_order(a, b, sa, sb, MT, NT);
  o[0] = t.raster_n;
  o[1] = t.group;
}
void tile_of(int raster_n, int group, int MT, int NT, int local, int* at) {
  const moe::TileAt t = moe::tile_at(moe::TileOrder{raster_n, group}, MT, NT, local);
  at[0] = t.m;
  at[1] = t.n;
}
int most_rows() { return moe::kMostRows; }
}
"""


@pytest.fixture(scope="module")
def order(tmp_path_factory):
    at = tmp_path_factory.mktemp("order")
    (at / "order.cpp").write_text(SOURCE)
    subprocess.run([cbuild.compiler(), "-std=c++17", "-O1", "-shared", "-fPIC", "-fsanitize=signed-integer-overflow,integer-divide-by-zero,bounds",
                    "-fsanitize-undefined-trap-on-error", "-I" + mbuild.CSRC, str(at / "order.cpp"), "-o", str(at / "order.so")], check=True)
    L = ctypes.CDLL(str(at / "order.so"))
    L.order_of.argtypes = [ctypes.c_longlong] * 6 + [ctypes.c_void_p]
    return L


def _call(f, *args):
    out = (ctypes.c_int * 2)()
    f(*args, out)
    return tuple(out)


def _want(raster_n, group, MT, NT, local):
    wide, along = (NT, MT) if raster_n else (MT, NT)
    band, r = divmod(local, group * along)
    size = min(group, wide - band * group)
    u, v = band * group + r % size, r // size
    return (v, u) if raster_n else (u, v)


# rows, K, N of one group: among them the products of 32 bits that were 0, negative or wrapped
FAR = [(2 ** 28, 16, 16), (2 ** 28 - 70000, 16, 16), (2 ** 28 + 256, 16, 16), (2 ** 27, 16, 16), (2 ** 27 + 300, 16, 256), (357900000, 64, 64),
       (400000001, 64, 64), (MOST_ROWS, 16, 16), (MOST_ROWS, 64, 16), (2 ** 30, 144, 16), (2 ** 28, 16, 512), (1, 16, 2 ** 20), (300, 2 ** 20, 2 ** 20)]
NEAR = [(16384, 4096, 14336), (192, 2048, 1408), (1037, 1104, 720), (1, 4096, 14336), (49152, 2048, 1408), (100, 4096, 4096), (70000, 128, 4096)]


@pytest.mark.parametrize("rows,K,N", FAR + NEAR)
def test_tiles_of_one_group(order, rows, K, N):
    MT, NT = -(-rows // 256), -(-N // 256)
    raster_n, group = _call(order.order_of, rows * K, K * N, 256 * K, 256 * K, MT, NT)
    assert 1 <= group <= (NT if raster_n else MT)
    tiles = MT * NT
    rng = random.Random(rows + K + N)
    some = {t for t in (0, 1, tiles // 2, tiles - 2, tiles - 1) if t >= 0} | {rng.randrange(tiles) for _ in range(300)}
    for local in some:
        at = _call(order.tile_of, raster_n, group, MT, NT, local)
        assert at == _want(raster_n, group, MT, NT, local)
        assert 0 <= at[0] < MT and 0 <= at[1] < NT
    for e in (7, MT - 1, MT):  # and of a group that has but a part of the rows
        if 0 < e <= MT:
            for local in {0, e * NT - 1, rng.randrange(e * NT)}:
                assert _call(order.tile_of, raster_n, group, e, NT, local) == _want(raster_n, group, e, NT, local)


def test_every_tile_comes_once(order):
    rng = random.Random(1)
    for _ in range(60):
        MT, NT, K = rng.randint(1, 40), rng.randint(1, 40), 16 * rng.randint(1, 4000)
        raster_n, group = _call(order.order_of, MT * 256 * K, K * NT * 256, 256 * K, 256 * K, MT, NT)
        assert {_call(order.tile_of, raster_n, group, MT, NT, t) for t in range(MT * NT)} == {(m, n) for m in range(MT) for n in range(NT)}


def test_rows_whose_numbers_leave_31_bits_are_refused(order):
    assert order.most_rows() == MOST_ROWS
    mbuild.build()
    for rows, ok in ((MOST_ROWS, True), (MOST_ROWS + 1, False), (2 ** 31 - 1, False)):
        assert (mb.moe_gemm_workspace_bytes(mb.gemm_dims(rows, 16, 16)) > 0) == ok
        for back in (0, 1):
            assert (mb.moe_ffn_workspace_bytes(mb.ffn_dims(rows, 64, 64), back) > 0) == ok
        for op in (mb.OP_LAYER_FWD_FP8_BLOCK, mb.OP_LAYER_BWD_FP8_BLOCK):
            assert (mb.moe_workspace_bytes(mb.dims(rows, 64, 64, 8, 1), op) > 0) == ok


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake device addresses: host-only check")
def test_calls_of_more_rows_are_refused():
    mbuild.build()
    L, at, room = mb.load(), 1 << 20, 1 << 50
    for rows in (MOST_ROWS + 1, 2 ** 31 - 1):
        g, f, d = ctypes.byref(mb.gemm_dims(rows, 16, 16)), ctypes.byref(mb.ffn_dims(rows, 64, 64)), ctypes.byref(mb.dims(rows, 64, 64, 8, 1))
        assert L.moe_gemm_fp8_block(g, *[at] * 7, room, None) == mb.MOE_ERR_UNSUPPORTED
        assert L.moe_gated_ffn_fwd(f, *[at] * 13, room, None) == mb.MOE_ERR_UNSUPPORTED
        assert L.moe_gated_ffn_bwd(f, *[at] * 17, room, None) == mb.MOE_ERR_UNSUPPORTED
        assert L.moe_layer_fwd_fp8_block(d, *[at] * 12, room, None) == mb.MOE_ERR_UNSUPPORTED
        assert L.moe_layer_bwd_fp8_block(d, *[at] * 16, room, None) == mb.MOE_ERR_UNSUPPORTED


@pytest.mark.skipif(torch.cuda.is_available(), reason="fake device addresses: host-only check")
def test_sides_whose_blocks_leave_31_bits_are_refused():
    """The quantisers' sides, and the layer's as the feed-forward block's."""
    mbuild.build()
    L, at, uns = mb.load(), 1 << 20, mb.MOE_ERR_UNSUPPORTED
    for far in (2 ** 31 - 16, 2 ** 31 - 128, 2 ** 31 - 496):
        assert L.moe_quantize_rows_fp8_block(at, 1, far, None, 1, 1, at, at, None) == uns
        assert L.moe_quantize_weights_fp8_block(at, 1, far, 16, at, at, None) == uns
        assert L.moe_quantize_weights_fp8_block(at, 1, 16, far, at, at, None) == uns
    for kw in (dict(h=2 ** 20 + 64), dict(f=2 ** 20 + 64), dict(h=2 ** 31 - 64)):
        d = mb.dims(**{**dict(T=1, h=64, f=64, E=2, k=1), **kw})
        assert L.moe_layer_fwd_fp8_block(ctypes.byref(d), *[at] * 12, 1 << 60, None) == uns
        assert L.moe_layer_bwd_fp8_block(ctypes.byref(d), *[at] * 16, 1 << 60, None) == uns
        assert mb.moe_workspace_bytes(d, mb.OP_LAYER_FWD_FP8_BLOCK) == mb.moe_workspace_bytes(d, mb.OP_LAYER_BWD_FP8_BLOCK) == 0
    assert mb.moe_workspace_bytes(mb.dims(1, 2 ** 20, 2 ** 20, 2, 1), mb.OP_LAYER_FWD_FP8_BLOCK) > 0
