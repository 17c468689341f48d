"""Which kernel, tile and piece of a block-scaled product comes when, on the CPU:
csrc/block_order.h compiled by the host compiler, where an operation that leaves
32 bits ends the run, against the same order in Python's integers; and that the
GPU tests' sizes reach every variant."""
import ctypes
import random
import subprocess

import pytest
import torch

from oracle import cbuild
from routing_grouped_expert_router_gb300 import binding as mb
from routing_grouped_expert_router_gb300 import build as mbuild
from tests import test_gpu_block_fp8 as near
from tests import test_gpu_block_fp8_edges as edges

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
int few(int rows, int E, int K, int N, int alone) { return alone ? moe::few_rows_alone(rows, E, K, N) : moe::few_rows(rows, E, K, N); }
int few_tile(int rows, int E) { return moe::few_tile_rows(rows, E); }
void share(int tiles, int nkb, int grid, int me, int* o) {
  const moe::Share s = moe::share_of(tiles, nkb, grid, me);
  const int all[6] = {s.per, s.each, s.longer, s.t, s.kb, s.count};
  for (int i = 0; i < 6; ++i) o[i] = all[i];
}
int owner(int tiles, int nkb, int grid, int step) { return moe::share_of(tiles, nkb, grid, 0).owner(step); }
int first_of(int tiles, int nkb, int grid, int c) { return moe::share_of(tiles, nkb, grid, 0).lo(c); }
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


# ---------------------------------------------------------------- few rows
SMS = 152


def _cut(order, tiles, nkb, grid):
    """Every block's steps as (tile, first step, steps, slot) and what they are: "whole", "even", or "parts" of tiles."""
    out, shares, slots = (ctypes.c_int * 6)(), [], False
    for me in range(grid):
        order.share(tiles, nkb, grid, me, out)
        per, each, longer, t, kb, left = out
        mine = []
        while left > 0:
            n, slot = min(nkb - kb, left), None
            if n < nkb:  # as the kernel finds the pieces of a shared tile, and its own slot
                if per:
                    first, last, first_slot = t * per, t * per + per - 1, 0
                else:
                    first, last = (order.owner(tiles, nkb, grid, s) for s in (t * nkb, t * nkb + nkb - 1))
                    first_slot = 0 if order.first_of(tiles, nkb, grid, first) == t * nkb else 1
                assert first <= me <= last and last - first < 160
                slot = (first, last, first_slot if me == first else 0)
                slots = slots or slot[2] == 1
            mine.append((t, kb, n, slot))
            left, kb = left - n, kb + n
            if kb == nkb:
                t, kb = t + 1, 0
        shares.append(mine)
    return shares, ("even" if out[0] > 1 else "whole") if out[0] else ("parts" if slots else "edges")


def _check_cut(order, tiles, nkb, grid):
    shares, kind = _cut(order, tiles, nkb, grid)
    done = sorted((t, kb, n) for mine in shares for t, kb, n, _ in mine)
    want = [0] * tiles
    for t, kb, n in done:  # each tile's steps once, in order
        assert kb == want[t]
        want[t] += n
    assert all(w == nkb for w in want)
    joins = {}
    for me, mine in enumerate(shares):
        at = [s[2] for *_, s in mine if s]
        assert len(at) == len(set(at)) <= 2  # no slot holds two tiles' sums
        for t, _, _, s in mine:
            if s:
                joins.setdefault(t, []).append((me, s))
    for t, who in joins.items():  # each piece of a shared tile agrees on which blocks they are
        first, last = who[0][1][:2]
        assert [me for me, _ in who] == list(range(first, last + 1)) and all(s[:2] == (first, last) for _, s in who)
    assert len({who[0][1][0] for who in joins.values()}) == len(joins)  # a counter to a tile
    return kind


def test_steps_of_few_rows_are_cut_once(order):
    rng = random.Random(3)
    kinds = {_check_cut(order, rng.choice([1, 2, 11, 56, 88, 112, 151, 152, 153, 384, rng.randint(1, 700)]),
                        rng.choice([1, 2, 3, 4, 7, 8, 9, 16, 32, rng.randint(1, 200)]), rng.choice([1, 2, 148, 152, 160])) for _ in range(400)}
    assert kinds >= {"whole", "even", "parts"}
    assert _check_cut(order, 0, 16, 152) in ("edges", "whole")


def test_the_gpu_tests_reach_every_variant(order):
    """By the rules as they stand: the pair kernel, and the one for few rows with each tile and each cut."""
    def variant(counts, K, N, alone, cols):
        R, E = sum(counts), len(counts)
        if not order.few(R, E, K, N, alone):
            return "pair"
        nt = order.few_tile(R, E)
        tiles = -(-N // cols) * sum(-(-c // nt) for c in counts)
        return nt, _check_cut(order, tiles, -(-K // 128), SMS)

    products = {variant(c, K, N, 1, 256) for c, K, N in near.SHAPES + edges.FEW}
    assert products >= {"pair", (16, "whole"), (16, "even"), (16, "parts"), (32, "even"), (32, "parts")}
    assert {n for n, _ in products - {"pair"}} == {16, 32}
    first = {variant(c, h, f, 0, 128) for c, h, f in near.FFN + edges.FEW_FFN}
    assert first >= {"pair", (16, "whole"), (16, "even"), (16, "parts"), (32, "whole"), (32, "parts")}
    second = {variant(c, f, h, 0, 256) for c, h, f in near.FFN + edges.FEW_FFN}
    assert second >= {"pair", (16, "whole"), (16, "even"), (16, "parts"), (32, "even"), (32, "parts")}
    # one group whose rows fill more than one tile of 32
    assert any(max(c) > 32 and order.few(sum(c), len(c), K, N, 1) for c, K, N in edges.FEW)
