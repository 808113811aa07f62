"""The tiles that the 16-bit linear is launched with, on the host: the sizes of
the GPU tests reach every kind that the planner has."""

import pytest

from linear_cases import DEEP, units

TILES = {"whole", "halves", "quarters", "split", "ragged quarters", "ragged split", "whole + halves",
         "whole + quarters"}


@pytest.mark.parametrize("M,K,N,product,tiles", DEEP)
def test_a_size_reaches_its_tiles(M, K, N, product, tiles):
    assert units(M, K, N, product)[0] == tiles
    depth = {"fwd": K, "dX": N, "dW": M}[product]
    assert depth > 8 * 32 and depth % 32 != 0


@pytest.mark.parametrize("product", ["fwd", "dX", "dW"])
def test_every_kind_of_tile_is_reached(product):
    assert {t for *_, p, t in DEEP if p == product} - {"skinny", "skinny split"} == TILES


def test_the_sizes_of_the_models_reach_tested_kinds():
    # PixArt-Sigma's up projection at 4096 tokens, Qwen3-8B's up and down at 1 to 2048
    for M, K, N in [(4096, 1152, 4608), (4096, 4608, 1152)] + [
            (M, k, n) for M in (1, 16, 48, 64, 200, 512, 2048) for k, n in ((4096, 12288), (12288, 4096))]:
        for product in ("fwd", "dX", "dW"):
            assert (product, units(M, K, N, product)[0]) in {(p, t) for *_, p, t in DEEP}


def test_whole_tiles_go_in_rounds():
    # 8 x 48 tiles on 256 CUs: one round of whole ones, the others in halves
    assert units(2048, 4096, 12288, "fwd") == ("whole + halves", 256 + 2 * 128)
