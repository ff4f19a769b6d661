"""The batches of test_latent_waits_gpu.py on the checked debug variant, whose rings have their
least depth, so that phases wrap as often as they can; no check may fire."""

import pytest

import test_latent_waits_gpu as W
from exact_attention_fattn_gb300 import _lib, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def debug_lib():
    lib = _lib.load(build.build(debug=True))
    saved = _lib._lib
    _lib._lib = lib
    try:
        yield lib
    finally:
        _lib._lib = saved


@pytest.mark.parametrize("rank,heads", [(256, 16), (512, 16), (256, 40), (512, 64), (512, 20)])
def test_tiles_of_one_page_and_of_two_in_turn(rank, heads):
    W.test_tiles_of_one_page_and_of_two_in_turn(rank, heads)


@pytest.mark.parametrize("page,step", [(64, 1), (128, 97)])
def test_references_that_move_in_every_tile(page, step):
    W.test_references_that_move_in_every_tile(page, step)
