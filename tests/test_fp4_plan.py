"""Which kernel, tile and split a 4-bit product takes, without a GPU: the sizes of the GPU tests reach
every one that the plan chooses for some product on a GB300 (152 SMs)."""

import itertools

import pytest

import dense_fp32_matrix_04_gb300 as sg
from dense_fp32_matrix_04_gb300 import build

SMS = 152

#: a product of each tile and split, its sides off the tiles' edges: (tokens, parts) -> (M, N, K)
REACHED = {(1, 1): (1, 4203, 5000), (16, 1): (13, 3001, 1130), (16, 2): (7, 4841, 3906), (16, 4): (9, 94, 14352),
           (32, 1): (26, 2300, 760), (32, 2): (17, 4697, 6408), (32, 4): (22, 539, 6624),
           (64, 1): (346, 1026, 2010), (64, 2): (1201, 247, 12617), (64, 4): (105, 577, 7645),
           (128, 1): (1812, 1441, 617), (128, 2): (2374, 145, 24387), (128, 4): (72, 2342, 23321), (256, 1): (985, 2992, 4036)}


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


@pytest.mark.parametrize("want,size", REACHED.items())
def test_sizes_reach_what_they_are_for(want, size):
    assert sg.sgemm_fp4_plan_model(*size, SMS) == want


def test_nothing_else_is_reached():
    steps = [1, 2, 3, 5, 8, 13, 17, 24, 33, 48, 65, 72, 100, 129, 200, 257, 300, 420, 600, 900, 1168, 1500, 2374, 3001, 4743, 8192, 16384]
    got = {sg.sgemm_fp4_plan_model(M, N, K, SMS)
           for M, N, K in itertools.product(steps, steps, [1, 64, 300, 1000, 2047, 4096, 6446, 8192, 12541, 16384, 23586, 90112, 90113, 300000])}
    assert got == set(REACHED)


def sizes(test):
    """The M, N, K (or M alone) of a parametrised test."""
    return [v for mark in test.pytestmark if mark.name == "parametrize" and mark.args[0] in ("M,N,K", "M,N", "M") for v in mark.args[1]]


def test_the_tests_of_pairs_reach_pairs():
    import test_fp4_gpu as t
    tiles = {size: sg.sgemm_fp4_plan_model(*size, SMS)[0] for size in sizes(t.test_product_on_pairs)}
    tiles.update({M: sg.sgemm_fp4_plan_model(M, 4300, 1130, SMS)[0] for M in sizes(t.test_strides_and_what_lies_around_on_pairs)})
    tiles.update({M: sg.sgemm_fp4_plan_model(M, 4100, 1024, SMS)[0] for M in sizes(t.test_another_stream_a_graph_and_the_same_bits_on_pairs)})
    tiles.update({N: sg.sgemm_fp4_plan_model(1301, N, 1450, SMS)[0] for N in (8000, 8001, 7937)})
    tiles["just before"] = sg.sgemm_fp4_plan_model(1300, 8000, 2048, SMS)[0]
    assert set(tiles.values()) == {256}, tiles
    # of the two sizes that stand for clusters of two the first has them
    assert sg.sgemm_fp4_plan_model(*sizes(t.test_product_of_halves)[0], SMS) == (16, 2)


@pytest.mark.parametrize("size", [(0, 1, 1, 152), (1, 0, 1, 152), (1, 1, 0, 152), (2 ** 30 + 1, 1, 1, 152), (1, 1, 2 ** 24 + 1, 152), (5, 5, 5, 1)])
def test_refusals(size):
    with pytest.raises(sg.SgemmError):
        sg.sgemm_fp4_plan_model(*size)
    assert sg.load().sgemm_fp4_plan_model(4, 4, 4, 152, None, None) == sg.SGEMM_ERR_INVALID_ARG
