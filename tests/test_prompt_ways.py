"""Which way short pieces go, by the size of their scratch (host arithmetic, no GPU), against times of both ways in
microseconds on a GB300: n = 8, 16, 24, 32, 48, 64, as a tree and from bf16 rows."""
import pytest

from reference_residual_kv_gb300 import build, rkv

NS = (8, 16, 24, 32, 48, 64)
TIMES = {  # S, T, N, H, D
    (1, 131072, 8, 32, 128): ((114, 220), (149, 222), (147, 225), (144, 229), (169, 248), (174, 253)),
    (16, 8192, 8, 32, 128): ((119, 228), (158, 235), (166, 242), (170, 250), (227, 271), (262, 272)),
    (4, 8192, 8, 32, 128): ((50, 70), (52, 73), (52, 76), (54, 79), (75, 85), (89, 88)),
    (64, 1024, 8, 32, 128): ((97, 131), (135, 137), (165, 142), (199, 149), (338, 162), (465, 168)),
    (1, 4096, 8, 32, 128): ((18, 37), (22, 37), (24, 38), (25, 39), (27, 41), (29, 42)),
    (16, 8192, 4, 28, 128): ((86, 124), (95, 129), (114, 145), (123, 151), (214, 200), (248, 201)),
    (4, 8192, 4, 28, 128): ((40, 51), (42, 52), (47, 56), (49, 57), (76, 71), (87, 72)),
    (16, 8192, 8, 64, 128): ((156, 228), (163, 236), (202, 264), (221, 271), (438, 380), (504, 401)),
    (256, 512, 4, 16, 128): ((137, 143), (201, 143), (259, 149), (323, 156), (584, 166), (829, 173)),
    (1, 32768, 2, 16, 128): ((33, 59), (38, 61), (35, 64), (40, 65), (51, 66), (53, 67)),
    (32, 4096, 8, 8, 128): ((60, 236), (83, 243), (126, 250), (134, 257), (184, 257), (203, 258)),
    (16, 8192, 8, 32, 64): ((74, 140), (103, 143), (110, 148), (119, 151), (182, 171), (208, 172)),
    (4, 8192, 8, 32, 64): ((35, 53), (38, 54), (39, 54), (41, 55), (65, 63), (73, 64)),
    (1, 131072, 4, 16, 256): ((125, 256), (213, 262), (323, 267), (424, 273), (622, 326), (924, 327)),
    (4, 8192, 4, 16, 256): ((53, 78), (73, 83), (101, 89), (135, 94), (196, 115), (270, 116)),
    (16, 2048, 4, 16, 256): ((56, 75), (87, 81), (126, 87), (158, 94), (240, 110), (340, 111)),
    (1, 4096, 4, 16, 256): ((19, 42), (25, 43), (31, 45), (32, 46), (42, 46), (57, 47)),
}


SHORT = {  # many short sequences: n = 1, 2, 4, 8
    (500, 100, 1, 8, 128): ((40, 40), (44, 40), (63, 40), (114, 42)),
    (2048, 128, 1, 8, 128): ((100, 120), (137, 121), (240, 123), (369, 127)),
    (500, 100, 1, 8, 64): ((29, 35), (37, 34), (51, 34), (88, 34)),
    (500, 100, 1, 8, 256): ((58, 57), (63, 58), (116, 60), (230, 65)),
    (64, 1024, 8, 32, 128): ((43, 134), (47, 135), (67, 137), (109, 141)),
    (256, 256, 8, 32, 128): ((82, 151), (91, 151), (137, 153), (240, 156)),
}


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()


def tree_bytes(p, H, n):
    """The scratch of the way of trees: that of the tree and the rows' parents."""
    return rkv.rkv_dense_attention_workspace(p, H, n) + (4 * p.S * n + 255) // 256 * 256


@pytest.mark.parametrize("sizes,ns,times,most", [(k, NS, v, 1.08) for k, v in TIMES.items()] + [(k, (1, 2, 4, 8), v, 1.21) for k, v in SHORT.items()])
def test_the_way_taken_is_the_faster_one(sizes, ns, times, most):
    S, T, N, H, D = sizes
    p = rkv.make_dense_params(S, T, N, D)
    for n, (tree, rows) in zip(ns, times):
        goes_as_tree = rkv.rkv_chunk_attention_workspace(p, H, n) == tree_bytes(p, H, n)
        assert (tree if goes_as_tree else rows) <= most * min(tree, rows), (n, goes_as_tree)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_fewer_rows_go_as_trees(D):
    # a piece that goes as a tree does so with fewer rows as well
    for S, T, N, H in ((1, 32, 1, 1), (3, 700, 2, 16), (40, 2048, 8, 8), (500, 100, 1, 8)):
        p = rkv.make_dense_params(S, T, N, D)
        way = [rkv.rkv_chunk_attention_workspace(p, H, n) == tree_bytes(p, H, n) for n in range(1, min(T, 64) + 1)]
        assert way == sorted(way, reverse=True)
