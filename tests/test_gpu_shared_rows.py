"""shared_attention where a group has few rows: every kernel that the shared
tokens' launch picks by their number, against 64-bit attention."""
import pytest

torch = pytest.importorskip("torch")
from test_gpu_decode import make_tree  # noqa: E402
from test_gpu_shared import attend, tk  # noqa: E402,F401

pytestmark = pytest.mark.gpu

# groups, requests of a group, nodes, query heads, cache heads: rows of a group's head
ROWS = {8: (12, 8, 1, 2, 2), 32: (12, 16, 1, 2, 1), 33: (10, 11, 3, 1, 1), 64: (8, 16, 1, 4, 1), 65: (8, 13, 5, 1, 1), 128: (6, 16, 2, 4, 1)}


def lengths(groups, size):
    """Shared tokens of each group (around a tile's end, none, several tiles) and each request's own."""
    shared = [(448, 0, 700, 64, 511, 129, 63, 333, 640, 65, 200, 575)[i % 12] for i in range(groups)]
    return shared, [(0, 1, 63, 64, 65, 17, 130)[i % 7] for i in range(groups * size)]


@pytest.mark.parametrize("dtype,cache", [("bf16", "own"), ("f16", "own"), ("bf16", "e4m3"), ("f16", "e4m3")])
# page sizes that TMA takes, and that it does not
@pytest.mark.parametrize("D,P", [(128, 16), (96, 12), (64, 64)])
@pytest.mark.parametrize("rows", sorted(ROWS))
def test_rows_of_a_group(tk, dtype, cache, D, P, rows):  # noqa: F811
    groups, size, T, Hq, Hkv = ROWS[rows]
    assert size * T * Hq // Hkv == rows
    shared, own = lengths(groups, size)
    # planned for contexts that take several parts of shared tokens, each shorter than a group's
    attend(tk, dtype, cache, shared, size, own, T, Hq, Hkv, D, P, seed=rows, max_context=5000, max_shared=4500, capacity=5000, launches=3)


@pytest.mark.parametrize("cache", ["own", "e4m3"])
@pytest.mark.parametrize("rows", [33, 65, 128])
def test_nodes_and_trees_of_few_rows(tk, cache, rows):  # noqa: F811
    groups, size, T, Hq, Hkv = ROWS[rows]
    shared, own = lengths(groups, size)
    nodes = [(T, 0, 1, T - 1)[i % 4] for i in range(groups * size)]
    kw = dict(seed=rows + 1, max_context=41000, max_shared=40500, capacity=41000, launches=3)
    attend(tk, "bf16", cache, shared, size, own, T, Hq, Hkv, 128, 16, nodes=nodes, **kw)
    attend(tk, "f16", cache, shared, size, own, T, Hq, Hkv, 80, 5, tree=make_tree(groups * size, T, rows), nodes=nodes, qview=True, **kw)


@pytest.mark.parametrize("dtype,cache", [("bf16", "own"), ("f16", "own"), ("bf16", "e4m3"), ("f16", "e4m3")])
@pytest.mark.parametrize("groups,size,T,Hq", [(6, 8, 1, 1), (4, 16, 1, 4), (2, 16, 2, 4)])
def test_long_prefixes_of_few_rows(tk, dtype, cache, groups, size, T, Hq):  # noqa: F811
    """Rings of keys and values that go round many times in one part."""
    shared = [(6000, 4097)[i % 2] for i in range(groups)]
    own = [(0, 700, 64)[i % 3] for i in range(groups * size)]
    attend(tk, dtype, cache, shared, size, own, T, Hq, 1, 128, 64, seed=size, max_context=200000, max_shared=199000, capacity=200000, launches=3)
