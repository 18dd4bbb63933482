"""embed_rows_grad where a token's run meets the edges of the chunks that the sorted
list is cut into: 32 numbers, or more past 262144 tokens. Bounds as in
test_embed_gpu."""

import pytest

torch = pytest.importorskip("torch")

from test_embed_gpu import BF, BF32, F32, H16, check_backward, rand

pytestmark = pytest.mark.gpu


def of_runs(sizes, seed, gone=0):
    """Token numbers whose sorted list has these runs, in any order, and `gone` negative."""
    ids = torch.cat([torch.full((n,), i, dtype=torch.int32) for i, n in enumerate(sizes)]
                    + [torch.full((gone,), -3, dtype=torch.int32)])
    g = torch.Generator().manual_seed(seed)
    return ids[torch.randperm(ids.numel(), generator=g)].cuda()


EDGES = [31, 32, 33, 63, 64, 65, 95, 96, 97, 1, 2, 128, 30]


@pytest.mark.parametrize("dtype", [F32, BF32, H16, BF])
@pytest.mark.parametrize("turn", range(len(EDGES)))
def test_runs_at_the_edges_of_32(turn, dtype):
    sizes = EDGES[turn:] + EDGES[:turn]  # every cut falls elsewhere
    ids = of_runs(sizes, turn, gone=turn * 7)
    check_backward(ids.numel(), len(sizes) + 2, 72, dtype, ids=ids, beta=turn % 3 / 2)


@pytest.mark.parametrize("M,chunk", [(262145, 64), (1100000, 160)])
def test_runs_at_the_edges_of_longer_chunks(M, chunk):
    sizes = [k * chunk + d for k in (1, 2, 3, 40) for d in (-1, 0, 1)]
    sizes += [1, chunk // 2, M - sum(sizes) - chunk // 2 - 1 - 5]
    assert sizes[-1] > 1000 * chunk
    for seed in range(2):
        ids = of_runs(sizes, seed, gone=5)
        assert ids.numel() == M
        check_backward(M, len(sizes) + 1, 24, BF32, ids=ids, scale=0.5)
        sizes = sizes[3:] + sizes[:3]


def test_frequent_neighbours():
    """All tokens are a few rows that lie side by side, one of them most of the time."""
    M = 300001
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = 40 + torch.randint(0, 5, (M,), generator=g, device="cuda")
    ids[torch.rand(M, generator=g, device="cuda") < 0.9] = 41
    for beta in (0.0, 0.5, 1.0):
        check_backward(M, 90, 40, BF32, ids=ids.int(), beta=beta)
