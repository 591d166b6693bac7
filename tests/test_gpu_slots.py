"""Moves between the slots of a state pool on the GPU against one assignment on
the CPU, bit for bit."""
import pytest
import torch

import selective_state_space_21_amd as ssm
from oracle import linear as O

pytestmark = pytest.mark.gpu


def pool_of(shape, dtype, seed=0):
    return torch.randint(-100, 100, shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def move(pool, src, dst, dim=0):
    src, dst = (torch.tensor(x, dtype=torch.int32) if not isinstance(x, torch.Tensor) else x for x in (src, dst))
    x = pool.clone().cuda()
    got = ssm.state_slots_copy(x, src.cuda(), dst.cuda(), dim=dim)
    assert got.data_ptr() == x.data_ptr()
    assert torch.equal(got.cpu(), O.slots_copy(pool, src, dst, dim))


SHAPES = [((6, 40), torch.float32, 0), ((6, 3), torch.uint8, 0), ((3, 6, 5, 7), torch.bfloat16, 1), ((6, 1), torch.float32, 0),
          ((2, 2, 6, 1024), torch.float32, 2), ((4, 6, 4 * 1024 + 4), torch.float32, 1), ((6, 515 * 3), torch.float32, 0),
          ((6, 2), torch.bfloat16, 0), ((6,), torch.int64, 0), ((1, 6, 70000), torch.uint8, 1)]


@pytest.mark.parametrize("shape, dtype, dim", SHAPES)
def test_every_kind_of_move(shape, dtype, dim):
    pool = pool_of(shape, dtype)
    move(pool, [0, 0, 0], [1, 2, 3], dim)                         # fork
    move(pool, [1, 2, 3, 4, 5, 0], [0, 1, 2, 3, 4, 5], dim)       # a cycle
    move(pool, [1, 0], [0, 1], dim)                               # two change places
    move(pool, [5, 4], [0, 1], dim)                               # compact
    move(pool, [-1, -7], [2, 4], dim)                             # clear
    move(pool, [3, 3], [3, 0], dim)                               # onto itself
    move(pool, [0, 1, 2, -1], [5, 5, 5, 5], dim)                  # one destination: the last counts
    move(pool, [2, 4, 4], [4, 4, 2], dim)
    move(pool, [6, 1, 9, 1], [0, -1, 1, 6], dim)                  # slots that are not there
    move(pool, [6, 1], [3, 3], dim)
    move(pool, [1, 6], [3, 3], dim)
    move(pool, [], [], dim)


@pytest.mark.parametrize("n, slots, size", [(2, 3, 5000), (16, 20, 5000), (17, 30, 100), (64, 64, 3001), (255, 300, 64),
                                            (256, 256, 33), (257, 300, 1000), (1024, 1500, 48), (1025, 1500, 64),
                                            (2048, 2048, 100), (2048, 100000, 3)])
def test_random_maps(n, slots, size):
    g = torch.Generator().manual_seed(n)
    pool = pool_of((2, slots, size), torch.float32, n)
    src = torch.randint(-2, slots + 1, (n,), generator=g, dtype=torch.int32)
    dst = torch.randint(-1, slots + 1, (n,), generator=g, dtype=torch.int32)
    move(pool, src, dst, 1)                                       # destinations named twice among them
    order = torch.randperm(slots, generator=g)[:n].int()
    move(pool, order[torch.randint(0, n, (n,), generator=g)], order, 1)


def test_unaligned_pools():
    for dtype, first in ((torch.uint8, 1), (torch.uint8, 4), (torch.bfloat16, 1), (torch.float32, 1), (torch.float32, 4)):
        base = pool_of((first + 6 * 64,), dtype).cuda()
        pool = base[first:].view(6, 64)
        want = O.slots_copy(pool, torch.tensor([1, 0, 5]), torch.tensor([0, 1, 2]))
        head = base[:first].clone()
        ssm.state_slots_copy(pool, torch.tensor([1, 0, 5], dtype=torch.int32).cuda(),
                             torch.tensor([0, 1, 2], dtype=torch.int32).cuda())
        assert torch.equal(pool.cpu(), want) and torch.equal(base[:first], head)


def test_offsets_past_32_bits():
    pool = torch.empty(2, 40, 1 << 26, dtype=torch.uint8, device="cuda")      # 5.4 GB
    for i in range(40):
        pool[:, i] = i + 1
    ssm.state_slots_copy(pool, torch.tensor([39, 0, -1], dtype=torch.int32).cuda(),
                         torch.tensor([0, 39, 20], dtype=torch.int32).cuda(), dim=1)
    for i, v in ((0, 40), (39, 1), (20, 0), (38, 39), (21, 22)):
        assert (pool[:, i] == v).all()


def test_captured_and_replayed():
    pool = pool_of((3, 8, 100), torch.float32).cuda()
    src = torch.tensor([1, 2, 3], dtype=torch.int32).cuda()
    dst = torch.tensor([0, 1, 2], dtype=torch.int32).cuda()
    ssm.state_slots_copy(pool, src, dst, dim=1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ssm.state_slots_copy(pool, src, dst, dim=1)
    for n in range(4):
        src.copy_(torch.randint(-1, 8, (3,), generator=torch.Generator().manual_seed(n)).int())
        want = O.slots_copy(pool, src.cpu(), dst.cpu(), 1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(pool.cpu(), want), n
