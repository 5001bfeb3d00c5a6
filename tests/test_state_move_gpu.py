"""Moves of cache rows against indexing on the host: bits have to be equal."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lr():
    import linear_recurrence_gb300 as m
    m.load_library()
    return m


def run(lr, cache, src, dst, layers):
    at = 1 if layers else 0
    want = cache.clone()
    for a, b in zip(src, dst):
        if b < 0 or b >= cache.shape[at] or a >= cache.shape[at]:
            continue
        value = cache.select(at, a) if a >= 0 else torch.zeros_like(cache.select(at, 0))
        want.select(at, b).copy_(value)
    dev = cache.cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    lr.state_move(dev, torch.tensor(src, **i32), torch.tensor(dst, **i32), layers=layers)
    got = dev.cpu()
    assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.uint8, torch.int64])
@pytest.mark.parametrize("shape", [(40, 64, 16), (40, 5, 3), (40, 1, 1), (40, 1030, 3), (40, 333, 7)], ids=str)
@pytest.mark.parametrize("layers", [0, 3])
def test_permutations_forks_and_frees(lr, dtype, shape, layers):
    g = torch.Generator().manual_seed(shape[1])
    full = (layers, *shape) if layers else shape
    cache = torch.randint(0, 255, full, generator=g).to(dtype)
    n = shape[0]
    perm = torch.randperm(n, generator=g).tolist()
    run(lr, cache, perm, list(range(n)), bool(layers))                      # a permutation: every row is source and target
    run(lr, cache, [3] * 7, [9, 1, 2, 0, 39, 20, 21], bool(layers))         # a fork, row 3 itself untouched
    run(lr, cache, [5, 6, -1, 3, 8], [6, 5, 7, -1, 3], bool(layers))        # a swap, a free, a skipped move, a chain
    run(lr, cache, [4], [4], bool(layers))
    assert lr.get_last_error() == lr.SSCAN_OK


@pytest.mark.parametrize("dtype", [torch.float32, torch.uint8])
def test_off_a_vector_boundary(lr, dtype):
    g = torch.Generator().manual_seed(1)
    whole = torch.randint(0, 255, (1 + 20 * 48,), generator=g).to(dtype).cuda()
    cache = whole[1:].view(20, 48)
    want = cache.clone()
    want[7], want[2] = cache[2], cache[7]
    i32 = dict(dtype=torch.int32, device="cuda")
    first = whole[0].clone()
    lr.state_move(cache, torch.tensor([2, 7], **i32), torch.tensor([7, 2], **i32))
    assert torch.equal(cache, want) and whole[0] == first


def test_many_moves(lr):
    g = torch.Generator().manual_seed(2)
    n = lr.STATE_MOVE_MAX
    cache = torch.randn(n, 9, generator=g)
    run(lr, cache, torch.randperm(n, generator=g).tolist(), torch.randperm(n, generator=g).tolist(), False)
    cache = torch.randn(n, 12, generator=g)
    run(lr, cache, torch.randperm(n, generator=g).tolist(), torch.randperm(n, generator=g).tolist(), False)


def test_values_of_rows_are_kept_bit_for_bit(lr):
    cache = torch.tensor([[float("nan"), float("inf"), -0.0, 1e-45]] * 4)
    cache[1] = 0
    run(lr, cache, [0], [1], False)


def test_rows_out_of_range_are_skipped_and_reported(lr):
    cache = torch.arange(40.0).view(10, 4)
    run(lr, cache, [10, 3, 2], [1, 11, 4], False)
    assert lr.get_last_error() == lr.SSCAN_ERR_INVALID
    assert lr.get_last_error() == lr.SSCAN_OK


def test_nothing_to_do(lr):
    cache = torch.arange(8.0, device="cuda").view(2, 4)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert torch.equal(lr.state_move(cache, none, none), torch.arange(8.0, device="cuda").view(2, 4))


def test_beyond_32_bits(lr):
    """Rows whose place in the cache passes 2^32 bytes."""
    cache = torch.zeros(18, 300_000_000, dtype=torch.uint8, device="cuda")
    cache[17] = 7
    cache[3, -1] = 9
    i32 = dict(dtype=torch.int32, device="cuda")
    lr.state_move(cache, torch.tensor([17, 3], **i32), torch.tensor([3, 16], **i32))
    assert bool((cache[3] == 7).all()) and int(cache[16, -1]) == 9 and int(cache[16].long().sum()) == 9 and not cache[:3].any()


def test_captured(lr):
    cache = torch.randn(6, 100, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    src, dst = torch.tensor([0, 1], **i32), torch.tensor([1, 0], **i32)
    before = cache.clone()
    lr.state_move(cache, src, dst)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lr.state_move(cache, src, dst)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(cache, before)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(cache[0], before[1]) and torch.equal(cache[1], before[0])
