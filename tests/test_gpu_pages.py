"""GPU: pages of a state pool, copied, cleared and compacted: exact."""
import pytest
import torch

import ssd_chunked_scan_fwd_amd as ssd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ssd.lib()


def pool_of(layers, slots, *page, dtype=torch.float32, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-120, 120, (layers, slots) + page, generator=g).to(dtype).cuda()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def copied(pool, src, dst):
    old, new = pool.clone(), pool.clone()
    for a, b in zip(src, dst):
        if 0 <= a < pool.shape[1] and 0 <= b < pool.shape[1]:
            new[:, b] = old[:, a]
    return new


PAGES = [((2, 8, 64), torch.float32), ((1, 3), torch.float32), ((5,), torch.bfloat16), ((7, 129), torch.int8),
         ((4, 64, 64), torch.float32), ((1,), torch.float32)]


@pytest.mark.parametrize("page,dtype", PAGES)
@pytest.mark.parametrize("layers", [1, 3])
def test_copy(page, dtype, layers):
    """A fork, a swap, a rotation, a chain, pairs left out, the last of several to one page."""
    lists = [([0], [1]), ([0, 0, 0], [1, 2, 3]), ([0, 1], [1, 0]), ([1, 2, 3, 4, 0], [0, 1, 2, 3, 4]), ([0, 1, 2, 3], [1, 2, 3, 4]),
             ([0, -1, 3, 99, 2], [5, 6, -1, 1, 900]), ([1, 2, 3], [0, 0, 0]), ([4, 5], [4, 5]), ([0, 9, 1], [9, 9, 0]),
             ([2, 99, 3], [7, 7, -5])]
    for src, dst in lists:
        print(f"[pages] copy {page} {dtype} x{layers} {src}->{dst}", flush=True)
        p = pool_of(layers, 10, *page, dtype=dtype)
        want = copied(p, src, dst)
        ssd.pages_copy(p, i32(src), i32(dst))
        assert torch.equal(p, want), (src, dst)


@pytest.mark.parametrize("n", [64, 65, 128, 200, 257, 512, 700, 1024])
def test_copy_permutes_many(n):
    print(f"[pages] permutation of {n}", flush=True)
    p = pool_of(2, n, 3, 40)
    perm = torch.randperm(n, generator=torch.Generator().manual_seed(n)).to(torch.int32)
    want = p.clone()
    want[:, torch.arange(n)] = p[:, perm.long()]
    ssd.pages_copy(p, perm.cuda(), torch.arange(n, dtype=torch.int32, device="cuda"))
    assert torch.equal(p, want)


def test_copy_nothing():
    p = pool_of(1, 4, 8)
    want = p.clone()
    ssd.pages_copy(p, i32([]), i32([]))
    ssd.pages_clear(p, i32([]))
    assert torch.equal(p, want)


@pytest.mark.parametrize("page,dtype", PAGES)
def test_clear(page, dtype):
    p = pool_of(2, 6, *page, dtype=dtype) + 1
    want = p.clone()
    want[:, [1, 4]] = 0
    ssd.pages_clear(p, i32([4, 1, -1, 6, 1]))
    assert torch.equal(p, want)


def compacted(pool, live):
    count = sum(live)
    holes = [i for i in range(count) if not live[i]]
    high = [i for i in range(count, len(live)) if live[i]]
    where = [i if live[i] else -1 for i in range(len(live))]
    new = pool.clone()
    for a, b in zip(high, holes):
        new[:, b] = pool[:, a]
        where[a] = b
    return new, where, count


@pytest.mark.parametrize("slots", [1, 2, 63, 64, 65, 500, 1024, 1025, 5000])
@pytest.mark.parametrize("share", [0.0, 0.03, 0.5, 0.97, 1.0])
def test_compact(slots, share):
    live = torch.rand(slots, generator=torch.Generator().manual_seed(slots)) < share
    print(f"[pages] compact {slots} slots, {int(live.sum())} live", flush=True)
    p = pool_of(2, slots, 3, 20)
    want, where, count = compacted(p, live.int().tolist())
    w, c = ssd.pages_compact(p, live.cuda())
    assert torch.equal(p, want) and w.tolist() == where and c.tolist() == [count]


@pytest.mark.parametrize("page,dtype", PAGES)
def test_compact_pages(page, dtype):
    live = [0, 1, 0, 0, 1, 1, 0, 2, 255]
    p = pool_of(3, 9, *page, dtype=dtype)
    want, where, count = compacted(p, [int(v != 0) for v in live])
    w, c = ssd.pages_compact(p, torch.tensor(live, dtype=torch.uint8, device="cuda"))
    assert torch.equal(p, want) and w.tolist() == where and c.tolist() == [count]


def test_pool_not_on_a_boundary():
    """A pool that starts 4 bytes into its allocation."""
    raw = pool_of(1, 1, 6 * 64 + 1).view(-1)
    p = raw[1:].view(1, 6, 64)
    want = copied(p, [0, 1], [1, 0])
    ssd.pages_copy(p, i32([0, 1]), i32([1, 0]))
    assert torch.equal(p, want)


def test_pool_beyond_32_bits():
    """A pool of 6 GiB: pages whose offsets pass 2^32 bytes."""
    p = torch.zeros(1, 6, 1 << 30, dtype=torch.uint8, device="cuda")
    for i in range(6):
        p[0, i, :4] = i + 1
        p[0, i, -4:] = 10 * (i + 1)
    ssd.pages_copy(p, i32([5, 0]), i32([0, 5]))
    assert p[0, :, 0].tolist() == [6, 2, 3, 4, 5, 1] and p[0, :, -1].tolist() == [60, 20, 30, 40, 50, 10]
    w, c = ssd.pages_compact(p, torch.tensor([0, 1, 0, 0, 0, 1], dtype=torch.uint8, device="cuda"))
    assert w.tolist() == [-1, 1, -1, -1, -1, 0] and c.item() == 2 and p[0, 0, -1].item() == 10
    ssd.pages_clear(p, i32([4]))
    assert p[0, :, -1].tolist() == [10, 20, 30, 40, 0, 10]
