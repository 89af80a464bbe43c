"""The paged cache's page operations and append on the GPU against the same
steps on host lists: whole numbers and moved bytes must be equal."""
import random

import pytest
import torch

from routed_expert_ffn_router_gb300 import _lib
from routed_expert_ffn_router_gb300 import build as libbuild
from routed_expert_ffn_router_gb300.paged import PagedKV
from tests._kv_ref import Books

pytestmark = pytest.mark.gpu
OK, DEVICE = _lib.MOE_OK, _lib.MOE_ERR_DEVICE


@pytest.fixture(scope="module", autouse=True)
def _built():
    libbuild.build()
    _lib.load()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(n_layers=2, n_pages=64, page=16, Hkv=2, D=64, n_slots=12, max_pages=10, dtype=torch.bfloat16, seed=0):
    kv = PagedKV(n_layers, n_pages, page, Hkv, D, n_slots, max_pages, dtype=dtype, max_rows=64)
    g = torch.Generator(device="cuda").manual_seed(seed)
    for pool in (kv.k, kv.v):
        pool.copy_(torch.randn(pool.shape, generator=g, device="cuda"))
    return kv, books(kv)


def books(kv):
    return Books(kv.k, kv.v, kv.table, kv.lens, kv.refs, kv.free, kv.n_free)


def same(kv, b, what=""):
    torch.cuda.synchronize()
    assert kv.status() == (OK, 0), what
    b.check(kv, what)


@pytest.mark.parametrize("shape", [dict(), dict(page=1, Hkv=1, D=8, n_pages=200, max_pages=40),
                                   dict(page=24, D=80, n_layers=1), dict(page=64, Hkv=3, D=128, n_pages=40, max_pages=4),
                                   dict(n_pages=9000, n_slots=40, max_pages=300, Hkv=1, D=8, n_layers=1),
                                   dict(page=8, D=256, n_pages=70, dtype=torch.float16)])
def test_a_life_of_random_operations(shape):
    kv, b = make(**shape)
    rng = random.Random(len(str(shape)))
    n_slots, cap = kv.n_slots, kv.table.shape[1] * kv.k.shape[3]
    for step in range(60):
        busy = [s for s in range(n_slots) if b.lens[s] > 0]
        idle = [s for s in range(n_slots) if b.lens[s] == 0]
        op = rng.choice(["grow", "grow", "fork", "free", "compact"])
        if op == "grow":
            slots, add, free = [], [], len(b.stack)
            for s in rng.sample(range(n_slots), rng.randint(1, n_slots)):
                a = rng.choice([0, 1, 2, rng.randint(0, cap)])
                a = min(a, cap - b.lens[s])
                need = b.n(b.lens[s] + a) - b.n(b.lens[s])
                # a partly filled page that is shared must not grow: forks copy it, so it never is
                if need <= free:
                    slots.append(s), add.append(a)
                    free -= need
            if slots:
                kv.grow(i32(slots), i32(add))
                b.grow(slots, add)
        elif op == "fork" and busy and idle:
            dst = rng.sample(idle, rng.randint(1, len(idle)))
            src = [rng.choice(busy) for _ in dst]
            if sum(b.lens[a] % b.page > 0 for a in src) <= len(b.stack):
                kv.fork(i32(src), i32(dst))
                b.fork(src, dst)
        elif op == "free" and busy:
            gone = rng.sample(range(n_slots), rng.randint(1, max(1, n_slots // 2)))  # idle ones among them
            kv.free_slots(i32(gone))
            b.free(gone)
        elif op == "compact":
            moved = i32([-1])
            kv.compact(moved)
            assert int(moved) == b.compact()
        same(kv, b, f"step {step}: {op}")


def test_large_pool_of_small_pages():
    kv, b = make(n_layers=1, n_pages=70001, page=1, Hkv=1, D=8, n_slots=1500, max_pages=50)
    slots = list(range(1500))
    add = [(i * 7) % 47 for i in slots]
    kv.grow(i32(slots), i32(add))
    b.grow(slots, add)
    same(kv, b, "grow")
    kv.free_slots(i32(slots[::2]))
    b.free(slots[::2])
    same(kv, b, "free")
    kv.compact()
    b.compact()
    same(kv, b, "compact")


def test_out_of_pages_changes_nothing():
    kv, b = make(n_pages=8, max_pages=8, n_slots=6)
    kv.grow(i32([0, 1]), i32([16 * 3 + 1, 16 * 2]))   # 4 and 2 pages: 2 are left
    b.grow([0, 1], [16 * 3 + 1, 16 * 2])
    same(kv, b, "grow")
    kv.grow(i32([2, 3]), i32([17, 17]))               # 4 more
    assert kv.status() == (DEVICE, 32)
    kv.clear_status()
    same(kv, b, "a growth that does not fit")
    kv.fork(i32([0, 0, 0]), i32([2, 3, 4]))           # 3 copies of the last page
    assert kv.status() == (DEVICE, 32)
    kv.clear_status()
    same(kv, b, "forks that do not fit")
    kv.fork(i32([0, 0]), i32([2, 3]))
    b.fork([0, 0], [2, 3])
    same(kv, b, "forks that fit")


def test_refused_arguments_change_nothing():
    kv, b = make()
    kv.grow(i32([0]), i32([40]))
    b.grow([0], [40])
    calls = [lambda: kv.grow(i32([1, 12]), i32([1, 1])), lambda: kv.grow(i32([1, -1]), i32([1, 1])),
             lambda: kv.grow(i32([1, 2]), i32([1, -1])), lambda: kv.grow(i32([1]), i32([161])),
             lambda: kv.grow(i32([0]), i32([2147483647])),
             lambda: kv.fork(i32([0]), i32([12])), lambda: kv.fork(i32([12]), i32([1])),
             lambda: kv.fork(i32([0, 0]), i32([1, 0])), lambda: kv.fork(i32([-1]), i32([1]))]
    for i, call in enumerate(calls):
        call()
        assert kv.status() == (DEVICE, 64), i
        kv.clear_status()
        same(kv, b, f"call {i}")
    kv.free_slots(i32([12, -3]))
    assert kv.status() == (DEVICE, 2)
    kv.clear_status()
    same(kv, b, "slots out of range")


def test_copy_pages():
    kv, b = make(page=16, Hkv=3, D=80, n_pages=33)
    src, dst = [0, 5, 5, 32], [1, 2, 31, 9]
    kv.copy_pages(i32(src), i32(dst))
    b.copy(src, dst)
    same(kv, b, "copy")
    kv.copy_pages(i32([0, 40, 3, -1]), i32([4, 6, 33, 7]))
    assert kv.status() == (DEVICE, 2)
    kv.clear_status()
    b.copy([0], [4])
    same(kv, b, "pairs out of range are skipped")


@pytest.mark.parametrize("D,page,dtype", [(64, 16, torch.bfloat16), (8, 1, torch.float16), (80, 24, torch.bfloat16),
                                          (256, 64, torch.float16)])
def test_append(D, page, dtype):
    kv, b = make(n_layers=3, n_pages=80, page=page, Hkv=2, D=D, max_pages=60, n_slots=6, dtype=dtype)
    lens = [0, 1, 5, 17, 30]
    kv.grow(i32([0, 1, 2, 3, 4]), i32(lens))
    b.grow([0, 1, 2, 3, 4], lens)
    slots = i32([4, 1, 0, 3])           # 2 rows each: slot 0 has no token, slot 1 only the second
    wide = torch.randn(8, 5, D, device="cuda").to(dtype)
    k, v = wide[:, 1:3], wide[:, 3:5]
    kv.append(1, k, v, slots=slots)
    news = [3, 0, 0, 5]
    start = i32([0, 3, 3, 3, 8])
    kv.append(2, k, v, slots=slots, row_start=start)
    torch.cuda.synchronize()

    def put(layer, t, s, tok):
        if tok < 0:
            return
        p = b.table[s][tok // page]
        b.k[layer, p, :, tok % page], b.v[layer, p, :, tok % page] = k[t].cpu(), v[t].cpu()

    for i, s in enumerate(slots.tolist()):
        for j in range(2):
            put(1, 2 * i + j, s, lens[s] - 2 + j)
        for j in range(news[i]):
            put(2, int(start[i]) + j, s, lens[s] - news[i] + j)
    same(kv, b, "append")
    # a page out of range: the row is not written
    kv.table[4, (30 - 1) // page] = 80
    before = kv.k.clone()
    kv.append(0, k[:1], v[:1], slots=i32([4]))
    assert kv.status() == (DEVICE, 2)
    assert torch.equal(kv.k.view(torch.int16), before.view(torch.int16))


def test_operations_in_a_graph_on_another_stream():
    kv, b = make(n_pages=100)
    s = torch.cuda.Stream()
    src, dst, gone, add = i32([0, 1]), i32([4, 5]), i32([0, 4, 5]), i32([33, 20])
    two = i32([0, 1])
    torch.cuda.synchronize()

    def cycle():
        kv.grow(two, add)
        kv.fork(src, dst)
        kv.free_slots(gone)
        kv.compact()
        kv.free_slots(two)

    def host():
        b.grow([0, 1], [33, 20])
        b.fork([0, 1], [4, 5])
        b.free([0, 4, 5])
        b.compact()
        b.free([0, 1])

    with torch.cuda.stream(s):
        cycle()
    host()
    s.synchronize()
    same(kv, b, "once")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        cycle()
    for i in range(3):
        g.replay()
        host()
        torch.cuda.synchronize()
        same(kv, b, f"replay {i}")


def test_pools_beyond_2_to_the_32_elements():
    page, Hkv, D = 64, 8, 128
    n_pages = (1 << 32) // (page * Hkv * D) + 64
    kv = PagedKV(1, n_pages, page, Hkv, D, n_slots=4, max_pages=n_pages)
    kv.grow(i32([0, 1]), i32([(n_pages - 10) * page, 70]))   # slot 1 at the end of the pool
    k = torch.randn(70, Hkv, D, device="cuda").bfloat16()
    kv.append(0, k, -k, slots=i32([1]))
    kv.fork(i32([1]), i32([2]))
    torch.cuda.synchronize()
    assert kv.status() == (OK, 0)
    t = kv.table[1, :2].tolist()
    assert t == [n_pages - 10, n_pages - 9] and kv.table[2, :2].tolist() == [n_pages - 10, n_pages - 8]
    for p in (t[1], n_pages - 8):
        assert torch.equal(kv.k[0, p, :, :6], k[64:].transpose(0, 1)) and torch.equal(kv.v[0, p, :, :6], -k[64:].transpose(0, 1))
    kv.free_slots(i32([0]))
    kv.compact()
    torch.cuda.synchronize()
    assert kv.table[1, :2].tolist() == [0, 1] and kv.table[2, :2].tolist() == [0, 2] and int(kv.n_free) == n_pages - 3
    assert torch.equal(kv.k[0, 0], k[:64].transpose(0, 1)) and torch.equal(kv.v[0, 2, :, :6], -k[64:].transpose(0, 1))
    del kv
    torch.cuda.empty_cache()
