"""Pages: the allocator's compaction and resizing (CPU), and the copies of all layers' pools (GPU)."""
import ctypes as C

import numpy as np
import pytest

from continuous_batching_gb300 import binding as bd

torch = pytest.importorskip("torch")


def _filled(seed, nb=40, bs=16):
    """An allocator with admitted, forked, trimmed and freed sequences."""
    rng = np.random.default_rng(seed)
    a = bd.Allocator(nb, bs)
    for s in range(6):
        a.admit(s, int(rng.integers(1, 6)) * bs - int(rng.integers(0, bs)))
    a.fork(1, 10)
    a.cow(10, 0, 1)
    a.free_seq(int(rng.integers(2, 4)))
    a.free_seq(0)
    a.trim(5, 3)
    return a


def _seqs(a):
    out = {}
    for s in range(16):
        try:
            out[s] = a.table(s)
        except bd.PagedAttnError:
            pass
    return out


@pytest.mark.parametrize("seed", range(8))
def test_compaction_moves_the_live_blocks_down(seed):
    a = _filled(seed)
    before, free = _seqs(a), a.num_free
    refs = {b: a.refcount(b) for b in range(a.num_blocks)}
    pairs = a.compact()
    a.check_consistent()
    live = a.num_blocks - free
    move = dict(pairs)
    assert a.num_free == free
    assert all(old >= live and new < live and refs[old] > 0 and refs[new] == 0 for old, new in pairs)
    assert len(set(move)) == len(pairs) == len(set(move.values()))
    after = _seqs(a)
    assert after == {s: [move.get(b, b) for b in t] for s, t in before.items()}
    assert {b for t in after.values() for b in t} == set(range(live))
    assert all(a.refcount(move.get(b, b)) == n for b, n in refs.items() if n)
    assert a.compact() == []
    if free:
        assert a.alloc() == live                          # the lowest free id is next
        a.free(live)
    a.resize(live)
    a.check_consistent()
    assert a.num_free == 0
    with pytest.raises(bd.PoolExhausted):
        a.ensure_capacity(5, 16 * 30)
    a.resize(live + 7)
    a.check_consistent()
    assert a.num_free == 7 and a.alloc() == live


def test_compaction_changes_nothing_on_an_error():
    a = _filled(2)
    before = _seqs(a)
    lib, k = bd.load(), C.c_int32()
    pairs = np.full(2, -5, np.int32)
    need = len(_filled(2).compact())
    assert need > 1
    assert lib.pa_alloc_compact(a._h, pairs.ctypes.data_as(C.POINTER(C.c_int32)), 1, C.byref(k)) == bd.PA_ERR_INVALID
    assert k.value == need and _seqs(a) == before and (pairs == -5).all()
    a.check_consistent()
    assert lib.pa_alloc_compact(None, None, 0, C.byref(k)) == bd.PA_ERR_INVALID
    # a block held outside the tables cannot be renamed
    b = bd.Allocator(8, 16)
    held = [b.alloc() for _ in range(3)]
    b.free(held[0])
    with pytest.raises(bd.PagedAttnError) as e:
        b.compact()
    assert e.value.status == bd.PA_ERR_STATE and b.refcount(held[2]) == 1 and b.refcount(held[0]) == 0


def test_resize_refuses_live_tails_and_empties():
    a = bd.Allocator(10, 8)
    a.admit(3, 30)
    with pytest.raises(bd.PagedAttnError) as e:
        a.resize(3)
    assert e.value.status == bd.PA_ERR_STATE and a.num_blocks == 10 and a.num_free == 6
    a.resize(4)
    a.check_consistent()
    a.free_seq(3)
    a.resize(0)
    assert a.compact() == [] and a.num_free == 0
    with pytest.raises(bd.PagedAttnError):
        a.resize(-1)


def test_copy_refuses():
    lib = bd.load()
    one = (bd.Pages * 1)(bd.Pages(4096, 64))
    call = lambda pools=one, n=1, pairs=4096, n_pairs=2, nb=4: lib.paged_copy_pages(pairs, n_pairs, pools, n, nb, None, None)
    assert call(n_pairs=-1) == bd.PA_ERR_INVALID and call(nb=-1) == bd.PA_ERR_INVALID and call(pools=None) == bd.PA_ERR_INVALID
    assert call(pairs=None) == bd.PA_ERR_INVALID
    for bad in (bd.Pages(4100, 64), bd.Pages(None, 64), bd.Pages(4096, 60), bd.Pages(4096, 0), bd.Pages(4096, -16)):
        assert call(pools=(bd.Pages * 1)(bad)) == bd.PA_ERR_INVALID
    assert call(n_pairs=0, pairs=None) == bd.PA_OK and call(n=0, pools=None) == bd.PA_OK


# -------------------------------------------------------------------------------------- GPU

@pytest.mark.gpu
@pytest.mark.parametrize("n_pools", [1, 7, 130])          # 130: two launches
@pytest.mark.parametrize("page", [16, 2064, 5120])
def test_pages_of_every_pool_move(n_pools, page):
    rng = np.random.default_rng(page)
    nb = 23
    # pools of other page sizes among them
    sizes = [page if i % 3 else 16 * (1 + i % 5) for i in range(n_pools)]
    pools = [torch.randint(0, 256, (nb, s), dtype=torch.uint8, device="cuda") for s in sizes]
    ids = rng.permutation(nb)[:18].astype(np.int32).reshape(-1, 2)
    ids[3] = ids[3][0]                                    # a page onto itself: skipped
    ids[5, 1] = nb                                        # outside the pools: skipped
    want = [p.cpu().clone() for p in pools]
    for w in want:
        for a, b in ids.tolist():
            if b < nb:
                w[b] = w[a]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    bd.paged_copy_pages(torch.from_numpy(ids).cuda(), pools, err=err)
    assert all(torch.equal(p.cpu(), w) for p, w in zip(pools, want))
    assert int(err.item()) == bd.PA_DEVERR_BLOCK


@pytest.mark.gpu
def test_pools_of_any_type_and_a_captured_compaction():
    """bf16, e4m3 and 4-bit pools in one call, captured; replayed after the pairs were rewritten."""
    nb = 12
    pools = [torch.randn(nb, 16, 2, 64, device="cuda").bfloat16(), torch.randint(0, 256, (nb, 16, 2, 64), dtype=torch.uint8, device="cuda"),
             torch.randint(0, 256, (nb, 2, 16 * 40), dtype=torch.uint8, device="cuda")]
    pairs = torch.tensor([[9, 1], [11, 4]], dtype=torch.int32, device="cuda")
    bd.paged_copy_pages(pairs, pools)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bd.paged_copy_pages(pairs, pools)
    pairs.copy_(torch.tensor([[8, 0], [10, 5]], dtype=torch.int32))
    before = [p.clone() for p in pools]
    graph.replay()
    torch.cuda.synchronize()
    for p, b in zip(pools, before):
        w = b.clone()
        w[0], w[5] = b[8], b[10]
        assert torch.equal(p.view(torch.uint8), w.view(torch.uint8))
    with pytest.raises(ValueError):
        bd.paged_copy_pages(pairs, [pools[0], pools[1][:5]])


@pytest.mark.gpu
def test_pages_behind_four_gigabytes():
    nb, page = 70000, 1 << 16
    pool = torch.empty(nb, page, dtype=torch.uint8, device="cuda")
    pool[nb - 1] = 5
    pool[nb - 2] = 0
    pool[3] = 0
    bd.paged_copy_pages(torch.tensor([[nb - 1, 3]], dtype=torch.int32, device="cuda"), [pool])
    bd.paged_copy_pages(torch.tensor([[3, nb - 2]], dtype=torch.int32, device="cuda"), [pool])
    assert bool((pool[3] == 5).all()) and bool((pool[nb - 2] == 5).all())
