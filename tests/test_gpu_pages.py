"""Page copies, row compaction and batched forks on the device, against indexed copies."""
import numpy as np
import pytest
import torch

import paged_kv_cache_decode_gb300 as pkv

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def filled(L, pages, H, D, P, dtype, seed=0, **kw):
    pool = pkv.Pool(L, pages, H, D, P, dtype, P * pages, **kw)
    g = torch.Generator("cuda").manual_seed(seed)
    views = [x for l in range(L) for x in pool.kv_pages(l)]
    for x in views:
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
    return pool, views, [x.clone() for x in views]


def i32(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


SHAPES = [(1, 2, 2, 16, "bf16"), (3, 1, 8, 16, "f32"), (2, 5, 64, 48, "bf16"), (12, 12, 64, 16, "f32"),
          (2, 32, 128, 64, "bf16"), (1, 3, 256, 16, "bf16"), (1, 1, 2, 16, "bf16"), (1, 1, 4, 16, "f32")]


@pytest.mark.parametrize("L,H,D,P,dtype", SHAPES)
@pytest.mark.parametrize("n,src", [(1, 1), (7, 7), (30, 1), (500, 90)])
def test_copy_pages(L, H, D, P, dtype, n, src):
    pages = n + src + 3
    pool, views, was = filled(L, pages, H, D, P, dtype, n)
    try:
        rng = np.random.default_rng(n)
        perm = rng.permutation(pages)
        dst, s = perm[:n], rng.choice(perm[n:n + src], size=n)
        pool.copy_pages(i32(s), i32(dst))
        assert pool.check_device_status() == 0
        for x, y in zip(views, was):
            y[torch.from_numpy(dst).cuda()] = y[torch.from_numpy(s).cuda()]
            assert torch.equal(x, y)
    finally:
        pool.close()


def test_copy_pages_skips_ids_outside_the_pool():
    pool, views, was = filled(2, 6, 2, 64, 16, "bf16")
    try:
        pool.copy_pages(i32([0, 1, -1, 2, 6]), i32([3, 6, 4, 5, 4]))
        assert pool.device_status_bits() == pkv.PKV_DEVERR_PAGE_ID
        for x, y in zip(views, was):
            y[3], y[5] = y[0], y[2]
            assert torch.equal(x, y)
        pool.copy_pages(i32([]), i32([]))
        with pytest.raises(ValueError):
            pool.copy_pages(i32([0, 1]), i32([2]))
        with pytest.raises(ValueError):
            pool.copy_pages(torch.zeros(1, dtype=torch.int64, device="cuda"), i32([2]))
    finally:
        pool.close()


def test_copy_pages_past_32_bit_offsets():
    """A pool of more than 2^31 elements a layer: the last pages are reached."""
    pool = pkv.Pool(1, 33000, 32, 128, 16, "bf16", 64)
    try:
        k, v = pool.kv_pages(0)
        k[32998].fill_(3.0)
        v[32999].fill_(4.0)
        pool.copy_pages(i32([32998, 32999]), i32([32997, 0]))
        assert pool.check_device_status() == 0
        assert (k[32997] == 3).all() and (v[0] == 4).all() and (k[0] == 0).all() and (v[32997] == 0).all()
    finally:
        pool.close()


@pytest.mark.parametrize("L,H,D,P,dtype", SHAPES)
@pytest.mark.parametrize("lens,share", [([1], 1.0), ([40, 0, 200, 16], 0.5), ([100, 33], 0.0), ([700], 0.9)])
def test_compact_pages(L, H, D, P, dtype, lens, share):
    rng = np.random.default_rng(len(lens))
    keep = [np.flatnonzero(rng.random(t) < share) for t in lens]
    if lens == [40, 0, 200, 16]:
        keep[2] = rng.permutation(keep[2])              # any order
    need, out = [-(-t // P) for t in lens], [-(-len(k) // P) for k in keep]
    pages = sum(need) + sum(out) + 2
    pool, views, was = filled(L, pages, H, D, P, dtype, 3)
    try:
        perm = list(rng.permutation(pages))
        tables = np.full((len(lens), max(need) + 1), -1, np.int32)
        new = np.full((len(lens), max(out) + 1), -1, np.int32)
        for b in range(len(lens)):
            tables[b, :need[b]] = [perm.pop() for _ in range(need[b])]
            new[b, :out[b]] = [perm.pop() for _ in range(out[b])]
        cu = np.concatenate([[0], np.cumsum([len(k) for k in keep])])
        pool.compact_pages(i32(np.concatenate(keep)), i32(cu), i32(tables), i32(lens), i32(new))
        assert pool.check_device_status() == 0
        for x, y in zip(views, was):
            want = y.clone()
            for b, k in enumerate(keep):
                for i, pos in enumerate(k):
                    want[new[b, i // P], :, i % P] = y[tables[b, pos // P], :, pos % P]
            assert torch.equal(x, want)
    finally:
        pool.close()


def test_compact_pages_refuses_rows_that_do_not_fit():
    pool, views, was = filled(1, 8, 2, 64, 16, "f32")
    try:
        tables, new = i32([[0, 1, -1]]), i32([[4]])
        # position 20 past the length, -1, and a 17th row past the new table
        pool.compact_pages(i32([3, 20, -1]), i32([0, 3]), tables, i32([20]), new)
        assert pool.device_status_bits() == pkv.PKV_DEVERR_SEQ_LEN
        want = was[0].clone()
        want[4, :, 0] = was[0][0, :, 3]
        assert torch.equal(views[0], want)
        pool.compact_pages(i32(list(range(17))), i32([0, 17]), tables, i32([20]), new)
        assert pool.device_status_bits() == pkv.PKV_DEVERR_SEQ_LEN
        pool.compact_pages(i32([3, 40]), i32([0, 2]), tables, i32([48]), i32([[5]]))
        assert pool.device_status_bits() == pkv.PKV_DEVERR_PAGE_ID
        pool.compact_pages(i32([]), i32([0, 0]), tables, i32([20]), new)
        assert pool.check_device_status() == 0
    finally:
        pool.close()


def test_pages_captured_on_a_stream_and_replayed():
    pool, views, was = filled(2, 12, 4, 64, 16, "bf16")
    try:
        src, dst = i32([0, 1]), i32([4, 5])
        keep, cu, tables, lens, new = i32([1, 18, 30]), i32([0, 3]), i32([[2, 3]]), i32([31]), i32([[6]])
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            pool.copy_pages(src, dst)
            pool.compact_pages(keep, cu, tables, lens, new)
        dst.copy_(i32([8, 9]))
        keep.copy_(i32([0, 16, 29]))
        g.replay()
        assert pool.check_device_status() == 0
        for x, y in zip(views, was):
            y[8], y[9] = y[0].clone(), y[1].clone()
            y[6, :, 0], y[6, :, 1], y[6, :, 2] = y[2, :, 0], y[3, :, 0], y[3, :, 13]
            assert torch.equal(x, y)
    finally:
        pool.close()


@pytest.mark.parametrize("n", [1, 3, 600])
def test_fork_batch_copies_the_tail_once_for_every_layer(n):
    L, H, D = 3, 2, 64
    pool = pkv.Pool(L, n + 8, H, D, 16, "bf16", 64)
    try:
        req = pool.request()
        k = torch.randn(37, H, D, device="cuda").bfloat16()
        req.begin_chunk(37)
        for l in range(L):
            req.prefill_chunk(l, torch.randn(37, H, D, device="cuda").bfloat16(), k + l, k - l)
        req.commit_token()
        kids = req.fork_batch(n)
        table = req.page_table()
        for l in range(L):
            kp, vp = pool.kv_pages(l)
            for c in kids[:5] + kids[-5:]:
                t = c.page_table()
                assert t[:2] == table[:2] and t[2] != table[2] and c.length == 37
                assert torch.equal(kp[t[2]], kp[table[2]]) and torch.equal(vp[t[2]], vp[table[2]])
        assert pool.page_refs(table[0]) == n + 1 and pool.page_refs(table[2]) == 1
        assert pool.check_device_status() == 0
    finally:
        pool.close()


def grown(pool, n, seed=0):
    """A request of n committed positions, every layer filled by a chunk."""
    g = torch.Generator("cuda").manual_seed(seed)
    req = pool.request()
    req.begin_chunk(n)
    for l in range(pool.layers):
        x = lambda h: torch.randn(n, h, pool.head_dim, generator=g, device="cuda").to(pool.torch_dtype)  # noqa: E731
        req.prefill_chunk(l, x(pool.query_heads), x(pool.heads), x(pool.heads))
    req.commit_token()
    return req


def rows(pool, req):
    """Every layer's K and V rows of a request, in order."""
    t = torch.tensor(req.page_table(), device="cuda")
    return [x[t].transpose(1, 2).flatten(0, 1)[:req.length].clone() for l in range(pool.layers)
            for x in pool.kv_pages(l)]


def test_request_compact_and_truncate_bookkeeping():
    pool = pkv.Pool(2, 20, 2, 64, 16, "bf16", 128, seed=4)
    try:
        req = grown(pool, 70)
        kid = req.fork()
        was, table, free = rows(pool, req), req.page_table(), pool.free_list()
        keep = torch.arange(1, 70, 3, dtype=torch.int32, device="cuda")
        before = req.counters()
        req.compact(keep)
        assert req.length == 23 and req.counters() == before
        assert req.page_table() == free[:2]
        assert [pool.page_refs(p) for p in table] == [1] * 5           # the child's now
        for x, y in zip(rows(pool, req), was):
            assert torch.equal(x, y[keep.long()])
        for x, y in zip(rows(pool, kid), was):
            assert torch.equal(x, y)
        kid.truncate(33)
        assert kid.page_table() == table[:3] and pool.free_list() == free[2:] + table[3:]
        req.compact(torch.arange(23, dtype=torch.int32, device="cuda"))     # all of them: moved as they are
        for x, y in zip(rows(pool, req), was):
            assert torch.equal(x, y[keep.long()])
        with pytest.raises(pkv.PkvError):
            req.truncate(24)
        req.compact(torch.empty(0, dtype=torch.int32, device="cuda"))
        assert req.length == 0 and req.page_table() == []
        req.begin_token()
        req.abort_token()
        assert pool.check_device_status() == 0
    finally:
        pool.close()


def test_compact_position_outside_the_length_is_reported():
    pool = pkv.Pool(1, 8, 2, 64, 16, "f32", 64)
    try:
        req = grown(pool, 20)
        req.compact(torch.tensor([0, 20], dtype=torch.int32, device="cuda"))
        assert pool.device_status_bits() == pkv.PKV_DEVERR_SEQ_LEN and req.length == 2
    finally:
        pool.close()


def test_calls_that_cannot_lease_change_nothing():
    pool = pkv.Pool(1, 6, 2, 64, 16, "bf16", 64)
    try:
        req = grown(pool, 40)
        table, free = req.page_table(), pool.free_list()
        keep = torch.arange(33, dtype=torch.int32, device="cuda")

        def refused(call):
            with pytest.raises(pkv.PkvError) as e:
                call()
            assert e.value.status == pkv.PKV_ERR_OUT_OF_PAGES
            assert req.page_table() == table and pool.free_list() == free and req.length == 40
            assert [pool.page_refs(p) for p in table] == [1] * 3

        refused(lambda: req.fork_batch(4))              # 3 free
        for n in (1, 3):
            pool.inject_fault(pkv.PKV_INJECT_LEASE, n)
            refused(lambda: req.fork_batch(3))
            pool.inject_fault(pkv.PKV_INJECT_LEASE, n)
            refused(lambda: req.compact(keep))
        req.lease_pages(1)
        table, free = req.page_table(), pool.free_list()
        with pytest.raises(pkv.PkvError):
            req.compact(keep)
        assert req.page_table() == table and pool.free_list() == free
        kids = req.fork_batch(2)
        assert all(k.page_table()[:2] == table[:2] and len(k.page_table()) == 3 for k in kids)
    finally:
        pool.close()
