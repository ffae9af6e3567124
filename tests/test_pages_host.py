"""Bookkeeping and refusals of batched forks, truncation, compaction and of differential
pools that need no device (host-only pools hold no rows, so lengths stay 0)."""
import ctypes

import pytest

import paged_kv_cache_decode_gb300 as pkv


@pytest.fixture
def pool():
    p = pkv.Pool(2, 24, 2, 4, 16, "f32", 160, seed=5, host_only=True)
    yield p
    for r in list(p._requests):
        r.close()
    assert p.free_pages == 24
    p.close()


def status(call):
    with pytest.raises(pkv.PkvError) as e:
        call()
    return e.value.status


def test_truncate_and_compact_refuse_what_does_not_fit(pool):
    r = pool.request()
    r.lease_pages(3)
    for bad in (-1, 1):
        assert status(lambda: r.truncate(bad)) == pkv.PKV_ERR_INVALID_ARGUMENT
        assert status(lambda: r.compact(bad)) == pkv.PKV_ERR_INVALID_ARGUMENT
    assert status(lambda: r.fork_batch(-1)) == pkv.PKV_ERR_INVALID_ARGUMENT
    r.begin_token()
    for call in (lambda: r.truncate(0), lambda: r.compact(0), lambda: r.fork_batch(2)):
        assert status(call) == pkv.PKV_ERR_BAD_STATE
    r.abort_token()
    assert len(r.page_table()) == 3 and pool.free_pages == 21


def test_truncate_gives_leased_pages_back_in_logical_order(pool):
    r = pool.request()
    r.lease_pages(4)
    table, free = r.page_table(), pool.free_list()
    r.truncate(0)
    assert r.page_table() == [] and pool.free_list() == free + table
    r.truncate(0)
    r.begin_token()                                 # the request goes on
    r.abort_token()


def test_compact_to_nothing_drops_every_reference(pool):
    r = pool.request()
    r.lease_pages(2)
    child = r.fork()
    table, free = r.page_table(), pool.free_list()
    r.compact(0)
    assert r.page_table() == [] and r.length == 0
    assert child.page_table() == table and [pool.page_refs(p) for p in table] == [1, 1]
    assert pool.free_list() == free
    child.compact([])
    assert pool.free_list() == free + table


def test_fork_batch_of_an_empty_request(pool):
    r = pool.request()
    r.lease_pages(2)                                # leased ahead: not shared
    kids = r.fork_batch(5)
    assert [k.page_table() for k in kids] == [[]] * 5 and pool.free_pages == 22
    assert r.fork_batch(0) == []
    kids[3].lease_pages(1)
    assert pool.free_pages == 21


def test_null_arguments():
    lib = pkv.lib
    assert lib.pkv_request_truncate(None, 0) == pkv.PKV_ERR_INVALID_ARGUMENT
    assert lib.pkv_request_compact(None, 0, None, None) == pkv.PKV_ERR_INVALID_ARGUMENT
    assert lib.pkv_request_fork_batch(None, 0, None, None) == pkv.PKV_ERR_INVALID_ARGUMENT
    assert lib.pkv_copy_pages(None, 0, None, None, None) == pkv.PKV_ERR_INVALID_ARGUMENT
    assert lib.pkv_compact_pages(None, 0, 0, None, None, None, 1, None, None, 1,
                                 None) == pkv.PKV_ERR_INVALID_ARGUMENT
    assert lib.pkv_differential_workspace_size(None, 1, 1, None) == pkv.PKV_ERR_INVALID_ARGUMENT


def test_device_calls_on_a_host_only_pool():
    plain = pkv.Pool(1, 4, 2, 64, 16, "bf16", 64, host_only=True)
    pool = pkv.Pool(1, 4, 2, 64, 16, "bf16", 64, host_only=True, differential=True)
    lib, n = pkv.lib, ctypes.c_size_t()
    try:
        assert lib.pkv_copy_pages(pool.handle, -1, None, None, None) == pkv.PKV_ERR_INVALID_ARGUMENT
        assert lib.pkv_copy_pages(pool.handle, 1, None, None, None) == pkv.PKV_ERR_INVALID_ARGUMENT
        assert lib.pkv_copy_pages(pool.handle, 0, None, None, None) == pkv.PKV_ERR_NO_STORAGE
        assert lib.pkv_compact_pages(pool.handle, -1, 0, None, None, None, 1, None, None, 1,
                                     None) == pkv.PKV_ERR_INVALID_ARGUMENT
        assert lib.pkv_compact_pages(pool.handle, 0, 0, None, None, None, 1, None, None, 1,
                                     None) == pkv.PKV_ERR_NO_STORAGE
        for p, want in ((plain, pkv.PKV_ERR_UNSUPPORTED), (pool, pkv.PKV_ERR_NO_STORAGE)):
            assert lib.pkv_differential_workspace_size(p.handle, 1, 16, ctypes.byref(n)) == want
            assert lib.pkv_differential_prefill_workspace_size(p.handle, 1, 16, ctypes.byref(n)) == want
        assert lib.pkv_differential_workspace_size(pool.handle, -1, 16,
                                                   ctypes.byref(n)) == pkv.PKV_ERR_INVALID_ARGUMENT
        one = ctypes.c_float(0.5)
        diff = pkv.pkv_differential(ctypes.addressof(one), None, 0, 0.0, 1.0)
        call = lambda p, d, out=None: lib.pkv_paged_differential_decode(  # noqa: E731
            p.handle, 0, 0, None, None, None, None, 1, None, 16, d, out, None, 0, None)
        assert call(plain, ctypes.byref(diff)) == pkv.PKV_ERR_UNSUPPORTED
        assert call(pool, None) == pkv.PKV_ERR_INVALID_ARGUMENT
        assert call(pool, ctypes.byref(diff), 8) == pkv.PKV_ERR_INVALID_ARGUMENT      # out alignment
        assert call(pool, ctypes.byref(diff)) == pkv.PKV_ERR_NO_STORAGE
        diff.normalise = 1                          # norm_eps is 0
        assert call(pool, ctypes.byref(diff)) == pkv.PKV_ERR_INVALID_ARGUMENT
        diff.normalise, diff.out_scale = 0, float("nan")
        assert call(pool, ctypes.byref(diff)) == pkv.PKV_ERR_INVALID_ARGUMENT
    finally:
        plain.close()
        pool.close()


def test_odd_heads_cannot_be_paired():
    with pytest.raises(pkv.PkvError, match="odd"):
        pkv.Pool(1, 4, 3, 64, 16, "bf16", 64, host_only=True, differential=True)


def test_injected_lease_failure_reaches_the_new_calls(pool):
    r = pool.request()
    pool.inject_fault(pkv.PKV_INJECT_LEASE, 1)
    r.truncate(0)
    r.compact(0)                                    # leases nothing: not its turn
    assert status(lambda: r.lease_pages(1)) == pkv.PKV_ERR_OUT_OF_PAGES
