"""Differential attention over paged caches against its formula in 64 bits: decode and
prefill, every storage type and head layout, ragged and empty requests, windows, the
transactions, streams and captured graphs, device-side refusals."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_decode_gb300 as pkv
from tests._differential import Case, formula

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def checked(case, what="", **kw):
    try:
        case.run(**kw)
        torch.cuda.synchronize()
        return case.check(what)
    finally:
        case.close()


LENS = [1, 2, 15, 16, 17, 31, 33, 100, 255, 256, 257, 700]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_decode_lengths(dtype, D, G):
    checked(Case(LENS, 4, G, D, dtype=dtype, seed=D + G))


@pytest.mark.parametrize("dtype,D", [("f32", 2), ("f32", 4), ("f32", 8), ("f32", 16), ("f32", 32),
                                     ("bf16", 2), ("bf16", 4), ("bf16", 8), ("bf16", 16), ("bf16", 32),
                                     ("bf16", 256)])
def test_decode_other_head_widths(dtype, D):
    checked(Case([1, 16, 40, 300], 2, 1, D, dtype=dtype, seed=D))
    checked(Case([40, 9], 2, 1, D, dtype=dtype, seed=D, new=[20, 9]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("G", [16, 128])
def test_decode_many_query_heads(dtype, G):
    checked(Case([1, 50, 333], 2, G, 64, dtype=dtype, seed=G))


@pytest.mark.parametrize("dtype,G", [("f32", 1), ("bf16", 1), ("bf16", 4)])
@pytest.mark.parametrize("P", [16, 48, 256])
def test_decode_page_sizes(dtype, G, P):
    checked(Case([P - 1, P, P + 1, 5 * P + 3, 1], 2, G, 128, P=P, dtype=dtype, seed=P))


@pytest.mark.parametrize("dtype,G", [("f32", 2), ("bf16", 2), ("bf16", 8)])
@pytest.mark.parametrize("window", [1, 16, 37, 5000])
def test_decode_window(dtype, G, window):
    checked(Case([1, 16, 36, 37, 38, 200, 1001], 4, G, 64, dtype=dtype, window=window, seed=window))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decode_empty_slots(dtype):
    c = Case([0, 5, 0, 0, 200, 0], 4, 2, 64, dtype=dtype, seed=3)
    try:
        c.run()
        assert c.check() >= 0
        assert (c.out[[0, 2, 3, 5]] == 0).all()
    finally:
        c.close()
    c = Case([0, 0], 2, 1, 128, dtype=dtype, seed=3)
    try:
        c.run()
        c.check()
        assert (c.out == 0).all()
    finally:
        c.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decode_one_long_request_split_over_the_gpu(dtype):
    checked(Case([40001], 2, 1, 128, dtype=dtype, seed=5))
    checked(Case([33000, 3], 2, 8, 64, dtype=dtype, seed=6))


@pytest.mark.parametrize("dtype,D,G", [("f32", 64, 1), ("f32", 128, 4), ("bf16", 64, 1), ("bf16", 128, 2),
                                       ("bf16", 128, 8), ("f32", 16, 1)])
@pytest.mark.parametrize("window", [0, 50])
def test_decode_single_requests(dtype, D, G, window):
    """One request: its lanes run in the warps of one CTA up to a length, over the GPU past it."""
    for t in (0, 1, 16, 17, 100, 192, 193, 383, 384, 385, 768, 769, 3000):
        checked(Case([t], 2, G, D, dtype=dtype, seed=t, window=window), f"t={t}")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,G", [(64, 1), (64, 16), (128, 4)])
@pytest.mark.parametrize("window", [0, 33])
def test_decode_few_short_requests(dtype, D, G, window):
    """Lanes of a CTA each: ragged lengths, empty slots, several row blocks a pair."""
    checked(Case([1, 0, 16, 17, 100, 0, 184, 5], 4, G, D, dtype=dtype, seed=D + G, window=window))
    checked(Case([0, 0, 1], 2, G, D, dtype=dtype, seed=D + G, window=window))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decode_few_short_requests_with_bad_entries(dtype):
    c = Case([30, 60, 5], 2, 2, 64, dtype=dtype, seed=1)
    try:
        assert c.pool.differential_workspace_size(3, c.max_len) == 0
        for bad in (-1, c.max_len + 1):
            c.dlens[0] = bad
            c.out.fill_(math.nan)
            c.run()
            assert c.pool.device_status_bits() == pkv.PKV_DEVERR_SEQ_LEN
            assert near(c, 1)
        c.dlens[0] = 30
        c.tables[0, 1] = c.pool.pages
        c.run()
        assert c.pool.device_status_bits() == pkv.PKV_DEVERR_PAGE_ID
        assert near(c, 1)
    finally:
        c.close()


def test_decode_single_request_of_a_bad_length():
    for dtype in ("f32", "bf16"):
        c = Case([40], 2, 1, 64, dtype=dtype)
        try:
            c.dlens[0] = 41
            c.run()
            assert c.pool.device_status_bits() == pkv.PKV_DEVERR_SEQ_LEN
            c.dlens[0] = 40
            c.tables[0, 1] = -1
            c.run()
            assert c.pool.device_status_bits() == pkv.PKV_DEVERR_PAGE_ID
        finally:
            c.close()


@pytest.mark.parametrize("B", [512, 513, 1025, 2500])
def test_decode_large_batches(B):
    lens = np.random.default_rng(B).integers(0, 40, size=B)
    checked(Case(lens, 2, 1, 64, dtype="bf16", seed=B))


@pytest.mark.parametrize("dtype,D,P", [("bf16", 128, 16), ("f32", 64, 32)])
def test_pages_past_32_bit_offsets(dtype, D, P):
    """Pages behind more than 2^31 elements of a layer: read, appended to, attended."""
    first = (1 << 31) // (32 * P * D) + 5
    checked(Case([P + 3, 200, 1], 32, 1, D, P=P, dtype=dtype, seed=2, first_page=first), "decode")
    checked(Case([P + 3, 200], 32, 1, D, P=P, dtype=dtype, seed=3, new=[P, 70], first_page=first), "prefill")


def test_decode_without_norm_and_without_weight():
    for dtype in ("f32", "bf16"):
        checked(Case([7, 300], 4, 2, 64, dtype=dtype, norm=False))
        checked(Case([7, 300], 4, 2, 64, dtype=dtype, weight=False))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decode_scores_far_apart(dtype):
    """Scores tens of units apart: the maximum moves late and the weights underflow."""
    checked(Case([900, 64], 2, 2, 128, dtype=dtype, amp=8.0, seed=9))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decode_infinite_rows_behind_the_length(dtype):
    """Whatever the slots behind a length, and those before the window, hold is not read into
    the result."""
    c = Case([5, 37, 130], 2, 1, 128, dtype=dtype, window=20, seed=4)
    try:
        for b, t in enumerate((5, 37, 130)):
            for pos in range(max(0, t - 20)):
                pg = int(c.tables[b, pos // 16])
                c.v[pg, :, pos % 16] = math.inf
                c.k[pg, :, pos % 16] = -math.inf
        c.run()
        assert c.pool.check_device_status() == 0
        ref, bound = c.reference()
        assert ((c.out.double() - ref).abs() <= bound).all()
    finally:
        c.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decode_same_bits_every_time(dtype):
    c = Case([5000, 1, 77, 20000], 4, 2, 128, dtype=dtype, seed=8)
    try:
        first = c.run().clone()
        for _ in range(4):
            c.out.fill_(math.nan)
            assert torch.equal(c.run(), first)
        ws = torch.full((c.pool.differential_workspace_size(c.B, c.max_len),), 255, dtype=torch.uint8,
                        device="cuda")
        assert torch.equal(c.run(workspace=ws), first)      # scratch needs no initialisation
    finally:
        c.close()


def test_decode_on_a_stream_and_two_at_once():
    a = Case([300, 2000], 4, 1, 128, dtype="bf16", seed=1)
    b = Case([1500, 9], 4, 2, 64, dtype="f32", seed=2)
    try:
        s, t = torch.cuda.Stream(), torch.cuda.Stream()
        torch.cuda.synchronize()
        for _ in range(3):
            a.run(stream=s)
            b.run(stream=t)
        torch.cuda.synchronize()
        a.check()
        b.check()
    finally:
        a.close()
        b.close()


@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_two_graphs_and_an_eager_call_share_no_scratch(kind):
    """Scratch made by the call itself: two captured graphs replayed at once on two streams,
    with an eager call beside them."""
    new = None if kind == "decode" else [30, 90]
    cases = [Case([700, 3000 + i], 4, 1, 64, dtype="f32", seed=20 + i, new=new) for i in range(3)]
    try:
        for c in cases:
            c.run()
        torch.cuda.synchronize()
        graphs = []
        for c in cases[:2]:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                c.run()
            graphs.append(g)
        streams = [torch.cuda.Stream() for _ in range(2)]
        for c in cases:
            c.out.fill_(math.nan)
        torch.cuda.synchronize()
        for _ in range(5):
            for g, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    g.replay()
            cases[2].run()
        torch.cuda.synchronize()
        for c in cases:
            c.check()
    finally:
        for c in cases:
            c.close()


@pytest.mark.parametrize("kind", ["decode", "prefill"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_captured_and_replayed(dtype, kind):
    """A graph of the call, replayed on other inputs and lengths in the same buffers."""
    new = None if kind == "decode" else [3, 60]
    c = Case([40, 700], 4, 2, 64, dtype=dtype, seed=11, new=new)
    try:
        n = (c.pool.differential_workspace_size(c.B, c.max_len) if new is None
             else c.pool.differential_prefill_workspace_size(c.B, c.rows))
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        c.run(workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(workspace=ws)
        for seed in (1, 2):
            c.q.copy_(torch.randn(c.q.shape, generator=torch.Generator("cuda").manual_seed(seed),
                                  device="cuda").to(c.q.dtype))
            c.out.fill_(math.nan)
            g.replay()
            c.check(f"replay {seed}")
    finally:
        c.close()


# -------------------------------------------------------------- prefill --

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_prefill_ragged(dtype, D, G):
    new = [1, 5, 0, 128, 33, 257]
    cached = [0, 11, 40, 0, 300, 16]
    checked(Case(np.add(new, cached), 4, G, D, dtype=dtype, new=new, seed=G))


@pytest.mark.parametrize("dtype,G", [("f32", 1), ("bf16", 1), ("bf16", 16), ("f32", 16)])
@pytest.mark.parametrize("window", [1, 20, 130])
def test_prefill_window(dtype, G, window):
    new, cached = [40, 200, 1], [0, 90, 500]
    checked(Case(np.add(new, cached), 2, G, 64, dtype=dtype, new=new, window=window, seed=window))


@pytest.mark.parametrize("dtype,D", [("f32", 128), ("bf16", 64), ("bf16", 128)])
def test_prefill_long_chunk(dtype, D):
    checked(Case([1400, 700], 2, 2, D, dtype=dtype, new=[1000, 700], seed=2))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("P", [48, 256])
def test_prefill_page_sizes(dtype, P):
    new, cached = [P, 300, 7], [0, P + 5, 2 * P]
    checked(Case(np.add(new, cached), 2, 2, 128, P=P, dtype=dtype, new=new, seed=P))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B", [255, 300, 1500])
def test_prefill_many_short_requests(dtype, B):
    rng = np.random.default_rng(B)
    new = rng.integers(0, 4, size=B)
    new[-1] = 3
    checked(Case(new + rng.integers(0, 20, size=B), 2, 1, 64, dtype=dtype, new=new, seed=B))


@pytest.mark.parametrize("D", [64, 128])
def test_prefill_maximum_that_grows_tile_by_tile(D):
    """Keys whose scores grow along the cache move the exponent base again and again, in both
    maps and at different tiles."""
    c = Case([1500], 2, 1, D, dtype="bf16", new=[300], seed=7)
    try:
        ramp = torch.linspace(0.0, 30.0, 1500, device="cuda")[:, None, None]
        sign = torch.tensor([1.0, -1.0], device="cuda")[None, :, None]
        c.K[0] = (c.K[0].float() * 0.1 + ramp * sign / D ** 0.5).bfloat16()
        c.q = (c.q.float() * 0.1 + 1.0).bfloat16()
        pos = torch.arange(1200, device="cuda")
        c.k[c.tables[0, pos // 16].long(), :, pos % 16] = c.K[0][:1200]
        c.k_new = c.K[0][1200:].contiguous()
        c.run()
        c.check()
    finally:
        c.close()


def test_prefill_reports_overlapping_rows():
    c = Case([40, 40, 40], 2, 1, 64, dtype="bf16", new=[30, 0, 30], seed=1)
    try:
        c.cu.copy_(torch.tensor([0, 30, 10, 60], dtype=torch.int32))        # not ascending
        c.run()
        assert c.pool.device_status_bits() == pkv.PKV_DEVERR_SEQ_LEN
    finally:
        c.close()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prefill_scores_far_apart_without_norm(dtype):
    checked(Case([500], 2, 1, 128, dtype=dtype, new=[400], amp=8.0, norm=False, seed=1))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prefill_rows_behind_the_last_request_stay(dtype):
    """total_new counts more rows than the requests take: the others are left as they were."""
    c = Case([30, 12], 2, 1, 64, dtype=dtype, new=[20, 12], seed=6)
    try:
        pad = 9
        grow = lambda x: torch.cat([x, torch.zeros(pad, *x.shape[1:], dtype=x.dtype, device="cuda")])  # noqa: E731
        out = torch.full((c.rows + pad, 1, 128), 7.0, device="cuda")
        c.pool.paged_differential_prefill(0, grow(c.q), grow(c.k_new), grow(c.v_new), c.cu, c.tables,
                                          c.dlens, c.diff, out=out)
        c.out.copy_(out[:c.rows])
        c.check()
        assert (out[c.rows:] == 7.0).all()
    finally:
        c.close()


# --------------------------------------------------------- transactions --

@pytest.mark.parametrize("dtype,D,G", [("f32", 64, 1), ("bf16", 128, 2), ("bf16", 64, 8), ("f32", 8, 1)])
def test_transaction_chunk_then_tokens_then_fork_and_compact(dtype, D, G):
    """A request as it is used: a chunk, tokens, a batch of forks that go on by themselves, an
    aborted token, truncation, compaction -- each step against the formula on the rows kept."""
    H, L = 2, 2
    HQ = H * G
    pool = pkv.Pool(L, 64, H, D, 16, dtype, 200, query_heads=HQ, differential=True, seed=3)
    gen = torch.Generator("cuda").manual_seed(5)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    lam = [0.3 * torch.ones(HQ // 2, device="cuda"), 0.7 * torch.ones(HQ // 2, device="cuda")]
    diff = [pkv.Differential(x, norm_eps=1e-5, out_scale=0.8) for x in lam]
    try:
        req = pool.request()
        K = [[torch.empty(0, H, D, device="cuda", dtype=dt) for _ in range(L)] for _ in range(2)]

        def step(r, K, n, commit=True):
            k = [[rnd(n, H, D).to(dt) for _ in range(L)] for _ in range(2)]
            q = [rnd(n, HQ, D) for _ in range(L)]
            r.begin_token() if n == 1 else r.begin_chunk(n)
            outs = []
            for l in range(L):
                if n == 1:
                    o = r.append_and_attend_differential(l, q[l][0], k[0][l][0], k[1][l][0], diff[l])[None]
                else:
                    q[l] = q[l].to(dt)
                    o = r.prefill_chunk_differential(l, q[l], k[0][l], k[1][l], diff[l])
                outs.append(o)
            now = [[torch.cat([K[i][l], k[i][l]]) for l in range(L)] for i in range(2)]
            for l in range(L):
                ref, bound = formula(q[l], now[0][l], now[1][l], lam[l], None, True, 0, dtype == "bf16")
                assert ((outs[l].double() - ref).abs() <= bound).all()
            if commit:
                r.commit_token()
                return now
            r.abort_token()
            return K

        K = step(req, K, 37)
        K = step(req, K, 1)
        K = step(req, K, 1, commit=False)
        kids = req.fork_batch(3)
        assert [k.length for k in kids] == [38] * 3
        assert len({k.page_table()[2] for k in kids} | {req.page_table()[2]}) == 4
        assert all(k.page_table()[:2] == req.page_table()[:2] for k in kids)
        KK = [step(k, K, 1) for k in kids]
        KK = [step(k, x, 20) for k, x in zip(kids, KK)]
        K = step(req, K, 1)
        kids[0].truncate(33)
        KK[0] = [[x[:33] for x in side] for side in KK[0]]
        KK[0] = step(kids[0], KK[0], 1)
        keep = torch.tensor([0, 3, 4, 5, 17, 30, 31, 40, 58], dtype=torch.int32, device="cuda")
        kids[1].compact(keep)
        assert kids[1].length == 9 and len(kids[1].page_table()) == 1
        KK[1] = [[x[keep.long()] for x in side] for side in KK[1]]
        KK[1] = step(kids[1], KK[1], 1)
        KK[1] = step(kids[1], KK[1], 30)
        kids[1].compact(torch.arange(1, 40, dtype=torch.int32, device="cuda"))
        KK[1] = [[x[1:40] for x in side] for side in KK[1]]
        KK[1] = step(kids[1], KK[1], 1)
        KK[2] = step(kids[2], KK[2], 1)
        K = step(req, K, 1)
        assert pool.check_device_status() == 0
    finally:
        pool.close()
    del KK


def test_plain_and_differential_layers_of_one_request():
    """A differential pool serves the plain calls too, with the same results as any pool."""
    outs = []
    for differential in (False, True):
        pool = pkv.Pool(2, 8, 2, 64, 16, "bf16", 64, query_heads=4, differential=differential)
        gen = torch.Generator("cuda").manual_seed(1)
        req = pool.request()
        for _ in range(3):
            req.begin_token()
            q = torch.randn(4, 64, generator=gen, device="cuda")
            k, v = (torch.randn(2, 64, generator=gen, device="cuda").bfloat16() for _ in range(2))
            last = req.append_and_attend(0, q, k, v).clone()
            if differential:
                req.append_and_attend_differential(1, q, k, v, pkv.Differential(torch.ones(2, device="cuda")))
            else:
                req.append_and_attend(1, q, k, v)
            req.commit_token()
        outs.append(last)
        assert pool.check_device_status() == 0
        pool.close()
    assert torch.equal(*outs)


# ------------------------------------------------------------- refusals --

def near(c, first):
    """The rows from `first` on agree with the formula (the split of the work over the GPU, and
    with it the order of the sums, depends on every length of the batch)."""
    ref, bound = c.reference()
    return bool(((c.out.double() - ref).abs() <= bound)[first:].all())


def test_device_refusals_set_the_error_word_and_nothing_else_breaks():
    c = Case([30, 100, 5], 2, 1, 64, dtype="bf16", seed=1)
    try:
        good = c.run().clone()
        lens = c.dlens.clone()
        for bad in (-1, c.max_len + 1):
            c.dlens[0] = bad
            c.out.fill_(math.nan)
            c.run()
            with pytest.raises(pkv.PkvError):
                c.pool.check_device_status()
            assert near(c, 1)
        c.dlens.copy_(lens)
        keep = c.tables.clone()
        for bad in (-1, c.pool.pages):
            c.tables[0, 0] = bad
            c.out.fill_(math.nan)
            c.run()
            assert c.pool.device_status_bits() == pkv.PKV_DEVERR_PAGE_ID
            assert near(c, 1)
        c.tables.copy_(keep)
        assert torch.equal(c.run(), good)
        assert c.pool.check_device_status() == 0
    finally:
        c.close()


def test_prefill_device_refusals():
    for dtype in ("f32", "bf16"):
        c = Case([30, 100], 2, 1, 64, dtype=dtype, new=[10, 20], seed=1)
        try:
            c.run()
            c.dlens[0] = 5                              # shorter than its chunk
            c.out.fill_(math.nan)
            c.run()
            assert c.pool.device_status_bits() == pkv.PKV_DEVERR_SEQ_LEN
            assert near(c, 10)
            c.dlens[0] = 30
            c.tables[0, 0] = c.pool.pages
            c.out.fill_(math.nan)
            c.run()
            assert c.pool.device_status_bits() == pkv.PKV_DEVERR_PAGE_ID
            assert near(c, 10)
        finally:
            c.close()


def test_host_refusals():
    c = Case([30, 3000], 2, 1, 64, dtype="bf16")       # long enough for scratch
    plain = pkv.Pool(1, 4, 2, 64, 16, "bf16", 64)
    try:
        args = (0, c.q, c.k_new, c.v_new, c.tables, c.dlens, c.max_len)
        with pytest.raises(pkv.PkvError, match="PKV_POOL_DIFFERENTIAL"):
            plain.paged_differential_decode(*args, c.diff, workspace=torch.empty(1, dtype=torch.uint8, device="cuda"))
        with pytest.raises(ValueError, match="lam"):
            c.pool.paged_differential_decode(*args, pkv.Differential(torch.ones(2, device="cuda")))
        with pytest.raises(ValueError, match="norm_weight"):
            c.pool.paged_differential_decode(
                *args, pkv.Differential(c.lam, norm_weight=torch.ones(64, device="cuda")))
        with pytest.raises(pkv.PkvError, match="norm_eps"):
            c.pool.paged_differential_decode(*args, pkv.Differential(c.lam, norm_eps=0.0))
        with pytest.raises(pkv.PkvError, match="out_scale"):
            c.pool.paged_differential_decode(*args, pkv.Differential(c.lam, out_scale=math.inf))
        with pytest.raises(pkv.PkvError, match="workspace"):
            c.pool.paged_differential_decode(*args, c.diff, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
        with pytest.raises(pkv.PkvError, match="layer"):
            c.pool.paged_differential_decode(1, *args[1:], c.diff)
        out = torch.empty(c.out.numel() + 1, device="cuda")[1:].view(c.out.shape)
        with pytest.raises(pkv.PkvError, match="aligned"):
            c.pool.paged_differential_decode(*args, c.diff, out=out)
        req = c.pool.request()
        with pytest.raises(pkv.PkvError, match="no token pending"):
            req.append_and_attend_differential(0, c.q[0], c.k_new[0], c.v_new[0], c.diff)
        req.close()
        assert torch.isnan(c.out).all() and c.pool.check_device_status() == 0
    finally:
        plain.close()
        c.close()
    with pytest.raises(pkv.PkvError, match="odd"):
        pkv.Pool(1, 4, 3, 64, 16, "bf16", 64, differential=True)
