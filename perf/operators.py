"""Timed cases of the differential-attention and page operators, with a plain form of each.

Operators (see include/pkv.h):
  decode   paged_differential_decode: one new token per request attends, through two softmax
           maps per output head, over the request's pages;
  prefill  paged_differential_prefill: a chunk of new tokens per request, causally;
  copy     copy_pages: whole pages, K and V of every layer (forking a prompt's tail page);
  compact  compact_pages: the kept token rows of each request, packed into new pages.

``own`` false: the plain form, elementary torch operations in 32 bits.  ``own`` true: the
library's calls.
"""
from __future__ import annotations

import json
import math
import zlib

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-5


# ---------------------------------------------------------------- cases --

def listed():
    return [
        # decode ---------------------------------------------------------------------------
        # one chat request of a 12-head fp32 model early in its answer: latency is what counts
        dict(name="token_f32_t128", op="decode", dtype="f32", B=1, pad=0, H=12, G=1, D=64, P=16,
             tmin=128, tmax=128, window=0),
        # a serving batch of 64 requests of every age, 32 KV heads, two of the 64 slots empty
        dict(name="decode_bf16_h32", op="decode", dtype="bf16", B=64, pad=2, H=32, G=1, D=128, P=16,
             tmin=1, tmax=4096, window=0),
        # the same batch on a grouped-query model: 4 query pairs per KV pair
        dict(name="decode_bf16_gqa4", op="decode", dtype="bf16", B=64, pad=0, H=8, G=4, D=128, P=16,
             tmin=1, tmax=8192, window=0),
        # long documents: the cache read is everything
        dict(name="decode_bf16_long", op="decode", dtype="bf16", B=16, pad=0, H=8, G=1, D=128, P=16,
             tmin=131072, tmax=131072, window=0),
        # sliding-window fp32 model of narrow heads, grouped queries, odd lengths
        dict(name="decode_f32_window", op="decode", dtype="f32", B=33, pad=1, H=8, G=2, D=64, P=32,
             tmin=1, tmax=7001, window=1000),
        # prefill --------------------------------------------------------------------------
        # chunked prefill of four prompts behind cached prefixes, grouped-query model
        dict(name="chunk_bf16_d128", op="prefill", dtype="bf16", B=4, H=8, G=2, D=128, P=16,
             nmin=2048, nmax=2048, cmin=0, cmax=2048, window=0),
        # two long prompts taken at once on a model of narrow heads
        dict(name="chunk_bf16_d64", op="prefill", dtype="bf16", B=2, H=8, G=4, D=64, P=16,
             nmin=3500, nmax=4096, cmin=0, cmax=1000, window=0),
        # short ragged chunks of an fp32 model (speculative drafts being verified)
        dict(name="chunk_f32_ragged", op="prefill", dtype="f32", B=6, H=8, G=1, D=128, P=16,
             nmin=0, nmax=120, cmin=1, cmax=1500, window=0),
        # copy -----------------------------------------------------------------------------
        # eight samples forked from one prompt: its tail page, in every layer
        dict(name="copy_fork_tail", op="copy", dtype="f32", L=12, H=12, D=64, P=16, pages=96, n=8,
             src=1),
        # moving whole requests' pages: a gigabyte
        dict(name="copy_bf16_many", op="copy", dtype="bf16", L=2, H=32, D=128, P=16, pages=6144,
             n=2048, src=2048),
        # compact --------------------------------------------------------------------------
        # one request of a small model keeps a quarter of its tokens
        dict(name="compact_f32_one", op="compact", dtype="f32", L=12, H=12, D=64, P=16, B=1,
             tmin=512, tmax=512, share=0.25, run=1),
        # heavy-hitter eviction over a batch: about half of each request's tokens stay
        dict(name="compact_bf16_batch", op="compact", dtype="bf16", L=2, H=8, D=128, P=16, B=64,
             tmin=100, tmax=8192, share=0.5, run=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prefill", "prefill", "copy", "compact"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    D, P = rng.choice([64, 128]), rng.choice([16, 16, 32, 64])
    H = rng.choice([2, 4, 8, 12, 16, 32])
    if op == "decode":
        G = rng.choice([1, 1, 2, 4, 8])
        B = _log(rng, 1, 96)
        tmax = _log(rng, 16, min(32768, 400_000_000 // (B * H * D)))
        return dict(op=op, dtype=dtype, B=B, pad=rng.choice([0, 0, min(1, B - 1)]), H=H, G=G, D=D, P=P,
                    tmin=rng.choice([1, max(1, tmax // 2)]), tmax=tmax,
                    window=rng.choice([0, 0, 0, _log(rng, 5, 4096)]))
    if op == "prefill":
        H = rng.choice([2, 4, 8])
        G = rng.choice([1, 2, 4])
        B = _log(rng, 1, 12)
        most = 2048 if dtype == "bf16" else 256
        nmax = _log(rng, 1, most // B + 8)
        cmax = _log(rng, 1, 2048)
        return dict(op=op, dtype=dtype, B=B, H=H, G=G, D=D, P=P, nmin=rng.choice([0, nmax]), nmax=nmax,
                    cmin=0, cmax=cmax, window=rng.choice([0, 0, _log(rng, 5, 2048)]))
    L = rng.choice([1, 2, 5, 12])
    if op == "copy":
        n = _log(rng, 1, min(1500, 400_000_000 // (L * H * D * P * 4)))
        return dict(op=op, dtype=dtype, L=L, H=H, D=D, P=P, pages=3 * n + 5, n=n,
                    src=rng.choice([1, n, max(1, n // 3)]))
    B = _log(rng, 1, 48)
    tmax = _log(rng, 16, min(8192, 400_000_000 // (L * H * D * 4 * B)))
    return dict(op=op, dtype=dtype, L=L, H=H, D=D, P=P, B=B, tmin=rng.choice([1, tmax]), tmax=tmax,
                share=rng.choice([0.1, 0.5, 0.9]), run=rng.choice([1, 4, 32]))


# --------------------------------------------------------------- inputs --

class _Held:
    """A pool that goes with the last of its state and of the page views that are outputs."""

    def __init__(self, pool):
        self.pool = pool

    def __del__(self):
        self.pool.close()


def _lens(rng, lo, hi, n):
    return rng.integers(lo, hi + 1, size=n).astype(np.int64) if hi > lo else np.full(n, lo, np.int64)


def _sizes(c):
    """The case's lengths: the case alone says them, so that other inputs have the same shapes."""
    said = json.dumps({k: v for k, v in c.items() if k != "name"}, sort_keys=True)
    rng = np.random.default_rng(zlib.crc32(said.encode()))
    z = {}
    if c["op"] == "decode":
        z["t"] = _lens(rng, c["tmin"], c["tmax"], c["B"])
        z["t"][0] = c["tmax"]                 # the longest length takes part
        z["t"][c["B"] - c["pad"]:] = 0        # empty slots of the batch
    elif c["op"] == "prefill":
        z["n"] = _lens(rng, c["nmin"], c["nmax"], c["B"])
        z["n"][0] = c["nmax"]
        z["t"] = z["n"] + _lens(rng, c["cmin"], c["cmax"], c["B"])
    elif c["op"] == "compact":
        z["t"] = _lens(rng, c["tmin"], c["tmax"], c["B"])
        z["t"][0] = c["tmax"]
        z["keep"] = []
        for tb in z["t"]:                     # runs of `run` tokens, each kept with the share
            runs = rng.random(-(-int(tb) // c["run"])) < c["share"]
            z["keep"].append(np.flatnonzero(np.repeat(runs, c["run"])[:int(tb)]))
    return z


def _tables(rng, need, pages):
    """[B, max] page ids, -1 behind each request's last page; the pages in a shuffled order."""
    perm = rng.permutation(pages)
    t = np.full((len(need), max(1, int(need.max()))), -1, np.int32)
    at = 0
    for b, k in enumerate(need):
        t[b, :k] = perm[at:at + k]
        at += int(k)
    return t, perm[at:]


def _inputs(c, seed):
    """Everything before the call, in plain tensors on the GPU."""
    rng = np.random.default_rng([seed, 77])
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DT[c["dtype"]]

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)

    def dev(a):
        return torch.from_numpy(np.ascontiguousarray(a)).cuda()

    s = {"case": c}
    P, D, H = c["P"], c["D"], c["H"]
    if c["op"] in ("decode", "prefill"):
        B, HQ = c["B"], c["H"] * c["G"]
        z = _sizes(c)
        t = z["t"]
        if c["op"] == "decode":
            s["rows"] = B - c["pad"]
        else:
            s["n"] = n = z["n"]
            s["cu"] = dev(np.concatenate([[0], np.cumsum(n)]).astype(np.int32))
            s["rows"] = int(n.sum())
        need = -(-t // P)
        pages = int(need.sum()) + 3
        tables, _ = _tables(rng, need, pages)
        s.update(lens=dev(t.astype(np.int32)), t=t, tables=dev(tables), pages=pages,
                 max_len=int(t.max()))
        rows = B if c["op"] == "decode" else s["rows"]
        s["k"] = [normal(pages, H, P, D, dtype=dt)]
        s["v"] = [normal(pages, H, P, D, dtype=dt)]
        s["q"] = normal(rows, HQ, D, dtype=torch.float32 if c["op"] == "decode" else dt)
        s["k_new"] = normal(rows, H, D, dtype=dt)
        s["v_new"] = normal(rows, H, D, dtype=dt)
        s["lam"] = 0.2 + 0.6 * torch.rand(HQ // 2, generator=g, device="cuda")
        s["weight"] = 1.0 + 0.1 * normal(2 * D)
        s["scale"] = 0.8
    else:
        L = c["L"]
        if c["op"] == "copy":
            pages = c["pages"]
            perm = rng.permutation(pages)
            src = rng.choice(perm[c["n"]:c["n"] + c["src"]], size=c["n"], replace=c["src"] < c["n"])
            s["src"], s["dst"] = dev(src.astype(np.int32)), dev(perm[:c["n"]].astype(np.int32))
        else:
            z = _sizes(c)
            t, keep = z["t"], z["keep"]
            m = np.array([len(k) for k in keep], np.int64)
            need, out = -(-t // P), -(-m // P)
            pages = int(need.sum() + out.sum()) + 2
            tables, rest = _tables(rng, need, pages)
            dst = np.full((c["B"], max(1, int(out.max()))), -1, np.int32)
            at = 0
            for b, k in enumerate(out):
                dst[b, :k] = rest[at:at + k]
                at += int(k)
            s["keep"] = dev(np.concatenate(keep).astype(np.int32))
            s["cu"] = dev(np.concatenate([[0], np.cumsum(m)]).astype(np.int32))
            s["kept"] = int(m.sum())
            s["tables"], s["new_tables"] = dev(tables), dev(dst)
            s["lens"] = dev(t.astype(np.int32))
        s["pages"] = pages
        s["k"] = [normal(pages, H, P, D, dtype=dt) for _ in range(L)]
        s["v"] = [normal(pages, H, P, D, dtype=dt) for _ in range(L)]
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import paged_kv_cache_decode_gb300 as pkv
        c = case
        attn = c["op"] in ("decode", "prefill")
        pool = pkv.Pool(c.get("L", 1), s["pages"], c["H"], c["D"], c["P"], c["dtype"],
                        max_context=max(c["P"], s.get("max_len", c["P"])),
                        query_heads=c["H"] * c.get("G", 1), window=c.get("window", 0),
                        differential=attn)
        held, s["pool"] = _Held(pool), pool
        for i in range(c.get("L", 1)):
            k, v = pool.kv_pages(i)
            k.copy_(s["k"][i])
            v.copy_(s["v"][i])
            k.held = v.held = held            # views of the pool's memory
            s["k"][i], s["v"][i] = k, v
        if attn:
            s["diff"] = pkv.Differential(s["lam"], norm_weight=s["weight"], norm_eps=EPS,
                                         out_scale=s["scale"])
    return s


# ------------------------------------------------------------ plain form --

def _rows_of(pages, tables):
    """Each request's rows in logical order, 32 bits: [B, H, T, D]."""
    x = pages[tables.clamp(min=0).long()]                    # [B, N, H, P, D]
    B, N, H, P, D = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(B, H, N * P, D).float()


def _maps(q, k, v, mask, lam, weight, scale):
    """q [B, Hp, 2, R, D], k [B, Hp, 2, T, D], v [B, Hp, T, 2D], mask [B, 1, 1, R, T],
    lam [Hp, R, 1] (or broadcast) -> normalised difference [B, Hp, R, 2D]."""
    s = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(q.shape[-1])
    s.masked_fill_(~mask, -math.inf)
    m = s.amax(-1, keepdim=True)
    s = torch.exp_(s.sub_(torch.where(m == -math.inf, 0.0, m)))
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s, v.unsqueeze(2)) / torch.where(total == 0, 1.0, total)
    d = o[:, :, 0] - lam * o[:, :, 1]
    return scale * weight * d / torch.sqrt((d * d).mean(-1, keepdim=True) + EPS)


def _plain_decode(s):
    c = s["case"]
    B, H, G, D, P, real = c["B"], c["H"], c["G"], c["D"], c["P"], s["rows"]
    kp, vp, tables, lens = s["k"][0], s["v"][0], s["tables"], s["lens"].long()
    last = lens[:real] - 1
    page = tables[:real].gather(1, (last // P)[:, None])[:, 0].long()
    kp[page, :, last % P] = s["k_new"][:real]
    vp[page, :, last % P] = s["v_new"][:real]
    k, v = _rows_of(kp, tables), _rows_of(vp, tables)
    T = k.shape[2]
    at = torch.arange(T, device="cuda")
    mask = at < lens[:, None]
    if c["window"]:
        mask &= at >= lens[:, None] - c["window"]
    # rows behind a request's last are whatever the page holds: their weight is nothing
    v.masked_fill_(~mask[:, None, :, None], 0.0)
    q = s["q"].view(B, H // 2, G, 2, D).transpose(2, 3)
    v2 = v.view(B, H // 2, 2, T, D).transpose(2, 3).reshape(B, H // 2, T, 2 * D)
    out = _maps(q, k.view(B, H // 2, 2, T, D), v2, mask[:, None, None, None], s["lam"].view(H // 2, G, 1),
                s["weight"], s["scale"])
    return {"out": out.reshape(B, H * G // 2, 2 * D), "k": kp, "v": vp}


def _plain_prefill(s):
    c = s["case"]
    B, H, G, D, P = c["B"], c["H"], c["G"], c["D"], c["P"]
    N, most = s["rows"], int(s["n"].max())
    kp, vp, tables, lens, cu = s["k"][0], s["v"][0], s["tables"], s["lens"].long(), s["cu"].long()
    n = cu[1:] - cu[:-1]
    b = torch.repeat_interleave(torch.arange(B, device="cuda"), n, output_size=N)
    i = torch.arange(N, device="cuda") - cu[b]               # place in the chunk
    pos = lens[b] - n[b] + i
    page = tables[b, pos // P].long()
    kp[page, :, pos % P] = s["k_new"]
    vp[page, :, pos % P] = s["v_new"]
    k, v = _rows_of(kp, tables), _rows_of(vp, tables)
    T = k.shape[2]
    at = torch.arange(T, device="cuda")
    qpos = (lens - n)[:, None] + torch.arange(most, device="cuda")      # [B, most]
    mask = at <= qpos[:, :, None]
    if c["window"]:
        mask &= at > qpos[:, :, None] - c["window"]
    v.masked_fill_((at >= lens[:, None])[:, None, :, None], 0.0)
    q = torch.zeros(B, most, H * G, D, device="cuda")
    q[b, i] = s["q"].float()
    # rows of a KV pair: chunk token by chunk token, its G query pairs in order
    q = q.view(B, most, H // 2, G, 2, D).permute(0, 2, 4, 1, 3, 5).reshape(B, H // 2, 2, most * G, D)
    v2 = v.view(B, H // 2, 2, T, D).transpose(2, 3).reshape(B, H // 2, T, 2 * D)
    rows = mask.repeat_interleave(G, 1)[:, None, None]
    lam = s["lam"].view(H // 2, 1, G).expand(-1, most, -1).reshape(H // 2, most * G, 1)
    out = _maps(q, k.view(B, H // 2, 2, T, D), v2, rows, lam, s["weight"], s["scale"])
    out = out.view(B, H // 2, most, G, 2 * D).transpose(1, 2).reshape(B, most, H * G // 2, 2 * D)
    return {"out": out[b, i], "k": kp, "v": vp}


def _plain_copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    for x in s["k"] + s["v"]:                # one pair of indexed operations a layer
        x[dst] = x[src]
    return {"k": s["k"], "v": s["v"]}


def _plain_compact(s):
    c = s["case"]
    P, N = c["P"], s["kept"]
    cu, keep = s["cu"].long(), s["keep"].long()
    b = torch.repeat_interleave(torch.arange(c["B"], device="cuda"), cu[1:] - cu[:-1], output_size=N)
    to = torch.arange(N, device="cuda") - cu[b]
    src, dst = s["tables"][b, keep // P].long(), s["new_tables"][b, to // P].long()
    for x in s["k"] + s["v"]:
        x[dst, :, to % P] = x[src, :, keep % P]
    return {"k": s["k"], "v": s["v"]}


def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        pool = s["pool"]
        if op == "decode":
            out = pool.paged_differential_decode(0, s["q"], s["k_new"], s["v_new"], s["tables"], s["lens"],
                                                 s["max_len"], s["diff"])
            return {"out": out, "k": s["k"][0], "v": s["v"][0]}
        if op == "prefill":
            out = pool.paged_differential_prefill(0, s["q"], s["k_new"], s["v_new"], s["cu"], s["tables"],
                                                  s["lens"], s["diff"])
            return {"out": out, "k": s["k"][0], "v": s["v"][0]}
        if op == "copy":
            pool.copy_pages(s["src"], s["dst"])
        else:
            pool.compact_pages(s["keep"], s["cu"], s["tables"], s["lens"], s["new_tables"])
        return {"k": s["k"], "v": s["v"]}
    if op == "decode":
        return _plain_decode(s)
    if op == "prefill":
        return _plain_prefill(s)
    return _plain_copy(s) if op == "copy" else _plain_compact(s)


# ----------------------------------------------------------------- work --

def work(case):
    c = case
    es = 4 if c["dtype"] == "f32" else 2
    H, D, P = c["H"], c["D"], c["P"]
    if c["op"] == "copy":
        block = H * P * D * es * 2 * c["L"]
        return {"bytes": (min(c["src"], c["n"]) + c["n"]) * block + 8 * c["n"], "flops": 0}
    z = _sizes(c)
    if c["op"] == "compact":
        kept = sum(len(k) for k in z["keep"])
        return {"bytes": kept * (H * D * es * 2 * c["L"] * 2 + 4) + 8 * c["B"], "flops": 0}
    HQ, w = H * c["G"], c["window"] or (1 << 40)
    t = z["t"]
    if c["op"] == "decode":
        # one query attends min(t, window) keys; each is read once
        keys = pairs = int(np.minimum(t, w).sum())
        rows, new, qbytes = c["B"] - c["pad"], c["B"] - c["pad"], 4
    else:
        # the chunk's keys come in as k_new / v_new and are stored once; cached ones are read once
        n = z["n"]
        pairs = sum(int(np.minimum(np.arange(tb - nb + 1, tb + 1), w).sum()) for tb, nb in zip(t, n))
        keys = int(np.minimum(t - n, w).sum())
        rows = new = int(n.sum())
        qbytes = es
    moved = (keys + 2 * new) * H * D * es * 2 + rows * HQ * D * (qbytes + 4) + 4 * int((-(-t // P)).sum())
    if c["op"] == "decode":
        moved -= new * H * D * es * 2         # a new row counts as one of the keys already
    return {"bytes": moved, "flops": pairs * (HQ // 2) * 12 * D}


# ---------------------------------------------------------------- exact --

def exact(case, seed):
    """The definition in 64 bits, request by request and head by head."""
    s = _inputs(case, seed)
    c = case
    P = c["P"]
    K, V = s["k"], s["v"]
    if c["op"] == "copy":
        pairs = list(zip(s["src"].tolist(), s["dst"].tolist()))
        for x in K + V:
            old = x.clone()
            for a, b in pairs:
                x[b] = old[a]
        return {"k": K, "v": V}
    if c["op"] == "compact":
        cu = s["cu"].tolist()
        for b in range(c["B"]):
            kept = s["keep"][cu[b]:cu[b + 1]].long()
            if not len(kept):
                continue
            for x in K + V:
                line = x[s["tables"][b].clamp(min=0).long()].transpose(1, 2).flatten(0, 1)   # [T, H, D]
                rows = line[kept]
                for j in range(-(-len(kept) // P)):
                    part = rows[j * P:(j + 1) * P]
                    x[int(s["new_tables"][b, j]), :, :len(part)] = part.transpose(0, 1)
        return {"k": K, "v": V}
    H, G, D = c["H"], c["G"], c["D"]
    heads = H * G // 2
    decode = c["op"] == "decode"
    n = np.where(s["t"] > 0, 1, 0) if decode else s["n"]
    out = torch.zeros(s["q"].shape[0], heads, 2 * D, dtype=torch.float64, device="cuda")
    lam, w = s["lam"].double(), s["weight"].double()
    at = 0
    for b in range(c["B"]):
        t, nb = int(s["t"][b]), int(n[b])
        if nb == 0:
            continue
        pos = np.arange(t - nb, t)
        for j, x in enumerate(pos):
            page = int(s["tables"][b, x // P]) if nb == 1 else None
            if page is None:
                break
            K[0][page, :, x % P] = s["k_new"][at + j]
            V[0][page, :, x % P] = s["v_new"][at + j]
        if nb > 1:
            dest = s["tables"][b].long()[torch.from_numpy(pos // P).cuda()]
            slot = torch.from_numpy(pos % P).cuda()
            for x, new in ((K[0], s["k_new"]), (V[0], s["v_new"])):
                for h in range(H):
                    x[dest, h, slot] = new[at:at + nb, h]
        ids = s["tables"][b, :-(-t // P)].long()
        qpos = torch.arange(t - nb, t, device="cuda")[:, None]
        keys = torch.arange(t, device="cuda")[None]
        hidden = keys > qpos
        if c["window"]:
            hidden |= keys <= qpos - c["window"]
        for p in range(H // 2):
            kk = K[0][ids, 2 * p:2 * p + 2].double().transpose(0, 1).reshape(2, -1, D)[:, :t]
            vv = V[0][ids, 2 * p:2 * p + 2].double().transpose(0, 1).reshape(2, -1, D)[:, :t]
            vv = torch.cat([vv[0], vv[1]], dim=1)
            for i in range(p * G, (p + 1) * G):
                side = []
                for m in range(2):
                    logits = s["q"][at:at + nb, 2 * i + m].double() @ kk[m].T * D ** -0.5
                    logits[hidden] = -math.inf
                    side.append(torch.softmax(logits, dim=1) @ vv)
                d = side[0] - lam[i] * side[1]
                rms = torch.rsqrt(d.square().mean(1, keepdim=True) + EPS)
                out[at:at + nb, i] = s["scale"] * d * rms * w
        at += nb
    return {"out": out, "k": K, "v": V}
