// Differential attention over the paged KV cache for sm_103a: decode of one new
// token per request, and prefill of chunks through the same lanes.
//
// What is computed.  KV heads come in pairs (2p, 2p + 1) and query heads in pairs
// (2i, 2i + 1); query pair i reads KV pair p = i / G.  Per pair, with the keys K of
// head 2p (map 0) and of head 2p + 1 (map 1) and the values of both heads side by
// side, V_j = [v_2p,j | v_2p+1,j] (2 d_h wide):
//     A_m = softmax_j(q_(2i+m) . K_(2p+m),j / sqrt(d_h)),   m = 0, 1
//     d   = sum_j A_0,j V_j - lambda_i sum_j A_1,j V_j
//     out = s * w * d / sqrt(mean(d^2) + eps)       (without the norm: s * d)
// Both maps run as online softmaxes over one pass of the cache: each K row is read
// once for its map, each V row once for both maps.
//
// Work decomposition.  A lane is (request, KV pair, row block): up to R query rows
// that share every key -- the G query pairs of a token, and in a prefill those of
// several consecutive chunk tokens, each with its own causal end.  A lane's keys
// are cut into tiles of 16 positions (one page holds whole tiles); all tiles of all
// lanes are laid end to end and cut into W equal pieces, one per worker (a warp of
// a grid that fills the GPU once), so that any mix of lengths is balanced to one
// tile.  Every CTA derives the tile prefix from the lengths by itself: no plan
// kernel runs first.  A lane inside one worker's piece is finished by it.  A lane
// that crosses pieces leaves one partial (m, l, o) per row, map and worker in the
// workspace; the merge kernel, launched as the split kernel's programmatic
// dependent, joins them in worker order (no atomics: the same bits every time):
//     o = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s,   M = max_s m_s.
//
// A few short requests instead give each lane to the warps of one CTA, which join it in
// shared memory: one launch, no scratch.
//
// Three engines take the tiles: bf16 at head width 64 and 128 on mma.sync, fp32 at the
// same widths on packed fp32 FMAs, every other width on a plain CUDA-core loop.
//
// Bound: the K and V bytes of the cache, read once (each query row adds 12 d_h flops
// per key to the 8 d_h bytes (bf16) of a key's pair of K and V rows): 16 x 131072
// positions, 4 KV pairs of width 128, bf16: 1240 us, 1.02 of the copy bandwidth; 64 requests
// of up to 4096, 16 pairs: 324 us, 0.97; of up to 8192, 4 pairs x 4 query pairs: 195 us,
// 0.89 (start and merge take about 12 us of it).
//
// Precision.  Scores, maxima, sums and accumulators are fp32; exponents are taken
// in log2 units with log2(e) / sqrt(d_h) folded into q.  2e-7 to 6e-7 off the formula.
//
// Faults are not raised by trapping: bad lengths and page ids, and waits that run
// out, set bits of the pool's device error word and the work is skipped.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "pkv.h"
#include "pkv_internal.h"
#include "ptx.cuh"

namespace pkv {

namespace {

constexpr uint64_t kWaitNs = 4000000000ull;     // 4 s per bounded wait
constexpr int kPrefix = 512;                    // entries of the tile prefix in shared memory
constexpr int kRingBudget = 196608;             // stage-ring bytes of one CTA (one CTA per SM)
// What a lane costs beside its tiles, in tiles.  64 requests of up to 4096 positions, 16 KV
// pairs: 343 us at 1, 337 at 2, 331 at 4; short windows (64 tiles a lane): 37.7, 36.5, 37.0.
constexpr int kLaneCost = 3;

struct DfParams {
    const void* q;              // [token][2 * Hp * G][D], fp32 or (q_bf16) bf16
    bool q_bf16;
    const void* k_new;          // [B][2 * Hp][D] storage dtype; nullptr: rows are in the pages
    const void* v_new;
    void* k_pages;              // [pages][2 * Hp][P][D]
    void* v_pages;
    int64_t n_pages;
    const int32_t* tables;
    int max_pages;
    const int32_t* table_rows;  // table row of request x; nullptr: x
    const int32_t* seq_lens;    // nullptr: one request of length single_t
    int single_t;
    int64_t max_seq_len;
    const int32_t* tok0;        // prefill blocks: first chunk row and token count of block x
    const int32_t* ntok;        //   (nullptr: one token, row x)
    int B, Hp, G, subs, P;      // subs: row blocks per (request, pair)
    int tile;                   // positions of a tile (16, or 8)
    int64_t window;
    float qscale;               // log2(e) / sqrt(D)
    const float* lambda;        // [Hp * G]
    const float* norm_weight;   // [2 D] or nullptr
    int normalise;
    float norm_eps, out_scale;
    float* out;                 // [token][Hp * G][2 D]
    int alone;                  // > 0: a CTA for each lane, split over this many of its warps,
                                //   which join it in shared memory (no rec, no partials)
    int4* rec;                  // [W] lane that starts in worker w and ends after it:
                                //   (request, pair * subs + sub, last worker, 1), or w = 0
    float2* part_ml;            // [2 W][R][2]
    float* part_o;              // [2 W][R][2][2 D]
    int W, R;
    unsigned* err;
};

__device__ __forceinline__ int len_at(const DfParams& p, int x) {
    return p.seq_lens ? __ldg(p.seq_lens + x) : p.single_t;
}

__device__ __forceinline__ int ntok_at(const DfParams& p, int x) {
    return p.ntok ? __ldg(p.ntok + x) : 1;
}

// First position any row of request x reads at length t: the window's first position
// for its earliest token.
__device__ __forceinline__ int first_pos(const DfParams& p, int t, int nt) {
    if (p.window <= 0) return 0;
    const int64_t s = (int64_t)t - (nt - 1) - p.window;
    return s > 0 ? (int)s : 0;
}

__device__ __forceinline__ bool len_ok(const DfParams& p, int t) {
    return t >= 0 && t <= p.max_seq_len && ((int64_t)t + p.P - 1) / p.P <= p.max_pages;
}

// Tiles of one lane of request x (0: an empty slot, or a length that is refused).
__device__ __forceinline__ int tiles_at(const DfParams& p, int x) {
    const int t = len_at(p, x);
    if (t <= 0 || !len_ok(p, t)) return 0;
    return (t + p.tile - 1) / p.tile - first_pos(p, t, ntok_at(p, x)) / p.tile;
}

// The same in units of work: a lane is charged kLaneCost units, before its tiles, for what
// its start and end take (queries, epilogue), so that a worker with many short lanes
// gets fewer tiles.
__device__ __forceinline__ int units_at(const DfParams& p, int x) {
    const int n = tiles_at(p, x);
    return n > 0 ? n + kLaneCost : 0;
}

// Unit prefix over requests, every `stride` of them, in shared memory; all threads of
// the CTA.  pre[e] = units of one lane of the requests below e * stride; returns the total.
struct Prefix {
    int64_t pre[kPrefix + 1];
    int64_t warp_sum[32];
};

__device__ int64_t build_prefix(const DfParams& p, Prefix& s, int& stride, int& entries) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x;
    if (p.B == 1) {                             // nothing to scan
        if (tid == 0 && blockIdx.x == 0 && !len_ok(p, len_at(p, 0))) atomicOr(p.err, PKV_DEVERR_SEQ_LEN);
        stride = entries = 1;
        return units_at(p, 0);
    }
    const int nw = nt >> 5;
    stride = (p.B + kPrefix - 1) / kPrefix;
    entries = (p.B + stride - 1) / stride;
    // units of every entry: a thread for each request, or (stride > 1) a warp for each entry
    for (int e = stride == 1 ? tid : warp; e < entries; e += stride == 1 ? nt : nw) {
        int64_t n = 0;
        const int x1 = min((e + 1) * stride, p.B);
        for (int x = e * stride + (stride == 1 ? 0 : lane); x < x1; x += 32) {
            n += units_at(p, x);
            if (blockIdx.x == 0 && !len_ok(p, len_at(p, x))) atomicOr(p.err, PKV_DEVERR_SEQ_LEN);
        }
        if (stride > 1) {
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
        }
        s.pre[e] = n;
    }
    __syncthreads();
    // exclusive prefix: a thread a run of entries
    const int per = (entries + nt - 1) / nt;
    const int e0 = min(tid * per, entries), e1 = min(e0 + per, entries);
    int64_t n = 0;
    for (int e = e0; e < e1; ++e) n += s.pre[e];
    int64_t incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) s.warp_sum[warp] = incl;
    __syncthreads();
    int64_t at = incl - n, total = 0;
    for (int w = 0; w < nw; ++w) {
        if (w < warp) at += s.warp_sum[w];
        total += s.warp_sum[w];
    }
    for (int e = e0; e < e1; ++e) {
        const int64_t v = s.pre[e];
        s.pre[e] = at;
        at += v;
    }
    if (tid == 0) s.pre[entries] = total;
    __syncthreads();
    return total;
}

// A place in the flattened (request, lane, unit) sequence, always at a tile.
struct Cursor {
    int64_t f;                  // flattened unit
    int x, ln, tile;            // request, lane of it, tile of the lane
    int n, tile0;               // the request's tiles per lane, first tile
    int h, sub;                 // the lane's KV pair and row block
    int page, slot;             // the tile's page of the request, tile of that page
};

__device__ __forceinline__ void cursor_load(const DfParams& p, Cursor& c) {
    c.n = tiles_at(p, c.x);
    c.tile0 = first_pos(p, len_at(p, c.x), ntok_at(p, c.x)) / p.tile;
}

// Places within the pages for the cursor's tile.
__device__ __forceinline__ void cursor_place(const DfParams& p, Cursor& c) {
    const int gt = c.tile0 + c.tile, tpp = p.P / p.tile;
    c.page = gt / tpp;
    c.slot = gt - c.page * tpp;
}

// Cursor at the first tile at or behind flattened unit f.
__device__ Cursor cursor_at(const DfParams& p, const Prefix& s, int stride, int entries, int64_t f) {
    const int LN = p.Hp * p.subs;
    int lo = 0, hi = entries - 1;               // largest e with LN * pre[e] <= f
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (LN * s.pre[mid] <= f) lo = mid;
        else hi = mid - 1;
    }
    int64_t base = p.B == 1 ? 0 : LN * s.pre[lo];
    Cursor c;
    c.x = lo * stride;
    for (;;) {
        const int n = units_at(p, c.x);
        if (f < base + (int64_t)LN * n || c.x == p.B - 1) break;
        base += (int64_t)LN * n;
        ++c.x;
    }
    cursor_load(p, c);
    const int64_t local = f - base;
    const int per = c.n + kLaneCost;
    c.ln = local < INT32_MAX ? (int)local / per : (int)(local / per);
    c.tile = (int)(local - (int64_t)c.ln * per) - kLaneCost;
    c.f = f;
    if (c.tile < 0) {
        c.f -= c.tile;
        c.tile = 0;
    }
    c.h = c.ln / p.subs;
    c.sub = c.ln - c.h * p.subs;
    cursor_place(p, c);
    return c;
}

__device__ __forceinline__ void cursor_next(const DfParams& p, Cursor& c) {
    ++c.f;
    if (++c.tile < c.n) {
        if (++c.slot * p.tile == p.P) {
            c.slot = 0;
            ++c.page;
        }
        return;
    }
    c.tile = 0;
    c.f += kLaneCost;
    if (++c.sub == p.subs) {
        c.sub = 0;
        ++c.h;
    }
    if (++c.ln == p.Hp * p.subs) {
        c.ln = c.h = c.sub = 0;
        do {
            ++c.x;
        } while (c.x < p.B && tiles_at(p, c.x) == 0);
        if (c.x >= p.B) return;
        cursor_load(p, c);
    }
    cursor_place(p, c);
}

// Page ids of a cursor's tiles, 32 table entries at a time: lane i holds entry base + i.
struct Pager {
    int x = -1, base = 0;
    int32_t val = -1;

    __device__ __forceinline__ int32_t page(const DfParams& p, const Cursor& c) {
        const int index = c.page;
        if (c.x != x || index < base || index >= base + 32) {
            x = c.x;
            base = index;
            const int e = index + (int)(threadIdx.x & 31);
            const int64_t row = p.table_rows ? __ldg(p.table_rows + x) : x;
            val = e < p.max_pages ? __ldg(p.tables + row * p.max_pages + e) : -1;
        }
        return __shfl_sync(0xffffffffu, val, index - base);
    }
};

// One worker's share of the flattened units (every worker that works has one at least).
struct Share {
    int64_t all, begin, end;    // units of the launch, first of this worker, one past its last
    int workers;                // workers with work
};

__device__ __forceinline__ Share share_of(const DfParams& p, int64_t requests_units, int w) {
    Share s;
    s.all = (int64_t)p.Hp * p.subs * requests_units;
    s.workers = (int)(s.all < p.W ? s.all : p.W);
    s.begin = s.end = 0;
    if (w >= s.workers) return s;
    if (s.all < (1 << 20)) {                    // 32-bit divisions while w * all fits
        s.begin = (uint32_t)w * (uint32_t)s.all / (uint32_t)s.workers;
        s.end = (uint32_t)(w + 1) * (uint32_t)s.all / (uint32_t)s.workers;
    } else {
        s.begin = w * s.all / s.workers;
        s.end = (w + 1) * s.all / s.workers;
    }
    return s;
}

// The last worker of a lane that ends before flattened unit `lane_end`: the inverse of
// `begin` above.
__device__ __forceinline__ int last_worker(const Share& s, int64_t lane_end) {
    return (int)((lane_end * s.workers - 1) / s.all);
}

// Empty slots of the batch: their rows of the output are zeros.  All threads of all CTAs.
__device__ __forceinline__ void zero_empty(const DfParams& p, int D) {
    if (p.tok0) return;
    const int n = p.Hp * p.G * 2 * D;
    for (int x = blockIdx.x; x < p.B; x += gridDim.x) {
        if (tiles_at(p, x) > 0) continue;
        for (int i = threadIdx.x; i < n; i += blockDim.x) p.out[(int64_t)x * n + i] = 0.f;
    }
}

// A wait ran out: report it and let the copies in flight behind stage s land.
__device__ __forceinline__ void give_up(const DfParams& p, uint64_t* bars, int stages, int s, uint32_t parity,
                                        int ahead) {
    if ((threadIdx.x & 31) != 0) return;
    atomicOr(p.err, PKV_DEVERR_TIMEOUT);
    for (int i = 1; i < stages && i < ahead; ++i)
        mbar_wait_bounded(&bars[(s + i) % stages], parity ^ (s + i >= stages ? 1u : 0u), kWaitNs);
}

// The rows of one lane: row r is query pair `head` of one token, at output row `row`
// ([token][Hp * G]), attending positions start .. end - 1.
struct LaneRows {
    int t, nt, tok0, h, sub;
    int lo;                     // first position any row reads
};

__device__ __forceinline__ LaneRows lane_rows(const DfParams& p, int x, int h, int sub) {
    LaneRows L;
    L.t = len_at(p, x);
    L.nt = ntok_at(p, x);
    L.tok0 = p.tok0 ? __ldg(p.tok0 + x) : x;
    L.h = h;
    L.sub = sub;
    L.lo = first_pos(p, L.t, L.nt);
    return L;
}

__device__ __forceinline__ bool row_at(const DfParams& p, const LaneRows& L, int r, int64_t& row,
                                       int& head, int& start, int& end) {
    const int idx = L.sub * p.R + r;
    const bool ok = idx < L.nt * p.G;
    const int tok = ok ? idx / p.G : 0;
    head = L.h * p.G + (ok ? idx - tok * p.G : 0);
    row = (int64_t)(L.tok0 + tok) * (p.Hp * p.G) + head;
    end = ok ? L.t - (L.nt - 1 - tok) : 0;
    start = (p.window > 0 && end > p.window) ? (int)(end - p.window) : 0;
    return ok;
}

// Fetch a tensor map into the descriptor cache.
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// A CTA that has one lane (p.alone): this warp's tiles of it as share and cursor.  Returns
// the lane's tiles; 0: an empty slot (its rows are zeros) or a refused length.
__device__ __forceinline__ int alone_start(const DfParams& p, int D, int warp, Share& share, Cursor& c) {
    const int LN = p.Hp * p.subs;
    c.x = blockIdx.x / LN;
    c.ln = blockIdx.x - c.x * LN;
    c.h = c.ln / p.subs;
    c.sub = c.ln - c.h * p.subs;
    cursor_load(p, c);
    if (c.ln == 0 && threadIdx.x == 0 && !len_ok(p, len_at(p, c.x))) atomicOr(p.err, PKV_DEVERR_SEQ_LEN);
    share.all = share.workers = 0;
    share.begin = warp * c.n / p.alone;
    share.end = (warp + 1) * c.n / p.alone;
    if (c.n == 0) {
        const LaneRows L = lane_rows(p, c.x, c.h, c.sub);
        for (int r = warp; r < p.R; r += p.alone) {
            int64_t row;
            int head, st, en;
            if (!row_at(p, L, r, row, head, st, en)) continue;
            for (int i = threadIdx.x & 31; i < 2 * D; i += 32) p.out[row * 2 * D + i] = 0.f;
        }
    }
    c.tile = (int)share.begin;
    c.f = share.begin < share.end ? share.begin : share.end;
    cursor_place(p, c);
    return c.n;
}

// A warp, a few tiles ahead: fetch into L1 the queries that the lane at `c` starts with, or
// the new key and value rows that it ends with.
template <int D, int ES>
__device__ __forceinline__ void prefetch_rows(const DfParams& p, const Cursor& c) {
    const int lane = threadIdx.x & 31;
    auto fetch = [](const char* at) { asm volatile("prefetch.global.L1 [%0];" ::"l"(at)); };
    const LaneRows L = lane_rows(p, c.x, c.h, c.sub);
    if (c.tile == 0) {
        const int es = p.q_bf16 ? 2 : 4, per = (2 * D * es + 127) / 128;    // lines of one row
        for (int i = lane; i < p.R * per; i += 32) {
            int64_t row;
            int head, st, en;
            if (row_at(p, L, i / per, row, head, st, en))
                fetch(static_cast<const char*>(p.q) + row * 2 * D * es + (i % per) * 128);
        }
    }
    if (c.tile == c.n - 1) {
        // what the epilogue reads
        if (lane == 0) fetch(reinterpret_cast<const char*>(p.lambda + L.h * p.G));
        if (p.norm_weight && lane < (2 * D * 4 + 127) / 128)
            fetch(reinterpret_cast<const char*>(p.norm_weight) + lane * 128);
    }
    if (p.k_new != nullptr && c.tile == c.n - 1) {
        constexpr int per = (2 * D * ES + 127) / 128;
        const int64_t at = ((int64_t)c.x * p.Hp + L.h) * 2 * D * ES;
        for (int i = lane; i < 2 * per; i += 32)
            fetch(static_cast<const char*>(i < per ? p.k_new : p.v_new) + at + (i % per) * 128);
    }
}

// A warp's output row from the differences `d` (vector v of lane l: columns 4 (32 v + l) ..)
// and the sum of their squares.
template <int D>
__device__ __forceinline__ void store_row(const DfParams& p, int64_t row, const float4* d, float sq) {
    float c = p.out_scale;
    if (p.normalise) c *= 1.f / sqrtf(sq / (2 * D) + p.norm_eps);
#pragma unroll
    for (int v = 0; v < 2 * D / 128; ++v) {
        const int col = (v * 32 + (threadIdx.x & 31)) * 4;
        float4 nw = make_float4(1.f, 1.f, 1.f, 1.f);
        if (p.normalise && p.norm_weight) {
            nw.x = __ldg(p.norm_weight + col), nw.y = __ldg(p.norm_weight + col + 1);
            nw.z = __ldg(p.norm_weight + col + 2), nw.w = __ldg(p.norm_weight + col + 3);
        }
        *reinterpret_cast<float4*>(p.out + row * 2 * D + col) =
            make_float4(d[v].x * c * nw.x, d[v].y * c * nw.y, d[v].z * c * nw.z, d[v].w * c * nw.w);
    }
}

// A lane split over p.alone warps of one CTA: after the warps' pieces, their partials are
// joined in shared memory.  A warp's partial lies in its own part of the ring (its tiles
// are used up): (m, l) [R][2], then o [R][2][2 D].
constexpr int kPartOffset = 128;

template <int D, int R>
__device__ __forceinline__ void join_alone(const DfParams& p, unsigned char* smem, int warp_bytes, int warp,
                                           bool worked) {
    const int lane = threadIdx.x & 31;
    if (!worked && lane < 2 * R)
        reinterpret_cast<float2*>(smem + warp * warp_bytes)[lane] = make_float2(-INFINITY, 0.f);
    asm volatile("bar.sync 2, %0;" ::"r"(32 * p.alone) : "memory");
    const int LN = p.Hp * p.subs, req = blockIdx.x / LN, ln = blockIdx.x - req * LN, h = ln / p.subs;
    const LaneRows L = lane_rows(p, req, h, ln - h * p.subs);
    for (int r = warp; r < R; r += p.alone) {
        int64_t row;
        int head, st, en;
        if (!row_at(p, L, r, row, head, st, en)) continue;
        constexpr int NV = 2 * D / 128;             // vectors of 4 columns a lane
        float4 o[2][NV];
        float inv[2];
#pragma unroll
        for (int mm = 0; mm < 2; ++mm) {
            const float2 ml = lane < p.alone ? reinterpret_cast<const float2*>(smem + lane * warp_bytes)[r * 2 + mm]
                                             : make_float2(-INFINITY, 0.f);
            float mx = ml.x;
#pragma unroll
            for (int x = 16; x >= 1; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
            const float wt = ml.y > 0.f ? exp2f(ml.x - mx) : 0.f;
            float lt = wt * ml.y;
#pragma unroll
            for (int x = 16; x >= 1; x >>= 1) lt += __shfl_xor_sync(0xffffffffu, lt, x);
            inv[mm] = lt > 0.f ? 1.f / lt : 0.f;
#pragma unroll
            for (int v = 0; v < NV; ++v) o[mm][v] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int j = 0; j < p.alone; ++j) {
                const float c = __shfl_sync(0xffffffffu, wt, j);
                if (c == 0.f) continue;             // no partial, or one that weighs nothing
                const float4* x = reinterpret_cast<const float4*>(smem + j * warp_bytes + kPartOffset) +
                                  (r * 2 + mm) * (2 * D / 4) + lane;
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    const float4 y = x[v * 32];
                    o[mm][v].x = fmaf(c, y.x, o[mm][v].x), o[mm][v].y = fmaf(c, y.y, o[mm][v].y);
                    o[mm][v].z = fmaf(c, y.z, o[mm][v].z), o[mm][v].w = fmaf(c, y.w, o[mm][v].w);
                }
            }
        }
        inv[1] *= __ldg(p.lambda + head);
        float4 d[NV];
        float sq = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            d[v].x = o[0][v].x * inv[0] - o[1][v].x * inv[1], d[v].y = o[0][v].y * inv[0] - o[1][v].y * inv[1];
            d[v].z = o[0][v].z * inv[0] - o[1][v].z * inv[1], d[v].w = o[0][v].w * inv[0] - o[1][v].w * inv[1];
            sq += d[v].x * d[v].x + d[v].y * d[v].y + d[v].z * d[v].z + d[v].w * d[v].w;
        }
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, x);
        store_row<D>(p, row, d, sq);
    }
}

// ------------------------------------------------------- CUDA-core engine --

// One warp's view of a tile: 16 rows of K and V of both heads of the pair, staged
// by 1-D bulk copies as [K0 | K1 | Va | Vb], each 16 x D contiguous.  Lane l owns FPL
// features of every row: partial dot products of 16 keys x 2 maps are reduced with a
// transposed butterfly (31 shuffles per query row) that leaves lane l the score of
// key l % 16 of map l / 16; the weights go through shared memory so that every lane
// reads all 32 of a row with 8 broadcast loads, and V is read once for all rows and
// both maps.
template <typename T, int D, int R>
struct CoreGeo {
    static constexpr int ES = sizeof(T);
    static constexpr int TB = kTile * D * ES;              // one head's rows of a tile
    static constexpr int STAGE_BYTES = 4 * TB;
    static constexpr int FIT = kRingBudget / (2 * STAGE_BYTES);
    static constexpr int WARPS = FIT < 8 ? FIT : 8;
    static constexpr int STAGES_FIT = kRingBudget / (WARPS * STAGE_BYTES);
    static constexpr int STAGES = STAGES_FIT < 4 ? STAGES_FIT : 4;
    static constexpr int FPL = D >= 32 ? D / 32 : 1;       // features of one lane
    static constexpr int P_BYTES = R * 32 * 4;             // a warp's weights
    static constexpr int SMEM = WARPS * (STAGES * (STAGE_BYTES + 16) + P_BYTES);
    static_assert(WARPS >= 1 && STAGES >= 2 && SMEM <= 215 * 1024, "CTA does not fit an SM");
};

template <typename T, int N>
__device__ __forceinline__ void load_feats(const T* src, float* dst) {
    if constexpr (sizeof(T) == 4) {
        if constexpr (N == 8) {
            load_feats<T, 4>(src, dst);
            load_feats<T, 4>(src + 4, dst + 4);
        } else if constexpr (N == 4) {
            const float4 v = *reinterpret_cast<const float4*>(src);
            dst[0] = v.x, dst[1] = v.y, dst[2] = v.z, dst[3] = v.w;
        } else if constexpr (N == 2) {
            const float2 v = *reinterpret_cast<const float2*>(src);
            dst[0] = v.x, dst[1] = v.y;
        } else {
            dst[0] = *src;
        }
    } else {
        if constexpr (N == 1) {
            dst[0] = __bfloat162float(*src);
        } else {
            uint32_t w[N / 2];
            if constexpr (N == 8) {
                const uint4 v = *reinterpret_cast<const uint4*>(src);
                w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
            } else if constexpr (N == 4) {
                const uint2 v = *reinterpret_cast<const uint2*>(src);
                w[0] = v.x, w[1] = v.y;
            } else {
                w[0] = *reinterpret_cast<const uint32_t*>(src);
            }
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                dst[2 * i] = __uint_as_float(w[i] << 16);
                dst[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    }
}

template <typename T, int D, int R>
__global__ void __launch_bounds__(CoreGeo<T, D, R>::WARPS * 32, 1)
differential_core_kernel(const __grid_constant__ DfParams p) {
    using M = CoreGeo<T, D, R>;
    constexpr int F = M::FPL;
    pdl_launch_dependents();                    // the merge grid waits for this grid's end
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ Prefix prefix;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int w = warp * gridDim.x + blockIdx.x;
    constexpr int stages = M::STAGES;
    unsigned char* ring = smem + warp * stages * M::STAGE_BYTES;
    unsigned char* after = smem + M::WARPS * M::STAGES * M::STAGE_BYTES;
    float* pw = reinterpret_cast<float*>(after + warp * M::P_BYTES);
    uint64_t* bars = reinterpret_cast<uint64_t*>(after + M::WARPS * M::P_BYTES) + warp * stages;
    int32_t* stage_page = reinterpret_cast<int32_t*>(after + M::WARPS * (M::P_BYTES + M::STAGES * 8)) +
                          warp * stages;
    if (lane == 0 && w < p.W) {
        for (int s = 0; s < stages; ++s) mbar_init(&bars[s], 1);
        fence_mbar_init();
        p.rec[w] = make_int4(0, 0, 0, 0);
    }
    int stride, entries;
    const int64_t total = build_prefix(p, prefix, stride, entries);
    zero_empty(p, D);
    const Share share = share_of(p, total, w);
    if (share.begin == share.end) return;
    Cursor cur = cursor_at(p, prefix, stride, entries, share.begin);
    if (cur.f >= share.end) return;
    Cursor prod = cur;
    Pager pager;
    const uint64_t policy = l2_stream_policy();
    auto issue = [&](int s) {
        const int32_t page = pager.page(p, prod);
        if (lane == 0) {
            stage_page[s] = page;
            if (page < 0 || page >= p.n_pages) {
                atomicOr(p.err, PKV_DEVERR_PAGE_ID);
                mbar_arrive(&bars[s]);
            } else {
                const int64_t row = ((int64_t)page * 2 * p.Hp + 2 * prod.h) * p.P + prod.slot * kTile;
                const T* k = static_cast<const T*>(p.k_pages) + row * D;
                const T* v = static_cast<const T*>(p.v_pages) + row * D;
                unsigned char* dst = ring + s * M::STAGE_BYTES;
                mbar_arrive_expect_tx(&bars[s], M::STAGE_BYTES);
                bulk_copy_g2s(dst, k, M::TB, &bars[s], policy);
                bulk_copy_g2s(dst + M::TB, k + (int64_t)p.P * D, M::TB, &bars[s], policy);
                bulk_copy_g2s(dst + 2 * M::TB, v, M::TB, &bars[s], policy);
                bulk_copy_g2s(dst + 3 * M::TB, v + (int64_t)p.P * D, M::TB, &bars[s], policy);
            }
        }
        if (prod.tile == 0 || prod.tile == prod.n - 1) prefetch_rows<D, sizeof(T)>(p, prod);
        cursor_next(p, prod);
    };
    int ahead = 0;                                  // tiles staged and not yet used
    for (; ahead < stages && prod.f < share.end; ++ahead) issue(ahead);

    const bool own = lane * F < D;                  // D < 32: the lanes past D idle
    const int feat = own ? lane * F : 0;
    const int key = lane & 15, half = lane >> 4;
    float q[R][2][F], acc[R][2][2][F];
    float m[R], l[R];                               // of this half's map
    int r_start[R], r_end[R];
    LaneRows L{};
    bool has_start = false;
    int s = 0;
    uint32_t parity = 0;

    for (bool first = true; cur.f < share.end; first = false) {
        if (first || cur.tile == 0) {               // a new lane piece
            has_start = cur.tile == 0;
            L = lane_rows(p, cur.x, cur.h, cur.sub);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                int64_t row;
                int head;
                const bool ok = row_at(p, L, r, row, head, r_start[r], r_end[r]);
                // unconditional loads, so that they overlap (a row that is none reads the
                // lane's first)
#pragma unroll
                for (int mm = 0; mm < 2; ++mm) {
                    const int64_t at = (row * 2 + mm) * D + feat;
                    if (p.q_bf16) load_feats<__nv_bfloat16, F>(static_cast<const __nv_bfloat16*>(p.q) + at, q[r][mm]);
                    else load_feats<float, F>(static_cast<const float*>(p.q) + at, q[r][mm]);
#pragma unroll
                    for (int i = 0; i < F; ++i) {
                        q[r][mm][i] = ok && own ? q[r][mm][i] * p.qscale : 0.f;
                        acc[r][mm][0][i] = acc[r][mm][1][i] = 0.f;
                    }
                }
                m[r] = -INFINITY;
                l[r] = 0.f;
            }
        }
        if (!mbar_wait_bounded(&bars[s], parity, kWaitNs)) {
            give_up(p, bars, stages, s, parity, ahead);
            return;
        }
        unsigned char* stage = ring + s * M::STAGE_BYTES;
        T* rows = reinterpret_cast<T*>(stage);      // [K0 | K1 | Va | Vb][16][D]
        const int gt = cur.tile0 + cur.tile, k0 = gt * kTile;
        const int32_t page = stage_page[s];
        if (page >= 0 && page < p.n_pages) {
            const int lo = L.lo;
            const bool edge = k0 < lo || k0 + kTile > L.t;
            if (edge) {
                // rows that no query of the lane reads may hold anything: zeros, so that
                // a weight of 0 times them is 0
                for (int i = lane; i < kTile * 2 * D; i += 32) {
                    const int row = (i / D) % kTile;
                    if (k0 + row < lo || k0 + row >= L.t) rows[2 * kTile * D + i] = T(0.f);
                }
                __syncwarp();
            }
            if (p.k_new != nullptr && L.t - 1 >= k0 && L.t - 1 < k0 + kTile) {
                // the new token's rows: into the staged tile and into the page
                const int slot = L.t - 1 - k0;
                const int64_t src = ((int64_t)cur.x * 2 * p.Hp + 2 * L.h) * D;
                const int64_t dst =
                    (((int64_t)page * 2 * p.Hp + 2 * L.h) * p.P + (L.t - 1) % p.P) * D;
                for (int i = lane; i < 2 * D; i += 32) {
                    const int hd = i / D, c = i - hd * D;
                    const T kv = static_cast<const T*>(p.k_new)[src + i];
                    const T vv = static_cast<const T*>(p.v_new)[src + i];
                    rows[(hd * kTile + slot) * D + c] = kv;
                    rows[((2 + hd) * kTile + slot) * D + c] = vv;
                    if (L.sub == 0) {
                        static_cast<T*>(p.k_pages)[dst + (int64_t)hd * p.P * D + c] = kv;
                        static_cast<T*>(p.v_pages)[dst + (int64_t)hd * p.P * D + c] = vv;
                    }
                }
                __syncwarp();
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float v[32];                        // partial scores: 16 keys of map 0, of map 1
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    float kf[F];
                    load_feats<T, F>(rows + j * D + feat, kf);
                    float x = q[r][j >> 4][0] * kf[0];
#pragma unroll
                    for (int i = 1; i < F; ++i) x = fmaf(q[r][j >> 4][i], kf[i], x);
                    v[j] = own ? x : 0.f;
                }
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) {
                    const bool up = (lane & o) != 0;
#pragma unroll
                    for (int i = 0; i < o; ++i) {
                        const float mine = up ? v[i + o] : v[i], other = up ? v[i] : v[i + o];
                        v[i] = mine + __shfl_xor_sync(0xffffffffu, other, o);
                    }
                }
                const float sc =
                    (k0 + key >= r_start[r] && k0 + key < r_end[r]) ? v[0] : -INFINITY;
                float mx = sc;
#pragma unroll
                for (int o = 8; o >= 1; o >>= 1)
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                const float m_new = fmaxf(m[r], mx);
                const float mb = m_new == -INFINITY ? 0.f : m_new;
                const float alpha = exp2f(m[r] - mb);
                const float pr = exp2f(sc - mb);
                l[r] = fmaf(l[r], alpha, pr);
                m[r] = m_new;
                pw[r * 32 + lane] = pr;
                if (__any_sync(0xffffffffu, alpha != 1.f)) {
                    const float a0 = __shfl_sync(0xffffffffu, alpha, 0);
                    const float a1 = __shfl_sync(0xffffffffu, alpha, 16);
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                        for (int i = 0; i < F; ++i) {
                            acc[r][0][hf][i] *= a0;
                            acc[r][1][hf][i] *= a1;
                        }
                }
            }
            __syncwarp();
#pragma unroll
            for (int kq = 0; kq < kTile; kq += 4) {
                float4 w0[R], w1[R];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    w0[r] = *reinterpret_cast<const float4*>(pw + r * 32 + kq);
                    w1[r] = *reinterpret_cast<const float4*>(pw + r * 32 + 16 + kq);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float va[F], vb[F];
                    load_feats<T, F>(rows + (2 * kTile + kq + j) * D + feat, va);
                    load_feats<T, F>(rows + (3 * kTile + kq + j) * D + feat, vb);
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const float x0 = (&w0[r].x)[j], x1 = (&w1[r].x)[j];
#pragma unroll
                        for (int i = 0; i < F; ++i) {
                            acc[r][0][0][i] = fmaf(x0, va[i], acc[r][0][0][i]);
                            acc[r][0][1][i] = fmaf(x0, vb[i], acc[r][0][1][i]);
                            acc[r][1][0][i] = fmaf(x1, va[i], acc[r][1][0][i]);
                            acc[r][1][1][i] = fmaf(x1, vb[i], acc[r][1][1][i]);
                        }
                    }
                }
            }
        }
        // the stage is free again: hand it to the copy engine
        fence_proxy_async_smem();
        __syncwarp();
        if (prod.f < share.end) issue(s);
        else --ahead;
        if (++s == stages) {
            s = 0;
            parity ^= 1u;
        }

        const bool has_end = cur.tile == cur.n - 1;
        if (has_end || cur.f + 1 >= share.end) {    // the piece ends
            const int slot = 2 * w + (has_start ? 1 : 0);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                int64_t row;
                int head, st, en;
                const bool ok = row_at(p, L, r, row, head, st, en);
                float lt = l[r];
#pragma unroll
                for (int o = 8; o >= 1; o >>= 1) lt += __shfl_xor_sync(0xffffffffu, lt, o);
                if (has_start && has_end) {
                    if (!ok) continue;
                    const float l0 = __shfl_sync(0xffffffffu, lt, 0);
                    const float l1 = __shfl_sync(0xffffffffu, lt, 16);
                    const float i0 = l0 > 0.f ? 1.f / l0 : 0.f;
                    const float i1 = l1 > 0.f ? __ldg(p.lambda + head) / l1 : 0.f;
                    float d[2][F], sq = 0.f;
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                        for (int i = 0; i < F; ++i) {
                            d[hf][i] = acc[r][0][hf][i] * i0 - acc[r][1][hf][i] * i1;
                            if (own) sq = fmaf(d[hf][i], d[hf][i], sq);
                        }
#pragma unroll
                    for (int o = 16; o >= 1; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
                    float c = p.out_scale;
                    if (p.normalise) c *= 1.f / sqrtf(sq / (2 * D) + p.norm_eps);
                    if (own) {
                        float* op = p.out + row * 2 * D + feat;
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                            for (int i = 0; i < F; ++i) {
                                const int col = hf * D + i;
                                const float nw =
                                    p.norm_weight && p.normalise ? __ldg(p.norm_weight + feat + col) : 1.f;
                                op[col] = d[hf][i] * c * nw;
                            }
                    }
                } else {
                    const int64_t at = ((int64_t)slot * R + r) * 2;
                    if (key == 0) p.part_ml[at + half] = make_float2(m[r], lt);
                    if (own) {
#pragma unroll
                        for (int mm = 0; mm < 2; ++mm)
#pragma unroll
                            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                                for (int i = 0; i < F; ++i)
                                    p.part_o[(at + mm) * 2 * D + hf * D + feat + i] = acc[r][mm][hf][i];
                    }
                }
            }
            if (has_start && !has_end && lane == 0) {
                p.rec[w] = make_int4(cur.x, cur.ln, last_worker(share, cur.f - cur.tile + cur.n), 1);
            }
        }
        cursor_next(p, cur);
    }
}

// ----------------------------------------------------------- fp32 engine --

// fp32, head width 64 or 128, R = 1, 2 or 4 query rows a lane, CUDA cores (fp32 products
// as they are: tensor cores would take each operand in three parts).  A stage holds a
// tile of KT positions as TMA leaves it, K then V: [head][32-column chunk][KT rows][128
// bytes], 128-byte swizzle (one box of a 5-D map for both heads).
//   scores   lane (s, part): the dot products of keys s and s + KT/2 over D * KT / 64
//            features of both maps -- the swizzle spreads 8 keys' 16-byte pieces over all
//            banks, queries come from shared memory as broadcasts for both keys -- then
//            a transposed butterfly over the parts that leaves a lane one key of one map
//   weights  one exponential a lane and row (map lane / 16), through shared memory
//   values   a lane owns 4 or 8 of the 2 D columns for all rows and both maps: V is read
//            once, weights as broadcasts; packed two-lane FMAs
// KT = 8 at D = 128: the same ring holds twice the warps, and with several rows the kernel
// is bound by their instruction latency (ragged chunks in lanes of 4 tokens: 124 us, with
// KT = 16 139 us); at D = 64 both are alike (window of 1000, 2 rows: 35 us).
template <int D, int R, int KT>
struct F32Geo {
    static constexpr int CH = D / 32;                      // 128-byte chunks of a row
    static constexpr int HEAD = CH * KT * 128;             // one head's rows of a tile
    static constexpr int STAGE_BYTES = 4 * HEAD;
    static constexpr int FIT = kRingBudget / (2 * STAGE_BYTES);
    static constexpr int WARPS = FIT < 12 ? FIT : 12;
    static constexpr int STAGES = kRingBudget / (WARPS * STAGE_BYTES);
    static constexpr int KS = KT / 2;                      // a lane takes keys s and s + KS
    static constexpr int PARTS = 32 / KS;                  // lanes that share the two
    static constexpr int PIECES = D / 4 / PARTS;           // 16-byte pieces of one lane's part
    static constexpr int NV = 2 * D / 128;                 // 4-column vectors of a lane
    static constexpr int Q_BYTES = R * 2 * D * 4, P_BYTES = R * 2 * KT * 4;
    static constexpr int SMEM = 1024 + WARPS * (STAGES * (STAGE_BYTES + 12) + Q_BYTES + P_BYTES);
    static_assert(STAGES >= 2 && SMEM <= 222 * 1024, "CTA does not fit an SM");
};

__device__ __forceinline__ float2 lo2(const float4& v) { return make_float2(v.x, v.y); }
__device__ __forceinline__ float2 hi2(const float4& v) { return make_float2(v.z, v.w); }

template <int D, int R, int KT>
__global__ void __launch_bounds__(F32Geo<D, R, KT>::WARPS * 32, 1)
differential_f32_kernel(const __grid_constant__ DfParams p, const __grid_constant__ CUtensorMap tmk,
                        const __grid_constant__ CUtensorMap tmv) {
    using M = F32Geo<D, R, KT>;
    pdl_launch_dependents();                    // the merge grid waits for this grid's end
    extern __shared__ unsigned char smem_raw[];
    __shared__ Prefix prefix;
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (p.alone && warp >= p.alone) return;
    const int w = p.alone ? blockIdx.x * p.alone + warp : warp * gridDim.x + blockIdx.x;
    constexpr int stages = M::STAGES;
    unsigned char* ring = smem + warp * stages * M::STAGE_BYTES;
    unsigned char* after = smem + M::WARPS * M::STAGES * M::STAGE_BYTES;
    float* qs = reinterpret_cast<float*>(after + warp * M::Q_BYTES);            // [R][2][D], scaled
    float* pw = reinterpret_cast<float*>(after + M::WARPS * M::Q_BYTES + warp * M::P_BYTES);
    after += M::WARPS * (M::Q_BYTES + M::P_BYTES);
    uint64_t* bars = reinterpret_cast<uint64_t*>(after) + warp * stages;
    int32_t* stage_page = reinterpret_cast<int32_t*>(after + M::WARPS * M::STAGES * 8) + warp * stages;
    if (lane == 0 && w < p.W) {
        prefetch_map(&tmk);
        prefetch_map(&tmv);
        for (int s = 0; s < stages; ++s) mbar_init(&bars[s], 1);
        fence_mbar_init();
        if (!p.alone) p.rec[w] = make_int4(0, 0, 0, 0);
    }
    Share share;
    Cursor cur;
    int alone_tiles = 0;
    if (p.alone) {
        alone_tiles = alone_start(p, D, warp, share, cur);
        if (alone_tiles == 0) return;
    } else {
        int stride, entries;
        const int64_t total = build_prefix(p, prefix, stride, entries);
        zero_empty(p, D);
        share = share_of(p, total, w);
        if (share.begin == share.end) return;
        cur = cursor_at(p, prefix, stride, entries, share.begin);
    }
    const bool worked = share.begin < share.end;
    Cursor prod = cur;
    Pager pager;
    const uint64_t policy = l2_stream_policy();
    auto issue = [&](int s) {
        const int32_t page = pager.page(p, prod);
        if (lane == 0) {
            stage_page[s] = page;
            if (page < 0 || page >= p.n_pages) {
                atomicOr(p.err, PKV_DEVERR_PAGE_ID);
                mbar_arrive(&bars[s]);
            } else {
                const int slot = prod.slot * KT;
                unsigned char* dst = ring + s * M::STAGE_BYTES;
                mbar_arrive_expect_tx(&bars[s], M::STAGE_BYTES);
                tma_load_5d(dst, &tmk, 0, slot, 0, 2 * prod.h, page, &bars[s], policy);
                tma_load_5d(dst + 2 * M::HEAD, &tmv, 0, slot, 0, 2 * prod.h, page, &bars[s], policy);
            }
        }
        if (prod.tile == 0 || prod.tile == prod.n - 1) prefetch_rows<D, 4>(p, prod);
        cursor_next(p, prod);
    };
    int ahead = 0;                                  // tiles staged and not yet used
    for (; ahead < stages && prod.f < share.end; ++ahead) issue(ahead);

    // dot products of keys slot and slot + KS; then the score of key `key` of map `half`
    const int slot_k = lane % M::KS, part = lane / M::KS, half = lane >> 4, upper = (lane >> 3) & 1;
    const int key = slot_k + upper * M::KS;
    const bool writes = KT == 16 || (lane & 4) == 0;          // KT = 8: lanes l, l ^ 4 hold the same
    auto over_keys = [](float x, auto f) {
        x = f(x, __shfl_xor_sync(0xffffffffu, x, 1));
        x = f(x, __shfl_xor_sync(0xffffffffu, x, 2));
        if constexpr (KT == 16) x = f(x, __shfl_xor_sync(0xffffffffu, x, 4));
        return f(x, __shfl_xor_sync(0xffffffffu, x, 8));
    };
    // 16-byte piece u of key row `key` and head hd is at hd * HEAD + (u / 8) * KT * 128 +
    // key * 128 + ((u % 8) ^ (key % 8)) * 16
    auto piece_at = [](int hd, int u, int row) {
        return hd * M::HEAD + (u >> 3) * (KT * 128) + row * 128 + (((u & 7) ^ (row & 7)) << 4);
    };
    float2 acc[R][2][M::NV][2];                     // [row][map][vector][column pair]
    float m[R], l[R];                               // of this half's map
    int r_start[R], r_end[R];
    LaneRows L{};
    bool has_start = false;
    int s = 0;
    uint32_t parity = 0;

    for (bool first = true; cur.f < share.end; first = false) {
        if (first || cur.tile == 0) {               // a new lane piece
            has_start = cur.tile == 0;
            L = lane_rows(p, cur.x, cur.h, cur.sub);
            float4 x[R][2 * D / 128];
            bool ok[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                int64_t row;
                int head;
                ok[r] = row_at(p, L, r, row, head, r_start[r], r_end[r]);
                const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + row * 2 * D);
#pragma unroll
                for (int i = 0; i < 2 * D / 128; ++i) x[r][i] = __ldg(q + i * 32 + lane);
            }
            __syncwarp();                           // the last piece's reads of qs are done
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float c = ok[r] ? p.qscale : 0.f;
#pragma unroll
                for (int i = 0; i < 2 * D / 128; ++i)
                    reinterpret_cast<float4*>(qs + r * 2 * D)[i * 32 + lane] =
                        make_float4(x[r][i].x * c, x[r][i].y * c, x[r][i].z * c, x[r][i].w * c);
                m[r] = -INFINITY;
                l[r] = 0.f;
#pragma unroll
                for (int mm = 0; mm < 2; ++mm)
#pragma unroll
                    for (int v = 0; v < M::NV; ++v)
                        acc[r][mm][v][0] = acc[r][mm][v][1] = make_float2(0.f, 0.f);
            }
            __syncwarp();
        }
        if (!mbar_wait_bounded(&bars[s], parity, kWaitNs)) {
            give_up(p, bars, stages, s, parity, ahead);
            break;
        }
        unsigned char* stage = ring + s * M::STAGE_BYTES;
        const int k0 = (cur.tile0 + cur.tile) * KT;
        const int32_t page = stage_page[s];
        if (page >= 0 && page < p.n_pages) {
            const int lo = L.lo;
            if (k0 < lo || k0 + KT > L.t) {
                // value rows that no query of the lane reads may hold anything: zeros, so that
                // a weight of 0 times them is 0
                for (int i = lane; i < KT * 2 * M::CH * 8; i += 32) {
                    const int rw = (i >> 3) % KT;
                    if (k0 + rw < lo || k0 + rw >= L.t)
                        *reinterpret_cast<uint4*>(stage + 2 * M::HEAD + i * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                __syncwarp();
            }
            if (p.k_new != nullptr && L.t - 1 >= k0 && L.t - 1 < k0 + KT) {
                // the new token's rows: into the staged tile and into the page
                const int slot = L.t - 1 - k0;
                const int64_t src = ((int64_t)cur.x * 2 * p.Hp + 2 * L.h) * D;
                const int64_t dst = (((int64_t)page * 2 * p.Hp + 2 * L.h) * p.P + (L.t - 1) % p.P) * D;
                for (int i = lane; i < D; i += 32) {            // 2 x 2 rows of D / 4 pieces
                    const bool value = i >= D / 2;
                    const int c = value ? i - D / 2 : i, hd = c / (D / 4), u = c - hd * (D / 4);
                    const uint4 x = *reinterpret_cast<const uint4*>(
                        static_cast<const float*>(value ? p.v_new : p.k_new) + src + c * 4);
                    *reinterpret_cast<uint4*>(stage + (value ? 2 : 0) * M::HEAD + piece_at(hd, u, slot)) = x;
                    if (L.sub == 0)
                        *reinterpret_cast<uint4*>(static_cast<float*>(value ? p.v_pages : p.k_pages) + dst +
                                                  (int64_t)hd * p.P * D + u * 4) = x;
                }
                __syncwarp();
            }
            float sc[R];                            // this half's map, key `key`
            {
                float2 d[R][2][2];                  // [row][map][key]
#pragma unroll
                for (int mm = 0; mm < 2; ++mm) {
#pragma unroll
                    for (int r = 0; r < R; ++r) d[r][mm][0] = d[r][mm][1] = make_float2(0.f, 0.f);
#pragma unroll
                    for (int u = 0; u < M::PIECES; ++u) {
                        const int pu = part * M::PIECES + u;
                        float4 kv[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            kv[i] = *reinterpret_cast<const float4*>(stage + piece_at(mm, pu, slot_k + i * M::KS));
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            const float4 qv =
                                reinterpret_cast<const float4*>(qs + (r * 2 + mm) * D)[pu];
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                d[r][mm][i] = __ffma2_rn(lo2(qv), lo2(kv[i]), d[r][mm][i]);
                                d[r][mm][i] = __ffma2_rn(hi2(qv), hi2(kv[i]), d[r][mm][i]);
                            }
                        }
                    }
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    // lanes of the other half want the other map, lanes l ^ 8 the other key
                    float v[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float a = d[r][0][i].x + d[r][0][i].y, b = d[r][1][i].x + d[r][1][i].y;
                        v[i] = (half ? b : a) + __shfl_xor_sync(0xffffffffu, half ? a : b, 16);
                    }
                    float x = (upper ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, upper ? v[0] : v[1], 8);
                    if constexpr (KT == 8) x += __shfl_xor_sync(0xffffffffu, x, 4);
                    sc[r] = x;
                }
            }
            bool moved = false;
            float alpha[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (k0 + key < r_start[r] || k0 + key >= r_end[r]) sc[r] = -INFINITY;
                const float mx = over_keys(sc[r], [](float a, float b) { return fmaxf(a, b); });
                alpha[r] = 1.f;
                if (mx > m[r] + 8.f || (m[r] == -INFINITY && mx > m[r])) {
                    alpha[r] = exp2f(m[r] - mx);    // 0 for the first
                    m[r] = mx;
                    moved = true;
                }
                const float pr = exp2f(sc[r] - (m[r] == -INFINITY ? 0.f : m[r]));
                l[r] = fmaf(l[r], alpha[r], pr);
                if (writes) pw[(r * 2 + half) * KT + key] = pr;
            }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float a0 = __shfl_sync(0xffffffffu, alpha[r], 0);
                    const float a1 = __shfl_sync(0xffffffffu, alpha[r], 16);
#pragma unroll
                    for (int v = 0; v < M::NV; ++v)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            acc[r][0][v][i].x *= a0, acc[r][0][v][i].y *= a0;
                            acc[r][1][v][i].x *= a1, acc[r][1][v][i].y *= a1;
                        }
                }
            }
            __syncwarp();
#pragma unroll
            for (int kq = 0; kq < KT; kq += 4) {
                float4 wt[R][2];
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int mm = 0; mm < 2; ++mm)
                        wt[r][mm] = *reinterpret_cast<const float4*>(pw + (r * 2 + mm) * KT + kq);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float4 vv[M::NV];
#pragma unroll
                    for (int v = 0; v < M::NV; ++v) {
                        const int u = v * 32 + lane, hd = u / (D / 4);
                        vv[v] = *reinterpret_cast<const float4*>(
                            stage + 2 * M::HEAD + piece_at(hd, u - hd * (D / 4), kq + j));
                    }
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int mm = 0; mm < 2; ++mm) {
                            const float x = (&wt[r][mm].x)[j];
                            const float2 x2 = make_float2(x, x);
#pragma unroll
                            for (int v = 0; v < M::NV; ++v) {
                                acc[r][mm][v][0] = __ffma2_rn(x2, lo2(vv[v]), acc[r][mm][v][0]);
                                acc[r][mm][v][1] = __ffma2_rn(x2, hi2(vv[v]), acc[r][mm][v][1]);
                            }
                        }
                }
            }
        }
        // the stage is free again: hand it to the copy engine
        fence_proxy_async_smem();
        __syncwarp();
        if (prod.f < share.end) issue(s);
        else --ahead;
        if (++s == stages) {
            s = 0;
            parity ^= 1u;
        }

        const bool has_end = cur.tile == cur.n - 1;
        if (has_end || cur.f + 1 >= share.end) {    // the piece ends
            const int64_t slot = 2 * w + (has_start ? 1 : 0);
            float2* ml = p.alone ? reinterpret_cast<float2*>(ring) : p.part_ml + slot * R * 2;
            float* po = p.alone ? reinterpret_cast<float*>(ring + kPartOffset) : p.part_o + slot * R * 4 * D;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                int64_t row;
                int head, st, en;
                const bool ok = row_at(p, L, r, row, head, st, en);
                const float lt = over_keys(l[r], [](float a, float b) { return a + b; });
                if (has_start && has_end) {
                    if (!ok) continue;              // alike in all lanes
                    const float l0 = __shfl_sync(0xffffffffu, lt, 0);
                    const float l1 = __shfl_sync(0xffffffffu, lt, 16);
                    const float i0 = l0 > 0.f ? 1.f / l0 : 0.f;
                    const float i1 = l1 > 0.f ? __ldg(p.lambda + head) / l1 : 0.f;
                    float4 d[M::NV];
                    float sq = 0.f;
#pragma unroll
                    for (int v = 0; v < M::NV; ++v) {
                        const float2* a = acc[r][0][v];
                        const float2* b = acc[r][1][v];
                        d[v] = make_float4(a[0].x * i0 - b[0].x * i1, a[0].y * i0 - b[0].y * i1,
                                           a[1].x * i0 - b[1].x * i1, a[1].y * i0 - b[1].y * i1);
                        sq += d[v].x * d[v].x + d[v].y * d[v].y + d[v].z * d[v].z + d[v].w * d[v].w;
                    }
#pragma unroll
                    for (int o = 16; o >= 1; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
                    store_row<D>(p, row, d, sq);
                } else {
                    if (lane % 16 == 0) ml[r * 2 + half] = make_float2(m[r], lt);
#pragma unroll
                    for (int mm = 0; mm < 2; ++mm)
#pragma unroll
                        for (int v = 0; v < M::NV; ++v)
                            *reinterpret_cast<float4*>(po + (r * 2 + mm) * 2 * D + (v * 32 + lane) * 4) =
                                make_float4(acc[r][mm][v][0].x, acc[r][mm][v][0].y, acc[r][mm][v][1].x,
                                            acc[r][mm][v][1].y);
                }
            }
            if (has_start && !has_end && lane == 0 && !p.alone)
                p.rec[w] = make_int4(cur.x, cur.ln, last_worker(share, cur.f - cur.tile + cur.n), 1);
        }
        cursor_next(p, cur);
    }
    // a lane of one tile, or of one warp, is finished already
    if (p.alone > 1 && alone_tiles > 1)
        join_alone<D, R>(p, smem, M::STAGES * M::STAGE_BYTES, warp, worked);
}

// ------------------------------------------------------ tensor-core engine --

// bf16, head width 64 or 128, R = 1, 2, 4 or 8 query rows a lane.  A stage holds a tile as
// TMA leaves it, K then V: [head][64-column chunk][16 rows][128 bytes], 128-byte swizzle
// (one box of a 5-D map for both heads).  Products are m16n8k16 with the cache as the
// 16-row operand, so that few queries still fill the 8 columns:
//   S_m = K_m Q_m^T   16 keys x 8 columns of queries.  fp32 queries go in as bf16 parts
//                     (hi, mid, lo: 24 bits) on columns of their own where there is
//                     room, else as further products into the same columns
//   O += V^T P^T      16 value columns x 8 columns of (query, map, part of the weight);
//                     P^T is the scores' fragment transposed by movmatrix, weights as
//                     three bf16 parts too.  Both maps share every V fragment
// Column layouts (lane = 4 g + t holds columns 2t, 2t + 1 of row g and row g + 8):
//   R   S columns 2t, 2t+1              O columns 2t, 2t+1               MMAs a tile (D 128)
//   1   t even: hi, mid; odd: lo, 0     map t/2; t even: hi, mid; odd: lo, 0    16 + 16
//   2   query t/2, as above             query t/2, map t%2: hi, mid; + lo, 0    16 + 32
//   4   query t: hi, mid; + lo, 0       query t: map 0, map 1; parts added      32 + 48
//   8   queries 2t, 2t+1; parts added   the same, an accumulator a map          32 + 96
// (R = 8 at D = 128 takes two parts of q, 2^-18: three do not fit the registers.)
// mma.sync, not tcgen05: at most 16 columns of queries would use 16 of tcgen05's 128
// rows, and the kernel waits for memory.  Each tile's V product is added to O by
// rounding adds: the MMA's own accumulation truncates, which over a long cache adds up
// (1.3e-5 of the result at 131072 keys).  The maximum is only followed when it grows by
// more than 8 in log2 units: weights stay below 2^8.
template <int D>
struct MmaGeo {
    static constexpr int CH = D / 64;                      // 128-byte chunks of a row
    static constexpr int HEAD = CH * kTile * 128;          // one head's rows of a tile
    static constexpr int STAGE_BYTES = 4 * HEAD;
    static constexpr int WARPS = D == 64 ? 12 : 6;
    static constexpr int STAGES = kRingBudget / (WARPS * STAGE_BYTES);
    static constexpr int KS = D / 16, NB = 2 * D / 16;     // k-steps of S, 16-column blocks of O
    static constexpr int SMEM = 1024 + WARPS * STAGES * (STAGE_BYTES + 12);
    static_assert(STAGES >= 2 && SMEM <= 215 * 1024, "CTA does not fit an SM");
};

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// x as three bf16 parts: x = part[0] + part[1] + part[2] to 2^-24.
__device__ __forceinline__ void split3(float x, float (&part)[3]) {
    part[0] = __bfloat162float(__float2bfloat16_rn(x));
    const float r = x - part[0];
    part[1] = __bfloat162float(__float2bfloat16_rn(r));
    part[2] = r - part[1];
}

__device__ __forceinline__ uint32_t pack(float x, float y) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// 8 x 8 transpose: in, lane 4 g + t holds columns 2t, 2t + 1 of row g; out, rows 2t,
// 2t + 1 of column g.
__device__ __forceinline__ uint32_t transpose(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void add2(float* to, const float* x) {
    const float2 r = __fadd2_rn(make_float2(to[0], to[1]), make_float2(x[0], x[1]));
    to[0] = r.x, to[1] = r.y;
}

template <int D, int R>
__global__ void __launch_bounds__(MmaGeo<D>::WARPS * 32, 1)
differential_mma_kernel(const __grid_constant__ DfParams p, const __grid_constant__ CUtensorMap tmk,
                        const __grid_constant__ CUtensorMap tmv) {
    using M = MmaGeo<D>;
    constexpr int QB = R <= 2 ? 1 : R == 4 ? 2 : D == 128 ? 2 : 3;   // products of S (B operands of Q)
    constexpr int SETS = R == 8 ? 2 : 1;        // accumulators of O
    constexpr int NC = R <= 2 ? 1 : R == 4 ? 2 : 4;      // (query, map) pairs of a lane
    pdl_launch_dependents();                    // the merge grid waits for this grid's end
    extern __shared__ unsigned char smem_raw[];
    __shared__ Prefix prefix;
    unsigned char* smem = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (p.alone && warp >= p.alone) return;
    const int w = p.alone ? blockIdx.x * p.alone + warp : warp * gridDim.x + blockIdx.x;
    constexpr int stages = M::STAGES;
    unsigned char* ring = smem + warp * stages * M::STAGE_BYTES;
    unsigned char* after = smem + M::WARPS * M::STAGES * M::STAGE_BYTES;
    uint64_t* bars = reinterpret_cast<uint64_t*>(after) + warp * stages;
    int32_t* stage_page = reinterpret_cast<int32_t*>(after + M::WARPS * M::STAGES * 8) + warp * stages;
    if (lane == 0 && w < p.W) {
        prefetch_map(&tmk);
        prefetch_map(&tmv);
        for (int s = 0; s < stages; ++s) mbar_init(&bars[s], 1);
        fence_mbar_init();
        if (!p.alone) p.rec[w] = make_int4(0, 0, 0, 0);
    }
    Share share;
    Cursor cur;
    int alone_tiles = 0;
    if (p.alone) {
        alone_tiles = alone_start(p, D, warp, share, cur);
        if (alone_tiles == 0) return;
    } else {
        int stride, entries;
        const int64_t total = build_prefix(p, prefix, stride, entries);
        zero_empty(p, D);
        share = share_of(p, total, w);
        if (share.begin == share.end) return;
        cur = cursor_at(p, prefix, stride, entries, share.begin);
    }
    const bool worked = share.begin < share.end;
    Cursor prod = cur;
    Pager pager;
    const uint64_t policy = l2_stream_policy();
    auto issue = [&](int s) {
        const int32_t page = pager.page(p, prod);
        if (lane == 0) {
            stage_page[s] = page;
            if (page < 0 || page >= p.n_pages) {
                atomicOr(p.err, PKV_DEVERR_PAGE_ID);
                mbar_arrive(&bars[s]);
            } else {
                const int slot = prod.slot * kTile;
                unsigned char* dst = ring + s * M::STAGE_BYTES;
                mbar_arrive_expect_tx(&bars[s], M::STAGE_BYTES);
                tma_load_5d(dst, &tmk, 0, slot, 0, 2 * prod.h, page, &bars[s], policy);
                tma_load_5d(dst + 2 * M::HEAD, &tmv, 0, slot, 0, 2 * prod.h, page, &bars[s], policy);
            }
        }
        if (prod.tile == 0 || prod.tile == prod.n - 1) prefetch_rows<D, sizeof(__nv_bfloat16)>(p, prod);
        cursor_next(p, prod);
    };
    int ahead = 0;                                  // tiles staged and not yet used
    for (; ahead < stages && prod.f < share.end; ++ahead) issue(ahead);

    const int g = lane >> 2, t = lane & 3;          // fragment row, column pair
    const int mj = lane >> 3, mr = lane & 7;        // ldmatrix: matrix and row of this address
    // inside a stage, chunk c (16 bytes) of key row `key` is at
    // (c / 8) * 2048 + key * 128 + ((c % 8) ^ (key % 8)) * 16, heads HEAD apart
    const uint32_t k_row = (uint32_t)((((mj & 1) << 3) + mr) * 128);
    const uint32_t v_row = (uint32_t)((((mj >> 1) << 3) + mr) * 128) + 2 * M::HEAD;
    // combo i of this lane: query row and map
    auto combo_row = [&](int i) { return R == 1 ? 0 : R == 2 ? t >> 1 : R == 4 ? t : 2 * t + (i & 1); };
    auto combo_map = [&](int i) { return R == 1 ? t >> 1 : R == 2 ? t & 1 : R == 4 ? i : i >> 1; };
    uint32_t qb[2][M::KS][QB][2];
    float o[SETS][M::NB][4];
    float m[NC], l[NC];
    bool has_start = false;
    LaneRows L{};
    int s = 0;
    uint32_t parity = 0;

    for (bool first = true; cur.f < share.end; first = false) {
        if (first || cur.tile == 0) {               // a new lane piece
            has_start = cur.tile == 0;
            L = lane_rows(p, cur.x, cur.h, cur.sub);
            // B operand column g: this lane's query and part of it
            const int qr = R == 1 ? 0 : R == 2 ? g >> 2 : R == 4 ? g >> 1 : g;
            int64_t row;
            int head, st, en;
            const bool ok = row_at(p, L, qr, row, head, st, en);
#pragma unroll
            for (int mm = 0; mm < 2; ++mm) {
                // all loads first: one latency, not one for each (a row that is none reads the
                // lane's first)
                const float* q = static_cast<const float*>(p.q) + (row * 2 + mm) * D + 2 * t;
                const float scale = ok ? p.qscale : 0.f;
                float2 x[M::KS][2];
#pragma unroll
                for (int ks = 0; ks < M::KS; ++ks)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        x[ks][i] = *reinterpret_cast<const float2*>(q + ks * 16 + 8 * i);
#pragma unroll
                for (int ks = 0; ks < M::KS; ++ks) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        // what is left after 0, 1, 2 parts; rounding it gives the next part
                        const float a0 = x[ks][i].x * scale, b0 = x[ks][i].y * scale;
                        const uint32_t h0 = pack(a0, b0);
                        const float a1 = a0 - __uint_as_float(h0 << 16);
                        const float b1 = b0 - __uint_as_float(h0 & 0xffff0000u);
                        const uint32_t h1 = pack(a1, b1);
                        const float a2 = a1 - __uint_as_float(h1 << 16);
                        const float b2 = b1 - __uint_as_float(h1 & 0xffff0000u);
                        const uint32_t h2 = pack(a2, b2);
#pragma unroll
                        for (int u = 0; u < QB; ++u) {
                            // parts: R <= 2 g % 4, R = 4 (hi, mid) then (lo, 0), R = 8 part u
                            const int part = R <= 2 ? g & 3 : R == 4 ? 2 * u + (g & 1) : u;
                            qb[mm][ks][u][i] = part == 0 ? h0 : part == 1 ? h1 : part == 2 ? h2 : 0u;
                        }
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                m[i] = -INFINITY;
                l[i] = 0.f;
            }
#pragma unroll
            for (int u = 0; u < SETS; ++u)
#pragma unroll
                for (int nb = 0; nb < M::NB; ++nb)
                    o[u][nb][0] = o[u][nb][1] = o[u][nb][2] = o[u][nb][3] = 0.f;
        }
        if (!mbar_wait_bounded(&bars[s], parity, kWaitNs)) {
            give_up(p, bars, stages, s, parity, ahead);
            break;
        }
        unsigned char* stage = ring + s * M::STAGE_BYTES;
        const int k0 = (cur.tile0 + cur.tile) * kTile;
        const int32_t page = stage_page[s];
        if (page >= 0 && page < p.n_pages) {
            const int lo = L.lo;
            const bool edge = k0 < lo || k0 + kTile > L.t;
            if (edge) {
                // value rows that no query of the lane reads may hold anything: zeros, so that
                // a weight of 0 times them is 0
                for (int i = lane; i < kTile * 2 * M::CH * 8; i += 32) {
                    const int rw = (i >> 3) % kTile;
                    if (k0 + rw < lo || k0 + rw >= L.t)
                        *reinterpret_cast<uint4*>(stage + 2 * M::HEAD + i * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                __syncwarp();
            }
            if (p.k_new != nullptr && L.t - 1 >= k0 && L.t - 1 < k0 + kTile) {
                // the new token's rows: into the staged tile and into the page
                const int slot = L.t - 1 - k0;
                const int64_t src = ((int64_t)cur.x * 2 * p.Hp + 2 * L.h) * D;
                const int64_t dst = (((int64_t)page * 2 * p.Hp + 2 * L.h) * p.P + (L.t - 1) % p.P) * D;
                constexpr int PIECES = 2 * D / 8;   // of both heads' rows
                for (int i = lane; i < 2 * PIECES; i += 32) {
                    const bool value = i >= PIECES;
                    const int c = value ? i - PIECES : i, hd = c / (D / 8), cc = c - hd * (D / 8);
                    const uint4 x = *reinterpret_cast<const uint4*>(
                        static_cast<const __nv_bfloat16*>(value ? p.v_new : p.k_new) + src + c * 8);
                    *reinterpret_cast<uint4*>(stage + (value ? 2 : 0) * M::HEAD + hd * M::HEAD +
                                              (cc >> 3) * kTile * 128 + slot * 128 +
                                              (((cc & 7) ^ (slot & 7)) << 4)) = x;
                    if (L.sub == 0)
                        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(value ? p.v_pages : p.k_pages) +
                                                  dst + (int64_t)hd * p.P * D + cc * 8) = x;
                }
                __syncwarp();
            }
            const uint32_t base = smem_u32(stage);
            float sm[2][4];                         // S of map 0, 1: keys g, g + 8
#pragma unroll
            for (int mm = 0; mm < 2; ++mm) {
                float a[4] = {0.f, 0.f, 0.f, 0.f}, b[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int ks = 0; ks < M::KS; ++ks) {
                    // matrices: (keys 0-7, chunk 2ks), (keys 8-15, 2ks), then chunk 2ks + 1
                    const int c = 2 * ks;
                    uint32_t kf[4];
                    ldsm_x4(base + mm * M::HEAD + (c >> 3) * (kTile * 128) + k_row +
                                ((((c & 7) + (mj >> 1)) ^ mr) << 4), kf);
#pragma unroll
                    for (int u = 0; u < QB; ++u) mma_bf16(ks & 1 ? b : a, kf, qb[mm][ks][u][0], qb[mm][ks][u][1]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) sm[mm][i] = a[i] + b[i];
            }
            float sc[NC][2];                        // scores of the lane's combos at keys g, g + 8
            if constexpr (R <= 2) {
                // both lanes of a pair get hi + mid + lo of their query
#pragma unroll
                for (int mm = 0; mm < 2; ++mm)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float x = sm[mm][2 * i] + sm[mm][2 * i + 1];
                        sm[mm][i] = x + __shfl_xor_sync(0xffffffffu, x, 1);
                    }
                const bool second = combo_map(0) != 0;
                sc[0][0] = second ? sm[1][0] : sm[0][0];
                sc[0][1] = second ? sm[1][1] : sm[0][1];
            } else if constexpr (R == 4) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    sc[i][0] = sm[i][0] + sm[i][1], sc[i][1] = sm[i][2] + sm[i][3];
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[i][0] = sm[i >> 1][i & 1], sc[i][1] = sm[i >> 1][2 + (i & 1)];
            }
            if (edge || L.nt > 1) {
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    int64_t row;
                    int head, st, en;
                    if (!row_at(p, L, combo_row(i), row, head, st, en)) en = 0;
                    if (k0 + g < st || k0 + g >= en) sc[i][0] = -INFINITY;
                    if (k0 + 8 + g < st || k0 + 8 + g >= en) sc[i][1] = -INFINITY;
                }
            }
            float alpha[NC], pr[NC][2];
            bool moved = false;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                float mx = fmaxf(sc[i][0], sc[i][1]);
#pragma unroll
                for (int x = 4; x <= 16; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
                alpha[i] = 1.f;
                if (mx > m[i] + 8.f || (m[i] == -INFINITY && mx > m[i])) {
                    alpha[i] = exp2f(m[i] - mx);    // 0 for the first
                    m[i] = mx;
                    l[i] *= alpha[i];
                    moved = true;
                }
                const float mb = m[i] == -INFINITY ? 0.f : m[i];
                pr[i][0] = exp2f(sc[i][0] - mb), pr[i][1] = exp2f(sc[i][1] - mb);
                l[i] += pr[i][0] + pr[i][1];
            }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int u = 0; u < SETS; ++u) {
                    const float a0 = alpha[R == 8 ? 2 * u : 0], a1 = alpha[R <= 2 ? 0 : 2 * u + 1];
#pragma unroll
                    for (int nb = 0; nb < M::NB; ++nb) {
                        o[u][nb][0] *= a0, o[u][nb][1] *= a1;
                        o[u][nb][2] *= a0, o[u][nb][3] *= a1;
                    }
                }
            }
            // B operands of O: keys 0-7 and 8-15, transposed; smallest parts first
            constexpr int PB = R == 1 ? 1 : R == 2 ? 2 : 3;
            uint32_t pb[SETS][PB][2];
            float part[NC][2][3];
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                split3(pr[i][0], part[i][0]);
                split3(pr[i][1], part[i][1]);
            }
#pragma unroll
            for (int u = 0; u < SETS; ++u)
#pragma unroll
                for (int v = 0; v < PB; ++v)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float* x = part[R == 8 ? 2 * u : 0][i];
                        const float* y = part[R <= 2 ? 0 : 2 * u + 1][i];
                        uint32_t z;
                        if constexpr (R == 1) z = t & 1 ? pack(x[2], 0.f) : pack(x[0], x[1]);
                        else if constexpr (R == 2) z = v == 0 ? pack(x[2], 0.f) : pack(x[0], x[1]);
                        else z = pack(x[2 - v], y[2 - v]);
                        pb[u][v][i] = transpose(z);
                    }
#pragma unroll
            for (int nb = 0; nb < M::NB; ++nb) {
                // matrices: (keys 0-7, chunk 2nb), (keys 0-7, 2nb + 1), then keys 8-15
                constexpr int per = D / 8;          // chunks of one head's row
                const int hd = 2 * nb / per, c = 2 * nb - hd * per;
                uint32_t vf[4];
                ldsm_x4_trans(base + hd * M::HEAD + (c >> 3) * (kTile * 128) + v_row +
                                  ((((c & 7) + (mj & 1)) ^ mr) << 4), vf);
#pragma unroll
                for (int u = 0; u < SETS; ++u) {
                    float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int v = 0; v < PB; ++v) mma_bf16(a, vf, pb[u][v][0], pb[u][v][1]);
                    add2(o[u][nb], a);
                    add2(o[u][nb] + 2, a + 2);
                }
            }
        }
        // the stage is free again: hand it to the copy engine
        fence_proxy_async_smem();
        __syncwarp();
        if (prod.f < share.end) issue(s);
        else --ahead;
        if (++s == stages) {
            s = 0;
            parity ^= 1u;
        }

        const bool has_end = cur.tile == cur.n - 1;
        if (has_end || cur.f + 1 >= share.end) {    // the piece ends
#pragma unroll
            for (int i = 0; i < NC; ++i)
#pragma unroll
                for (int x = 4; x <= 16; x <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
            if constexpr (R <= 2) {
                // columns 2t, 2t + 1 are parts of one value (R = 1: of lanes t, t ^ 1 too)
#pragma unroll
                for (int nb = 0; nb < M::NB; ++nb)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float x = o[0][nb][2 * i] + o[0][nb][2 * i + 1];
                        if constexpr (R == 1) x += __shfl_xor_sync(0xffffffffu, x, 1);
                        o[0][nb][i] = x;
                    }
            }
            // value column nb * 16 + g + 8 i of combo c
            auto value = [&](int c, int nb, int i) {
                return R <= 2 ? o[0][nb][i] : o[R == 8 ? c >> 1 : 0][nb][2 * i + (c & 1)];
            };
            if (has_start && has_end) {
                constexpr int NQ = R == 8 ? 2 : 1;  // queries of a lane
#pragma unroll
                for (int qi = 0; qi < NQ; ++qi) {
                    int64_t row;
                    int head, st, en;
                    const bool ok = row_at(p, L, combo_row(qi), row, head, st, en);
                    const float lam = ok ? __ldg(p.lambda + head) : 0.f;
                    const int c0 = qi, c1 = R == 8 ? 2 + qi : R == 4 ? 1 : 0;    // combos of map 0, 1
                    float d[M::NB][2], sq = 0.f;
                    // R <= 2: the other map is in another lane
                    constexpr int other = R == 1 ? 2 : 1;
                    const bool second = R <= 2 && combo_map(0) != 0;
                    const float mine = R > 2 ? 0.f : l[0] > 0.f ? (second ? -lam : 1.f) / l[0] : 0.f;
                    const float i0 = l[c0] > 0.f ? 1.f / l[c0] : 0.f;
                    const float i1 = l[c1] > 0.f ? lam / l[c1] : 0.f;
#pragma unroll
                    for (int nb = 0; nb < M::NB; ++nb)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            if constexpr (R <= 2) {
                                const float x = value(0, nb, i) * mine;
                                d[nb][i] = x + __shfl_xor_sync(0xffffffffu, x, other);
                            } else {
                                d[nb][i] = value(c0, nb, i) * i0 - value(c1, nb, i) * i1;
                            }
                            sq = fmaf(d[nb][i], d[nb][i], sq);
                        }
#pragma unroll
                    for (int x = 4; x <= 16; x <<= 1) sq += __shfl_xor_sync(0xffffffffu, sq, x);
                    float c = p.out_scale;
                    if (p.normalise) c *= 1.f / sqrtf(sq / (2 * D) + p.norm_eps);
                    if (!ok) continue;
                    const bool weighted = p.normalise && p.norm_weight != nullptr;
                    if (R == 1 && t >= 2) continue; // lanes 0, 1 hold all of it
                    float* op = p.out + row * 2 * D;
                    auto store = [&](int col, float x) {
                        op[col] = x * c * (weighted ? __ldg(p.norm_weight + col) : 1.f);
                    };
#pragma unroll
                    for (int nb = 0; nb < M::NB; ++nb) {
                        if constexpr (R <= 2) {
                            // two lanes hold the same values: one column of each block each
                            store(nb * 16 + g + 8 * (t & 1), t & 1 ? d[nb][1] : d[nb][0]);
                        } else {
                            store(nb * 16 + g, d[nb][0]);
                            store(nb * 16 + g + 8, d[nb][1]);
                        }
                    }
                }
            } else {
                const int64_t slot = 2 * w + (has_start ? 1 : 0);
                float2* ml = p.alone ? reinterpret_cast<float2*>(ring) : p.part_ml + slot * R * 2;
                float* part = p.alone ? reinterpret_cast<float*>(ring + kPartOffset) : p.part_o + slot * R * 4 * D;
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    const int at = combo_row(i) * 2 + combo_map(i);
                    if (g == 0 && (R > 1 || (t & 1) == 0)) ml[at] = make_float2(m[i], l[i]);
                    float* po = part + at * 2 * D + g;
#pragma unroll
                    for (int nb = 0; nb < M::NB; ++nb) {
                        const float x = value(i, nb, 0), y = value(i, nb, 1);
                        if constexpr (R == 1) {
                            po[nb * 16 + 8 * (t & 1)] = t & 1 ? y : x;
                        } else {
                            po[nb * 16] = x;
                            po[nb * 16 + 8] = y;
                        }
                    }
                }
                if (has_start && lane == 0 && !p.alone)
                    p.rec[w] = make_int4(cur.x, cur.ln, last_worker(share, cur.f - cur.tile + cur.n), 1);
            }
        }
        cursor_next(p, cur);
    }
    // a lane of one tile, or of one warp, is finished already
    if (p.alone > 1 && alone_tiles > 1)
        join_alone<D, R>(p, smem, M::STAGES * M::STAGE_BYTES, warp, worked);
}

// ------------------------------------------------------------------ merge --

constexpr int kMergeThreads = 256;
constexpr int kMaxWorkers = 2048;

// CTA (w, r): joins row r of the lane that starts in worker w and ends in a later one
// from the partials of its workers, then takes the difference and the norm.
__global__ void __launch_bounds__(kMergeThreads) differential_merge_kernel(const DfParams p, int D) {
    __shared__ float wgt[2][kMaxWorkers];
    __shared__ float inv[2];
    __shared__ float4 red[kMergeThreads];
    __shared__ float sums[kMergeThreads / 32];
    pdl_wait_primary();
    const int w0 = blockIdx.x, r = blockIdx.y;
    const int4 rc = p.rec[w0];
    if (rc.w == 0) return;
    const LaneRows L = lane_rows(p, rc.x, rc.y / p.subs, rc.y % p.subs);
    int64_t row;
    int head, st, en;
    if (!row_at(p, L, r, row, head, st, en)) return;
    const int n = rc.z - w0 + 1;                    // pieces: slot 2 w0 + 1, then 2 (w0 + i)
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto slot = [&](int i) { return (int64_t)(2 * (w0 + i) + (i == 0 ? 1 : 0)) * p.R + r; };
    if (warp < 2) {
        float mx = -INFINITY;
        for (int i = lane; i < n; i += 32) mx = fmaxf(mx, p.part_ml[slot(i) * 2 + warp].x);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float mb = mx == -INFINITY ? 0.f : mx;
        float lt = 0.f;
        for (int i = lane; i < n; i += 32) {
            const float2 ml = p.part_ml[slot(i) * 2 + warp];
            const float x = exp2f(ml.x - mb);
            wgt[warp][i] = x;
            lt = fmaf(x, ml.y, lt);
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) lt += __shfl_xor_sync(0xffffffffu, lt, o);
        if (lane == 0) inv[warp] = lt > 0.f ? 1.f / lt : 0.f;
    }
    __syncthreads();
    // 2 maps x D / 2 vectors of 4 columns; the threads left over split the pieces
    const int vecs = 2 * D / 4, lanes = 2 * vecs, groups = kMergeThreads / lanes;
    const int g = tid / lanes, at = tid - g * lanes, mm = at / vecs, v = at - mm * vecs;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (g < groups) {
#pragma unroll 4
        for (int i = g; i < n; i += groups) {
            const float4 x =
                __ldcg(reinterpret_cast<const float4*>(p.part_o + (slot(i) * 2 + mm) * 2 * D) + v);
            const float c = wgt[mm][i];
            a.x = fmaf(c, x.x, a.x), a.y = fmaf(c, x.y, a.y);
            a.z = fmaf(c, x.z, a.z), a.w = fmaf(c, x.w, a.w);
        }
    }
    red[tid] = a;
    __syncthreads();
    float4 d = make_float4(0.f, 0.f, 0.f, 0.f);
    float sq = 0.f;
    if (tid < vecs) {
        float4 o[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            o[k] = red[k * vecs + tid];
            for (int i = 1; i < groups; ++i) {
                const float4 x = red[i * lanes + k * vecs + tid];
                o[k].x += x.x, o[k].y += x.y, o[k].z += x.z, o[k].w += x.w;
            }
        }
        const float i0 = inv[0], i1 = inv[1] * __ldg(p.lambda + head);
        d.x = o[0].x * i0 - o[1].x * i1, d.y = o[0].y * i0 - o[1].y * i1;
        d.z = o[0].z * i0 - o[1].z * i1, d.w = o[0].w * i0 - o[1].w * i1;
        sq = d.x * d.x + d.y * d.y + d.z * d.z + d.w * d.w;
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
    if (lane == 0) sums[warp] = sq;
    __syncthreads();
    if (tid >= vecs) return;
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < kMergeThreads / 32; ++i) t += sums[i];
    float c = p.out_scale;
    float4 nw = make_float4(1.f, 1.f, 1.f, 1.f);
    if (p.normalise) {
        c *= 1.f / sqrtf(t / (2 * D) + p.norm_eps);
        if (p.norm_weight) {
            nw.x = __ldg(p.norm_weight + 4 * tid), nw.y = __ldg(p.norm_weight + 4 * tid + 1);
            nw.z = __ldg(p.norm_weight + 4 * tid + 2), nw.w = __ldg(p.norm_weight + 4 * tid + 3);
        }
    }
    reinterpret_cast<float4*>(p.out + row * 2 * D)[tid] =
        make_float4(d.x * c * nw.x, d.y * c * nw.y, d.z * c * nw.z, d.w * c * nw.w);
}

// ----------------------------------------------------------- prefill lanes --

struct ChunkParams {
    int B, H, D, P, es, bt;         // bt: chunk tokens of one block
    int64_t N, X, n_pages;
    const int32_t* cu_new;          // nullptr: one request of N rows, length single_t
    const int32_t* seq_lens;
    int single_t;
    const int32_t* tables;
    int max_pages;
    const void* k_new;
    const void* v_new;
    void* k_pages;
    void* v_pages;
    int32_t *rows, *lens, *tok0, *ntok, *first;
    unsigned* err;
};

__device__ __forceinline__ int chunk_cu(const ChunkParams& p, int b) {
    return p.cu_new ? __ldg(p.cu_new + b) : (b == 0 ? 0 : (int)p.N);
}

__device__ __forceinline__ int64_t chunk_len(const ChunkParams& p, int b) {
    return p.seq_lens ? __ldg(p.seq_lens + b) : p.single_t;
}

__device__ __forceinline__ bool chunk_ok(const ChunkParams& p, int b) {
    const int64_t c0 = chunk_cu(p, b), c1 = chunk_cu(p, b + 1), t = chunk_len(p, b);
    return c0 >= 0 && c1 >= c0 && c1 <= p.N && t - (c1 - c0) >= 0 && t <= (int64_t)p.max_pages * p.P;
}

// Every new key / value row into its page: VEC bytes a thread.
template <int VEC>
__global__ void __launch_bounds__(256) differential_append_kernel(const ChunkParams p) {
    pdl_launch_dependents();                    // an attention grid may start; it waits for the rows
    const int pieces = p.D * p.es / VEC;
    const int64_t total = p.N * p.H * pieces;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t x = i / (p.H * pieces);
        const int rem = (int)(i - x * p.H * pieces);
        const int h = rem / pieces, u = rem - h * pieces;
        int lo = 0, hi = p.B;                       // last request with cu_new[b] <= x
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (chunk_cu(p, mid) <= x) lo = mid;
            else hi = mid;
        }
        if (!chunk_ok(p, lo)) continue;             // the plan reports it
        const int64_t c0 = chunk_cu(p, lo), c1 = chunk_cu(p, lo + 1);
        if (x < c0 || x >= c1) continue;
        const int64_t pos = chunk_len(p, lo) - (c1 - c0) + (x - c0);
        const int32_t page = p.tables[(int64_t)lo * p.max_pages + pos / p.P];
        if (page < 0 || page >= p.n_pages) {
            atomicOr(p.err, PKV_DEVERR_PAGE_ID);
            continue;
        }
        const int64_t dst = ((((int64_t)page * p.H + h) * p.P + pos % p.P) * p.D) * p.es + (int64_t)u * VEC;
        const int64_t src = ((x * p.H + h) * p.D) * p.es + (int64_t)u * VEC;
        const char *ks = static_cast<const char*>(p.k_new) + src, *vs = static_cast<const char*>(p.v_new) + src;
        char *kd = static_cast<char*>(p.k_pages) + dst, *vd = static_cast<char*>(p.v_pages) + dst;
        if constexpr (VEC == 16) {
            *reinterpret_cast<uint4*>(kd) = *reinterpret_cast<const uint4*>(ks);
            *reinterpret_cast<uint4*>(vd) = *reinterpret_cast<const uint4*>(vs);
        } else {
            *reinterpret_cast<uint32_t*>(kd) = *reinterpret_cast<const uint32_t*>(ks);
            *reinterpret_cast<uint32_t*>(vd) = *reinterpret_cast<const uint32_t*>(vs);
        }
    }
}

// Blocks of bt chunk tokens, request by request: table row, length after the block's
// last token, first chunk row, tokens.  Blocks past the last have length 0.  One CTA.
__global__ void __launch_bounds__(1024) differential_blocks_kernel(const ChunkParams p) {
    __shared__ int warp_sum[32];
    __shared__ int carry_s;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    if (tid == 0) carry_s = 0;
    __syncthreads();
    for (int base = 0; base < p.B; base += 1024) {
        const int b = base + tid;
        int nb = 0;
        if (b < p.B) {
            if (!chunk_ok(p, b)) atomicOr(p.err, PKV_DEVERR_SEQ_LEN);
            else nb = (chunk_cu(p, b + 1) - chunk_cu(p, b) + p.bt - 1) / p.bt;
        }
        int incl = nb;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) warp_sum[wid] = incl;
        __syncthreads();
        int at = carry_s + incl - nb, all = 0;
        for (int w = 0; w < 32; ++w) {
            if (w < wid) at += warp_sum[w];
            all += warp_sum[w];
        }
        if (b < p.B) p.first[b] = at;
        __syncthreads();
        if (tid == 0) carry_s += all;
        __syncthreads();
    }
    const int total = carry_s;
    // requests whose row ranges overlap can hold more blocks than the launch has room for
    if (total > p.X && tid == 0) atomicOr(p.err, PKV_DEVERR_SEQ_LEN);
    for (int64_t x = tid; x < p.X; x += 1024) {
        int row = 0, len = 0, t0 = 0, nt = 0;
        if (x < total) {
            int lo = 0, hi = p.B;                   // last request with first[b] <= x
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (p.first[mid] <= x) lo = mid;
                else hi = mid;
            }
            const int c0 = chunk_cu(p, lo), n = chunk_cu(p, lo + 1) - c0;
            const int k = (int)(x - p.first[lo]) * p.bt;
            row = lo;
            t0 = c0 + k;
            nt = n - k < p.bt ? n - k : p.bt;
            len = (int)(chunk_len(p, lo) - n + k + nt);
        }
        p.rows[x] = row;
        p.lens[x] = len;
        p.tok0[x] = t0;
        p.ntok[x] = nt;
    }
}

// ------------------------------------------------------------------- host --

// Opt a kernel into its dynamic shared memory, once per device.
template <typename K>
cudaError_t configure(K kernel, int bytes, bool* done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && done[dev]) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) done[dev] = true;
    return e;
}

// bf16 at head width 64 and 128 runs on the tensor cores.
bool use_mma(int dtype, int D) { return dtype == PKV_BF16 && (D == 64 || D == 128); }

// Most query rows of one lane.
int most_rows(int dtype, int D) { return use_mma(dtype, D) ? 8 : D == 64 || D == 128 ? 4 : 1; }

// Other head widths, one row a lane: f(T, D, R).
#define PKV_DF_CORE(F)                                                                    \
    F(float, 2, 1) F(float, 4, 1) F(float, 8, 1) F(float, 16, 1) F(float, 32, 1)           \
    F(__nv_bfloat16, 2, 1) F(__nv_bfloat16, 4, 1) F(__nv_bfloat16, 8, 1)                  \
    F(__nv_bfloat16, 16, 1) F(__nv_bfloat16, 32, 1) F(__nv_bfloat16, 256, 1)

// CTAs of a launch: workers go to CTA after CTA; or one lane a CTA.
int grid_of(const DfParams& p, int sms) {
    return p.alone ? p.W / p.alone : p.W < sms ? p.W : sms;
}

template <typename T, int D, int R>
cudaError_t launch_core(const DfParams& p, int sms, cudaStream_t stream) {
    using M = CoreGeo<T, D, R>;
    static bool done[64] = {};
    cudaError_t e = configure(differential_core_kernel<T, D, R>, M::SMEM, done);
    if (e != cudaSuccess) return e;
    const int grid = grid_of(p, sms);
    differential_core_kernel<T, D, R><<<grid, M::WARPS * 32, M::SMEM, stream>>>(p);
    return cudaGetLastError();
}

template <int D, int R>
cudaError_t launch_mma(const DfParams& p, const void* tmap_k, const void* tmap_v, int sms,
                       cudaStream_t stream) {
    using M = MmaGeo<D>;
    static bool done[64] = {};
    cudaError_t e = configure(differential_mma_kernel<D, R>, M::SMEM, done);
    if (e != cudaSuccess) return e;
    CUtensorMap tmk, tmv;
    std::memcpy(&tmk, tmap_k, sizeof tmk);
    std::memcpy(&tmv, tmap_v, sizeof tmv);
    const int grid = grid_of(p, sms);
    differential_mma_kernel<D, R><<<grid, M::WARPS * 32, M::SMEM, stream>>>(p, tmk, tmv);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_mma_rows(const DfParams& p, const void* tmap_k, const void* tmap_v, int sms,
                            cudaStream_t stream) {
    switch (p.R) {
        case 1: return launch_mma<D, 1>(p, tmap_k, tmap_v, sms, stream);
        case 2: return launch_mma<D, 2>(p, tmap_k, tmap_v, sms, stream);
        case 4: return launch_mma<D, 4>(p, tmap_k, tmap_v, sms, stream);
        case 8: return launch_mma<D, 8>(p, tmap_k, tmap_v, sms, stream);
        default: return cudaErrorInvalidValue;
    }
}

// fp32 at head width 64 and 128: f(D, R, KT).
constexpr int kTileF32_64 = 16, kTileF32_128 = 8;
#define PKV_DF_F32(F)                                                                     \
    F(64, 1, kTileF32_64) F(64, 2, kTileF32_64) F(64, 4, kTileF32_64)                      \
    F(128, 1, kTileF32_128) F(128, 2, kTileF32_128) F(128, 4, kTileF32_128)

int tile_of(int dtype, int D) {
    return dtype == PKV_F32 && D == 64 ? kTileF32_64 : dtype == PKV_F32 && D == 128 ? kTileF32_128 : kTile;
}

template <int D, int R, int KT>
cudaError_t launch_f32(const DfParams& p, const void* tmap_k, const void* tmap_v, int sms,
                       cudaStream_t stream) {
    using M = F32Geo<D, R, KT>;
    static bool done[64] = {};
    cudaError_t e = configure(differential_f32_kernel<D, R, KT>, M::SMEM, done);
    if (e != cudaSuccess) return e;
    CUtensorMap tmk, tmv;
    std::memcpy(&tmk, tmap_k, sizeof tmk);
    std::memcpy(&tmv, tmap_v, sizeof tmv);
    const int grid = grid_of(p, sms);
    differential_f32_kernel<D, R, KT><<<grid, M::WARPS * 32, M::SMEM, stream>>>(p, tmk, tmv);
    return cudaGetLastError();
}

// A decode of up to kAloneTiles tiles a warp, and no more lanes than SMs, gives each lane to
// the warps of one CTA, which join it in shared memory: one launch, no scan of the lengths,
// no scratch.  On the device, against the split over the GPU and its merge, at 128 / 256
// positions a request: 12 heads of 64, fp32, 1 request 8.2 / 9.7 us against 10.5 / 11.6, 8
// requests 10.0 / 11.4 against 14.1 / 14.9, 24 requests 10.3 / 12.2 against 14.9 / 16.7; 8
// heads of 128, bf16, 1 request 11.6 / 13.0 against 14.1 / 14.8, 8 requests 13.3 / 14.7
// against 17.6 / 18.5, 36 requests 13.5 / 15.4 against 18.5 / 20.1.  At 512 positions the
// split wins for one request (12.7 against 15.0; 17.3, 17.5).
// Both forms are one kernel: as two, both were within 2 % of this, for a third more to compile.
constexpr int kAloneTiles = 4;

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

bool differential_needs_maps(int dtype, int D) { return D == 64 || D == 128; }

int differential_tile(int dtype, int D) { return tile_of(dtype, D); }

int differential_rows(int dtype, int D, int G) {
    const int most = most_rows(dtype, D);
    return G < most ? G : most;
}

int differential_block_tokens(int dtype, int D, int G) {
    const int most = most_rows(dtype, D);
    return G <= most ? most / G : 1;
}

namespace {

// Warps of a CTA of the split kernel.
int warps_of(int dtype, int D, int rows) {
    int warps = use_mma(dtype, D) ? (D == 64 ? MmaGeo<64>::WARPS : MmaGeo<128>::WARPS) : 0;
#define PKV_DF_WARPS(T, DD, RR) \
    if (dtype == (sizeof(T) == 4 ? PKV_F32 : PKV_BF16) && D == DD && rows == RR) warps = CoreGeo<T, DD, RR>::WARPS;
    PKV_DF_CORE(PKV_DF_WARPS)
#undef PKV_DF_WARPS
#define PKV_DF_WARPS(DD, RR, KT) \
    if (dtype == PKV_F32 && D == DD && rows == RR) warps = F32Geo<DD, RR, KT>::WARPS;
    PKV_DF_F32(PKV_DF_WARPS)
#undef PKV_DF_WARPS
    return warps;
}

}  // namespace

DifferentialSplit differential_split(int dtype, int D, int rows, int num_sms, bool decode, int64_t lanes,
                                     int64_t max_len) {
    const int warps = warps_of(dtype, D, rows), tile = tile_of(dtype, D);
    const int64_t per = (max_len + tile - 1) / tile, tiles = lanes * per;
    DifferentialSplit s{};
    if (decode && (D == 64 || D == 128) && per <= (int64_t)kAloneTiles * warps && lanes <= num_sms) {
        s.alone = per < warps ? (int)per : warps;
        s.workers = (int)lanes * s.alone;
        return s;
    }
    int64_t w = (int64_t)warps * num_sms;
    if (w > kMaxWorkers) w = kMaxWorkers / num_sms * num_sms;
    s.workers = (int)(tiles < w ? (tiles < 1 ? 1 : tiles) : w);
    return s;
}

DifferentialLayout differential_layout(int D, int rows, DifferentialSplit split) {
    DifferentialLayout L{};
    if (split.alone) return L;
    const int workers = split.workers;
    L.rec = 0;
    L.part_ml = up256(L.rec + sizeof(int4) * (size_t)workers);
    L.part_o = up256(L.part_ml + sizeof(float2) * 2 * 2 * (size_t)workers * rows);
    L.total = up256(L.part_o + sizeof(float) * 2 * 2 * 2 * (size_t)workers * rows * D);
    return L;
}

cudaError_t launch_differential(const DifferentialArgs& a, cudaStream_t stream) {
    DfParams p{};
    p.q = a.q;
    p.q_bf16 = a.q_bf16;
    p.k_new = a.k_new;
    p.v_new = a.v_new;
    p.k_pages = a.k_pages;
    p.v_pages = a.v_pages;
    p.n_pages = a.n_pages;
    p.tables = a.tables;
    p.max_pages = a.max_pages;
    p.table_rows = a.table_rows;
    p.seq_lens = a.seq_lens;
    p.single_t = a.single_t;
    p.max_seq_len = a.max_seq_len;
    p.tok0 = a.tok0;
    p.ntok = a.ntok;
    p.B = a.B;
    p.Hp = a.H / 2;
    p.G = a.G;
    p.R = a.rows;
    p.subs = a.ntok ? (a.block_tokens * a.G + a.rows - 1) / a.rows : (a.G + a.rows - 1) / a.rows;
    p.P = a.P;
    p.tile = tile_of(a.dtype, a.D);
    p.window = a.window;
    p.qscale = (float)(1.4426950408889634 / std::sqrt((double)a.D));
    p.lambda = a.diff.lambda;
    p.norm_weight = a.diff.norm_weight;
    p.normalise = a.diff.normalise;
    p.norm_eps = a.diff.norm_eps;
    p.out_scale = a.diff.out_scale;
    p.out = a.out;
    p.W = a.split.workers;
    p.err = a.dev_error;
    p.alone = a.split.alone;
    const DifferentialLayout L = differential_layout(a.D, a.rows, a.split);
    unsigned char* ws = static_cast<unsigned char*>(a.workspace);
    p.rec = reinterpret_cast<int4*>(ws + L.rec);
    p.part_ml = reinterpret_cast<float2*>(ws + L.part_ml);
    p.part_o = reinterpret_cast<float*>(ws + L.part_o);
    if (a.ev_before) cudaEventRecord(a.ev_before, stream);
    cudaError_t e = cudaErrorInvalidValue;
    if (use_mma(a.dtype, a.D))
        e = a.D == 64 ? launch_mma_rows<64>(p, a.tmap_k, a.tmap_v, a.sms, stream)
                      : launch_mma_rows<128>(p, a.tmap_k, a.tmap_v, a.sms, stream);
#define PKV_DF_LAUNCH(T, DD, RR)                                                              \
    if (a.dtype == (sizeof(T) == 4 ? PKV_F32 : PKV_BF16) && a.D == DD && a.rows == RR)        \
        e = launch_core<T, DD, RR>(p, a.sms, stream);
    PKV_DF_CORE(PKV_DF_LAUNCH)
#undef PKV_DF_LAUNCH
#define PKV_DF_LAUNCH(DD, RR, KT)                                                             \
    if (a.dtype == PKV_F32 && a.D == DD && a.rows == RR)                                      \
        e = launch_f32<DD, RR, KT>(p, a.tmap_k, a.tmap_v, a.sms, stream);
    PKV_DF_F32(PKV_DF_LAUNCH)
#undef PKV_DF_LAUNCH
    if (e != cudaSuccess) return e;
    if (a.ev_after) cudaEventRecord(a.ev_after, stream);
    if (p.alone) return cudaSuccess;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)p.W, (unsigned)p.R);
    cfg.blockDim = dim3(kMergeThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, differential_merge_kernel, p, a.D);
}

DifferentialChunkLayout differential_chunk_layout(int64_t N, int batch, int block_tokens, int D, int rows,
                                                  DifferentialSplit split) {
    DifferentialChunkLayout L{};
    L.blocks = N / block_tokens + batch;
    size_t at = differential_layout(D, rows, split).total;
    auto take = [&](int64_t n) {
        const size_t o = at;
        at = up256(at + sizeof(int32_t) * (size_t)n);
        return o;
    };
    L.rows = take(L.blocks);
    L.lens = take(L.blocks);
    L.tok0 = take(L.blocks);
    L.ntok = take(L.blocks);
    L.first = take(batch + 1);
    L.total = at;
    return L;
}

namespace {

ChunkParams chunk_params(const DifferentialArgs& a, int batch, int64_t total_new, const int32_t* cu_new) {
    ChunkParams c{};
    c.B = batch;
    c.H = a.H;
    c.D = a.D;
    c.P = a.P;
    c.es = a.dtype == PKV_F32 ? 4 : 2;
    c.bt = a.block_tokens;
    c.N = total_new;
    c.n_pages = a.n_pages;
    c.cu_new = cu_new;
    c.seq_lens = a.seq_lens;
    c.single_t = a.single_t;
    c.tables = a.tables;
    c.max_pages = a.max_pages;
    c.k_new = a.k_new;
    c.v_new = a.v_new;
    c.k_pages = a.k_pages;
    c.v_pages = a.v_pages;
    c.err = a.dev_error;
    return c;
}

}  // namespace

cudaError_t launch_differential_append(const DifferentialArgs& a, int batch, int64_t total_new,
                                       const int32_t* cu_new, cudaStream_t stream) {
    const ChunkParams c = chunk_params(a, batch, total_new, cu_new);
    const int vec = a.D * c.es >= 16 ? 16 : 4;
    const int64_t pieces = total_new * a.H * (a.D * c.es / vec);
    const int64_t want = (pieces + 255) / 256, most = (int64_t)a.sms * 8;
    const unsigned grid = (unsigned)(want < most ? want : most);
    if (vec == 16) differential_append_kernel<16><<<grid, 256, 0, stream>>>(c);
    else differential_append_kernel<4><<<grid, 256, 0, stream>>>(c);
    return cudaGetLastError();
}

cudaError_t launch_differential_chunks(const DifferentialArgs& args, int batch, int64_t total_new,
                                       const int32_t* cu_new, cudaStream_t stream) {
    DifferentialArgs a = args;
    const DifferentialChunkLayout L =
        differential_chunk_layout(total_new, batch, a.block_tokens, a.D, a.rows, a.split);
    unsigned char* ws = static_cast<unsigned char*>(a.workspace);
    ChunkParams c = chunk_params(a, batch, total_new, cu_new);
    c.X = L.blocks;
    c.rows = reinterpret_cast<int32_t*>(ws + L.rows);
    c.lens = reinterpret_cast<int32_t*>(ws + L.lens);
    c.tok0 = reinterpret_cast<int32_t*>(ws + L.tok0);
    c.ntok = reinterpret_cast<int32_t*>(ws + L.ntok);
    c.first = reinterpret_cast<int32_t*>(ws + L.first);
    cudaError_t e = launch_differential_append(a, batch, total_new, cu_new, stream);
    if (e != cudaSuccess) return e;
    differential_blocks_kernel<<<1, 1024, 0, stream>>>(c);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    a.k_new = a.v_new = nullptr;                    // stored already
    a.B = (int)L.blocks;
    a.table_rows = c.rows;
    a.seq_lens = c.lens;
    a.tok0 = c.tok0;
    a.ntok = c.ntok;
    a.max_seq_len = (int64_t)a.max_pages * a.P;
    return launch_differential(a, stream);
}

}  // namespace pkv
