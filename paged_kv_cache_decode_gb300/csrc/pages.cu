// Moving tokens between pages of a pool: whole pages (copies for forked requests)
// and selected rows (compaction of an evicted cache), K and V of every layer in one
// launch.
//
// copy:     pages[dst_i] = pages[src_i], i < n, in each of the 2 x layers pools
//           [pages][H][P][D]; a page of one pool is one contiguous block.
// compact:  row cu[b] + i of `keep` names a position of request b; that row of every
//           head moves to position i of the request's new table.
//
// Bound: bytes read plus bytes written at the copy bandwidth of the memory; nothing
// is computed.
//
// Ids and positions that do not fit set bits of the pool's device error word and
// their bytes are not moved.

#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "pkv.h"
#include "pkv_internal.h"

namespace pkv {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;                          // 16-byte pieces of one thread in flight

struct CopyParams {
    char* k_base;                                   // [layers][pages][page_bytes]
    char* v_base;
    int64_t layer_bytes, page_bytes, n_pages;
    int layers, n;
    int64_t chunks;                                 // units of one page: kThreads * kUnroll * 16 bytes
    unsigned* err;
};

// Where the ids of pair i come from: device lists, or a host list that travels with the
// launch.
struct DeviceIds {
    const int32_t* src;
    const int32_t* dst;
    __device__ int2 at(int i) const { return make_int2(__ldg(src + i), __ldg(dst + i)); }
};

struct ListIds {
    int2 pair[kInlinePairs];
    __device__ int2 at(int i) const { return pair[i]; }
};

// One unit per turn: a chunk (16 KB; with 8 KB 314 us instead of 311 for 2 GB) of one
// page of one pool.
template <typename IDS>
__global__ void __launch_bounds__(kThreads)
copy_pages_kernel(const __grid_constant__ CopyParams p, const __grid_constant__ IDS ids) {
    const int64_t units = (int64_t)p.n * p.layers * 2 * p.chunks;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t page_unit = u / p.chunks, chunk = u - page_unit * p.chunks;
        const int64_t pool = page_unit / p.n;
        const int i = (int)(page_unit - pool * p.n);
        const int2 pair = ids.at(i);
        const int src = pair.x, dst = pair.y;
        if (src < 0 || src >= p.n_pages || dst < 0 || dst >= p.n_pages) {
            if (threadIdx.x == 0) atomicOr(p.err, PKV_DEVERR_PAGE_ID);
            continue;
        }
        char* base = ((pool & 1) ? p.v_base : p.k_base) + (pool >> 1) * p.layer_bytes;
        const char* s = base + (int64_t)src * p.page_bytes;
        char* d = base + (int64_t)dst * p.page_bytes;
        const int64_t at = (chunk * kThreads * kUnroll + threadIdx.x) * 16;
        uint4 v[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k)
            if (at + k * kThreads * 16 < p.page_bytes)
                v[k] = *reinterpret_cast<const uint4*>(s + at + k * kThreads * 16);
#pragma unroll
        for (int k = 0; k < kUnroll; ++k)
            if (at + k * kThreads * 16 < p.page_bytes)
                *reinterpret_cast<uint4*>(d + at + k * kThreads * 16) = v[k];
    }
}

constexpr int kGroup = 16;                          // kept rows whose places one CTA looks up

struct CompactParams {
    char* k_base;
    char* v_base;
    int64_t layer_bytes, n_pages;
    int layers, H, P, row_bytes, batch;
    int64_t total;
    const int32_t* keep;                            // [total] positions
    const int32_t* cu;                              // [batch + 1]; nullptr: one request, `total` rows
    const int32_t* tables;                          // [batch][max_pages]
    int max_pages;
    const int32_t* seq_lens;                        // [batch]; nullptr: single_t
    int64_t single_t;
    const int32_t* new_tables;                      // [batch][new_max_pages]
    int new_max_pages;
    int per_cta;                                    // (layer, K or V, head) blocks of one CTA
    unsigned* err;
};

// CTA (group, part): kGroup consecutive kept rows, per_cta of the 2 x layers x heads
// blocks.  The rows' places are looked up once, by the group's first threads.
template <int VEC>
__global__ void __launch_bounds__(kThreads) compact_kernel(const __grid_constant__ CompactParams p) {
    using V = typename std::conditional<VEC == 16, uint4, uint32_t>::type;
    __shared__ int64_t from_s[kGroup], to_s[kGroup];    // first row of the page's head 0, or -1
    const int64_t j0 = (int64_t)blockIdx.x * kGroup;
    if (threadIdx.x < kGroup) {
        const int64_t j = j0 + threadIdx.x;
        int64_t from = -1, to = -1;
        if (j < p.total) {
            int lo = 0, hi = p.cu ? p.batch : 1;        // last request with cu[b] <= j
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (__ldg(p.cu + mid) <= j) lo = mid;
                else hi = mid;
            }
            const int64_t c0 = p.cu ? __ldg(p.cu + lo) : 0, c1 = p.cu ? __ldg(p.cu + lo + 1) : p.total;
            const int64_t len = p.seq_lens ? __ldg(p.seq_lens + lo) : p.single_t;
            const int64_t pos = __ldg(p.keep + j), at = j - c0;
            if (j < c0 || j >= c1 || pos < 0 || pos >= len || pos / p.P >= p.max_pages ||
                at / p.P >= p.new_max_pages) {
                atomicOr(p.err, PKV_DEVERR_SEQ_LEN);
            } else {
                const int32_t a = __ldg(p.tables + (int64_t)lo * p.max_pages + pos / p.P);
                const int32_t b = __ldg(p.new_tables + (int64_t)lo * p.new_max_pages + at / p.P);
                if (a < 0 || a >= p.n_pages || b < 0 || b >= p.n_pages) {
                    atomicOr(p.err, PKV_DEVERR_PAGE_ID);
                } else {
                    from = ((int64_t)a * p.H) * p.P + pos % p.P;
                    to = ((int64_t)b * p.H) * p.P + at % p.P;
                }
            }
        }
        from_s[threadIdx.x] = from;
        to_s[threadIdx.x] = to;
    }
    __syncthreads();
    const int pieces = p.row_bytes / VEC;
    const int blocks = p.layers * 2 * p.H;
    const int b0 = blockIdx.y * p.per_cta, b1 = min(b0 + p.per_cta, blocks);
    const int work = (b1 - b0) * kGroup * pieces;
    for (int i0 = threadIdx.x; i0 < work; i0 += kThreads * kUnroll) {
        V v[kUnroll];
        char* to[kUnroll];
#pragma unroll
        for (int k = 0; k < kUnroll; ++k) {
            const int i = i0 + k * kThreads;
            to[k] = nullptr;
            if (i >= work) continue;
            const int blk = b0 + i / (kGroup * pieces), rem = i % (kGroup * pieces);
            const int row = rem / pieces, u = rem - row * pieces;
            const int64_t from = from_s[row];
            if (from < 0) continue;
            const int pool = blk / p.H, h = blk - pool * p.H;
            char* base = ((pool & 1) ? p.v_base : p.k_base) + (int64_t)(pool >> 1) * p.layer_bytes;
            const int64_t off = (int64_t)h * p.P;
            v[k] = *reinterpret_cast<const V*>(base + (from + off) * p.row_bytes + u * VEC);
            to[k] = base + (to_s[row] + off) * p.row_bytes + u * VEC;
        }
#pragma unroll
        for (int k = 0; k < kUnroll; ++k)
            if (to[k]) *reinterpret_cast<V*>(to[k]) = v[k];
    }
}

CopyParams copy_params(const PageStore& s, int n) {
    CopyParams p{};
    p.k_base = static_cast<char*>(s.k_base);
    p.v_base = static_cast<char*>(s.v_base);
    p.layer_bytes = s.layer_bytes;
    p.page_bytes = (int64_t)s.H * s.P * s.row_bytes;
    p.n_pages = s.n_pages;
    p.layers = s.layers;
    p.n = n;
    p.chunks = (p.page_bytes + kThreads * kUnroll * 16 - 1) / (kThreads * kUnroll * 16);
    p.err = s.dev_error;
    return p;
}

// A CTA for each unit: 2048 pages of 131 KB in two layers take 311 us (1.02 of the copy
// bandwidth), with eight CTAs an SM that loop over the units 343 us.
unsigned copy_grid(const CopyParams& p) {
    const int64_t units = (int64_t)p.n * p.layers * 2 * p.chunks, most = 1 << 30;
    return (unsigned)(units < most ? units : most);
}

}  // namespace

cudaError_t launch_copy_pages(const PageStore& s, int n, const int32_t* src, const int32_t* dst,
                              cudaStream_t stream) {
    const CopyParams p = copy_params(s, n);
    copy_pages_kernel<<<copy_grid(p), kThreads, 0, stream>>>(p, DeviceIds{src, dst});
    return cudaGetLastError();
}

cudaError_t launch_copy_page_list(const PageStore& s, int n, const int32_t* src, const int32_t* dst,
                                  cudaStream_t stream) {
    for (int i = 0; i < n; i += kInlinePairs) {
        const int m = n - i < kInlinePairs ? n - i : kInlinePairs;
        const CopyParams p = copy_params(s, m);
        ListIds list{};
        for (int k = 0; k < m; ++k) list.pair[k] = make_int2(src[i + k], dst[i + k]);
        copy_pages_kernel<<<copy_grid(p), kThreads, 0, stream>>>(p, list);
        cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_compact(const PageStore& s, const CompactArgs& a, cudaStream_t stream) {
    CompactParams p{};
    p.k_base = static_cast<char*>(s.k_base);
    p.v_base = static_cast<char*>(s.v_base);
    p.layer_bytes = s.layer_bytes;
    p.n_pages = s.n_pages;
    p.layers = s.layers;
    p.H = s.H;
    p.P = s.P;
    p.row_bytes = s.row_bytes;
    p.batch = a.batch;
    p.total = a.total;
    p.keep = a.keep;
    p.cu = a.cu_keep;
    p.tables = a.tables;
    p.max_pages = a.max_pages;
    p.seq_lens = a.seq_lens;
    p.single_t = a.single_t;
    p.new_tables = a.new_tables;
    p.new_max_pages = a.new_max_pages;
    p.err = s.dev_error;
    const int vec = s.row_bytes % 16 == 0 ? 16 : 4;
    const int64_t groups = (a.total + kGroup - 1) / kGroup;
    const int blocks = s.layers * 2 * s.H;
    // at least one turn of every thread a CTA, and CTAs for two full waves of the GPU (64
    // requests, about half of up to 8192 rows each, two layers: 347 us, 0.96 of the copy
    // bandwidth; 8 pieces in flight a thread: 429 us, 2: 374 us)
    const int least = (kThreads * kUnroll + kGroup * (s.row_bytes / vec) - 1) / (kGroup * (s.row_bytes / vec));
    const int64_t want = ((int64_t)s.sms * 16 + groups - 1) / groups;       // parts per group
    int64_t per = (blocks + want - 1) / want;
    if (per < least) per = least;
    if (per > blocks) per = blocks;
    p.per_cta = (int)per;
    const dim3 grid((unsigned)groups, (unsigned)((blocks + per - 1) / per));
    if (vec == 16) compact_kernel<16><<<grid, kThreads, 0, stream>>>(p);
    else compact_kernel<4><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace pkv
