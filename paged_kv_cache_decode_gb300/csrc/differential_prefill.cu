// Differential attention of prefill chunks on the sm_103a tensor cores (bf16 pools of
// head width 64 or 128); differential.cu holds the formula and every other pool.
//
// Two launches per call: the chunk's rows are stored in their pages, then one CTA
// per (query tile, KV pair, output half) attends them.
//
// Attention CTA.  A query tile is 128 rows: 128/G consecutive chunk tokens times the
// G query pairs that share one KV pair.  Map 0 and map 1 of the same rows are two
// score tiles, A and B, against the keys of the pair's first and second head; both
// multiply the same values:
//     S_A = Q_0 K_0^T, S_B = Q_1 K_1^T   tcgen05.mma, M=128 N=128 K=d_h, fp32 in TMEM
//     P_x = 2^(c S_x - c m_x)            softmax warps: TMEM -> registers -> bf16 hi + lo
//                                        back into TMEM over the S columns already read
//     O_x += P_hi,x V + P_lo,x V         tcgen05.mma, A = P from TMEM, M=128 N=128 K=128
// with c = log2(e) / sqrt(d_h).  S_A, S_B, O_A and O_B of 128 columns each fill the
// 512 columns of TMEM, so one CTA holds 128 of the pair's 2 d_h value columns: both
// heads' at d_h = 64; at d_h = 128 the two CTAs of a cluster take one head's each
// and compute the scores twice (12 units of MMA work per key tile where one CTA per
// map would need 10, but the same code for both widths and no exchange of O).
// Warp roles (320 threads):
//   warps 0-3, 4-7  softmax of A, B: one query row per thread; they stage Q, write P,
//              rescale O.  At the end each group takes 64 output columns of the
//              same rows: d = O_A / l_A - lambda O_B / l_B, mean square over all
//              2 d_h columns (across the cluster through distributed shared
//              memory), store;
//   warp 8     producer: eight lanes issue the K / V tile copies, one 16-row group
//              each (a group never straddles a page);
//   warp 9     MMA: allocates TMEM, one thread issues the MMAs and commits.
// The MMA order P V_A(j), S_A(j+1), P V_B(j), S_B(j+1) ... keeps the tensor cores on
// one map while the other map's softmax runs; MMAs of one thread run in issue order,
// so S_A(j+1) overwrites P_A(j) only after P V_A(j) has read it.
//
// Bound: the tensor cores (P V twice for the hi and lo parts of the weights, which
// carry each to about 2^-17; one bf16 part alone would be off by 2^-9).  The row
// maximum is only followed when it grows by more than 8 in log2 units (the weights
// stay below 2^8 and O / l uses the same base in both).
//
// Faults: bad lengths and page ids set bits of the device error word (a bad page
// reads as zeros); a wait that runs out sets the timeout bit and ends the CTA's work.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "pkv.h"
#include "pkv_internal.h"
#include "ptx.cuh"
#include "tc05.cuh"

namespace pkv {

namespace {

constexpr int kRows = 128;                  // query rows per tile = TMEM lanes
constexpr int kKeys = 128;                  // key positions per key tile
constexpr int kCols = 128;                  // value columns of one CTA
constexpr int kThreads = 320;

template <int D>
struct DpGeo {
    static constexpr int HALVES = 2 * D / kCols;             // CTAs (a cluster) per pair and tile
    static constexpr int CHUNKS = D / 64;                    // 128-byte swizzle columns of Q, K
    static constexpr int COL_BYTES = kKeys * 128;            // one such column of 128 rows
    static constexpr int Q_BYTES = CHUNKS * COL_BYTES;       // Q of one map
    static constexpr int SLOT = 2 * COL_BYTES;               // 128 keys x 128 columns
    // loads of one key tile, one slot each: D = 64 the pair's K, its V; D = 128 K of map 0,
    // K of map 1, V of this CTA's head
    static constexpr int LOADS = D == 64 ? 2 : 3;
    static constexpr int BAR_BYTES = 256;
    static constexpr int XCH_BYTES = HALVES > 1 ? 2 * kRows * 4 : 0;   // sums from the other CTA
    static constexpr int FIXED = 1024 + 2 * Q_BYTES + BAR_BYTES + XCH_BYTES;
    static constexpr int SLOTS_FIT = (227 * 1024 - FIXED) / SLOT;
    static constexpr int SLOTS = SLOTS_FIT < 6 ? SLOTS_FIT : 6;
    static constexpr int SMEM = FIXED + SLOTS * SLOT;
    static constexpr uint32_t S_COL = 0, O_COL = 256, TMEM_COLS = 512;
    static_assert(D == 64 || D == 128, "head width 64 or 128");
    static_assert(SLOTS >= LOADS + 1 && SMEM <= 227 * 1024, "CTA does not fit an SM");
    static_assert(2 * SLOTS * 8 + 8 * 8 + 16 <= BAR_BYTES, "barrier area");
};

struct DpParams {
    int B, Hp, G, P, max_pages;
    int64_t window, n_pages, total_new;
    int pool_rows;                 // rows of one layer's 2-D pool view (pages * H * P)
    const __nv_bfloat16* q;        // [N][2 Hp G][D]
    const int32_t* cu_new;         // [B + 1]; nullptr: one request of single_n rows
    const int32_t* seq_lens;       // [B]; nullptr: single_t
    int single_n, single_t;
    const int32_t* tables;         // [B][max_pages]
    const float* lambda;
    const float* norm_weight;
    int normalise;
    float norm_eps, out_scale;
    float* out;                    // [N][Hp G][2 D]
    float scale_log2;              // log2(e) / sqrt(D)
    unsigned* dev_error;
};

__device__ __forceinline__ int cu_at(const DpParams& p, int b) {
    return p.cu_new ? __ldg(p.cu_new + b) : (b == 0 ? 0 : p.single_n);
}

__device__ __forceinline__ int len_at(const DpParams& p, int b) {
    return p.seq_lens ? __ldg(p.seq_lens + b) : p.single_t;
}

// One warp: the query tile that is number `item` of the call -- requests in order, each
// request's last (heaviest) tile first -- as (request, tile), or (-1, 0) past the last.
__device__ int2 find_tile(const DpParams& p, int item, bool report) {
    const int lane = threadIdx.x & 31, T = kRows / p.G;
    int before = 0;
    for (int base = 0; base < p.B; base += 32) {
        const int b = base + lane;
        int tiles = 0;
        if (b < p.B) {
            const int64_t c0 = cu_at(p, b), c1 = cu_at(p, b + 1), t = len_at(p, b);
            const bool ok = c0 >= 0 && c1 >= c0 && c1 <= p.total_new && t - (c1 - c0) >= 0 &&
                            t <= (int64_t)p.max_pages * p.P;
            if (ok) tiles = (int)((c1 - c0 + T - 1) / T);
            else if (report) atomicOr(p.dev_error, PKV_DEVERR_SEQ_LEN);
        }
        int incl = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        const int first = before + incl - tiles;
        const unsigned hit = __ballot_sync(0xffffffffu, item >= first && item < first + tiles);
        if (hit && !report) {
            const int src = __ffs(hit) - 1;
            const int f = __shfl_sync(0xffffffffu, first, src), n = __shfl_sync(0xffffffffu, tiles, src);
            return make_int2(base + src, n - 1 - (item - f));
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
    return make_int2(-1, 0);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
differential_prefill_kernel(const __grid_constant__ DpParams p, const __grid_constant__ CUtensorMap tmk,
                            const __grid_constant__ CUtensorMap tmv) {
    using M = DpGeo<D>;
    constexpr int HV = M::HALVES;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    unsigned char* Qs = sm;                                   // maps A, B
    unsigned char* ring = Qs + 2 * M::Q_BYTES;
    uint64_t* bars = reinterpret_cast<uint64_t*>(ring + M::SLOTS * M::SLOT);
    uint64_t* slot_full = bars;                  // per slot: copy landed
    uint64_t* slot_empty = bars + M::SLOTS;      //           MMAs reading it done
    uint64_t* s_full = bars + 2 * M::SLOTS;      // per map: S computed
    uint64_t* p_full = s_full + 2;               //          P written
    uint64_t* o_done = p_full + 2;               // last P V of both maps done
    uint64_t* q_ready = o_done + 1;
    uint64_t* drain = q_ready + 1;               // MMA completion on the abort path
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* tile_s = const_cast<int*>(abort_flag) + 1;           // request, tile
    float* peer_sums = reinterpret_cast<float*>(reinterpret_cast<unsigned char*>(bars) + M::BAR_BYTES);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // CTAs: item-major, then KV pair, then (cluster) half
    const int half = HV == 2 ? (int)(blockIdx.x & 1) : 0;
    const int unit = blockIdx.x / HV;
    const int item = unit / p.Hp, h = unit - item * p.Hp;
    if (warp == 0) {
        if (blockIdx.x == 0) find_tile(p, 0, true);
        const int2 it = find_tile(p, item, false);
        if (lane == 0) {
            tile_s[0] = it.x;
            tile_s[1] = it.y;
            *abort_flag = (*reinterpret_cast<volatile unsigned*>(p.dev_error) & PKV_DEVERR_TIMEOUT) ? 1 : 0;
        }
    }
    if (threadIdx.x == 32) {
        for (int s = 0; s < M::SLOTS; ++s) {
            mbar_init(&slot_full[s], 1);
            mbar_init(&slot_empty[s], 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(&s_full[x], 1);
            mbar_init(&p_full[x], 128);
        }
        mbar_init(o_done, 1);
        mbar_init(q_ready, 256);
        mbar_init(drain, 1);
        fence_mbar_init();
    }
    __syncthreads();
    const int b = tile_s[0];
    if (b < 0) return;                           // both CTAs of a cluster alike
    if (warp == 9) tmem_alloc(tmem_slot, M::TMEM_COLS);
    tc_fence_before();
    if constexpr (HV == 2) cluster_sync_all();   // the other CTA runs: its shared memory may be written
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    const int G = p.G, T = kRows / G;
    const int c0 = cu_at(p, b), n = cu_at(p, b + 1) - c0;
    const int t_b = len_at(p, b), L0 = t_b - n;
    const int i0 = tile_s[1] * T, i_end = min(n, i0 + T);
    const int pos_last = L0 + i_end - 1;
    const int lo_first = p.window > 0 && L0 + i0 + 1 > p.window ? (int)(L0 + i0 + 1 - p.window) : 0;
    const int kt0 = lo_first / kKeys, ntiles = pos_last / kKeys - kt0 + 1;

    // rows of the output and what the epilogue needs of them
    const int r = threadIdx.x & 127;                          // softmax warps: row = TMEM lane
    const int g = r % G, i = i0 + r / G;
    const bool valid = i < i_end;
    const int heads = p.Hp * G, head = h * G + g;
    const int64_t row_x = (int64_t)c0 + i;

    if (warp < 8) {
        // ------------------------------------------------------ softmax --
        const int x = warp >> 2;                              // map A (0) or B (1)
        unsigned char* Qx = Qs + x * M::Q_BYTES;
        {
            const uint4* src =
                reinterpret_cast<const uint4*>(p.q + ((row_x * heads + head) * 2 + x) * D);
#pragma unroll
            for (int u = 0; u < D / 8; ++u) {
                const uint4 v = valid ? __ldg(src + u) : make_uint4(0u, 0u, 0u, 0u);
                *reinterpret_cast<uint4*>(Qx + sw_off(r, u)) = v;
            }
        }
        fence_proxy_async_smem();
        mbar_arrive(q_ready);

        const int pos = L0 + i;
        const int hi = valid ? pos : -1;                      // keys lo .. hi
        const int lo = p.window > 0 && pos + 1 > p.window ? (int)(pos + 1 - p.window) : 0;
        const float c = p.scale_log2;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t t_s = lanes + M::S_COL + x * kKeys;
        const uint32_t t_o = lanes + M::O_COL + x * kCols;
        float m_used = -INFINITY, l = 0.f;
        bool ok = true;
        for (int j = 0; j < ntiles; ++j) {
            if (!pf_warp_wait(&s_full[x], j & 1, abort_flag, p.dev_error)) {
                ok = false;
                break;
            }
            tc_fence_after();
            // keys e_lo .. e_hi of the tile are this row's (none when e_lo > e_hi)
            const int k0 = (kt0 + j) * kKeys;
            const bool full = k0 >= lo && k0 + kKeys - 1 <= hi;
            const int e_lo = min(max(lo - k0, 0), kKeys), e_hi = max(min(hi - k0, kKeys - 1), -1);
            // the row maximum first (keys 64..127 read for it alone), then the weights of keys
            // 0..63 from registers and of 64..127 from a second read; P_hi and P_lo of a half
            // go over that half's S columns: 32 columns of pairs each
            const float2 c2 = make_float2(c, c);
            float m2[2] = {-INFINITY, -INFINITY};
            auto mask = [&](uint32_t* s, int first) {
                if (full) return;
#pragma unroll
                for (int e = 0; e < 64; ++e)
                    if (first + e < e_lo || first + e > e_hi) s[e] = 0xff800000u;
            };
            auto largest = [&](const uint32_t* s) {
#pragma unroll
                for (int e = 0; e < 64; e += 4) {
                    m2[0] = fmax3(m2[0], __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
                    m2[1] = fmax3(m2[1], __uint_as_float(s[e + 2]), __uint_as_float(s[e + 3]));
                }
            };
            {
                uint32_t sv[64];
                tmem_ld32(t_s + 64, sv);
                tmem_ld32(t_s + 96, sv + 32);
                tmem_wait_ld();
                mask(sv, 64);
                largest(sv);
            }
            uint32_t s0[64];
            tmem_ld32(t_s, s0);
            tmem_ld32(t_s + 32, s0 + 32);
            tmem_wait_ld();
            mask(s0, 0);
            largest(s0);
            const float mx = fmaxf(m2[0], m2[1]);
            float alpha = 1.f;
            if (mx > m_used && (m_used == -INFINITY || (mx - m_used) * c > 8.f)) {
                alpha = m_used == -INFINITY ? 0.f : ex2((m_used - mx) * c);
                m_used = mx;
                l *= alpha;
            }
            // S of this tile was committed after P V of the previous one, so that P V is
            // complete: O may be rescaled
            if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
                for (int cc = 0; cc < kCols / 32; ++cc) {
                    uint32_t ov[32];
                    tmem_ld32(t_o + cc * 32, ov);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                    tmem_st32(t_o + cc * 32, ov);
                }
                tmem_wait_st();
            }
            const float mb = m_used == -INFINITY ? 0.f : m_used * c;
            const float2 nmb2 = make_float2(-mb, -mb);
            float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            auto weights = [&](const uint32_t* sv, uint32_t col) {
                uint32_t phi[32], plo[32];
#pragma unroll
                for (int e = 0; e < 64; e += 2) {
                    const float2 xe = __ffma2_rn(
                        make_float2(__uint_as_float(sv[e]), __uint_as_float(sv[e + 1])), c2, nmb2);
                    const float2 pr = make_float2(ex2(xe.x), ex2(xe.y));
                    acc[(e >> 1) & 1] = __fadd2_rn(acc[(e >> 1) & 1], pr);
                    const __nv_bfloat162 hb = __floats2bfloat162_rn(pr.x, pr.y);
                    const __nv_bfloat162 lb =
                        __floats2bfloat162_rn(pr.x - __low2float(hb), pr.y - __high2float(hb));
                    phi[e >> 1] = *reinterpret_cast<const uint32_t*>(&hb);
                    plo[e >> 1] = *reinterpret_cast<const uint32_t*>(&lb);
                }
                tmem_st32(t_s + col, phi);
                tmem_st32(t_s + col + 32, plo);
            };
            weights(s0, 0);
            {
                uint32_t sv[64];
                tmem_ld32(t_s + 64, sv);
                tmem_ld32(t_s + 96, sv + 32);
                tmem_wait_ld();
                mask(sv, 64);
                weights(sv, 64);
            }
            tmem_wait_st();
            const float2 a = __fadd2_rn(acc[0], acc[1]);
            l += a.x + a.y;
            tc_fence_before();
            mbar_arrive(&p_full[x]);
        }
        if (ok) ok = pf_warp_wait(o_done, 0, abort_flag, p.dev_error);
        // Q is no longer read: its first bytes carry 1 / l and the partial sums of squares
        float* linv = reinterpret_cast<float*>(Qs);           // [2][128]
        float* sums = linv + 2 * kRows;                       // [2][128]
        if (ok) linv[x * kRows + r] = l > 0.f ? 1.f / l : 0.f;
        asm volatile("bar.sync 1, 256;" ::: "memory");
        float d[64];
        float sq = 0.f;
        if (ok) {
            tc_fence_after();
            const float i0v = linv[r];
            const float i1v = valid ? linv[kRows + r] * __ldg(p.lambda + head) : 0.f;
            const uint32_t oa = lanes + M::O_COL + x * 64, ob = oa + kCols;
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) {
                uint32_t va[32], vb[32];
                tmem_ld32(oa + cc * 32, va);
                tmem_ld32(ob + cc * 32, vb);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const float v = __uint_as_float(va[e]) * i0v - __uint_as_float(vb[e]) * i1v;
                    d[cc * 32 + e] = v;
                    sq = fmaf(v, v, sq);
                }
            }
        }
        if (p.normalise) {
            sums[x * kRows + r] = sq;
            if constexpr (HV == 2) {
                const uint32_t to = cluster_map(smem_u32(peer_sums + x * kRows + r), half ^ 1);
                st_cluster_f32(to, sq);
                cluster_sync_all();
            } else {
                asm volatile("bar.sync 1, 256;" ::: "memory");
            }
        }
        if (ok && valid) {
            float scale = p.out_scale;
            const float* nw = p.norm_weight ? p.norm_weight + half * kCols + x * 64 : nullptr;
            if (p.normalise) {
                // the halves' sums in the same order in both CTAs
                float t = sums[r] + sums[kRows + r];
                if constexpr (HV == 2) t += peer_sums[r] + peer_sums[kRows + r];
                scale *= 1.f / sqrtf(t / (2 * D) + p.norm_eps);
            }
            const bool weighted = p.normalise && nw != nullptr;
            float4* dst = reinterpret_cast<float4*>(p.out + (row_x * heads + head) * 2 * D + half * kCols +
                                                    x * 64);
#pragma unroll
            for (int e = 0; e < 64; e += 4) {
                float4 v = make_float4(d[e] * scale, d[e + 1] * scale, d[e + 2] * scale, d[e + 3] * scale);
                if (weighted) {
                    v.x *= __ldg(nw + e), v.y *= __ldg(nw + e + 1);
                    v.z *= __ldg(nw + e + 2), v.w *= __ldg(nw + e + 3);
                }
                dst[e / 4] = v;
            }
        }
    } else if (warp == 8) {
        // ----------------------------------------------------- producer --
        // load ld goes to slot ld % SLOTS once the MMAs that read the slot's previous tile
        // are done.  Lane gi < 8 looks up the page of the tile's 16-row group gi and issues
        // its boxes; groups outside lo_first .. pos_last read zeros (past the pool's rows).
        const uint64_t pol = l2_normal_policy();
        const int32_t* table = p.tables + (int64_t)b * p.max_pages;
        const int gi = lane & 7, H = 2 * p.Hp;
        pdl_wait_primary();                                   // the chunk's rows are stored
        int issued = 0;
        bool aborted = false;
        for (int j = 0; j < ntiles && !aborted; ++j) {
            const int key = (kt0 + j) * kKeys + 16 * gi;
            int y = p.pool_rows, y1 = p.pool_rows;            // this group's rows of head 2h, 2h + 1
            if (lane < 8 && key <= pos_last && key + 15 >= lo_first) {
                const int32_t page = __ldg(table + key / p.P);
                if (page >= 0 && page < p.n_pages) {
                    y = (int)(((int64_t)page * H + 2 * h) * p.P + key % p.P);
                    y1 = y + p.P;
                } else {
                    atomicOr(p.dev_error, PKV_DEVERR_PAGE_ID);
                }
            }
#pragma unroll
            for (int w = 0; w < M::LOADS; ++w) {
                const int ld = M::LOADS * j + w, s = ld % M::SLOTS;
                if (ld >= M::SLOTS && !pf_warp_wait(&slot_empty[s], ((ld / M::SLOTS) - 1) & 1,
                                                    abort_flag, p.dev_error)) {
                    aborted = true;
                    break;
                }
                if (lane == 0) mbar_arrive_expect_tx(&slot_full[s], M::SLOT);
                __syncwarp();
                if (lane < 8) {
                    unsigned char* dst = ring + s * M::SLOT + gi * 2048;
                    const bool value = w == M::LOADS - 1;
                    const CUtensorMap* map = value ? &tmv : &tmk;
#pragma unroll
                    for (int cc = 0; cc < 2; ++cc) {
                        // D = 64: one column of either head; D = 128: both columns of one head
                        const bool second = D == 64 ? cc == 1 : (value ? half == 1 : w == 1);
                        tma_load_2d(dst + cc * M::COL_BYTES, map, D == 64 ? 0 : cc * 64, second ? y1 : y,
                                    &slot_full[s], pol);
                    }
                }
                ++issued;
            }
        }
        if (lane == 0 && (aborted || *abort_flag)) {
            // let the copies in flight land before the CTA's shared memory goes away
            for (int ld = issued - M::SLOTS > 0 ? issued - M::SLOTS : 0; ld < issued; ++ld)
                mbar_wait_bounded(&slot_full[ld % M::SLOTS], (ld / M::SLOTS) & 1, kTcWaitLimitNs);
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------- MMA --
        constexpr uint32_t idS = idesc_bf16(kKeys, false);
        constexpr uint32_t idO = idesc_bf16(kCols, true);
        const uint32_t q_addr = smem_u32(Qs), ring_addr = smem_u32(ring);
        constexpr int NL = M::LOADS;
        auto wait_slot = [&](int ld) {
            return pf_warp_wait(&slot_full[ld % M::SLOTS], (ld / M::SLOTS) & 1, abort_flag,
                                p.dev_error);
        };
        auto ld_k = [&](int j, int x) { return NL * j + (NL == 3 ? x : 0); };
        auto ld_v = [&](int j) { return NL * j + NL - 1; };
        auto issue_s = [&](int j, int x) {
            const uint32_t k_addr = ring_addr + (ld_k(j, x) % M::SLOTS) * M::SLOT +
                                    (NL == 2 ? x * M::COL_BYTES : 0);
            const uint64_t da = sw128_desc(q_addr + x * M::Q_BYTES, 16, 1024);
            const uint64_t db = sw128_desc(k_addr, 16, 1024);
            const uint32_t d = tmem + M::S_COL + x * kKeys;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint64_t dk = (uint64_t)(((k >> 2) * M::COL_BYTES + (k & 3) * 32) >> 4);
                umma_bf16(d, da + dk, db + dk, idS, k > 0);
            }
            umma_commit(&s_full[x]);
            // the keys' slot is free once its last reader is done
            if (NL == 3 || x == 1) umma_commit(&slot_empty[ld_k(j, x) % M::SLOTS]);
        };
        auto issue_pv = [&](int j, int x) {
            // V is MN-major: two 64-column swizzle atoms COL_BYTES apart, 8-row groups 1024
            const uint64_t dv =
                sw128_desc(ring_addr + (ld_v(j) % M::SLOTS) * M::SLOT, M::COL_BYTES, 1024);
            // P in TMEM: keys 16k .. 16k+15 are P_hi columns 64(k/4) + 8(k%4) .. +7 and the
            // P_lo columns 32 further on
            const uint32_t pa = tmem + M::S_COL + x * kKeys;
            const uint32_t o = tmem + M::O_COL + x * kCols;
#pragma unroll
            for (int k = 0; k < kKeys / 16; ++k) {
                const uint64_t dvk = dv + (uint64_t)((k * 16 * 128) >> 4);
                const uint32_t ph = pa + (k >> 2) * 64 + (k & 3) * 8;
                umma_bf16_tmem_a(o, ph, dvk, idO, (j > 0 || k > 0) ? 1u : 0u);
                umma_bf16_tmem_a(o, ph + 32, dvk, idO, 1u);
            }
        };
        // rows [r0, r1) of tile j's values to zero: slots that no row of the CTA may read can
        // hold anything, and their weight is 0
        auto clear = [&](int j, int r0, int r1) {
            unsigned char* Vs = ring + (ld_v(j) % M::SLOTS) * M::SLOT;
            for (int idx = lane; idx < (r1 - r0) * 16; idx += 32) {
                const int row = r0 + idx / 16, piece = idx % 16;
                *reinterpret_cast<uint4*>(Vs + (piece >> 3) * M::COL_BYTES + row * 128 + (piece & 7) * 16) =
                    make_uint4(0u, 0u, 0u, 0u);
            }
        };
        bool ok = pf_warp_wait(q_ready, 0, abort_flag, p.dev_error) && wait_slot(ld_k(0, 0)) &&
                  (NL == 2 || wait_slot(ld_k(0, 1)));
        bool issued_any = false;
        if (ok) {
            tc_fence_after();
            if (lane == 0) {
                issue_s(0, 0);
                issue_s(0, 1);
            }
            issued_any = true;
            __syncwarp();
        }
        for (int j = 0; ok && j < ntiles; ++j) {
            const bool more = j + 1 < ntiles;
            if (!pf_warp_wait(&p_full[0], j & 1, abort_flag, p.dev_error) || !wait_slot(ld_v(j))) {
                ok = false;
                break;
            }
            const int k0 = (kt0 + j) * kKeys;
            const int last = !more ? ((pos_last - k0) / 16 + 1) * 16 : 0;    // rows copied, last tile
            const bool clear_end = !more && t_b - k0 < last;
            const bool clear_start = j == 0 && lo_first > k0;
            if (clear_end || clear_start) {
                if (clear_end) clear(j, t_b - k0, last);
                if (clear_start) clear(j, (lo_first - k0) / 16 * 16, lo_first - k0);
                fence_proxy_async_smem();
                __syncwarp();
            }
            tc_fence_after();
            if (lane == 0) issue_pv(j, 0);
            __syncwarp();
            if (more) {
                if (!wait_slot(ld_k(j + 1, 0))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (lane == 0) issue_s(j + 1, 0);
                __syncwarp();
            }
            if (!pf_warp_wait(&p_full[1], j & 1, abort_flag, p.dev_error) ||
                (more && NL == 3 && !wait_slot(ld_k(j + 1, 1)))) {
                ok = false;
                break;
            }
            tc_fence_after();
            if (lane == 0) {
                issue_pv(j, 1);
                umma_commit(&slot_empty[ld_v(j) % M::SLOTS]);
                if (more) issue_s(j + 1, 1);
                else umma_commit(o_done);
            }
            __syncwarp();
        }
        if (issued_any && *abort_flag) {
            // MMAs still in flight read shared memory and write TMEM: let them finish
            if (lane == 0) {
                umma_commit(drain);
                mbar_wait_bounded(drain, 0, kTcWaitLimitNs);
            }
            __syncwarp();
        }
    }
    if constexpr (HV == 2) {
        // producer and MMA warps join the softmax warps' exchange
        if (warp >= 8 && p.normalise) cluster_sync_all();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, M::TMEM_COLS);
    }
}

template <int D>
cudaError_t launch(const DpParams& p, const void* tmap_k, const void* tmap_v, cudaStream_t stream) {
    using M = DpGeo<D>;
    static bool done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !done[dev]) {
        e = cudaFuncSetAttribute(differential_prefill_kernel<D>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, M::SMEM);
        if (e != cudaSuccess) return e;
        if (dev < 64) done[dev] = true;
    }
    CUtensorMap tmk, tmv;
    std::memcpy(&tmk, tmap_k, sizeof tmk);
    std::memcpy(&tmv, tmap_v, sizeof tmv);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(differential_prefill_tiles(p.B, p.G, p.total_new) * p.Hp * M::HALVES));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = M::SMEM;
    cfg.stream = stream;
    // behind the append: the producer waits for it, everything before runs beside it
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (M::HALVES > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = M::HALVES;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, differential_prefill_kernel<D>, p, tmk, tmv);
}

}  // namespace

int64_t differential_prefill_tiles(int B, int G, int64_t total_new) { return total_new / (kRows / G) + B; }

bool differential_prefill_supported(int dtype, int D, int G) {
    return dtype == PKV_BF16 && (D == 64 || D == 128) && G >= 1 && G <= kRows && kRows % G == 0;
}

cudaError_t launch_differential_prefill(const DifferentialArgs& a, int batch, int64_t total_new,
                                        const int32_t* cu_new, const void* tmap_k, const void* tmap_v,
                                        cudaStream_t stream) {
    cudaError_t e = launch_differential_append(a, batch, total_new, cu_new, stream);
    if (e != cudaSuccess) return e;
    DpParams p{};
    p.B = batch;
    p.Hp = a.H / 2;
    p.G = a.G;
    p.P = a.P;
    p.max_pages = a.max_pages;
    p.window = a.window;
    p.n_pages = a.n_pages;
    p.total_new = total_new;
    p.pool_rows = (int)(a.n_pages * a.H * a.P);
    p.q = static_cast<const __nv_bfloat16*>(a.q);
    p.cu_new = cu_new;
    p.seq_lens = a.seq_lens;
    p.single_n = (int)total_new;
    p.single_t = a.single_t;
    p.tables = a.tables;
    p.lambda = a.diff.lambda;
    p.norm_weight = a.diff.norm_weight;
    p.normalise = a.diff.normalise;
    p.norm_eps = a.diff.norm_eps;
    p.out_scale = a.diff.out_scale;
    p.out = a.out;
    p.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)a.D));
    p.dev_error = a.dev_error;
    if (a.ev_before) cudaEventRecord(a.ev_before, stream);
    e = a.D == 64 ? launch<64>(p, tmap_k, tmap_v, stream) : launch<128>(p, tmap_k, tmap_v, stream);
    if (a.ev_after) cudaEventRecord(a.ev_after, stream);
    return e;
}

}  // namespace pkv
