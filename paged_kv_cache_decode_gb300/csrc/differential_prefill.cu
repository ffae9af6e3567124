// Differential attention of prefill chunks on the sm_103a tensor cores (bf16 pools of
// head width 64 or 128); differential.cu holds the formula and every other pool.
//
// Two launches per call: the chunk's rows are stored in their pages, then one cluster
// of two CTAs per (query tile, KV pair) attends them, one softmax map a CTA.
//
// Attention CTA.  A query tile is 128 rows: 128/G consecutive chunk tokens times the
// G query pairs that share one KV pair.  The CTA of map m takes the pair's queries
// q_(2i+m) against the keys of head 2p + m, and the values of both heads:
//     S  = Q_m K_m^T           tcgen05.mma, M=128 N=128 K=d_h, fp32 in TMEM
//     P  = 2^(c S - c base)    softmax warps: TMEM -> registers -> bf16 hi + lo
//                              back into TMEM over the S columns already read
//     O += P_hi V + P_lo V     tcgen05.mma, A = P from TMEM, M=128 N=2 d_h K=128
// with c = log2(e) / sqrt(d_h).  The softmax of a tile takes about 2000 cycles (two threads
// a row, 64 keys a thread), its MMAs 2600 (d_h = 128) or 1300 (64): something has to run
// beside it.
//   d_h = 128  O takes half of TMEM, so one CTA has the SM.  S has two buffers and a
//              group of eight softmax warps each: S of the next tile is there before a
//              tile's softmax ends, and the groups overlap.  They share one exponent base
//              per row, handed from tile to tile through shared memory as soon as a
//              tile's maximum is known.
//   d_h = 64   two CTAs share the SM, one S buffer and one group each.
// MMA order P V(j), S(j + buffers): MMAs of one thread run in issue order, so S overwrites
// P(j) only after P V(j) has read it.
//
// The base moves only when the maximum grows by more than 8 in log2 units (weights stay
// below 2^8; O / l uses the same base in both); the group that moves it waits for the
// previous P V and rescales O.
//
// At the end CTA m scales its O by 1 / l (map 1: lambda / l), sends the other CTA the
// d_h columns that that one finishes through distributed shared memory, and both take
// d = map 0 - map 1, its mean square over all 2 d_h columns, and store their half.
//
// Warp roles: 16 (8) softmax warps (they stage Q, write P, rescale O, store the output);
// producers, for K and for V (d_h = 64: one for both; copies of 16-row groups: a group
// never straddles a page); an MMA warp (allocates TMEM, one thread issues the MMAs and
// commits).  MMAs and copies are issued under elect.sync, V copies for both heads at
// once: in a branch on the lane number every operand is moved to uniform registers each
// time, at about 100 cycles an instruction, and that bounded the kernel (4 x 2048
// tokens, d_h = 128: 500 us with both maps in a CTA, 405 us like this, against 335).
//
// Bound: the tensor cores at d_h = 128 (3250 cycles a key tile for 2560 of MMAs at their
// nominal rate; beside that about 20000 cycles a CTA for its first copies and its
// output); at 64 the tensor cores and the exponentials about alike.
//
// Precision.  P V runs twice, for the hi and lo parts of the weights, which carry each to
// about 2^-17 (one bf16 part alone would be off by 2^-9; for a third TMEM has no columns
// at d_h = 128): 2e-6 to 3e-6 off the formula.  O accumulates inside the tensor cores,
// whose additions truncate, which adds up along the cache: 5e-6 at 4096 positions, 2e-5
// at 16384.
//
// Faults: bad lengths and page ids set bits of the device error word (a bad page
// reads as zeros); a wait that runs out sets the timeout bit and ends the CTA's work
// (it still meets the other CTA at the cluster barriers).

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

// Bounded wait of a whole warp; gives up early once another role of the CTA has given up.
__device__ __forceinline__ bool dp_warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                             unsigned* dev_error) {
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) {
        const uint64_t start = global_timer_ns();
        for (uint32_t i = 1; !ok; ++i) {
            ok = mbar_try_wait(bar, parity);
            if (!ok && (i & 63) == 0) {
                if (*abort_flag) break;
                if (global_timer_ns() - start > kTcWaitLimitNs) {
                    *abort_flag = 1;
                    atomicOr(dev_error, PKV_DEVERR_TIMEOUT);
                    break;
                }
            }
        }
    }
    return __all_sync(0xffffffffu, ok);
}

// 16 consecutive 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t x;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(x));
    return x != 0;
}

template <int D>
struct DpGeo {
    // S buffers = softmax groups of 128 SPLIT threads.  d_h = 128: one CTA fills an SM (O
    // alone takes half of TMEM) and hides a tile's softmax behind the other buffer's.
    // d_h = 64: two CTAs share an SM, one S buffer each -- a CTA's softmax, first copies
    // and output run beside the other's MMAs (458 us for 2 x ~4000 tokens with one CTA of
    // two buffers).
    static constexpr int CTAS = D == 64 ? 2 : 1;
    static constexpr int BUFS = D == 64 ? 1 : 2, SPLIT = 2;
    static constexpr int SOFTMAX = 128 * SPLIT * BUFS;       // softmax threads
    static constexpr int PRODUCERS = D == 64 ? 1 : 2;        // warps: K and V, or one each
    static constexpr int THREADS = SOFTMAX + 32 * PRODUCERS + 32;
    static constexpr int CHUNKS = D / 64;                    // 128-byte swizzle columns of Q, K
    static constexpr int COL_BYTES = kKeys * 128;            // one such column of 128 rows
    static constexpr int Q_BYTES = CHUNKS * COL_BYTES;       // Q, or the K of a tile
    static constexpr int V_BYTES = 2 * Q_BYTES;              // both heads' V of a tile
    static constexpr int V_GROUP = V_BYTES / 8;              // 16 positions of it
    static constexpr int STAGE = Q_BYTES + V_BYTES;
    static constexpr int BAR_BYTES = D == 64 ? 160 : 256;
    // either key half's maximum for each group and (two groups) the rows' exponent bases of
    // this tile and the last one, all bf16
    static constexpr int ROW_BYTES = (SPLIT * BUFS + (BUFS > 1 ? 2 : 0)) * kRows * 2;
    static constexpr int OUT_PITCH = D + 4;                  // floats of an output row in shared memory
    // (dynamic shared memory starts on a 1024-byte boundary; checked)
    static constexpr int FIXED = Q_BYTES + BAR_BYTES + ROW_BYTES;
    static constexpr int ROOM = CTAS == 2 ? 228 * 1024 / 2 - 1024 : 227 * 1024;
    static constexpr int STAGES = (ROOM - FIXED) / STAGE < 4 ? (ROOM - FIXED) / STAGE : 4;
    static constexpr int SMEM = FIXED + STAGES * STAGE;
    static constexpr uint32_t O_COL = BUFS * kKeys, TMEM_COLS = 512 / CTAS;
    static_assert(D == 64 || D == 128, "head width 64 or 128");
    static_assert(O_COL + 2 * D <= TMEM_COLS, "S buffers and O fill TMEM");
    static_assert(STAGES >= 2 && SMEM <= ROOM, "CTAs do not fit an SM");
    static_assert((4 * STAGES + 3 * BUFS + 3) * 8 + 28 <= BAR_BYTES, "barrier area");
    static_assert(STAGES * STAGE >= kRows * (D + OUT_PITCH) * 4, "the output goes over the ring");
    static_assert(kRows % (SOFTMAX / 32 * (128 / D)) == 0, "whole steps of the output rows");
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
// request's last (heaviest) tile first -- as (request, tile), or (-1, 0) past the last.  A
// lane looks at 8 requests at a time.  `report`: set the error bit of requests whose
// lengths do not fit, and of more tiles than the launch has room for (`items`).
__device__ int2 find_tile(const DpParams& p, int item, int items, bool report) {
    constexpr int PER = 8;
    const int lane = threadIdx.x & 31, T = kRows / p.G;
    const int per = p.B <= 32 ? 1 : PER;        // requests of a lane
    int64_t before = 0;
    for (int base = 0; base < p.B; base += 32 * per) {
        const int b0 = base + lane * per;
        int cu[PER + 1], len[PER], tiles[PER], sum = 0;
        cu[0] = b0 < p.B ? cu_at(p, b0) : 0;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            tiles[k] = 0;
            if (k >= per) continue;
            cu[k + 1] = b0 + k < p.B ? cu_at(p, b0 + k + 1) : 0;
            len[k] = b0 + k < p.B ? len_at(p, b0 + k) : 0;
        }
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            if (k >= per || b0 + k >= p.B) continue;
            const int64_t c0 = cu[k], c1 = cu[k + 1], t = len[k];
            const bool ok = c0 >= 0 && c1 >= c0 && c1 <= p.total_new && t - (c1 - c0) >= 0 &&
                            t <= (int64_t)p.max_pages * p.P;
            if (ok) tiles[k] = (int)((c1 - c0 + T - 1) / T);
            else if (report) atomicOr(p.dev_error, PKV_DEVERR_SEQ_LEN);
            sum += tiles[k];
        }
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        int64_t at = before + incl - sum;
        int2 found = make_int2(-1, 0);
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            if (k >= per) continue;
            if (item >= at && item < at + tiles[k]) found = make_int2(b0 + k, (int)(tiles[k] - 1 - (item - at)));
            at += tiles[k];
        }
        const unsigned hit = __ballot_sync(0xffffffffu, found.x >= 0);
        if (hit && !report) {
            const int src = __ffs(hit) - 1;
            return make_int2(__shfl_sync(0xffffffffu, found.x, src), __shfl_sync(0xffffffffu, found.y, src));
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
    // requests whose row ranges overlap
    if (report && lane == 0 && before > items) atomicOr(p.dev_error, PKV_DEVERR_SEQ_LEN);
    return make_int2(-1, 0);
}

template <int D>
__global__ void __launch_bounds__(DpGeo<D>::THREADS, DpGeo<D>::CTAS)
differential_prefill_kernel(const __grid_constant__ DpParams p, const __grid_constant__ CUtensorMap tmk,
                            const __grid_constant__ CUtensorMap tmv) {
    using M = DpGeo<D>;
    constexpr int NB = M::BUFS, NS = M::STAGES;
    extern __shared__ __align__(1024) unsigned char sm[];
    unsigned char* Qs = sm;
    unsigned char* ring = Qs + M::Q_BYTES;       // per stage: K, then V of both heads
    uint64_t* bars = reinterpret_cast<uint64_t*>(ring + NS * M::STAGE);
    uint64_t* k_full = bars;                     // per stage: K landed
    uint64_t* v_full = bars + NS;                //            V landed
    uint64_t* k_empty = bars + 2 * NS;           //            S that reads the K done
    uint64_t* v_empty = bars + 3 * NS;           //            P V that reads the V done
    uint64_t* s_full = bars + 4 * NS;            // per buffer: S computed
    uint64_t* p_full = s_full + NB;              //             P written
    uint64_t* pv_done = p_full + NB;             //             P V of the buffer's tile done
    uint64_t* o_done = pv_done + NB;             // the last P V done
    uint64_t* q_ready = o_done + 1;
    uint64_t* drain = q_ready + 1;               // MMA completion on the abort path
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int* tile_s = const_cast<int*>(abort_flag) + 1;           // request, tile, its cu_new, length
    __nv_bfloat16* row_max =
        reinterpret_cast<__nv_bfloat16*>(reinterpret_cast<unsigned char*>(bars) + M::BAR_BYTES);
                                                 // [group][half][128]
    __nv_bfloat16* base_s = row_max + M::SPLIT * NB * kRows;  // [2][128] (two groups)

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kProducer = M::SOFTMAX / 32, kMma = kProducer + M::PRODUCERS;
    // CTAs: item-major, then KV pair, then map (a cluster's two CTAs)
    const int map = blockIdx.x & 1;
    const int unit = blockIdx.x >> 1;
    const int item = unit / p.Hp, h = unit - item * p.Hp;
    if (warp == 0) {
        const int items = gridDim.x / 2 / p.Hp;
        if (blockIdx.x == 0) find_tile(p, 0, items, true);
        const int2 it = find_tile(p, item, items, false);
        if (lane == 0) {
            tile_s[0] = it.x;
            tile_s[1] = it.y;
            if (it.x >= 0) {
                tile_s[2] = cu_at(p, it.x);
                tile_s[3] = cu_at(p, it.x + 1);
                tile_s[4] = len_at(p, it.x);
            }
            *abort_flag = (*reinterpret_cast<volatile unsigned*>(p.dev_error) & PKV_DEVERR_TIMEOUT) ? 1 : 0;
        }
    }
    if (threadIdx.x == 32) {
        for (int s = 0; s < 4 * NS; ++s) mbar_init(&bars[s], 1);
        for (int b = 0; b < NB; ++b) {
            mbar_init(&s_full[b], 1);
            mbar_init(&p_full[b], 128 * M::SPLIT);
            mbar_init(&pv_done[b], 1);
        }
        mbar_init(o_done, 1);
        mbar_init(q_ready, M::SOFTMAX);
        mbar_init(drain, 1);
        fence_mbar_init();
    }
    __syncthreads();
    const int b = tile_s[0];
    if (b < 0) return;                           // both CTAs of a cluster alike
    if (smem_u32(sm) & 1023) {                   // the swizzle's pattern (alike in every CTA; reported
                                                 // as work that gave up)
        if (threadIdx.x == 0) atomicOr(p.dev_error, PKV_DEVERR_TIMEOUT);
        return;
    }
    if (warp == kMma) tmem_alloc(tmem_slot, M::TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    const int G = p.G, T = kRows / G;
    const int c0 = tile_s[2], n = tile_s[3] - c0;
    const int t_b = tile_s[4], L0 = t_b - n;
    const int i0 = tile_s[1] * T, i_end = min(n, i0 + T);
    const int pos_last = L0 + i_end - 1;
    const int lo_first = p.window > 0 && L0 + i0 + 1 > p.window ? (int)(L0 + i0 + 1 - p.window) : 0;
    const int kt0 = lo_first / kKeys, ntiles = pos_last / kKeys - kt0 + 1;

    if (warp < kProducer) {
        // ------------------------------------------------------ softmax --
        constexpr int SP = M::SPLIT, PARTS = SP * NB, KEYS = kKeys / SP;
        const int grp = warp / (4 * SP);                      // takes tiles grp, grp + NB, ...
        const int kh = SP == 2 ? (warp >> 2) & 1 : 0;         // keys KEYS kh .. + KEYS - 1 of them
        const int r = threadIdx.x & 127;                      // row of the tile = TMEM lane
        const int g = r % G, i = i0 + r / G;
        const bool valid = i < i_end;
        const int heads = p.Hp * G, head = h * G + g;
        const int64_t row_x = (int64_t)c0 + i;
        const int part = grp * SP + kh;
        const float weight = map ? __ldg(p.lambda + head) : 1.f;
        {
            const uint4* src =
                reinterpret_cast<const uint4*>(p.q + ((row_x * heads + head) * 2 + map) * D);
            uint4 v[(D / 8 + PARTS - 1) / PARTS];
#pragma unroll
            for (int u = 0; u * PARTS < D / 8; ++u) {
                const int piece = u * PARTS + part;
                v[u] = valid && piece < D / 8 ? __ldg(src + piece) : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int u = 0; u * PARTS < D / 8; ++u) {
                const int piece = u * PARTS + part;
                if (piece < D / 8) *reinterpret_cast<uint4*>(Qs + sw_off(r, piece)) = v[u];
            }
        }
        fence_proxy_async_smem();
        mbar_arrive(q_ready);

        const int pos = L0 + i;
        const int hi = valid ? pos : -1;                      // keys lo .. hi
        const int lo = p.window > 0 && pos + 1 > p.window ? (int)(pos + 1 - p.window) : 0;
        const float c = p.scale_log2;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t t_s = lanes + grp * kKeys + kh * KEYS;
        const uint32_t t_o = lanes + M::O_COL;
        // A named barrier for each group and row quarter: the SPLIT warps of tile j meet, and
        // those of tile j - 1 have arrived with its base (before tile 0: the last group).
        const int bar_in = 1 + grp * 4 + (warp & 3), bar_out = 1 + (grp + 1) % NB * 4 + (warp & 3);
        __nv_bfloat16* mine = row_max + part * kRows + r;
        const __nv_bfloat16* other = row_max + (part ^ 1) * kRows + r;
        if (NB > 1 && grp == NB - 1) {
            if (kh == 0) base_s[kRows + r] = __float2bfloat16_rn(-INFINITY);
            asm volatile("bar.arrive %0, %1;" ::"r"(bar_out), "n"(64 * SP) : "memory");
        }
        float m_used = -INFINITY, l = 0.f;
        bool ok = true;
        for (int j = grp; j < ntiles; j += NB) {
            if (!dp_warp_wait(&s_full[grp], (j / NB) & 1, abort_flag, p.dev_error)) ok = false;
            tc_fence_after();
            // keys e_lo .. e_hi of this half are this row's (none when e_lo > e_hi)
            const int k0 = (kt0 + j) * kKeys + kh * KEYS;
            const bool full = k0 >= lo && k0 + KEYS - 1 <= hi;
            const int e_lo = max(lo - k0, 0), e_hi = min(hi - k0, KEYS - 1);
            auto load = [&](uint32_t* sv, int chunk) {
                tmem_ld32(t_s + chunk * 32, sv);
                tmem_wait_ld();
                if (!full) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (chunk * 32 + e < e_lo || chunk * 32 + e > e_hi) sv[e] = 0xff800000u;
                }
            };
            // S is read twice, 32 columns at a time: for the maximum, then for the weights
            float m2[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int chunk = 0; chunk < KEYS / 32; ++chunk) {
                uint32_t sv[32];
                load(sv, chunk);
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    m2[0] = fmax3(m2[0], __uint_as_float(sv[e]), __uint_as_float(sv[e + 1]));
                    m2[1] = fmax3(m2[1], __uint_as_float(sv[e + 2]), __uint_as_float(sv[e + 3]));
                }
            }
            // Maxima and bases are bf16: any base near the maximum serves, as long as all warps
            // of a row take the same.  (The other warp has read `mine` of this group's last
            // tile before it arrived on p_full, without which this S would not be there.)
            const __nv_bfloat16 own = __float2bfloat16_rn(fmaxf(m2[0], m2[1]));
            *mine = own;
            constexpr int kMeet = NB > 1 ? 64 * SP : 32 * SP;
            asm volatile("bar.sync %0, %1;" ::"r"(bar_in), "n"(kMeet) : "memory");
            const float mx = fmaxf(__bfloat162float(own), __bfloat162float(*other));
            // the base of tile j - 1: from the other group's warps, or this thread's own
            const float before = NB > 1 ? __bfloat162float(base_s[((j + 1) & 1) * kRows + r]) : m_used;
            const float base =
                mx > before && (before == -INFINITY || (mx - before) * c > 8.f) ? mx : before;
            if (NB > 1) {
                if (kh == 0) base_s[(j & 1) * kRows + r] = __float2bfloat16_rn(base);
                if (j + 1 < ntiles) asm volatile("bar.arrive %0, %1;" ::"r"(bar_out), "n"(kMeet) : "memory");
            }
            // l is this thread's share, at the base of its last tile
            if (base != m_used) l *= m_used == -INFINITY ? 0.f : ex2((m_used - base) * c);
            m_used = base;
            if (j > 0 && __any_sync(0xffffffffu, base != before)) {
                // O was summed at the old base; it is whole once P V of tile j - 1 is done
                const float alpha = base == before ? 1.f : before == -INFINITY ? 0.f : ex2((before - base) * c);
                if (!dp_warp_wait(&pv_done[(j - 1) % NB], ((j - 1) / NB) & 1, abort_flag, p.dev_error))
                    ok = false;
                tc_fence_after();
#pragma unroll 1
                for (int cc = 0; cc < 2 * D / SP / 32; ++cc) {        // its share of O's columns
                    const uint32_t at = t_o + kh * (2 * D / SP) + cc * 32;
                    uint32_t ov[32];
                    tmem_ld32(at, ov);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                    tmem_st32(at, ov);
                }
                tmem_wait_st();
            }
            const float mb = base == -INFINITY ? 0.f : base * c;
            const float2 c2 = make_float2(c, c), nmb2 = make_float2(-mb, -mb), minus = make_float2(-1.f, -1.f);
            float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int chunk = 0; chunk < KEYS / 32; ++chunk) {
                uint32_t sv[32];
                load(sv, chunk);
#pragma unroll
                for (int k = 0; k < 32; k += 16) {
                    uint32_t pv[16];                          // 8 P_hi pairs, 8 P_lo pairs
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const float2 xe = __ffma2_rn(
                            make_float2(__uint_as_float(sv[k + e]), __uint_as_float(sv[k + e + 1])), c2, nmb2);
                        const float2 pr = make_float2(ex2(xe.x), ex2(xe.y));
                        acc[(e >> 1) & 1] = __fadd2_rn(acc[(e >> 1) & 1], pr);
                        const __nv_bfloat162 hb = __floats2bfloat162_rn(pr.x, pr.y);
                        const float2 rest = __ffma2_rn(__bfloat1622float2(hb), minus, pr);   // exact
                        const __nv_bfloat162 lb = __floats2bfloat162_rn(rest.x, rest.y);
                        pv[e >> 1] = *reinterpret_cast<const uint32_t*>(&hb);
                        pv[8 + (e >> 1)] = *reinterpret_cast<const uint32_t*>(&lb);
                    }
                    tmem_st16(t_s + chunk * 32 + k, pv);
                }
            }
            tmem_wait_st();
            const float2 a = __fadd2_rn(acc[0], acc[1]);
            l += a.x + a.y;
            tc_fence_before();
            mbar_arrive(&p_full[grp]);
        }
        if (ok) ok = dp_warp_wait(o_done, 0, abort_flag, p.dev_error);
        // Q is no longer read: it carries each thread's base and sum, and sums of squares
        float* gm = reinterpret_cast<float*>(Qs);             // [part][128]
        float* gl = gm + PARTS * kRows;
        float* sums = gl + PARTS * kRows;                     // [part][128]
        float* peer_sums = sums + PARTS * kRows;              // [128], from the other CTA
        if (ok) {
            gm[part * kRows + r] = m_used;
            gl[part * kRows + r] = l;
        }
        asm volatile("bar.sync 15, %0;" ::"n"(M::SOFTMAX) : "memory");
        float scale = 0.f;
        if (ok) {
            tc_fence_after();
            float top = -INFINITY, lt = 0.f;
#pragma unroll
            for (int k = 0; k < PARTS; ++k) top = fmaxf(top, gm[k * kRows + r]);
#pragma unroll
            for (int k = 0; k < PARTS; ++k) {
                const float mk = gm[k * kRows + r];
                lt += mk == -INFINITY ? 0.f : gl[k * kRows + r] * ex2((mk - top) * c);
            }
            if (valid && lt > 0.f) scale = weight / lt;
        }
        cluster_sync_all();                                   // both CTAs' Q and rings are free
        // Each CTA finishes the d_h columns of head 2h + map: what it has of the others goes to
        // the other CTA, as [column][row] (lanes side by side: stores of a lane's own 16 bytes
        // took distributed shared memory 2.5 times as long)
        constexpr int COLS = D / PARTS;                       // columns a thread sends, and finishes
        const int col = part * COLS;
        const uint32_t inbox = cluster_map(smem_u32(ring), map ^ 1);
#pragma unroll
        for (int cc = 0; cc < COLS; cc += 16) {
            uint32_t v[16];
            tmem_ld16(t_o + (map ^ 1) * D + col + cc, v);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e)
                st_cluster_f32(inbox + ((col + cc + e) * kRows + r) * 4, __uint_as_float(v[e]) * scale);
        }
        float d[COLS];
#pragma unroll
        for (int cc = 0; cc < COLS; cc += 16)
            tmem_ld16(t_o + map * D + col + cc, reinterpret_cast<uint32_t*>(d) + cc);
        tmem_wait_ld();
        cluster_sync_all();
        float sq = 0.f;
        {
            const float* in = reinterpret_cast<const float*>(ring) + col * kRows + r;
            const float f = map ? -scale : scale, g0 = map ? 1.f : -1.f;      // map 0 less map 1
#pragma unroll
            for (int e = 0; e < COLS; ++e) {
                d[e] = fmaf(g0, in[e * kRows], d[e] * f);
                sq = fmaf(d[e], d[e], sq);
            }
        }
        // the rows to shared memory, [row][OUT_PITCH], to be stored a row a warp
        float* rows = reinterpret_cast<float*>(ring) + D * kRows;
#pragma unroll
        for (int e = 0; e < COLS; e += 4)
            *reinterpret_cast<float4*>(rows + r * M::OUT_PITCH + col + e) =
                make_float4(d[e], d[e + 1], d[e + 2], d[e + 3]);
        sums[part * kRows + r] = sq;
        asm volatile("bar.sync 15, %0;" ::"n"(M::SOFTMAX) : "memory");
        float total = 0.f;
#pragma unroll
        for (int k = 0; k < PARTS; ++k) total += sums[k * kRows + r];
        if (p.normalise) {
            if (part == 0) st_cluster_f32(cluster_map(smem_u32(peer_sums + r), map ^ 1), total);
            cluster_sync_all();
        }
        if (part == 0) {
            float f = p.out_scale;
            // (both CTAs add the same two numbers)
            if (p.normalise) f *= 1.f / sqrtf((total + peer_sums[r]) / (2 * D) + p.norm_eps);
            gm[r] = f;
            reinterpret_cast<int*>(gl)[r] =                   // output row of this tile row, or -1
                ok && valid ? (i - i0) * heads + head : -1;
        }
        asm volatile("bar.sync 15, %0;" ::"n"(M::SOFTMAX) : "memory");
        // a lane 4 columns of a row, LPR lanes a row
        constexpr int LPR = D / 4, RPW = 32 / LPR, STEP = M::SOFTMAX / 32 * RPW;
        const int at = lane % LPR * 4;
        float4 nw = make_float4(1.f, 1.f, 1.f, 1.f);
        if (p.normalise && p.norm_weight) {
            const float* w = p.norm_weight + map * D + at;
            nw = make_float4(__ldg(w), __ldg(w + 1), __ldg(w + 2), __ldg(w + 3));
        }
        float* dst = p.out + ((int64_t)c0 + i0) * heads * 2 * D + map * D + at;
#pragma unroll
        for (int k = 0; k < kRows / STEP; ++k) {
            const int rr = warp * RPW + lane / LPR + k * STEP;
            const int row = reinterpret_cast<const int*>(gl)[rr];
            const float f = gm[rr];
            const float4 x = *reinterpret_cast<const float4*>(rows + rr * M::OUT_PITCH + at);
            if (row >= 0)
                *reinterpret_cast<float4*>(dst + (int64_t)row * 2 * D) =
                    make_float4(x.x * f * nw.x, x.y * f * nw.y, x.z * f * nw.z, x.w * f * nw.w);
        }
    } else if (warp < kMma) {
        // ---------------------------------------------------- producers --
        // (d_h = 128: a warp for K, one for V.)  Tile j goes to stage j % NS once the MMAs that read the
        // stage's last tile are done.  Lane gi < 8 looks up the page of the tile's 16-row
        // group gi (groups outside lo_first .. pos_last read zeros: a place past the pool);
        // one lane issues the copies, K a box of 16 rows x 64 columns at a time, V one of
        // 16 rows x both heads (issued by eight lanes box by box, the copies of a tile took
        // longer than its MMAs).
        const uint64_t pol = l2_normal_policy();
        const int32_t* table = p.tables + (int64_t)b * p.max_pages;
        const int gi = lane & 7, H = 2 * p.Hp;
        pdl_wait_primary();                                   // the chunk's rows are stored
        // this lane's table entry for tile j, or -1 where nothing is to be read; looked at a
        // tile later, so that no copy waits for the load
        auto lookup = [&](int j) {
            const int key = (kt0 + j) * kKeys + 16 * gi;
            const bool used = j < ntiles && lane < 8 && key <= pos_last && key + 15 >= lo_first;
            return used ? __ldg(table + key / p.P) : -2;
        };
        const bool keys = M::PRODUCERS == 1 || warp == kProducer, values = M::PRODUCERS == 1 || !keys;
        int k_issued = 0, v_issued = 0;
        int32_t next = lookup(0);
        for (int j = 0; j < ntiles; ++j) {
            const int s = j % NS;
            int32_t page = next;
            next = lookup(j + 1);
            if (page != -2 && (page < 0 || page >= p.n_pages)) {
                atomicOr(p.dev_error, PKV_DEVERR_PAGE_ID);
                page = -2;
            }
            const int slot = ((kt0 + j) * kKeys + 16 * gi) % p.P;
            // K: the group's row of the 2-D pool; V: its page
            const int row = page < 0 ? p.pool_rows : (int)(((int64_t)page * H + 2 * h + map) * p.P + slot);
            if (page < 0) page = (int32_t)p.n_pages;
            int rows[8], pages[8], slots[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                rows[k] = __shfl_sync(0xffffffffu, row, k);
                pages[k] = __shfl_sync(0xffffffffu, page, k);
                slots[k] = __shfl_sync(0xffffffffu, slot, k);
            }
            unsigned char* dst = ring + s * M::STAGE;
            const uint32_t past = ((j / NS) - 1) & 1;
            if (keys) {
                if (j >= NS && !dp_warp_wait(&k_empty[s], past, abort_flag, p.dev_error)) break;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&k_full[s], M::Q_BYTES);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
#pragma unroll
                        for (int cc = 0; cc < M::CHUNKS; ++cc)
                            tma_load_2d(dst + cc * M::COL_BYTES + k * 2048, &tmk, cc * 64, rows[k], &k_full[s],
                                        pol);
                }
                __syncwarp();
                ++k_issued;
            }
            if (values) {
                if (j >= NS && !dp_warp_wait(&v_empty[s], past, abort_flag, p.dev_error)) break;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&v_full[s], M::V_BYTES);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        tma_load_5d(dst + M::Q_BYTES + k * M::V_GROUP, &tmv, 0, slots[k], 0, 2 * h, pages[k],
                                    &v_full[s], pol);
                }
                __syncwarp();
                ++v_issued;
            }
        }
        if (lane == 0 && (k_issued + v_issued < ((int)keys + (int)values) * ntiles || *abort_flag)) {
            // let the copies in flight land before the CTA's shared memory goes away
            for (int j = max(k_issued - NS, 0); j < k_issued; ++j)
                mbar_wait_bounded(&k_full[j % NS], (j / NS) & 1, kTcWaitLimitNs);
            for (int j = max(v_issued - NS, 0); j < v_issued; ++j)
                mbar_wait_bounded(&v_full[j % NS], (j / NS) & 1, kTcWaitLimitNs);
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------- MMA --
        constexpr uint32_t idS = idesc_bf16(kKeys, false);
        constexpr uint32_t idO = idesc_bf16(2 * D, true);
        // a CTA that has all 512 columns has them from column 0: constants
        const uint32_t tS = M::CTAS == 1 ? 0 : tmem, tO = tS + M::O_COL;
        const uint32_t q_addr = smem_u32(Qs), ring_addr = smem_u32(ring);
        auto wait = [&](uint64_t* bar, int phase) {
            return dp_warp_wait(bar, phase & 1, abort_flag, p.dev_error);
        };
        auto issue_s = [&](int j) {
            const uint64_t da = sw128_desc(q_addr, 16, 1024);
            const uint64_t db = sw128_desc(ring_addr + (j % NS) * M::STAGE, 16, 1024);
            const uint32_t d = tS + (j % NB) * kKeys;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint64_t dk = (uint64_t)(((k >> 2) * M::COL_BYTES + (k & 3) * 32) >> 4);
                umma_bf16(d, da + dk, db + dk, idS, k > 0);
            }
            umma_commit(&s_full[j % NB]);
            umma_commit(&k_empty[j % NS]);
        };
        auto issue_pv = [&](int j) {
            // V is MN-major: a k-step is one 16-row group, its 64-column swizzle atoms 2048
            // bytes apart, 8-row groups 1024
            const uint64_t dv = sw128_desc(ring_addr + (j % NS) * M::STAGE + M::Q_BYTES, 2048, 1024);
            // P in TMEM: keys 16k .. 16k+15 are P_hi columns 16k .. +7 and the P_lo columns
            // behind them
            const uint32_t pa = tS + (j % NB) * kKeys;
#pragma unroll
            for (int k = 0; k < kKeys / 16; ++k) {
                const uint64_t dvk = dv + (uint64_t)((k * M::V_GROUP) >> 4);
                const uint32_t ph = pa + k * 16;
                umma_bf16_tmem_a(tO, ph, dvk, idO, (j > 0 || k > 0) ? 1u : 0u);
                umma_bf16_tmem_a(tO, ph + 8, dvk, idO, 1u);
            }
            umma_commit(&pv_done[j % NB]);
            umma_commit(&v_empty[j % NS]);
        };
        // rows [r0, r1) of tile j's values to zero: slots that no row of the CTA may read can
        // hold anything, and their weight is 0
        auto clear = [&](int j, int r0, int r1) {
            unsigned char* Vs = ring + (j % NS) * M::STAGE + M::Q_BYTES;
            constexpr int PER = 2 * M::CHUNKS * 8;            // 16-byte pieces of a row
            for (int idx = lane; idx < (r1 - r0) * PER; idx += 32) {
                const int row = r0 + idx / PER, piece = idx % PER;
                *reinterpret_cast<uint4*>(Vs + (row >> 4) * M::V_GROUP + (piece >> 3) * 2048 + (row & 15) * 128 +
                                          (piece & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
        };
        bool ok = wait(q_ready, 0);
        bool issued_any = false;
        for (int j = 0; ok && j < NB && j < ntiles; ++j) {
            if (!(ok = wait(&k_full[j % NS], j / NS))) break;
            tc_fence_after();
            if (elect_one()) issue_s(j);
            __syncwarp();
            issued_any = true;
        }
        for (int j = 0; ok && j < ntiles; ++j) {
            // copies first: they are there early, P comes last
            const bool end = j + 1 == ntiles;
            const int k0 = (kt0 + j) * kKeys;
            if (!wait(&v_full[j % NS], j / NS) ||
                (j + NB < ntiles && !wait(&k_full[(j + NB) % NS], (j + NB) / NS))) {
                ok = false;
                break;
            }
            const int last = end ? ((pos_last - k0) / 16 + 1) * 16 : 0;      // rows copied, last tile
            const bool clear_end = end && t_b - k0 < last;
            const bool clear_start = j == 0 && lo_first > k0;
            if (clear_end || clear_start) {
                if (clear_end) clear(j, t_b - k0, last);
                if (clear_start) clear(j, (lo_first - k0) / 16 * 16, lo_first - k0);
                fence_proxy_async_smem();
                __syncwarp();
            }
            if (!wait(&p_full[j % NB], j / NB)) {
                ok = false;
                break;
            }
            tc_fence_after();
            if (elect_one()) {
                issue_pv(j);
                if (end) umma_commit(o_done);
                if (j + NB < ntiles) issue_s(j + NB);
            }
            __syncwarp();
        }
        if (issued_any && *abort_flag) {
            // MMAs still in flight read shared memory and write TMEM: let them finish
            if (elect_one()) {
                umma_commit(drain);
                mbar_wait_bounded(drain, 0, kTcWaitLimitNs);
            }
            __syncwarp();
        }
    }
    if (warp >= kProducer) {
        // producer and MMA warps join the softmax warps' cluster barriers
        cluster_sync_all();
        cluster_sync_all();
        if (p.normalise) cluster_sync_all();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kMma) {
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
    cfg.gridDim = dim3((unsigned)(differential_prefill_tiles(p.B, p.G, p.total_new) * p.Hp * 2));
    cfg.blockDim = dim3(M::THREADS);
    cfg.dynamicSmemBytes = M::SMEM;
    cfg.stream = stream;
    // behind the append: the producer waits for it, everything before runs beside it
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    attr[1].id = cudaLaunchAttributeClusterDimension;         // the two maps
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
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
