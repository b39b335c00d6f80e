// Shared parts of the tensor-core attention kernels (tcgen05 + TMEM + TMA):
// tile geometry, barriers, the TMA producer of the K and V rings, the issue of
// the two products, and the online softmax of a key tile in registers.  Used
// by tree attention (attention_umma.cu) and chunk attention
// (chunk_attention.cu); the kernels' own files describe their use.
#pragma once

#include <cuda.h>

#include "sm100_ptx.cuh"
#include "tsd_common.cuh"

namespace tsd {

// A K or V cache, or a page pool, as the tensor map the kernels load from:
// [planes][rows][head_dim] bf16 in boxes of [1][box_rows][64] (a contiguous
// cache has planes = B * Hkv and rows = Lmax, a paged pool planes = num_pages *
// Hkv and rows = page_size).  False if the driver refuses it.
bool make_kv_map(CUtensorMap *m, const void *ptr, int head_dim, int rows, int planes, int box_rows);

namespace attn {

constexpr int BQ = 128;        // query rows per tile
constexpr uint32_t kSubQ = BQ * 128;         // Q [128 rows][64 bf16] sub-tile, 16 KB
constexpr uint32_t kOffQ = 0;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleThreshold = 8.0f;   // log2 units
constexpr float kLazyLimit = 18446744073709551616.0f;   // 2^64: headroom of a P tile sum
constexpr int kTableCache = 1024;   // block-table entries of a CTA's key range kept in smem

// Tile geometry of a kernel: keys per tile, K and V ring stages, TMEM
// columns; shared memory holds Q, the K ring, the V ring, the mbarriers.
template <int BN_, int NSK_, int NSV_, uint32_t TMEM_COLS, int HD_ = 128>
struct Geo {
    static constexpr int HD = HD_;                       // head dim, 64 or 128
    static constexpr uint32_t kTileQ = HD / 64 * kSubQ;  // Q tile [128][HD] bf16
    static constexpr int BN = BN_;                       // keys per tile
    static constexpr int NSK = NSK_;                     // K ring stages
    static constexpr int NSV = NSV_;                     // V ring stages
    static constexpr uint32_t kSub = BN * 128;           // [BN rows][64 bf16] sub-tile
    static constexpr uint32_t kTile = HD / 64 * kSub;    // [BN][HD] bf16
    static constexpr uint32_t kOffK = kOffQ + kTileQ;
    static constexpr uint32_t kOffV = kOffK + NSK * kTile;
    static constexpr uint32_t kOffBar = kOffV + NSV * kTile;
    static constexpr int kNumBars = 1 + 2 * NSK + 2 * NSV + 18;
    static constexpr uint32_t kOffMisc = kOffBar + 8 * kNumBars;
    static constexpr uint32_t kOffXchg = kOffMisc + 16;    // the softmax pairs' exchange slots
    static constexpr uint32_t kXchgBytes = 4 * 528;        // 4 x sizeof(PairXchg)
    static constexpr uint32_t kOffTable = kOffXchg + kXchgBytes;   // paged: block-table slice
    static constexpr uint32_t kSmemBytes = kOffTable + 4 * kTableCache + 1024;   // + alignment slack
    static constexpr uint32_t kTmemCols = TMEM_COLS;
};

// mbarrier addresses: q_full, k_full[NSK], k_empty[NSK], v_full[NSV],
// v_empty[NSV], s_full[4], p_full[4], o_ready[4], pair[4], drained (and one
// unused) -- consecutive 8-byte words.
template <class Gm>
struct Bars {
    static constexpr int NSK = Gm::NSK, NSV = Gm::NSV;
    uint32_t base;
    __device__ uint32_t q_full() const { return base; }
    __device__ uint32_t k_full(int s) const { return base + 8u * (1 + s); }
    __device__ uint32_t k_empty(int s) const { return base + 8u * (1 + NSK + s); }
    __device__ uint32_t v_full(int s) const { return base + 8u * (1 + 2 * NSK + s); }
    __device__ uint32_t v_empty(int s) const { return base + 8u * (1 + 2 * NSK + NSV + s); }
    __device__ uint32_t s_full(int i) const { return base + 8u * (1 + 2 * NSK + 2 * NSV + i); }
    __device__ uint32_t p_full(int i) const { return base + 8u * (5 + 2 * NSK + 2 * NSV + i); }
    __device__ uint32_t o_ready(int i) const { return base + 8u * (9 + 2 * NSK + 2 * NSV + i); }
    // the two softmax warps of TMEM lane quarter i meet here (two arrivals)
    __device__ uint32_t pair(int i) const { return base + 8u * (13 + 2 * NSK + 2 * NSV + i); }
    // only after a wait that gave up: every product issued is done
    __device__ uint32_t drained() const { return base + 8u * (17 + 2 * NSK + 2 * NSV); }
};

// A wait whose outcome is the same on every lane of the warp (the TMEM
// loads/stores that follow are warp-collective).
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int *abort)
{
    const bool ok = ptx::mbar_wait(bar, parity, abort);
    return __all_sync(0xffffffffu, ok);
}

// warp_wait for a phase that this warp already tested with ptx::mbar_test
// (`tested`, this lane's result) while it did other work: when every lane
// saw the phase complete the wait costs one vote.  The test must have been
// issued after the phase before it completed (else a stale phase passes).
__device__ __forceinline__ bool warp_wait_tested(uint32_t tested, uint32_t bar, uint32_t parity,
                                                 volatile int *abort)
{
    if (__all_sync(0xffffffffu, tested != 0u))
        return true;
    return warp_wait(bar, parity, abort);
}

// One arrival per warp: the lanes' prior writes (TMEM stores after their
// wait::st and fence, or shared-memory stores after their proxy fence) are
// ordered before lane 0's arrival by the warp barrier.
__device__ __forceinline__ void warp_arrive(uint32_t bar)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        ptx::mbar_arrive(bar);
}

// K-major, 128-byte-swizzled operand made of two [rows][64] sub-tiles `sub`
// bytes apart: the descriptor for the 16-wide slice kk of the 128-wide
// contraction dim is the base descriptor plus slice_off(kk, sub) (the
// address field is addr >> 4 and shared addresses stay below 256 KB, so
// adding to the packed word never carries out of it).
__device__ __forceinline__ uint64_t desc_kmajor(uint32_t tile)
{
    return ptx::smem_desc_sw128(tile, 16u, 1024u);
}
__device__ __forceinline__ uint64_t slice_off(int kk, uint32_t sub)
{
    return ((uint32_t)(kk >> 2) * sub + (uint32_t)(kk & 3) * 32u) >> 4;
}

// V tile as the MN-major B operand of O += P V (group kk of 16 keys at
// + kk * 2 KB); the two 64-wide halves of head_dim are `sub` bytes apart.
__device__ __forceinline__ uint64_t desc_v(uint32_t tile, uint32_t sub)
{
    return ptx::smem_desc_sw128(tile, sub, 1024u);
}

// Per-CTA set-up shared by both kernels: 1024-byte aligned carve-up of the
// dynamic shared memory, barrier initialisation, TMEM allocation (warp 1).
template <class Gm>
struct Setup {
    uint8_t *gbase;
    uint32_t base, sQ, sK, sV, tmem;
    Bars<Gm> bars;
    volatile int *abort_flag;
    volatile int *loads;   // K and V tiles the producer has issued, once it is done
};

template <class Gm>
__device__ __forceinline__ Setup<Gm> cta_setup(uint8_t *smem_raw, uint32_t q_arrivals,
                                               uint32_t p_arrivals)
{
    constexpr int NSK = Gm::NSK, NSV = Gm::NSV;
    constexpr uint32_t kOffMisc = Gm::kOffMisc;
    Setup<Gm> su;
    const uint32_t raw = ptx::smem_addr(smem_raw);
    su.base = (raw + 1023u) & ~1023u;
    su.gbase = smem_raw + (su.base - raw);
    su.sQ = su.base + kOffQ;
    su.sK = su.base + Gm::kOffK;
    su.sV = su.base + Gm::kOffV;
    su.bars = Bars<Gm>{su.base + Gm::kOffBar};
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(su.gbase + kOffMisc);
    su.abort_flag = reinterpret_cast<volatile int *>(su.gbase + kOffMisc + 4);
    su.loads = reinterpret_cast<volatile int *>(su.gbase + kOffMisc + 8);
    if (threadIdx.x == 0) {
        ptx::mbar_init(su.bars.q_full(), q_arrivals);
        for (int i = 0; i < NSK; ++i) {
            ptx::mbar_init(su.bars.k_full(i), 1);
            ptx::mbar_init(su.bars.k_empty(i), 1);
        }
        for (int i = 0; i < NSV; ++i) {
            ptx::mbar_init(su.bars.v_full(i), 1);
            ptx::mbar_init(su.bars.v_empty(i), 1);
        }
        for (int i = 0; i < 4; ++i) {
            ptx::mbar_init(su.bars.s_full(i), 1);
            ptx::mbar_init(su.bars.o_ready(i), 1);
            ptx::mbar_init(su.bars.p_full(i), p_arrivals);
            ptx::mbar_init(su.bars.pair(i), 2);
        }
        ptx::mbar_init(su.bars.drained(), 1);
        *su.abort_flag = 0;
        ptx::fence_barrier_init();
        ptx::fence_proxy_async_smem();
    }
    if ((threadIdx.x >> 5) == 1) {
        ptx::tmem_alloc(ptx::smem_addr((const void *)tmem_slot), Gm::kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    su.tmem = *tmem_slot;
    return su;
}

// After a wait that gave up: what this CTA still has in flight -- the products
// issued by this thread (the MMA warp's lane 0), and the last load of every ring
// slot -- lands before its shared memory and TMEM are given back.  Load i of a
// ring of n slots is phase i / n of slot i % n, and no later one was begun.  Each
// wait ends after 100 ms at the latest.
template <class Gm>
__device__ __forceinline__ void drain(const Setup<Gm> &su)
{
    const uint64_t t0 = ptx::global_timer_ns();
    auto landed = [&](uint32_t bar, int phase) {
        while (!ptx::mbar_try_wait(bar, phase & 1) &&
               ptx::global_timer_ns() - t0 <= 100000000ull) {
        }
    };
    ptx::mma_commit(su.bars.drained());
    landed(su.bars.drained(), 0);
    const int nk = su.loads[0], nv = su.loads[1];
    for (int i = max(nk - Gm::NSK, 0); i < nk; ++i)
        landed(su.bars.k_full(i % Gm::NSK), i / Gm::NSK);
    for (int i = max(nv - Gm::NSV, 0); i < nv; ++i)
        landed(su.bars.v_full(i % Gm::NSV), i / Gm::NSV);
}

template <class Gm>
__device__ __forceinline__ void cta_teardown(const Setup<Gm> &su, int32_t *dev_status)
{
    ptx::tc_fence_before();
    __syncthreads();
    const bool gave_up = *su.abort_flag != 0;
    if (gave_up && threadIdx.x == 0)
        flag(dev_status, TSD_DEV_TIMEOUT);
    if ((threadIdx.x >> 5) == 1) {
        if (gave_up) {
            if ((threadIdx.x & 31) == 0)
                drain(su);
            __syncwarp();
        }
        ptx::tc_fence_after();
        ptx::tmem_dealloc(su.tmem, Gm::kTmemCols);
    }
}

// The block-table entries of the pages a CTA's key range [kb, seq_end)
// touches, staged in shared memory by the producer warp before its first
// load (at most kTableCache of them; entries past that are read from global
// memory), so that a ring slot's reload does not wait for a global load.
struct PageCache {
    const int32_t *sm;   // entries blk0 .. blk0 + n - 1
    int blk0, n;
};

template <class Gm>
__device__ __forceinline__ PageCache stage_pages(const Setup<Gm> &su, const KvPages &pages, int b,
                                                 int kb, int seq_end, int lane)
{
    PageCache pc{reinterpret_cast<const int32_t *>(su.gbase + Gm::kOffTable), 0, 0};
    if (!pages.table || seq_end <= kb)
        return pc;
    pc.blk0 = kb >> pages.log2_page;
    pc.n = min(((seq_end - 1) >> pages.log2_page) - pc.blk0 + 1, kTableCache);
    int32_t *dst = reinterpret_cast<int32_t *>(su.gbase + Gm::kOffTable);
    for (int i = lane; i < pc.n; i += 32)
        dst[i] = pages.table[(size_t)b * pages.max_blocks + pc.blk0 + i];
    __syncwarp();
    return pc;
}

// The TMA loads of one [BN keys][128] K or V tile starting at logical key
// position pos0 into `dst` (two 64-column halves).  Contiguous cache: one box
// per half at (x, pos0, b * Hkv + hk).  Paged cache: one box per page the
// tile touches (box rows = min(BN, page_size); a box never straddles a page
// since both are powers of two and pos0 is a multiple of BN) at (x, row in
// page, page * Hkv + hk).  A box that starts at or beyond the sequence's end
// loads any valid page: those keys are masked and their V rows zeroed.
template <class Gm>
__device__ __forceinline__ void load_kv_tile(uint32_t dst, const CUtensorMap *tm, uint32_t bar,
                                             int pos0, int b, int hk, int Hkv,
                                             const KvPages &pages, const PageCache &pc,
                                             int seq_end, int32_t *dev_status)
{
    if (!pages.table) {
        ptx::tma_load_3d(dst, tm, 0, pos0, b * Hkv + hk, bar);
        if (Gm::HD == 128)
            ptx::tma_load_3d(dst + Gm::kSub, tm, 64, pos0, b * Hkv + hk, bar);
        return;
    }
    const int rows = min(Gm::BN, pages.page_size);
    for (int r0 = 0; r0 < Gm::BN; r0 += rows) {
        const int pos = pos0 + r0;
        int z = hk, y = 0;
        if (pos < seq_end) {
            const int blk = pos >> pages.log2_page, ci = blk - pc.blk0;
            const int page = (ci >= 0 && ci < pc.n)
                                 ? pc.sm[ci]
                                 : pages.table[(size_t)b * pages.max_blocks + blk];
            if (page < 0 || page >= pages.num_pages)
                flag(dev_status, TSD_DEV_BAD_PAGE);   // page 0 stands in
            else
                z = page * Hkv + hk;
            y = pos & (pages.page_size - 1);
        }
        ptx::tma_load_3d(dst + r0 * 128, tm, 0, y, z, bar);
        if (Gm::HD == 128)
            ptx::tma_load_3d(dst + Gm::kSub + r0 * 128, tm, 64, y, z, bar);
    }
}

// TMA producer (one lane).  Load order: K_0 .. K_{NSK-1} and V_0 .. V_{NSV-1}
// into the empty rings, then ... V_m, K_{m+L}, V_{m+1}, ... with L = NSK +
// LA - NSV, LA the MMA warp's QK lookahead (QK_{j+LA} is issued right after
// PV_j).  A ring slot is reused once the product that read it is complete,
// so V_m's slot frees with PV_{m-NSV} and K_{m+L}'s with QK_{m+L-NSK}, the
// QK issued right after that same PV: each reload is issued as soon as its
// slot is free, a K tile has about LA tile periods to land, and no V reload
// queues behind a K reload gated one product later.  Deadlock-free: the
// product a K wait needs reads V tiles below m only, and the one a V wait
// needs reads K tiles below the K index already issued.  NS_PROD = 0: the
// MMA warp commits every product to the rings' own empty barriers as well.
// NS_PROD = NS (the number of score buffers, equal to the K ring's depth):
// the producer waits on the products' own barriers instead -- QK_{i-NSK}
// completes on s_full[i % NS], PV_{j-NSV} on o_ready[(j - NSV) % NS] --
// which saves the MMA thread two commits per tile.  Either wait names a phase
// that cannot be stale or ahead: the phase before it was waited for by the
// previous reload of the same ring slot, and the phase after it needs K_i
// (or V_{j+1}), which this producer has not loaded yet.
template <class Gm, int NS_PROD>
__device__ __forceinline__ void produce_kv(const Setup<Gm> &su, const CUtensorMap *tmK,
                                           const CUtensorMap *tmV, int b, int hk, int Hkv,
                                           int kb, int ntiles, const KvPages &pages,
                                           const PageCache &pc, int seq_end,
                                           int32_t *dev_status)
{
    constexpr int NSK = Gm::NSK, NSV = Gm::NSV, BN = Gm::BN;
    constexpr uint32_t kTile = Gm::kTile;
    static_assert(NS_PROD == 0 || NS_PROD == NSK, "score buffers and K ring in step");
    // the QK lookahead: NS for the rows kernels, 2 for the key-split kernel
    constexpr int kLead = NSK + (NS_PROD ? NS_PROD : 2) - NSV;
    ptx::prefetch_tmap(tmK);
    ptx::prefetch_tmap(tmV);
    int i = 0, j = 0;   // next K tile, next V tile
    while (i < ntiles || j < ntiles) {
        const bool take_k =
            i < ntiles && (j >= ntiles || i < NSK || (j >= NSV && i <= j - 1 + kLead));
        if (take_k) {
            const int s = i % NSK;
            const uint32_t k_free = NS_PROD ? su.bars.s_full(s) : su.bars.k_empty(s);
            if (i >= NSK && !ptx::mbar_wait(k_free, ((i / NSK) - 1) & 1, su.abort_flag))
                break;
            ptx::mbar_arrive_expect_tx(su.bars.k_full(s), kTile);
            load_kv_tile<Gm>(su.sK + s * kTile, tmK, su.bars.k_full(s), kb + i * BN, b, hk, Hkv,
                             pages, pc, seq_end, dev_status);
            ++i;
        } else {
            const int s = j % NSV;
            if (j >= NSV) {
                const int r = j - NSV;   // PV_r read this slot last
                constexpr int NSP = NS_PROD ? NS_PROD : 1;
                // PV_r done: o_ready[r % NS] phase r / NS, or the ring's own
                // v_empty (which the MMA warp then commits as well)
                const bool ok =
                    !NS_PROD
                        ? ptx::mbar_wait(su.bars.v_empty(s), ((j / NSV) - 1) & 1, su.abort_flag)
                        : ptx::mbar_wait(su.bars.o_ready(r % NSP), (r / NSP) & 1,
                                         su.abort_flag);
                if (!ok)
                    break;
            }
            ptx::mbar_arrive_expect_tx(su.bars.v_full(s), kTile);
            load_kv_tile<Gm>(su.sV + s * kTile, tmV, su.bars.v_full(s), kb + j * BN, b, hk, Hkv,
                             pages, pc, seq_end, dev_status);
            ++j;
        }
    }
    su.loads[0] = i;
    su.loads[1] = j;
}

// MMA warp, S = Q K^T for key tile `t` into TMEM columns `col_s`.
template <class Gm, bool RING_COMMIT = true, bool COMMIT = true, bool WARP = true>
__device__ __forceinline__ void issue_qk(const Setup<Gm> &su, int lane, uint32_t col_s, int t,
                                         uint32_t s_full)
{
    constexpr uint32_t idesc = ptx::idesc_bf16(BQ, Gm::BN, false, false);
    const int st = t % Gm::NSK;
    if (lane == 0) {
        const uint64_t dq = desc_kmajor(su.sQ), dk = desc_kmajor(su.sK + st * Gm::kTile);
#pragma unroll
        for (int kk = 0; kk < Gm::HD / 16; ++kk)
            ptx::mma_ss(su.tmem + col_s, dq + slice_off(kk, kSubQ), dk + slice_off(kk, Gm::kSub),
                        idesc, kk > 0 ? 1u : 0u);
        if (COMMIT)
            ptx::mma_commit(s_full);
        if (COMMIT && RING_COMMIT)
            ptx::mma_commit(su.bars.k_empty(st));
    }
    if (WARP)
        __syncwarp();
}

// Zero the rows first_bad .. BN-1 of V ring slot vs (cache rows at or beyond
// P_b + T_b: masked keys whose P is 0, but 0 * NaN would not be), by one warp,
// then make the generic-proxy stores visible to the tensor cores.
template <class Gm>
__device__ __forceinline__ void zero_v_rows(const Setup<Gm> &su, int vs, int first_bad, int lane)
{
    uint8_t *vt = su.gbase + Gm::kOffV + vs * Gm::kTile;
    for (int row = max(first_bad, 0) + (lane >> 3); row < Gm::BN; row += 4) {
        const int c = lane & 7;
        *reinterpret_cast<uint4 *>(vt + row * 128 + c * 16) = make_uint4(0, 0, 0, 0);
        if (Gm::HD == 128)
            *reinterpret_cast<uint4 *>(vt + Gm::kSub + row * 128 + c * 16) = make_uint4(0, 0, 0, 0);
    }
    ptx::fence_proxy_async_smem();
    __syncwarp();
}

// MMA warp, O += P V for key tile `t` (P in TMEM columns col_p); zeroes the
// V rows at or beyond P_b + T_b first.  P_SPLIT: the packed P of keys
// 64 .. 127 sits 64 columns after that of keys 0 .. 63 (each softmax half
// writes into its own score columns) instead of right after it.
template <class Gm, bool RING_COMMIT = true, bool P_SPLIT = false, bool COMMIT = true,
          bool ZERO = true>
__device__ __forceinline__ void issue_pv(const Setup<Gm> &su, int lane, uint32_t col_p,
                                         uint32_t col_o, int t, bool accumulate, int first_bad,
                                         uint32_t o_ready)
{
    constexpr int BN = Gm::BN;
    constexpr uint32_t idesc = ptx::idesc_bf16(BQ, Gm::HD, false, true);
    const int vs = t % Gm::NSV;
    if (ZERO && first_bad < BN)
        zero_v_rows<Gm>(su, vs, first_bad, lane);
    ptx::tc_fence_after();
    if (lane == 0) {
        const uint64_t dv = desc_v(su.sV + vs * Gm::kTile, Gm::kSub);
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk) {
            const uint32_t pc = P_SPLIT ? (uint32_t)((kk >> 2) * 64 + (kk & 3) * 8)
                                        : (uint32_t)(kk * 8);
            ptx::mma_ts(su.tmem + col_o, su.tmem + col_p + pc,
                        dv + (uint64_t)((kk * 16u * 128u) >> 4), idesc,
                        (accumulate || kk > 0) ? 1u : 0u);
        }
        if (COMMIT && RING_COMMIT)
            ptx::mma_commit(su.bars.v_empty(vs));
        if (COMMIT)
            ptx::mma_commit(o_ready);
    }
    if (ZERO)
        __syncwarp();
}

// Q row `t` of the tile -> shared memory, 128-byte swizzled K-major layout;
// with SW = 2 warps per row, half hf loads the 64 dims hf*64 .. hf*64 + 63.
template <class Gm, int SW = 1>
__device__ __forceinline__ void load_q_row(const Setup<Gm> &su, const __nv_bfloat16 *__restrict__ q,
                                           bool row_ok, size_t q_off, int t, int hf = 0)
{
    uint8_t *dst = su.gbase + kOffQ;
    const uint4 *src = reinterpret_cast<const uint4 *>(q + q_off);
#pragma unroll
    for (int c = (SW == 2 ? hf * 8 : 0); c < (SW == 2 ? hf * 8 + 8 : Gm::HD / 8); ++c) {
        const uint4 x = row_ok ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
        const int sub = c >> 3, cc = c & 7;
        *reinterpret_cast<uint4 *>(dst + sub * kSubQ + t * 128 + ((cc ^ (t & 7)) * 16)) = x;
    }
    ptx::fence_proxy_async_smem();
}

// Rescale this row's O (TMEM columns col_o) by alpha.
template <int HD = 128>
__device__ __forceinline__ void rescale_o(uint32_t taddr_o, float alpha)
{
#pragma unroll
    for (int c = 0; c < HD / 32; ++c) {
        uint32_t o[32];
        ptx::tmem_ld32(taddr_o + c * 32, o);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 32; ++k)
            o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
        ptx::tmem_st32(taddr_o + c * 32, o);
    }
    ptx::tmem_wait_st();
}

// P = 2^(s * scale - m) for 64 scores (two 32-column chunks already loaded
// and masked), packed to bf16 into pk[32]; returns their sum.  The scaling
// and the sums run on packed fp32 pairs, the exponentials on MUFU.
__device__ __forceinline__ float exp_pack64(const uint32_t (&sa)[32], const uint32_t (&sb)[32],
                                            float scale_log2, float neg_m, uint32_t (&pk)[32])
{
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        float x0, x1, x2, x3;
        ptx::fma2_bc(x0, x1, __uint_as_float(sa[2 * k]), __uint_as_float(sa[2 * k + 1]),
                     scale_log2, neg_m);
        ptx::fma2_bc(x2, x3, __uint_as_float(sb[2 * k]), __uint_as_float(sb[2 * k + 1]),
                     scale_log2, neg_m);
        const float p0 = ptx::ex2(x0), p1 = ptx::ex2(x1), p2 = ptx::ex2(x2), p3 = ptx::ex2(x3);
        const int a = (k & 1) * 2;
        ptx::add2(acc[a], acc[a + 1], p0, p1);
        ptx::add2(acc[a], acc[a + 1], p2, p3);
        pk[k] = ptx::pack_bf16(p0, p1);
        pk[16 + k] = ptx::pack_bf16(p2, p3);
    }
    return (acc[0] + acc[1]) + (acc[2] + acc[3]);
}

// P for 32 scores (one 32-column chunk, loaded and masked), packed to bf16
// into pk[16]; returns their sum.
__device__ __forceinline__ float exp_pack32(const uint32_t (&sa)[32], float scale_log2,
                                            float neg_m, uint32_t (&pk)[16])
{
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        float x0, x1;
        ptx::fma2_bc(x0, x1, __uint_as_float(sa[2 * k]), __uint_as_float(sa[2 * k + 1]),
                     scale_log2, neg_m);
        const float p0 = ptx::ex2(x0), p1 = ptx::ex2(x1);
        const int a = (k & 1) * 2;
        ptx::add2(acc[a], acc[a + 1], p0, p1);
        pk[k] = ptx::pack_bf16(p0, p1);
    }
    return (acc[0] + acc[1]) + (acc[2] + acc[3]);
}

__device__ __forceinline__ void mask32(uint32_t (&s)[32], uint32_t bits)
{
#pragma unroll
    for (int k = 0; k < 32; ++k)
        s[k] = ((bits >> k) & 1u) ? s[k] : __float_as_uint(-INFINITY);
}

// Running maxima of 64 scores, 16 independent chains of 3-input maxima.
__device__ __forceinline__ void max32x2(const uint32_t (&sa)[32], const uint32_t (&sb)[32],
                                        float (&mx)[16])
{
#pragma unroll
    for (int k = 0; k < 32; ++k)
        mx[k & 15] = ptx::max3(mx[k & 15], __uint_as_float(sa[k]), __uint_as_float(sb[k]));
}

__device__ __forceinline__ float max16(const float (&mx)[16])
{
    float a = ptx::max3(mx[0], mx[1], mx[2]), b = ptx::max3(mx[3], mx[4], mx[5]);
    float c = ptx::max3(mx[6], mx[7], mx[8]), d = ptx::max3(mx[9], mx[10], mx[11]);
    float e = ptx::max3(mx[12], mx[13], mx[14]);
    return ptx::max3(ptx::max3(a, b, c), ptx::max3(d, e, mx[15]), -INFINITY);
}

// One key tile of the online softmax of the rows kernels, for this thread's
// query row: the BN scores in TMEM columns taddr_s are read into registers
// at once and masked where the tile reaches the tree or the range end.  P is
// written against the running max speculatively; the row max is only taken
// (and O rescaled) when some exponent may exceed the headroom -- the tile's
// sum above 2^64 or not finite, which always happens on a query tile's first
// key tile (m_run = -inf).  One exp loop, run a second time only by a warp
// that took the max.  `wait_prev` waits for the previous PV product before
// O is rescaled.  `vis` says which keys the row sees: vis.clear(pos0, BN),
// the same on every lane, that a whole tile is visible, vis.bits(pos) the
// visibility of the 32 keys from pos on.  Returns false on abort.
template <class Gm, class Vis, typename WaitPrev>
__device__ __forceinline__ bool softmax_rows_tile(uint32_t taddr_s, uint32_t taddr_o, int pos0,
                                                  const Vis &vis, float scale_log2, bool first, float &m_run,
                                                  float &l_run, WaitPrev wait_prev)
{
    constexpr int BN = Gm::BN;
    constexpr int NC = BN / 32;   // 32-column score chunks
    uint32_t sr[NC][32];
#pragma unroll
    for (int c = 0; c < NC; ++c)
        ptx::tmem_ld32(taddr_s + c * 32, sr[c]);
    ptx::tmem_wait_ld();
    if (!vis.clear(pos0, BN)) {   // only where the tree or the range end is
#pragma unroll
        for (int c = 0; c < NC; ++c)
            mask32(sr[c], vis.bits(pos0 + c * 32));
    }
    float lsum = 0.f;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        const float neg_m = m_run == -INFINITY ? 0.f : -m_run;
        lsum = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            uint32_t pk[16];
            lsum += exp_pack32(sr[c], scale_log2, neg_m, pk);
            ptx::tmem_st16(taddr_s + c * 16, pk);
        }
        const bool redo = !(lsum <= kLazyLimit) || m_run == -INFINITY;
        if (pass == 1 || !__any_sync(0xffffffffu, redo))
            break;
        float mx[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
            mx[i] = -INFINITY;
#pragma unroll
        for (int c = 0; c < NC; c += 2)
            max32x2(sr[c], sr[c + 1], mx);
        const float mt = max16(mx) * scale_log2;
        const bool need = mt > m_run + kRescaleThreshold;   // false if mt is -inf
        const float m_new = need ? mt : m_run;
        const float alpha = need ? ptx::ex2(m_run - m_new) : 1.f;   // 0 when m_run = -inf
        if (__any_sync(0xffffffffu, need) && !first) {
            // O holds the products of the earlier key tiles: wait for the last.
            if (!wait_prev())
                return false;
            ptx::tc_fence_after();
            rescale_o<Gm::HD>(taddr_o, alpha);
        }
        l_run *= alpha;
        m_run = m_new;
        ptx::tmem_wait_st();   // the speculative P is overwritten next pass
    }
    l_run += lsum;
    ptx::tmem_wait_st();
    return true;
}

// Final O row (TMEM) -> output row (bf16, normalised) or split partial (fp32).
template <int HD = 128>
__device__ __forceinline__ void write_row(uint32_t taddr_o, float inv, bool row_ok, size_t row,
                                          int nsplit, int split, size_t nrows,
                                          __nv_bfloat16 *__restrict__ out,
                                          float *__restrict__ part_o, int col0, int ncols)
{
    for (int c = 0; c < ncols; c += 32) {
        uint32_t o[32];
        ptx::tmem_ld32(taddr_o + c, o);
        ptx::tmem_wait_ld();
        if (!row_ok)
            continue;
        if (nsplit == 1) {
            uint4 *dst = reinterpret_cast<uint4 *>(out + row * HD + col0 + c);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                uint4 x;
                x.x = ptx::pack_bf16(__uint_as_float(o[8 * v + 0]) * inv,
                                     __uint_as_float(o[8 * v + 1]) * inv);
                x.y = ptx::pack_bf16(__uint_as_float(o[8 * v + 2]) * inv,
                                     __uint_as_float(o[8 * v + 3]) * inv);
                x.z = ptx::pack_bf16(__uint_as_float(o[8 * v + 4]) * inv,
                                     __uint_as_float(o[8 * v + 5]) * inv);
                x.w = ptx::pack_bf16(__uint_as_float(o[8 * v + 6]) * inv,
                                     __uint_as_float(o[8 * v + 7]) * inv);
                dst[v] = x;
            }
        } else {
            float4 *dst = reinterpret_cast<float4 *>(part_o + ((size_t)split * nrows + row) * HD +
                                                     col0 + c);
#pragma unroll
            for (int v = 0; v < 8; ++v)
                dst[v] = make_float4(__uint_as_float(o[4 * v]) * inv,
                                     __uint_as_float(o[4 * v + 1]) * inv,
                                     __uint_as_float(o[4 * v + 2]) * inv,
                                     __uint_as_float(o[4 * v + 3]) * inv);
        }
    }
}

}  // namespace attn
}  // namespace tsd
