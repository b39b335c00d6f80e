// Causal attention of a chunk of new tokens over a paged KV cache.
//
// Sequence b has T_b new tokens behind P_b cached ones; their K and V rows
// are in the cache already.  Token t, query head h:
//     out[b][t][h] = sum_{j <= P_b + t} softmax_j(scale q . k_j) v_j
// over KV head h / G (G = Hq / Hkv).  One token per sequence (T = 1) is the
// decode step, thousands a prompt.
//
// The rows of one KV head are packed r = t * G + g, so a block of BQ rows
// reads each key once for all the query heads that share it, and its keys end
// at the last row's position.  Two kernels:
//   * bf16: tcgen05 products with S and O in TMEM (attn_umma.cuh), 64-key tiles
//     at two CTAs per SM: where the KV stream is the bound they keep twice the
//     loads in flight, and in prompts one's products run beside the other's
//     exponentials and its start and end (128-key tiles at one CTA per SM: 697
//     against 611 us for 2048 tokens on 4096, 64/8 heads, two sequences; the
//     same when the power limit paces both).  head_dim 64 or 128.
//   * fp32: FMA tiles in registers (the tensor cores have no fp32 product).
//
// Work is divided in one of two ways.
//   * Blocks: one CTA per (block, KV head, sequence), those with the most keys
//     first.  Always taken from some number of blocks on (`chunk_plan`).
//   * Ranges: the key tiles of all blocks in a row are cut into as many equal
//     ranges as there are CTA slots, so every CTA streams the same number of
//     tiles whatever the sequences' lengths, and its rings keep loading over the
//     border from one block to the next.  A block that a border cuts leaves
//     partial results, which a second kernel joins by their running maxima and
//     sums.
// With few blocks the lengths decide, and they are on the device: each warp of
// each CTA sums and scans the blocks of one KV head (no extra launch; `chunk_plan`
// limits those of all heads together to 591 in bf16 and 1183 in fp32 on 148 SMs),
// estimates both ways (`prefer_ranges`) and finds its share of the better one.
// (Ranges against pieces of blocks, one CTA each: 63 against 75 to 98 us for 32
// sequences of 512 to 4096 keys; pieces cannot be equal when lengths are not,
// and every CTA pays 4 us to start.)

#include <algorithm>
#include <atomic>

#include "attn_umma.cuh"

namespace tsd {

namespace {

using namespace attn;

constexpr int kMinTiles = 2;   // key tiles of a range at least

struct Sizes {
    int B, Tmax, Hq, Hkv, Lmax, nrb;   // nrb: row blocks of the longest chunk
    int ranges;                        // per KV head; 0: blocks, whatever the lengths
    int part_rows;                     // rows of a partial result
    float start, border, join;         // costs in key tiles, for prefer_ranges
};

// Whether ranges end sooner than blocks: `total` key tiles (of one KV head) in
// `blocks` blocks, the longest of `longest`.  A range pays its tiles, a start,
// one border per block, and the join; a block its tiles and a start, and what
// more blocks than slots cost: about 0.6 of the longest at the end.  In tiles of
// about 1 us (bf16), measured: 2 x 512 new tokens of 8/8 heads 15 us as blocks and 34
// as ranges; 256 on 8192, 64/8 heads, 125 and 94; 40 single tokens on 2048 81 and 65,
// on 64 to 512 18 and 28.
__device__ __forceinline__ bool prefer_ranges(const Sizes &z, long long total, int blocks,
                                              int longest)
{
    const float slots = (float)z.ranges, share = (float)total / slots;
    const float busy = (float)blocks / slots;   // blocks per slot
    const float as_ranges = share + z.start + z.border * busy + z.join;
    const float as_blocks = busy <= 1.f ? (float)longest + 0.5f * z.start
                                        : share + 0.6f * (float)longest + z.border * busy;
    return as_ranges < as_blocks;
}

// Key tiles of block rb of a sequence; 0 for no rows (or a bad header).
template <int BQ, int BN>
__device__ __forceinline__ int block_tiles(const Sizes &z, int rb, int T, int P)
{
    if (T < 1 || T > z.Tmax || P < 0 || P > z.Lmax - T)
        return 0;
    const int G = z.Hq / z.Hkv, R = T * G, r0 = rb * BQ;   // at most 2^30 rows
    if (r0 >= R)
        return 0;
    const int t_last = (min(r0 + BQ, R) - 1) / G;
    return (P + t_last + BN) / BN;   // ceil of P + t_last + 1 keys
}

// Partial results in the workspace: (first range, how many, which of the first
// one's two slots) per (item, KV head), then per slot the rows' (max, sum),
// then their unnormalised rows.  A CTA has two slots: a block that its range
// begins in the middle of, and one that its range ends in the middle of.
struct Parts {
    int4 *meta;
    float2 *ml;
    float *o;
};

// A CTA's walk through its range: the blocks (items) it touches, one at a
// time.  Every warp makes the same walk by itself.
template <int BQ, int BN>
struct Walk {
    // the current segment: key tiles [tile0, tile0 + n) of block rb of sequence b
    int item, b, hk, rb, T, P, tile0, n;
    bool whole;     // the whole block: its rows are final
    int slot;       // of a partial result
    int left;       // tiles of the range behind the segment
    int done;       // tiles of the range in front of the segment

    __device__ __forceinline__ int load_item(const Sizes &z, const int32_t *prefix_len,
                                             const int32_t *chunk_len)
    {
        b = item / z.nrb;
        rb = item - b * z.nrb;
        T = chunk_len[b];
        P = prefix_len[b];
        return block_tiles<BQ, BN>(z, rb, T, P);
    }

    // This CTA's block; with `meta`, notes that there is nothing to join.
    __device__ __forceinline__ bool begin_block(const Sizes &z, const int32_t *prefix_len,
                                                const int32_t *chunk_len, int4 *meta)
    {
        const int pairs = z.B * z.Hkv, order = blockIdx.x / pairs, pair = blockIdx.x - order * pairs;
        if (order >= z.nrb)
            return false;
        b = pair / z.Hkv;
        hk = pair - b * z.Hkv;
        item = b * z.nrb + z.nrb - 1 - order;   // most keys first
        tile0 = 0;
        n = load_item(z, prefix_len, chunk_len);
        whole = true;
        left = 0;
        if (meta && (threadIdx.x & 31) == 0)
            meta[item * z.Hkv + hk] = make_int4(0, 1, 0, 0);
        return n > 0;
    }

    // The first segment; false if the CTA has no work.  With `meta`, notes
    // where the pieces of every block that begins in this range will be.
    __device__ __forceinline__ bool begin(const Sizes &z, const int32_t *prefix_len,
                                          const int32_t *chunk_len, int4 *meta)
    {
        done = 0;
        slot = 0;
        if (z.ranges == 0)
            return begin_block(z, prefix_len, chunk_len, nullptr);
        const int lane = threadIdx.x & 31, items = z.B * z.nrb;
        auto tiles_of = [&](int i) {
            const int s = i / z.nrb;
            return i < items ? block_tiles<BQ, BN>(z, i - s * z.nrb, chunk_len[s], prefix_len[s])
                             : 0;
        };
        const int tiles_first = tiles_of(lane);   // kept for the second pass
        long long total = tiles_first;
        int longest = tiles_first, blocks = tiles_first > 0;
        for (int i = lane + 32; i < items; i += 32) {
            const int tiles = tiles_of(i);
            total += tiles;
            longest = max(longest, tiles);
            blocks += tiles > 0;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            total += __shfl_xor_sync(0xffffffffu, total, o);
            longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, o));
            blocks += __shfl_xor_sync(0xffffffffu, blocks, o);
        }
        if (!prefer_ranges(z, total, blocks, longest))
            return begin_block(z, prefix_len, chunk_len, meta);
        const int c = blockIdx.x / z.Hkv;
        hk = blockIdx.x - c * z.Hkv;
        const long long ranges = min((long long)z.ranges, (total + kMinTiles - 1) / kMinTiles);
        if (c >= ranges)
            return false;
        const long long lo = c * total / ranges, hi = (c + 1) * total / ranges;
        auto owner = [&](long long tile) {   // the range that holds a tile
            return (int)(((tile + 1) * ranges + total - 1) / total) - 1;
        };
        long long before = 0;
        bool found = false;
        for (int i0 = 0; i0 < items; i0 += 32) {
            const int tiles = i0 ? tiles_of(i0 + lane) : tiles_first;
            long long incl = tiles;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long x = __shfl_up_sync(0xffffffffu, incl, o);
                incl += lane >= o ? x : 0;
            }
            const long long first = before + incl - tiles, end = before + incl;
            if (meta && tiles > 0 && first >= lo && first < hi)
                meta[(i0 + lane) * z.Hkv + hk] =
                    make_int4(c, owner(end - 1) - c + 1, first > lo ? 1 : 0, 0);
            const uint32_t here = __ballot_sync(0xffffffffu, tiles > 0 && first <= lo && lo < end);
            if (here) {
                const int src = __ffs(here) - 1;
                item = i0 + src;
                tile0 = (int)(lo - __shfl_sync(0xffffffffu, first, src));
                found = true;
            }
            before = __shfl_sync(0xffffffffu, end, 31);
            if (before >= hi)
                break;
        }
        if (!found)
            return false;
        left = (int)(hi - lo);
        const int all = load_item(z, prefix_len, chunk_len);
        n = min(all - tile0, left);
        whole = tile0 == 0 && n == all;
        left -= n;
        return true;
    }

    __device__ __forceinline__ bool next(const Sizes &z, const int32_t *prefix_len,
                                         const int32_t *chunk_len)
    {
        if (left == 0)
            return false;
        done += n;
        int all;
        do {   // the tiles left belong to a later item
            if (++item >= z.B * z.nrb)
                return false;   // only if the lengths change under the kernel
            all = load_item(z, prefix_len, chunk_len);
        } while (all == 0);
        tile0 = 0;
        n = min(all, left);
        whole = n == all;
        slot = 1;
        left -= n;
        return true;
    }
    // row of the partial results where this segment's row r is
    __device__ __forceinline__ size_t part_row(const Sizes &z, int r) const
    {
        return (size_t)(2 * blockIdx.x + slot) * z.part_rows + r;
    }
    // checked build: the row is one of the partial results'
    __device__ __forceinline__ bool part_ok(const Sizes &z, size_t at, int32_t *dev_status) const
    {
        return in_bounds((long long)at, 2LL * z.ranges * z.Hkv * z.part_rows, dev_status);
    }
};

// A malformed header is reported by the first CTA that can see it.
__device__ __forceinline__ void check_headers(const Sizes &z, const int32_t *prefix_len,
                                              const int32_t *chunk_len, int32_t *dev_status)
{
    if (blockIdx.x != 0)
        return;
    for (int b = threadIdx.x; b < z.B; b += blockDim.x) {
        const int T = chunk_len[b], P = prefix_len[b];
        if (T < 0 || T > z.Tmax || P < 0 || P > z.Lmax - T)
            flag(dev_status, TSD_DEV_BAD_PREFIX);
    }
}

// ------------------------------------------------------------------- bf16
template <int HD> using Half = Geo<64, 2, 2, 256, HD>;   // 64-key tiles, two CTAs per SM

// What a token's rows see: the keys in front of `end`; `all` of the block's
// rows see those in front of the first row's end.
struct CausalVis {
    int end, all;
    __device__ __forceinline__ bool clear(int pos0, int n) const { return pos0 + n <= all; }
    __device__ __forceinline__ uint32_t bits(int pos) const
    {
        const int n = end - pos;
        return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
    }
};

// TMA producer: the K and V tiles of all segments in one stream, in the order
// of produce_kv (K_0 .., V_0 .., then V_m, K_{m+L}, ...), ring slots and barrier
// phases counted over the whole range.  Lane r issues the boxes of the r-th
// page of a tile, so that the block-table entries of a tile are read side by
// side; those of the next K tile are read one turn ahead, and the V tile finds
// them in L1.
template <class Gm, int NS, int BQ_>
__device__ __forceinline__ void produce_range(const Setup<Gm> &su, const CUtensorMap *tmK,
                                              const CUtensorMap *tmV, const Sizes &z,
                                              const Walk<BQ_, Gm::BN> &start,
                                              const int32_t *prefix_len, const int32_t *chunk_len,
                                              const KvPages &pages, int32_t *dev_status)
{
    constexpr int NSK = Gm::NSK, NSV = Gm::NSV, BN = Gm::BN;
    constexpr int kLead = NSK + NS - NSV;
    const int lane = threadIdx.x & 31;
    const int rows = min(BN, pages.page_size), boxes = BN / rows;
    Walk<BQ_, BN> wk = start, wv = start;   // where the K and the V loads are
    int jk = 0, jv = 0;                     // tiles of their segments
    auto entry = [&](const Walk<BQ_, BN> &w, int j) -> int {   // this lane's page of a tile
        const int pos = (w.tile0 + j) * BN + lane * rows;
        return lane < boxes && pos < w.P + w.T
                   ? pages.table[(size_t)w.b * pages.max_blocks + (pos >> pages.log2_page)]
                   : 0;
    };
    auto load = [&](uint32_t dst, const CUtensorMap *tm, uint32_t bar, const Walk<BQ_, BN> &w, int j,
                    int page) {
        if (lane == 0)
            ptx::mbar_arrive_expect_tx(bar, Gm::kTile);
        __syncwarp();
        if (lane >= boxes)
            return;
        // a box behind the sequence's end loads any page: masked and zeroed
        const int pos = (w.tile0 + j) * BN + lane * rows;
        int zc = w.hk, y = 0;
        if (pos < w.P + w.T) {
            if (page < 0 || page >= pages.num_pages)
                flag(dev_status, TSD_DEV_BAD_PAGE);   // page 0 stands in
            else
                zc = page * z.Hkv + w.hk;
            y = pos & (pages.page_size - 1);
        }
        ptx::tma_load_3d(dst + lane * rows * 128, tm, 0, y, zc, bar);
        if (Gm::HD == 128)
            ptx::tma_load_3d(dst + Gm::kSub + lane * rows * 128, tm, 64, y, zc, bar);
    };
    if (lane == 0) {
        ptx::prefetch_tmap(tmK);
        ptx::prefetch_tmap(tmV);
    }
    bool more_k = true, more_v = true;
    int page_k = entry(wk, 0);
    int i = 0, j = 0;   // next K tile, next V tile of the range
    while (more_k || more_v) {
        if (more_k && (!more_v || i < NSK || (j >= NSV && i <= j - 1 + kLead))) {
            const int s = i % NSK;
            if (i >= NSK && !warp_wait(su.bars.s_full(s), ((i / NSK) - 1) & 1, su.abort_flag))
                break;
            load(su.sK + s * Gm::kTile, tmK, su.bars.k_full(s), wk, jk, page_k);
            ++i;
            if (++jk == wk.n) {
                jk = 0;
                more_k = wk.next(z, prefix_len, chunk_len);
            }
            if (more_k)
                page_k = entry(wk, jk);
        } else {
            const int s = j % NSV, r = j - NSV;   // PV_r read this slot last
            if (j >= NSV && !warp_wait(su.bars.o_ready(r % NS), (r / NS) & 1, su.abort_flag))
                break;
            load(su.sV + s * Gm::kTile, tmV, su.bars.v_full(s), wv, jv, entry(wv, jv));
            ++j;
            if (++jv == wv.n) {
                jv = 0;
                more_v = wv.next(z, prefix_len, chunk_len);
            }
        }
    }
    if (lane == 0) {
        su.loads[0] = i;
        su.loads[1] = j;
    }
}

// The warps and barriers of tree attention's rows kernel: warp 0 the TMA
// producer, warp 1 the MMA issuer (QK_0 .. QK_{NS-1}, then PV_j QK_{j+NS}),
// warps 2 .. 5 the softmax, one query row per thread.  Tiles, and with them
// ring slots and barrier phases, are counted over the CTA's whole range (g0 +
// j); q_full completes once per segment.  The border between two segments: a
// softmax warp that has written out O (whose last product it waited for, so
// all of the segment's products are done) loads the next Q rows and arrives on
// q_full; the MMA warp then issues the next segment's first products, and its
// first PV, which overwrites O, waits for the P that these warps write later
// still.  The K and V rings run on meanwhile.
template <class Gm, int NS, int kMinBlocks>
__global__ void __launch_bounds__(192, kMinBlocks)
    chunk_attn_umma_kernel(const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV,
                           const __nv_bfloat16 *__restrict__ q,
                           const int32_t *__restrict__ prefix_len,
                           const int32_t *__restrict__ chunk_len, Sizes z, float scale_log2,
                           __nv_bfloat16 *__restrict__ out, Parts parts, int32_t *dev_status,
                           KvPages pages)
{
    extern __shared__ uint8_t smem_raw[];
    constexpr int BN = Gm::BN, NSK = Gm::NSK, NSV = Gm::NSV, HD = Gm::HD;
    static_assert(NS * BN + HD <= (int)Gm::kTmemCols && BN % 64 == 0, "TMEM layout");
    static_assert(NS == NSK, "the producer reuses K slots on the score barriers");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    check_headers(z, prefix_len, chunk_len, dev_status);
    Walk<BQ, BN> w;
    // the join's indices are written before any wait: valid even after a timeout
    if (!w.begin(z, prefix_len, chunk_len, warp == 5 ? parts.meta : nullptr))
        return;
    const int G = z.Hq / z.Hkv;
    const Setup<Gm> su = cta_setup<Gm>(smem_raw, 4, 4);   // arrivals: softmax warps
    auto col_s = [](int i) { return (uint32_t)(i % NS) * (uint32_t)BN; };
    constexpr uint32_t kO = NS * BN;

    if (warp == 0) {
        produce_range<Gm, NS, BQ>(su, &tmK, &tmV, z, w, prefix_len, chunk_len, pages, dev_status);
    } else if (warp == 1) {
        auto kbar = [&](int i) { return su.bars.k_full(i % NSK); };
        auto kpar = [&](int i) { return (uint32_t)(i / NSK) & 1u; };
        auto vbar = [&](int i) { return su.bars.v_full(i % NSV); };
        auto vpar = [&](int i) { return (uint32_t)(i / NSV) & 1u; };
        bool ok = true;
        int seg = 0;
        do {
            const int g0 = w.done, g1 = g0 + w.n;
            ok = warp_wait(su.bars.q_full(), seg & 1, su.abort_flag);
            ++seg;
            ptx::tc_fence_after();
            for (int i = g0; ok && i < min(g0 + NS, g1); ++i) {
                ok = warp_wait(kbar(i), kpar(i), su.abort_flag);
                ptx::tc_fence_after();
                if (ok)
                    issue_qk<Gm, false>(su, lane, col_s(i), i, su.bars.s_full(i % NS));
            }
            uint32_t v_tested = ptx::mbar_test(vbar(g0), vpar(g0));
            for (int j = g0; ok && j < g1; ++j) {
                if (!warp_wait(su.bars.p_full(j % NS), (j / NS) & 1, su.abort_flag) ||
                    !warp_wait_tested(v_tested, vbar(j), vpar(j), su.abort_flag)) {
                    ok = false;
                    break;
                }
                const int i = j + NS;
                const uint32_t k_tested = i < g1 ? ptx::mbar_test(kbar(i), kpar(i)) : 1u;
                issue_pv<Gm, false>(su, lane, col_s(j), kO, j, j > g0,
                                    w.P + w.T - (w.tile0 + j - g0) * BN, su.bars.o_ready(j % NS));
                if (i < g1 && !warp_wait_tested(k_tested, kbar(i), kpar(i), su.abort_flag)) {
                    ok = false;
                    break;
                }
                v_tested = j + 1 < g1 ? ptx::mbar_test(vbar(j + 1), vpar(j + 1)) : 1u;
                if (i < g1) {
                    ptx::tc_fence_after();
                    issue_qk<Gm, false>(su, lane, col_s(i), i, su.bars.s_full(i % NS));
                }
            }
        } while (ok && w.next(z, prefix_len, chunk_len));
    } else {
        const int quarter = warp & 3, tr = quarter * 32 + lane;   // row of the block
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const uint32_t taddr_o = su.tmem + lane_off + kO;
        bool ok = true;
        do {
            const int g0 = w.done, g1 = g0 + w.n;
            const int r = w.rb * BQ + tr, R = w.T * G;
            const int t = min(r, R - 1) / G, h = w.hk * G + min(r, R - 1) - t * G;
            const size_t row = ((size_t)w.b * z.Tmax + t) * z.Hq + h;
            const bool row_ok =
                r < R && in_bounds((long long)row, (long long)z.B * z.Tmax * z.Hq, dev_status);
            load_q_row<Gm>(su, q, row_ok, row * HD, tr);
            warp_arrive(su.bars.q_full());
            CausalVis vis;
            vis.end = w.P + t + 1;
            vis.all = w.P + w.rb * BQ / G + 1;
            float m_run = -INFINITY, l_run = 0.f;
            uint32_t s_tested = 0u;
            for (int j = g0; ok && j < g1; ++j) {
                if (!warp_wait_tested(s_tested, su.bars.s_full(j % NS), (j / NS) & 1,
                                      su.abort_flag)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                s_tested = j + 1 < g1
                               ? ptx::mbar_test(su.bars.s_full((j + 1) % NS), ((j + 1) / NS) & 1)
                               : 1u;
                ok = softmax_rows_tile<Gm>(su.tmem + lane_off + col_s(j), taddr_o,
                                           (w.tile0 + j - g0) * BN, vis, scale_log2, j == g0, m_run,
                                           l_run, [&]() {
                                               return warp_wait(su.bars.o_ready((j - 1) % NS),
                                                                ((j - 1) / NS) & 1, su.abort_flag);
                                           });
                if (!ok)
                    break;
                ptx::tc_fence_before();
                warp_arrive(su.bars.p_full(j % NS));
            }
            ok = ok && warp_wait(su.bars.o_ready((g1 - 1) % NS), ((g1 - 1) / NS) & 1, su.abort_flag);
            if (ok) {
                ptx::tc_fence_after();
                if (w.whole) {
                    const float inv = l_run > 0.f ? 1.f / l_run : 0.f;
                    write_row<HD>(taddr_o, inv, row_ok, row, 1, 0, 0, out, nullptr, 0, HD);
                } else {
                    const size_t at = w.part_row(z, tr);
                    const bool keep =
                        row_ok && tr < z.part_rows && w.part_ok(z, at, dev_status);
                    write_row<HD>(taddr_o, 1.f, keep, at, 2, 0, 0, out, parts.o, 0, HD);
                    if (keep)
                        parts.ml[at] = make_float2(m_run, l_run);
                }
                ptx::tc_fence_before();   // O has been read when the next P is published
            }
        } while (ok && w.next(z, prefix_len, chunk_len));
    }
    cta_teardown(su, dev_status);
}

// ------------------------------------------------------------------- fp32
// BQ rows by 64 keys a tile, 256 threads.  Scores: thread (i, j) of a 16 x 16
// grid has BQ/16 rows by the keys j, j + 16, j + 32, j + 48; output: the same
// rows by D/16 dims.  All operands are read as 16-byte vectors along the head
// dimension (rows padded by 16 bytes: no bank conflicts), 12 shared-memory
// wavefronts for 64 FMAs of a warp at BQ = 64, so the FMA pipes are the bound.
// The next tile's keys and values are copied (cp.async) while this one is
// computed.  BQ = 16 for decode and short chunks (a 64-row tile would spend
// four times the FMAs of the KV stream's time), 64 otherwise.
constexpr int kFmaThreads = 256;
constexpr int kFmaKeys = 64;

template <int BQ_, int D> struct FmaSmem {
    static constexpr int LD = D + 4, LP = kFmaKeys + 4;   // row steps, in floats
    static constexpr int kQ = 0, kK = kQ + BQ_ * LD, kV = kK + 2 * kFmaKeys * LD,
                         kP = kV + 2 * kFmaKeys * D, kFloats = kP + BQ_ * LP;
    static constexpr size_t kBytes = sizeof(float) * kFloats;
};

__device__ __forceinline__ void copy16(float *dst, const float *src, bool ok)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(ptx::smem_addr(dst)),
                 "l"(src), "r"(ok ? 16 : 0)
                 : "memory");   // zeros where there is no key
}

template <int BQ_, int D>
__global__ void __launch_bounds__(kFmaThreads)
    chunk_attn_fma_kernel(const float *__restrict__ q, const float *__restrict__ kp,
                          const float *__restrict__ vp, const int32_t *__restrict__ prefix_len,
                          const int32_t *__restrict__ chunk_len, Sizes z, float scale_log2,
                          float *__restrict__ out, Parts parts, int32_t *dev_status, KvPages pages)
{
    using Sm = FmaSmem<BQ_, D>;
    constexpr int BN = kFmaKeys, RT = BQ_ / 16, DT = D / 16;   // rows, dims of a thread
    constexpr int LD = Sm::LD, LP = Sm::LP, VEC = D / 4;
    extern __shared__ float smem[];
    float *const sQ = smem + Sm::kQ, *const sP = smem + Sm::kP;
    check_headers(z, prefix_len, chunk_len, dev_status);
    Walk<BQ_, BN> w;
    const int tid = threadIdx.x, ti = tid >> 4, tj = tid & 15;
    if (!w.begin(z, prefix_len, chunk_len, tid < 32 ? parts.meta : nullptr))
        return;
    const int G = z.Hq / z.Hkv;
    do {
        const int r0 = w.rb * BQ_, R = w.T * G, seq_end = w.P + w.T, tile1 = w.tile0 + w.n;
        auto out_row = [&](int lr) {   // row of q and out of local row lr
            const int r = min(r0 + lr, R - 1), t = r / G;
            return ((size_t)w.b * z.Tmax + t) * z.Hq + w.hk * G + r - t * G;
        };
        auto fetch = [&](int kt) {   // the copies of tile kt
            float *const sK = smem + Sm::kK + (kt & 1) * BN * LD;
            float *const sV = smem + Sm::kV + (kt & 1) * BN * D;
#pragma unroll 4
            for (int i = tid; i < BN * VEC; i += kFmaThreads) {
                const int j = i / VEC, c = i % VEC, pos = kt * BN + j;
                bool ok = pos < seq_end;
                long long row = 0;
                if (ok) {
                    const int page =
                        pages.table[(size_t)w.b * pages.max_blocks + (pos >> pages.log2_page)];
                    ok = page >= 0 && page < pages.num_pages;
                    if (ok)
                        row = ((long long)page * z.Hkv + w.hk) * pages.page_size +
                              (pos & (pages.page_size - 1));
                    else if (c == 0)
                        flag(dev_status, TSD_DEV_BAD_PAGE);   // that key reads as zero
                    ok = ok && in_bounds(row, kv_rows_total(pages, z.B, z.Hkv, 0), dev_status);
                }
                copy16(sK + j * LD + 4 * c, kp + row * D + 4 * c, ok);
                copy16(sV + j * D + 4 * c, vp + row * D + 4 * c, ok);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        fetch(w.tile0);
        for (int i = tid; i < BQ_ * VEC; i += kFmaThreads) {
            const int lr = i / VEC, c = i % VEC;
            const bool ok = r0 + lr < R && in_bounds((long long)out_row(lr),
                                                     (long long)z.B * z.Tmax * z.Hq, dev_status);
            const float4 x = ok ? __ldg(reinterpret_cast<const float4 *>(q + out_row(lr) * D) + c)
                                : make_float4(0.f, 0.f, 0.f, 0.f);
            *reinterpret_cast<float4 *>(sQ + lr * LD + 4 * c) = x;
        }
        float o[RT][DT], m[RT], l[RT];
        int end[RT];   // keys the row sees
#pragma unroll
        for (int a = 0; a < RT; ++a) {
            m[a] = -INFINITY;
            l[a] = 0.f;
            end[a] = w.P + min(r0 + ti * RT + a, R - 1) / G + 1;
#pragma unroll
            for (int c = 0; c < DT; ++c)
                o[a][c] = 0.f;
        }
        for (int kt = w.tile0; kt < tile1; ++kt) {
            const int pos0 = kt * BN;
            const float *const sK = smem + Sm::kK + (kt & 1) * BN * LD;
            const float *const sV = smem + Sm::kV + (kt & 1) * BN * D;
            if (kt + 1 < tile1) {   // into the buffers that the barrier below the tile before freed
                fetch(kt + 1);
                asm volatile("cp.async.wait_group 1;" ::: "memory");
            } else {
                asm volatile("cp.async.wait_group 0;" ::: "memory");
            }
            __syncthreads();
            float s[RT][4];
#pragma unroll
            for (int a = 0; a < RT; ++a)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    s[a][c] = 0.f;
#pragma unroll 4
            for (int d = 0; d < D; d += 4) {
                float4 y[4];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    y[c] = *reinterpret_cast<const float4 *>(sK + (tj + 16 * c) * LD + d);
#pragma unroll
                for (int a = 0; a < RT; ++a) {
                    const float4 x = *reinterpret_cast<const float4 *>(sQ + (ti * RT + a) * LD + d);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        s[a][c] = fmaf(x.x, y[c].x, s[a][c]);
                        s[a][c] = fmaf(x.y, y[c].y, s[a][c]);
                        s[a][c] = fmaf(x.z, y[c].z, s[a][c]);
                        s[a][c] = fmaf(x.w, y[c].w, s[a][c]);
                    }
                }
            }
            // a row's 64 scores are on 16 lanes of one half warp
#pragma unroll
            for (int a = 0; a < RT; ++a) {
                float mx = -INFINITY;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    s[a][c] = pos0 + tj + 16 * c < end[a] ? s[a][c] * scale_log2 : -INFINITY;
                    mx = fmaxf(mx, s[a][c]);
                }
#pragma unroll
                for (int k = 8; k > 0; k >>= 1)
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
                const float m_new = fmaxf(m[a], mx);
                const float base = m_new == -INFINITY ? 0.f : m_new;   // nothing visible yet
                const float alpha = exp2f(m[a] - base);
                float sum = 0.f;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float p = exp2f(s[a][c] - base);
                    sum += p;
                    sP[(ti * RT + a) * LP + tj + 16 * c] = p;
                }
#pragma unroll
                for (int k = 8; k > 0; k >>= 1)
                    sum += __shfl_xor_sync(0xffffffffu, sum, k);
                l[a] = l[a] * alpha + sum;
                m[a] = m_new;
#pragma unroll
                for (int c = 0; c < DT; ++c)
                    o[a][c] *= alpha;
            }
            __syncwarp();   // a row's probabilities stay within its half warp
#pragma unroll 2
            for (int j = 0; j < BN; j += 4) {
                float4 p[RT];
#pragma unroll
                for (int a = 0; a < RT; ++a)
                    p[a] = *reinterpret_cast<const float4 *>(sP + (ti * RT + a) * LP + j);
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int c = 0; c < DT; c += 4) {
                        const float4 y = *reinterpret_cast<const float4 *>(sV + (j + k) * D +
                                                                           (c / 4) * 64 + tj * 4);
#pragma unroll
                        for (int a = 0; a < RT; ++a) {
                            const float f = k == 0 ? p[a].x : k == 1 ? p[a].y : k == 2 ? p[a].z : p[a].w;
                            o[a][c] = fmaf(f, y.x, o[a][c]);
                            o[a][c + 1] = fmaf(f, y.y, o[a][c + 1]);
                            o[a][c + 2] = fmaf(f, y.z, o[a][c + 2]);
                            o[a][c + 3] = fmaf(f, y.w, o[a][c + 3]);
                        }
                    }
            }
            __syncthreads();   // this tile's buffers may be refilled
        }
#pragma unroll
        for (int a = 0; a < RT; ++a) {
            const int lr = ti * RT + a;
            if (r0 + lr >= R || !in_bounds((long long)out_row(lr), (long long)z.B * z.Tmax * z.Hq,
                                           dev_status))
                continue;
            const size_t at = w.part_row(z, lr);
            if (!w.whole && !w.part_ok(z, at, dev_status))
                continue;
            float *dst = w.whole ? out + out_row(lr) * D : parts.o + at * D;
            const float f = w.whole ? (l[a] > 0.f ? 1.f / l[a] : 0.f) : 1.f;
#pragma unroll
            for (int c = 0; c < DT; c += 4)
                *reinterpret_cast<float4 *>(dst + (c / 4) * 64 + tj * 4) =
                    make_float4(o[a][c] * f, o[a][c + 1] * f, o[a][c + 2] * f, o[a][c + 3] * f);
            if (!w.whole && tj == 0)
                parts.ml[at] = make_float2(m[a], l[a]);
        }
    } while (w.next(z, prefix_len, chunk_len));
}

// -------------------------------------------------------------------- join
// One warp per row of a block that was cut: weights 2^(m_i - max m) over its
// pieces (those of one range after the other), the weighted sum of their rows over
// the weighted sum of their sums.  A piece none of whose keys the row sees has sum
// 0; a sum that is no number (a q row with NaN) makes the row one.
constexpr int kJoinRows = 8;   // rows (warps) of a CTA

template <typename T, int D, int BQ_>
__global__ void __launch_bounds__(32 * kJoinRows)
    chunk_join_kernel(Parts parts, const int32_t *__restrict__ prefix_len,
                      const int32_t *__restrict__ chunk_len, Sizes z, T *__restrict__ out,
                      int32_t *dev_status)
{
    constexpr int DL = D / 32;   // dims of a lane
    const int item = blockIdx.x / z.Hkv, hk = blockIdx.x - item * z.Hkv;
    const int b = item / z.nrb, rb = item - b * z.nrb;
    const int n_tok = chunk_len[b], G = z.Hq / z.Hkv;
    const int lr = blockIdx.y * kJoinRows + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (block_tiles<BQ_, 64>(z, rb, n_tok, prefix_len[b]) == 0 || rb * BQ_ + lr >= n_tok * G ||
        lr >= z.part_rows)
        return;
    const int4 meta = parts.meta[blockIdx.x];
    if (meta.y < 2)
        return;
    auto piece = [&](int i) {   // this row in piece i
        return (size_t)(2 * ((meta.x + i) * z.Hkv + hk) + (i == 0 ? meta.z : 0)) * z.part_rows + lr;
    };
    float M = -INFINITY;
    for (int i = lane; i < meta.y; i += 32) {
        const float2 ml = parts.ml[piece(i)];
        M = fmaxf(M, ml.y == 0.f ? -INFINITY : ml.x);
    }
    M = warp_max(M);
    float acc[DL], L = 0.f;
#pragma unroll
    for (int k = 0; k < DL; ++k)
        acc[k] = 0.f;
    for (int i0 = 0; i0 < meta.y; i0 += 32) {
        float f = 0.f;   // lane's piece: its weight
        if (i0 + lane < meta.y) {
            const float2 ml = parts.ml[piece(i0 + lane)];
            f = ml.y == 0.f ? 0.f : exp2f(ml.x - M);
            L = fmaf(f, ml.y, L);
        }
        const int n = min(32, meta.y - i0);
#pragma unroll 8
        for (int i = 0; i < n; ++i) {
            const float w = __shfl_sync(0xffffffffu, f, i);
            const size_t at = piece(i0 + i);
            float x[DL];
            if (DL == 2) {
                const float2 v = *reinterpret_cast<const float2 *>(parts.o + at * D + lane * DL);
                x[0] = v.x;
                x[1] = v.y;
            } else {
                const float4 v = *reinterpret_cast<const float4 *>(parts.o + at * D + lane * DL);
                x[0] = v.x;
                x[1] = v.y;
                x[DL > 2 ? 2 : 0] = v.z;
                x[DL > 3 ? 3 : 0] = v.w;
            }
#pragma unroll
            for (int k = 0; k < DL; ++k)
                acc[k] = w > 0.f ? fmaf(w, x[k], acc[k]) : acc[k];
        }
    }
    L = warp_sum(L);
    const int r = rb * BQ_ + lr;
    const size_t row = ((size_t)b * z.Tmax + r / G) * z.Hq + hk * G + r % G;
    const float inv = L == 0.f ? 0.f : 1.f / L;
    if (in_bounds((long long)row, (long long)z.B * z.Tmax * z.Hq, dev_status))
#pragma unroll
        for (int k = 0; k < DL; ++k)
            out[row * D + lane * DL + k] = from_float<T>(acc[k] * inv);
}

// -------------------------------------------------------------------- host
struct Plan {
    Sizes z;
    int bq;
    long long grid;
    dim3 join;          // grid of the join
    size_t meta_bytes, ml_bytes, o_bytes;
};

// CTAs of an SM: two, or the one that fits its 228 KB of shared memory (1 KB of
// them reserved for each CTA): fp32 at head_dim 128.
template <int BQ_, int D> constexpr int fma_ctas()
{
    return std::min<int>(2, (228 * 1024) / (FmaSmem<BQ_, D>::kBytes + 1024));
}

int ctas_per_sm(const ChunkArgs &a, int bq)
{
    if (a.dtype != TSD_F32)
        return 2;
    return a.D == 64 ? (bq == 16 ? fma_ctas<16, 64>() : fma_ctas<64, 64>())
                     : (bq == 16 ? fma_ctas<16, 128>() : fma_ctas<64, 128>());
}

Plan chunk_plan(const ChunkArgs &a, int num_sms)
{
    Plan p;
    const int G = a.Hq / a.Hkv;
    const long long rows = (long long)a.Tmax * G;
    const bool f32 = a.dtype == TSD_F32;
    p.bq = f32 && rows > 16 ? 64 : f32 ? 16 : BQ;
    p.z.B = a.B;
    p.z.Tmax = a.Tmax;
    p.z.Hq = a.Hq;
    p.z.Hkv = a.Hkv;
    p.z.Lmax = a.pages.max_blocks * a.pages.page_size;
    p.z.nrb = (int)((rows + p.bq - 1) / p.bq);
    p.z.part_rows = (int)std::min<long long>(rows, p.bq);
    // in key tiles: of 1 us (bf16), 2 (fp32, 16 rows) and 5 (fp32, 64 rows);
    // joining blocks of many rows costs more than a few rows
    p.z.start = f32 ? (p.bq == 16 ? 5.f : 2.f) : 10.f;
    p.z.border = 0.5f * p.z.start;
    p.z.join = p.z.part_rows > 16 ? 1.5f * p.z.start : 0.f;
    // CTA slots of the GPU (for two CTAs per SM where one fits, fp32 at head_dim 128,
    // 32 single tokens on 1024 took 77 us, not 67).  From some number of blocks a slot they even out by
    // themselves, and the few that end last cost less than partial results do:
    // half a block where blocks are full (choosing and joining cost 5 us: 16/16
    // heads, 2048 new tokens, 256 blocks, 51 without and 60 with), two where a
    // sequence is one block (single tokens on 2048, 1024 blocks: 180 and 183;
    // 320 blocks: 81 and 65), four for fp32
    const int slots = num_sms * ctas_per_sm(a, p.bq);
    const long long blocks = (long long)a.B * a.Hkv * p.z.nrb;
    const long long most = f32 ? 4LL * slots : rows <= BQ ? 2LL * slots : slots / 2;
    size_t items = 0, parts = 0;
    if (blocks < most) {
        p.z.ranges = std::max(slots / a.Hkv, 1);
        const long long cut = (long long)p.z.ranges * a.Hkv;
        p.grid = std::max(cut, blocks);   // the lengths decide which of the two
        items = (size_t)a.B * p.z.nrb;
        parts = (size_t)cut * 2;
        p.join = dim3((unsigned)(items * a.Hkv), (p.z.part_rows + kJoinRows - 1) / kJoinRows);
    } else {
        p.z.ranges = 0;
        p.grid = blocks;
    }
    auto up = [](size_t n) { return (n + 255) & ~(size_t)255; };
    p.meta_bytes = up(items * a.Hkv * sizeof(int4));
    p.ml_bytes = up(parts * p.z.part_rows * sizeof(float2));
    p.o_bytes = parts * p.z.part_rows * a.D * sizeof(float);
    return p;
}

// The dynamic shared memory limit of `kern` on the current device, raised once.
cudaError_t raise_smem(const void *kern, size_t bytes, bool max_carveout)
{
    cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           (int)bytes);
    if (err == cudaSuccess && max_carveout)
        err = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout,
                                   (int)cudaSharedmemCarveoutMaxShared);
    return err;
}

cudaError_t set_smem_attributes()
{
    constexpr int kMaxDevices = 64;
    static std::atomic<bool> done[kMaxDevices];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess)
        return err;
    if (dev < 0 || dev >= kMaxDevices)
        return cudaErrorInvalidDevice;
    if (done[dev].load())
        return cudaSuccess;
    struct {
        const void *kern;
        size_t bytes;
    } const all[] = {
        {(const void *)chunk_attn_umma_kernel<Half<128>, 2, 2>, Half<128>::kSmemBytes},
        {(const void *)chunk_attn_umma_kernel<Half<64>, 2, 2>, Half<64>::kSmemBytes},
        {(const void *)chunk_attn_fma_kernel<16, 64>, FmaSmem<16, 64>::kBytes},
        {(const void *)chunk_attn_fma_kernel<64, 64>, FmaSmem<64, 64>::kBytes},
        {(const void *)chunk_attn_fma_kernel<16, 128>, FmaSmem<16, 128>::kBytes},
        {(const void *)chunk_attn_fma_kernel<64, 128>, FmaSmem<64, 128>::kBytes}};
    for (const auto &k : all)
        if (err == cudaSuccess)
            err = raise_smem(k.kern, k.bytes, true);
    if (err == cudaSuccess)
        done[dev].store(true);
    return err;
}

template <int D>
int launch_umma(const ChunkArgs &a, const Plan &p, const Parts &parts, float sl2,
                cudaStream_t stream)
{
    CUtensorMap tmK, tmV;
    const int box = std::min(Half<D>::BN, a.pages.page_size);
    const int planes = a.pages.num_pages * a.Hkv;
    if (!make_kv_map(&tmK, a.k, D, a.pages.page_size, planes, box) ||
        !make_kv_map(&tmV, a.v, D, a.pages.page_size, planes, box))
        return TSD_ERR_CUDA;
    chunk_attn_umma_kernel<Half<D>, 2, 2><<<(unsigned)p.grid, 192, Half<D>::kSmemBytes, stream>>>(
        tmK, tmV, static_cast<const __nv_bfloat16 *>(a.q), a.prefix_len, a.chunk_len, p.z, sl2,
        static_cast<__nv_bfloat16 *>(a.out), parts, a.dev_status, a.pages);
    TSD_LAUNCH_CHECK();
    if (p.z.ranges) {
        chunk_join_kernel<__nv_bfloat16, D, BQ><<<p.join, 32 * kJoinRows, 0, stream>>>(
            parts, a.prefix_len, a.chunk_len, p.z, static_cast<__nv_bfloat16 *>(a.out),
            a.dev_status);
        TSD_LAUNCH_CHECK();
    }
    return TSD_OK;
}

template <int BQ_, int D>
int launch_fma(const ChunkArgs &a, const Plan &p, const Parts &parts, float sl2,
               cudaStream_t stream)
{
    chunk_attn_fma_kernel<BQ_, D>
        <<<(unsigned)p.grid, kFmaThreads, FmaSmem<BQ_, D>::kBytes, stream>>>(
        static_cast<const float *>(a.q), static_cast<const float *>(a.k),
        static_cast<const float *>(a.v), a.prefix_len, a.chunk_len, p.z, sl2,
        static_cast<float *>(a.out), parts, a.dev_status, a.pages);
    TSD_LAUNCH_CHECK();
    if (p.z.ranges) {
        chunk_join_kernel<float, D, BQ_><<<p.join, 32 * kJoinRows, 0, stream>>>(
            parts, a.prefix_len, a.chunk_len, p.z, static_cast<float *>(a.out), a.dev_status);
        TSD_LAUNCH_CHECK();
    }
    return TSD_OK;
}

}  // namespace

size_t chunk_attention_workspace(const ChunkArgs &a, int num_sms)
{
    const Plan p = chunk_plan(a, num_sms);
    return p.meta_bytes + p.ml_bytes + p.o_bytes;
}

int launch_chunk_attention(const ChunkArgs &a, void *ws, int num_sms, cudaStream_t stream)
{
    const Plan p = chunk_plan(a, num_sms);
    if (p.grid > 0x7fffffffLL)
        return TSD_ERR_SHAPE;
    TSD_CUDA_TRY(set_smem_attributes());
    Parts parts{};
    if (p.z.ranges) {
        char *base = static_cast<char *>(ws);
        parts.meta = reinterpret_cast<int4 *>(base);
        parts.ml = reinterpret_cast<float2 *>(base + p.meta_bytes);
        parts.o = reinterpret_cast<float *>(base + p.meta_bytes + p.ml_bytes);
    }
    const float sl2 = a.scale * kLog2e;
    if (a.dtype == TSD_BF16)
        return a.D == 64 ? launch_umma<64>(a, p, parts, sl2, stream)
                         : launch_umma<128>(a, p, parts, sl2, stream);
    if (p.bq == 16)
        return a.D == 64 ? launch_fma<16, 64>(a, p, parts, sl2, stream)
                         : launch_fma<16, 128>(a, p, parts, sl2, stream);
    return a.D == 64 ? launch_fma<64, 64>(a, p, parts, sl2, stream)
                     : launch_fma<64, 128>(a, p, parts, sl2, stream);
}

}  // namespace tsd
