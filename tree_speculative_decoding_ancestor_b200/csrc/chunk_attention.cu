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
//   * bf16: tcgen05 products with S and O in TMEM (attn_umma.cuh), the
//     geometry of tree attention: 128-key tiles at one CTA per SM, or, where a
//     sequence's rows are one block of 128, 64-key tiles at two CTAs per SM
//     (the KV stream is the bound there).  head_dim 64 or 128.
//   * fp32: FMA tiles in registers (the tensor cores have no fp32 product).
//
// Work is divided in one of two ways.
//   * Many blocks (prompts): one CTA per (block, KV head, sequence), the
//     blocks with the most keys first.
//   * Few blocks (decode, short chunks): every block's keys are split so that
//     all CTAs get about the same number of key tiles, whatever the sequences'
//     lengths.  The lengths are on the device, so each warp of each CTA finds
//     its own piece from them (a sum and a scan over at most a few hundred
//     items, no extra launch), and a second kernel joins the pieces of a block
//     by their running maxima and sums.
#include <algorithm>
#include <atomic>

#include "attn_umma.cuh"

namespace tsd {

namespace {

using namespace attn;

constexpr int kMinTiles = 2;   // key tiles of a piece at least, when keys are split

struct Sizes {
    int B, Tmax, Hq, Hkv, Lmax, nrb;   // nrb: row blocks of the longest chunk
    int slots;                         // 0: one CTA per block; else pieces aimed at
    int part_rows;                     // rows of a partial result
};

// One CTA's share: rows [rb * BQ, ..) of sequence b and KV head hk, key tiles
// [tile0, tile1).
struct Piece {
    int b, hk, rb, T, P, tile0, tile1, pieces, first, item;
};

// Key tiles of block rb of sequence b; 0 for no rows (or a bad header).
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

// This CTA's piece (every warp finds the same one); false if it has none.
template <int BQ, int BN>
__device__ __forceinline__ bool find_piece(const Sizes &z, const int32_t *prefix_len,
                                           const int32_t *chunk_len, Piece &w)
{
    if (z.slots == 0) {
        const int pairs = z.B * z.Hkv;
        const int pair = blockIdx.x % pairs;
        w.rb = z.nrb - 1 - blockIdx.x / pairs;   // most keys first
        w.b = pair / z.Hkv;
        w.hk = pair % z.Hkv;
        w.T = chunk_len[w.b];
        w.P = prefix_len[w.b];
        w.tile0 = 0;
        w.tile1 = block_tiles<BQ, BN>(z, w.rb, w.T, w.P);
        w.pieces = 1;
        w.first = 0;
        w.item = 0;
        return w.tile1 > 0;
    }
    const int lane = threadIdx.x & 31;
    const int items = z.B * z.nrb;
    auto tiles_of = [&](int i) {
        const int b = i / z.nrb;
        return block_tiles<BQ, BN>(z, i - b * z.nrb, chunk_len[b], prefix_len[b]);
    };
    long long total = 0;
    for (int i = lane; i < items; i += 32)
        total += tiles_of(i);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        total += __shfl_xor_sync(0xffffffffu, total, o);
    const int per = (int)max((total * z.Hkv + z.slots - 1) / z.slots, (long long)kMinTiles);
    w.hk = blockIdx.x % z.Hkv;
    const int mine = blockIdx.x / z.Hkv;
    int before = 0;
    for (int i0 = 0; i0 < items; i0 += 32) {
        const int tiles = i0 + lane < items ? tiles_of(i0 + lane) : 0;
        const int n = (tiles + per - 1) / per;
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, o);
            incl += lane >= o ? x : 0;
        }
        const int total_n = __shfl_sync(0xffffffffu, incl, 31);
        if (mine < before + total_n) {
            const bool here = mine >= before + incl - n && mine < before + incl;
            const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
            const int first = __shfl_sync(0xffffffffu, before + incl - n, src);
            w.pieces = __shfl_sync(0xffffffffu, n, src);
            const int all = __shfl_sync(0xffffffffu, tiles, src);
            const int s = mine - first;
            w.item = i0 + src;
            w.b = w.item / z.nrb;
            w.rb = w.item - w.b * z.nrb;
            w.T = chunk_len[w.b];
            w.P = prefix_len[w.b];
            const int each = all / w.pieces, more = all - each * w.pieces;
            w.tile0 = s * each + min(s, more);
            w.tile1 = w.tile0 + each + (s < more ? 1 : 0);
            w.first = first * z.Hkv + w.hk;   // the CTA of piece 0; the others Hkv apart
            return true;
        }
        before += total_n;
    }
    return false;
}

// Partial results in the workspace: (first piece, pieces) per (item, KV
// head), then per piece the rows' (max, sum), then their unnormalised rows.
struct Parts {
    int2 *meta;
    float2 *ml;
    float *o;
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
template <int HD> using Wide = Geo<128, 3, 2, 512, HD>;
template <int HD> using Half = Geo<64, 2, 2, 256, HD>;

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

// The warps and barriers of tree attention's rows kernel: warp 0 the TMA
// producer, warp 1 the MMA issuer (QK_0 .. QK_{NS-1}, then PV_j QK_{j+NS}),
// warps 2 .. 5 the softmax, one query row per thread.
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
    check_headers(z, prefix_len, chunk_len, dev_status);
    Piece w;
    if (!find_piece<BQ, BN>(z, prefix_len, chunk_len, w))
        return;
    const int G = z.Hq / z.Hkv;
    const int kb = w.tile0 * BN, ntiles = w.tile1 - w.tile0;
    const int seq_end = w.P + w.T;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // before any wait, so that the join reads valid indices even after a timeout
    if (z.slots && blockIdx.x == (unsigned)w.first && threadIdx.x == 0)
        parts.meta[w.item * z.Hkv + w.hk] = make_int2(w.first, w.pieces);
    const Setup<Gm> su = cta_setup<Gm>(smem_raw, 4, 4);   // arrivals: softmax warps
    auto col_s = [](int i) { return (uint32_t)(i % NS) * (uint32_t)BN; };
    constexpr uint32_t kO = NS * BN;

    if (warp == 0) {
        const PageCache pc = stage_pages(su, pages, w.b, kb, min(w.tile1 * BN, seq_end), lane);
        if (lane == 0)
            produce_kv<Gm, NS>(su, &tmK, &tmV, w.b, w.hk, z.Hkv, kb, ntiles, pages, pc, seq_end,
                               dev_status);
    } else if (warp == 1) {
        auto kbar = [&](int i) { return su.bars.k_full(i % NSK); };
        auto kpar = [&](int i) { return (uint32_t)(i / NSK) & 1u; };
        auto vbar = [&](int i) { return su.bars.v_full(i % NSV); };
        auto vpar = [&](int i) { return (uint32_t)(i / NSV) & 1u; };
        bool ok = warp_wait(su.bars.q_full(), 0, su.abort_flag);
        ptx::tc_fence_after();
        for (int i = 0; ok && i < min(NS, ntiles); ++i) {
            ok = warp_wait(kbar(i), kpar(i), su.abort_flag);
            ptx::tc_fence_after();
            if (ok)
                issue_qk<Gm, false>(su, lane, col_s(i), i, su.bars.s_full(i % NS));
        }
        uint32_t v_tested = ptx::mbar_test(vbar(0), vpar(0));
        for (int j = 0; ok && j < ntiles; ++j) {
            if (!warp_wait(su.bars.p_full(j % NS), (j / NS) & 1, su.abort_flag) ||
                !warp_wait_tested(v_tested, vbar(j), vpar(j), su.abort_flag)) {
                ok = false;
                break;
            }
            const int i = j + NS;
            const uint32_t k_tested = i < ntiles ? ptx::mbar_test(kbar(i), kpar(i)) : 1u;
            issue_pv<Gm, false>(su, lane, col_s(j), kO, j, j > 0, seq_end - (kb + j * BN),
                                su.bars.o_ready(j % NS));
            if (i < ntiles && !warp_wait_tested(k_tested, kbar(i), kpar(i), su.abort_flag)) {
                ok = false;
                break;
            }
            v_tested = j + 1 < ntiles ? ptx::mbar_test(vbar(j + 1), vpar(j + 1)) : 1u;
            if (i < ntiles) {
                ptx::tc_fence_after();
                issue_qk<Gm, false>(su, lane, col_s(i), i, su.bars.s_full(i % NS));
            }
        }
    } else {
        const int quarter = warp & 3, tr = quarter * 32 + lane;   // row of the block
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
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
        const uint32_t taddr_o = su.tmem + lane_off + kO;
        float m_run = -INFINITY, l_run = 0.f;
        bool ok = true;
        uint32_t s_tested = ptx::mbar_test(su.bars.s_full(0), 0);
        for (int j = 0; ok && j < ntiles; ++j) {
            if (!warp_wait_tested(s_tested, su.bars.s_full(j % NS), (j / NS) & 1,
                                  su.abort_flag)) {
                ok = false;
                break;
            }
            ptx::tc_fence_after();
            s_tested = j + 1 < ntiles
                           ? ptx::mbar_test(su.bars.s_full((j + 1) % NS), ((j + 1) / NS) & 1)
                           : 1u;
            ok = softmax_rows_tile<Gm>(su.tmem + lane_off + col_s(j), taddr_o, kb + j * BN, vis,
                                       scale_log2, j == 0, m_run, l_run, [&]() {
                                           return warp_wait(su.bars.o_ready((j - 1) % NS),
                                                            ((j - 1) / NS) & 1, su.abort_flag);
                                       });
            if (!ok)
                break;
            ptx::tc_fence_before();
            warp_arrive(su.bars.p_full(j % NS));
        }
        if (ok && warp_wait(su.bars.o_ready((ntiles - 1) % NS), ((ntiles - 1) / NS) & 1,
                            su.abort_flag)) {
            ptx::tc_fence_after();
            if (w.pieces == 1) {
                const float inv = l_run > 0.f ? 1.f / l_run : 0.f;
                write_row<HD>(taddr_o, inv, row_ok, row, 1, 0, 0, out, nullptr, 0, HD);
            } else {
                const size_t at = (size_t)blockIdx.x * z.part_rows + tr;
                const bool keep = row_ok && tr < z.part_rows;
                write_row<HD>(taddr_o, 1.f, keep, at, 2, 0, 0, out, parts.o, 0, HD);
                if (keep)
                    parts.ml[at] = make_float2(m_run, l_run);
            }
        }
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
    Piece w;
    if (!find_piece<BQ_, BN>(z, prefix_len, chunk_len, w))
        return;
    const int G = z.Hq / z.Hkv, seq_end = w.P + w.T;
    const int tid = threadIdx.x, ti = tid >> 4, tj = tid & 15;
    if (z.slots && blockIdx.x == (unsigned)w.first && tid == 0)
        parts.meta[w.item * z.Hkv + w.hk] = make_int2(w.first, w.pieces);
    const int r0 = w.rb * BQ_, R = w.T * G;
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
    for (int kt = w.tile0; kt < w.tile1; ++kt) {
        const int pos0 = kt * BN;
        const float *const sK = smem + Sm::kK + (kt & 1) * BN * LD;
        const float *const sV = smem + Sm::kV + (kt & 1) * BN * D;
        if (kt + 1 < w.tile1) {   // into the buffers that the barrier below the tile before freed
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
        const size_t at = (size_t)blockIdx.x * z.part_rows + lr;
        float *dst = w.pieces == 1 ? out + out_row(lr) * D : parts.o + at * D;
        const float f = w.pieces == 1 ? (l[a] > 0.f ? 1.f / l[a] : 0.f) : 1.f;
#pragma unroll
        for (int c = 0; c < DT; c += 4)
            *reinterpret_cast<float4 *>(dst + (c / 4) * 64 + tj * 4) =
                make_float4(o[a][c] * f, o[a][c + 1] * f, o[a][c + 2] * f, o[a][c + 3] * f);
        if (w.pieces > 1 && tj == 0)
            parts.ml[at] = make_float2(m[a], l[a]);
    }
}

// -------------------------------------------------------------------- join
// One warp per row of a block that was split: weights 2^(m_i - max m) over its
// pieces (Hkv CTAs apart), the weighted sum of their rows over the weighted sum
// of their sums.  A piece none of whose keys the row sees has sum 0.
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
    const int2 meta = parts.meta[blockIdx.x];
    if (meta.y < 2)
        return;
    float M = -INFINITY;
    for (int i = lane; i < meta.y; i += 32) {
        const float2 ml = parts.ml[(size_t)(meta.x + i * z.Hkv) * z.part_rows + lr];
        M = fmaxf(M, ml.y > 0.f ? ml.x : -INFINITY);
    }
    M = warp_max(M);
    float acc[DL], L = 0.f;
#pragma unroll
    for (int k = 0; k < DL; ++k)
        acc[k] = 0.f;
    for (int i0 = 0; i0 < meta.y; i0 += 32) {
        float f = 0.f;   // lane's piece: its weight
        if (i0 + lane < meta.y) {
            const float2 ml = parts.ml[(size_t)(meta.x + (i0 + lane) * z.Hkv) * z.part_rows + lr];
            f = ml.y > 0.f ? exp2f(ml.x - M) : 0.f;
            L = fmaf(f, ml.y, L);
        }
        const int n = min(32, meta.y - i0);
#pragma unroll 8
        for (int i = 0; i < n; ++i) {
            const float w = __shfl_sync(0xffffffffu, f, i);
            const size_t at = (size_t)(meta.x + (i0 + i) * z.Hkv) * z.part_rows + lr;
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
    const float inv = L > 0.f ? 1.f / L : 0.f;
    if (in_bounds((long long)row, (long long)z.B * z.Tmax * z.Hq, dev_status))
#pragma unroll
        for (int k = 0; k < DL; ++k)
            out[row * D + lane * DL + k] = from_float<T>(acc[k] * inv);
}

// -------------------------------------------------------------------- host
struct Plan {
    Sizes z;
    bool paired;        // bf16: 64-key tiles, two CTAs per SM
    int bq;
    long long grid;
    dim3 join;          // grid of the join
    size_t meta_bytes, ml_bytes, o_bytes;
};

Plan chunk_plan(const ChunkArgs &a, int num_sms)
{
    Plan p;
    const int G = a.Hq / a.Hkv;
    const long long rows = (long long)a.Tmax * G;
    const bool f32 = a.dtype == TSD_F32;
    p.bq = f32 && rows > 16 ? 64 : f32 ? 16 : BQ;
    p.paired = !f32 && rows <= BQ;
    p.z.B = a.B;
    p.z.Tmax = a.Tmax;
    p.z.Hq = a.Hq;
    p.z.Hkv = a.Hkv;
    p.z.Lmax = a.pages.max_blocks * a.pages.page_size;
    p.z.nrb = (int)((rows + p.bq - 1) / p.bq);
    p.z.part_rows = (int)std::min<long long>(rows, p.bq);
    // CTA slots of the GPU; keys are split while the blocks alone would leave
    // the last wave mostly empty (fewer than four blocks a slot).
    const int slots = num_sms * (f32 || p.paired ? 2 : 1);
    const long long blocks = (long long)a.B * a.Hkv * p.z.nrb;
    size_t items = 0;
    if (blocks < 4LL * slots) {
        p.z.slots = slots;
        items = (size_t)a.B * p.z.nrb;
        p.join = dim3((unsigned)(items * a.Hkv), (p.z.part_rows + kJoinRows - 1) / kJoinRows);
        p.grid = (long long)slots + blocks + a.Hkv;
    } else {
        p.z.slots = 0;
        p.grid = blocks;
    }
    auto up = [](size_t n) { return (n + 255) & ~(size_t)255; };
    p.meta_bytes = p.z.slots ? up(items * a.Hkv * sizeof(int2)) : 0;
    p.ml_bytes = p.z.slots ? up((size_t)p.grid * p.z.part_rows * sizeof(float2)) : 0;
    p.o_bytes = p.z.slots ? (size_t)p.grid * p.z.part_rows * a.D * sizeof(float) : 0;
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
        {(const void *)chunk_attn_umma_kernel<Wide<128>, 3, 1>, Wide<128>::kSmemBytes},
        {(const void *)chunk_attn_umma_kernel<Wide<64>, 3, 1>, Wide<64>::kSmemBytes},
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
    const int box = std::min(p.paired ? 64 : 128, a.pages.page_size);
    const int planes = a.pages.num_pages * a.Hkv;
    if (!make_kv_map(&tmK, a.k, D, a.pages.page_size, planes, box) ||
        !make_kv_map(&tmV, a.v, D, a.pages.page_size, planes, box))
        return TSD_ERR_CUDA;
    auto kern = p.paired ? chunk_attn_umma_kernel<Half<D>, 2, 2>
                         : chunk_attn_umma_kernel<Wide<D>, 3, 1>;
    const uint32_t smem = p.paired ? Half<D>::kSmemBytes : Wide<D>::kSmemBytes;
    kern<<<(unsigned)p.grid, 192, smem, stream>>>(
        tmK, tmV, static_cast<const __nv_bfloat16 *>(a.q), a.prefix_len, a.chunk_len, p.z, sl2,
        static_cast<__nv_bfloat16 *>(a.out), parts, a.dev_status, a.pages);
    TSD_LAUNCH_CHECK();
    if (p.z.slots) {
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
    if (p.z.slots) {
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
    if (p.z.slots) {
        char *base = static_cast<char *>(ws);
        parts.meta = reinterpret_cast<int2 *>(base);
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
