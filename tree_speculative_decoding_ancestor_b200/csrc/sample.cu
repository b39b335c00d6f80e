// Tokens from filtered logits and given uniforms.
//
// One row of logits l, temperature T: w_i = exp((l_i - max l) / T).  The kept
// set is the top_k largest entries, of these the smallest prefix (in
// descending order) that holds top_p of their sum, of these the entries with
// w_i >= min_p; equal logits are ordered by token id.  p is w over the kept
// set's sum, and draw s is the smallest kept i whose ascending cumulative sum
// of p exceeds u_s.
//
// Weights are held as integers, w_i = round(2^s exp(..)) with V 2^s <= 2^63:
// every sum is exact, so its value does not depend on the order in which the
// threads and atomics add, and the thresholds and draws of two runs are equal
// by construction.  The exponentials are fp64 (fp32 ones would move a CDF
// by 1e-7 and with it one draw in some thousands); the rounding to 2^-s
// (s = 46 at V = 128256) moves it by about 1e-11.
//
// A row belongs to a cluster of C CTAs; each loads its chunk of the row once
// into shared memory, and every later pass reads it there.
//   1  the largest logit, and a bound below which no entry can be kept: the
//      threads are grouped into at least top_k groups, and the smallest of the
//      groups' largest logits has at least top_k entries at or above it
//      (top_p alone: one thread per group, and the bound holds if the mass
//      above it turns out to reach top_p)
//   2  each warp lists the entries at or above the bound in its segment of the
//      chunk, in token order; with top_k = 50 of 32000 that leaves about 2%,
//      and the passes below walk these lists
//   3  a histogram of the listed entries over 1024 equal steps of the logit:
//      count and mass per step, added up over the cluster; a scan finds the
//      step in which the k-th entry, or the top_p mass, falls
//   4  that step's entries (usually a few) are gathered, and every entry sums
//      the count and mass in front of it; the one at which the limit is
//      passed is the threshold, as a 64-bit (logit, token id) key.  More than
//      kList entries: the same histogram over the keys' range inside the
//      step, ten bits of the key a round, until few are left -- keys are
//      distinct, so this ends also when all logits are equal
//   5  the kept sums of each warp's segment, from them each draw's segment,
//      which its warp walks; the probabilities of the kept entries, over zeros
//      that were written while the row was being searched
// Bound: the read of the logits and the write of the probabilities; for rows
// cut by top_p alone, or not at all, the fp64 exponentials of all entries.
#include <algorithm>
#include <atomic>

#include "cluster_xchg.cuh"
#include "fp64_exp.cuh"
#include "tsd_common.cuh"

namespace tsd {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2 * kThreads;     // steps of a histogram
constexpr int kList = 512;              // entries gathered at most
constexpr int kMaxCluster = 8;
constexpr int kMaxChunk = 45056;        // logits of a CTA, 176 KB of shared memory
constexpr int kListChunk = 40000;       // up to here there is room for the warps' lists
constexpr float kReach = 40.f;          // e^-40 2^s < 1/2: weights from there on are 0

typedef unsigned long long u64;

struct Shared {
    double table[kExpTable];
    u64 mass[kBins];
    uint32_t count[kBins];
    u64 key[kList], weight[kList];      // gathered entries of this CTA
    u64 all_key[kList], all_weight[kList];
    u64 warp_sum[kWarps];
    u64 scan_mass[kWarps];
    uint32_t scan_count[kWarps];
    float warp_hi[kWarps], warp_bound[kWarps];
    float hi, bound;                    // the CTA's largest logit and bound
    u64 rest;                           // the CTA's mass below the bound
    u64 key_hi, key_lo;                 // of the entries in question
    uint32_t listed;
    // the step (or entry) a search ended at
    u64 found_mass, found_before_mass, found_key;
    uint32_t found_bin, found_count, found_before;
};

__device__ __forceinline__ u64 remote_u64(const void *p, uint32_t rank)
{
    u64 v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];"
                 : "=l"(v)
                 : "r"(cluster_map(xchg_smem_addr(p), rank))
                 : "memory");
    return v;
}

__device__ __forceinline__ uint32_t remote_u32(const void *p, uint32_t rank)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];"
                 : "=r"(v)
                 : "r"(cluster_map(xchg_smem_addr(p), rank))
                 : "memory");
    return v;
}

// Larger logit first, then lower token id: descending order of this key.
__device__ __forceinline__ u64 order_key(float l, uint32_t token)
{
    uint32_t u = __float_as_uint(l);
    u ^= (u >> 31) ? 0xffffffffu : 0x80000000u;
    return ((u64)u << 32) | (0xffffffffu - token);
}

struct Row {
    const float *l;       // this CTA's logits (shared memory)
    int n, first;         // how many, and the token id of the first
    int C, rank;
    float top;            // the row's largest logit
    double inv_t;
    float step;           // histogram steps per logit unit
    // what this warp walks: its segment [s0, s1), or `listed` entries of it
    const uint16_t *list;
    int s0, s1, listed;   // listed < 0: the whole segment

    __device__ __forceinline__ int entries() const { return listed < 0 ? s1 - s0 : listed; }
    __device__ __forceinline__ int entry(int i) const { return s0 + (listed < 0 ? i : list[i]); }

    __device__ __forceinline__ u64 weight(float x, const double *table) const
    {
        const double d = x == top ? 0.0 : ((double)x - (double)top) * inv_t;   // inf - inf
        return __double2ull_rn(table_exp(d, table));
    }
    // Where x falls on the scale of histogram steps; kBins and above: out of
    // reach, weight 0.
    __device__ __forceinline__ float place(float x) const
    {
        return x == top ? 0.f : (top - x) * step;
    }
};

// The histogram of every CTA added up: thread t has steps 2t and 2t + 1 with
// what lies in front of each.
struct Scan {
    u64 mass[2], before_mass[2];
    uint32_t count[2], before[2];
};

__device__ __forceinline__ void combine_and_scan(Shared &sh, int C, Scan &sc,
                                                 bool with_rest = false, u64 *rest = nullptr)
{
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    cluster_sync_all();   // the histograms are complete
    if (with_rest) {
        u64 all = 0;
        for (int r = 0; r < C; ++r)
            all += remote_u64(&sh.rest, r);
        *rest = all;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        sc.mass[i] = 0;
        sc.count[i] = 0;
        for (int r = 0; r < C; ++r) {
            sc.mass[i] += remote_u64(&sh.mass[2 * t + i], r);
            sc.count[i] += remote_u32(&sh.count[2 * t + i], r);
        }
    }
    u64 m = sc.mass[0] + sc.mass[1];
    uint32_t c = sc.count[0] + sc.count[1];
    const u64 own_m = m;
    const uint32_t own_c = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 pm = __shfl_up_sync(0xffffffffu, m, o);
        const uint32_t pc = __shfl_up_sync(0xffffffffu, c, o);
        if (lane >= o) {
            m += pm;
            c += pc;
        }
    }
    if (lane == 31) {
        sh.scan_mass[warp] = m;
        sh.scan_count[warp] = c;
    }
    __syncthreads();
    m -= own_m;
    c -= own_c;
    for (int w = 0; w < warp; ++w) {
        m += sh.scan_mass[w];
        c += sh.scan_count[w];
    }
    sc.before_mass[0] = m;
    sc.before[0] = c;
    sc.before_mass[1] = m + sc.mass[0];
    sc.before[1] = c + sc.count[0];
    cluster_sync_all();   // every CTA has read the histograms: they may be reused
}

// Where the limit (an entry count, or a mass) falls; sh.found_* for all.
// Some step holds it: 0 < limit <= the total.
__device__ __forceinline__ void find_step(Shared &sh, const Scan &sc, bool by_mass, u64 limit)
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const bool here = by_mass ? sc.before_mass[i] < limit &&
                                        limit <= sc.before_mass[i] + sc.mass[i]
                                  : sc.before[i] < limit && limit <= sc.before[i] + sc.count[i];
        if (here) {
            sh.found_bin = 2 * threadIdx.x + i;
            sh.found_before = sc.before[i];
            sh.found_before_mass = sc.before_mass[i];
            sh.found_count = sc.count[i];
            sh.found_mass = sc.mass[i];
        }
    }
    __syncthreads();
}

// The entry of step `bin` (found_count entries behind found_before and
// found_before_mass) at which the limit is passed.  Returns its key, and in
// mass_incl the mass up to and including it.
__device__ u64 resolve(Shared &sh, const Row &row, int bin, bool by_mass, u64 limit, u64 *mass_incl)
{
    const int lane = threadIdx.x & 31, n_mine = row.entries();
    const float from = (float)bin, to = (float)(bin + 1);
    auto in_step = [&](float x) {
        const float f = row.place(x);
        return f >= from && f < to;
    };
    u64 lo = 0, hi = ~0ull;   // keys in question
    uint32_t count = sh.found_count, before = sh.found_before;
    u64 before_mass = sh.found_before_mass;
    __syncthreads();
    while (count > (uint32_t)kList) {
        if (threadIdx.x == 0) {
            sh.key_hi = 0;
            sh.key_lo = ~0ull;
        }
        __syncthreads();
        u64 khi = 0, klo = ~0ull;
        for (int e = lane; e < n_mine; e += 32) {
            const int i = row.entry(e);
            const float x = row.l[i];
            if (!in_step(x))
                continue;
            const u64 k = order_key(x, row.first + i);
            if (k < lo || k > hi)
                continue;
            khi = max(khi, k);
            klo = min(klo, k);
        }
        atomicMax(&sh.key_hi, khi);
        atomicMin(&sh.key_lo, klo);
        for (int i = threadIdx.x; i < kBins; i += kThreads) {
            sh.mass[i] = 0;
            sh.count[i] = 0;
        }
        cluster_sync_all();
        for (int r = 0; r < row.C; ++r) {
            khi = max(khi, remote_u64(&sh.key_hi, r));
            klo = min(klo, remote_u64(&sh.key_lo, r));
        }
        hi = khi;
        lo = klo;
        const int shift = max(0, 64 - __clzll((long long)(hi - lo)) - 10);   // 1024 steps
        for (int e = lane; e < n_mine; e += 32) {
            const int i = row.entry(e);
            const float x = row.l[i];
            if (!in_step(x))
                continue;
            const u64 k = order_key(x, row.first + i);
            if (k < lo || k > hi)
                continue;
            const int s = (int)((hi - k) >> shift);
            atomicAdd(&sh.count[s], 1u);
            atomicAdd(&sh.mass[s], row.weight(x, sh.table));
        }
        Scan sc;
        combine_and_scan(sh, row.C, sc);
        find_step(sh, sc, by_mass, by_mass ? limit - before_mass : limit - before);
        hi -= (u64)sh.found_bin << shift;
        lo = max(lo, hi - (((u64)1 << shift) - 1));
        count = sh.found_count;
        before += sh.found_before;
        before_mass += sh.found_before_mass;
        __syncthreads();
    }
    if (threadIdx.x == 0)
        sh.listed = 0;
    __syncthreads();
    for (int e = lane; e < n_mine; e += 32) {
        const int i = row.entry(e);
        const float x = row.l[i];
        if (!in_step(x))
            continue;
        const u64 k = order_key(x, row.first + i);
        if (k < lo || k > hi)
            continue;
        const uint32_t at = atomicAdd(&sh.listed, 1u);
        sh.key[at] = k;
        sh.weight[at] = row.weight(x, sh.table);
    }
    cluster_sync_all();
    int n = 0;
    for (int r = 0; r < row.C; ++r) {
        const int m = (int)remote_u32(&sh.listed, r);
        for (int i = threadIdx.x; i < m; i += kThreads) {
            sh.all_key[n + i] = remote_u64(&sh.key[i], r);
            sh.all_weight[n + i] = remote_u64(&sh.weight[i], r);
        }
        n += m;
    }
    cluster_sync_all();   // lists read everywhere (and all_* complete here)
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const u64 k = sh.all_key[i], w = sh.all_weight[i];
        u64 m = before_mass;
        uint32_t c = before;
        for (int j = 0; j < n; ++j) {
            const bool ahead = sh.all_key[j] > k;
            c += ahead ? 1u : 0u;
            m += ahead ? sh.all_weight[j] : 0ull;
        }
        if (by_mass ? m < limit && limit <= m + w : c + 1 == limit) {
            sh.found_key = k;
            sh.found_mass = m + w;
        }
    }
    __syncthreads();
    *mass_incl = sh.found_mass;
    return sh.found_key;
}

// Each lane's 4 consecutive entries from i on that are at or above the bound,
// appended to the warp's list in token order.  Returns the list's new length.
__device__ __forceinline__ int append(const float4 &x, int i, int left, float bound, uint16_t *list,
                                      int at, int room)
{
    const uint32_t below = (1u << (threadIdx.x & 31)) - 1u;
    const bool c0 = left > 0 && x.x >= bound, c1 = left > 1 && x.y >= bound;
    const bool c2 = left > 2 && x.z >= bound, c3 = left > 3 && x.w >= bound;
    if (!__any_sync(0xffffffffu, c0 | c1 | c2 | c3))
        return at;
    const uint32_t b0 = __ballot_sync(0xffffffffu, c0), b1 = __ballot_sync(0xffffffffu, c1);
    const uint32_t b2 = __ballot_sync(0xffffffffu, c2), b3 = __ballot_sync(0xffffffffu, c3);
    int p = at + __popc(b0 & below) + __popc(b1 & below) + __popc(b2 & below) + __popc(b3 & below);
    if (c0 && p < room)
        list[p] = (uint16_t)i;
    p += c0;
    if (c1 && p < room)
        list[p] = (uint16_t)(i + 1);
    p += c1;
    if (c2 && p < room)
        list[p] = (uint16_t)(i + 2);
    p += c2;
    if (c3 && p < room)
        list[p] = (uint16_t)(i + 3);
    return at + __popc(b0) + __popc(b1) + __popc(b2) + __popc(b3);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2)
    sample_kernel(SampleArgs a, int C, int chunk, double scale)
{
    extern __shared__ uint4 smem_raw[];
    // the chunk (a multiple of 128 logits), the warps' lists, the rest
    float *l = reinterpret_cast<float *>(smem_raw);
    uint16_t *lists = reinterpret_cast<uint16_t *>(l + chunk);
    const int room = chunk <= kListChunk ? chunk / kWarps / 2 : 0;   // of a warp's list
    Shared &sh = *reinterpret_cast<Shared *>(lists + room * kWarps);
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    Row row;
    row.C = C;
    row.rank = (int)cluster_ctarank();
    const long long r = blockIdx.x / C;
    row.l = l;
    row.first = row.rank * chunk;
    row.n = max(0, min(chunk, a.V - row.first));
    const int seg = chunk / kWarps;
    row.s0 = min(warp * seg, row.n);
    row.s1 = min(row.s0 + seg, row.n);
    row.listed = -1;
    uint16_t *const list = lists + warp * room;
    row.list = list;

    float T_ = a.temperature ? a.temperature[r] : 1.f;
    int top_k = a.top_k ? a.top_k[r] : 0;
    float top_p = a.top_p ? a.top_p[r] : 1.f;
    float min_p = a.min_p ? a.min_p[r] : 0.f;
    bool bad = !(T_ >= 0.f && T_ <= 1e30f) || top_p != top_p || min_p != min_p;
    if (T_ == 0.f) {   // the largest logit, lowest token id
        T_ = 1.f;
        top_k = 1;
        top_p = 1.f;
        min_p = 0.f;
    }
    top_k = top_k >= a.V ? 0 : max(top_k, 0);
    const bool cut = top_k > 0 || top_p < 1.f;

    // 1: the chunk into shared memory; NaN counts as -inf, -0 as +0
    const T *src = static_cast<const T *>(a.logits) + r * a.ld + row.first;
    float hi = -INFINITY;
    auto clean = [&](float x) {
        x = fmaxf(x, -INFINITY) + 0.f;
        hi = fmaxf(hi, x);
        return x;
    };
    constexpr int N = 16 / sizeof(T);
    int done = 0;
    if ((reinterpret_cast<uintptr_t>(src) & 15u) == 0) {   // whole 16-byte vectors
        const int nv = row.n / N;
#pragma unroll 4
        for (int i = t; i < nv; i += kThreads) {
            union {
                uint4 raw;
                T e[N];
            } x;
            x.raw = __ldg(reinterpret_cast<const uint4 *>(src) + i);
#pragma unroll
            for (int j = 0; j < N; j += 4)
                *reinterpret_cast<float4 *>(l + i * N + j) =
                    make_float4(clean(to_float(x.e[j])), clean(to_float(x.e[j + 1])),
                                clean(to_float(x.e[j + 2])), clean(to_float(x.e[j + 3])));
        }
        done = nv * N;
    }
    for (int i = done + t; i < row.n; i += kThreads)
        l[i] = clean(to_float(src[i]));
    float *const probs = a.probs ? a.probs + r * a.probs_ld + row.first : nullptr;
    const bool sparse = cut || min_p > 0.f || bad;
    if (probs && sparse) {   // most stay 0: written while the row is searched
        int from = row.s0;
        if ((reinterpret_cast<uintptr_t>(probs) & 15u) == 0) {
            for (int i = row.s0 + 4 * lane; i + 3 < row.s1; i += 128)
                *reinterpret_cast<float4 *>(probs + i) = make_float4(0.f, 0.f, 0.f, 0.f);
            from += (row.s1 - row.s0) & ~3;
        }
        for (int i = from + lane; i < row.s1; i += 32)
            probs[i] = 0.f;
    }
    fill_exp_table(sh.table, scale);
    for (int i = t; i < kBins; i += kThreads) {
        sh.mass[i] = 0;
        sh.count[i] = 0;
    }
    // groups of g threads, at least top_k of them in the cluster
    int g = top_k > 0 ? 32 : 1;
    while (g > 1 && C * kThreads / g < top_k)
        g >>= 1;
    float bound = hi;
    for (int o = 1; o < g; o <<= 1)
        bound = fmaxf(bound, __shfl_xor_sync(0xffffffffu, bound, o));
    bound = cut && top_k <= C * kThreads ? -warp_max(-bound) : -INFINITY;
    hi = warp_max(hi);
    if (lane == 0) {
        sh.warp_hi[warp] = hi;
        sh.warp_bound[warp] = bound;
    }
    __syncthreads();
    if (t == 0) {
        for (int w = 1; w < kWarps; ++w) {
            hi = fmaxf(hi, sh.warp_hi[w]);
            bound = fminf(bound, sh.warp_bound[w]);
        }
        sh.hi = hi;
        sh.bound = bound;
    }
    cluster_sync_all();
    for (int q = 0; q < C; ++q) {
        hi = fmaxf(hi, __uint_as_float(remote_u32(&sh.hi, q)));
        bound = fminf(bound, __uint_as_float(remote_u32(&sh.bound, q)));
    }
    row.top = hi;
    bad = bad || !(hi > -INFINITY);
    if (bad) {   // the same on every CTA of the cluster
        if (row.rank == 0) {
            if (t == 0)
                flag(a.dev_status, TSD_DEV_BAD_ROW);
            for (int s = t; s < a.S; s += kThreads)
                a.tokens[r * a.S + s] = -1;
        }
        for (int i = row.s0 + lane; probs && !sparse && i < row.s1; i += 32)
            probs[i] = 0.f;
        cluster_sync_all();   // no CTA leaves while a peer reads its extremes
        return;
    }
    row.inv_t = 1.0 / (double)T_;

    // 2 .. 4: the threshold
    u64 threshold = 0;      // kept: keys from here up
    float keep_from = -INFINITY;   // and so logits from here up
    while (cut) {
        const bool with_mass = top_p < 1.f, with_rest = with_mass && top_k == 0;
        const bool all = !(bound > -INFINITY);
        row.step = (float)(kBins - 1) / fmaxf(fminf(hi - bound, kReach * T_), 1e-30f);
        u64 rest = 0;
        row.listed = -1;
        if (!all) {
            int at = 0;
            for (int i0 = row.s0; i0 < row.s1; i0 += 128) {
                const int i = i0 + 4 * lane, left = row.s1 - i;
                const float4 x = left > 0 ? *reinterpret_cast<const float4 *>(l + i)
                                          : make_float4(0.f, 0.f, 0.f, 0.f);
                at = append(x, i - row.s0, left, bound, list, at, room);
                if (with_rest) {
                    rest += left > 0 && x.x < bound ? row.weight(x.x, sh.table) : 0;
                    rest += left > 1 && x.y < bound ? row.weight(x.y, sh.table) : 0;
                    rest += left > 2 && x.z < bound ? row.weight(x.z, sh.table) : 0;
                    rest += left > 3 && x.w < bound ? row.weight(x.w, sh.table) : 0;
                }
            }
            row.listed = at <= room ? at : -1;
            __syncwarp();
        }
        for (int e = lane; e < row.entries(); e += 32) {
            const float x = l[row.entry(e)];
            const float f = row.place(x);
            if (x < bound || !(f < (float)kBins))
                continue;
            atomicAdd(&sh.count[(int)f], 1u);
            if (with_mass)
                atomicAdd(&sh.mass[(int)f], row.weight(x, sh.table));
        }
        if (with_rest) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                rest += __shfl_xor_sync(0xffffffffu, rest, o);
            if (lane == 0)
                sh.warp_sum[warp] = rest;
            __syncthreads();
            if (t == 0) {
                rest = 0;
                for (int w = 0; w < kWarps; ++w)
                    rest += sh.warp_sum[w];
                sh.rest = rest;
            }
        }
        Scan sc;
        combine_and_scan(sh, C, sc, with_rest, &rest);
        if (t == kThreads - 1) {
            sh.found_count = sc.before[1] + sc.count[1];
            sh.found_mass = sc.before_mass[1] + sc.mass[1];
        }
        __syncthreads();
        const u64 above = sh.found_mass;
        u64 total = above + (with_rest ? rest : 0);
        const uint32_t entries = sh.found_count;
        __syncthreads();
        if (top_k > 0 && (uint32_t)top_k < entries) {
            find_step(sh, sc, false, (u64)top_k);
            threshold = resolve(sh, row, (int)sh.found_bin, false, (u64)top_k, &total);
            __syncthreads();
        }
        if (with_mass) {
            const u64 want = (u64)fmax(ceil((double)top_p * (double)total), 1.0);
            const u64 limit = min(max(want, (u64)1), total);
            if (top_k == 0 && limit > above) {   // the mass above the bound is short of top_p
                bound = -INFINITY;
                for (int i = t; i < kBins; i += kThreads) {
                    sh.mass[i] = 0;
                    sh.count[i] = 0;
                }
                __syncthreads();
                continue;
            }
            find_step(sh, sc, true, limit);
            u64 incl;
            threshold = resolve(sh, row, (int)sh.found_bin, true, limit, &incl);
            __syncthreads();
        }
        break;
    }
    if (!cut)
        row.step = (float)(kBins - 1) / fmaxf(kReach * T_, 1e-30f);
    if (threshold) {   // the logit of the threshold's key
        const uint32_t u = (uint32_t)(threshold >> 32);
        keep_from = __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xffffffffu));
    }

    // 5: kept sums of the warps' segments
    const u64 floor_w = (u64)ceil((double)fminf(fmaxf(min_p, 0.f), 1.f) * scale);
    if (min_p > 0.f)   // no logit below this one (a step's width of margin) has weight min_p
        keep_from = fmaxf(keep_from, __double2float_rd((double)hi + (double)T_ *
                                                       (log((double)fminf(min_p, 1.f)) - 1e-3)));
    auto kept = [&](int i) -> u64 {   // the weight of entry i, 0 if it is not kept
        const float x = l[i];
        if (x < keep_from || !(x > -INFINITY) || order_key(x, row.first + i) < threshold)
            return 0;
        const u64 w = row.weight(x, sh.table);
        return w >= floor_w ? w : 0;
    };
    const int n_mine = row.entries();
    u64 sum = 0;
    for (int e = lane; e < n_mine; e += 32)
        sum += kept(row.entry(e));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncthreads();   // warp_sum's last readers are done
    if (lane == 0)
        sh.warp_sum[warp] = sum;
    cluster_sync_all();
    u64 total = 0, before = 0;   // of the row, and in front of this warp's segment
    for (int i = lane; i < C * kWarps; i += 32) {
        const u64 w = remote_u64(&sh.warp_sum[i % kWarps], i / kWarps);
        total += w;
        before += i < row.rank * kWarps + warp ? w : 0;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        total += __shfl_xor_sync(0xffffffffu, total, o);
        before += __shfl_xor_sync(0xffffffffu, before, o);
    }
    for (int s = 0; s < a.S; ++s) {
        const double x = a.u[r * a.S + s] * (double)total;
        const u64 at = x > 0.0 ? min((u64)x, total - 1) : 0;   // first cumulative sum above it
        if (at < before || at >= before + sum)
            continue;
        u64 run = before;
        for (int e = 0; e < n_mine; e += 32) {
            u64 c = e + lane < n_mine ? kept(row.entry(e + lane)) : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 p = __shfl_up_sync(0xffffffffu, c, o);
                c += lane >= o ? p : 0;
            }
            const uint32_t over = __ballot_sync(0xffffffffu, run + c > at);
            if (over) {
                if (lane == 0)
                    a.tokens[r * a.S + s] = row.first + row.entry(e + __ffs(over) - 1);
                break;
            }
            run += __shfl_sync(0xffffffffu, c, 31);
        }
    }
    if (probs) {
        const double inv = 1.0 / (double)total;
        __syncwarp();   // the zeros of this warp's segment are written
        for (int e = lane; e < n_mine; e += 32) {
            const int i = row.entry(e);
            const u64 w = kept(i);
            if (w || !sparse)
                probs[i] = (float)((double)w * inv);
        }
    }
    cluster_sync_all();   // no CTA leaves while a peer reads its sums
}

// the chunk, half as many 16-bit list entries, the rest
size_t sample_smem(int chunk)
{
    return (size_t)chunk * (chunk <= kListChunk ? 5 : 4) + sizeof(Shared);
}

}  // namespace

int sample_max_vocab() { return kMaxCluster * kMaxChunk; }

int launch_sample(const SampleArgs &a, int R, int dtype, int num_sms, cudaStream_t stream)
{
    // CTAs per row: as few as hold the row at two CTAs per SM; more (down to
    // 4096 logits each) while the rows alone leave SMs idle.
    int C = 1;
    while (C < kMaxCluster && (a.V + C - 1) / C > 16384)
        C *= 2;
    while (C < kMaxCluster && (long long)R * C < num_sms && (a.V + C - 1) / C > 4096)
        C *= 2;
    const int chunk = ((a.V + C - 1) / C + 127) & ~127;   // warps' segments of whole vectors
    int log2v = 0;
    while ((1LL << log2v) < a.V)
        ++log2v;
    const int s = std::min(50, 63 - log2v);
    const size_t smem = sample_smem(chunk);
    auto kern = dtype == TSD_BF16 ? sample_kernel<__nv_bfloat16> : sample_kernel<float>;
    constexpr int kMaxDevices = 64;
    static std::atomic<bool> raised[kMaxDevices][2];
    int dev = 0;
    TSD_CUDA_TRY(cudaGetDevice(&dev));
    if (dev < 0 || dev >= kMaxDevices)
        return TSD_ERR_CUDA;
    if (!raised[dev][dtype == TSD_BF16].load()) {
        TSD_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          (int)std::max(sample_smem(kMaxChunk), sample_smem(kListChunk))));
        raised[dev][dtype == TSD_BF16].store(true);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)R * C));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = C;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kern, a, C, chunk, ldexp(1.0, s));
    if (err != cudaSuccess) {
        (void)cudaGetLastError();
        return TSD_ERR_CUDA;
    }
    TSD_LAUNCH_CHECK();
    return TSD_OK;
}

}  // namespace tsd
