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
// into shared memory, and every later pass reads it there, a segment to each
// warp.  Four CTAs of 256 threads share an SM: a search is a chain of short
// dependent steps, and the others' passes fill its waits.  (1024 rows of 32000
// with mixed settings: 259 us; before the guess of step 3, 276, and then 293 us
// as two CTAs of 512 threads, 450 to 650 us where the passes read the row from
// L2 instead and twice as many rows are in flight.)
//   1  the largest logit, and with top_k a bound below which no entry can be
//      kept: the threads' largest logits are sorted; the (top_k / C)-th of each
//      CTA's 256, the least of them over the cluster, has at least top_k
//      entries at or above it, and not many more
//   2  the entries at or above the bound are listed (top_k = 50 of 32000: some
//      60).  At most kList of them in the row: every CTA sorts them, and one
//      scan of their weights answers top_k, top_p and min_p; sorted by token
//      id, another scan answers the draws.  Otherwise:
//   3  a histogram of the entries above the bound over 256 equal steps of the
//      logit: count and mass per step, added up over the cluster; a scan finds
//      the step in which the k-th entry, or the top_p mass, falls.  For top_p
//      alone the steps cover what a guess is worth: a histogram of fp32 weights
//      (one add an entry instead of four) says about where the mass falls, and
//      the exact masses above and below the steps around that are summed in
//      registers.  If the limit is not among the steps after all, they are laid
//      over the whole reach and the pass is repeated.  (1024 rows of 32000, top_p
//      0.9 of twice normal logits: 308 us; 458 with steps over what the least of
//      the threads' largest logits bounds, which is often short of top_p)
//   4  that step's entries (usually some tens) are listed and sorted; the one
//      at which the limit is passed is the threshold, as a 64-bit (logit,
//      token id) key.  More than kList entries: the same histogram over the
//      keys' range inside the step, eight bits of the key a round, until few
//      are left -- keys are distinct, so this ends also when all logits are
//      equal
//   5  the probabilities, and the kept sums of each warp's segment; from them
//      each draw's segment, which its warp walks
// Bound: the read of the logits and the write of the probabilities; for rows
// cut by top_p alone, or not at all, the exponentials of all entries; the chain of
// a search's steps.  Rows off a 16-byte boundary (most rows of an odd vocabulary) are
// loaded and stored element by element: 1024 rows of 50257 fp32 498 us, of 50304 467.
#include <algorithm>
#include <atomic>

#include "cluster_xchg.cuh"
#include "fp64_exp.cuh"
#include "tsd_common.cuh"

namespace tsd {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = kThreads;         // steps of a histogram, one per thread
constexpr int kList = kThreads;         // entries listed at most, one per thread
constexpr int kListTop = kThreads / 2;  // top_k / C up to which listing is tried: about
                                        // -256 ln(1 - top_k / (256 C)) entries of a CTA pass
constexpr int kMaxCluster = 8;
constexpr int kMaxChunk = 49152;        // logits of a CTA, 192 KB of shared memory
constexpr float kReach = 40.f;          // e^-40 2^s < 1/2: weights from there on are 0
constexpr int kGuessBins = 4 * kThreads;   // steps of the guess, four per thread
constexpr float kGuessReach = 12.f;        // e^-12 2^16 < 1/2: guessed weights from there on are 0

typedef unsigned long long u64;

struct Shared {
    double table[kExpTable];
    union {
        // Count and mass per step.  A 64-bit add in shared memory is a
        // compare-and-swap loop, so the mass is kept as three sums of 16, 16
        // and the remaining bits of the weights: with V 2^s <= 2^63 none
        // overflows.
        uint32_t hist[4][kBins];
        u64 by_rank[kList];             // weights, then cumulative sums
    };
    u64 key[kList];                     // listed entries of this CTA
    union {
        u64 swap[2][kThreads];          // of the sorts
        uint4 guess[kThreads];          // guessed mass per step
    };
    u64 warp_sum[kWarps], warp_over[kWarps], scan_mass[kWarps];
    float warp_hi[kWarps];
    float hi, bound;                    // the CTA's largest logit and bound
    u64 over, rest;                     // the CTA's mass above and below the steps
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

__device__ __forceinline__ uint4 remote_uint4(const void *p, uint32_t rank)
{
    uint4 v;
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
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

__device__ __forceinline__ float key_logit(u64 key)
{
    const uint32_t u = (uint32_t)(key >> 32);
    return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ uint32_t key_token(u64 key) { return 0xffffffffu - (uint32_t)key; }

// The chunk of the row in shared memory, in the logits' own type, as this warp
// sees it.
template <typename T> struct Row {
    const T *l;           // the chunk (-inf behind its end, up to a multiple of four)
    int first;            // token id of its first logit
    int s0, s1;           // this warp's segment (s0 a multiple of four)
    int C, rank;
    bool deep;            // logits so large that top - 45 T is no float next to it
    float top, low;       // the row's largest logit, and one whose weight is 0
    double top_d, per_t;  // weight of x: 2^(((x - top) per_t) / 128)
    float from, step;     // upper end of the histogram's steps, and steps per logit unit
    float bound;          // entries below it are in no step

    // Logits i .. i + 3 (i a multiple of four); -inf beyond the segment.
    __device__ __forceinline__ float4 load(int i) const
    {
        if (i >= s1)
            return make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (sizeof(T) == 4)
            return *reinterpret_cast<const float4 *>(l + i);
        const uint2 v = *reinterpret_cast<const uint2 *>(l + i);   // bf16: the upper halves
        return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                           __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
    }
    // f(i, x) for every four logits x at i of the segment; every lane takes
    // part in every call (i may be at or beyond s1).
    template <typename F> __device__ __forceinline__ void walk(F f) const
    {
        const int lane = threadIdx.x & 31;
        for (int i0 = s0; i0 < s1; i0 += 128)
            f(i0 + 4 * lane, load(i0 + 4 * lane));
    }
    // round(2^s exp((x - top) / T)): a = (x - top) 128 / (T ln 2) = n + r with n
    // an integer, then 2^(n / 128) from the table (scaled by 2^s) and
    // 2^(r / 128) from its series to degree 4 (|r| <= 1/2: 1.3e-15).  Rounded
    // to an integer by adding 2^52 (weights are at most 2^50); the conversion
    // instruction would be slower.
    __device__ __forceinline__ u64 weight(float x, const double *table) const
    {
        constexpr double kRound = 6755399441055744.0;   // 1.5 * 2^52
        constexpr double c1 = 0.6931471805599453 / 128.0, c2 = c1 * c1 / 2.0;
        constexpr double c3 = c1 * c2 / 3.0, c4 = c1 * c3 / 4.0;
        double a = ((double)fmaxf(x, low) - top_d) * per_t;
        if (deep)   // low is -inf
            a = fmax(a, -45.0 * 184.6649652337873);
        const double sum = a + kRound;
        const double r = a - (sum - kRound);
        const int n = __double2loint(sum);
        const double p = r * fma(r, fma(r, fma(r, c4, c3), c2), c1);
        const double t = table[n & (kExpTable - 1)];
        const double y = __hiloint2double(__double2hiint(fma(t, p, t)) + ((n >> 7) << 20),
                                          __double2loint(fma(t, p, t)));
        return (u64)__double_as_longlong(y + 4503599627370496.0) & 0xfffffffffffffull;
    }
    // Where x falls on the scale of histogram steps: below 0 above them, from
    // kBins on below them (with the whole reach: weight 0).
    __device__ __forceinline__ float place(float x) const { return (from - x) * step; }
};

__device__ __forceinline__ void mass_in(Shared &sh, int step, u64 w)
{
    atomicAdd(&sh.hist[1][step], (uint32_t)w & 0xffffu);
    atomicAdd(&sh.hist[2][step], (uint32_t)(w >> 16) & 0xffffu);
    atomicAdd(&sh.hist[3][step], (uint32_t)(w >> 32));
}

__device__ __forceinline__ void count_in(Shared &sh, int step) { atomicAdd(&sh.hist[0][step], 1u); }

__device__ __forceinline__ void clear_hist(Shared &sh)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        sh.hist[i][threadIdx.x] = 0u;
}

// The histogram of every CTA added up: thread t has step t with what lies in
// front of it.
struct Scan {
    u64 mass, before_mass;
    uint32_t count, before;
};

// Inclusive sums of v over the threads in front of and including this one;
// `total` of all.  Ends with a barrier behind the last read.
__device__ __forceinline__ u64 block_scan(Shared &sh, u64 v, u64 &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 p = __shfl_up_sync(0xffffffffu, v, o);
        v += lane >= o ? p : 0;
    }
    if (lane == 31)
        sh.scan_mass[warp] = v;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const u64 m = sh.scan_mass[w];
        v += w < warp ? m : 0;
        total += m;
    }
    __syncthreads();
    return v;
}

// Peers may read this CTA's histogram until the next cluster barrier.
__device__ __forceinline__ void combine_and_scan(Shared &sh, int C, Scan &sc)
{
    const int t = threadIdx.x;
    cluster_sync_all();   // the histograms are complete
    sc.mass = 0;
    sc.count = 0;
#pragma unroll 1
    for (int r = 0; r < C; r += 4) {
        uint32_t h[4][4];   // sixteen remote loads in flight
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                h[i][k] = r + i < C ? remote_u32(&sh.hist[k][t], r + i) : 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            sc.mass += (u64)h[i][1] + ((u64)h[i][2] << 16) + ((u64)h[i][3] << 32);
            sc.count += h[i][0];
        }
    }
    u64 total;
    sc.before_mass = block_scan(sh, sc.mass, total) - sc.mass;
    sc.before = (uint32_t)block_scan(sh, sc.count, total) - sc.count;
}

// Where the limit (an entry count, or a mass) falls; sh.found_* for all.
// Some step holds it: 0 < limit <= the total.
__device__ __forceinline__ void find_step(Shared &sh, const Scan &sc, bool by_mass, u64 limit)
{
    const bool here = by_mass ? sc.before_mass < limit && limit <= sc.before_mass + sc.mass
                              : sc.before < limit && limit <= sc.before + sc.count;
    if (here) {
        sh.found_bin = threadIdx.x;
        sh.found_before = sc.before;
        sh.found_before_mass = sc.before_mass;
        sh.found_count = sc.count;
        sh.found_mass = sc.mass;
    }
    __syncthreads();
}

// Bitonic sort, descending, of one key per thread; n of them count, the others
// are 0.  Strides within a warp are shuffles; warps of zeros only keep step.
__device__ __forceinline__ u64 sort_descending(Shared &sh, u64 v, int n)
{
    const int t = threadIdx.x;
    const int n2 = n > 1 ? 1 << (32 - __clz(n - 1)) : 1;   // what the network spans
    const bool active = (t & ~31) < n2;
    int buf = 0;
    __syncthreads();   // the buffers' last readers are done
#pragma unroll
    for (int size = 2; size <= kThreads; size <<= 1) {
        if (size > n2)
            break;
#pragma unroll
        for (int stride = size >> 1; stride > 0; stride >>= 1) {
            if (stride >= 32) {   // two buffers: one barrier an exchange
                sh.swap[buf][t] = v;
                __syncthreads();
                const u64 w = sh.swap[buf][t ^ stride];
                buf ^= 1;
                v = (((t & stride) == 0) == ((t & size) == 0)) == (v > w) ? v : w;
            } else if (active) {
                const u64 w = __shfl_xor_sync(0xffffffffu, v, stride);
                v = (((t & stride) == 0) == ((t & size) == 0)) == (v > w) ? v : w;
            }
        }
    }
    return v;
}

// The q-th largest of the threads' values (a bitonic sort of them).  Begins
// behind the last readers of sh.swap.
__device__ __forceinline__ float nth_largest(Shared &sh, float v, int q)
{
    const int t = threadIdx.x;
    float *swap = reinterpret_cast<float *>(sh.swap);
    int buf = 0;
#pragma unroll
    for (int size = 2; size <= kThreads; size <<= 1)
#pragma unroll
        for (int stride = size >> 1; stride > 0; stride >>= 1) {
            float w;
            if (stride >= 32) {   // two buffers: one barrier an exchange
                swap[buf + t] = v;
                __syncthreads();
                w = swap[buf + (t ^ stride)];
                buf ^= kThreads;
            } else {
                w = __shfl_xor_sync(0xffffffffu, v, stride);
            }
            v = ((t & stride) == 0) == ((t & size) == 0) ? fmaxf(v, w) : fminf(v, w);
        }
    if (t == q - 1)
        swap[2 * kThreads] = v;
    __syncthreads();
    return swap[2 * kThreads];
}

// A guess at the step (of kGuessBins, of `unit` each, nearest one) in which
// top_p of the row's sum is reached: weights in fp32, rounded to 2^-16 and added
// up as integers (a chunk's are below 2^32), one atomic each.  Peers may read
// sh.guess until the next cluster barrier.
template <typename T>
__device__ __forceinline__ int guess_step(Shared &sh, const Row<T> &row, float top_p, float unit)
{
    constexpr float kInt = 8388608.f;   // 2^23: x + 2^23 holds round(x) in its low bits
    constexpr float kLog2 = -1.4426950408889634f * kGuessReach / kGuessBins;
    uint32_t *const sums = &sh.guess[0].x;
    const int t = threadIdx.x;
    const float per = 1.f / unit;
    row.walk([&](int, const float4 &x) {
        const float e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float f = (row.top - e[j]) * per;
            if (f < kGuessBins - 1)
                atomicAdd(&sums[__float_as_uint(f + kInt) & (kGuessBins - 1)],
                          __float_as_uint(fmaf(exp2f(f * kLog2), 65536.f, kInt)) & 0x7fffffu);
        }
    });
    cluster_sync_all();   // the sums are complete
    u64 own[4] = {0, 0, 0, 0};   // of steps 4 t .. 4 t + 3
#pragma unroll 1
    for (int r = 0; r < row.C; r += 4) {
        uint4 g[4];   // four remote loads in flight
#pragma unroll
        for (int i = 0; i < 4; ++i)
            g[i] = r + i < row.C ? remote_uint4(&sh.guess[t], r + i) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            own[0] += g[i].x;
            own[1] += g[i].y;
            own[2] += g[i].z;
            own[3] += g[i].w;
        }
    }
    const u64 all = own[0] + own[1] + own[2] + own[3];
    u64 total;
    u64 run = block_scan(sh, all, total) - all;
    const u64 want = max((u64)1, (u64)(fmax((double)top_p, 0.0) * (double)total));
    if (run < want && want <= run + all) {
        int k = 0;
        while (k < 3 && run + own[k] < want)
            run += own[k++];
        sh.found_bin = 4 * t + k;
    }
    __syncthreads();
    return (int)sh.found_bin;
}

// Every CTA's listed keys, one per thread (0 beyond their number, n).  The
// lists are complete behind the cluster barrier that this begins with.  More
// than kList: n alone.
__device__ __forceinline__ u64 all_keys(Shared &sh, int C, int &n)
{
    const int lane = threadIdx.x & 31;
    cluster_sync_all();
    uint32_t end = lane < C ? remote_u32(&sh.listed, lane) : 0;   // where a CTA's keys end
#pragma unroll
    for (int o = 1; o < kMaxCluster; o <<= 1) {
        const uint32_t p = __shfl_up_sync(0xffffffffu, end, o);
        end += lane >= o ? p : 0;
    }
    n = (int)min(__shfl_sync(0xffffffffu, end, kMaxCluster - 1), (uint32_t)kList + 1u);
    int r = 0;
    uint32_t from = 0;
#pragma unroll
    for (int q = 0; q < kMaxCluster - 1; ++q) {
        const uint32_t x = __shfl_sync(0xffffffffu, end, q);
        r = threadIdx.x >= x ? q + 1 : r;
        from = threadIdx.x >= x ? x : from;
    }
    return n <= kList && (int)threadIdx.x < n ? remote_u64(&sh.key[threadIdx.x - from], r) : 0;
}

// The entries of four that are chosen, appended to the CTA's list (counted
// beyond its end, too).  Every lane of the warp takes part.
__device__ __forceinline__ void list_in(Shared &sh, const float4 &x, int i, bool c0, bool c1, bool c2,
                                        bool c3)
{
    if (!__any_sync(0xffffffffu, c0 | c1 | c2 | c3))
        return;
    const int lane = threadIdx.x & 31;
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t b0 = __ballot_sync(0xffffffffu, c0), b1 = __ballot_sync(0xffffffffu, c1);
    const uint32_t b2 = __ballot_sync(0xffffffffu, c2), b3 = __ballot_sync(0xffffffffu, c3);
    uint32_t p = 0;
    if (lane == 0)
        p = atomicAdd(&sh.listed, (uint32_t)(__popc(b0) + __popc(b1) + __popc(b2) + __popc(b3)));
    p = __shfl_sync(0xffffffffu, p, 0) + __popc(b0 & below) + __popc(b1 & below) +
        __popc(b2 & below) + __popc(b3 & below);
    if (c0 && p < kList)
        sh.key[p] = order_key(x.x, i);
    p += c0;
    if (c1 && p < kList)
        sh.key[p] = order_key(x.y, i + 1);
    p += c1;
    if (c2 && p < kList)
        sh.key[p] = order_key(x.z, i + 2);
    p += c2;
    if (c3 && p < kList)
        sh.key[p] = order_key(x.w, i + 3);
}

// The entry of step `bin` (found_count entries behind found_before and
// found_before_mass) at which the limit is passed.  Returns its key, and in
// mass_incl the mass up to and including it.  Peers may read this CTA's list
// until the next cluster barrier.
template <typename T>
__device__ __forceinline__ u64 resolve(Shared &sh, const Row<T> &row, int bin, bool by_mass, u64 limit,
                                    u64 *mass_incl)
{
    const float from = (float)bin, to = (float)(bin + 1);
    // keys in question: like the histogram, none below the bound
    u64 lo = order_key(row.bound, 0xffffffffu), hi = ~0ull;
    auto in_question = [&](float x, int i) {
        const float f = row.place(x);
        if (!(f >= from && f < to))
            return false;
        const u64 k = order_key(x, row.first + i);
        return k >= lo && k <= hi;
    };
    uint32_t count = sh.found_count, before = sh.found_before;
    u64 before_mass = sh.found_before_mass;
    __syncthreads();
    while (count > (uint32_t)kList) {
        if (threadIdx.x == 0) {
            sh.key_hi = 0;
            sh.key_lo = ~0ull;
        }
        cluster_sync_all();   // and every CTA has read the last histogram
        u64 khi = 0, klo = ~0ull;
        row.walk([&](int i, const float4 &x) {
            const float e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (in_question(e[j], i + j)) {
                    khi = max(khi, order_key(e[j], row.first + i + j));
                    klo = min(klo, order_key(e[j], row.first + i + j));
                }
        });
        atomicMax(&sh.key_hi, khi);
        atomicMin(&sh.key_lo, klo);
        clear_hist(sh);
        cluster_sync_all();
        for (int r = 0; r < row.C; ++r) {
            khi = max(khi, remote_u64(&sh.key_hi, r));
            klo = min(klo, remote_u64(&sh.key_lo, r));
        }
        hi = khi;
        lo = klo;
        const int shift = max(0, 64 - __clzll((long long)(hi - lo)) - 8);   // 256 steps
        row.walk([&](int i, const float4 &x) {
            const float e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (in_question(e[j], i + j)) {
                    const int s = (int)((hi - order_key(e[j], row.first + i + j)) >> shift);
                    count_in(sh, s);
                    mass_in(sh, s, row.weight(e[j], sh.table));
                }
        });
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
    row.walk([&](int i, const float4 &x) {
        list_in(sh, x, row.first + i, in_question(x.x, i), in_question(x.y, i + 1), in_question(x.z, i + 2),
                in_question(x.w, i + 3));
    });
    int n;
    u64 key = all_keys(sh, row.C, n);
    key = sort_descending(sh, key, n);
    const u64 w = key ? row.weight(key_logit(key), sh.table) : 0;
    u64 all;
    const u64 incl = before_mass + block_scan(sh, w, all);
    if (key && (by_mass ? incl - w < limit && limit <= incl : before + threadIdx.x + 1 == limit)) {
        sh.found_key = key;
        sh.found_mass = incl;
    }
    __syncthreads();
    *mass_incl = sh.found_mass;
    const u64 key_found = sh.found_key;
    __syncthreads();
    return key_found;
}

// The mass that top_p of `total` asks for: an entry is kept if less lies in
// front of it.
__device__ __forceinline__ u64 mass_limit(float top_p, u64 total)
{
    const u64 want = (u64)fmax(ceil((double)top_p * (double)total), 1.0);
    return min(max(want, (u64)1), total);
}

// A weight (below 2^52) as a double, without the slow conversion instruction.
__device__ __forceinline__ double weight_double(u64 w)
{
    return __longlong_as_double((long long)(w | 0x4330000000000000ull)) - 4503599627370496.0;
}

// A draw takes the first entry whose cumulative sum exceeds this.
__device__ __forceinline__ u64 draw_at(double u, u64 total)
{
    const double x = u * (double)total;
    return x > 0.0 ? min((u64)x, total - 1) : 0;
}

// Step 2 behind the listing: n keys of the row, one per thread; the kept ones'
// probabilities (over zeros) and the draws.  [first, last) are this CTA's
// tokens, probs its part of the row.
template <typename T>
__device__ __forceinline__ void finish_list(Shared &sh, const SampleArgs &a, const Row<T> &row, u64 key,
                                            int n, int top_k, float top_p, u64 floor_w, long long r,
                                            int first, int last, float *probs)
{
    const int t = threadIdx.x, k = min(top_k, n);
    key = sort_descending(sh, key, n);
    const u64 w = key ? row.weight(key_logit(key), sh.table) : 0;
    u64 all;
    const u64 incl = block_scan(sh, w, all);
    if (t == k - 1)
        sh.found_mass = incl;
    __syncthreads();
    const u64 limit = top_p < 1.f ? mass_limit(top_p, sh.found_mass) : ~0ull;
    // the kept entries are a prefix of the order
    const bool keep = t < k && incl - w < limit && w >= floor_w && w > 0;
    const int kept = __syncthreads_count(keep);
    if (t == kept - 1)
        sh.found_before_mass = incl;
    sh.by_rank[t] = w;
    __syncthreads();
    const u64 total = sh.found_before_mass;
    const int token = (int)key_token(key);
    if (probs && keep && token >= first && token < last &&
        in_bounds(token, a.V, a.dev_status))
        probs[token - first] = (float)((double)w * (1.0 / (double)total));
    if (row.rank != 0 || a.S == 0)
        return;
    // in token order: the complement of (token, rank), descending
    const u64 id = sort_descending(
        sh, keep ? ~(((u64)key_token(key) << 32) | (uint32_t)t) : 0, kept);
    const u64 cum = block_scan(sh, id ? sh.by_rank[(uint32_t)~id] : 0, all);
    sh.by_rank[t] = cum;
    sh.swap[0][t] = ~id >> 32;
    __syncthreads();
    for (int s = t; s < a.S; s += kThreads) {
        const u64 at = draw_at(a.u[r * a.S + s], total);
        int lo = 0, up = kept - 1;   // first cumulative sum above it
        while (lo < up) {
            const int mid = (lo + up) >> 1;
            if (sh.by_rank[mid] > at)
                up = mid;
            else
                lo = mid + 1;
        }
        const int32_t drawn = (int32_t)sh.swap[0][lo];
        if (in_bounds(drawn, a.V, a.dev_status))
            a.tokens[r * a.S + s] = drawn;
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4)
    sample_kernel(SampleArgs a, int C, int steps, double scale)
{
    extern __shared__ float4 smem_raw[];
    Shared &sh = *reinterpret_cast<Shared *>(smem_raw);
    T *const l = reinterpret_cast<T *>(smem_raw + (sizeof(Shared) + 15) / 16);
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const long long r = blockIdx.x / C;
    Row<T> row;
    row.C = C;
    row.rank = (int)cluster_ctarank();
    row.l = l;
    // whole steps of 128 logits, spread evenly over the cluster's warps
    auto begin = [&](int w) {
        return (int)min((long long)steps * w / (C * kWarps) * 128, (long long)a.V);
    };
    const int first = begin(row.rank * kWarps), last = begin((row.rank + 1) * kWarps);
    row.first = first;
    row.s0 = begin(row.rank * kWarps + warp) - first;
    row.s1 = begin(row.rank * kWarps + warp + 1) - first;

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
    float *const probs = a.probs ? a.probs + r * a.probs_ld + first : nullptr;
    const bool probs_vec = (reinterpret_cast<uintptr_t>(probs) & 15u) == 0;
    auto put4 = [&](int i, float p0, float p1, float p2, float p3) {
        if (probs_vec && i + 3 < row.s1) {
            if (in_bounds(first + i + 3, a.V, a.dev_status))
                *reinterpret_cast<float4 *>(probs + i) = make_float4(p0, p1, p2, p3);
            return;
        }
        const float p[4] = {p0, p1, p2, p3};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + j < row.s1 && in_bounds(first + i + j, a.V, a.dev_status))
                probs[i + j] = p[j];
    };
    auto zeros = [&]() {
        for (int i = row.s0 + 4 * lane; i < row.s1; i += 128)
            put4(i, 0.f, 0.f, 0.f, 0.f);
    };

    // 1: the chunk into shared memory, its largest logit and the bound; NaN
    // counts as -inf, -0 as +0
    const T *src = static_cast<const T *>(a.logits) + r * a.ld + first;
    const int n_own = last - first;
    float hi = -INFINITY;
    auto clean = [&](float x) {
        x = fmaxf(x, -INFINITY) + 0.f;
        hi = fmaxf(hi, x);
        return x;
    };
    constexpr int N = 16 / sizeof(T);
    const int room = (steps + C - 1) / C * 128;   // logits that the chunk may hold
    auto fits = [&](int i, int n) {   // logits i .. i + n - 1 of the chunk
        return in_bounds(i + n - 1, room, a.dev_status) &&
               in_bounds(first + i + n - 1, a.V, a.dev_status);
    };
    int done = 0;
    if ((reinterpret_cast<uintptr_t>(src) & 15u) == 0) {   // whole 16-byte vectors
        const int nv = n_own / N;
#pragma unroll 4
        for (int i = t; i < nv; i += kThreads) {
            if (!fits(i * N, N))
                continue;
            union {
                uint4 raw;
                T e[N];
            } x;
            x.raw = __ldg(reinterpret_cast<const uint4 *>(src) + i);
#pragma unroll
            for (int j = 0; j < N; ++j)
                x.e[j] = from_float<T>(clean(to_float(x.e[j])));
            *(reinterpret_cast<uint4 *>(l) + i) = x.raw;
        }
        done = nv * N;
    }
    for (int i = done + t; i < ((n_own + 3) & ~3); i += kThreads)
        if (i < n_own ? fits(i, 1) : in_bounds(i, room, a.dev_status))
            l[i] = from_float<T>(i < n_own ? clean(to_float(src[i])) : -INFINITY);
    fill_exp_table(sh.table, scale);
    clear_hist(sh);
    if (top_k == 0)
        sh.guess[t] = make_uint4(0, 0, 0, 0);
    if (t == 0)
        sh.listed = 0;
    // the bound: the q-th largest of the threads' largest logits, q such that
    // C of these cover top_k
    const int q = (top_k + C - 1) / C;
    float bound = -INFINITY;
    if (top_k > 0 && q <= kThreads)
        bound = nth_largest(sh, hi, q);
    hi = warp_max(hi);
    if (lane == 0)
        sh.warp_hi[warp] = hi;
    __syncthreads();
    hi = warp_max(lane < kWarps ? sh.warp_hi[lane] : -INFINITY);
    if (t == 0) {
        sh.hi = hi;
        sh.bound = bound;
    }
    cluster_sync_all();
    hi = lane < C ? __uint_as_float(remote_u32(&sh.hi, lane)) : -INFINITY;
    bound = lane < C ? __uint_as_float(remote_u32(&sh.bound, lane)) : INFINITY;
    hi = warp_max(hi);
    bound = -warp_max(-bound);
    bad = bad || !(hi > -INFINITY);
    if (bad) {   // the same on every CTA of the cluster
        if (row.rank == 0) {
            if (t == 0)
                flag(a.dev_status, TSD_DEV_BAD_ROW);
            for (int s = t; s < a.S; s += kThreads)
                a.tokens[r * a.S + s] = -1;
        }
        if (probs)
            zeros();
        cluster_sync_all();   // no CTA leaves while a peer reads its extremes
        return;
    }
    if (hi == INFINITY) {   // +inf stands for 0, everything else for -inf
        for (int i = t; i < ((n_own + 3) & ~3); i += kThreads)
            l[i] = from_float<T>(to_float(l[i]) == INFINITY ? 0.f : -INFINITY);
        hi = 0.f;
        bound = -INFINITY;
        __syncthreads();
    }
    row.top = hi;
    row.top_d = (double)hi;
    row.per_t = 184.6649652337873 / (double)T_;   // 128 / ln 2 / T
    row.low = hi - 45.f * T_;
    row.deep = !(fabs((double)hi - (double)row.low - 45.0 * (double)T_) <= (double)T_);
    row.low = row.deep ? -INFINITY : row.low;
    row.from = hi;
    row.step = (float)(kBins - 1) / fmaxf(fminf(hi - bound, kReach * T_), 1e-30f);
    row.bound = bound;
    const u64 floor_w = (u64)ceil((double)fminf(fmaxf(min_p, 0.f), 1.f) * scale);

    // 2: few entries
    if (bound > -INFINITY && q <= kListTop) {
        row.walk([&](int i, const float4 &x) {
            list_in(sh, x, first + i, x.x >= bound, x.y >= bound, x.z >= bound, x.w >= bound);
        });
        if (probs)
            zeros();
        int n;
        const u64 key = all_keys(sh, C, n);
        if (n <= kList) {
            finish_list(sh, a, row, key, n, top_k, top_p, floor_w, r, first, last, probs);
            cluster_sync_all();   // no CTA leaves while a peer reads its list
            return;
        }
    }

    // 3, 4: the threshold
    const bool with_mass = top_p < 1.f, with_rest = with_mass && top_k == 0;
    u64 threshold = 0, total = 0;   // kept: keys from here up
    bool guessed = with_rest;
    if (guessed) {   // the steps: those around the guess, or everything below it near the reach
        const float unit = fmaxf(kGuessReach * T_, 1e-30f) / kGuessBins;
        const int g = guess_step(sh, row, top_p, unit);
        row.from = g > 1 ? hi - ((float)g - 1.5f) * unit : hi;
        const float to = g < kGuessBins - 3 ? hi - ((float)g + 1.5f) * unit : hi - kReach * T_;
        row.step = (float)(kBins - 1) / fmaxf(row.from - to, 1e-30f);
    }
    while (cut) {
        u64 rest = 0, over = 0;
        row.walk([&](int i, const float4 &x) {
            const float e[4] = {x.x, x.y, x.z, x.w};
            u64 w[4] = {0, 0, 0, 0};
            if (with_rest) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[j] = row.weight(e[j], sh.table);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float f = row.place(e[j]);
                if (f < 0.f) {
                    over += w[j];
                } else if (e[j] >= bound && f < (float)kBins) {
                    count_in(sh, (int)f);
                    if (with_mass)
                        mass_in(sh, (int)f, with_rest ? w[j] : row.weight(e[j], sh.table));
                } else {
                    rest += w[j];
                }
            }
        });
        if (with_rest) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                over += __shfl_xor_sync(0xffffffffu, over, o);
                rest += __shfl_xor_sync(0xffffffffu, rest, o);
            }
            if (lane == 0) {
                sh.warp_sum[warp] = rest;
                sh.warp_over[warp] = over;
            }
            __syncthreads();
            if (t == 0) {
                rest = over = 0;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    rest += sh.warp_sum[w];
                    over += sh.warp_over[w];
                }
                sh.rest = rest;
                sh.over = over;
            }
        }
        Scan sc;
        combine_and_scan(sh, C, sc);
        if (t == kThreads - 1) {
            sh.found_count = sc.before + sc.count;
            sh.found_mass = sc.before_mass + sc.mass;
        }
        if (with_rest) {
            rest = lane < C ? remote_u64(&sh.rest, lane) : 0;
            over = lane < C ? remote_u64(&sh.over, lane) : 0;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                rest += __shfl_xor_sync(0xffffffffu, rest, o);
                over += __shfl_xor_sync(0xffffffffu, over, o);
            }
        }
        __syncthreads();
        const u64 within = sh.found_mass;
        const uint32_t entries = sh.found_count;
        total = within + (with_rest ? over + rest : 0);
        __syncthreads();
        // (top_k entries or more lie at or above the bound, so with fewer inside the
        // reach all that have weight are kept; with just as many the last of them is
        // still the threshold, for others lie below the bound)
        if (top_k > 0 && (uint32_t)top_k <= entries) {
            find_step(sh, sc, false, (u64)top_k);
            threshold = resolve(sh, row, (int)sh.found_bin, false, (u64)top_k, &total);
            if (with_mass)
                cluster_sync_all();   // every CTA has read the list
        }
        if (with_mass) {
            const u64 limit = mass_limit(top_p, total) - (with_rest ? over : 0);
            if (guessed && !(0 < (long long)limit && limit <= within)) {   // a wrong guess: all steps
                guessed = false;
                row.from = hi;
                row.step = (float)(kBins - 1) / fmaxf(kReach * T_, 1e-30f);
                cluster_sync_all();   // every CTA has read the others' sums
                clear_hist(sh);
                __syncthreads();
                continue;
            }
            find_step(sh, sc, true, limit);
            threshold = resolve(sh, row, (int)sh.found_bin, true, limit, &total);
            total += with_rest ? over : 0;
        }
        break;
    }

    // 5: probabilities, kept sums of the warps' segments, draws
    float keep_from = threshold ? key_logit(threshold) : -INFINITY;
    // the kept sum is known if top_p was asked for and min_p takes nothing off it
    const bool known = with_mass && threshold &&
                       row.weight(keep_from, sh.table) >= floor_w;
    if (min_p > 0.f)   // no logit below this one (with some margin) has weight min_p
        keep_from = fmaxf(keep_from, __double2float_rd((double)hi + (double)T_ *
                                                       (log((double)fminf(min_p, 1.f)) - 1e-3)));
    // of the entries at keep_from itself those up to the threshold's token
    const int last_tied =
        threshold && keep_from == key_logit(threshold) ? (int)key_token(threshold) - first : a.V;
    auto kept4 = [&](int i, const float4 &x, u64 (&w)[4]) {
        const float e[4] = {x.x, x.y, x.z, x.w};
        bool keep[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            keep[j] = e[j] > keep_from || (e[j] == keep_from && i + j <= last_tied);
            w[j] = 0;
        }
        if (!__any_sync(0xffffffffu, keep[0] | keep[1] | keep[2] | keep[3]))
            return false;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const u64 v = row.weight(e[j], sh.table);
            w[j] = keep[j] ? v : 0;
        }
        if (min_p > 0.f) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[j] = w[j] >= floor_w ? w[j] : 0;
        }
        return true;
    };
    u64 sum = 0;
    auto write = [&](u64 all, bool count) {
        const double inv = 1.0 / (double)all;
        row.walk([&](int i, const float4 &x) {
            u64 w[4];
            if (kept4(i, x, w)) {
                if (count)
                    sum += (w[0] + w[1]) + (w[2] + w[3]);
                if (i < row.s1)
                    put4(i, (float)(weight_double(w[0]) * inv), (float)(weight_double(w[1]) * inv),
                         (float)(weight_double(w[2]) * inv), (float)(weight_double(w[3]) * inv));
            } else if (i < row.s1) {
                put4(i, 0.f, 0.f, 0.f, 0.f);
            }
        });
    };
    const bool at_once = probs && known;
    if (at_once) {
        write(total, true);
    } else {
        row.walk([&](int i, const float4 &x) {
            u64 w[4];
            if (kept4(i, x, w))
                sum += (w[0] + w[1]) + (w[2] + w[3]);
        });
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncthreads();   // warp_sum's last readers are done
    if (lane == 0)
        sh.warp_sum[warp] = sum;
    cluster_sync_all();
    total = 0;
    u64 before = 0;   // in front of this warp's segment
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
    if (probs && !at_once)
        write(total, false);
    for (int s = 0; s < a.S; ++s) {
        const u64 at = draw_at(a.u[r * a.S + s], total);   // first cumulative sum above it
        if (at < before || at >= before + sum)
            continue;
        u64 run = before;
        for (int i0 = row.s0; i0 < row.s1; i0 += 128) {
            const int i = i0 + 4 * lane;
            u64 w[4];
            if (!kept4(i, row.load(i), w))
                continue;
            const u64 own = (w[0] + w[1]) + (w[2] + w[3]);
            u64 c = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 p = __shfl_up_sync(0xffffffffu, c, o);
                c += lane >= o ? p : 0;
            }
            const uint32_t over = __ballot_sync(0xffffffffu, run + c > at);
            if (over) {
                if (lane == __ffs(over) - 1) {
                    u64 m = run + c - own;
                    int j = 0;
                    while (j < 3 && m + w[j] <= at)
                        m += w[j++];
                    if (in_bounds(first + i + j, a.V, a.dev_status))
                        a.tokens[r * a.S + s] = first + i + j;
                }
                break;
            }
            run += __shfl_sync(0xffffffffu, c, 31);
        }
    }
    cluster_sync_all();   // no CTA leaves while a peer reads its sums
}

}  // namespace

int sample_max_vocab() { return kMaxCluster * kMaxChunk; }

int launch_sample(const SampleArgs &a, int R, int dtype, int num_sms, cudaStream_t stream)
{
    // CTAs per row: as few as hold the row at four CTAs per SM (32 KB of logits
    // each, or what eight of them have to hold); more (down to 2048 logits
    // each) while the rows alone leave SMs idle.
    const int es = dtype == TSD_BF16 ? 2 : 4;
    int C = 1;
    while (C < kMaxCluster && ((long long)(a.V + C - 1) / C * es > 32768 ||
                               ((long long)R * C < 2LL * num_sms && a.V / C >= 4096)))
        C *= 2;
    const int steps = (a.V + 127) / 128;
    const int chunk = (steps + C - 1) / C * 128;   // of a CTA at most
    int log2v = 0;
    while ((1LL << log2v) < a.V)
        ++log2v;
    const int s = std::min(50, 63 - log2v);
    const auto smem = [es](int n) { return (sizeof(Shared) + 15) / 16 * 16 + (size_t)n * es; };
    auto kern = dtype == TSD_BF16 ? sample_kernel<__nv_bfloat16> : sample_kernel<float>;
    constexpr int kMaxDevices = 64;
    static std::atomic<bool> raised[kMaxDevices][2];
    int dev = 0;
    TSD_CUDA_TRY(cudaGetDevice(&dev));
    if (dev < 0 || dev >= kMaxDevices)
        return TSD_ERR_CUDA;
    if (!raised[dev][dtype == TSD_BF16].load()) {
        TSD_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          (int)smem(kMaxChunk + 256)));
        raised[dev][dtype == TSD_BF16].store(true);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)R * C));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem(chunk);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = C;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, a, C, steps, ldexp(1.0, s)) != cudaSuccess) {
        (void)cudaGetLastError();
        return TSD_ERR_CUDA;
    }
    TSD_LAUNCH_CHECK();
    return TSD_OK;
}

}  // namespace tsd
