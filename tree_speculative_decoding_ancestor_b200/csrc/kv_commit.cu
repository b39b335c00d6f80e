// Commit of the accepted path (SpecInfer explainer, "Tree Attention のカーネル
// 融合", item 2: the tree's KV entries stay consistent with the existing KV
// cache; the flatkey.ai guide's verification diagram: the accepted prefix is
// committed).  After verification the K and V rows of the accepted nodes
// u_0 < u_1 < ... < u_{n-1} move from cache positions P_b + u_i to P_b + i,
// for every KV head, and the prefix grows to P_b + n.
//
// One CTA per (group of KV heads, sequence).  The path is checked before
// anything moves: entries strictly increasing, in [0, Tmax), and P + u < Lmax;
// over a paged cache also the page of every row that is read or written (the
// same logical positions, each row found through the block table once).
// A destination can be another accepted row's source (path [0, 2, 3]: position
// P+2 is read for i = 1 and written for i = 2), but only one of a row in front:
// u_j = i with u_j > j means j < i.  So the rows move in ascending i, a batch
// of 16-byte vectors in the threads' registers at a time, read by every thread
// before any is written.  Rows already in place (u_i = i, a prefix of the path)
// are neither read nor written.
// Bound: a chain of five dependent accesses (count, path, page, row, store), so
// all CTAs should be resident at once: few registers, no staging buffer, and
// several heads a CTA where one would make more CTAs than fit (128 sequences of
// 32 heads, 8 to 16 rows, 25 MB: 10.3 us; with one head a CTA and rows staged in
// shared memory 19.5 us, with 4 or 8 vectors in flight 11.0 and 12.5 us).
#include <algorithm>

#include "tsd_common.cuh"

namespace tsd {

namespace {

constexpr int kCommitThreads = 256;
constexpr int kCommitBatch = 2;   // 16-byte vectors of a thread in flight

__global__ void __launch_bounds__(kCommitThreads)
    kv_commit_kernel(uint4 *k, uint4 *v, KvPages pages, const int32_t *__restrict__ prefix_len,
                     const int32_t *__restrict__ out_path,
                     const int32_t *__restrict__ n_accepted, int Tmax, int Hkv, int heads, int Lmax,
                     int vec, int32_t *__restrict__ new_prefix, int32_t *dev_status)
{
    __shared__ int s_path[kMaxTree];
    __shared__ long long s_src[kMaxTree], s_dst[kMaxTree];   // a move's rows, KV head 0
    const int h0 = blockIdx.x * heads, b = blockIdx.y;
    const int n = n_accepted[b], P = prefix_len[b];
    if (n < 0) {   // malformed upstream (already reported there): nothing moves
        if (h0 == 0 && threadIdx.x == 0)
            new_prefix[b] = P;
        return;
    }
    bool ok = n <= Tmax && P >= 0;
    if (ok && (int)threadIdx.x < n)
        s_path[threadIdx.x] = out_path[(size_t)b * Tmax + threadIdx.x];
    __syncthreads();
    if (ok && (int)threadIdx.x < n) {
        const int i = threadIdx.x, u = s_path[i];
        ok = u >= 0 && u < Tmax && (i == 0 || u > s_path[i - 1]) && u < Lmax - P;
    }
    ok = __syncthreads_and(ok) != 0;
    bool bad_page = false, stays = false;
    if (ok && (int)threadIdx.x < n) {
        const int i = threadIdx.x, u = s_path[i];
        stays = u == i;   // no page needed
        s_src[i] = stays ? 0 : kv_row(pages, b, 0, Hkv, Lmax, P + u);
        s_dst[i] = stays ? 0 : kv_row(pages, b, 0, Hkv, Lmax, P + i);
        bad_page = s_src[i] < 0 || s_dst[i] < 0;
    }
    bad_page = __syncthreads_or(bad_page) != 0;
    const int first = __syncthreads_count(stays);   // rows in front that are in place
    if (h0 == 0 && threadIdx.x == 0) {
        new_prefix[b] = ok && !bad_page ? P + n : P;
        if (!ok)
            flag(dev_status, TSD_DEV_BAD_PATH);
        if (bad_page)
            flag(dev_status, TSD_DEV_BAD_PAGE);
    }
    if (!ok || bad_page)
        return;
    const int nh = min(heads, Hkv - h0);
    const int per_row = 2 * nh * vec;   // vectors of a path entry: K and V of nh heads
    const int total = (n - first) * per_row;
    const long long head_rows = pages.table ? pages.page_size : Lmax;
    // extent of the cache in vectors
    const long long all_vec = kv_rows_total(pages, gridDim.y, Hkv, Lmax) * vec;
    for (int base = 0; base < total; base += kCommitThreads * kCommitBatch) {
        uint4 x[kCommitBatch];
        long long to[kCommitBatch];
        bool is_v[kCommitBatch];
#pragma unroll
        for (int e = 0; e < kCommitBatch; ++e) {
            const int idx = base + e * kCommitThreads + threadIdx.x;
            to[e] = -1;
            if (idx >= total)
                continue;
            const int i = idx / per_row, r = idx - i * per_row;
            const int hv = r / vec, c = r - hv * vec;   // 2 * head + (0: K, 1: V)
            is_v[e] = hv & 1;
            const long long head = (h0 + (hv >> 1)) * head_rows;
            const long long from = (s_src[first + i] + head) * vec + c;
            const long long at = (s_dst[first + i] + head) * vec + c;
            if (!in_bounds(from, all_vec, dev_status) || !in_bounds(at, all_vec, dev_status))
                continue;
            x[e] = (is_v[e] ? v : k)[from];
            to[e] = at;
        }
        __syncthreads();   // every row of the batch is read
#pragma unroll
        for (int e = 0; e < kCommitBatch; ++e)
            if (to[e] >= 0)
                (is_v[e] ? v : k)[to[e]] = x[e];
    }
}

}  // namespace

int launch_kv_commit(void *k_cache, void *v_cache, const KvPages &pages,
                     const int32_t *prefix_len, const int32_t *out_path,
                     const int32_t *n_accepted, int B, int Tmax, int Hkv, int Lmax, int row_bytes,
                     int32_t *new_prefix, int32_t *dev_status, int num_sms, cudaStream_t stream)
{
    if (B == 0)
        return TSD_OK;
    // KV heads of a CTA: one, and more while the CTAs would not fit the GPU at
    // once (8 per SM)
    int heads = 1;
    while (heads < Hkv && (long long)B * ((Hkv + heads - 1) / heads) > 8LL * num_sms)
        heads *= 2;
    kv_commit_kernel<<<dim3((Hkv + heads - 1) / heads, B), kCommitThreads, 0, stream>>>(
        static_cast<uint4 *>(k_cache), static_cast<uint4 *>(v_cache), pages, prefix_len, out_path,
        n_accepted, Tmax, Hkv, heads, Lmax, row_bytes / 16, new_prefix, dev_status);
    TSD_LAUNCH_CHECK();
    return TSD_OK;
}

}  // namespace tsd
