// Rotary positions of new tokens, appended to a paged KV cache.
//
// The token in slot u of sequence b sits at position pos = P_b + u (a chunk)
// or P_b + depth[u] - 1 (a node of a token tree: its depth counts the nodes
// of its root path), and its K/V rows go to logical cache position P_b + u.
// Pair i of the rotated part of a head turns by pos * inv_freq[i]:
//     (x, y) -> (x c - y s, y c + x s),  c = g cos(angle), s = g sin(angle)
// with pairs (i, i + rot/2) or (2i, 2i + 1); dimensions from rot on pass
// through.  The angle is a product of a position that may need 20 bits and a
// frequency: its fp32 rounding alone would be 2^-24 * 10^5 = 0.006 radians,
// so it is formed and reduced to half a turn in fp64; the cosine and sine are
// fp32, and each output is rounded once.
//
// Every row is read and written once: HBM-bound for chunks, launch latency
// for single tokens.  A thread keeps two 16-byte slots of a row -- for pairs
// (i, i + rot/2) the two that hold each other's partners -- with their cosines
// and sines in registers, and walks the heads of its token with them, so the
// trigonometry and its shared-memory reads are paid once per token and not per
// head, and no element is loaded twice.  Measured (bf16, D = 128, 64/8 heads):
// 4096 tokens 33.3 us = 5.0 TB/s, 77% of a plain copy; 2048 tree tokens 15.7
// us; 8 single tokens 2.8 us.  One slot a thread, its partners loaded again:
// 37.6 and 19.8 us; two or four rows in flight, three or six CTAs per SM: 34 to
// 73 us and 15 to 28 (spills where the registers end).
#include <algorithm>

#include "tsd_common.cuh"

namespace tsd {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 4;      // tokens per CTA at most
constexpr int kRopeRows = 3;        // rows a thread has in flight
constexpr int kRopeCtas = 4;        // CTAs per SM
constexpr int kRopeMaxPairs = 128;  // rot / 2 at most (rows of 512 bytes, 16-bit elements)

template <typename T> struct Vec16 {
    static constexpr int N = 16 / sizeof(T);
    union {
        uint4 raw;
        T e[N];
    };
    __device__ Vec16() {}
};

// How the pairs of a head lie: (2i, 2i + 1), or (i, i + rot / 2) with the
// partners of a 16-byte slot a slot themselves, or anywhere.
enum Pairs { kInterleaved, kHalves, kOddHalves };

template <typename T, Pairs P_>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas)
    rope_append_kernel(RopeArgs a, int tokens_per_cta, int heads_per_cta)
{
    constexpr int N = Vec16<T>::N;
    __shared__ float s_cos[kRopeTokens][kRopeMaxPairs], s_sin[kRopeTokens][kRopeMaxPairs];
    __shared__ long long s_row[kRopeTokens];   // pool row of (token, KV head 0), -1: none
    const int b = blockIdx.y;
    const int P = a.prefix_len[b], n = a.n_new[b];
    const int cap = a.pages.max_blocks << a.pages.log2_page;
    if (n < 0 || n > a.Tmax || P < 0 || P > cap - n) {
        if (blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0)
            flag(a.dev_status, TSD_DEV_BAD_PREFIX);
        return;
    }
    const int t0 = blockIdx.x * tokens_per_cta, t1 = min(t0 + tokens_per_cta, n);
    if (t0 >= t1)
        return;
    const int half = a.rot / 2;
    for (int i = threadIdx.x; i < (t1 - t0) * half; i += kRopeThreads) {
        const int t = i / half, p = i - t * half;
        const int off = a.depth ? a.depth[(size_t)b * a.Tmax + t0 + t] - 1 : t0 + t;
        // in turns, of which only the part behind the point matters
        const double turns = (double)((long long)P + off) * a.inv_freq[p] * 0.15915494309189535;
        float s, c;
        sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
        s_cos[t][p] = c * a.rot_scale;
        s_sin[t][p] = s * a.rot_scale;
    }
    if ((int)threadIdx.x < t1 - t0) {
        const int pos = P + t0 + threadIdx.x;
        const int page = a.pages.table[(size_t)b * a.pages.max_blocks + (pos >> a.pages.log2_page)];
        const bool ok = page >= 0 && page < a.pages.num_pages;
        if (!ok && blockIdx.z == 0)
            flag(a.dev_status, TSD_DEV_BAD_PAGE);
        s_row[threadIdx.x] = ok ? (long long)page * a.Hkv * a.pages.page_size +
                                      (pos & (a.pages.page_size - 1))
                                : -1;
    }
    __syncthreads();
    const int slots = a.D / N, units = (slots + 1) / 2;   // 16-byte slots of a row, two a thread
    const int par = kRopeThreads / units;                 // rows side by side
    const int j = threadIdx.x % units, hp = threadIdx.x / units;
    if (hp >= par)
        return;
    // this thread's slots: partners, or the next two
    const int turned = P_ == kHalves ? half / N : 0;
    const int sa = P_ == kHalves ? (j < turned ? j : 2 * j) : 2 * j;
    const int sb = P_ == kHalves && j < turned ? j + turned : sa + 1;
    const bool two = sb < slots;
    const int ea = sa * N, eb = sb * N;
    const int h_end = min((int)(blockIdx.z + 1) * heads_per_cta, a.Hq + 2 * a.Hkv);
    for (int t = t0; t < t1; ++t) {
        // cosines and sines: of slot a's N pairs (halves), or of the N / 2 pairs
        // of each slot (interleaved)
        float c[N], s[N];
        if (P_ != kOddHalves) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int p = P_ == kHalves ? ea + i : ea / 2 + i;
                const bool turn = P_ == kHalves ? j < turned : p < half;
                c[i] = turn ? s_cos[t - t0][p] : 1.f;
                s[i] = turn ? s_sin[t - t0][p] : 0.f;
            }
        }
        const long long row = s_row[t - t0];
        const T *const q = static_cast<const T *>(a.q) + b * a.q_batch + t * a.q_token;
        const T *const k = static_cast<const T *>(a.k) + b * a.k_batch + t * a.k_token;
        const T *const v = static_cast<const T *>(a.v) + b * a.v_batch + t * a.v_token;
        const bool turn = P_ == kHalves ? j < turned : ea < a.rot;
        auto source = [&](int h) {
            return h < a.Hq            ? q + (size_t)h * a.D
                   : h < a.Hq + a.Hkv ? k + (size_t)(h - a.Hq) * a.D
                                      : v + (size_t)(h - a.Hq - a.Hkv) * a.D;
        };
        for (int h0 = blockIdx.z * heads_per_cta + hp; h0 < h_end; h0 += kRopeRows * par) {
            // all rows' loads in flight before the first is used
            Vec16<T> x[kRopeRows], y[kRopeRows];
#pragma unroll
            for (int i = 0; i < kRopeRows; ++i) {
                const int h = h0 + i * par;
                if (h >= h_end)
                    continue;
                const T *const src = source(h);
                x[i].raw = __ldg(reinterpret_cast<const uint4 *>(src + ea));
                if (two)
                    y[i].raw = __ldg(reinterpret_cast<const uint4 *>(src + eb));
            }
#pragma unroll
            for (int i = 0; i < kRopeRows; ++i) {
                const int h = h0 + i * par;
                if (h >= h_end || (h >= a.Hq && row < 0))
                    continue;
                if (turn && h < a.Hq + a.Hkv) {
                    if (P_ == kHalves) {
#pragma unroll
                        for (int n = 0; n < N; ++n) {
                            const float f = to_float(x[i].e[n]), g = to_float(y[i].e[n]);
                            x[i].e[n] = from_float<T>(f * c[n] - g * s[n]);
                            y[i].e[n] = from_float<T>(g * c[n] + f * s[n]);
                        }
                    } else if (P_ == kInterleaved) {
#pragma unroll
                        for (int n = 0; n < N; n += 2) {   // dimensions from rot on stay as they are
                            if (ea + n < a.rot) {
                                const float f = to_float(x[i].e[n]), g = to_float(x[i].e[n + 1]);
                                x[i].e[n] = from_float<T>(f * c[n / 2] - g * s[n / 2]);
                                x[i].e[n + 1] = from_float<T>(g * c[n / 2] + f * s[n / 2]);
                            }
                            if (eb + n < a.rot) {
                                const int m = (N + n) / 2;
                                const float f = to_float(y[i].e[n]), g = to_float(y[i].e[n + 1]);
                                y[i].e[n] = from_float<T>(f * c[m] - g * s[m]);
                                y[i].e[n + 1] = from_float<T>(g * c[m] + f * s[m]);
                            }
                        }
                    } else {   // element by element
                        const T *const src = source(h);
                        for (int n = 0; n < 2 * N; ++n) {
                            const int e = ea + n;
                            if (e >= a.rot)
                                break;
                            const int p = e < half ? e : e - half;
                            const float f = to_float(src[e]);
                            const float g = to_float(src[e < half ? e + half : p]);
                            const float z = f * s_cos[t - t0][p] +
                                            (e < half ? -g : g) * s_sin[t - t0][p];
                            if (n < N)
                                x[i].e[n] = from_float<T>(z);
                            else
                                y[i].e[n - N] = from_float<T>(z);
                        }
                    }
                }
                T *dst;
                long long at, extent;
                if (h < a.Hq) {
                    at = (((long long)b * a.Tmax + t) * a.Hq + h) * a.D;
                    extent = (long long)gridDim.y * a.Tmax * a.Hq * a.D;
                    dst = static_cast<T *>(a.q_out);
                } else {
                    const bool is_k = h < a.Hq + a.Hkv;
                    at = (row + (long long)(h - a.Hq - (is_k ? 0 : a.Hkv)) * a.pages.page_size) *
                         a.D;
                    extent = kv_rows_total(a.pages, gridDim.y, a.Hkv, 0) * a.D;
                    dst = static_cast<T *>(is_k ? a.k_pages : a.v_pages);
                }
                if (in_bounds(at, extent - a.D + 1, a.dev_status)) {
                    *reinterpret_cast<uint4 *>(dst + at + ea) = x[i].raw;
                    if (two)
                        *reinterpret_cast<uint4 *>(dst + at + eb) = y[i].raw;
                }
            }
        }
    }
}

}  // namespace

int launch_rope_append(const RopeArgs &a, int B, int dtype, int num_sms, cudaStream_t stream)
{
    // Tokens per CTA: four share one round of trigonometry, fewer while the
    // grid would leave SMs without a CTA; then the heads are divided too, down
    // to one pass of the CTA's threads over them.
    const int heads = a.Hq + 2 * a.Hkv;
    const int slots = a.D * (dtype == TSD_F32 ? 4 : 2) / 16;
    const int par = kRopeThreads / ((slots + 1) / 2);
    int per = kRopeTokens;
    while (per > 1 && (long long)B * ((a.Tmax + per - 1) / per) < 2LL * num_sms)
        per >>= 1;
    const long long ctas = (long long)B * ((a.Tmax + per - 1) / per);
    int parts = (int)std::min<long long>(std::max<long long>(num_sms / ctas, 1), (heads + par - 1) / par);
    const int hpc = (heads + parts - 1) / parts;
    parts = (heads + hpc - 1) / hpc;
    const dim3 grid((a.Tmax + per - 1) / per, B, parts);
    const bool whole = a.rot / 2 % (dtype == TSD_F32 ? 4 : 8) == 0;
    auto kern = dtype == TSD_BF16
                    ? (a.interleaved ? rope_append_kernel<__nv_bfloat16, kInterleaved>
                       : whole       ? rope_append_kernel<__nv_bfloat16, kHalves>
                                     : rope_append_kernel<__nv_bfloat16, kOddHalves>)
                    : (a.interleaved ? rope_append_kernel<float, kInterleaved>
                       : whole       ? rope_append_kernel<float, kHalves>
                                     : rope_append_kernel<float, kOddHalves>);
    kern<<<grid, kRopeThreads, 0, stream>>>(a, per, hpc);
    TSD_LAUNCH_CHECK();
    return TSD_OK;
}

}  // namespace tsd
