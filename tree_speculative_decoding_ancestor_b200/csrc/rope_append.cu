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
// so it is formed and reduced to [-pi, pi] in fp64; the cosine and sine are
// fp32, and each output is rounded once.
//
// Every row is read and written once: HBM-bound for chunks, launch latency
// for single tokens.  A thread keeps one 16-byte slot of a row (and that
// slot's cosines and sines in registers) and walks the heads of its token
// with it, so the trigonometry and its shared-memory reads are paid once per
// token and not per head.
#include <algorithm>

#include "tsd_common.cuh"

namespace tsd {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 4;      // tokens per CTA at most
constexpr int kRopeMaxPairs = 128;  // rot / 2 at most (rows of 512 bytes, 16-bit elements)

template <typename T> struct Vec16 {
    static constexpr int N = 16 / sizeof(T);
    union {
        uint4 raw;
        T e[N];
    };
    __device__ Vec16() {}
};

template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads)
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
        const double angle = (double)((long long)P + off) * a.inv_freq[p];
        const double turns = rint(angle * 0.15915494309189535);   // 1 / (2 pi)
        // 2 pi as the sum of two doubles: the reduced angle keeps fp32 accuracy
        double r = fma(turns, -6.283185307179586, angle);
        r = fma(turns, -2.4492935982947064e-16, r);
        float s, c;
        sincosf((float)r, &s, &c);
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
    const int slots = a.D / N;   // 16-byte slots of a row
    const int par = kRopeThreads / slots;
    const int j = threadIdx.x % slots, hp = threadIdx.x / slots;
    if (hp >= par)
        return;
    const int e0 = j * N;
    const int h_end = min((int)(blockIdx.z + 1) * heads_per_cta, a.Hq + 2 * a.Hkv);
    const bool paired = !INTERLEAVED && half % N == 0;   // a slot's partners are a slot
    for (int t = t0; t < t1; ++t) {
        float c[N], s[N];   // out = x * c + partner * s
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int e = e0 + i;
            const bool turn = e < a.rot;
            const int p = !turn ? 0 : INTERLEAVED ? e >> 1 : (e < half ? e : e - half);
            const bool first = INTERLEAVED ? (e & 1) == 0 : e < half;
            c[i] = turn ? s_cos[t - t0][p] : 1.f;
            s[i] = turn ? (first ? -s_sin[t - t0][p] : s_sin[t - t0][p]) : 0.f;
        }
        const long long row = s_row[t - t0];
#pragma unroll 4
        for (int h = blockIdx.z * heads_per_cta + hp; h < h_end; h += par) {
            const bool is_q = h < a.Hq, is_k = !is_q && h < a.Hq + a.Hkv;
            const int hk = h - a.Hq - (is_k ? 0 : a.Hkv);   // KV head (k and v rows)
            if (!is_q && row < 0)
                continue;
            const T *src =
                is_q   ? static_cast<const T *>(a.q) + b * a.q_batch + t * a.q_token + (size_t)h * a.D
                : is_k ? static_cast<const T *>(a.k) + b * a.k_batch + t * a.k_token + (size_t)hk * a.D
                       : static_cast<const T *>(a.v) + b * a.v_batch + t * a.v_token + (size_t)hk * a.D;
            Vec16<T> x, y;
            x.raw = *reinterpret_cast<const uint4 *>(src + e0);
            const bool turn = (is_q || is_k) && e0 < a.rot;
            if (turn) {
                float f[N];
#pragma unroll
                for (int i = 0; i < N; ++i)
                    f[i] = to_float(x.e[i]);
                if (INTERLEAVED) {
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        y.e[i] = from_float<T>(f[i] * c[i] + f[i ^ 1] * s[i]);
                } else if (paired) {
                    Vec16<T> o;
                    o.raw = *reinterpret_cast<const uint4 *>(src + (e0 < half ? e0 + half : e0 - half));
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        y.e[i] = from_float<T>(f[i] * c[i] + to_float(o.e[i]) * s[i]);
                } else {
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const int e = e0 + i;
                        const float o =
                            e < a.rot ? to_float(src[e < half ? e + half : e - half]) : 0.f;
                        y.e[i] = e < a.rot ? from_float<T>(f[i] * c[i] + o * s[i]) : x.e[i];
                    }
                }
                // dimensions from rot on inside the slot pass through bit for bit
                if (e0 + N > a.rot) {
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        if (e0 + i >= a.rot)
                            y.e[i] = x.e[i];
                }
            } else {
                y.raw = x.raw;
            }
            T *dst;
            long long at, extent;
            if (is_q) {
                at = (((long long)b * a.Tmax + t) * a.Hq + h) * a.D + e0;
                extent = (long long)gridDim.y * a.Tmax * a.Hq * a.D;
                dst = static_cast<T *>(a.q_out);
            } else {
                at = (row + (long long)hk * a.pages.page_size) * a.D + e0;
                extent = kv_rows_total(a.pages, gridDim.y, a.Hkv, 0) * a.D;
                dst = static_cast<T *>(is_k ? a.k_pages : a.v_pages);
            }
            if (in_bounds(at, extent - N + 1, a.dev_status))
                *reinterpret_cast<uint4 *>(dst + at) = y.raw;
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
    const int par = kRopeThreads / (a.D * (dtype == TSD_F32 ? 4 : 2) / 16);
    int per = kRopeTokens;
    while (per > 1 && (long long)B * ((a.Tmax + per - 1) / per) < 2LL * num_sms)
        per >>= 1;
    const long long ctas = (long long)B * ((a.Tmax + per - 1) / per);
    int parts = (int)std::min<long long>(std::max<long long>(num_sms / ctas, 1), (heads + par - 1) / par);
    const int hpc = (heads + parts - 1) / parts;
    parts = (heads + hpc - 1) / hpc;
    const dim3 grid((a.Tmax + per - 1) / per, B, parts);
    auto kern = dtype == TSD_BF16
                    ? (a.interleaved ? rope_append_kernel<__nv_bfloat16, true>
                                     : rope_append_kernel<__nv_bfloat16, false>)
                    : (a.interleaved ? rope_append_kernel<float, true>
                                     : rope_append_kernel<float, false>);
    kern<<<grid, kRopeThreads, 0, stream>>>(a, per, hpc);
    TSD_LAUNCH_CHECK();
    return TSD_OK;
}

}  // namespace tsd
