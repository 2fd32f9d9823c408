// prefill_simple.cu -- causal attention of many new tokens of each sequence, over packed keys and
// values or over a paged cache, on the CUDA cores.
//
// What is computed: the i-th of a sequence's n new tokens, of L keys in all, has position
// p = L - n + i and sees the keys t <= p (window > 0: of them t > p - window or t < n_sink):
//   s_t = scale q.k_t,  out = sum_t exp(s_t - lse) v_t,  lse = log(sum_t exp(s_t) [+ exp(sink)]).
//
// One CTA takes 64 rows (token, head of the KV head's group) of one sequence and KV head and walks
// its visible keys 32 at a time with a running maximum and sum, everything in float32.

#include <algorithm>

#include "kvd_device.cuh"
#include "kvd_host.h"

namespace kvd {

namespace {

constexpr int kRows = 64, kKeys = 32, kThreads = 128;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f32(float* d, float x) { *d = x; }
__device__ __forceinline__ void from_f32(__nv_bfloat16* d, float x) { *d = __float2bfloat16_rn(x); }

template <int D>
struct Smem {
    float q[kRows][D + 1];
    float k[kKeys][D + 1];
    float v[kKeys][D];
    float s[kRows][kKeys + 1];
};

template <int D, typename T>
__global__ void __launch_bounds__(kThreads) prefill_simple_kernel(const PrefillParams p) {
    extern __shared__ __align__(16) uint8_t raw[];
    Smem<D>& sm = *reinterpret_cast<Smem<D>*>(raw);
    griddep_wait();
    // the sequence: block x is tile x - (first row / 64 + b) of sequence b
    const int x = blockIdx.x, h = blockIdx.y;
    auto first_row = [&](int b) -> long long { return p.cu_q ? p.cu_q[b] : b; };
    auto start = [&](int b) { return first_row(b) * p.G / kRows + b; };
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int b = threadIdx.x; b < p.B; b += kThreads) {
            const long long c0 = first_row(b), c1 = first_row(b + 1);
            bool bad = c0 < 0 || c1 < c0 || c1 > p.T || (b == 0 && c0 != 0);
            if (p.block_table) {
                const int L = p.seq_lens[b];
                bad |= L < c1 - c0 || L > static_cast<long long>(p.max_pages) << p.page_shift;
            } else {
                const int k0 = p.cu_k[b], k1 = p.cu_k[b + 1];
                bad |= k0 < 0 || k1 < k0 || k1 > p.Tk || (b == 0 && k0 != 0);
            }
            if (bad) record_error(p.err, KVD_ERR_DEVICE_OOB);
        }
    int lo = 0, hi = p.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (start(mid) <= x) lo = mid; else hi = mid - 1;
    }
    const int b = lo;
    const long long c0 = first_row(b), c1 = first_row(b + 1);
    if (c0 < 0 || c1 < c0 || c1 > p.T) return;
    const int n = static_cast<int>(c1 - c0);
    const long long r0 = (x - start(b)) * kRows, n_rows = static_cast<long long>(n) * p.G;
    if (r0 < 0 || r0 >= n_rows) return;
    int L;
    long long k0 = 0;
    if (p.block_table) {
        L = min(max(p.seq_lens[b], 0), p.max_pages << p.page_shift);
    } else {
        k0 = p.cu_k[b];
        const long long k1 = p.cu_k[b + 1];
        if (k0 < 0 || k1 < k0 || k1 > p.Tk) return;
        L = static_cast<int>(k1 - k0);
    }
    const T* q = static_cast<const T*>(p.q);
    const T* kp = static_cast<const T*>(p.k);
    const T* vp = static_cast<const T*>(p.v);
    for (int i = threadIdx.x; i < kRows * D; i += kThreads) {
        const int r = i / D, d = i % D;
        const long long row = r0 + r;
        sm.q[r][d] = row < n_rows
                         ? to_f32(q[(c0 + row / p.G) * p.q_stride +
                                    (h * p.G + row % p.G) * static_cast<long long>(D) + d]) *
                               p.scale_log2
                         : 0.f;
    }
    const int ty = threadIdx.x / 8, tx = threadIdx.x % 8;  // rows 4 ty + i; keys tx + 8 j
    float o[4][D / 8], m[4], l[4];
    int pos[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
        const long long row = r0 + ty * 4 + i;
        pos[i] = row < n_rows ? static_cast<int>(L - n + row / p.G) : -1;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) o[i][c] = 0.f;
    }
    const int last = static_cast<int>(L - n + (min(r0 + kRows, n_rows) - 1) / p.G);
    const int first = static_cast<int>(L - n + r0 / p.G);
    const int w0 = p.window > 0 ? max(0, first - p.window + 1) : 0;
    for (int t0 = 0; t0 <= last; t0 += kKeys) {
        if (t0 + kKeys <= w0 && t0 >= p.n_sink) {
            t0 = w0 / kKeys * kKeys;  // behind the sinks: on to the window
            if (t0 > last) break;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < kKeys * D; i += kThreads) {
            const int r = i / D, d = i % D, t = t0 + r;
            float kv = 0.f, vv = 0.f;
            if (t <= last) {
                if (p.block_table) {
                    int pg = p.block_table[static_cast<size_t>(b) * p.max_pages + (t >> p.page_shift)];
                    if (pg < 0 || pg >= p.num_pages) {
                        record_error(p.err, KVD_ERR_DEVICE_OOB);
                        pg = 0;
                    }
                    const size_t at =
                        (((static_cast<size_t>(pg) * p.Hkv + h) << p.page_shift) +
                         (t & ((1 << p.page_shift) - 1))) * D + d;
                    kv = to_f32(kp[at]);
                    vv = to_f32(vp[at]);
                } else {
                    kv = to_f32(kp[(k0 + t) * p.k_stride + static_cast<long long>(h) * D + d]);
                    vv = to_f32(vp[(k0 + t) * p.v_stride + static_cast<long long>(h) * D + d]);
                }
            }
            sm.k[r][d] = kv;
            sm.v[r][d] = vv;
        }
        __syncthreads();
        float s[4][4] = {};
        for (int d = 0; d < D; ++d) {
            float a[4], c[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = sm.q[ty * 4 + i][d];
#pragma unroll
            for (int j = 0; j < 4; ++j) c[j] = sm.k[tx + 8 * j][d];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[i][j] = fmaf(a[i], c[j], s[i][j]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = t0 + tx + 8 * j;
                const bool seen = t <= pos[i] && (p.window <= 0 || t > pos[i] - p.window || t < p.n_sink);
                if (!seen) s[i][j] = -INFINITY;
                top = fmaxf(top, s[i][j]);
            }
            for (int off = 4; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            const float mn = fmaxf(m[i], top), ref = mn == -INFINITY ? 0.f : mn;
            const float fade = exp2f(m[i] - ref);
            m[i] = mn;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float e = exp2f(s[i][j] - ref);
                sm.s[ty * 4 + i][tx + 8 * j] = e;
                sum += e;
            }
            for (int off = 4; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            l[i] = l[i] * fade + sum;
#pragma unroll
            for (int c = 0; c < D / 8; ++c) o[i][c] *= fade;
        }
        __syncwarp();
        for (int t = 0; t < kKeys; ++t) {
            float e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) e[i] = sm.s[ty * 4 + i][t];
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                const float y = sm.v[t][tx + 8 * c];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (e[i] != 0.f) o[i][c] = fmaf(e[i], y, o[i][c]);  // (a hidden value may be NaN)
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const long long row = r0 + ty * 4 + i;
        if (row >= n_rows) continue;
        const int head = h * p.G + static_cast<int>(row % p.G);
        const long long at = (c0 + row / p.G) * p.Hq + head;
        float ref = m[i] == -INFINITY ? 0.f : m[i];
        float mm = m[i], ll = l[i], fade = 1.f;
        if (p.sink_logit) {
            const float sink = p.sink_logit[head] * 1.4426950408889634f;
            mm = fmaxf(m[i], sink);
            ref = mm == -INFINITY ? 0.f : mm;
            fade = exp2f(m[i] - ref);
            ll = l[i] * fade + exp2f(sink - ref);
        }
        const float inv = ll == 0.f ? 0.f : fade / ll;
        T* out = static_cast<T*>(p.out) + at * D;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) from_f32(out + tx + 8 * c, o[i][c] * inv);
        if (p.lse_out && tx == 0)
            p.lse_out[at] = ll == 0.f ? -INFINITY : (ref + log2f(ll)) * 0.6931471805599453f;
    }
}

template <int D, typename T>
int launch(const PrefillParams& p, cudaStream_t stream) {
    auto kernel = prefill_simple_kernel<D, T>;
    static const cudaError_t set = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(sizeof(Smem<D>)));
    if (set != cudaSuccess) return KVD_ERR_CUDA;
    const long long tiles = static_cast<long long>(p.T) * p.G / kRows + p.B;
    if (launch_kernel(kernel, dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(p.Hkv)),
                      dim3(kThreads), sizeof(Smem<D>), stream, p) != cudaSuccess)
        return KVD_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? KVD_OK : KVD_ERR_CUDA;
}

}  // namespace

int prefill_f32_launch(const PrefillParams& p, int D, cudaStream_t stream) {
    return D == 64 ? launch<64, float>(p, stream) : launch<128, float>(p, stream);
}

}  // namespace kvd
