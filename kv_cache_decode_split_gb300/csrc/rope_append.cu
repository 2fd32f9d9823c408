// rope_append.cu -- new tokens' keys and values written into a paged or rolling cache, the
// position rotation applied on the way; the cache in the tensors' own type or in 4 bits.
//
// What is computed. Row x of a new token at position t is rotated by the table's cosines c and
// sines s of that position (rot channels, the others pass unchanged):
//   halves       y_i = x_i c_i - x_{i+rot/2} s_i,  y_{i+rot/2} = x_{i+rot/2} c_i + x_i s_i
//   interleaved  y_2i = x_2i c_i - x_{2i+1} s_i,   y_{2i+1} = x_{2i+1} c_i + x_2i s_i
// each product and each sum rounded to float32 (no fused multiply-add: the 4-bit codes then follow
// from the inputs by IEEE arithmetic alone, whatever computes them). Queries and keys are rotated,
// values are not. Queries go to q_out; keys and values go to the cache slot of t (slot t, or, in a
// rolling cache of n_sink + window slots, t for t < n_sink and n_sink + (t - n_sink) mod window;
// a token that a later one of the same call replaces there is not written). For the 4-bit cache
// see kvd_q4.cuh.
//
// GB300: no reuse, so bytes are the bound. A row is handled by D/16 lanes, each with two pieces of
// 8 channels (the two halves of the rotated pairs, so a pair never leaves its thread); the row's
// data is requested before the token's sequence, length, page and table row are looked up, which
// is a chain of dependent reads.

#include <algorithm>

#include "kvd_device.cuh"
#include "kvd_host.h"
#include "kvd_q4.cuh"

namespace kvd {

namespace {

struct TokenAt {
    int b, slot, pos;   // slot < 0: the cache is not written
    bool ok;            // false: the row belongs to no token, or the token's length is bad
};

// Sequence of token i: the last b with cu[b] <= i, by 32-way search (one warp).
__device__ __forceinline__ int find_seq(const int32_t* cu, int B, int i, int lane) {
    int lo = 0, n = B + 1;
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int k = lane * step;
        const bool le = k < n && __ldg(cu + lo + k) <= i;
        const int cnt = __popc(__ballot_sync(0xffffffffu, le));
        if (cnt == 0) return -1;
        lo += (cnt - 1) * step;
        n = min(step, n - (cnt - 1) * step);
    }
    return lo;
}

// Where token i goes (the same answer in every lane of the warp).
__device__ __forceinline__ TokenAt locate(const RopeAppendParams& p, int i, int lane) {
    TokenAt a;
    a.ok = false;
    a.slot = -1;
    a.pos = 0;
    a.b = i;
    int before = i, n = 1;  // the sequence's first row, its new tokens
    if (p.cu_seqlens) {
        a.b = find_seq(p.cu_seqlens, p.B, i, lane);
        if (a.b < 0 || a.b >= p.B) return a;  // in front of the first or behind the last sequence
        before = __ldg(p.cu_seqlens + a.b);
        const int next = __ldg(p.cu_seqlens + a.b + 1);
        n = next - before;
        if (before > i || i >= next) {  // offsets that do not ascend
            record_error(p.err, KVD_ERR_DEVICE_OOB);
            return a;
        }
    }
    const int L = __ldg(p.seq_lens + a.b);
    const long long cap = static_cast<long long>(p.max_pages) << p.page_shift;
    a.pos = L - n + (i - before);
    if (n > L || a.pos >= p.max_pos || (p.window <= 0 && L > cap)) {
        record_error(p.err, KVD_ERR_DEVICE_OOB);
        return a;
    }
    a.ok = true;
    if (p.window <= 0 || a.pos < p.n_sink)
        a.slot = a.pos;
    else if (a.pos >= L - p.window)
        a.slot = p.n_sink + (a.pos - p.n_sink) % p.window;
    return a;
}

template <typename T>
struct Piece;  // 8 channels as loaded
template <>
struct Piece<__nv_bfloat16> {
    uint4 v;
    __device__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
    __device__ void get(float (&x)[8]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            x[2 * k] = __uint_as_float(w[k] << 16);
            x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        }
    }
    static __device__ void put(__nv_bfloat16* p, const float (&x)[8]) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                                  pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    }
};
template <>
struct Piece<float> {
    float4 a, b;
    __device__ void load(const float* p) {
        a = *reinterpret_cast<const float4*>(p);
        b = *reinterpret_cast<const float4*>(p + 4);
    }
    __device__ void get(float (&x)[8]) const {
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
        x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
    static __device__ void put(float* p, const float (&x)[8]) {
        *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
    }
};

__device__ __forceinline__ void rotate_pair(float& x, float& y, float c, float s) {
    const float a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
    y = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
    x = a;
}

// Nibble m of lane j's word becomes nibble j of lane m's word, among 8 neighbouring lanes.
__device__ __forceinline__ uint32_t transpose_nibbles(uint32_t w, int lane) {
    uint32_t o = __shfl_xor_sync(0xffffffffu, w, 4);
    w = (lane & 4) ? ((w & 0xffff0000u) | (o >> 16)) : ((w & 0x0000ffffu) | (o << 16));
    o = __shfl_xor_sync(0xffffffffu, w, 2);
    w = (lane & 2) ? ((w & 0xff00ff00u) | ((o >> 8) & 0x00ff00ffu))
                   : ((w & 0x00ff00ffu) | ((o & 0x00ff00ffu) << 8));
    o = __shfl_xor_sync(0xffffffffu, w, 1);
    return (lane & 1) ? ((w & 0xf0f0f0f0u) | ((o >> 4) & 0x0f0f0f0fu))
                      : ((w & 0x0f0f0f0fu) | ((o & 0x0f0f0f0fu) << 4));
}

// One warp: one token, 32 / (D/16) rows at a time, R rows a lane.
template <typename T, int D, bool kQ4, int R>
__global__ void __launch_bounds__(256) rope_append_kernel(const RopeAppendParams p) {
    griddep_wait();
    using L4 = Q4<D>;
    constexpr int kTeam = D / 16;       // lanes of a row
    constexpr int kTeams = 32 / kTeam;  // rows of a warp's step
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int team = lane / kTeam, j = lane % kTeam;
    const long long item = static_cast<long long>(blockIdx.x) * 8 + warp;
    const int parts = (p.rows + kTeams * R - 1) / (kTeams * R);
    if (item >= static_cast<long long>(p.T) * parts) return;
    const int i = static_cast<int>(item / parts);
    const int row0 = static_cast<int>(item % parts) * kTeams * R + team;

    // pieces of a rotated row: (c, c + rot/16) for the pairs, then neighbours; of a value row
    // (j, j + D/16)
    const int rp = p.rot / 16;
    const int ca = j < rp ? j : 2 * j, cb = j < rp ? j + rp : 2 * j + 1;
    Piece<T> a[R], b[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int row = row0 + k * kTeams;
        if (row >= p.rows) continue;
        const T* src;
        int pa = ca, pb = cb;
        if (row < p.Hq) {
            src = static_cast<const T*>(p.q) + i * p.q_stride + row * D;
        } else if (row < p.Hq + p.Hkv) {
            src = static_cast<const T*>(p.k) + i * p.k_stride + (row - p.Hq) * D;
        } else {
            src = static_cast<const T*>(p.v) + i * p.v_stride + (row - p.Hq - p.Hkv) * D;
            pa = j, pb = j + kTeam;
        }
        a[k].load(src + 8 * pa);
        b[k].load(src + 8 * pb);
    }
    const TokenAt at = locate(p, i, lane);
    if (!at.ok) return;
    // the token's row in the cache
    int page = -1;
    if (at.slot >= 0) {
        page = __ldg(p.block_table + static_cast<size_t>(at.b) * p.max_pages +
                     (at.slot >> p.page_shift));
        if (page < 0 || page >= p.num_pages) {
            record_error(p.err, KVD_ERR_DEVICE_OOB);
            page = -1;
        }
    }
    const int in_page = at.slot & ((1 << p.page_shift) - 1);
    // cosines and sines of this lane's pairs: halves share them (8 + 8), interleaved pieces have
    // four pairs each
    float cs[8], sn[8];
    {
        const float* row = p.cos_sin + static_cast<size_t>(at.pos) * p.rot;
        const int h = p.rot / 2;
        if (j < rp) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int o = p.interleaved ? (e ? cb : ca) * 4 : ca * 8 + 4 * e;
                const float4 c = __ldg(reinterpret_cast<const float4*>(row + o));
                const float4 s = __ldg(reinterpret_cast<const float4*>(row + h + o));
                cs[4 * e] = c.x, cs[4 * e + 1] = c.y, cs[4 * e + 2] = c.z, cs[4 * e + 3] = c.w;
                sn[4 * e] = s.x, sn[4 * e + 1] = s.y, sn[4 * e + 2] = s.z, sn[4 * e + 3] = s.w;
            }
        }
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int row = row0 + k * kTeams;
        const bool have = row < p.rows;
        const bool is_q = row < p.Hq, is_v = row >= p.Hq + p.Hkv;
        float x[8], y[8];
        if (have) {
            a[k].get(x);
            b[k].get(y);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = y[e] = 0.f;
        }
        if (have && !is_v && j < rp) {
            if (p.interleaved) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    rotate_pair(x[2 * e], x[2 * e + 1], cs[e], sn[e]);
                    rotate_pair(y[2 * e], y[2 * e + 1], cs[4 + e], sn[4 + e]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) rotate_pair(x[e], y[e], cs[e], sn[e]);
            }
        }
        const int pa = is_v ? j : ca, pb = is_v ? j + kTeam : cb;
        if (have && is_q) {
            T* dst = static_cast<T*>(p.q_out) + (static_cast<size_t>(i) * p.Hq + row) * D;
            Piece<T>::put(dst + 8 * pa, x);
            Piece<T>::put(dst + 8 * pb, y);
        }
        const int h = row - p.Hq - (is_v ? p.Hkv : 0);
        if constexpr (!kQ4) {
            if (have && !is_q && page >= 0) {
                T* dst = static_cast<T*>(is_v ? p.v_pool : p.k_pool) +
                         (((static_cast<size_t>(page) * p.Hkv + h) << p.page_shift) + in_page) * D;
                Piece<T>::put(dst + 8 * pa, x);
                Piece<T>::put(dst + 8 * pb, y);
            }
        } else {
            if (!__any_sync(0xffffffffu, have && !is_q)) continue;
            // scale and minimum of the row's groups (piece c belongs to group c / 8)
            const int ga = pa >> 3, gb = pb >> 3;
            bool fa = true, fb = true;
            float lo_a = 65504.f, hi_a = -65504.f, lo_b = 65504.f, hi_b = -65504.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                fa = fa && isfinite(x[e]);
                fb = fb && isfinite(y[e]);
                x[e] = fminf(fmaxf(x[e], -65504.f), 65504.f);
                y[e] = fminf(fmaxf(y[e], -65504.f), 65504.f);
                lo_a = fminf(lo_a, x[e]), hi_a = fmaxf(hi_a, x[e]);
                lo_b = fminf(lo_b, y[e]), hi_b = fmaxf(hi_b, y[e]);
            }
            __half2 par[L4::kGroups];
            float base[L4::kGroups], step[L4::kGroups], inv[L4::kGroups];
#pragma unroll
            for (int g = 0; g < L4::kGroups; ++g) {
                float lo = fminf(ga == g ? lo_a : 65504.f, gb == g ? lo_b : 65504.f);
                float hi = fmaxf(ga == g ? hi_a : -65504.f, gb == g ? hi_b : -65504.f);
                int bad = (ga == g && !fa) || (gb == g && !fb);
#pragma unroll
                for (int off = 1; off < kTeam; off <<= 1) {
                    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
                    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
                    bad |= __shfl_xor_sync(0xffffffffu, bad, off);
                }
                __half hb = __float2half_rn(lo);
                const __half hs = __float2half_rn(__fmul_rn(__fsub_rn(hi, lo), 1.0f / 15.0f));
                step[g] = __half2float(hs);
                base[g] = __half2float(hb);
                inv[g] = step[g] > 0.f ? __frcp_rn(step[g]) : 0.f;
                if (bad) {
                    hb = __ushort_as_half(0x7fff);
                    inv[g] = 0.f;
                }
                par[g] = __halves2half2(hs, hb);
            }
            auto code = [&](float v, int g) {
                const float c = rintf(__fmul_rn(__fsub_rn(v, base[g]), inv[g]));
                return static_cast<uint32_t>(fminf(fmaxf(c, 0.f), 15.f));
            };
            uint32_t wa = 0, wb = 0;
            float va[8], vb[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int g0 = L4::kGroups == 1 ? 0 : ga, g1 = L4::kGroups == 1 ? 0 : gb;
                const uint32_t c0 = g0 ? code(x[e], L4::kGroups - 1) : code(x[e], 0);
                const uint32_t c1 = g1 ? code(y[e], L4::kGroups - 1) : code(y[e], 0);
                wa |= c0 << (4 * e);
                wb |= c1 << (4 * e);
                const __half2 q0 = g0 ? par[L4::kGroups - 1] : par[0];
                const __half2 q1 = g1 ? par[L4::kGroups - 1] : par[0];
                va[e] = fmaf(__low2float(q0), static_cast<float>(c0), __high2float(q0));
                vb[e] = fmaf(__low2float(q1), static_cast<float>(c1), __high2float(q1));
            }
            uint32_t ta = wa, tb = wb;
            if (__any_sync(0xffffffffu, have && is_v)) {
                if constexpr (D == 128) {
                    ta = transpose_nibbles(wa, j);
                    tb = transpose_nibbles(wb, j);
                } else {  // pieces j and j + 4 of the 8: the first exchange stays in the thread
                    const uint32_t u = (wa & 0x0000ffffu) | (wb << 16);
                    const uint32_t v = (wa >> 16) | (wb & 0xffff0000u);
                    uint32_t o = __shfl_xor_sync(0xffffffffu, u, 2);
                    uint32_t u1 = (j & 2) ? ((u & 0xff00ff00u) | ((o >> 8) & 0x00ff00ffu))
                                          : ((u & 0x00ff00ffu) | ((o & 0x00ff00ffu) << 8));
                    o = __shfl_xor_sync(0xffffffffu, v, 2);
                    uint32_t v1 = (j & 2) ? ((v & 0xff00ff00u) | ((o >> 8) & 0x00ff00ffu))
                                          : ((v & 0x00ff00ffu) | ((o & 0x00ff00ffu) << 8));
                    o = __shfl_xor_sync(0xffffffffu, u1, 1);
                    ta = (j & 1) ? ((u1 & 0xf0f0f0f0u) | ((o >> 4) & 0x0f0f0f0fu))
                                 : ((u1 & 0x0f0f0f0fu) | ((o & 0x0f0f0f0fu) << 4));
                    o = __shfl_xor_sync(0xffffffffu, v1, 1);
                    tb = (j & 1) ? ((v1 & 0xf0f0f0f0u) | ((o >> 4) & 0x0f0f0f0fu))
                                 : ((v1 & 0x0f0f0f0fu) | ((o & 0x0f0f0f0fu) << 4));
                }
            }
            if (!have || is_q) continue;
            void* vals = is_v ? p.v_out : p.k_out;
            if (vals) {
                T* dst = static_cast<T*>(vals) + (static_cast<size_t>(i) * p.Hkv + h) * D;
                Piece<T>::put(dst + 8 * pa, va);
                Piece<T>::put(dst + 8 * pb, vb);
            }
            if (page < 0) continue;
            uint8_t* blk = static_cast<uint8_t*>(is_v ? p.v_pool : p.k_pool) +
                           (((static_cast<size_t>(page) * p.Hkv + h) << (p.page_shift - 4)) +
                            (in_page >> 4)) * L4::kBlockBytes;
            const int r = in_page & 15;
            uint32_t* words = reinterpret_cast<uint32_t*>(blk);
            if (is_v) {
                if constexpr (D == 128) {
                    *reinterpret_cast<uint2*>(words + L4::v_word(r, j, 0)) = make_uint2(ta, tb);
                } else {
                    words[L4::v_word(r, j, 0)] = ta;
                    words[L4::v_word(r, j + 4, 0)] = tb;
                }
            } else {
                words[L4::k_word(r, pa)] = __funnelshift_l(wa, wa, 3);
                words[L4::k_word(r, pb)] = __funnelshift_l(wb, wb, 3);
            }
            if (j < L4::kGroups)
                *reinterpret_cast<__half2*>(blk + L4::param(r, j)) = j ? par[L4::kGroups - 1] : par[0];
        }
    }
}

template <typename T, int D, bool kQ4, int R>
int launch_rows(const RopeAppendParams& p, cudaStream_t stream) {
    constexpr int per = 32 / (D / 16) * R;
    const long long items = static_cast<long long>(p.T) * ((p.rows + per - 1) / per);
    const long long blocks = (items + 7) / 8;
    if (blocks > 0x7fffffffLL) return KVD_ERR_UNSUPPORTED;
    if (launch_kernel(rope_append_kernel<T, D, kQ4, R>, dim3(static_cast<unsigned>(blocks)),
                      dim3(256), 0, stream, p) != cudaSuccess)
        return KVD_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? KVD_OK : KVD_ERR_CUDA;
}

template <typename T, int D>
int launch_type(const RopeAppendParams& p, bool q4, cudaStream_t stream) {
    return q4 ? launch_rows<T, D, true, 1>(p, stream) : launch_rows<T, D, false, 1>(p, stream);
}

}  // namespace

int rope_append_launch(const RopeAppendParams& p, bool q4, int D, int dtype,
                       cudaStream_t stream) {
    if (dtype == KVD_BF16)
        return D == 128 ? launch_type<__nv_bfloat16, 128>(p, q4, stream)
                        : launch_type<__nv_bfloat16, 64>(p, q4, stream);
    return D == 128 ? launch_type<float, 128>(p, q4, stream)
                    : launch_type<float, 64>(p, q4, stream);
}

}  // namespace kvd
