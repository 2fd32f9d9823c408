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
// is a chain of dependent reads. Measured: one token of each of 32 sequences, 32 query and 8 KV
// heads of 128 bf16 channels, 1.9 us (2.3 into 4 bits); 9 prompts, 400 MB in all, 61 us, 98% of the
// rate of a copy (into 4 bits, with the stored values handed back, 71 us, 88%). What bounds the 4-bit
// form is the codes' instructions for each key and value row: with as many KV heads as query heads
// (8 and 8 of 128 bf16 channels, 365 MB) it takes 80 us, two thirds of the rate of a copy, the other
// form 51 us, 97%; 5 and 5 of 64, where a step of a warp has 8 row slots, 90 and 62 us, 37% and 50%.

#include <algorithm>

#include "kvd_device.cuh"
#include "kvd_host.h"
#include "kvd_q4.cuh"

namespace kvd {

namespace {

struct TokenAt {
    int slot, pos;      // slot < 0: the cache is not written
    bool ok;            // false: the row belongs to no token, or the token's length is bad
    int b, len, end;    // its sequence, that one's length, and the row behind its last new token's
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
// The same by one lane.
__device__ __forceinline__ int find_seq(const int32_t* cu, int B, int i) {
    int lo = -1, hi = B + 1;  // cu[lo] <= i < cu[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        (__ldg(cu + mid) <= i ? lo : hi) = mid;
    }
    return lo;
}

// Where token pos of a sequence with this length goes.
__device__ __forceinline__ int slot_of(const RopeAppendParams& p, int pos, int len) {
    if (p.window <= 0 || pos < p.n_sink) return pos;
    return pos >= len - p.window ? p.n_sink + (pos - p.n_sink) % p.window : -1;
}

// Where token i of sequence b goes.
__device__ __forceinline__ TokenAt place(const RopeAppendParams& p, int b, int i) {
    TokenAt a = {-1, 0, false, b, 0, 0};
    int before = i, n = 1;  // the sequence's first row, its new tokens
    if (p.cu_seqlens) {
        if (b < 0 || b >= p.B) return a;  // in front of the first or behind the last sequence
        before = __ldg(p.cu_seqlens + b);
        const int next = __ldg(p.cu_seqlens + b + 1);
        n = next - before;
        if (before > i || i >= next) {  // offsets that do not ascend
            record_error(p.err, KVD_ERR_DEVICE_OOB);
            return a;
        }
    }
    const int L = __ldg(p.seq_lens + b);
    const long long cap = static_cast<long long>(p.max_pages) << p.page_shift;
    a.pos = L - n + (i - before);
    if (n > L || a.pos >= p.max_pos || (p.window <= 0 && L > cap)) {
        record_error(p.err, KVD_ERR_DEVICE_OOB);
        return a;
    }
    a.ok = true;
    a.len = L;
    a.end = before + n;
    a.slot = slot_of(p, a.pos, L);
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

// One step of a transposition among neighbouring lanes: lane pairs kLane apart exchange the parts of
// kBits bits that belong to the other.
template <int kLane, int kBits>
__device__ __forceinline__ uint32_t swap_parts(uint32_t w, int lane) {
    constexpr uint32_t kLow = kBits == 16 ? 0x0000ffffu : kBits == 8 ? 0x00ff00ffu : 0x0f0f0f0fu;
    const uint32_t o = __shfl_xor_sync(0xffffffffu, w, kLane);
    return (lane & kLane) ? (w & ~kLow) | ((o >> kBits) & kLow)
                          : (w & kLow) | ((o & kLow) << kBits);
}
// Nibble m of lane j's word becomes nibble j of lane m's word, among 8 neighbouring lanes.
__device__ __forceinline__ uint32_t transpose_nibbles(uint32_t w, int lane) {
    return swap_parts<1, 4>(swap_parts<2, 8>(swap_parts<4, 16>(w, lane), lane), lane);
}

// Minimum and maximum that keep a NaN.
__device__ __forceinline__ float min3(float a, float b, float c) {
    float d;
    asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
template <int N>
__device__ __forceinline__ float least(const float (&x)[N]) {
    float d = min3(x[0], x[1], x[2]);
#pragma unroll
    for (int e = 3; e < N; e += 2) d = min3(d, x[e], x[e + 1 < N ? e + 1 : e]);
    return d;
}
template <int N>
__device__ __forceinline__ float most(const float (&x)[N]) {
    float d = max3(x[0], x[1], x[2]);
#pragma unroll
    for (int e = 3; e < N; e += 2) d = max3(d, x[e], x[e + 1 < N ? e + 1 : e]);
    return d;
}

// 4-bit codes of a row whose lane has pieces pa and pb (x, y): stored in the token's block, and,
// where `vals` is given, as the values that they stand for. Every lane of the warp comes here;
// `store` and `vals` say whether this lane's row is written.
template <typename T, int D, bool kV>
__device__ __forceinline__ void put_q4(float (&x)[8], float (&y)[8], int pa, int pb, int j,
                                       uint8_t* blk, int r, bool store, T* vals) {
    using L4 = Q4<D>;
    constexpr int kTeam = D / 16, NG = L4::kGroups;
    constexpr float kInf = __builtin_huge_valf();
    // Scale and minimum of the row's groups (piece c belongs to group c / 8). Clamping to the
    // float16 range commutes with minimum and maximum; a NaN stays in them, an infinity shows in
    // one of them.
    const float lo_a = least<8>(x), hi_a = most<8>(x), lo_b = least<8>(y), hi_b = most<8>(y);
    // (one group: both pieces are of it; two: pieces a and b are of groups 0 and 1, or, with fewer
    // channels rotated, of any)
    float lo[NG], hi[NG];
    if constexpr (NG == 1) {
        lo[0] = min3(lo_a, lo_b, lo_b), hi[0] = max3(hi_a, hi_b, hi_b);
    } else {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const bool ag = pa >> 3 == g, bg = pb >> 3 == g;
            const float la = ag ? lo_a : kInf, lb = bg ? lo_b : kInf;
            const float ha = ag ? hi_a : -kInf, hb = bg ? hi_b : -kInf;
            lo[g] = min3(la, lb, lb), hi[g] = max3(ha, hb, hb);
        }
    }
#pragma unroll
    for (int off = 1; off < kTeam; off <<= 1)
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const float ol = __shfl_xor_sync(0xffffffffu, lo[g], off);
            const float oh = __shfl_xor_sync(0xffffffffu, hi[g], off);
            lo[g] = min3(lo[g], ol, ol), hi[g] = max3(hi[g], oh, oh);
        }
    // The values themselves: below -65504 (then b is that) a code is 0 either way, but past 65504 it
    // would follow the value instead of its clamp where the minimum is next to 65504 as well. Rare,
    // so one comparison a row decides.
    if (hi[0] > 65504.f || hi[NG - 1] > 65504.f) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = fminf(x[e], 65504.f), y[e] = fminf(y[e], 65504.f);
    }
    float step[NG], base[NG], inv[NG];
    uint32_t par[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        const bool bad = !(lo[g] > -kInf && hi[g] < kInf);
        const float l = fminf(fmaxf(lo[g], -65504.f), 65504.f);
        const float h = fminf(fmaxf(hi[g], -65504.f), 65504.f);
        const __half hb = bad ? __ushort_as_half(0x7fff) : __float2half_rn(l);
        const __half hs = bad ? __ushort_as_half(0)
                              : __float2half_rn(__fmul_rn(__fsub_rn(h, l), 1.0f / 15.0f));
        step[g] = __half2float(hs);
        base[g] = __half2float(hb);
        inv[g] = step[g] > 0.f ? __frcp_rn(step[g]) : 0.f;
        par[g] = __half_as_ushort(hs) | static_cast<uint32_t>(__half_as_ushort(hb)) << 16;
    }
    const bool a1 = NG == 2 && pa >= 8, b1 = NG == 2 && pb >= 8;
    const float base_a = a1 ? base[NG - 1] : base[0], base_b = b1 ? base[NG - 1] : base[0];
    const float inv_a = a1 ? inv[NG - 1] : inv[0], inv_b = b1 ? inv[NG - 1] : inv[0];
    // rounding by adding 1.5 2^23: the code is then the sum's low bits (a NaN group has factor 0
    // and a NaN minimum: the comparison makes it 0)
    constexpr float kMagic = 12582912.f;
    auto code = [&](float v, float from, float by) {
        const float c = __fmul_rn(__fsub_rn(v, from), by);
        return __fadd_rn(fminf(fmaxf(c, 0.f), 15.f), kMagic);
    };
    uint32_t wa = 0, wb = 0;
#pragma unroll
    for (int e = 7; e >= 0; --e) {  // x and y become the codes (plus kMagic)
        x[e] = code(x[e], base_a, inv_a);
        y[e] = code(y[e], base_b, inv_b);
        wa = wa * 16 + __float_as_uint(x[e]);
        wb = wb * 16 + __float_as_uint(y[e]);
    }
    wa -= 0x4B400000u * 0x11111111u;
    wb -= 0x4B400000u * 0x11111111u;
    if (vals) {
        const float step_a = a1 ? step[NG - 1] : step[0], step_b = b1 ? step[NG - 1] : step[0];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] = fmaf(step_a, x[e] - kMagic, base_a);
            y[e] = fmaf(step_b, y[e] - kMagic, base_b);
        }
        Piece<T>::put(vals + 8 * pa, x);
        Piece<T>::put(vals + 8 * pb, y);
    }
    uint32_t* words = reinterpret_cast<uint32_t*>(blk);
    if constexpr (!kV) {
        if (store) {
            words[L4::k_word(r, pa)] = __funnelshift_l(wa, wa, 3);
            words[L4::k_word(r, pb)] = __funnelshift_l(wb, wb, 3);
        }
    } else if constexpr (D == 128) {
        wa = transpose_nibbles(wa, j);
        wb = transpose_nibbles(wb, j);
        if (store)
            *reinterpret_cast<uint2*>(words + L4::v_word(r, j, 0)) = make_uint2(wa, wb);
    } else {  // pieces j and j + 4 of the 8: the first exchange stays in the thread
        const uint32_t u = (wa & 0x0000ffffu) | (wb << 16), v = (wa >> 16) | (wb & 0xffff0000u);
        wa = swap_parts<1, 4>(swap_parts<2, 8>(u, j), j);
        wb = swap_parts<1, 4>(swap_parts<2, 8>(v, j), j);
        if (store) {
            words[L4::v_word(r, j, 0)] = wa;
            words[L4::v_word(r, j + 4, 0)] = wb;
        }
    }
    if (store && j < NG)
        *reinterpret_cast<uint32_t*>(blk + L4::param(r, j)) = j ? par[NG - 1] : par[0];
}

// Rows begin .. end - 1 of one kind (0 queries, 1 keys, 2 values) of token i0, by one warp, R rows of
// a lane at a time. kFew: all rows (at most half of those that a warp has lanes for), 1 << log_rows
// lanes' rows for each, of token i0 and the ones behind it; their sequence is i0's mostly.
template <typename T, int D, bool kQ4, int R, int kKind, bool kFew>
__device__ __forceinline__ void append_rows(const RopeAppendParams& p, int i0, int begin, int end,
                                            int lane, int log_rows) {
    using L4 = Q4<D>;
    constexpr int kTeam = D / 16;       // lanes of a row
    constexpr int kTeams = 32 / kTeam;  // rows of a warp at once
    static_assert(!kFew || R == 1, "one step");
    const int team = kFew ? lane / kTeam & ((1 << log_rows) - 1) : lane / kTeam, j = lane % kTeam;
    const int i = kFew ? i0 + (lane / kTeam >> log_rows) : i0;
    const T* src = kKind == 0   ? static_cast<const T*>(p.q) + i * p.q_stride
                   : kKind == 1 ? static_cast<const T*>(p.k) + i * p.k_stride
                                : static_cast<const T*>(p.v) + i * p.v_stride;
    // pieces of a rotated row: (c, c + rot/16) for the pairs, then neighbours; of a value row
    // (j, j + D/16)
    const int rp = p.rot / 16;
    const int pa = kKind == 2 || j < rp ? j : 2 * j;
    const int pb = kKind == 2 ? j + kTeam : j < rp ? j + rp : 2 * j + 1;
    Piece<T> a[R], b[R];
    auto load = [&](int k, int row) {
        if (row < end && (!kFew || i < p.T)) {
            a[k].load(src + row * D + 8 * pa);
            b[k].load(src + row * D + 8 * pb);
        }
    };
#pragma unroll
    for (int k = 0; k < R; ++k) load(k, begin + team + k * kTeams);
    TokenAt at = place(p, p.cu_seqlens ? find_seq(p.cu_seqlens, p.B, i0, lane) : i0, i0);
    if constexpr (kFew) {
        if (i >= p.T) {
            at.ok = false;
        } else if (i > i0) {
            if (at.ok && i < at.end && at.pos + (i - i0) < p.max_pos) {
                at.pos += i - i0;
                at.slot = slot_of(p, at.pos, at.len);
            } else {
                at = place(p, p.cu_seqlens ? find_seq(p.cu_seqlens, p.B, i) : i, i);
            }
        }
        if (!at.ok) at.slot = -1;
    } else {
        if (!at.ok) return;
    }
    const bool turns = kKind != 2 && j < rp && (!kFew || at.ok);
    // where the rows go: queries, or the cache's rows of this token
    T* dst = nullptr;    // (null: not written)
    uint8_t* blk = nullptr;
    T* vals = nullptr;
    size_t dst_row = D;  // elements, or bytes of 4-bit pages, between heads
    const int in_page = at.slot & ((1 << p.page_shift) - 1);
    if constexpr (kKind == 0) {
        if (!kFew || at.ok) dst = static_cast<T*>(p.q_out) + static_cast<size_t>(i) * p.Hq * D;
    } else {
        void* pool = kKind == 2 ? p.v_pool : p.k_pool;
        int page = -1;
        if (at.slot >= 0) {
            page = __ldg(p.block_table + static_cast<size_t>(at.b) * p.max_pages +
                         (at.slot >> p.page_shift));
            if (page < 0 || page >= p.num_pages) {
                record_error(p.err, KVD_ERR_DEVICE_OOB);
                page = -1;
            }
        }
        if constexpr (kQ4) {
            dst_row = static_cast<size_t>(L4::kBlockBytes) << (p.page_shift - 4);
            if (page >= 0)
                blk = static_cast<uint8_t*>(pool) + page * (p.Hkv * dst_row) +
                      (in_page >> 4) * L4::kBlockBytes;
            if (!kFew || at.ok) vals = static_cast<T*>(kKind == 2 ? p.v_out : p.k_out);
            if (vals) vals += static_cast<size_t>(i) * p.Hkv * D;
        } else {
            dst_row = static_cast<size_t>(D) << p.page_shift;
            if (page >= 0)
                dst = static_cast<T*>(pool) + page * (p.Hkv * dst_row) +
                      static_cast<size_t>(in_page) * D;
        }
    }
    // cosines and sines of this lane's pairs: halves share them (8 + 8), interleaved pieces have
    // four pairs each
    float cs[8], sn[8];
    if (turns) {
        const float* row = p.cos_sin + static_cast<size_t>(at.pos) * p.rot;
        const int h = p.rot / 2;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int o = p.interleaved ? (e ? pb : pa) * 4 : pa * 8 + 4 * e;
            const float4 c = __ldg(reinterpret_cast<const float4*>(row + o));
            const float4 s = __ldg(reinterpret_cast<const float4*>(row + h + o));
            cs[4 * e] = c.x, cs[4 * e + 1] = c.y, cs[4 * e + 2] = c.z, cs[4 * e + 3] = c.w;
            sn[4 * e] = s.x, sn[4 * e + 1] = s.y, sn[4 * e + 2] = s.z, sn[4 * e + 3] = s.w;
        }
    }
    for (int row0 = begin; row0 < end; row0 += kTeams * R) {
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if (k > 0 && row0 + k * kTeams >= end) break;
            const int row = row0 + k * kTeams + team;
            float x[8], y[8];
            a[k].get(x);
            b[k].get(y);
            load(k, row + kTeams * R);  // the next step's
            if (turns) {
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
            if constexpr (kQ4 && kKind != 0) {
                const bool have = row < end;
                put_q4<T, D, kKind == 2>(x, y, pa, pb, j, blk + row * dst_row, in_page & 15,
                                         have && blk, have && vals ? vals + row * D : nullptr);
            } else if (row < end && dst) {
                Piece<T>::put(dst + row * dst_row + 8 * pa, x);
                Piece<T>::put(dst + row * dst_row + 8 * pb, y);
            }
        }
    }
}

// A warp's token, kind and rows. The kinds have code of their own (the queries' registers are not the
// codes'), but one launch. kBlocks: CTAs that an SM is to hold at least.
template <typename T, int D, bool kQ4, int R, int kBlocks>
__global__ void __launch_bounds__(256, kBlocks) rope_append_kernel(const RopeAppendParams p) {
    griddep_wait();
    const uint32_t item = blockIdx.x * 8 + threadIdx.x / 32;
    const uint32_t per = p.q_items + 2 * p.kv_items;
    const int i = static_cast<int>(item / per);
    if (i >= p.T) return;
    int part = static_cast<int>(item % per);
    const int lane = threadIdx.x % 32;
    if (part < p.q_items) {
        append_rows<T, D, kQ4, R, 0, false>(p, i, part * p.q_rows, min(p.Hq, (part + 1) * p.q_rows),
                                            lane, 0);
        return;
    }
    part -= p.q_items;
    const bool values = part >= p.kv_items;
    if (values) part -= p.kv_items;
    const int begin = part * p.kv_rows, end = min(p.Hkv, begin + p.kv_rows);
    constexpr int kR = kQ4 ? 1 : R;  // (the codes take the registers)
    if (values)
        append_rows<T, D, kQ4, kR, 2, false>(p, i, begin, end, lane, 0);
    else
        append_rows<T, D, kQ4, kR, 1, false>(p, i, begin, end, lane, 0);
}

// Few heads: a warp has lanes for the keys (or values, or queries, if they are few as well) of several
// tokens. Warps of queries come first, then those of keys, then of values; q_items, kv_items: all.
template <typename T, int D, bool kQ4>
__global__ void __launch_bounds__(256, 3) rope_append_few_kernel(const RopeAppendParams p) {
    constexpr int kTeams = 32 / (D / 16);
    griddep_wait();
    uint32_t item = blockIdx.x * 8 + threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    if (item < static_cast<uint32_t>(p.q_items)) {
        if (p.q_log >= 0) {
            append_rows<T, D, kQ4, 1, 0, true>(p, item * (kTeams >> p.q_log), 0, p.Hq, lane, p.q_log);
        } else {
            const int per = (p.Hq + p.q_rows - 1) / p.q_rows, begin = item % per * p.q_rows;
            append_rows<T, D, kQ4, 1, 0, false>(p, item / per, begin, min(p.Hq, begin + p.q_rows),
                                                lane, 0);
        }
        return;
    }
    item -= p.q_items;
    const int step = kTeams >> p.kv_log;
    if (item < static_cast<uint32_t>(p.kv_items))
        append_rows<T, D, kQ4, 1, 1, true>(p, item * step, 0, p.Hkv, lane, p.kv_log);
    else if (item < 2u * p.kv_items)
        append_rows<T, D, kQ4, 1, 2, true>(p, (item - p.kv_items) * step, 0, p.Hkv, lane, p.kv_log);
}

template <typename... P>
int launch_items(void (*kernel)(P...), const RopeAppendParams& p, long long items,
                 cudaStream_t stream) {
    if (items >= (1LL << 31) - 8) return KVD_ERR_UNSUPPORTED;
    if (launch_kernel(kernel, dim3(static_cast<unsigned>((items + 7) / 8)), dim3(256), 0, stream,
                      p) != cudaSuccess)
        return KVD_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? KVD_OK : KVD_ERR_CUDA;
}

// `steps`: steps of a warp (its rows are that many times a step's).
template <typename T, int D, bool kQ4, int R, int kBlocks>
int launch_rows(RopeAppendParams p, int steps, cudaStream_t stream) {
    p.q_rows = p.kv_rows = 32 / (D / 16) * R * steps;
    p.q_items = (p.Hq + p.q_rows - 1) / p.q_rows;
    p.kv_items = (p.Hkv + p.kv_rows - 1) / p.kv_rows;
    return launch_items(rope_append_kernel<T, D, kQ4, R, kBlocks>, p,
                        static_cast<long long>(p.T) * (p.q_items + 2 * p.kv_items), stream);
}

template <typename T, int D, bool kQ4>
int launch_few(RopeAppendParams p, cudaStream_t stream) {
    constexpr int teams = 32 / (D / 16);
    auto log_of = [](int heads) {
        int n = 0;
        while (1 << n < heads) ++n;
        return n;
    };
    auto warps_of_log = [&](int n) { return (p.T + (teams >> n) - 1LL) / (teams >> n); };
    p.q_rows = 2 * teams;
    p.q_log = 2 * p.Hq <= teams ? log_of(p.Hq) : -1;  // (-1: the general form)
    p.kv_log = log_of(p.Hkv);
    const long long q = p.Hq == 0 ? 0
                        : p.q_log >= 0 ? warps_of_log(p.q_log)
                                       : static_cast<long long>(p.T) * ((p.Hq + p.q_rows - 1) / p.q_rows);
    const long long kv = warps_of_log(p.kv_log);
    if (q + 2 * kv >= (1LL << 31) - 8) return KVD_ERR_UNSUPPORTED;
    p.q_items = static_cast<int>(q);
    p.kv_items = static_cast<int>(kv);
    return launch_items(rope_append_few_kernel<T, D, kQ4>, p, q + 2 * kv, stream);
}

template <typename T, int D, bool kQ4>
int launch_type(const RopeAppendParams& p, cudaStream_t stream) {
    constexpr int teams = 32 / (D / 16);
    const long long warps = static_cast<long long>(p.T) *
                            ((p.Hq + teams - 1) / teams + 2 * ((p.Hkv + teams - 1) / teams));
    // Few rows: one step a warp, as many warps as there are, for the shortest chain of reads.
    // Many: two steps of a warp share the token's look-up, with more warps on an SM. Measured (us,
    // 40 rows of 128 bf16 a token and 8 of values; one step against two): 192 tokens 2.59 / 2.78,
    // 384 3.72 / 3.36, 3000 19.9 / 14.1; into 4 bits 192 3.07 / 3.87, 384 4.67 / 4.72, 3000 28.9 /
    // 16.4; float32 192 3.18 / 3.15, 3000 33.2 / 25.6. 20 warps an SM are about 250 such tokens.
    if (warps <= 20LL * num_sms()) return launch_rows<T, D, kQ4, 1, 1>(p, 1, stream);
    // Few heads: the lanes of several tokens in a warp, from two (bf16) or four (float32, whose rows are
    // longer) on. 12000 tokens of 1 head of 128 5.0 us (14.4 otherwise), into 4 bits 7.6 (23.1); 3000 of
    // 2 heads of 128 bf16 4.4 (5.2), float32 7.6 (7.1); 8000 of 1 head of 64 float32 8.3 (11.9).
    if ((sizeof(T) == 2 ? 2 : 4) * p.Hkv <= teams) return launch_few<T, D, kQ4>(p, stream);
    // (Registers are held to 64 and 80 a thread for the warps that the loads need; the 4-bit kernels then
    // spill 56 to 72 bytes of a thread in bf16, 20 to 32 in float32.)
    if constexpr (sizeof(T) == 2)
        return launch_rows<T, D, kQ4, 2, 4>(p, 2, stream);
    else  // (a float32 row is two bf16 ones)
        return launch_rows<T, D, kQ4, 1, 3>(p, 2, stream);
}

}  // namespace

int rope_append_launch(const RopeAppendParams& p, bool q4, int D, int dtype,
                       cudaStream_t stream) {
    if (dtype == KVD_BF16) {
        if (D == 128)
            return q4 ? launch_type<__nv_bfloat16, 128, true>(p, stream)
                      : launch_type<__nv_bfloat16, 128, false>(p, stream);
        return q4 ? launch_type<__nv_bfloat16, 64, true>(p, stream)
                  : launch_type<__nv_bfloat16, 64, false>(p, stream);
    }
    if (D == 128)
        return q4 ? launch_type<float, 128, true>(p, stream)
                  : launch_type<float, 128, false>(p, stream);
    return q4 ? launch_type<float, 64, true>(p, stream) : launch_type<float, 64, false>(p, stream);
}

}  // namespace kvd
