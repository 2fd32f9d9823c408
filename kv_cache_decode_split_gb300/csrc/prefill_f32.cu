// prefill_f32.cu -- causal attention of many new tokens of each sequence, float32, over packed keys and
// values or over a paged cache (the formulas are in prefill_bf16.cu).
//
// Products. A float32 number is the sum of three bfloat16 numbers (3 x 8 bits of significand, the same
// exponents), x = x1 + x2 + x3, each the rounding of what the ones before it leave. Of the nine products
// of two such sums the six of at least 2^-16 are kept, x1 y1 + x1 y2 + x2 y1 + x2 y2 + x1 y3 + x3 y1; the
// three left out are below 2^-24 of |x||y| each. (Three products of two tf32 numbers cost as much time
// at half the rate, and a third more shared memory. On CUDA cores the chunks below took 3.9 ms.)
// The smallest products are added first. A tensor core cuts what it adds, so the weighted sums of one
// 64-key tile at most are left to it: every tile's outputs start from zero and are added to float32
// registers, rounded.
//
// Bound by the converting warps: 500 instructions for 64 rows, two such items a tile, and one buffer for
// each (at D = 128, where a set of operands takes 192 KB, there is no room for a second; at D = 64 there
// would be), so that a tile of D = 128 takes 6600 cycles where the products take 3800
// and shared memory, which the score product's operands fill (6 KB for 128 x 64 x 16), 4400. Six chunks of
// 1 to 301 tokens behind 400 to 5003, 14/2 heads of 128: 118 us, 96 TFLOP/s of the formula's operations,
// a sixth of those issued; the windowed prompts below 118 us. (Pages looked up two items ahead, or 32-byte
// loads, change nothing.)
//
// One persistent CTA an SM takes units of one query tile (128 rows: the G query heads of a KV head of
// 128 / G tokens) from the list of prefill_common.cuh. Roles:
//   * eight warps read queries, keys and values, split them and write the parts to shared memory in the
//     tensor core's layout; values that are not finite are cleared (their split is NaN), and the rows
//     that see them get them back at the end;
//   * a warp issues S = Q K^T (6 x D / 16 steps), another O = P V (6 x 4 steps): the scores of the next
//     tile are under way while this tile's softmax runs;
//   * four warps, a row a thread: running maximum and sum, weights split into three parts for tensor
//     memory, outputs in registers. They read the scores twice, 32 at a time, in rolled loops (with a row's
//     64 in registers and all loops unrolled the kernel was 145 KB of code, now 90, and the chunks took
//     169 us), and add a tile's outputs behind the next tile's weights.

#include <algorithm>

#include "prefill_common.cuh"

namespace kvd {

namespace {

using namespace prefill;

constexpr int kN = 64;       // keys of a tile
constexpr int kThreads = 512;
constexpr int kSoftWarps = 4, kConvWarps = 8;
constexpr int kWarpConv = 4, kWarpWalk = 12, kWarpQk = 13, kWarpPv = 14;
// registers of a thread of the softmax's, the two converting and the last warpgroup, of 128 at launch
constexpr int kRegsSoft = 232, kRegsConv = 104, kRegsOther = 72;
static_assert(kRegsSoft + 2 * kRegsConv + kRegsOther <= 4 * 128, "registers");
constexpr uint32_t kColS = 0, kColP = 128, kColO = 256;  // two score tiles; 3 x 32; two of D

template <int D>
struct Smem {
    uint8_t q[3][kM * D * 2];  // offset 0; every part is a multiple of 1024 bytes
    uint8_t k[3][kN * D * 2];
    uint8_t v[3][kN * D * 2];
    uint64_t qfull, qempty, kfull, kempty, vfull, vempty, sfull[2], pready[2], ofull;
    uint64_t pfull[kPieces], pempty[kPieces], end[2], never;
    Piece piece[kPieces];
    uint32_t bad[kPieces];  // tiles with values that are not finite
    uint32_t tmem_base;
};

// Two numbers as three pairs of bfloat16 numbers.
__device__ __forceinline__ void split2(float x, float y, uint32_t& a, uint32_t& b, uint32_t& c) {
    a = pack_bf16(x, y);
    x -= __uint_as_float(a << 16);
    y -= __uint_as_float(a & 0xffff0000u);
    b = pack_bf16(x, y);
    x -= __uint_as_float(b << 16);
    y -= __uint_as_float(b & 0xffff0000u);
    c = pack_bf16(x, y);
}

// The products that are kept, smallest first: part of the left and of the right operand.
__device__ __forceinline__ int left_part(int i) { return (0x001102 >> (4 * i)) & 3; }   // 2 0 1 1 0 0
__device__ __forceinline__ int right_part(int i) { return (0x010120 >> (4 * i)) & 3; }  // 0 2 1 0 1 0

// ---------------------------------------------------------------------------------- converting
// Eight channels (chunk c8) of a row into their three places; part: bytes of a part, rows: of a tile.
__device__ __forceinline__ void put_split(uint8_t* base, int part, int rows, int row, int c8,
                                          const float4& lo, const float4& hi) {
    uint4 a, b, c;
    split2(lo.x, lo.y, a.x, b.x, c.x);
    split2(lo.z, lo.w, a.y, b.y, c.y);
    split2(hi.x, hi.y, a.z, b.z, c.z);
    split2(hi.z, hi.w, a.w, b.w, c.w);
    uint8_t* at = base + swz128(row, c8 * 8, rows);
    *reinterpret_cast<uint4*>(at) = a;
    *reinterpret_cast<uint4*>(at + part) = b;
    *reinterpret_cast<uint4*>(at + 2 * part) = c;
}

__device__ __forceinline__ bool splits4(const float4& v) {
    return splits(v.x) && splits(v.y) && splits(v.z) && splits(v.w);
}
__device__ __forceinline__ void clear4(float4& v) {
    v.x = splits(v.x) ? v.x : 0.f;
    v.y = splits(v.y) ? v.y : 0.f;
    v.z = splits(v.z) ? v.z : 0.f;
    v.w = splits(v.w) ? v.w : 0.f;
}

// A unit's items of 64 rows: the queries (two), then keys and values, K(0), K(1), V(0), K(2), V(1), ...
// An item's rows are on their way while the one before it is split. (One loop for all of them: code that
// is not in the instruction caches costs more than its selects.)
template <int D>
__device__ void convert_role(const PrefillParams& p, Smem<D>& sm, int tid, int lane) {
    constexpr int kRow = D / 8;                    // chunks of a row
    constexpr int kEach = kN * kRow / 256;         // chunks of an item that a thread takes
    constexpr int kStep = 256 / kRow;              // in rows r0 + i * kStep
    struct Rows {
        float4 x[kEach][2];
    };
    const int TM = kM / p.G;
    int* err = p.err;
    const int c8 = tid % kRow, r0 = tid / kRow;
    uint32_t nq = 0, nk = 0, nv = 0;
    bool ok = !stalls(p, &sm.never, 4);
    for (int k = 0; ok; ++k) {
        const int slot = k % kPieces;
        if (!wait(&sm.pfull[slot], (k / kPieces) & 1, p)) break;
        const Piece pc = sm.piece[slot];
        if (pc.t0 < 0) break;
        const int nt = pc.t1 - pc.t0, items = nt > 0 ? 2 * nt : -2;
        // the first key in the first row's window: those before it, that are no sinks, no row of the unit sees
        // (and their pages may be gone)
        const int low = p.window > 0 ? pc.L - pc.n + pc.tok0 - p.window + 1 : 0;
        // item i: -2 and -1 are the queries
        auto is_value = [&](int i) { return i == items - 1 || (i > 0 && i % 2 == 0); };
        auto load = [&](Rows& rows, int i) {
            const bool is_v = is_value(i);
            const int t0 = i < 0 ? 0 : tile_of(pc, pc.t0 + (is_v ? (i == items - 1 ? nt : i / 2) - 1 : (i + 1) / 2)) * kN;
            const float* base = static_cast<const float*>(i < 0 ? p.q : is_v ? p.v : p.k);
            const long long stride = is_v ? p.v_stride : p.k_stride;
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const int r = r0 + e * kStep;
                const float* at = nullptr;  // the row; null for one of zeros
                if (i < 0) {
                    const int row = (i + 2) * kN + r, t = row / p.G, token = pc.tok0 + t;
                    if (t < TM && token < pc.n)
                        at = base + (pc.c0 + token) * p.q_stride +
                             (pc.h * p.G + (row - t * p.G)) * static_cast<long long>(D);
                } else if (t0 + r < pc.L && (t0 + r >= low || t0 + r < p.n_sink)) {
                    if (p.block_table) {
                        const int key = t0 + r;
                        const int pg = load_page(p.block_table, p.max_pages, p.num_pages, pc.k0,
                                                 key >> p.page_shift, err);
                        at = base + (((static_cast<size_t>(pg) * p.Hkv + pc.h) << p.page_shift) +
                                     (key & ((1 << p.page_shift) - 1))) * D;
                    } else {
                        at = base + (pc.k0 + t0 + r) * stride + pc.h * D;
                    }
                }
                rows.x[e][0] = rows.x[e][1] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (at) {
                    rows.x[e][0] = reinterpret_cast<const float4*>(at)[2 * c8];
                    rows.x[e][1] = reinterpret_cast<const float4*>(at)[2 * c8 + 1];
                }
            }
        };
        Rows rows, next;
        if (items > 0) load(next, -2);
#pragma unroll 1
        for (int i = -2; i < items; ++i) {
            rows = next;
            if (i + 1 < items) load(next, i + 1);
            const bool is_v = is_value(i);
            uint64_t* full = i < 0 ? &sm.qfull : is_v ? &sm.vfull : &sm.kfull;
            if (i != -1) {  // (the queries' halves are one wait and one arrival)
                uint32_t& n = i < 0 ? nq : is_v ? nv : nk;
                if (!(ok = wait(i < 0 ? &sm.qempty : is_v ? &sm.vempty : &sm.kempty, (n & 1) ^ 1, p))) break;
                ++n;
            }
            if (is_v) {
                bool bad = false;
#pragma unroll
                for (int e = 0; e < kEach; ++e)
                    if (!(splits4(rows.x[e][0]) && splits4(rows.x[e][1]))) {
                        clear4(rows.x[e][0]);
                        clear4(rows.x[e][1]);
                        bad = true;
                    }
                if (bad)
                    atomicOr(&sm.bad[slot], 1u << (((i == items - 1 ? nt : i / 2) - 1) >> odd_shift(pc)));
            }
            uint8_t* dst = i < 0 ? sm.q[0] : is_v ? sm.v[0] : sm.k[0];
            const int height = i < 0 ? kM : kN, first = i == -1 ? kN : 0;
#pragma unroll
            for (int e = 0; e < kEach; ++e)
                put_split(dst, height * D * 2, height, first + r0 + e * kStep, c8, rows.x[e][0], rows.x[e][1]);
            if (i == -2) continue;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(full);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.pempty[slot]);
    }
}

// ---------------------------------------------------------------------------------- products
// Scores and outputs are issued by a warp each, so that the tensor core has the one's products while the
// other waits or commits; all lanes take the loops, so that descriptors are in uniform registers, which a
// product's instruction reads. (Five windowed prompts of 33 to 1500 tokens, 16/4 heads of 64: 117 us; one
// thread for both: 142; two threads: 134.)
template <int D>
__device__ void qk_role(const PrefillParams& p, Smem<D>& sm, int lane) {
    constexpr uint32_t id = idesc_bf16_f32(kM, kN, 0, 0);
    const uint64_t q = sw128_kmajor_desc(smem_u32(sm.q[0])), kk = sw128_kmajor_desc(smem_u32(sm.k[0]));
    const bool one = lane == 0;
    uint32_t nq = 0, nk = 0;  // query tiles, key tiles taken
    bool ok = !stalls(p, &sm.never, 2);
    for (int k = 0; ok; ++k) {
        const int i = k % kPieces;
        if (!wait(&sm.pfull[i], (k / kPieces) & 1, p)) break;
        const int t0 = sm.piece[i].t0, nt = sm.piece[i].t1 - t0;
        __syncwarp();
        if (one) mbar_arrive(&sm.pempty[i]);
        if (t0 < 0) break;
        if (nt == 0) continue;
        if (!(ok = wait(&sm.qfull, nq++ & 1, p))) break;
#pragma unroll 1
        for (int t = 0; t < nt; ++t, ++nk) {
            // (the scores two tiles ago have been read)
            if (!(ok = wait(&sm.pready[nk & 1], ((nk >> 1) & 1) ^ 1, p) && wait(&sm.kfull, nk & 1, p))) break;
            tc_fence_after();
            const uint32_t s = sm.tmem_base + kColS + kN * (nk & 1);
#pragma unroll 1
            for (int j = 0; j < 6; ++j) {
                const uint64_t a = q + ((left_part(j) * kM * D * 2) >> 4);
                const uint64_t b = kk + ((right_part(j) * kN * D * 2) >> 4);
                if (one) {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    tc_mma_bf16(s, a + (((ks >> 2) * kM * 128 + (ks & 3) * 32) >> 4),
                                b + (((ks >> 2) * kN * 128 + (ks & 3) * 32) >> 4), id, j + ks > 0 ? 1u : 0u);
                }
            }
            if (one) {
                tc_commit(&sm.sfull[nk & 1]);
                tc_commit(&sm.kempty);
            }
        }
        if (ok && one) tc_commit(&sm.qempty);
    }
    if (one) tc_commit(&sm.end[0]);  // all products complete before tensor memory is released
    drain(&sm.end[0], 0, p);
}

template <int D>
__device__ void pv_role(const PrefillParams& p, Smem<D>& sm, int lane) {
    constexpr uint32_t id = idesc_bf16_f32(kM, D, 0, 1);
    const uint64_t v = sw128_mnmajor_desc(smem_u32(sm.v[0]), kN * 128);
    const bool one = lane == 0;
    uint32_t np = 0;  // value tiles taken
    bool ok = !stalls(p, &sm.never, 3);
    for (int k = 0; ok; ++k) {
        const int i = k % kPieces;
        if (!wait(&sm.pfull[i], (k / kPieces) & 1, p)) break;
        const int t0 = sm.piece[i].t0, nt = sm.piece[i].t1 - t0;
        __syncwarp();
        if (one) mbar_arrive(&sm.pempty[i]);
        if (t0 < 0) break;
#pragma unroll 1
        for (int t = 0; t < nt; ++t, ++np) {
            if (!(ok = wait(&sm.vfull, np & 1, p) && wait(&sm.pready[np & 1], (np >> 1) & 1, p))) break;
            tc_fence_after();
            const uint32_t o = sm.tmem_base + kColO + 128 * (np & 1);
#pragma unroll 1
            for (int j = 0; j < 6; ++j) {
                const uint32_t a = sm.tmem_base + kColP + left_part(j) * (kN / 2);
                const uint64_t b = v + ((right_part(j) * kN * D * 2) >> 4);
                if (one) {
#pragma unroll
                    for (int ks = 0; ks < kN / 16; ++ks)
                        tc_mma_bf16_ts(o, a + ks * 8, b + ((ks * 16 * 128) >> 4), id, j + ks > 0 ? 1u : 0u);
                }
            }
            if (one) {
                tc_commit(&sm.ofull);
                tc_commit(&sm.vempty);
            }
        }
    }
    if (one) tc_commit(&sm.end[1]);
    drain(&sm.end[1], 0, p);
}

// ----------------------------------------------------------------------------------- softmax
// Values that are not finite, put back into the row (of the piece's 128) that a lane has written.
template <int D>
__device__ __noinline__ void put_back_rows(const PrefillParams& p, const Piece& pc, uint32_t marks, int r) {
    const int TM = kM / p.G, t = r / p.G, token = pc.tok0 + t;
    const long long at = pc.slot < 0 ? static_cast<long long>(pc.c0 + token) * p.Hq + pc.h * p.G + (r - t * p.G)
                                     : static_cast<long long>(pc.slot) * 2 * kM + r;
    put_back<D, kN, float, false>(p, pc, marks, TM, t < TM && token < pc.n, pc.L - pc.n + token,
                                  (pc.slot < 0 ? static_cast<float*>(p.out) : p.part_o) + at * D, false,
                                  threadIdx.x % 32);
}

__device__ __forceinline__ uint64_t first_bits(int n) {
    return n <= 0 ? 0 : n >= 64 ? ~0ull : (1ull << n) - 1;
}

template <int D>
__device__ void softmax_role(const PrefillParams& p, Smem<D>& sm, int warp, int lane) {
    const int r = warp * 32 + lane;  // row of the tile, lane of tensor memory
    const int TM = kM / p.G, U = TM;
    const uint32_t quad = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t tmem = sm.tmem_base + quad;
    const bool negative = p.scale_log2 < 0.f;
    const float c = fmaxf(fabsf(p.scale_log2), 0x1p-100f);  // (0: -inf times it stays -inf)
    const int tok_r = r / p.G, head_r = r - tok_r * p.G;
    uint32_t ns = 0, no = 0;  // score tiles and output tiles taken
    if (stalls(p, &sm.never, 5)) return;
    for (int k = 0;; ++k) {
        const int i = k % kPieces;
        if (!wait(&sm.pfull[i], (k / kPieces) & 1, p)) break;
        const Piece pc = sm.piece[i];
        if (pc.t0 < 0) break;
        const int token = pc.tok0 + tok_r;
        const bool valid = tok_r < TM && token < pc.n;
        const bool busy = __any_sync(0xffffffffu, valid);
        const int pos = valid ? pc.L - pc.n + token : 0x3fffffff;
        const Edge<kN> at_edge(p, pc, U);
        float m = -INFINITY, l = 0.f, f = 1.f;  // maximum (raw score units), sum, the last rise's factor
        uint64_t o[D / 2];
#pragma unroll
        for (int e = 0; e < D / 2; ++e) o[e] = 0;
        bool ok = true;
        // the last tile's outputs are added to the row's
        auto add_tile = [&]() {
            const uint32_t at = tmem + kColO + 128 * ((no - 1) & 1);
            const uint64_t f2 = pair64(f, f);
            tc_fence_after();
#pragma unroll
            for (int a = 0; a < D / 32; ++a) {
                uint32_t x[32];
                tmem_ld_32x32b_x32(at + 32 * a, x);
                tmem_ld_wait(x);
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    o[16 * a + e] = fma2(o[16 * a + e], f2,
                                         pair64(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])));
            }
            tc_fence_before();
        };
#pragma unroll 1
        for (int t = pc.t0; t < pc.t1; ++t) {
            if (!(ok = wait(&sm.sfull[ns & 1], (ns >> 1) & 1, p))) break;
            const uint32_t s_at = tmem + kColS + kN * (ns & 1);
            const int tile = tile_of(pc, t);
            const bool edge = at_edge(tile);
            // the keys seen, a bit each: up to the row's own, in its window or a sink
            uint32_t seen_lo = 0, seen_hi = 0;
            if (edge) {
                const int hi = pos - tile * kN, lo = p.window > 0 && valid ? hi - p.window + 1 : 0;
                const uint64_t seen = first_bits(hi + 1) & (~first_bits(lo) | first_bits(p.n_sink - tile * kN));
                seen_lo = static_cast<uint32_t>(seen);
                seen_hi = static_cast<uint32_t>(seen >> 32);
            }
            // scores 32a .. 32a + 31 of the row, with the sign of the scale, -inf where they are masked
            auto scores = [&](int a, uint32_t (&x)[32]) {
                tmem_ld_32x32b_x32(s_at + 32 * a, x);
                tmem_ld_wait(x);
                if (negative) {
                    uint32_t sign = 0x80000000u;
                    asm volatile("" : "+r"(sign));  // (kept behind the branch)
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] ^= sign;
                }
                if (edge) {
                    uint32_t word = a ? seen_hi : seen_lo;
                    asm volatile("" : "+r"(word));
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (!(word >> e & 1)) x[e] = 0xff800000u;
                }
            };
            float rise = 1.f;
            if (busy) {
                tc_fence_after();
                float top = m;
#pragma unroll 1
                for (int a = 0; a < kN / 32; ++a) {
                    uint32_t x[32];
                    scores(a, x);
                    float other = -INFINITY;
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        top = max3(top, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
                        other = max3(other, __uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]));
                    }
                    top = fmaxf(top, other);
                }
                if (top > m) {
                    rise = fast_exp2((m - top) * c);  // (m = -inf: 0)
                    m = top;
                    l *= rise;
                }
            }
            // (the weights before are read, and their outputs there: P is free)
            if (t > pc.t0) {
                if (!(ok = wait(&sm.ofull, no & 1, p))) break;
                ++no;
            }
            if (busy) {
                const float mc = m == -INFINITY ? 0.f : -m * c;
                const uint64_t c2 = pair64(c, c), mc2 = pair64(mc, mc);
                uint64_t sum = 0;
                tc_fence_after();
#pragma unroll 1
                for (int a = 0; a < kN / 32; ++a) {
                    uint32_t x[32], y[3][16];
                    scores(a, x);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float w0, w1;
                        unpair64(fma2(pair64(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), c2, mc2),
                                 w0, w1);
                        w0 = fast_exp2(w0);
                        w1 = fast_exp2(w1);
                        sum = add2(sum, pair64(w0, w1));
                        split2(w0, w1, y[0][e], y[1][e], y[2][e]);
                    }
#pragma unroll
                    for (int b = 0; b < 3; ++b) tmem_st_x16(tmem + kColP + b * (kN / 2) + 16 * a, y[b]);
                }
                float s0, s1;
                unpair64(sum, s0, s1);
                l += s0 + s1;
                tmem_st_wait();
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.pready[ns & 1]);
            ++ns;
            // (the next tile's outputs go to the other place)
            if (busy && t > pc.t0) add_tile();
            f = rise;
        }
        if (ok && pc.t1 > pc.t0) {
            ok = wait(&sm.ofull, no & 1, p);
            ++no;
            if (ok && busy) add_tile();
        }
        if (!ok) break;
        // ---- the piece's end
        const int head = pc.h * p.G + head_r;
        const long long row = static_cast<long long>(pc.c0 + token) * p.Hq + head;
        const float top = m == -INFINITY ? -INFINITY : m * c;  // log2 units
        if (valid) {
            float scale = 1.f;
            float* dst;
            if (pc.slot < 0) {
                float ref = top, sum = l;
                if (p.sink_logit) {
                    const float sink = p.sink_logit[head] * kLog2e;
                    ref = fmaxf(top, sink);
                    scale = top == -INFINITY ? 1.f : fast_exp2(top - ref);
                    sum = sum * scale + (sink == -INFINITY ? 0.f : fast_exp2(sink - ref));
                }
                scale = sum == 0.f ? 0.f : scale / sum;
                if (p.lse_out)
                    p.lse_out[row] = sum == 0.f ? -INFINITY
                                                : ((ref == -INFINITY ? 0.f : ref) + log2f(sum)) * kLn2;
                dst = static_cast<float*>(p.out) + row * D;
            } else {
                const size_t at = static_cast<size_t>(pc.slot) * 2 * kM + r;
                reinterpret_cast<float2*>(p.part_ml)[at] = make_float2(top, l);
                dst = p.part_o + at * D;
            }
#pragma unroll
            for (int e = 0; e < D / 4; ++e) {
                float4 y;
                unpair64(o[2 * e], y.x, y.y);
                unpair64(o[2 * e + 1], y.z, y.w);
                reinterpret_cast<float4*>(dst)[e] = make_float4(y.x * scale, y.y * scale, y.z * scale, y.w * scale);
            }
        }
        const uint32_t marks = *reinterpret_cast<volatile uint32_t*>(&sm.bad[i]);
        if (marks && busy) put_back_rows<D>(p, sm.piece[i], marks, r);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.pempty[i]);
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) prefill_f32_kernel(const PrefillParams p) {
    extern __shared__ __align__(1024) uint8_t raw[];
    Smem<D>& sm = *reinterpret_cast<Smem<D>*>(raw);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (smem_u32(raw) & 1023u) {  // the layout needs a 1024-byte aligned window
        griddep_wait();
        if (threadIdx.x == 0) {
            record_error(p.err, KVD_ERR_CUDA);
            p.head[blockIdx.x].nt = 0;
        }
        return;
    }
    if (threadIdx.x == 0) {
        mbar_init(&sm.qfull, kConvWarps);
        mbar_init(&sm.kfull, kConvWarps);
        mbar_init(&sm.vfull, kConvWarps);
        mbar_init(&sm.qempty, 1);
        mbar_init(&sm.kempty, 1);
        mbar_init(&sm.vempty, 1);
        mbar_init(&sm.sfull[0], 1);
        mbar_init(&sm.sfull[1], 1);
        mbar_init(&sm.pready[0], kSoftWarps);
        mbar_init(&sm.pready[1], kSoftWarps);
        mbar_init(&sm.ofull, 1);
        mbar_init(&sm.end[0], 1);
        mbar_init(&sm.end[1], 1);
        mbar_init(&sm.never, 1);
        for (int i = 0; i < kPieces; ++i) {
            mbar_init(&sm.pfull[i], 1);
            mbar_init(&sm.pempty[i], 2 + kSoftWarps + kConvWarps);
        }
        fence_mbar_init();
    }
    if (warp == kWarpQk) tmem_alloc(&sm.tmem_base, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_wait();
    if (warp < kSoftWarps) {
        regs_more<kRegsSoft>();
        softmax_role<D>(p, sm, warp, lane);
    } else if (warp < kWarpWalk) {
        regs_fewer<kRegsConv>();
        convert_role<D>(p, sm, threadIdx.x - kWarpConv * 32, lane);
    } else {
        regs_fewer<kRegsOther>();
        if (warp == kWarpWalk) {
            int ps = 0;
            auto publish = [&](const Piece& u) {
                const int i = ps % kPieces;
                bool ok = true;
                if (lane == 0) {
                    ok = wait(&sm.pempty[i], ((ps / kPieces) & 1) ^ 1, p);
                    if (ok) {
                        sm.piece[i] = u;
                        sm.bad[i] = 0;
                        mbar_arrive(&sm.pfull[i]);
                    }
                }
                ++ps;
                return __shfl_sync(0xffffffffu, ok, 0) != 0;
            };
            bool ok = !stalls(p, &sm.never, 1);
            const int TM = kM / p.G;
            walk<kN>(p, TM, TM, lane, [&](const Piece& u) { return ok = ok && publish(u); });
            if (ok) {
                Piece last;
                last.t0 = -1;
                last.t1 = 0;
                publish(last);
            }
        } else if (warp == kWarpQk) {
            qk_role<D>(p, sm, lane);
        } else if (warp == kWarpPv) {
            pv_role<D>(p, sm, lane);
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWarpQk) tmem_dealloc(sm.tmem_base, 512);
}

template <int D>
int launch(PrefillParams p, void* ws, cudaStream_t stream) {
    auto kernel = prefill_f32_kernel<D>;
    constexpr int smem = static_cast<int>(sizeof(Smem<D>));
    static_assert(smem <= 227 * 1024, "prefill shared memory");
    static const cudaError_t set =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (set != cudaSuccess) return KVD_ERR_CUDA;
    set_plan(p, D, ws, 64, 4 * kN);
    if (launch_kernel(kernel, dim3(static_cast<unsigned>(p.n_cta)), dim3(kThreads), smem, stream, p) !=
            cudaSuccess ||
        launch_merge<D, float, kN>(p, kM / p.G, stream) != cudaSuccess)
        return KVD_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? KVD_OK : KVD_ERR_CUDA;
}

}  // namespace

int prefill_f32_launch(const PrefillParams& p, int D, void* ws, cudaStream_t stream) {
    return D == 64 ? launch<64>(p, ws, stream) : launch<128>(p, ws, stream);
}

}  // namespace kvd
