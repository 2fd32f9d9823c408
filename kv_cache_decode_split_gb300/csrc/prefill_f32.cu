// prefill_f32.cu -- causal attention of many new tokens of each sequence, float32, over packed keys and
// values or over a paged cache (the formulas are in prefill_bf16.cu).
//
// Products. A float32 number is the sum of three bfloat16 numbers (3 x 8 bits of significand, the same
// exponents), x = x1 + x2 + x3, each the rounding of what the ones before it leave. Of the nine products
// of two such sums the six of at least 2^-16 are kept, x1 y1 + x1 y2 + x2 y1 + x2 y2 + x1 y3 + x3 y1; the
// three left out are below 2^-24 of |x||y| each. (Three products of two tf32 numbers cost as much time
// at half the rate, and a third more shared memory. CUDA cores took 78 ms for 16385 tokens of 32 heads of
// 128 in bfloat16, and 3.9 ms for the ragged float32 chunks that take less than 0.2 here.)
// The smallest products are added first. A tensor core cuts what it adds, so the weighted sums of one
// 64-key tile at most are left to it: every tile's outputs start from zero and are added to float32
// registers, rounded.
//
// One persistent CTA an SM takes units of one query tile (128 rows: the G query heads of a KV head of
// 128 / G tokens) from the list of prefill_common.cuh. Roles:
//   * eight warps read queries, keys and values, split them and write the parts to shared memory in the
//     tensor core's layout; values that are not finite are cleared (their split is NaN), and the rows
//     that see them get them back at the end;
//   * one thread issues S = Q K^T (6 x D / 16 steps) and O = P V (6 x 4 steps): the scores of the next
//     tile are under way while this tile's softmax runs;
//   * four warps, a row a thread: running maximum and sum, weights split into three parts for tensor
//     memory, outputs in registers.

#include <algorithm>

#include "prefill_common.cuh"

namespace kvd {

namespace {

using namespace prefill;

constexpr int kN = 64;       // keys of a tile
constexpr int kThreads = 512;
constexpr int kSoftWarps = 4, kConvWarps = 8;
constexpr int kWarpConv = 4, kWarpWalk = 12, kWarpMma = 13;
// registers of a thread of the softmax's, the two converting and the last warpgroup, of 128 at launch
constexpr int kRegsSoft = 232, kRegsConv = 104, kRegsOther = 72;
static_assert(kRegsSoft + 2 * kRegsConv + kRegsOther <= 4 * 128, "registers");
constexpr uint32_t kColS = 0, kColP = 128, kColO = 256;  // two score tiles; 3 x 32; D

template <int D>
struct Smem {
    uint8_t q[3][kM * D * 2];  // offset 0; every part is a multiple of 1024 bytes
    uint8_t k[3][kN * D * 2];
    uint8_t v[3][kN * D * 2];
    uint64_t qfull, qempty, kfull, kempty, vfull, vempty, sfull[2], pready, ofull;
    uint64_t pfull[kPieces], pempty[kPieces], end;
    Piece piece[kPieces];
    int bad[kPieces];  // a value was not finite
    uint32_t tmem_base;
};

__device__ __forceinline__ void tmem_st_x8(uint32_t t, const uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t), "r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
        : "memory");
}

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
__device__ constexpr int kLeft[6] = {2, 0, 1, 1, 0, 0}, kRight[6] = {0, 2, 1, 0, 1, 0};

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

__device__ __forceinline__ bool finite4(const float4& v) {
    return isfinite(v.x) && isfinite(v.y) && isfinite(v.z) && isfinite(v.w);
}
__device__ __forceinline__ void clear4(float4& v) {
    v.x = isfinite(v.x) ? v.x : 0.f;
    v.y = isfinite(v.y) ? v.y : 0.f;
    v.z = isfinite(v.z) ? v.z : 0.f;
    v.w = isfinite(v.w) ? v.w : 0.f;
}

template <int D>
__device__ void convert_role(const PrefillParams& p, Smem<D>& sm, int tid, int lane) {
    constexpr int kRow = D / 8;                    // chunks of a row
    constexpr int kEach = kN * kRow / 256;         // chunks of a key or value tile that a thread takes
    const int TM = kM / p.G;
    int* err = p.err;
    const int c8 = tid % kRow, r0 = tid / kRow;    // row r0 + i * (256 / kRow)
    constexpr int kStep = 256 / kRow;
    uint32_t nq = 0, nk = 0, nv = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
        const int slot = k % kPieces;
        if (!wait(&sm.pfull[slot], (k / kPieces) & 1, err)) break;
        const Piece pc = sm.piece[slot];
        if (pc.t0 < 0) break;
        const int nt = pc.t1 - pc.t0;
        auto done = [&](uint64_t* bar) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        auto item = [&](int t, bool is_v) {
            const float* src = static_cast<const float*>(is_v ? p.v : p.k);
            const long long stride = is_v ? p.v_stride : p.k_stride;
            const int t0 = tile_of(pc, pc.t0 + t) * kN;
            float4 x[kEach][2];
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                const int key = t0 + r0 + i * kStep;
                x[i][0] = x[i][1] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (key < pc.L) {
                    const float* at;
                    if (p.block_table) {
                        const int pg = load_page(p.block_table, p.max_pages, p.num_pages, pc.k0,
                                                 key >> p.page_shift, err);
                        at = src + (((static_cast<size_t>(pg) * p.Hkv + pc.h) << p.page_shift) +
                                    (key & ((1 << p.page_shift) - 1))) * D;
                    } else {
                        at = src + (pc.k0 + key) * stride + pc.h * D;
                    }
                    x[i][0] = reinterpret_cast<const float4*>(at)[2 * c8];
                    x[i][1] = reinterpret_cast<const float4*>(at)[2 * c8 + 1];
                }
            }
            uint32_t& n = is_v ? nv : nk;
            if (!(ok = wait(is_v ? &sm.vempty : &sm.kempty, (n & 1) ^ 1, err))) return;
            ++n;
#pragma unroll
            for (int i = 0; i < kEach; ++i) {
                if (is_v && !(finite4(x[i][0]) && finite4(x[i][1]))) {
                    clear4(x[i][0]);
                    clear4(x[i][1]);
                    sm.bad[slot] = 1;
                }
                put_split(is_v ? sm.v[0] : sm.k[0], kN * D * 2, kN, r0 + i * kStep, c8, x[i][0], x[i][1]);
            }
            done(is_v ? &sm.vfull : &sm.kfull);
        };
        if (nt > 0) {
            if (!(ok = wait(&sm.qempty, (nq & 1) ^ 1, err))) break;
            ++nq;
            for (int r = r0; r < kM; r += kStep) {
                const int t = r / p.G, token = pc.tok0 + t;
                float4 lo = make_float4(0.f, 0.f, 0.f, 0.f), hi = lo;
                if (t < TM && token < pc.n) {
                    const float4* at = reinterpret_cast<const float4*>(
                        static_cast<const float*>(p.q) + (pc.c0 + token) * p.q_stride +
                        (pc.h * p.G + (r - t * p.G)) * static_cast<long long>(D));
                    lo = at[2 * c8];
                    hi = at[2 * c8 + 1];
                }
                put_split(sm.q[0], kM * D * 2, kM, r, c8, lo, hi);
            }
            done(&sm.qfull);
            item(0, false);
            for (int t = 0; t < nt && ok; ++t) {
                if (t + 1 < nt) item(t + 1, false);
                if (ok) item(t, true);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.pempty[slot]);
    }
}

// ---------------------------------------------------------------------------------- products
template <int D>
__device__ void mma_role(const PrefillParams& p, Smem<D>& sm) {
    constexpr uint32_t id_qk = idesc_bf16_f32(kM, kN, 0, 0), id_pv = idesc_bf16_f32(kM, D, 0, 1);
    const uint32_t tmem = sm.tmem_base;
    const uint64_t q = sw128_kmajor_desc(smem_u32(sm.q[0])), kk = sw128_kmajor_desc(smem_u32(sm.k[0]));
    const uint64_t v = sw128_mnmajor_desc(smem_u32(sm.v[0]), kN * 128);
    int* err = p.err;
    uint32_t nq = 0, nk = 0, np = 0;  // query tiles, key tiles, value tiles taken
    bool ok = true;
    auto qk = [&](bool last) {
        if (!wait(&sm.kfull, nk & 1, err)) return false;
        tc_fence_after();
        const uint32_t s = tmem + kColS + kN * (nk & 1);
#pragma unroll
        for (int i = 0; i < 6; ++i)
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
                tc_mma_bf16(s, q + ((kLeft[i] * kM * D * 2 + (ks >> 2) * kM * 128 + (ks & 3) * 32) >> 4),
                            kk + ((kRight[i] * kN * D * 2 + (ks >> 2) * kN * 128 + (ks & 3) * 32) >> 4),
                            id_qk, i + ks > 0 ? 1u : 0u);
        tc_commit(&sm.sfull[nk & 1]);
        tc_commit(&sm.kempty);
        if (last) tc_commit(&sm.qempty);
        ++nk;
        return true;
    };
    for (int k = 0; ok; ++k) {
        const int i = k % kPieces;
        if (!wait(&sm.pfull[i], (k / kPieces) & 1, err)) break;
        const int t0 = sm.piece[i].t0, nt = sm.piece[i].t1 - t0;
        mbar_arrive(&sm.pempty[i]);
        if (t0 < 0) break;
        if (nt == 0) continue;
        if (!(ok = wait(&sm.qfull, nq++ & 1, err) && qk(nt == 1))) break;
        for (int t = 0; t < nt; ++t) {
            if (t + 1 < nt && !(ok = qk(t + 2 == nt))) break;
            if (!(ok = wait(&sm.vfull, np & 1, err) && wait(&sm.pready, np & 1, err))) break;
            ++np;
            tc_fence_after();
#pragma unroll
            for (int j = 0; j < 6; ++j)
#pragma unroll
                for (int ks = 0; ks < kN / 16; ++ks)
                    tc_mma_bf16_ts(tmem + kColO, tmem + kColP + kLeft[j] * (kN / 2) + ks * 8,
                                   v + ((kRight[j] * kN * D * 2 + ks * 16 * 128) >> 4), id_pv,
                                   j + ks > 0 ? 1u : 0u);
            tc_commit(&sm.ofull);
            tc_commit(&sm.vempty);
        }
    }
    tc_commit(&sm.end);  // all products complete before tensor memory is released
    wait(&sm.end, 0, err);
}

// ----------------------------------------------------------------------------------- softmax
// What a row gets back, in one column, of the values that were cleared: v itself, where the row sees it.
template <int D>
__device__ __noinline__ float cleared(const PrefillParams& p, const Piece& pc, int pos, int col) {
    float sum = 0.f;
    for (int t = pc.t0; t < pc.t1; ++t) {
        const int t0 = tile_of(pc, t) * kN;
        for (int key = t0; key < min(t0 + kN, min(pc.L, pos + 1)); ++key) {
            if (p.window > 0 && key <= pos - p.window && key >= p.n_sink) continue;
            const float* v = static_cast<const float*>(p.v);
            if (p.block_table) {
                const int pg = load_page(p.block_table, p.max_pages, p.num_pages, pc.k0,
                                         key >> p.page_shift, nullptr);
                v += (((static_cast<size_t>(pg) * p.Hkv + pc.h) << p.page_shift) +
                      (key & ((1 << p.page_shift) - 1))) * D;
            } else {
                v += (pc.k0 + key) * p.v_stride + pc.h * D;
            }
            if (!isfinite(v[col])) sum += v[col];
        }
    }
    return sum;
}

template <int D>
__device__ void softmax_role(const PrefillParams& p, Smem<D>& sm, int warp, int lane) {
    const int r = warp * 32 + lane;  // row of the tile, lane of tensor memory
    const int TM = kM / p.G, U = TM;
    const uint32_t quad = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t tmem = sm.tmem_base + quad;
    int* err = p.err;
    const bool negative = p.scale_log2 < 0.f;
    const float c = fmaxf(fabsf(p.scale_log2), 0x1p-100f);  // (0: -inf times it stays -inf)
    const int tok_r = r / p.G, head_r = r - tok_r * p.G;
    uint32_t ns = 0, no = 0;  // score tiles and output tiles taken
    for (int k = 0;; ++k) {
        const int i = k % kPieces;
        if (!wait(&sm.pfull[i], (k / kPieces) & 1, err)) break;
        const Piece pc = sm.piece[i];
        if (pc.t0 < 0) break;
        const int token = pc.tok0 + tok_r;
        const bool valid = tok_r < TM && token < pc.n;
        const bool busy = __any_sync(0xffffffffu, valid);
        const int pos = valid ? pc.L - pc.n + token : 0x3fffffff;
        const Edge<kN> at_edge(p, pc, U);
        float m = -INFINITY, l = 0.f;  // maximum (raw score units), sum
        float o[D];
#pragma unroll
        for (int e = 0; e < D; ++e) o[e] = 0.f;
        bool ok = true;
        // the tile's outputs are added to the row's
        auto add_tile = [&](float f) {
            if (!wait(&sm.ofull, no & 1, err)) return false;
            ++no;
            if (!busy) return true;
            tc_fence_after();
            const bool same = __all_sync(0xffffffffu, f == 1.f);
#pragma unroll
            for (int a = 0; a < D / 16; ++a) {
                uint32_t x[16];
                tmem_ld_x16(tmem + kColO + 16 * a, x);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[16 * a + e] += __uint_as_float(x[e]);
            }
            if (!same) {
#pragma unroll
                for (int e = 0; e < D; ++e) o[e] *= f;
            }
            return true;
        };
        for (int t = pc.t0; t < pc.t1; ++t) {
            if (!(ok = wait(&sm.sfull[ns & 1], (ns >> 1) & 1, err))) break;
            float f = 1.f, s[kN];
            if (busy) {
                tc_fence_after();
                {
                    uint32_t x[32];
#pragma unroll
                    for (int a = 0; a < 2; ++a) {
                        tmem_ld_32x32b_x32(tmem + kColS + kN * (ns & 1) + 32 * a, x);
                        tmem_ld_wait(x);
#pragma unroll
                        for (int e = 0; e < 32; ++e) s[32 * a + e] = __uint_as_float(x[e]);
                    }
                }
                if (negative) {
#pragma unroll
                    for (int e = 0; e < kN; ++e) s[e] = -s[e];
                }
                const int tile = tile_of(pc, t);
                if (at_edge(tile)) {
                    const int hi = pos - tile * kN;  // last key seen
                    const int lo = p.window > 0 && valid ? hi - p.window + 1 : 0;
                    const int sk = p.n_sink - tile * kN;
#pragma unroll
                    for (int e = 0; e < kN; ++e)
                        if (e > hi || (e < lo && e >= sk)) s[e] = -INFINITY;
                }
                float top = fmaxf(m, s[0]);
#pragma unroll
                for (int e = 1; e < kN - 1; e += 2) top = max3(top, s[e], s[e + 1]);
                top = fmaxf(top, s[kN - 1]);
                if (top > m) {
                    f = fast_exp2((m - top) * c);  // (m = -inf: 0)
                    m = top;
                    l *= f;
                }
                const float mc = m == -INFINITY ? 0.f : m * c;
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int e = 0; e < kN; ++e) {
                    s[e] = fast_exp2(fmaf(s[e], c, -mc));
                    sum[e % 4] += s[e];
                }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            }
            ++ns;
            if (t > pc.t0 && !(ok = add_tile(f))) break;  // (the weights before are read: P is free)
            if (busy) {
#pragma unroll
                for (int a = 0; a < kN / 16; ++a) {
                    uint32_t x[3][8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        split2(s[16 * a + 2 * e], s[16 * a + 2 * e + 1], x[0][e], x[1][e], x[2][e]);
#pragma unroll
                    for (int b = 0; b < 3; ++b) tmem_st_x8(tmem + kColP + b * (kN / 2) + 8 * a, x[b]);
                }
                tmem_st_wait();
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.pready);
        }
        if (!ok || (pc.t1 > pc.t0 && !add_tile(1.f))) break;
        tc_fence_before();
        // ---- the piece's end
        const int bad = *reinterpret_cast<volatile int*>(&sm.bad[i]);
        if (bad) {
            const int seen = valid ? pos : -1;
#pragma unroll
            for (int e = 0; e < D; ++e) o[e] += cleared<D>(p, pc, seen, e);
        }
        const int head = pc.h * p.G + head_r;
        const long long row = static_cast<long long>(pc.c0 + token) * p.Hq + head;
        const float top = m == -INFINITY ? -INFINITY : m * c;  // log2 units
        if (valid && pc.slot < 0) {
            float ref = top, sum = l, scale = 1.f;
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
            float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + row * D);
#pragma unroll
            for (int e = 0; e < D / 4; ++e)
                dst[e] = make_float4(o[4 * e] * scale, o[4 * e + 1] * scale, o[4 * e + 2] * scale,
                                     o[4 * e + 3] * scale);
        } else if (valid) {
            const size_t at = static_cast<size_t>(pc.slot) * 2 * kM + r;
            reinterpret_cast<float2*>(p.part_ml)[at] = make_float2(top, l);
            float4* dst = reinterpret_cast<float4*>(p.part_o + at * D);
#pragma unroll
            for (int e = 0; e < D / 4; ++e)
                dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
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
        mbar_init(&sm.pready, kSoftWarps);
        mbar_init(&sm.ofull, 1);
        mbar_init(&sm.end, 1);
        for (int i = 0; i < kPieces; ++i) {
            mbar_init(&sm.pfull[i], 1);
            mbar_init(&sm.pempty[i], 1 + kSoftWarps + kConvWarps);
        }
        fence_mbar_init();
    }
    if (warp == kWarpMma) tmem_alloc(&sm.tmem_base, 512);
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
                    ok = wait(&sm.pempty[i], ((ps / kPieces) & 1) ^ 1, p.err);
                    if (ok) {
                        sm.piece[i] = u;
                        sm.bad[i] = 0;
                        mbar_arrive(&sm.pfull[i]);
                    }
                }
                ++ps;
                return __shfl_sync(0xffffffffu, ok, 0) != 0;
            };
            bool ok = true;
            const int TM = kM / p.G;
            walk<kN>(p, TM, TM, lane, [&](const Piece& u) { return ok = publish(u); });
            if (ok) {
                Piece last;
                last.t0 = -1;
                last.t1 = 0;
                publish(last);
            }
        } else if (warp == kWarpMma && lane == 0) {
            mma_role<D>(p, sm);
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWarpMma) tmem_dealloc(sm.tmem_base, 512);
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
