// prefill_bf16.cu -- causal attention of many new tokens of each sequence, bfloat16, over packed keys
// and values or over a paged cache.
//
// What is computed: the i-th of a sequence's n new tokens, of L keys in all, has position
// p = L - n + i and sees the keys t <= p (window > 0: of them t > p - window or t < n_sink):
//   s_t = scale q.k_t,  out = sum_t exp(s_t - lse) v_t,  lse = log(sum_t exp(s_t) [+ exp(sink)]).
//
// Rows. A KV head's G query heads read the same keys, so the G heads of 128 / G tokens make the 128
// rows of one tensor-core tile (row = token * G + head), and a unit of work is two such tiles of one
// sequence and KV head: every key and value tile is read once for 256 rows.
//
// One persistent CTA an SM, roles by warp:
//   * loads: query tiles and rings of 128-token key and value tiles, all by TMA;
//   * products: S = Q K^T (tcgen05, 128 x 64, operands in shared memory) and O += P V (P in tensor memory,
//     where it takes the place of its S), each of the two streams' by a warp of its own;
//   * softmax: two warpgroups, one row a thread, each with two score buffers of 64 keys and an output
//     accumulator of its own in tensor memory, so that one's exponentials run under the other's products.
//     The row's reference maximum is only raised, and O rescaled, when a maximum grows by more than 2^8;
//     weights are taken against 2^8 times it, so that they are at most 1 and a large value's product stays a
//     number (against the maximum itself a weight of 2^7.5 made 2.5e36 infinite). They are rounded to bfloat16
//     (the value product's operands have one type), their sums are float32 sums of the unrounded weights.
//   * values: at the edges of the mask three warps clear the value rows behind the sequence's end and
//     every value that is not finite, before a zero weight can meet them; the rows that see such a
//     value get it back at the end.
//   * a unit's end: a warpgroup divides and writes the outputs while the softmax goes on with the next unit.
// A unit of at most 128 rows (draft tokens, a prompt's end) is one query tile: the two streams then
// take its key tiles in turn, and their accumulators are merged.
//
// Work is cut as a list: all units one behind the other, each as long as the keys that it walks and a
// fixed part for its start and end, in equal ranges, one for each CTA. A unit that a cut divides is
// left as partial results of its pieces, which a second launch merges by log-sum-exp (in the order of
// the pieces: the result does not depend on timing).
//
// Bound, in long units, by the softmax's chain (some 1400 cycles for 64 keys, two such warps a scheduler, issue
// slots busy 48 %) next to the products, whose pipe is busy 75 %: a 128 x 128 tile is 512 cycles of
// QK (768 in the halves of 64 keys that let the exponentials start early; it is shared memory's rate then),
// 512 of PV and 512 of exponentials, two tiles at a time. 16385 tokens of 32/8 heads of 128 take 1.60 ms,
// 1.38 PFLOP/s (72 % of what a library matrix product reaches); 2048-token chunks behind 28 thousand 1.34 to
// 1.50. Short units are bound by their ends: the next unit's queries take the last one's place, so that 1500
// to 3000 cycles pass without products, and code that a unit runs once is not in the instruction caches
// (nine prompts of 61 to 3581 tokens: 390 us, 0.87 PFLOP/s). Loading the next unit's first keys ahead of its
// queries did not help (5 % slower). A call of one short unit an SM (513 tokens: 18.8 us) is a chain: 5 us to
// the first load (lengths, then the CTA's range), 3 to the first scores, 2 a tile, 3 for the end.
// Draft tokens (32 sequences, 1 to 8 tokens behind 4096 to 8184) read the cache at 5.6 TB/s: 143 us.

#include <algorithm>

#include "prefill_common.cuh"

namespace kvd {

namespace {

using namespace prefill;

constexpr int kN = 128;     // keys of a tile, as it is loaded
constexpr int kSub = 64;    // keys of a score buffer
// Tiles that tensor memory adds up. A tensor core cuts what it adds, so that a sum over many keys shrinks: by
// 1e-4 over 2048 tiles, 0.2 to 1.2 % over 32768 (4 million keys), where an output's own rounding is 0.2 %. Longer
// pieces go in parts, which are added up in float32 arithmetic in the workspace: for loads and scores they are
// one piece, but its statistics and outputs are handed over kMost tiles at a time.
constexpr int kMost = 512;
constexpr int kSoftWarps = 8;
constexpr int kWarpLoad = 8, kWarpQk = 9, kWarpPv = 11, kWarpFix = 13,
              kWarpEnd = 16;  // products: + stream
constexpr int kFixWarps = 3;
constexpr int kThreads = 640;
// registers of a thread of the softmax's two and the other three warpgroups, of 96 at launch
constexpr int kRegsSoft = 120, kRegsOther = 80;
static_assert(2 * kRegsSoft + 3 * kRegsOther <= 5 * 96, "registers");
constexpr float kGrowth = 8.0f;  // log2 units
constexpr uint32_t kColS = 0, kColO = 256;  // + 128 * stream

template <int D>
struct Layout {
    static constexpr int kTile = kN * D * 2;   // bytes of a key, value or query tile
    static constexpr int kK = D == 128 ? 2 : 4, kV = D == 128 ? 3 : 4;  // rings of key and value tiles
};

template <int D>
struct Smem {
    uint8_t q[2][Layout<D>::kTile];                   // offset 0, 1024-aligned
    uint8_t k[Layout<D>::kK][Layout<D>::kTile];
    uint8_t v[Layout<D>::kV][Layout<D>::kTile];
    float stat[2][kM][2];                             // each stream's rows' (maximum, sum)
    uint64_t kfull[Layout<D>::kK], kempty[Layout<D>::kK], vfull[Layout<D>::kV], vempty[Layout<D>::kV];
    // values at a mask's edge: under way (a look at `vfull` alone could take an earlier round of the ring
    // for this one), and looked through
    uint64_t issued[Layout<D>::kV], fixed[Layout<D>::kV];
    uint64_t qfull, qempty, sfull[2][2], pready[2][2], pvdone[2][2], ofull[2], ofree[2], pfull[kPieces], pempty[kPieces];
    uint64_t statw[2], statr[2];                      // a stream's stat written, read
    uint64_t end[4], never;
    Piece piece[kPieces];
    uint32_t bad[kPieces];                            // tiles at a mask's edge with values that are not finite
    uint32_t tmem_base;
};

// The halves (of 64 keys) of a tile that some row of a stream sees: bits 0 and 1.
struct Need {
    int first, last, window, n_sink;  // positions of the stream's first and last row
    __device__ __forceinline__ Need(const PrefillParams& p, const Piece& u, int w, int TM)
        : window(p.window), n_sink(p.n_sink) {
        const int tok = u.tok0 + (u.pair ? w * TM : 0);
        first = u.L - u.n + tok;
        last = u.L - u.n + min(u.n, tok + TM) - 1;
    }
    __device__ __forceinline__ int operator()(int tile) const {
        int bits = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int a = tile * kN + h * kSub;
            const bool before = window > 0 && a + kSub - 1 <= first - window && a >= n_sink;
            if (a <= last && !before) bits |= 1 << h;
        }
        return bits;
    }
};
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int x,
                                            int y, int z, int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

// S (tensor memory) = Q (128 rows) K^T (64 keys), both K-major in shared memory.
template <int D>
__device__ __forceinline__ void issue_qk(uint32_t s, uint32_t q, uint32_t k) {
    constexpr uint32_t idesc = idesc_bf16_f32(kM, kSub, 0, 0);
    const uint64_t a = sw128_kmajor_desc(q), b = sw128_kmajor_desc(k);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
        const uint64_t step = static_cast<uint64_t>(((ks >> 2) * kN * 128 + (ks & 3) * 32) >> 4);
        tc_mma_bf16(s, a + step, b + step, idesc, ks > 0 ? 1u : 0u);
    }
}

// O (tensor memory) (+)= P (tensor memory, 128 x 64) V (64 tokens, read MN-major).
template <int D>
__device__ __forceinline__ void issue_pv(uint32_t o, uint32_t pt, uint32_t v, bool accumulate) {
    constexpr uint32_t idesc = idesc_bf16_f32(kM, D, 0, 1);
    const uint64_t b = sw128_mnmajor_desc(v, kN * 128);
#pragma unroll
    for (int ks = 0; ks < kSub / 16; ++ks)
        tc_mma_bf16_ts(o, pt + ks * 8, b + static_cast<uint64_t>((ks * 16 * 128) >> 4), idesc,
                       (accumulate || ks > 0) ? 1u : 0u);
}

// ------------------------------------------------------------------------------------- loads
template <int D>
__device__ void load_role(const PrefillParams& p, Smem<D>& sm, const CUtensorMap* tq,
                          const CUtensorMap* tk, const CUtensorMap* tv, int lane) {
    using Ly = Layout<D>;
    const int TM = kM / p.G, U = 2 * TM;
    int* err = p.err;
    int ps = 0;               // pieces published
    uint32_t gk = 0, gv = 0, nq = 0;  // key tiles, value tiles and query loads issued
    bool ok = !stalls(p, &sm.never, 1);
    auto publish = [&](const Piece& u) {
        const int i = ps % kPieces;
        if (lane == 0) {
            ok = wait(&sm.pempty[i], ((ps / kPieces) & 1) ^ 1, p);
            if (ok) {
                sm.piece[i] = u;
                sm.bad[i] = 0;
                mbar_arrive(&sm.pfull[i]);
            }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        ++ps;
    };

    walk<kN>(p, U, TM, lane, [&](const Piece& pc) {
        if (ok) publish(pc);
        if (!ok) return false;
        const int nt = pc.t1 - pc.t0, la = pc.pair ? 1 : 2;
        if (nt == 0) return true;
        const Edge<kN> edge(p, pc, U);
        // queries
        if (lane == 0) {
            ok = wait(&sm.qempty, (nq & 1) ^ 1, p);
            if (ok) {
                const int rows = TM * p.G;
                mbar_arrive_expect_tx(&sm.qfull, (pc.pair ? 2 : 1) * rows * D * 2);
                for (int i = 0; i <= pc.pair; ++i)
                    for (int k = 0; k < D / 64; ++k)
                        tma_load_4d(sm.q[i] + k * kM * 128, tq, &sm.qfull, 0, pc.h * p.G,
                                    pc.c0 + pc.tok0 + i * TM, k);
            }
        }
        ++nq;
        ok = __shfl_sync(0xffffffffu, ok, 0);
        // keys and values. Item i of the piece: key tiles 0 .. la - 1, then value tile t and key tile
        // t + la in turn. Paged: a tile is `per` copies of a page's rows; lane e holds the row of copy e of
        // the next 32, of the keys' in kcur and knxt, of the values' in vcur.
        const bool paged = p.block_table != nullptr;
        const int shift = min(p.page_shift, 7), per = paged ? kN >> shift : 1;
        auto row_of = [&](int e) -> int {
            const int t = e / per;
            if (t >= nt) return 0;
            const int tok = tile_of(pc, pc.t0 + t) * kN + ((e % per) << shift);
            int key = min(tok, pc.L - 1);
            // (a page that no row of the unit sees may be gone: any other, all of it is masked)
            if (p.window > 0 && tok >= p.n_sink && tok + (1 << shift) <= pc.L - pc.n + pc.tok0 - p.window + 1)
                key = pc.L - 1;
            const int pg =
                load_page(p.block_table, p.max_pages, p.num_pages, pc.k0, key >> p.page_shift, err);
            return ((pg * p.Hkv + pc.h) << p.page_shift) + (tok & ((1 << p.page_shift) - 1));
        };
        int kb = -32, vb = -32, kcur = 0, knxt = 0, vcur = 0;
        if (paged) knxt = row_of(lane);
#pragma unroll 1
        for (int i = 0; i < 2 * nt && ok; ++i) {
            // of the items behind the first ones the even are values; as many at the end are values too
            const int lead = min(la, nt), at = i - lead;
            const bool tail = i + lead >= 2 * nt, is_v = at >= 0 && (at % 2 == 0 || tail);
            const int t = tail ? i - nt : is_v ? at / 2 : at < 0 ? i : (at - 1) / 2 + la;
            const uint32_t n = is_v ? gv : gk, size = is_v ? Ly::kV : Ly::kK, s_ = n % size;
            uint64_t* full = is_v ? &sm.vfull[s_] : &sm.kfull[s_];
            if (lane == 0) {
                ok = wait(is_v ? &sm.vempty[s_] : &sm.kempty[s_], ((n / size) & 1) ^ 1, p);
                if (ok) {
                    mbar_arrive_expect_tx(full, Ly::kTile);
                    if (is_v && edge(tile_of(pc, pc.t0 + t))) mbar_arrive(&sm.issued[s_]);
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            if (is_v) ++gv; else ++gk;
            const CUtensorMap* map = is_v ? tv : tk;
            int row = pc.k0 + tile_of(pc, pc.t0 + t) * kN, e = lane;
            if (paged) {
                const int e0 = t * per;
                if (e0 >= (is_v ? vb : kb) + 32) {
                    if (is_v) {
                        vb += 32;
                        vcur = vb == kb ? kcur : row_of(vb + lane);
                    } else {
                        kb += 32;
                        kcur = knxt;
                        knxt = row_of(kb + 32 + lane);
                    }
                }
                // copy i of the tile is with lane e0 - base + i, which issues it
                e = lane - (e0 - (is_v ? vb : kb));
                row = is_v ? vcur : kcur;
            }
            if (e >= 0 && e < per) {
                uint8_t* dst = (is_v ? sm.v[s_] : sm.k[s_]) + ((e << shift) * 128);
                tma_load_4d(dst, map, full, 0, row, 0, paged ? 0 : pc.h);
                if (per > 1 && D == 128) tma_load_4d(dst + kN * 128, map, full, 0, row, 1, 0);
            }
            __syncwarp();
        }
        return ok;
    });
    if (ok) {
        Piece last;
        last.t0 = -1;
        publish(last);
    }
    // every copy lands before the CTA ends, also after a wait gave up
    if (lane == 0) {
        for (uint32_t i = gk > Ly::kK ? gk - Ly::kK : 0; i < gk; ++i)
            drain(&sm.kfull[i % Ly::kK], (i / Ly::kK) & 1, p);
        for (uint32_t i = gv > Ly::kV ? gv - Ly::kV : 0; i < gv; ++i)
            drain(&sm.vfull[i % Ly::kV], (i / Ly::kV) & 1, p);
        if (nq > 0) drain(&sm.qfull, (nq - 1) & 1, p);
    }
    __syncwarp();
}

// ---------------------------------------------------------------------------------- products
// Four threads: each stream's score products, and its value products. A wait or a commit holds its thread
// up for some 100 cycles even where it has nothing to wait for, and a product's instructions until the one
// before has begun: with one thread for a stream's products the tensor cores were idle half of the time
// (16385 tokens: 1.80 ms; one thread for both streams: 2.18).
// A stream has two score buffers, one for each half of a tile. The score product into a buffer waits for
// the value product that reads its weights, the other buffer's softmax runs meanwhile. All threads of a
// kind pass every tile of their ring in order, also one that is the other stream's.

// A ring's next slot and the parity of its round.
template <int N>
struct Turn {
    uint32_t slot = 0, round = 0;
    __device__ __forceinline__ void next() {
        if (++slot == N) {
            slot = 0;
            round ^= 1;
        }
    }
};

template <int D>
__device__ void qk_role(const PrefillParams& p, Smem<D>& sm, const int w, const int lane) {
    using Ly = Layout<D>;
    const int TM = kM / p.G, U = 2 * TM;
    const uint32_t tS = sm.tmem_base + kColS + 128 * w, k0 = smem_u32(sm.k[0]);
    const bool one = lane == 0;
    Turn<Ly::kK> at;
    uint32_t nq = 0, used = 0;  // used: a parity bit for each buffer's score tiles
    bool ok = !stalls(p, &sm.never, 2);
    for (int k = 0; ok; ++k) {
        const int i = k % kPieces;
        if (!wait(&sm.pfull[i], (k / kPieces) & 1, p)) break;
        const Piece pc = sm.piece[i];
        __syncwarp();
        if (one) mbar_arrive(&sm.pempty[i]);
        if (pc.t0 < 0) break;
        if (pc.t1 == pc.t0) continue;
        const uint32_t q = smem_u32(sm.q[pc.pair ? w : 0]);
        const Need need(p, pc, w, TM);
        const Edge<kN> edge(p, pc, U);
        if (!(ok = wait(&sm.qfull, nq++ & 1, p))) break;
#pragma unroll 1
        for (int t = pc.t0; t < pc.t1; ++t) {
            const bool own = pc.pair || ((t - pc.t0) & 1) == w;
            const int tile = tile_of(pc, t), m = !own ? 0 : edge(tile) ? need(tile) : 3;
            if (!(ok = wait(&sm.kfull[at.slot], at.round, p))) break;
            const uint32_t kt = k0 + at.slot * Ly::kTile;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (m >> h & 1) {
                    if (!(ok = wait(&sm.pvdone[w][h], (used >> h & 1) ^ 1, p))) break;
                    used ^= 1u << h;
                    tc_fence_after();
                    if (one) {
                        issue_qk<D>(tS + kSub * h, q, kt + h * kSub * 128);
                        tc_commit(&sm.sfull[w][h]);
                    }
                }
            if (!ok) break;
            if (one) {
                if (own)
                    tc_commit(&sm.kempty[at.slot]);
                else
                    mbar_arrive(&sm.kempty[at.slot]);
            }
            at.next();
        }
        if (ok && one) tc_commit(&sm.qempty);
    }
    // all products complete before tensor memory is released
    if (one) tc_commit(&sm.end[w]);
    drain(&sm.end[w], 0, p);
}

template <int D>
__device__ void pv_role(const PrefillParams& p, Smem<D>& sm, const int w, const int lane) {
    using Ly = Layout<D>;
    const int TM = kM / p.G, U = 2 * TM;
    const uint32_t tS = sm.tmem_base + kColS + 128 * w, tO = sm.tmem_base + kColO + 128 * w;
    const uint32_t v0 = smem_u32(sm.v[0]);
    const bool one = lane == 0;
    Turn<Ly::kV> at;
    uint32_t fixed = 0, np = 0;  // a parity bit for each slot's `fixed`, each buffer's weights
    uint32_t parts = 0;
    bool ok = !stalls(p, &sm.never, 3);
    for (int k = 0; ok; ++k) {
        const int i = k % kPieces;
        if (!wait(&sm.pfull[i], (k / kPieces) & 1, p)) break;
        const Piece pc = sm.piece[i];
        __syncwarp();
        if (one) mbar_arrive(&sm.pempty[i]);
        if (pc.t0 < 0) break;
        const Need need(p, pc, w, TM);
        const Edge<kN> edge(p, pc, U);
        int t = pc.t0;
        do {
            if (!(ok = wait(&sm.ofree[w], (parts++ & 1) ^ 1, p))) break;
            bool first = true;  // the next product is the part's first
            const int end = min(pc.t1, t + kMost);
#pragma unroll 1
            for (; t < end; ++t) {
                const bool own = pc.pair || ((t - pc.t0) & 1) == w;
                const int tile = tile_of(pc, t);
                const bool e = edge(tile);
                const int m = !own ? 0 : e ? need(tile) : 3;
                if (e) {
                    ok = wait(&sm.fixed[at.slot], (fixed >> at.slot) & 1, p);
                    fixed ^= 1u << at.slot;
                } else {
                    ok = wait(&sm.vfull[at.slot], at.round, p);
                }
                if (!ok) break;
                const uint32_t v = v0 + at.slot * Ly::kTile;
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (m >> h & 1) {
                        if (!(ok = wait(&sm.pready[w][h], np >> h & 1, p))) break;
                        np ^= 1u << h;
                        tc_fence_after();
                        if (one) {
                            issue_pv<D>(tO, tS + kSub * h, v + h * kSub * 128, !first);
                            tc_commit(&sm.pvdone[w][h]);
                        }
                        first = false;
                    }
                if (!ok) break;
                if (one) {
                    if (own)
                        tc_commit(&sm.vempty[at.slot]);
                    else
                        mbar_arrive(&sm.vempty[at.slot]);
                }
                at.next();
            }
            if (ok && one) tc_commit(&sm.ofull[w]);
        } while (ok && t < pc.t1);
    }
    if (one) tc_commit(&sm.end[2 + w]);
    drain(&sm.end[2 + w], 0, p);
}

// ------------------------------------------------------------------------- values at the edges
template <int D>
__device__ void fix_role(const PrefillParams& p, Smem<D>& sm, int warp, int lane) {
    using Ly = Layout<D>;
    const int U = 2 * (kM / p.G);
    uint32_t g = 0, phase = 0;  // value tiles before the piece; a bit for each slot
    if (stalls(p, &sm.never, 4)) return;
    for (int k = 0;; ++k) {
        const int i = k % kPieces;
        if (!wait(&sm.pfull[i], (k / kPieces) & 1, p)) break;
        const Piece pc = sm.piece[i];
        if (pc.t0 < 0) break;
        const int nt = pc.t1 - pc.t0;
        const Edge<kN> edge(p, pc, U);
        bool ok = true;
        for (int t = 0; t < nt && ok; ++t) {
            const int tile = tile_of(pc, pc.t0 + t);
            if (!edge(tile)) continue;
            const uint32_t n = g + t;
            const int s = n % Ly::kV;
            ok = wait(&sm.issued[s], (phase >> s) & 1, p) && wait(&sm.vfull[s], (n / Ly::kV) & 1, p);
            if (!ok) break;
            phase ^= 1u << s;
            const int valid = pc.L - tile * kN;  // rows of the sequence
            bool bad = false;
#pragma unroll 2
            for (int c = warp * 32 + lane; c < Ly::kTile / 16; c += kFixWarps * 32) {
                uint4* at = reinterpret_cast<uint4*>(sm.v[s]) + c;
                uint4 v = *at;
                // bfloat16 pairs whose exponent bits are all ones
                auto odd = [](uint32_t x) { return ((x & 0x7f807f80u) + 0x00800080u) & 0x80008000u; };
                const int row = (c / 8) % kN;
                if (row >= valid) {
                    *at = make_uint4(0, 0, 0, 0);
                } else if (odd(v.x) | odd(v.y) | odd(v.z) | odd(v.w)) {
                    bad = true;
                    auto clear = [&](uint32_t x) {
                        const uint32_t o = odd(x);
                        return x & ~((o & 0x8000u ? 0xffffu : 0u) | (o & 0x80000000u ? 0xffff0000u : 0u));
                    };
                    *at = make_uint4(clear(v.x), clear(v.y), clear(v.z), clear(v.w));
                }
            }
            if (bad) atomicOr(&sm.bad[i], 1u << (t >> odd_shift(pc)));
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.fixed[s]);
        }
        if (lane == 0) mbar_arrive(&sm.pempty[i]);
        if (!ok) break;
        g += nt;
    }
}

// ----------------------------------------------------------------------------------- softmax
template <int D>
__device__ void softmax_role(const PrefillParams& p, Smem<D>& sm, int warp, int lane) {
    const int w = warp / 4;                       // stream
    const int r = (warp % 4) * 32 + lane;         // row of the tile, lane of tensor memory
    const int TM = kM / p.G, U = 2 * TM;
    const uint32_t quad = static_cast<uint32_t>((warp % 4) * 32) << 16;
    const uint32_t tS = sm.tmem_base + quad + kColS + 128 * w;
    const uint32_t tO = sm.tmem_base + quad + kColO;
    const bool negative = p.scale_log2 < 0.f;
    const float c = fmaxf(fabsf(p.scale_log2), 0x1p-100f);  // (0: -inf times it stays -inf)
    const int tok_r = r / p.G;
    uint32_t ns = 0, parts = 0;  // a parity bit for each score buffer; parts handed over
    if (stalls(p, &sm.never, 5)) return;
    for (int k = 0;; ++k) {
        const int i = k % kPieces;
        if (!wait(&sm.pfull[i], (k / kPieces) & 1, p)) break;
        const Piece pc = sm.piece[i];
        if (pc.t0 < 0) break;
        const int token = pc.tok0 + (pc.pair ? w * TM : 0) + tok_r;
        const bool valid = tok_r < TM && token < pc.n;
        const bool busy = __any_sync(0xffffffffu, valid);
        const int pos = valid ? pc.L - pc.n + token : 0x3fffffff;
        const Need need(p, pc, w, TM);
        const Edge<kN> at_edge(p, pc, U);
        float m = -INFINITY, l = 0.f;  // reference maximum (raw score units), sum
        bool ok = true, any = false;   // any: a product of this part has been or will be added to O
        int t = pc.t0 + (pc.pair ? 0 : w), end = pc.t0;
        do {
            end = min(pc.t1, end + kMost);
            for (; t < end && ok; t += pc.pair ? 1 : 2) {
                const int tile = tile_of(pc, t), halves = at_edge(tile) ? need(tile) | 4 : 3;  // 4: at an edge
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    if (!(halves >> h & 1)) continue;
                    if (!(ok = wait(&sm.sfull[w][h], ns >> h & 1, p))) break;
                    ns ^= 1u << h;
                    if (busy) {
                        tc_fence_after();
                        uint32_t s[2][32];
                        tmem_ld_32x32b_x32(tS + kSub * h, s[0]);
                        tmem_ld_32x32b_x32(tS + kSub * h + 32, s[1]);
                        tmem_ld_wait(s[0]);
                        tmem_ld_wait(s[1]);
                        if (negative) {
                            uint32_t sign = 0x80000000u;
                            asm volatile("" : "+r"(sign));  // (nor of this)
#pragma unroll
                            for (int a = 0; a < kSub; ++a) s[a / 32][a % 32] ^= sign;
                        }
                        if (halves & 4) {
                            // the keys seen, a bit each: up to the row's own, in its window or a sink
                            const int ts = tile * kN + kSub * h;
                            const int hi = pos - ts, lo = p.window > 0 && valid ? hi - p.window + 1 : 0;
                            auto below = [](int n) -> uint64_t {  // the first n of 64 bits
                                return n <= 0 ? 0 : n >= 64 ? ~0ull : (1ull << n) - 1;
                            };
                            const uint64_t seen = below(hi + 1) & (~below(lo) | below(p.n_sink - ts));
                            uint32_t word[2] = {static_cast<uint32_t>(seen), static_cast<uint32_t>(seen >> 32)};
                            asm volatile("" : "+r"(word[0]), "+r"(word[1]));  // (nothing of this ahead of the branch)
#pragma unroll
                            for (int a = 0; a < kSub; ++a)
                                if (!(word[a / 32] >> (a % 32) & 1)) s[a / 32][a % 32] = 0xff800000u;
                        }
                        float mx[4];
#pragma unroll
                        for (int a = 0; a < 4; ++a) mx[a] = __uint_as_float(s[a / 2][16 * (a % 2)]);
#pragma unroll
                        for (int e = 1; e < 15; e += 2)
#pragma unroll
                            for (int a = 0; a < 4; ++a)
                                mx[a] = max3(mx[a], __uint_as_float(s[a / 2][16 * (a % 2) + e]),
                                             __uint_as_float(s[a / 2][16 * (a % 2) + e + 1]));
                        const float top = max3(max3(mx[0], mx[1], __uint_as_float(s[0][15])),
                                               max3(mx[2], mx[3], __uint_as_float(s[0][31])),
                                               fmaxf(__uint_as_float(s[1][15]), __uint_as_float(s[1][31])));
                        const bool raise = (top - m) * c > kGrowth;  // (m = -inf: always)
                        float fade = 1.f;
                        if (raise) {
                            fade = fast_exp2((m - top) * c);
                            m = top;
                            l *= fade;
                        }
                        if (any && __any_sync(0xffffffffu, raise)) {
                            // this buffer's last product is complete (its scores waited for it); the
                            // other's when its barrier says so
                            ok = wait(&sm.pvdone[w][1 - h], (ns >> (1 - h) & 1) ^ 1, p);
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll 1
                            for (int a = 0; a < D / 16; ++a) {
                                uint32_t o[16];
                                tmem_ld_x16(tO + 128 * w + 16 * a, o);
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    o[e] = __float_as_uint(__uint_as_float(o[e]) * fade);
                                tmem_st_x16(tO + 128 * w + 16 * a, o);
                            }
                        }
                        const float mc = m == -INFINITY ? 0.f : fmaf(m, c, kGrowth);
                        const uint64_t c2 = pair64(c, c), n2 = pair64(-mc, -mc);
                        uint64_t sum[2] = {pair64(0.f, 0.f), pair64(0.f, 0.f)};
#pragma unroll
                        for (int a = 0; a < 2; ++a) {
                            uint32_t pr[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const uint64_t y = fma2(pair64(__uint_as_float(s[a][2 * e]),
                                                               __uint_as_float(s[a][2 * e + 1])), c2, n2);
                                float u, v;
                                unpair64(y, u, v);
                                u = fast_exp2(u);
                                v = fast_exp2(v);
                                sum[e & 1] = add2(sum[e & 1], pair64(u, v));
                                pr[e] = pack_bf16(u, v);
                            }
                            tmem_st_x16(tS + kSub * h + 16 * a, pr);
                        }
                        float x0, x1;
                        unpair64(add2(sum[0], sum[1]), x0, x1);
                        l += x0 + x1;  // (once for 64 keys: one by one, small weights are rounded away)
                        tmem_st_wait();
                        tc_fence_before();
                    }
                    any = true;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.pready[w][h]);
                }
            }
            // what the unit's end needs; the softmax goes on with the next part or piece
            if (!ok || !(ok = wait(&sm.statr[w], (parts++ & 1) ^ 1, p))) break;
            sm.stat[w][r][0] = m == -INFINITY ? -INFINITY : fmaf(m, c, kGrowth);  // log2 units
            sm.stat[w][r][1] = any ? l : -1.f;  // (below 0: nothing has been added)
            l = 0.f;
            any = false;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.statw[w]);
        } while (end < pc.t1);
        if (!ok) break;
        if (lane == 0) mbar_arrive(&sm.pempty[i]);
    }
}

// ------------------------------------------------------------------------------------ unit's end
// 32 bytes (wide: from a multiple of 32).
__device__ __forceinline__ void store32(char* dst, bool wide, const uint32_t* x) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(x[0]), "r"(x[1]),
                     "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(dst)[0] = make_uint4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<uint4*>(dst)[1] = make_uint4(x[4], x[5], x[6], x[7]);
    }
}

// What a piece with values that are not finite (marks), or a part of one, needs behind its stores, to the output or
// to a slot: the thread's rows are row r of each query tile. (Behind both tiles, and not a function of its own: the
// call, made where much is in registers, spilled what a unit's end needs, and 513 tokens took 19.6 us for 18.3.)
template <int D>
__device__ __forceinline__ void end_more(const PrefillParams& p, const Piece& pc, uint32_t marks, int slot, int end,
                                      int r) {
    const int TM = kM / p.G, t = r / p.G;
    const bool first = end - kMost <= pc.t0, last = end >= pc.t1;
    if (marks && last) {
#pragma unroll 1
        for (int w = 0; w <= pc.pair; ++w) {
            const int token = pc.tok0 + w * TM + t;
            const long long at =
                slot < 0 ? static_cast<long long>(pc.c0 + token) * p.Hq + pc.h * p.G + (r - t * p.G)
                         : static_cast<long long>(slot) * 2 * kM + w * kM + r;
            put_back<D, kN, __nv_bfloat16, true>(
                p, pc, marks, 2 * TM, t < TM && token < pc.n, pc.L - pc.n + token,
                slot < 0 ? static_cast<void*>(static_cast<__nv_bfloat16*>(p.out) + at * D) : p.part_o + at * D,
                slot < 0, threadIdx.x % 32);
        }
    }
    if (!(first && last)) add_part<D, __nv_bfloat16>(p, pc, slot, first, last, r);
    __syncwarp();
}

// A piece's rows: from their sums and, as soon as their products are complete, their outputs. (Done by the
// softmax's warps, this kept them from the next unit's scores for some 9000 cycles a unit.)
template <int D>
__device__ void end_role(const PrefillParams& p, Smem<D>& sm, int quarter, int lane) {
    const int r = quarter * 32 + lane;  // row of the tile, lane of tensor memory
    const int TM = kM / p.G;
    const uint32_t tO = sm.tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + kColO;
    const int tok_r = r / p.G, head_r = r - tok_r * p.G;
    uint32_t parts = 0;  // taken over
    if (stalls(p, &sm.never, 6)) return;
    for (int k = 0;; ++k) {
        const int i = k % kPieces;
        if (!wait(&sm.pfull[i], (k / kPieces) & 1, p)) break;
        const Piece& pc = sm.piece[i];
        if (pc.t0 < 0) break;
        const int head = pc.h * p.G + head_r;
        bool ok = true;
        int end = pc.t0;
        do {
            end += kMost;
            const int slot = pc.t1 - pc.t0 > kMost ? 2 * p.n_cta + static_cast<int>(blockIdx.x) : pc.slot;
            const bool last = slot < 0;
            // two query tiles: stream w's rows in turn; one: its rows, from both streams
#pragma unroll 1
            for (int w = 0; w <= pc.pair && ok; ++w) {
                ok = wait(&sm.statw[w], parts & 1, p) && (pc.pair || wait(&sm.statw[1], parts & 1, p));
                if (!ok) break;
                const int token = pc.tok0 + (pc.pair ? w * TM : 0) + tok_r;
                const bool valid = tok_r < TM && token < pc.n;
                float m0 = sm.stat[w][r][0], l0 = sm.stat[w][r][1], m1 = -INFINITY, l1 = -1.f;
                if (!pc.pair) {
                    m1 = sm.stat[1][r][0];
                    l1 = sm.stat[1][r][1];
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&sm.statr[w]);
                    if (!pc.pair) mbar_arrive(&sm.statr[1]);
                }
                const bool has0 = !(l0 < 0.f), has1 = !(l1 < 0.f);  // (the same for all rows)
                l0 = has0 ? l0 : 0.f;
                l1 = has1 ? l1 : 0.f;
                const float top = fmaxf(m0, m1);
                float f0 = m0 == -INFINITY ? 0.f : fast_exp2(m0 - top), f1 = m1 == -INFINITY ? 0.f : fast_exp2(m1 - top);
                // (a sum that is NaN has a maximum of -inf where all of its scores are NaN)
                float sum = (m0 == -INFINITY ? l0 : l0 * f0) + (m1 == -INFINITY ? l1 : l1 * f1);
                if (top == -INFINITY) f0 = f1 = 1.f;
                const long long row = static_cast<long long>(pc.c0 + token) * p.Hq + head;
                if (last) {
                    float ref = top, scale = 1.f;
                    if (p.sink_logit && valid) {
                        const float sink = p.sink_logit[head] * kLog2e;
                        ref = fmaxf(top, sink);
                        scale = top == -INFINITY ? 1.f : fast_exp2(top - ref);
                        sum = sum * scale + (sink == -INFINITY ? 0.f : fast_exp2(sink - ref));
                    }
                    scale = sum == 0.f ? 0.f : scale / sum;
                    f0 *= scale;
                    f1 *= scale;
                    if (valid && p.lse_out)
                        p.lse_out[row] =
                            sum == 0.f ? -INFINITY : ((ref == -INFINITY ? 0.f : ref) + log2f(sum)) * kLn2;
                } else if (valid) {
                    reinterpret_cast<float2*>(p.part_ml)[static_cast<size_t>(slot) * 2 * kM + w * kM + r] =
                        make_float2(top, sum);
                }
                char* dst = last ? static_cast<char*>(p.out) + row * D * 2
                                 : reinterpret_cast<char*>(
                                       p.part_o + (static_cast<long long>(slot) * 2 * kM + w * kM + r) * D);
                const bool wide = (reinterpret_cast<uintptr_t>(dst) & 31) == 0;  // (the same for all rows)
                ok = wait(&sm.ofull[w], parts & 1, p) && (pc.pair || wait(&sm.ofull[1], parts & 1, p));
                if (!ok) break;
                tc_fence_after();
                if (__any_sync(0xffffffffu, valid)) {
                    // 32 bytes a store: the rows that a store's lanes touch, 2.7 cycles each, set its pace.
                    // (Exchanging pieces between lanes first, for runs of 64 bytes, takes more instructions
                    // than that saves.)
#pragma unroll 1
                    for (int col = 0; col < D; col += 16) {
                        float f[16];
                        uint32_t o[16];
                        if (has0) tmem_ld_x16(tO + 128 * w + col, o);
#pragma unroll
                        for (int e = 0; e < 16; ++e) f[e] = has0 ? __uint_as_float(o[e]) * f0 : 0.f;
                        if (has1) {
                            tmem_ld_x16(tO + 128 + col, o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) f[e] = fmaf(__uint_as_float(o[e]), f1, f[e]);
                        }
                        if (valid && last) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) o[e] = pack_bf16(f[2 * e], f[2 * e + 1]);
                            store32(dst + col * 2, wide, o);
                        } else if (valid) {
                            store32(dst + col * 4, wide, reinterpret_cast<uint32_t*>(f));
                            store32(dst + col * 4 + 32, wide, reinterpret_cast<uint32_t*>(f) + 8);
                        }
                        __syncwarp();
                    }
                    __syncwarp();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&sm.ofree[w]);
                    if (!pc.pair) mbar_arrive(&sm.ofree[1]);
                }
            }
            if (!ok) break;
            ++parts;
            __syncwarp();
            const uint32_t bad = *reinterpret_cast<volatile uint32_t*>(&sm.bad[i]);
            if (__builtin_expect(bad || pc.t1 - pc.t0 > kMost, 0)) end_more<D>(p, sm.piece[i], bad, slot, end, r);
        } while (end < pc.t1);
        if (!ok) break;
        if (lane == 0) mbar_arrive(&sm.pempty[i]);
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_bf16_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                        const __grid_constant__ CUtensorMap tv, const PrefillParams p) {
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
        for (int i = 0; i < Layout<D>::kK; ++i) {
            mbar_init(&sm.kfull[i], 1);
            mbar_init(&sm.kempty[i], 2);
        }
        for (int i = 0; i < Layout<D>::kV; ++i) {
            mbar_init(&sm.vfull[i], 1);
            mbar_init(&sm.vempty[i], 2);
            mbar_init(&sm.issued[i], 1);
            mbar_init(&sm.fixed[i], kFixWarps);
        }
        mbar_init(&sm.qfull, 1);
        mbar_init(&sm.qempty, 2);
        for (int i = 0; i < 2; ++i) {
            for (int h = 0; h < 2; ++h) {
                mbar_init(&sm.sfull[i][h], 1);
                mbar_init(&sm.pready[i][h], 4);
                mbar_init(&sm.pvdone[i][h], 1);
            }
            mbar_init(&sm.ofull[i], 1);
            mbar_init(&sm.ofree[i], 4);
            mbar_init(&sm.statw[i], 4);
            mbar_init(&sm.statr[i], 4);
            mbar_init(&sm.end[i], 1);
            mbar_init(&sm.end[2 + i], 1);
        }
        mbar_init(&sm.never, 1);
        for (int i = 0; i < kPieces; ++i) {
            mbar_init(&sm.pfull[i], 1);
            mbar_init(&sm.pempty[i], 4 + kFixWarps + kSoftWarps + 4);
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
    } else {
        regs_fewer<kRegsOther>();
        if (warp == kWarpLoad)
            load_role<D>(p, sm, &tq, &tk, &tv, lane);
        else if (warp < kWarpPv)
            qk_role<D>(p, sm, warp - kWarpQk, lane);
        else if (warp < kWarpFix)
            pv_role<D>(p, sm, warp - kWarpPv, lane);
        else if (warp >= kWarpEnd)
            end_role<D>(p, sm, warp - kWarpEnd, lane);
        else
            fix_role<D>(p, sm, warp - kWarpFix, lane);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWarpQk) tmem_dealloc(sm.tmem_base, 512);
}

template <int D>
int launch(PrefillParams p, void* ws, cudaStream_t stream) {
    CUtensorMap tq, tk, tv;
    const uint64_t blocks = D / 64;
    {
        const uint64_t dims[4] = {64, static_cast<uint64_t>(p.Hq), static_cast<uint64_t>(p.T), blocks};
        const uint64_t strides[3] = {D * 2, static_cast<uint64_t>(p.q_stride) * 2, 128};
        const uint32_t box[4] = {64, static_cast<uint32_t>(p.G), static_cast<uint32_t>(kM / p.G), 1};
        if (make_tmap_bf16_4d(&tq, p.q, dims, strides, box) != KVD_OK) return KVD_ERR_CUDA;
    }
    for (int i = 0; i < 2; ++i) {
        CUtensorMap* map = i ? &tv : &tk;
        if (p.block_table) {
            const uint32_t rows = 1u << std::min(p.page_shift, 7);
            const uint64_t dims[4] = {64, (static_cast<uint64_t>(p.num_pages) * p.Hkv) << p.page_shift, blocks, 1};
            const uint64_t strides[3] = {D * 2, 128, D * 2};
            const uint32_t box[4] = {64, rows, rows == kN ? static_cast<uint32_t>(blocks) : 1, 1};
            if (make_tmap_bf16_4d(map, i ? p.v : p.k, dims, strides, box) != KVD_OK) return KVD_ERR_CUDA;
        } else {
            // (without keys nothing is loaded; any address makes a map)
            const void* at = p.Tk > 0 ? (i ? p.v : p.k) : p.q;
            const uint64_t stride = static_cast<uint64_t>(i ? p.v_stride : p.k_stride) * 2;
            const uint64_t dims[4] = {64, static_cast<uint64_t>(std::max(p.Tk, 1)), blocks,
                                      static_cast<uint64_t>(p.Hkv)};
            const uint64_t strides[3] = {stride, 128, D * 2};
            const uint32_t box[4] = {64, kN, static_cast<uint32_t>(blocks), 1};
            if (make_tmap_bf16_4d(map, at, dims, strides, box) != KVD_OK) return KVD_ERR_CUDA;
        }
    }
    auto kernel = prefill_bf16_kernel<D>;
    constexpr int smem = static_cast<int>(sizeof(Smem<D>));
    static_assert(smem <= 227 * 1024, "prefill shared memory");
    static const cudaError_t set =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (set != cudaSuccess) return KVD_ERR_CUDA;
    // A unit's start and end count as 320 keys (nine prompts of 61 to 3581 tokens, 32/8 heads of 128: 500 us
    // with 0, 395 with 192, 390 with 320, 385 with 512, 391 with 768; one of 16385: 1.67 ms, 1.59, 1.60, 1.61,
    // 1.63). A call of fewer units than SMs is left uncut if that makes its longest range at most 8 tiles
    // longer (5 draft tokens behind 1024: 19.1 us; with 24 tiles 20.9).
    set_plan(p, D, ws, 320, 8 * kN);
    if (launch_kernel(kernel, dim3(static_cast<unsigned>(p.n_cta)), dim3(kThreads), smem, stream, tq, tk,
                      tv, p) != cudaSuccess ||
        launch_merge<D, __nv_bfloat16, kN>(p, 2 * (kM / p.G), stream) != cudaSuccess)
        return KVD_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? KVD_OK : KVD_ERR_CUDA;
}

}  // namespace

size_t prefill_ws_bytes(int D) { return make_plan(D).total; }

int prefill_bf16_launch(const PrefillParams& p, int D, void* ws, cudaStream_t stream) {
    return D == 64 ? launch<64>(p, ws, stream) : launch<128>(p, ws, stream);
}

}  // namespace kvd
