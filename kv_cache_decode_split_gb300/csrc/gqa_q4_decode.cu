// gqa_q4_decode.cu -- single-token attention over a paged or rolling cache held in 4 bits.
//
// What is computed, with k and v the values that the codes stand for (kvd_q4.cuh):
//   o_h = sum_{t in V} e^{x_t} v_t / (sum_{t in V} e^{x_t} + [sink] e^{sigma_h}),
//   x_t = scale q_h . k_t, query head h reading KV head h / (Hq / Hkv),
// V the visible slots: all of the sequence, the window and the sink tokens, or what a rolling cache
// holds. With k = s code + b per group of 64 channels the score is sum_g s_g (q_g . code) + b_g sum(q_g),
// so the matrix product runs on the codes and scale and minimum enter once per token and group; with
// v = s code + b the weight p s multiplies the codes, and sum_t p b is one number per head and group.
//
// GB300. 4 bits quarter the bytes but not the elements: at the measured copy bandwidth an SM has
// about 2.7 lane operations for each element it reads, so what matters is instructions per
// element, logic and shift operations (half rate) first of all. Codes go from shared memory to
// matrix-instruction fragments with one shift and one three-input logic operation per two
// elements: code bits placed in the mantissa under a fixed exponent are the number 16 + c (keys,
// bf16) or 64 + c (values, float16), exactly. (Feeding tcgen05 would write every element back to
// shared memory as 16 bits first, which alone costs more than the whole budget; with at most 16
// query rows its rate is not needed. 8-bit matrix instructions on the codes were tried too: on this
// machine mma.sync's are slower than the 16-bit ones.) The scores' offset is taken out with the
// group's minimum, (b - 16 s) sum(q_g). Of the values, odd tokens are decoded with the sign
// flipped and the code complemented, -(64 + 15 - c) = c - 79: the offsets 64 and -79 average to
// the middle of the code range, so the sums stay small over long sequences; one more matrix
// product, of a constant with the same rounded weights, takes them out again.
//   scores^T [16 tokens x 8 heads] = K codes [16 x D] q^T           (mma.sync m16n8k16, fp32 sums)
//   O^T [16 channels x 8 heads]   += V codes^T [16 x 16 tokens] (p s)^T
// p s is a float16 number (11 bits; two for float32 queries), so that rounding the weights adds
// little to the output's own rounding. The softmax reference m is the largest score plus
// logarithm of its scale, rather than the largest score: then p s fits float16 whatever the
// values' sizes. It is raised only when a product leaves the range.
//
// A warp streams 64-token tiles through a ring of its own in shared memory (bulk copies, one per
// page piece, codes and scales together) and needs no other warp until its piece of a sequence
// ends. One CTA on each SM, with as many warps as registers and shared memory hold. Work is divided
// in one of two ways.
// List: the tiles of all (sequence, KV head, head block) units form one list, and each warp takes
// an equal share of it, whatever sequences it belongs to. A warp stores one partial (reference,
// sum, O) for each unit that it has a piece of, or the result itself if it had the whole unit;
// where units are cut into many pieces a CTA joins its warps' last ones in shared memory first. A
// second launch joins what was cut.
// Unit: in short calls a cluster of 1 to 8 CTAs takes one unit and joins it in distributed shared
// memory, in one launch.
//
// Measured (calls in a graph, inputs in turn, more of them than L2 holds). Full SMs read at the rate of
// a copy: 2 x 262144 more tokens of 8 heads of 128 channels at 6.6 TB/s. What a call costs beside that
// is about 11 us: start and tile look-up 2.5, first data, joining. 2 x 131072 tokens, 32 query heads:
// 56 us (floor 44); 32 ragged sequences of up to 8192: 46 us (33). With 9 to 16 heads to a KV head
// registers leave two warps to a scheduler, which wait for their own instructions: 96 ragged sequences
// 36 us (floor 10.6), 38% of issue slots used. Float32 queries have three and two products where
// bfloat16 ones have one: 32 x 4096 tokens 51 us (34; floor 22).
// The unit form against the list's, 32 query and 8 KV heads: 8 x 2048 tokens 11.8 us (14.1),
// 8 x 4096 15.9 (18.4), and one launch for the host to make, 2.8 us (4.3). It is chosen by what the
// block table has room for, so short sequences in a wide table take the list.
// The list costs every warp, and every CTA that joins, a look at all lengths, 32 at a time: nothing at
// a hundred sequences, most of the time at thousands of short ones (4096 x 64 tokens of one head 525 us).

#include <algorithm>
#include <type_traits>

#include "kvd_device.cuh"
#include "kvd_host.h"
#include "kvd_q4.cuh"

namespace kvd {

namespace {

constexpr int kTileTok = 64;   // tokens of a tile: four 16-token blocks, used two at a time
constexpr int kTileLog = 6;
constexpr int kPutBy = 32;     // tiles of a warp between two times that it puts its sums by
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// maximum of nothing: finite, so that differences with it are defined
constexpr float kNone = -3.0e38f;

__device__ __forceinline__ float neg_inf() { return -__int_as_float(0x7f800000); }

// Length of sequence b, within bounds.
__device__ __forceinline__ int seq_len(const Q4Params& p, int b) {
    const int L = __ldcg(p.seq_lens + b);  // (from L2: the joining launch reads it early)
    if (L >= 0 && (p.ring > 0 || L <= p.max_len)) return L;
    record_error(p.err, KVD_ERR_DEVICE_OOB);
    return L < 0 ? 0 : p.max_len;
}
// The visible slots of a sequence (at most two ranges), empty for a length of 0.
__device__ __forceinline__ Ranges slots_of(const Q4Params& p, int L) {
    if (p.ring > 0) return Ranges{0, min(L, p.ring), 0, 0};
    return visible_ranges(L, p.window, p.n_sink);
}
__device__ __forceinline__ int range_tiles(int lo, int hi) {
    return hi > lo ? ((hi - 1) >> kTileLog) - (lo >> kTileLog) + 1 : 0;
}
__device__ __forceinline__ int tiles_of(const Ranges& r) {
    return range_tiles(r.lo0, r.hi0) + range_tiles(r.lo1, r.hi1);
}

// Tiles of each unit of 32 sequences from b0 on, summed up to and with each lane's own (one warp);
// n: the lane's own, L: its sequence's length.
__device__ __forceinline__ int scan_tiles(const Q4Params& p, int b0, int lane, int& n, int& L) {
    L = b0 + lane < p.B ? seq_len(p, b0 + lane) : 0;
    n = tiles_of(slots_of(p, L));
    int inc = n;  // 32 sequences of fewer than 2^30 slots
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += o;
    }
    return inc;
}

// The list of all units' tiles in order (fewer than 2^31, which the host checks), shared evenly by n
// warps, in the list's order. Some warps have one tile more than the others (or one at all): the
// first of n (at most one for each tile), or, where CTAs join their warps' partials (`join`; warps
// c kCta .. are CTA c's), as many in each CTA, but for one more in the first ones.
template <int kCta>
struct Shares {
    uint32_t n, base, extra, each, more;
    bool join;
    __device__ Shares(const Q4Params& p, uint32_t tiles_of_units) {
        const uint32_t total = tiles_of_units * p.HU;
        join = p.join != 0;
        n = join ? static_cast<uint32_t>(p.n_warps) : min(static_cast<uint32_t>(p.n_warps), total);
        base = n > 0 ? total / n : 0;
        extra = total - base * n;
        each = extra / (n / kCta + !join);
        more = extra - each * (n / kCta);
    }
    __device__ uint32_t begin(uint32_t i) const {
        if (!join) return i * base + min(i, extra);
        const uint32_t c = i / kCta;
        return i * base + c * each + min(c, more) + min(i - c * kCta, each + (c < more));
    }
    __device__ int owner(uint32_t tile) const {
        if (!join) return find(tile, base, extra);
        const uint32_t all = kCta * base + each;  // tiles of a CTA, but for the first ones' one more
        const uint32_t c = find(tile, all, more);
        return static_cast<int>(c * kCta + find(tile - c * all - min(c, more), base, each + (c < more)));
    }
    // tile -> share, the first `longer` shares having size + 1 tiles and the others size
    __device__ static uint32_t find(uint32_t tile, uint32_t size, uint32_t longer) {
        const uint32_t t = longer * (size + 1);
        return tile < t ? tile / (size + 1) : longer + (tile - t) / size;
    }
};

// c[16x8] += a[16x16] * b[16x8], fp32 sums (not volatile: they may be reordered).
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// c = a * b (the accumulator starts at zero, without registers cleared for it).
__device__ __forceinline__ void mma_bf16_first(float (&c)[4], uint32_t a0, uint32_t a1,
                                               uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// Keys: 16 + c as bf16, code bits at mantissa bits 3-6.
constexpr uint32_t kKeyMask = 0x00780078u, kKey = 0x41804180u;
// Values: float16, code bits at mantissa bits 4-7: 64 + c, for odd tokens (the high halves)
// -(64 + 15 - c) = c - 79.
constexpr uint32_t kValMask = 0x00F000F0u, kVal = 0xD4F05400u, kVal64 = 0x54005400u;
constexpr uint32_t kValOff = 0x54F0D400u;  // minus the offsets: -64 and 79

// A constant that stays in a register (a logic instruction takes one immediate, and the compiler
// would rather split it in two): read back from shared memory.
__device__ __forceinline__ uint32_t read_shared(const uint32_t* p) {
    uint32_t r;
    asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(r) : "r"(smem_u32(p)));
    return r;
}

// One more copy's bytes for a barrier's phase to wait for.
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)),
                 "r"(bytes)
                 : "memory");
}

// Load from another CTA's shared memory (cluster address from map_peer).
__device__ __forceinline__ float2 ld_cluster_v2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                 : "=f"(v.x), "=f"(v.y)
                 : "r"(addr)
                 : "memory");
    return v;
}

// Codes with their offset -> c - 8 (exact), for float32 queries: nothing is left to cancel.
__device__ __forceinline__ uint32_t centre_key(uint32_t x) {
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&x),
                                     __floats2bfloat162_rn(24.f, 24.f));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t centre_val(uint32_t x) {
    const __half2 r = __hsub2(*reinterpret_cast<__half2*>(&x), __floats2half2_rn(72.f, 72.f));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// Two values as sums of kSplit bf16 numbers, part k of both packed.
template <int kSplit>
__device__ __forceinline__ void split_bf16(float x, float y, uint32_t (&part)[kSplit]) {
#pragma unroll
    for (int k = 0; k < kSplit; ++k) {
        part[k] = pack_bf16(x, y);
        if (k + 1 < kSplit) {
            x -= __uint_as_float(part[k] << 16);
            y -= __uint_as_float(part[k] & 0xffff0000u);
        }
    }
}

// A tile as the warp that uses it sees it: the unit, and bits 0 first tile of the warp's piece of
// the unit, 1 last, 2 first tile of the unit, 3 last, 4 not all of its tokens visible, 5 the sums are
// put by before it; from bit 8 the first visible token of the tile, from bit 16 the one behind the
// last.
using TileInfo = int2;

// One CTA on each SM; as many warps as its registers hold (a thread's products, sums and operands
// need 115 to 250) and, with 128 channels, its shared memory (two tiles of 18 KB a warp).
constexpr int warps_of(int d, int nt, bool f32) {
    return d == 128 ? (nt == 1 && !f32 ? 12 : 8) : f32 ? (nt == 1 ? 12 : 8) : (nt == 1 ? 16 : 11);
}

template <int D, int NT, bool kF32>
struct Q4Cfg {
    static constexpr int kWarps = warps_of(D, NT, kF32);
    static constexpr int kStages = 2;
    static constexpr int kTileBytes = 8 * Q4<D>::kBlockBytes;  // K and V, four blocks each
    static constexpr int kRing = kStages * kTileBytes;
    static constexpr int kPerWarp = kRing + kStages * static_cast<int>(sizeof(TileInfo) + 8);
    static constexpr int kSmem = kWarps * kPerWarp + 16 + kWarps * 8;
    // a warp's last piece, for the CTA's own joining: O, references, sums, over its ring
    static constexpr int kPieceFloats = NT * 8 * (D + 2);
    static_assert(kPieceFloats * 4 <= kRing, "a piece fits the ring");
};

// One more partial (references x, sums y, outputs v of two heads) into a running one.
__device__ __forceinline__ void add_piece(float& M0, float& M1, float& L0, float& L1, float4& acc,
                                          float x0, float x1, float y0, float y1, const float4& v) {
    const float t0 = fmaxf(M0, x0), t1 = fmaxf(M1, x1);
    const float a0 = fast_exp2(M0 - t0), a1 = fast_exp2(M1 - t1);
    const float w0 = fast_exp2(x0 - t0), w1 = fast_exp2(x1 - t1);
    M0 = t0, M1 = t1;
    L0 = fmaf(w0, y0, L0 * a0), L1 = fmaf(w1, y1, L1 * a1);
    acc.x = fmaf(w0, v.x, acc.x * a0), acc.z = fmaf(w0, v.z, acc.z * a0);
    acc.y = fmaf(w1, v.y, acc.y * a1), acc.w = fmaf(w1, v.w, acc.w * a1);
}

// kPair (128 channels, at most 4 heads): the matrix instructions' 8 columns are the heads once for
// each group of 64 channels. Column h takes the queries of group 0 (and zeros), column 4 + h those
// of group 1; a lane then scales its own group's products, adds the other half's (one exchange),
// and its weights carry its own group's scale: half the scaling, packing and transposing of the
// general form, where half the columns would be empty.
//
// kLong: the matrix instructions cut their float32 sums instead of rounding them, so that a sum over many
// tokens drifts: with 18,400 tokens of a warp (16 million of 2 KV heads, bfloat16) the outputs were off by
// 6.5e-3 of their size, where their own rounding is 1.7e-3. Every kPutBy tiles a warp therefore adds its
// sums, by float32 arithmetic, to its slot of the workspace and starts from zero again: 1.8e-3. Calls that
// have no more than kPutBy tiles for each warp, by their block table, do without the code, which costs the
// others 1 to 3% (2 x 524288 tokens 195 us, 188 without; 32 x 4096 in a table for 131072 34.7 and 34.2).
//
// kUnit: short calls. A cluster of CTAs takes one unit, its warps the unit's tiles in equal shares, and
// joins it in distributed shared memory: no list of all tiles to work out, no second launch.
template <int D, int NT, bool kF32, bool kPair, bool kUnit, bool kLong>
__global__ void __launch_bounds__(Q4Cfg<D, NT, kF32>::kWarps * 32, 1)
    gqa_q4_kernel(const __grid_constant__ Q4Params p) {
    using Cfg = Q4Cfg<D, NT, kF32>;
    using L4 = Q4<D>;
    constexpr int S = Cfg::kStages, kWarps = Cfg::kWarps;
    static_assert(!kPair || (D == 128 && NT == 1 && !kF32), "two groups, one column tile");
    static_assert(!kLong || (!kF32 && !kUnit), "not needed there");
    constexpr int NG = kPair ? 1 : L4::kGroups;  // groups that a lane scales
    constexpr int NQ = kPair ? 2 : NG;           // accumulators of a score
    constexpr int KW = D / 32;             // key words of a lane and row
    constexpr int MT = D / 16;             // 16-channel tiles of the output
    constexpr int kQ = kF32 ? 3 : 1;       // bf16 parts of a query
    constexpr int kP = kF32 ? 2 : 1;       // float16 parts of a weight
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int g = lane >> 2, t = lane & 3;
    const int own = kPair ? t >> 1 : 0;  // (kPair) this lane's group
    uint8_t* ring = smem + warp * Cfg::kRing;
    TileInfo* info = reinterpret_cast<TileInfo*>(smem + kWarps * Cfg::kRing) + warp * S;
    uint64_t* full = reinterpret_cast<uint64_t*>(
                         smem + kWarps * (Cfg::kRing + S * sizeof(TileInfo))) + warp * S;
    uint32_t* masks = reinterpret_cast<uint32_t*>(smem + kWarps * Cfg::kPerWarp);
    // of each warp: its last piece's unit and that unit's heads
    int2* last_piece = reinterpret_cast<int2*>(masks + 4);
    if (lane == 0) {
        for (int s = 0; s < S; ++s) mbar_init(&full[s], 1);
        fence_mbar_init();
        masks[0] = kKeyMask;  // (every warp writes the same)
        masks[1] = kValMask;
        // (a test of the give-up path: one phase that the tile's copies do not complete)
        if (p.stall > 0) mbar_expect_tx(&full[p.stall - 1], 16);
    }
    __syncwarp();
    const uint32_t key_mask = read_shared(masks), val_mask = read_shared(masks + 1);
    griddep_wait();

    uint32_t me = 0, begin = 0;
    int n_mine = 0;     // tiles
    bool join = false;  // the CTA joins its warps' last pieces
    int scan_n = 0, scan_inc = 0, scan_len = 0;
    // kUnit: this cluster's unit, its sequence's ranges, the tiles and the warps that have some
    const int cs = kUnit ? p.cluster : 1, rank = kUnit ? static_cast<int>(blockIdx.x) % cs : 0;
    const int my_unit = kUnit ? static_cast<int>(blockIdx.x) / cs : 0;
    Ranges unit_ranges{};
    int unit_tiles = 0;
    if constexpr (kUnit) {
        unit_ranges = slots_of(p, seq_len(p, my_unit / p.HU));
        unit_tiles = tiles_of(unit_ranges);
        const int i = warp * cs + rank, n = kWarps * cs;
        const int base = unit_tiles / n, extra = unit_tiles % n;
        begin = i * base + min(i, extra);
        n_mine = base + (i < extra ? 1 : 0);
    } else {
        // The joining launch may come up as soon as this grid's CTAs leave (it waits for all of them
        // before it reads a partial).
        griddep_launch_dependents();

        // ---- this warp's share of the tile list
        // Where a CTA joins, its warps have neighbouring shares; elsewhere neighbouring shares are in
        // different CTAs (with fewer tiles than warps, the first warps of all CTAs take one each).
        scan_inc = scan_tiles(p, 0, lane, scan_n, scan_len);  // of the first 32 sequences
        uint32_t tiles = __shfl_sync(0xffffffffu, scan_inc, 31);
        for (int b0 = 32; b0 < p.B; b0 += 32) {
            int n, L;
            tiles += __shfl_sync(0xffffffffu, scan_tiles(p, b0, lane, n, L), 31);
        }
        const Shares<kWarps> sh(p, tiles);
        join = sh.join;
        me = join ? blockIdx.x * kWarps + warp : warp * gridDim.x + blockIdx.x;
        if (me >= sh.n) return;
        begin = sh.begin(me);
        n_mine = static_cast<int>(sh.begin(me + 1) - begin);
    }
    // Tiles are looked up 32 at a time, lane k the k-th of the batch: its pieces' first blocks in
    // the pools (one piece, or two or four when pages hold 32 or 16 tokens) and its TileInfo.
    // That lane issues its copies.
    int blk[4] = {};
    TileInfo mine = make_int2(0, 0);
    uint32_t special = 0;  // tiles of the batch that begin or end a piece or need masks
    // the warp's i-th tile, the j-th of the n of unit u of sequence b
    auto describe = [&](int i, int b, int u, int j, int n, const Ranges& r) {
        const int n0 = range_tiles(r.lo0, r.hi0);
        const int kvh = u / p.NHG;
        const int lo = j < n0 ? r.lo0 : r.lo1, hi = j < n0 ? r.hi0 : r.hi1;
        const int T = ((lo >> kTileLog) + (j < n0 ? j : j - n0)) * kTileTok;
        const int v0 = max(lo - T, 0), v1 = min(hi - T, kTileTok);
        mine.x = b * p.HU + u;
        mine.y = ((i == 0 || j == 0) ? 1 : 0) |
                 ((i == n_mine - 1 || j == n - 1) ? 2 : 0) | (j == 0 ? 4 : 0) |
                 (j == n - 1 ? 8 : 0) | ((v0 > 0 || v1 < kTileTok) ? 16 : 0) | v0 << 8 | v1 << 16;
        if (kLong && i % kPutBy == 0 && !(mine.y & 1)) mine.y |= 32;
        // The pages of its (up to four) pieces: a piece is a page's part of the tile. Pieces
        // without a visible token take the page of one that has.
        const int32_t* row = p.block_table + static_cast<size_t>(b) * p.max_pages;
        const int piece = min(kTileTok, 1 << p.page_shift);
        int pg[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k * piece < kTileTok) {
                const int tok = T + min(max(k * piece, v0), v1 - 1);
                pg[k] = __ldg(row + (tok >> p.page_shift));
            }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k * piece < kTileTok) {
                if (static_cast<unsigned>(pg[k]) >= static_cast<unsigned>(p.num_pages)) {
                    record_error(p.err, KVD_ERR_DEVICE_OOB);
                    pg[k] = 0;
                }
                blk[k] = ((pg[k] * p.Hkv + kvh) << (p.page_shift - 4)) +
                         ((T & ((1 << p.page_shift) - 1)) >> 4);
            }
    };
    // the warp's i-th tile, the rem-th from the beginning of sequence b (of length L) on
    auto resolve = [&](int i, uint32_t rem, int b, int L) {
        Ranges r = slots_of(p, L);
        int n = tiles_of(r);
        while (rem >= static_cast<uint32_t>(n) * p.HU) {  // this lane's own tile is further on
            rem -= static_cast<uint32_t>(n) * p.HU;
            r = slots_of(p, seq_len(p, ++b));
            n = tiles_of(r);
        }
        const int u = static_cast<int>(rem / n), j = static_cast<int>(rem % n);
        describe(i, b, u, j, n, r);
    };
    auto look_up = [&](int base) {  // tiles base .. base + 31 of this warp
        if constexpr (kUnit) {
            mine.y = 0;
            if (base + lane < n_mine)
                describe(base + lane, my_unit / p.HU, my_unit % p.HU, begin + base + lane,
                         unit_tiles, unit_ranges);
            special = __ballot_sync(0xffffffffu, (mine.y & 51) != 0);
            return;
        }
        const uint32_t at = begin + base, row = at / static_cast<uint32_t>(p.HU);
        uint32_t before = 0;  // tiles of one unit of each sequence passed
        int b = 0, len = 0;
        for (int b0 = 0; b0 < p.B; b0 += 32) {  // the sequence that holds tile `base`
            int n, inc, L;
            if (b0 == 0)
                n = scan_n, inc = scan_inc, L = scan_len;
            else
                inc = scan_tiles(p, b0, lane, n, L);
            const uint32_t past = __ballot_sync(0xffffffffu, before + inc > row);
            if (past) {
                const int k = __ffs(past) - 1;
                b = b0 + k;
                len = __shfl_sync(0xffffffffu, L, k);
                before += __shfl_sync(0xffffffffu, inc - n, k);
                break;
            }
            before += __shfl_sync(0xffffffffu, inc, 31);
        }
        const uint32_t rem = at - before * p.HU;
        mine.y = 0;
        if (base + lane < n_mine) resolve(base + lane, rem + lane, b, len);
        special = __ballot_sync(0xffffffffu, (mine.y & 51) != 0);
    };
    const uint64_t pol = l2_evict_first_policy();  // keys and values are read once
    // copy the warp's i-th tile into stage s
    uint32_t queue = 0;  // bit k: the k-th tile from the current one is special
    auto issue = [&](int s, int i, int ahead) {
        if ((i & 31) == 0) look_up(i);
        queue |= ((special >> (i & 31)) & 1) << ahead;
        if (lane == (i & 31)) {
            info[s] = mine;
            uint8_t* st = ring + s * Cfg::kTileBytes;
            if (p.page_shift >= kTileLog) {
                const size_t off = static_cast<size_t>(blk[0]) * L4::kBlockBytes;
                mbar_arrive_expect_tx(&full[s], Cfg::kTileBytes);
                bulk_load(st, p.k_pool + off, Cfg::kTileBytes / 2, &full[s], pol);
                bulk_load(st + Cfg::kTileBytes / 2, p.v_pool + off, Cfg::kTileBytes / 2, &full[s],
                          pol);
            } else {  // a piece without visible tokens is not copied (all of it is masked)
                const int v0 = (mine.y >> 8) & 127, v1 = (mine.y >> 16) & 127;
                const int piece = 1 << p.page_shift;
                const uint32_t bytes = (piece >> 4) * L4::kBlockBytes;
                uint32_t total = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k * piece < v1 && (k + 1) * piece > v0) total += 2 * bytes;
                mbar_arrive_expect_tx(&full[s], total);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k * piece < v1 && (k + 1) * piece > v0) {
                        const size_t off = static_cast<size_t>(blk[k]) * L4::kBlockBytes;
                        bulk_load(st + k * bytes, p.k_pool + off, bytes, &full[s], pol);
                        bulk_load(st + Cfg::kTileBytes / 2 + k * bytes, p.v_pool + off, bytes,
                                  &full[s], pol);
                    }
            }
        }
    };
    for (int s = 0; s < min(S, n_mine); ++s) issue(s, s, s);

    // ---- state of the current piece
    uint32_t qf[kQ][NT][KW][4];
    float qsum[NT][NG][2];  // sums of q, heads 2t and 2t + 1
    const float sl2 = p.scale_log2;
    // o, and the values' offsets and minima in it: oo by the matrix product, ob in each lane
    float o[NT][MT][4], oo[NT][NG][4], ob[NT][NG][2], m[NT][2], l[NT][2];
    bool from_start = false;
    // (kLong) scale of the sums put by (0: none yet) against the present reference
    float put[NT][2];
    // this lane's quads of O in a partial, for heads 2t and 2t + 1 (kPair: 2 (t & 1) and the next, of its
    // group's half of the channels)
    constexpr int kHave = kPair ? MT / 2 : MT;
    auto quads_of = [&](int nt) {
        return nt * (D * 8) + (kPair ? own * (kHave * 128) + (4 * g + (t & 1)) * 4 : lane * 4);
    };

    // sequence, first query head, and number of heads of a unit
    auto unit_of = [&](int unit) {
        const int b = unit / p.HU, u = unit % p.HU;
        const int kvh = u / p.NHG, hg = u % p.NHG;
        return make_int4(b, kvh * p.G + hg * NT * 8, min(NT * 8, p.G - hg * NT * 8), 0);
    };
    int2 left = make_int2(-1, 0);  // unit and heads of a last piece that this CTA is to join
    // The first tile that the warp did not get. Every unit that it has tiles left of then gets NaN for a
    // result, never what the workspace or the output held before (a reference that is NaN makes a
    // joined piece so).
    int lost = n_mine;
    const float kNan = __int_as_float(0x7fffffff);
    float* held_m = reinterpret_cast<float*>(ring) + NT * D * 8;  // the last piece's references
    int s = 0, phase = 0;
    for (int i = 0; i < n_mine; ++i) {
        __syncwarp();
        TileInfo ti = make_int2(0, 0);
        if (queue & 1) ti = info[s];
        if ((queue & 1) && (ti.y & 1)) {
            const int4 un = unit_of(ti.x);
            from_start = (ti.y & 4) != 0;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float part[NG] = {};
                const int h = kPair ? g & 3 : nt * 8 + g;
                const bool ok = h < un.z;
                const size_t qrow = (static_cast<size_t>(un.x) * p.Hq + un.y + (ok ? h : 0)) * D;
#pragma unroll
                for (int w = 0; w < KW; ++w) {
                    float x[8];
                    if constexpr (kF32) {
                        const float* q = static_cast<const float*>(p.q) + qrow + 32 * w + 8 * t;
                        const float4 a = *reinterpret_cast<const float4*>(q);
                        const float4 c = *reinterpret_cast<const float4*>(q + 4);
                        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
                        x[4] = c.x, x[5] = c.y, x[6] = c.z, x[7] = c.w;
                    } else {
                        const uint4 v = *reinterpret_cast<const uint4*>(
                            static_cast<const __nv_bfloat16*>(p.q) + qrow + 32 * w + 8 * t);
                        const uint32_t r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            x[2 * e] = __uint_as_float(r[e] << 16);
                            x[2 * e + 1] = __uint_as_float(r[e] & 0xffff0000u);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if (!ok || (kPair && w / 2 != g >> 2)) x[e] = 0.f;
                        part[kPair ? 0 : w / 2] += x[e];
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) {  // fragments pair channels e and e + 4
                        uint32_t sp[kQ];
                        split_bf16<kQ>(x[e], x[e + 4], sp);
#pragma unroll
                        for (int k = 0; k < kQ; ++k) qf[k][nt][w][e] = sp[k];
                    }
                }
#pragma unroll
                for (int gr = 0; gr < NG; ++gr) {
                    part[gr] += __shfl_xor_sync(0xffffffffu, part[gr], 1);
                    part[gr] += __shfl_xor_sync(0xffffffffu, part[gr], 2);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        qsum[nt][gr][c] = __shfl_sync(0xffffffffu, part[gr], (2 * t + c) * 4);
                        ob[nt][gr][c] = 0.f;
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r) oo[nt][gr][r] = 0.f;
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    m[nt][c] = kNone;
                    l[nt][c] = 0.f;
                    put[nt][c] = 0.f;
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int r = 0; r < 4; ++r) o[nt][mt][r] = 0.f;
            }
        }
        // ---- the sums put by: in the warp's slot of the workspace, which is its own to the end of the
        // piece (ob is rounded as it grows and stays; oo goes to it)
        if (kLong && (queue & 1) && (ti.y & 32)) {
            const int4 un = unit_of(ti.x);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int h0 = kPair ? 2 * (t & 1) : nt * 8 + 2 * t;
                float* at = p.part_o + (static_cast<size_t>(me) + ti.x) * (NT * D * 8) + quads_of(nt);
#pragma unroll
                for (int mt = 0; mt < kHave; ++mt) {
                    float4 was = make_float4(0.f, 0.f, 0.f, 0.f);
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[e] = kPair && own ? o[nt][mt + MT - kHave][e] : o[nt][mt][e];
                        o[nt][mt][e] = 0.f;
                        o[nt][mt + MT - kHave][e] = 0.f;
                    }
                    if (h0 < un.z) {
                        float4* q = reinterpret_cast<float4*>(at + mt * 128);
                        if (put[nt][0] > 0.f || put[nt][1] > 0.f) was = __ldcg(q);
                        __stcg(q, make_float4(fmaf(was.x, put[nt][0], v[0]), fmaf(was.y, put[nt][1], v[1]),
                                              fmaf(was.z, put[nt][0], v[2]), fmaf(was.w, put[nt][1], v[3])));
                    }
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    put[nt][c] = 1.f;
#pragma unroll
                    for (int gr = 0; gr < NG; ++gr) {
                        if (g == 0) ob[nt][gr][c] += oo[nt][gr][c];
                        oo[nt][gr][c] = oo[nt][gr][2 + c] = 0.f;
                    }
                }
            }
        }
        if (!__all_sync(0xffffffffu, mbar_wait(&full[s], phase, p.err, p.wait_cycles))) {
            // the warp gives up, once the copies in flight have landed (or their own limits have passed)
            if (lane == 0)
                for (int k = i + 1; k < min(n_mine, i + S); ++k)
                    mbar_wait(&full[k % S], (k / S) & 1, p.err, p.wait_cycles);
            __syncwarp();
            lost = i;
            if (kUnit && lane < NT * 8) held_m[lane] = kNan;
            break;
        }
        const int v0 = (ti.y >> 8) & 127, v1 = (ti.y >> 16) & 127;  // (special tiles only)
        // half a tile: tokens 32 sub .. 32 sub + 31. This lane's score rows are tokens 16 bk +
        // 8 half + g of them, bit 2 bk + half of `seen` (two copies of the code: whole tiles do
        // not look at it)
        auto half_tile = [&](auto is_ragged, int sub) {
        const uint8_t* kt = ring + s * Cfg::kTileBytes + sub * (2 * L4::kBlockBytes);
        const uint8_t* vt = kt + Cfg::kTileBytes / 2;
        constexpr bool ragged = decltype(is_ragged)::value;
        uint32_t seen = 15;
        if constexpr (ragged) {
            seen = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int tok = 32 * sub + 8 * k + g;
                seen |= (tok >= v0 && tok < v1) ? 1u << k : 0u;
            }
        }

        // ---- scores of the two blocks (before the softmax scale)
        float x[2][NT][4];
#pragma unroll
        for (int bk = 0; bk < 2; ++bk) {
            const uint8_t* kb = kt + bk * L4::kBlockBytes;
            uint32_t wa[KW], wb[KW];
            if constexpr (D == 128) {
                *reinterpret_cast<uint4*>(wa) = *reinterpret_cast<const uint4*>(kb + g * 64 + t * 16);
                *reinterpret_cast<uint4*>(wb) =
                    *reinterpret_cast<const uint4*>(kb + (g + 8) * 64 + t * 16);
            } else {
                *reinterpret_cast<uint2*>(wa) = *reinterpret_cast<const uint2*>(kb + g * 32 + t * 8);
                *reinterpret_cast<uint2*>(wb) =
                    *reinterpret_cast<const uint2*>(kb + (g + 8) * 32 + t * 8);
            }
            // (float32 queries: their leading parts, and what the other parts add)
            float acc[NT][NQ][4], rest[NT][NQ][4];
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                uint32_t fa[4], fb[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    fa[e] = (__funnelshift_r(wa[w], wa[w], 4 * e) & key_mask) ^ kKey;
                    fb[e] = (__funnelshift_r(wb[w], wb[w], 4 * e) & key_mask) ^ kKey;
                    if (kF32) fa[e] = centre_key(fa[e]), fb[e] = centre_key(fb[e]);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < kQ; ++k) {
                        auto& sums = k == 0 ? acc : rest;
                        float(&c0)[4] = sums[nt][kPair ? 0 : w / 2];
                        float(&c1)[4] = sums[nt][kPair ? 1 : w / 2];
                        const bool fresh = k <= 1 && (kPair ? w == 0 : w % 2 == 0);
                        if (fresh)
                            mma_bf16_first(c0, fa[0], fb[0], fa[1], fb[1], qf[k][nt][w][0],
                                           qf[k][nt][w][1]);
                        else
                            mma_bf16(c0, fa[0], fb[0], fa[1], fb[1], qf[k][nt][w][0],
                                     qf[k][nt][w][1]);
                        if (fresh && kPair)
                            mma_bf16_first(c1, fa[2], fb[2], fa[3], fb[3], qf[k][nt][w][2],
                                           qf[k][nt][w][3]);
                        else
                            mma_bf16(c1, fa[2], fb[2], fa[3], fb[3], qf[k][nt][w][2],
                                     qf[k][nt][w][3]);
                    }
            }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const __half2* pr =
                    reinterpret_cast<const __half2*>(kb + L4::param(g + 8 * half, own));
#pragma unroll
                for (int gr = 0; gr < NG; ++gr) {
                    const float2 f = __half22float2(pr[gr]);  // scale, minimum
                    // codes were held as 16 + c, or centred as c - 8
                    const float base = fmaf(kF32 ? 8.f : -16.f, f.x, f.y);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float& v = x[bk][nt][2 * half + c];
                            v = gr ? fmaf(base, qsum[nt][gr][c], v) : base * qsum[nt][gr][c];
                            float a = acc[nt][gr][2 * half + c];
                            if (kF32) a += rest[nt][gr][2 * half + c];
                            if (kPair) a += acc[nt][NQ - 1][2 * half + c];
                            v = fmaf(f.x, a, v);
                            if (kPair) v += __shfl_xor_sync(0xffffffffu, v, 2);
                        }
                }
            }
        }
        // ---- weights: p = 2^{scaled score - m}, and p times the values' scales as float16
        float vs[4][NG];  // scales of token 2 bk + half's groups
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __half2* pr = reinterpret_cast<const __half2*>(
                vt + (k >> 1) * L4::kBlockBytes + L4::param(g + 8 * (k & 1), own));
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) {
                vs[k][gr] = __low2float(pr[gr]);
                if (ragged && !((seen >> k) & 1))  // a masked slot may hold anything, NaN included
                    vs[k][gr] = 0.f;
            }
        }
        uint32_t y[NT][NG][kP][4];
        float pw[2][NT][4];
        bool over;
        auto weights = [&]() {
            __half2 top = __floats2half2_rn(0.f, 0.f);
            float ptop = 0.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float* pr = &pw[k >> 1][nt][2 * (k & 1)];
                    const float* xr = &x[k >> 1][nt][2 * (k & 1)];
                    pr[0] = fast_exp2(fmaf(xr[0], sl2, -m[nt][0]));
                    pr[1] = fast_exp2(fmaf(xr[1], sl2, -m[nt][1]));
                    if (ragged && !((seen >> k) & 1)) pr[0] = pr[1] = 0.f;
                    ptop = fmaxf(ptop, fmaxf(pr[0], pr[1]));
#pragma unroll
                    for (int gr = 0; gr < NG; ++gr) {
                        const float y0 = pr[0] * vs[k][gr], y1 = pr[1] * vs[k][gr];
                        __half2 h = __floats2half2_rn(y0, y1);
                        y[nt][gr][0][k] = *reinterpret_cast<uint32_t*>(&h);
                        top = __hmax2(top, h);
                        if constexpr (kP == 2) {
                            const float2 back = __half22float2(h);
                            __half2 lo2 = __floats2half2_rn(y0 - back.x, y1 - back.y);
                            y[nt][gr][1][k] = *reinterpret_cast<uint32_t*>(&lo2);
                        }
                    }
                }
            over = ptop > 0x1p60f || __hmax(__low2half(top), __high2half(top)) >
                                         __ushort_as_half(0x7800);  // 2^15
        };
        weights();
        // Raise the reference m when a weight leaves float16's range: to where the largest
        // product of weight and scale is 2^8 (7 binary orders of room, 22 below it before a weight
        // loses bits), and the weights alone stay far from float32's limits.
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float v = kNone;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float sc = NG == 2 ? fmaxf(vs[k][0], vs[k][NG - 1]) : vs[k][0];
                        const float xs = x[k >> 1][nt][2 * (k & 1) + c] * sl2;
                        if ((seen >> k) & 1) v = fmaxf(v, xs + fmaxf(log2f(sc) - 8.f, -60.f));
                    }
#pragma unroll
                    for (int off = kPair ? 2 : 4; off < 32; off <<= 1)
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
                    v = fmaxf(v, m[nt][c]);
                    const float al = fast_exp2(m[nt][c] - v);
                    m[nt][c] = v;
                    l[nt][c] *= al;
                    if (kLong) put[nt][c] *= al;
#pragma unroll
                    for (int gr = 0; gr < NG; ++gr) {
                        ob[nt][gr][c] *= al;
                        oo[nt][gr][c] *= al;
                        oo[nt][gr][2 + c] *= al;
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        o[nt][mt][c] *= al;
                        o[nt][mt][2 + c] *= al;
                    }
                }
            weights();
        }
        // ---- O += values * weights
#pragma unroll
        for (int bk = 0; bk < 2; ++bk) {
            const uint8_t* vb = vt + bk * L4::kBlockBytes;
            float vm[2][NG];  // minima (and, codes centred on 8, 8 scales)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const __half2* pr =
                    reinterpret_cast<const __half2*>(vb + L4::param(g + 8 * half, own));
#pragma unroll
                for (int gr = 0; gr < NG; ++gr) {
                    vm[half][gr] = __high2float(pr[gr]);
                    if (kF32) vm[half][gr] = fmaf(8.f, __low2float(pr[gr]), vm[half][gr]);
                    if (ragged && !((seen >> (2 * bk + half)) & 1)) vm[half][gr] = 0.f;
                }
            }
            uint32_t pf[NT][NG][kP][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const float* pr = &pw[bk][nt][2 * half];
                    l[nt][0] += pr[0];
                    l[nt][1] += pr[1];
#pragma unroll
                    for (int gr = 0; gr < NG; ++gr) {
                        ob[nt][gr][0] = fmaf(pr[0], vm[half][gr], ob[nt][gr][0]);
                        ob[nt][gr][1] = fmaf(pr[1], vm[half][gr], ob[nt][gr][1]);
#pragma unroll
                        for (int k = 0; k < kP; ++k)
                            pf[nt][gr][k][half] = movmatrix_t(y[nt][gr][k][2 * bk + half]);
                    }
                }
            uint4 va, vc;  // words of tokens 2t, 2t + 1 and of 2t + 8, 2t + 9
            if constexpr (D == 128) {
                va = *reinterpret_cast<const uint4*>(vb + lane * 16);
                vc = *reinterpret_cast<const uint4*>(vb + 512 + lane * 16);
            } else {
                va = *reinterpret_cast<const uint4*>(vb + lane * 16);
            }
#pragma unroll
            for (int gr = 0; gr < L4::kGroups; ++gr) {
                const int gp = kPair ? 0 : gr;  // index of the group's weights
                uint32_t w0, w1, w2, w3;  // tokens 2t, 2t + 1, 2t + 8, 2t + 9
                if constexpr (D == 128) {
                    w0 = gr ? va.y : va.x, w1 = gr ? va.w : va.z;
                    w2 = gr ? vc.y : vc.x, w3 = gr ? vc.w : vc.z;
                } else {
                    w0 = va.x, w1 = va.y, w2 = va.z, w3 = va.w;
                }
#pragma unroll
                for (int hw = 0; hw < 2; ++hw) {  // codes 0-3, then 4-7 of the words
                    const uint32_t u = __byte_perm(w0, w1, hw ? 0x7632 : 0x5410);
                    const uint32_t v = __byte_perm(w2, w3, hw ? 0x7632 : 0x5410);
                    constexpr uint32_t kX = kF32 ? kVal64 : kVal;
                    uint32_t fu[4], fv[4];
                    fu[0] = ((u << 4) & val_mask) ^ kX;
                    fv[0] = ((v << 4) & val_mask) ^ kX;
                    fu[1] = (u & val_mask) ^ kX;
                    fv[1] = (v & val_mask) ^ kX;
                    const uint32_t u8 = u >> 8, v8 = v >> 8;
                    fu[2] = ((u8 << 4) & val_mask) ^ kX;
                    fv[2] = ((v8 << 4) & val_mask) ^ kX;
                    fu[3] = (u8 & val_mask) ^ kX;
                    fv[3] = (v8 & val_mask) ^ kX;
                    if constexpr (kF32) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            fu[e] = centre_val(fu[e]), fv[e] = centre_val(fv[e]);
                    }
                    const int mt = gr * 4 + hw * 2;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint32_t(&w)[2] = pf[nt][gp][0];
                        // The matrix instructions cut their sums where float32 arithmetic rounds: with
                        // float32 queries they add 16 tokens, the small parts first, and the rest is
                        // rounded (16 million tokens of 2 KV heads: off by 6e-7, not 4e-4).
                        if constexpr (kF32) {
                            const uint32_t(&low)[2] = pf[nt][gp][1];
                            float d0[4], d1[4];
                            mma_f16_first(d0, fu[0], fu[1], fv[0], fv[1], low[0], low[1]);
                            mma_f16_first(d1, fu[2], fu[3], fv[2], fv[3], low[0], low[1]);
                            mma_f16(d0, fu[0], fu[1], fv[0], fv[1], w[0], w[1]);
                            mma_f16(d1, fu[2], fu[3], fv[2], fv[3], w[0], w[1]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                o[nt][mt][e] += d0[e];
                                o[nt][mt + 1][e] += d1[e];
                            }
                        } else {
                            mma_f16(o[nt][mt], fu[0], fu[1], fv[0], fv[1], w[0], w[1]);
                            mma_f16(o[nt][mt + 1], fu[2], fu[3], fv[2], fv[3], w[0], w[1]);
                        }
                    }
                }
                if (!kF32 && gr < NG) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_f16(oo[nt][gr], kValOff, kValOff, kValOff, kValOff, pf[nt][gr][0][0],
                                pf[nt][gr][0][1]);
                }
            }
        }
        };
        if ((queue & 1) && (ti.y & 16)) {
#pragma unroll 1
            for (int sub = v0 >> 5; sub <= (v1 - 1) >> 5; ++sub) half_tile(std::true_type{}, sub);
        } else {
#pragma unroll 1
            for (int sub = 0; sub < 2; ++sub) half_tile(std::false_type{}, sub);
        }
        // ---- end of the warp's piece of this unit
        if ((queue & 1) && (ti.y & 2)) {
            const int4 un = unit_of(ti.x);
            const bool whole = !kUnit && from_start && (ti.y & 8);
            const size_t slot = static_cast<size_t>(me) + ti.x;
            // A cut piece goes to the workspace, the warp's last one to shared memory, where no
            // copy is in flight any more.
            const bool at_end = kUnit || (join && i == n_mine - 1);
            if (at_end && !whole) left = make_int2(ti.x, un.z);
            float* held = reinterpret_cast<float*>(ring);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float mul[2], add[NG][2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float lv = l[nt][c];
#pragma unroll
                    for (int gr = 0; gr < NG; ++gr) add[gr][c] = ob[nt][gr][c];
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) {
                        lv += __shfl_xor_sync(0xffffffffu, lv, off);
#pragma unroll
                        for (int gr = 0; gr < NG; ++gr)
                            add[gr][c] += __shfl_xor_sync(0xffffffffu, add[gr][c], off);
                    }
#pragma unroll
                    for (int gr = 0; gr < NG; ++gr) add[gr][c] += oo[nt][gr][c];
                    const int h = kPair ? 2 * (t & 1) + c : nt * 8 + 2 * t + c;
                    mul[c] = 1.f;
                    if (h >= un.z) continue;
                    if (whole) {  // nothing to join: the output itself
                        const int hq = un.y + h;
                        const float sig = p.sink_logit ? p.sink_logit[hq] * kLog2e : neg_inf();
                        const float M = fmaxf(m[nt][c], sig);
                        const float w = fast_exp2(m[nt][c] - M);
                        const float den = lv * w + (p.sink_logit ? fast_exp2(sig - M) : 0.f);
                        mul[c] = w / den;
                        if (p.lse_out && g == 0 && own == 0)
                            p.lse_out[static_cast<size_t>(un.x) * p.Hq + hq] =
                                (M + log2f(den)) * kLn2;
                    } else if (g == 0 && own == 0) {
                        if (at_end) {
                            held[NT * D * 8 + h] = m[nt][c];
                            held[NT * 8 * (D + 1) + h] = lv;
                        } else {
                            __stcg(p.part_m + slot * (NT * 8) + h, m[nt][c]);
                            __stcg(p.part_l + slot * (NT * 8) + h, lv);
                        }
                    }
                }
                // (kPair: this lane has its own group's half of the channels, of heads 0-3)
                const int h0 = kPair ? 2 * (t & 1) : nt * 8 + 2 * t;
                if (h0 >= un.z) continue;
                float r[kHave][4];
#pragma unroll
                for (int mt = 0; mt < kHave; ++mt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float v = kPair && own ? o[nt][mt + MT - kHave][e] : o[nt][mt][e];
                        r[mt][e] = v + add[kPair ? 0 : mt / 4][e & 1];
                    }
                float* dst = p.part_o + slot * (NT * D * 8) + quads_of(nt);
                if (kLong && (put[nt][0] > 0.f || put[nt][1] > 0.f)) {
#pragma unroll
                    for (int mt = 0; mt < kHave; ++mt) {
                        const float4 was = __ldcg(reinterpret_cast<const float4*>(dst + mt * 128));
                        r[mt][0] = fmaf(was.x, put[nt][0], r[mt][0]);
                        r[mt][1] = fmaf(was.y, put[nt][1], r[mt][1]);
                        r[mt][2] = fmaf(was.z, put[nt][0], r[mt][2]);
                        r[mt][3] = fmaf(was.w, put[nt][1], r[mt][3]);
                    }
                }
                if (!whole) {  // 16 bytes of 8 x 2 channels and heads each
#pragma unroll
                    for (int mt = 0; mt < kHave; ++mt) {
                        const float4 v = make_float4(r[mt][0], r[mt][1], r[mt][2], r[mt][3]);
                        if (at_end)
                            *reinterpret_cast<float4*>(held + quads_of(nt) + mt * 128) = v;
                        else
                            __stcg(reinterpret_cast<float4*>(dst + mt * 128), v);
                    }
                    continue;
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    if (h0 + c >= un.z) continue;
                    const size_t at = (static_cast<size_t>(un.x) * p.Hq + un.y + h0 + c) * D + g +
                                      own * (kHave * 16);
#pragma unroll
                    for (int mt = 0; mt < kHave; ++mt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float v = r[mt][2 * e + c] * mul[c];
                            if constexpr (kF32)
                                static_cast<float*>(p.out)[at + mt * 16 + 8 * e] = v;
                            else
                                static_cast<__nv_bfloat16*>(p.out)[at + mt * 16 + 8 * e] =
                                    __float2bfloat16(v);
                        }
                }
            }
        }
        __syncwarp();
        if (i + S < n_mine) issue(s, i + S, S);
        queue >>= 1;
        if (++s == S) s = 0, phase ^= 1;
    }
    if (!kUnit && lost < n_mine) {
        for (int base = lost & ~31; base < n_mine; base += 32) {
            look_up(base);
            uint32_t ends = __ballot_sync(0xffffffffu, base + lane >= lost && (mine.y & 2));
            for (; ends; ends &= ends - 1) {
                const int k = __ffs(ends) - 1;
                const int unit = __shfl_sync(0xffffffffu, mine.x, k);
                const bool whole = from_start && (__shfl_sync(0xffffffffu, mine.y, k) & 8);
                from_start = true;  // (the next units begin in this warp's share)
                const int4 un = unit_of(unit);
                const size_t h0 = static_cast<size_t>(un.x) * p.Hq + un.y;
                if (whole) {
                    for (int e = lane; e < un.z * D; e += 32) {
                        if constexpr (kF32)
                            static_cast<float*>(p.out)[h0 * D + e] = kNan;
                        else
                            static_cast<__nv_bfloat16*>(p.out)[h0 * D + e] = __float2bfloat16(kNan);
                    }
                    if (p.lse_out && lane < un.z) p.lse_out[h0 + lane] = kNan;
                } else if (join && base + k == n_mine - 1) {
                    left = make_int2(unit, un.z);
                    if (lane < NT * 8) held_m[lane] = kNan;
                } else if (lane < NT * 8) {
                    __stcg(p.part_m + (static_cast<size_t>(me) + unit) * (NT * 8) + lane, kNan);
                }
            }
        }
    }
    if constexpr (kUnit) {
        // ---- join the cluster's pieces (one of each warp that has tiles): CTA `rank` takes its share
        // of the quads of O, groups of threads every groups-th piece, from all the cluster's shared
        // memories
        __syncwarp();
        if (cs > 1)
            cluster_sync();
        else
            __syncthreads();
        constexpr int kThreads = kWarps * 32;
        const int quads = NT * D * 2 / cs;  // this CTA's
        const int nq = min(quads, kThreads), groups = kThreads / nq;
        const int tid = static_cast<int>(threadIdx.x), grp = tid / nq;
        const int4 un = unit_of(my_unit);
        const int pieces = min(unit_tiles, kWarps * cs), log_cs = __ffs(cs) - 1;
        // (behind a warp's own piece its ring is free)
        constexpr int kScratch = (Cfg::kPieceFloats * 4 + 15) / 16 * 16;
        static_assert(kScratch + 1024 <= Cfg::kRing, "the ring holds a piece and 32 bytes a lane");
        float4* mem = reinterpret_cast<float4*>(smem + kScratch);
        auto cell = [&](int i) { return mem + i / 32 * (Cfg::kRing / 16) + i % 32 * 2; };
        static_assert(NT * D <= kThreads, "with several CTAs one pass takes all quads of one");
        for (int q0 = 0; q0 < quads; q0 += nq) {  // (16 heads of 128 channels and one CTA: twice)
            const int quad = rank * quads + q0 + tid % nq;
            const int h = quad / (D * 2) * 8 + 2 * (quad & 3);  // heads h and h + 1
            const bool mine_q = grp < groups && q0 + tid % nq < quads && h < un.z;
            float M0 = kNone, M1 = kNone, L0 = 0.f, L1 = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            // kAtOnce of this thread's pieces in flight: one round trip (16 x 4000 tokens, 16 heads on a KV
            // head, 12.1 us one after another, 11.4), but two where there are no more (60 tokens each:
            // 6.4 us, with eight 6.9)
            auto gather = [&](auto at_once) {
                constexpr int kAtOnce = decltype(at_once)::value;
                for (int i0 = grp; mine_q && i0 < pieces; i0 += groups * kAtOnce) {
                    float2 x[kAtOnce], y[kAtOnce];
                    float4 v[kAtOnce];
#pragma unroll
                    for (int k = 0; k < kAtOnce; ++k) {
                        const int i = i0 + k * groups;
                        x[k] = make_float2(kNone, kNone);
                        y[k] = make_float2(0.f, 0.f);
                        v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (i < pieces) {
                            const uint32_t at = map_peer(smem_u32(smem) + (i >> log_cs) * Cfg::kRing,
                                                         static_cast<uint32_t>(i & (cs - 1)));
                            x[k] = ld_cluster_v2(at + (NT * D * 8 + h) * 4);
                            y[k] = ld_cluster_v2(at + (NT * 8 * (D + 1) + h) * 4);
                            v[k] = ld_cluster_v4(at + quad * 16);
                        }
                    }
                    float t0 = M0, t1 = M1;
#pragma unroll
                    for (int k = 0; k < kAtOnce; ++k) t0 = fmaxf(t0, x[k].x), t1 = fmaxf(t1, x[k].y);
                    const float a0 = fast_exp2(M0 - t0), a1 = fast_exp2(M1 - t1);
                    M0 = t0, M1 = t1;
                    L0 *= a0, L1 *= a1;
                    acc.x *= a0, acc.z *= a0, acc.y *= a1, acc.w *= a1;
#pragma unroll
                    for (int k = 0; k < kAtOnce; ++k) {
                        const float w0 = fast_exp2(x[k].x - t0), w1 = fast_exp2(x[k].y - t1);
                        L0 = fmaf(w0, y[k].x, L0), L1 = fmaf(w1, y[k].y, L1);
                        acc.x = fmaf(w0, v[k].x, acc.x), acc.z = fmaf(w0, v[k].z, acc.z);
                        acc.y = fmaf(w1, v[k].y, acc.y), acc.w = fmaf(w1, v[k].w, acc.w);
                    }
                }
            };
            if (pieces <= groups * 2)
                gather(std::integral_constant<int, 2>{});
            else
                gather(std::integral_constant<int, 8>{});
            if (q0 > 0) __syncthreads();  // the cells of the pass before are read
            cell(tid)[0] = acc;
            cell(tid)[1] = make_float4(M0, M1, L0, L1);
            __syncthreads();
            // Nothing is read from the other CTAs any more (with several there is one pass): they may
            // leave once all have come here.
            if (cs > 1) cluster_arrive_relaxed();
            if (grp != 0 || !mine_q) continue;
            for (int k = 1; k < groups; ++k) {
                const float4 v = cell(tid + k * nq)[0], x = cell(tid + k * nq)[1];
                add_piece(M0, M1, L0, L1, acc, x.x, x.y, x.z, x.w, v);
            }
            const float r[4] = {acc.x, acc.y, acc.z, acc.w};
            const int ln = quad % 32, mt = quad / 32 % MT;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (h + c >= un.z) continue;
                const int hq = un.y + h + c;
                const float sig = p.sink_logit ? p.sink_logit[hq] * kLog2e : neg_inf();
                const float m_c = c ? M1 : M0, top = fmaxf(m_c, sig), w = fast_exp2(m_c - top);
                const float den = fmaf(c ? L1 : L0, w, p.sink_logit ? fast_exp2(sig - top) : 0.f);
                const size_t at =
                    (static_cast<size_t>(un.x) * p.Hq + hq) * D + mt * 16 + (ln >> 2);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    // nothing visible: zeros, and the logarithm of the sink's share alone
                    const float v = pieces == 0 ? 0.f : r[2 * e + c] * (w / den);
                    if constexpr (kF32)
                        static_cast<float*>(p.out)[at + 8 * e] = v;
                    else
                        static_cast<__nv_bfloat16*>(p.out)[at + 8 * e] = __float2bfloat16(v);
                }
                if (mt == 0 && ln < 4 && p.lse_out)
                    p.lse_out[static_cast<size_t>(un.x) * p.Hq + hq] =
                        pieces == 0 ? sig * kLn2 : (top + log2f(den)) * kLn2;
            }
        }
        __syncwarp();
        if (cs > 1) cluster_wait();  // no CTA leaves while another reads its shared memory
        return;
    }
    // ---- join the CTA's last pieces, warps of one unit at a time, into one partial each: a twelfth
    // of the workspace traffic, and one round trip of the joining launch, for long sequences
    if (!join) return;
    if (lane == 0) last_piece[warp] = left;
    __syncthreads();
    const int2 piece = lane < kWarps ? last_piece[lane] : make_int2(-1, 0);
    const int before = __shfl_up_sync(0xffffffffu, piece.x, 1);
    // bits of the warps that begin a run of one unit, bit kWarps behind the last
    uint32_t starts = __ballot_sync(
        0xffffffffu, lane == kWarps || (lane < kWarps && (lane == 0 || before != piece.x)));
    for (int a = 0; a < kWarps;) {
        starts &= starts - 1;
        const int b = __ffs(starts) - 1;
        const int unit = __shfl_sync(0xffffffffu, piece.x, a);
        const int heads = __shfl_sync(0xffffffffu, piece.y, a);
        const size_t slot = static_cast<size_t>(blockIdx.x * kWarps + a) + unit;
        for (int quad = threadIdx.x; quad < NT * D * 2 && unit >= 0; quad += kWarps * 32) {
            const int h = quad / (D * 2) * 8 + 2 * (quad & 3);  // heads h and h + 1
            if (h >= heads) continue;
            const float* held = reinterpret_cast<const float*>(smem);
            float M0 = kNone, M1 = kNone;
#pragma unroll 4
            for (int w = a; w < b; ++w) {
                const float2 x = *reinterpret_cast<const float2*>(
                    held + w * (Cfg::kRing / 4) + NT * D * 8 + h);
                M0 = fmaxf(M0, x.x), M1 = fmaxf(M1, x.y);
            }
            float L0 = 0.f, L1 = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int w = a; w < b; ++w) {
                const float* of = held + w * (Cfg::kRing / 4);
                const float2 x = *reinterpret_cast<const float2*>(of + NT * D * 8 + h);
                const float2 y = *reinterpret_cast<const float2*>(of + NT * 8 * (D + 1) + h);
                const float4 v = *reinterpret_cast<const float4*>(of + quad * 4);
                const float w0 = fast_exp2(x.x - M0), w1 = fast_exp2(x.y - M1);
                L0 = fmaf(w0, y.x, L0), L1 = fmaf(w1, y.y, L1);
                acc.x = fmaf(w0, v.x, acc.x), acc.z = fmaf(w0, v.z, acc.z);
                acc.y = fmaf(w1, v.y, acc.y), acc.w = fmaf(w1, v.w, acc.w);
            }
            __stcg(reinterpret_cast<float4*>(p.part_o + slot * (NT * D * 8)) + quad, acc);
            if (quad % (D * 2) < 4) {
                __stcg(reinterpret_cast<float2*>(p.part_m + slot * (NT * 8) + h), make_float2(M0, M1));
                __stcg(reinterpret_cast<float2*>(p.part_l + slot * (NT * 8) + h), make_float2(L0, L1));
            }
        }
        a = b;
    }
}

// Joins the partials of one unit's block of 8 heads: out = sum_i 2^{m_i - M} O_i / (sum_i 2^{m_i - M}
// l_i + 2^{sigma - M}). A partial is 8 D floats as the main launch's lanes hold them; a thread takes
// one quad of it (two channels of two heads) of every kSplit-th partial, kAtOnce of them in flight
// with their references and sums, so that few partials cost one round trip and no barrier. A CTA
// has all quads (kSplit = 1), or, where few units are cut into many partials each, 32 of them
// (kSplit = 8), so that enough SMs read. Units that one warp had whole are written already; units
// without tiles get zeros. What there is to join follows from the lengths alone and is worked out
// while the main launch ends.
template <int D, int NT, bool kF32, int kSplit, bool kJoin>
__global__ void __launch_bounds__(kSplit == 1 ? D * 2 : 32 * kSplit)
    gqa_q4_combine_kernel(const Q4Params p) {
    constexpr int kQuads = kSplit == 1 ? D * 2 : 32, kAtOnce = 4, H = NT * 8;
    constexpr int kParts = D * 2 / kQuads;  // CTAs of a unit's 8 heads
    const int unit = blockIdx.x, nt = blockIdx.y / kParts;
    const int b = unit / p.HU, u = unit % p.HU;
    const int kvh = u / p.NHG, hg = u % p.NHG;
    const int hq0 = kvh * p.G + hg * H + nt * 8, heads = min(8, p.G - hg * H - nt * 8);
    const int quad = threadIdx.x % kQuads + blockIdx.y % kParts * kQuads;
    const int k0 = threadIdx.x / kQuads;
    const int lane = threadIdx.x % 32, mt = quad / 32, g = lane >> 2, h = 2 * (lane & 3);
    // The unit's partials: of warps first .. last, or, where CTAs have joined their warps' last
    // pieces, of the first warp in each CTA, and the last warp's own if it went on to another unit.
    constexpr int kCta = warps_of(D, NT, kF32);
    int first = 0, last = 0, n = 0, joined = 0;
    bool whole = false;
    {
        uint32_t tiles = 0, before = 0;
        int own = 0;
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            int x, L;
            const int inc = scan_tiles(p, b0, lane, x, L);
            if (b >= b0 && b < b0 + 32) {
                own = __shfl_sync(0xffffffffu, x, b - b0);
                before = tiles + __shfl_sync(0xffffffffu, inc, b - b0) - own;
            }
            tiles += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (own > 0 && heads > 0) {
            const Shares<kCta> sh(p, tiles);
            const uint32_t t0 = before * p.HU + static_cast<uint32_t>(u) * own;
            const uint32_t t1 = t0 + own - 1;
            first = sh.owner(t0);
            last = sh.owner(t1);
            whole = first == last;  // one warp had it: written already
            n = last - first + 1;
            if (kJoin && sh.join) {
                const bool goes_on = t1 + 1 != sh.begin(last + 1);
                joined = (goes_on ? last - 1 : last) / kCta - first / kCta + 1;
                n = joined + goes_on;
            }
        }
    }
    // Every CTA waits, those with nothing to do as well: this grid must not end before the main one,
    // or what follows it in the stream could start while the main launch is still writing.
    griddep_wait();
    if (heads <= 0 || whole) return;
    const bool mine = h < heads, both = h + 1 < heads;
    float sig[2] = {neg_inf(), neg_inf()};
    if (p.sink_logit) {
        if (mine) sig[0] = p.sink_logit[hq0 + h] * kLog2e;
        if (both) sig[1] = p.sink_logit[hq0 + h + 1] * kLog2e;
    }
    float M[2] = {kNone, kNone}, L[2] = {0.f, 0.f};
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto slot_of = [&](int i) -> size_t {
        const int w = !kJoin || joined == 0 ? first + i
                      : i == 0    ? first
                      : i < joined ? (first / kCta + i) * kCta
                                   : last;
        return static_cast<size_t>(w) + unit;
    };
    const float* pm = p.part_m + nt * 8 + h;
    const float* pl = p.part_l + nt * 8 + h;
    const float* po = p.part_o + nt * (D * 8) + quad * 4;
    if (mine) {
        for (int i0 = k0; i0 < n; i0 += kSplit * kAtOnce) {
            float2 mi[kAtOnce], li[kAtOnce];
            float4 v[kAtOnce];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const int i = i0 + kSplit * k;
                mi[k] = make_float2(kNone, kNone);
                li[k] = make_float2(0.f, 0.f);
                v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i < n) {
                    const size_t slot = slot_of(i);
                    mi[k] = __ldcg(reinterpret_cast<const float2*>(pm + slot * H));
                    li[k] = __ldcg(reinterpret_cast<const float2*>(pl + slot * H));
                    v[k] = __ldcg(reinterpret_cast<const float4*>(po + slot * (D * H)));
                }
            }
            float t0 = M[0], t1 = M[1];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                t0 = fmaxf(t0, mi[k].x);
                t1 = both ? fmaxf(t1, mi[k].y) : t1;  // (a head that is not there holds anything)
            }
            const float a0 = fast_exp2(M[0] - t0), a1 = fast_exp2(M[1] - t1);
            M[0] = t0, M[1] = t1;
            L[0] *= a0, L[1] *= a1;
            acc.x *= a0, acc.z *= a0, acc.y *= a1, acc.w *= a1;
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const float w0 = fast_exp2(mi[k].x - t0), w1 = both ? fast_exp2(mi[k].y - t1) : 0.f;
                L[0] = fmaf(w0, li[k].x, L[0]);
                acc.x = fmaf(w0, v[k].x, acc.x);
                acc.z = fmaf(w0, v[k].z, acc.z);
                if (both) {
                    L[1] = fmaf(w1, li[k].y, L[1]);
                    acc.y = fmaf(w1, v[k].y, acc.y);
                    acc.w = fmaf(w1, v[k].w, acc.w);
                }
            }
        }
    }
    if constexpr (kSplit > 1) {
        __shared__ float4 s_o[kSplit][kQuads], s_ml[kSplit][kQuads];
        s_o[k0][lane] = acc;
        s_ml[k0][lane] = make_float4(M[0], M[1], L[0], L[1]);
        __syncthreads();
        if (k0 != 0) return;
        float t0 = kNone, t1 = kNone;
#pragma unroll
        for (int k = 0; k < kSplit; ++k) {
            t0 = fmaxf(t0, s_ml[k][lane].x);
            t1 = fmaxf(t1, s_ml[k][lane].y);
        }
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
        M[0] = t0, M[1] = t1, L[0] = L[1] = 0.f;
#pragma unroll
        for (int k = 0; k < kSplit; ++k) {
            const float4 a = s_ml[k][lane], v = s_o[k][lane];
            const float w0 = fast_exp2(a.x - t0), w1 = fast_exp2(a.y - t1);
            L[0] = fmaf(w0, a.z, L[0]), L[1] = fmaf(w1, a.w, L[1]);
            acc.x = fmaf(w0, v.x, acc.x), acc.z = fmaf(w0, v.z, acc.z);
            acc.y = fmaf(w1, v.y, acc.y), acc.w = fmaf(w1, v.w, acc.w);
        }
    }
    const float r[4] = {acc.x, acc.y, acc.z, acc.w};
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        if (h + c >= heads) continue;
        const int hq = hq0 + h + c;
        const float top = fmaxf(M[c], sig[c]), w = fast_exp2(M[c] - top);
        const float den = fmaf(L[c], w, p.sink_logit ? fast_exp2(sig[c] - top) : 0.f);
        const size_t at = (static_cast<size_t>(b) * p.Hq + hq) * D + mt * 16 + g;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            // nothing visible: zeros, and the logarithm of the sink's share alone
            const float v = n == 0 ? 0.f : r[2 * e + c] * (w / den);
            if constexpr (kF32)
                static_cast<float*>(p.out)[at + 8 * e] = v;
            else
                static_cast<__nv_bfloat16*>(p.out)[at + 8 * e] = __float2bfloat16(v);
        }
        if (mt == 0 && g == 0 && p.lse_out)
            p.lse_out[static_cast<size_t>(b) * p.Hq + hq] =
                n == 0 ? sig[c] * kLn2 : (top + log2f(den)) * kLn2;
    }
}

// A cluster for each unit, with as many CTAs as give each of an SM's four schedulers a warp: where
// all are resident at once (of 8 CTAs 15 clusters fit, of 4 36), no warp has more than four tiles
// (the list evens out lengths that differ) and no SM ten tiles of 8 heads more than the list would
// give it. 2 x 8192 tokens of 8 KV heads, clusters of 4, 18 more: 14.3 us, list 12.6;
// 1 x 8192, clusters of 8, 9 more: 11.2, list 12.2; 4 x 16384, 10.2 more: 24.1, list 23.0.
template <int NT>
bool unit_form(const Q4Plan& plan, int cs, int warps) {
    return cs > 0 && plan.most <= std::min(4.f * cs * warps, cs * (plan.even + 10.f / NT));
}

template <int D, int NT, bool kF32, bool kPair>
int launch_q4(const Q4Plan& plan, const Q4Params& p, cudaStream_t stream) {
    using Cfg = Q4Cfg<D, NT, kF32>;
    constexpr bool kDrifts = !kF32;
    auto kern = gqa_q4_kernel<D, NT, kF32, kPair, false, false>;
    auto long_kern = gqa_q4_kernel<D, NT, kF32, kPair, false, kDrifts>;
    auto unit_kern = gqa_q4_kernel<D, NT, kF32, kPair, true, false>;
    static int configured = 0;
    static int fits[9] = {};  // clusters of this size that are resident at once, plus 1
    if (!configured) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::kSmem) !=
                cudaSuccess ||
            cudaFuncSetAttribute(long_kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Cfg::kSmem) != cudaSuccess ||
            cudaFuncSetAttribute(unit_kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Cfg::kSmem) != cudaSuccess)
            return KVD_ERR_CUDA;
        configured = 1;
    }
    Q4Params up = p;
    for (int cs = plan.cluster; unit_form<NT>(plan, cs, Cfg::kWarps); cs /= 2) {
        if (fits[cs] == 0) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(plan.units * cs);
            cfg.blockDim = dim3(Cfg::kWarps * 32);
            cfg.dynamicSmemBytes = Cfg::kSmem;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = static_cast<unsigned>(cs);
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int n = 0;
            if (cudaOccupancyMaxActiveClusters(&n, unit_kern, &cfg) != cudaSuccess) n = 0;
            cudaGetLastError();
            fits[cs] = n + 1;
        }
        if (plan.units < fits[cs]) {
            up.cluster = cs;
            if (launch_kernel_cluster(unit_kern, dim3(plan.units * cs), dim3(Cfg::kWarps * 32),
                                      Cfg::kSmem, cs > 1 ? cs : 0, stream, up) != cudaSuccess)
                return KVD_ERR_CUDA;
            return cudaGetLastError() == cudaSuccess ? KVD_OK : KVD_ERR_CUDA;
        }
    }
    if (static_cast<long long>(plan.units) * plan.most > kPutBy * static_cast<long long>(plan.n_warps))
        kern = long_kern;
    if (launch_kernel(kern, dim3(plan.ctas), dim3(Cfg::kWarps * 32), Cfg::kSmem, stream, p) !=
        cudaSuccess)
        return KVD_ERR_CUDA;
    // Few units: many partials each, so more CTAs and threads join one. 16 units of 8192 tokens
    // 12.6 us (14.4 with a CTA each), of 32768 22.8 (25.0); 64 units of 4096 19.9 (18.3).
    const bool few = plan.n_warps > 48 * plan.units;
    const dim3 all(plan.units, NT), parts(plan.units, NT * (D / 16));
    const cudaError_t e =
        !plan.join
            ? launch_kernel(gqa_q4_combine_kernel<D, NT, kF32, 1, false>, all, dim3(D * 2), 0, stream, p)
        : few
            ? launch_kernel(gqa_q4_combine_kernel<D, NT, kF32, 8, true>, parts, dim3(256), 0, stream, p)
            : launch_kernel(gqa_q4_combine_kernel<D, NT, kF32, 1, true>, all, dim3(D * 2), 0, stream, p);
    if (e != cudaSuccess) return KVD_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? KVD_OK : KVD_ERR_CUDA;
}

}  // namespace

// The plan with blocks of at most 8 nt query heads of a KV head; one CTA on each SM, or as many as
// the longest possible list of tiles keeps busy. CTAs join their warps' pieces where a unit has at
// least four warps.
static int plan_heads(int nt, int B, int Hkv, int G, int D, long long max_len, int most, int dtype,
                      Q4Plan* plan) {
    plan->nt = nt;
    plan->NHG = (G + nt * 8 - 1) / (nt * 8);
    const long long units = static_cast<long long>(B) * Hkv * plan->NHG;
    const long long tiles = units * ((max_len + kTileTok - 1) / kTileTok + 1);
    if (tiles >= (1LL << 31)) return KVD_ERR_UNSUPPORTED;
    plan->units = static_cast<int>(units);
    const int warps = warps_of(D, nt, dtype == KVD_F32);
    plan->ctas = static_cast<int>(std::max(1LL, std::min<long long>(num_sms(), tiles)));
    plan->n_warps = plan->ctas * warps;
    plan->join = plan->n_warps >= 4 * units;
    plan->most = most;
    plan->even = static_cast<float>(units) * plan->most / num_sms();
    int cs = 1;
    while (cs < 8 && 2 * cs * units <= num_sms() && plan->most > 4 * cs) cs *= 2;
    plan->cluster = units <= num_sms() ? cs : 0;
    const size_t slots = static_cast<size_t>(plan->n_warps) + units;
    const size_t heads = static_cast<size_t>(nt) * 8;
    auto round = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
    plan->off_m = 0;
    plan->off_l = round(slots * heads * 4);
    plan->off_o = plan->off_l + round(slots * heads * 4);
    plan->total = plan->off_o + slots * heads * D * 4;
    return KVD_OK;
}

// 9 to 16 heads of a KV head share the decoding of their codes, but where a call is short, two
// blocks of 8 have more warps and shorter ones (16 heads, 2000 tokens 7.4 us, together 9.2), and
// with float32 queries of 128 channels 16 heads do not fit the registers (2 x 32768 tokens of 8 KV
// heads 49 us, together 50; 32 x 4096 of 4 49 and 52). The workspace is that of the larger plan.
int q4_plan(int B, int Hq, int Hkv, int D, long long max_len, int most, int dtype, Q4Plan* plan) {
    const int G = Hq / Hkv;
    const bool f32 = dtype == KVD_F32;
    const int st = plan_heads(1, B, Hkv, G, D, max_len, most, dtype, plan);
    if (st != KVD_OK || G <= 8 || (D == 128 && f32)) return st;
    Q4Plan both;  // (half the units: no more tiles than the plan above)
    plan_heads(2, B, Hkv, G, D, max_len, most, dtype, &both);
    const size_t total = std::max(plan->total, both.total);
    if (!unit_form<1>(*plan, plan->cluster, warps_of(D, 1, f32))) *plan = both;
    plan->total = total;
    return KVD_OK;
}

int q4_launch(const Q4Plan& plan, const Q4Params& args, int D, int dtype, cudaStream_t stream) {
    Q4Params p = args;
    // (in a test of the give-up path about a millisecond, longer than any copy takes: only the wait
    // that the test holds up runs out)
    p.wait_cycles = p.stall ? 2000000 : kWaitCycles;
    if (dtype == KVD_F32) {
        if (D == 128) return launch_q4<128, 1, true, false>(plan, p, stream);
        return plan.nt == 1 ? launch_q4<64, 1, true, false>(plan, p, stream)
                            : launch_q4<64, 2, true, false>(plan, p, stream);
    }
    if (D == 128) {
        if (p.G <= 4) return launch_q4<128, 1, false, true>(plan, p, stream);
        return plan.nt == 1 ? launch_q4<128, 1, false, false>(plan, p, stream)
                            : launch_q4<128, 2, false, false>(plan, p, stream);
    }
    return plan.nt == 1 ? launch_q4<64, 1, false, false>(plan, p, stream)
                        : launch_q4<64, 2, false, false>(plan, p, stream);
}

}  // namespace kvd
