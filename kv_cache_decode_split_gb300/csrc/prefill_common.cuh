// prefill_common.cuh -- what the prefill attention kernels share: the work list and how CTAs cut it,
// the tiles that a unit walks, and the merge of units that a cut divides.
#pragma once

#include <algorithm>

#include "kvd_device.cuh"
#include "kvd_host.h"

namespace kvd {
namespace prefill {

constexpr int kM = 128;        // rows of a query tile
constexpr int kMaxCtas = 256;  // of the main launch
constexpr int kPieces = 4;     // ring of work descriptions
constexpr int kSlots = 3;      // partial results of a CTA: of its first and its last piece, and of a part
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;

// One piece of a unit: tiles [t0, t1) of its list.
struct Piece {
    int h;
    int c0, n, L;     // the sequence's first row, new tokens and keys
    int k0;           // its first key row (packed), or its sequence (paged)
    int tok0;         // the unit's first new token
    int nA, tB;       // the list: tiles 0 .. nA - 1, then from tB on
    int t0, t1, nt;   // nt: tiles of the whole unit; t0 < 0: no more pieces
    int slot;         // partial result, or -1: the piece is the whole unit
    int pair;         // two query tiles
};

struct Seq {
    int c0, n, L, k0;
};

// Sequence b; n = 0 where its offsets are bad. (b < B; every load is under way before the first is used)
static __device__ __noinline__ Seq load_seq(const PrefillParams& p, int b, int* err) {
    const bool paged = p.block_table != nullptr;
    const int32_t* keys = paged ? p.seq_lens : p.cu_k;
    Seq s;
    s.c0 = p.cu_q ? p.cu_q[b] : b;
    const int c1 = p.cu_q ? p.cu_q[b + 1] : b + 1;
    const int a = keys[b], k1 = keys[paged ? b : b + 1];
    bool bad = s.c0 < 0 || c1 < s.c0 || c1 > p.T || (b == 0 && s.c0 != 0);
    s.n = bad ? 0 : c1 - s.c0;
    if (paged) {
        s.L = min(max(a, 0), p.max_pages << p.page_shift);
        s.k0 = b;
        bad |= a != s.L || (s.L < s.n && p.cu_q);  // (without offsets: an empty sequence)
    } else {
        s.k0 = a;
        s.L = k1 - a;
        if (a < 0 || k1 < a || k1 > p.Tk || (b == 0 && a != 0)) {
            bad = true;
            s.n = 0;
        }
    }
    if (bad) record_error(err, KVD_ERR_DEVICE_OOB);
    return s;
}

// Length in the work list of a unit, and of a sequence's first m units (of one head): a fixed part and
// the keys up to the unit's last token, at most what a window leaves. (Only the balance depends on
// it. flat: every unit counts 1.)
struct Weigh {
    long long base, cap;
    int U, fixed, free;  // free: units before the window cuts their keys
    bool flat;
    __device__ __forceinline__ Weigh(const PrefillParams& p, const Seq& s, int u, bool f)
        : base(max(0, s.L - s.n)), cap(0), U(u), fixed(p.unit_cost), free(0x7fffffff), flat(f) {
        if (p.window > 0) {
            // (below 2^31 + 2^9: both of the first two may be 2^30)
            const unsigned c = static_cast<unsigned>(min(p.window, 1 << 30)) + U + 128 + min(p.n_sink, s.L) - 1;
            cap = c;
            free = c > base ? static_cast<int>(min((c - static_cast<unsigned>(base)) / U, 0x7fffffffu)) : 0;
        }
    }
    __device__ __noinline__ long long upto(int m) const {
        if (flat) return m;
        const long long m1 = min(m, free);
        return static_cast<long long>(m) * fixed + m1 * base + U * (m1 * (m1 + 1) / 2) + (m - m1) * cap;
    }
};

// The tiles that a unit walks: [0, nA) and nt - nA from tB on.
template <int kN>
__device__ __forceinline__ void unit_tiles(const PrefillParams& p, const Seq& s, int tok0, int U,
                                           int& nA, int& tB, int& nt) {
    const int first = s.L - s.n + tok0;                      // first and last position
    const int last = s.L - s.n + min(s.n, tok0 + U) - 1;
    nA = tB = nt = 0;
    if (last < 0) return;
    const int lo = p.window > 0 ? max(0, first - p.window + 1) / kN : 0;
    const int sink = p.window > 0 ? (min(p.n_sink, last + 1) + kN - 1) / kN : 0;
    nA = min(sink, lo);
    tB = lo;
    nt = nA + last / kN - lo + 1;
}

// The tiles at a mask's edge: some row of the unit does not see all of them. The mask is applied there,
// and their values are looked through.
template <int kN>
struct Edge {
    int from;          // tiles from here on reach past the first row's position
    int low, sink;     // tiles below `low` lie (in part) behind the last row's window, but those below
                       // `sink` hold sink tokens only
    __device__ __forceinline__ Edge(const PrefillParams& p, const Piece& u, int U) {
        const int first = u.L - u.n + u.tok0, last = u.L - u.n + min(u.n, u.tok0 + U) - 1;
        from = first < 0 ? 0 : (first + 1) / kN;
        low = p.window > 0 && last >= p.window ? (last - p.window) / kN + 1 : 0;
        sink = p.n_sink / kN;
    }
    __device__ __forceinline__ bool operator()(int tile) const {
        return tile >= from || (tile < low && tile >= sink);
    }
};

__device__ __forceinline__ int tile_of(const Piece& u, int t) {
    return t < u.nA ? t : u.tB + (t - u.nA);
}

// Values that are not finite are cleared in shared memory (a masked key's weight of zero would make NaN of
// them) and put back into the outputs of the rows that see them. Each piece has a word that says where: a
// bit for 1 << odd_shift() of its tiles.
__device__ __forceinline__ int odd_shift(const Piece& u) {
    return max(0, 27 - __clz(u.t1 - u.t0 - 1));
}

// Numbers of which the products' operands are made. (A float32 number goes in three bfloat16 parts, so what
// rounds to a bfloat16 infinity counts as infinite.)
__device__ __forceinline__ bool splits(float x) {
    return (__float_as_uint(x) & 0x7fffffffu) < 0x7f7f8000u;
}

// A lane's D / 32 columns of a value row.
template <int E>
__device__ __forceinline__ void get_row(const float* v, float (&x)[E]) {
    if (E == 4) {
        const float4 y = *reinterpret_cast<const float4*>(v);
        x[0] = y.x;
        x[1] = y.y;
        x[E - 2] = y.z;
        x[E - 1] = y.w;
    } else {
        const float2 y = *reinterpret_cast<const float2*>(v);
        x[0] = y.x;
        x[1] = y.y;
    }
}
template <int E>
__device__ __forceinline__ void get_row(const __nv_bfloat16* v, float (&x)[E]) {
#pragma unroll
    for (int e = 0; e < E; e += 2) {
        const uint32_t y = reinterpret_cast<const uint32_t*>(v)[e / 2];
        x[e] = __uint_as_float(y << 16);
        x[e + 1] = __uint_as_float(y & 0xffff0000u);
    }
}

// Puts back what was cleared into a warp's rows of outputs, one row a lane: dst, D numbers (half: bfloat16)
// of the row at position pos, valid or not. The marked tiles' values are read once more for all 32 rows, a
// lane taking columns of each key, and their signs collected, a bit a column, by the rows that see them:
// one infinity costs a row that sees it some hundred instructions and a read of a 32nd of its tiles.
template <int D, int kN, typename T, bool kEdgesOnly>
__device__ __forceinline__ void put_back(const PrefillParams& p, const Piece& pc, uint32_t marks, int U, bool valid,
                                      int pos, void* dst, bool half, int lane) {
    constexpr int E = D / 32, kBatch = 4;
    uint32_t up[E] = {}, down[E] = {};  // column i * E + e is bit i of word e; a NaN is in both
    const Edge<kN> edge(p, pc, U);
    const int shift = odd_shift(pc), top = __reduce_max_sync(0xffffffffu, valid ? pos : -1);
    bool full = false;  // all NaN: no more can come
#pragma unroll 1
    for (int t = pc.t0; t < pc.t1 && !full; ++t) {
        const int tile = tile_of(pc, t);
        if (!(marks >> ((t - pc.t0) >> shift) & 1) || (kEdgesOnly && !edge(tile))) continue;
        const int end = min(min(pc.L, top + 1), tile * kN + kN);
        auto row = [&](int key) -> const T* {
            const T* v = static_cast<const T*>(p.v) + lane * E;
            if (!p.block_table) return v + static_cast<long long>(pc.k0 + key) * p.v_stride + pc.h * D;
            const int pg =
                load_page(p.block_table, p.max_pages, p.num_pages, pc.k0, key >> p.page_shift, nullptr);
            return v + (((static_cast<size_t>(pg) * p.Hkv + pc.h) << p.page_shift) +
                        (key & ((1 << p.page_shift) - 1))) * D;
        };
#pragma unroll 1
        for (int k0 = tile * kN; k0 < end && !full; k0 += kBatch) {
            float x[kBatch][E];
            bool all = true;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) get_row(row(min(k0 + i, end - 1)), x[i]);
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
#pragma unroll
                for (int e = 0; e < E; ++e) all &= splits(x[i][e]);
            if (__all_sync(0xffffffffu, all)) continue;
#pragma unroll 1
            for (int key = k0; key < min(k0 + kBatch, end); ++key) {
                const bool sees =
                    valid && key <= pos && (p.window <= 0 || key > pos - p.window || key < p.n_sink);
                float y[E];
                get_row(row(key), y);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const uint32_t u = __ballot_sync(0xffffffffu, !splits(y[e]) && !(y[e] < 0.f));
                    const uint32_t d = __ballot_sync(0xffffffffu, !splits(y[e]) && !(y[e] > 0.f));
                    up[e] |= sees ? u : 0;
                    down[e] |= sees ? d : 0;
                }
            }
            uint32_t both = 0xffffffffu;
#pragma unroll
            for (int e = 0; e < E; ++e) both &= up[e] & down[e];
            full = __all_sync(0xffffffffu, !valid || both == 0xffffffffu);
        }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
#pragma unroll 1
        for (uint32_t left = up[e] | down[e]; left; left &= left - 1) {
            const int i = __ffs(left) - 1, col = i * E + e;
            const float x = (up[e] >> i & 1 ? INFINITY : 0.f) + (down[e] >> i & 1 ? -INFINITY : 0.f);
            if (half) {
                __nv_bfloat16* at = static_cast<__nv_bfloat16*>(dst) + col;
                *at = __float2bfloat16_rn(__bfloat162float(*at) + x);
            } else {
                static_cast<float*>(dst)[col] += x;
            }
        }
    }
    __syncwarp();
}
__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n)
                 : "memory");
}

// A bounded wait. (Code that a unit runs once is not in the instruction caches: it costs some 10 cycles an
// instruction, so that everything but the loops over tiles is kept short and rolled.)
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, const PrefillParams& p) {
    return mbar_wait(bar, parity, p.err, p.wait_cycles);
}
// For what is under way already: copies and products that must be complete before the CTA ends, also after a
// wait gave up.
__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity, const PrefillParams& p) {
    mbar_wait(bar, parity, p.err);
}
// The test of a wait that runs out: the role first waits for what nothing completes.
__device__ __forceinline__ bool stalls(const PrefillParams& p, uint64_t* never, int role) {
    return p.stall == role && !wait(never, 0, p);
}

// Registers of the executing warpgroup's threads, from the CTA's share at launch.
template <int N>
__device__ __forceinline__ void regs_more() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_fewer() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Two float32 operations in one instruction.
__device__ __forceinline__ uint64_t pair64(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair64(uint64_t v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// 16 columns of tensor memory, one lane a thread; the load's results are there behind the wait.
__device__ __forceinline__ void tmem_ld_x16(uint32_t t, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(t)
        : "memory");
}
__device__ __forceinline__ void tmem_st_x16(uint32_t t, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// Ranges: CTA c of n takes positions [range_start(c), range_start(c + 1)) of a list of length V. (No
// quotient: any rule will do that is the same for all CTAs and ascends from 0 to V.)
__device__ __forceinline__ long long range_start(const PrefillParams& p, long long V, int c) {
    return c >= p.n_cta ? V : static_cast<long long>(static_cast<double>(V) * (c * p.inv_cta));
}
// Tile at which offset y of a unit of length w and nt tiles cuts it.
template <int kN>
__device__ __forceinline__ int cut_tile(const PrefillParams& p, long long y, long long w, int nt) {
    if (y <= 0) return 0;
    if (y >= w) return nt;
    return static_cast<int>(min(static_cast<long long>(nt), max(0LL, (y - p.unit_cost) / kN)));
}

// Largest i in [0, n) with f(i) <= x, f ascending, f(0) <= x; by the warp, 32 at a time.
template <typename F>
__device__ __forceinline__ int last_below(int n, long long x, int lane, F&& f) {
    int lo = 0;
#pragma unroll 1
    while (n > 1) {
        const int step = (n + 31) / 32;
        const bool le = lane * step < n && f(lo + lane * step) <= x;
        const unsigned m = __ballot_sync(0xffffffffu, le);
        const int k = m ? 31 - __clz(m) : 0;
        lo += k * step;
        n = min(step, n - k * step);
    }
    return lo;
}

// Calls f(piece) for every piece of this CTA's range, in order, until it returns false: one warp, all
// lanes. U: tokens of a unit, TM: of a query tile.
template <int kN, typename F>
__device__ __forceinline__ void walk(const PrefillParams& p, int U, int TM, int lane, F&& f) {
    const int cta = blockIdx.x, n_cta = p.n_cta;
    if (lane == 0) p.head[cta].nt = 0;
    // how long the list is
    Seq mine{};             // of 32 sequences, one a lane
    long long my_head = 0;  // its length in the list, per head
    int my_units = 0;       // its units per head
    auto load_mine = [&](int b, int* err) {
        mine = b < p.B ? load_seq(p, b, err) : Seq{};
        my_units = (mine.n + U - 1) / U;
    };
    long long V = 0, units = 0, longest = 0;
#pragma unroll 1
    for (int b = lane; b < p.B; b += 32) {
        load_mine(b, cta == 0 ? p.err : nullptr);
        if (mine.n == 0) continue;
        const Weigh w(p, mine, U, false);
        my_head = w.upto(my_units);
        V += my_head * p.Hkv;
        units += static_cast<long long>(my_units) * p.Hkv;
        longest = max(longest, my_head - w.upto(my_units - 1));
    }
#pragma unroll 1
    for (int off = 16; off; off >>= 1) {
        V += __shfl_xor_sync(0xffffffffu, V, off);
        units += __shfl_xor_sync(0xffffffffu, units, off);
        longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, off));
    }
    // few short units: a CTA each, nothing is cut
    const bool flat = units <= n_cta && longest <= range_start(p, V, 1) + p.flat_slack;
    if (flat) V = units;
    const long long x0 = flat ? min(static_cast<long long>(cta), V) : range_start(p, V, cta);
    const long long x1 = flat ? min(cta + 1LL, V) : range_start(p, V, cta + 1);

    bool ok = true;
    // the sequence that position x0 falls in
    int b0 = 0;        // 32 sequences, one a lane
    long long at = 0;  // position of the first of them
    auto load_batch = [&]() {
        if (p.B > 32) {  // (up to 32 sequences are with their lanes)
            load_mine(b0 + lane, nullptr);
            my_head = Weigh(p, mine, U, flat).upto(my_units);
        } else if (flat) {
            my_head = my_units;
        }
    };
    int j = 32;
    if (x0 >= x1) return;
    bool first_seq = true;
#pragma unroll 1
    while (ok && at < x1) {
        if (j == 32) {  // the next 32 sequences; at first, those that x0 falls in
            if (b0 >= p.B) break;
            load_batch();
            j = 0;
            if (first_seq) {
                const long long my_len = my_head * p.Hkv;
                long long incl = my_len;
#pragma unroll 1
                for (int off = 1; off < 32; off <<= 1) {
                    const long long y = __shfl_up_sync(0xffffffffu, incl, off);
                    if (lane >= off) incl += y;
                }
                const unsigned m = __ballot_sync(0xffffffffu, at + incl > x0);
                if (!m) {
                    at += __shfl_sync(0xffffffffu, incl, 31);
                    b0 += 32;
                    j = 32;
                    continue;
                }
                j = __ffs(m) - 1;
                at += __shfl_sync(0xffffffffu, incl - my_len, j);
            }
        }
        Seq s;
        s.c0 = __shfl_sync(0xffffffffu, mine.c0, j);
        s.n = __shfl_sync(0xffffffffu, mine.n, j);
        s.L = __shfl_sync(0xffffffffu, mine.L, j);
        s.k0 = __shfl_sync(0xffffffffu, mine.k0, j);
        if (s.n > 0) {
            const int nm = (s.n + U - 1) / U;
            const Weigh wt(p, s, U, flat);
            const long long per_head = __shfl_sync(0xffffffffu, my_head, j);
            int h = 0, m = 0;
            long long u = at;  // position of the unit
            if (first_seq) {
                long long rem = x0 - at;
                h = last_below(p.Hkv, rem, lane, [&](int i) { return i * per_head; });
                rem -= h * per_head;
                m = last_below(nm, rem, lane, [&](int i) { return wt.upto(i); });
                u = at + h * per_head + wt.upto(m);
            }
#pragma unroll 1
            for (; h < p.Hkv && u < x1 && ok; ++h, m = 0) {
#pragma unroll 1
                for (; m < nm && u < x1 && ok; ++m) {
                    const long long w = wt.upto(m + 1) - wt.upto(m);
                    Piece pc;
                    pc.h = h;
                    pc.c0 = s.c0;
                    pc.n = s.n;
                    pc.L = s.L;
                    pc.k0 = s.k0;
                    pc.tok0 = m * U;
                    unit_tiles<kN>(p, s, pc.tok0, U, pc.nA, pc.tB, pc.nt);
                    pc.t0 = cut_tile<kN>(p, x0 - u, w, pc.nt);
                    pc.t1 = cut_tile<kN>(p, x1 - u, w, pc.nt);
                    pc.pair = U > TM && s.n - pc.tok0 > TM;
                    const bool whole = pc.t0 == 0 && pc.t1 == pc.nt;
                    pc.slot = whole ? -1 : 2 * cta + (pc.t0 == 0 ? 1 : 0);
                    const long long start = u;
                    u += w;
                    if (pc.nt == 0 ? start < x0 : pc.t0 == pc.t1) continue;
                    if (lane == 0 && !whole && pc.t0 == 0) {
                        // the unit's first piece: what the merge needs to know
                        PrefillHead& hd = p.head[cta];
                        hd.c0 = pc.c0;
                        hd.n = pc.n;
                        hd.h = h;
                        hd.tok0 = pc.tok0;
                        hd.tiles = pc.pair ? 2 : 1;
                        hd.u = start;
                        hd.w = w;
                        hd.V = V;
                        hd.nt = pc.nt;
                    }
                    ok = f(pc);
                }
            }
        }
        first_seq = false;
        at += __shfl_sync(0xffffffffu, my_head, j) * p.Hkv;
        if (++j == 32) b0 += 32;
    }
}

// A lane's E columns of a row.
template <int E>
__device__ __forceinline__ void put_row(__nv_bfloat16* dst, const float (&o)[E]) {
    if (E == 4)
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16(o[0], o[1]), pack_bf16(o[E - 2], o[E - 1]));
    else
        *reinterpret_cast<uint32_t*>(dst) = pack_bf16(o[0], o[1]);
}
template <int E>
__device__ __forceinline__ void put_row(float* dst, const float (&o)[E]) {
    if (E == 4)
        *reinterpret_cast<float4*>(dst) = make_float4(o[0], o[1], o[E - 2], o[E - 1]);
    else
        *reinterpret_cast<float2*>(dst) = make_float2(o[0], o[1]);
}

// Merges the pieces of the unit whose first piece CTA x of the main launch took, in their order: a warp
// a row, its lanes over the pieces for the weights and over the columns for the sums.
template <int D, typename T, int kN>
__global__ void __launch_bounds__(128) prefill_merge_kernel(const PrefillParams p) {
    __shared__ int slots[kMaxCtas + 1];
    __shared__ int n_slots;
    griddep_wait();
    const PrefillHead hd = p.head[blockIdx.x];
    if (hd.nt == 0) return;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (warp == 0) {
        // CTAs from x on whose range holds a tile of the unit
        int n = 0;
        for (int c0 = blockIdx.x; c0 < p.n_cta; c0 += 32) {
            const int c = c0 + lane;
            bool has = false, past = true;
            if (c < p.n_cta) {
                const long long a = range_start(p, hd.V, c) - hd.u, b = range_start(p, hd.V, c + 1) - hd.u;
                has = cut_tile<kN>(p, a, hd.w, hd.nt) < cut_tile<kN>(p, b, hd.w, hd.nt);
                past = b >= hd.w;
            }
            const unsigned m = __ballot_sync(0xffffffffu, has);
            if (has) slots[n + __popc(m & ((1u << lane) - 1))] = 2 * c + (c == static_cast<int>(blockIdx.x));
            n += __popc(m);
            if (__any_sync(0xffffffffu, past)) break;
        }
        if (lane == 0) n_slots = n;
    }
    __syncthreads();
    const int n = n_slots;
    const int TM = kM / p.G;
    // (a unit of one query tile leaves the second tile's rows out: their tokens are not its own)
    const int rows = hd.tiles * kM;
    constexpr int E = D / 32;
    for (int r = blockIdx.y * 4 + warp; r < rows; r += gridDim.y * 4) {
        const int t = r % kM / p.G, token = hd.tok0 + (r / kM) * TM + t;
        if (t >= TM || token >= hd.n) continue;
        const int head = hd.h * p.G + (r % kM - t * p.G);
        // the row's maximum, sink included
        const float sink = p.sink_logit ? p.sink_logit[head] * kLog2e : -INFINITY;
        const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
        float top = -INFINITY;
        for (int i = lane; i < n; i += 32) top = fmaxf(top, ml[static_cast<size_t>(slots[i]) * 2 * kM + r].x);
#pragma unroll
        for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
        top = fmaxf(top, sink);
        float sum = 0.f, o[E];
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = 0.f;
        for (int i0 = 0; i0 < n; i0 += 32) {
            float f = 0.f;
            if (i0 + lane < n) {
                const float2 v = ml[static_cast<size_t>(slots[i0 + lane]) * 2 * kM + r];
                // (a piece without a maximum: nothing seen, or all of it NaN)
                f = v.x == -INFINITY ? 1.f : fast_exp2(v.x - top);
                sum += v.y * f;
            }
            const int m = min(32, n - i0);
#pragma unroll 4
            for (int i = 0; i < m; ++i) {
                const float g = __shfl_sync(0xffffffffu, f, i);
                const float* src = p.part_o + (static_cast<size_t>(slots[i0 + i]) * 2 * kM + r) * D + lane * E;
                if (E == 4) {
                    const float4 v = *reinterpret_cast<const float4*>(src);
                    o[0] = fmaf(v.x, g, o[0]);
                    o[1] = fmaf(v.y, g, o[1]);
                    o[E - 2] = fmaf(v.z, g, o[E - 2]);
                    o[E - 1] = fmaf(v.w, g, o[E - 1]);
                } else {
                    const float2 v = *reinterpret_cast<const float2*>(src);
                    o[0] = fmaf(v.x, g, o[0]);
                    o[1] = fmaf(v.y, g, o[1]);
                }
            }
        }
#pragma unroll
        for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (sink != -INFINITY) sum += fast_exp2(sink - top);
        const float scale = sum == 0.f ? 0.f : 1.f / sum;
        const long long row = static_cast<long long>(hd.c0 + token) * p.Hq + head;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] *= scale;
        put_row<E>(static_cast<T*>(p.out) + row * D + lane * E, o);
        if (p.lse_out && lane == 0)
            p.lse_out[row] = sum == 0.f ? -INFINITY
                                        : ((top == -INFINITY ? 0.f : top) + log2f(sum)) * kLn2;
    }
}

// Adds a part of a piece, which lies in slot `from`, to the parts before it (first: there are none), or ends the
// piece (last): one row a thread, r of each query tile, which it has written. A whole unit's parts are added up
// in the slot of the CTA's last piece, which comes behind it.
template <int D, typename T>
__device__ __forceinline__ void add_part(const PrefillParams& p, const Piece& pc, int from, bool first, bool last,
                                         int r) {
    const int TM = kM / p.G, t = r / p.G, head = pc.h * p.G + (r - t * p.G);
    float2* ml = reinterpret_cast<float2*>(p.part_ml);
#pragma unroll 1
    for (int w = 0; w <= pc.pair; ++w) {
        const int token = pc.tok0 + w * TM + t;
        if (t >= TM || token >= pc.n) continue;
        const long long own = (static_cast<long long>(from) * 2 + w) * kM + r;
        const long long sum_at =
            (static_cast<long long>(pc.slot < 0 ? 2 * blockIdx.x + 1 : pc.slot) * 2 + w) * kM + r;
        float top = ml[own].x, sum = ml[own].y, f = 1.f, fp = 0.f;
        if (!first) {
            const float2 was = ml[sum_at];
            const float both = fmaxf(top, was.x);
            // (a part without a maximum: nothing seen, or all of it NaN)
            f = top == -INFINITY ? 1.f : fast_exp2(top - both);
            fp = was.x == -INFINITY ? 1.f : fast_exp2(was.x - both);
            sum = sum * f + was.y * fp;
            top = both;
        }
        const long long row = static_cast<long long>(pc.c0 + token) * p.Hq + head;
        const bool done = last && pc.slot < 0;
        if (done) {
            float scale = 1.f;
            if (p.sink_logit) {
                const float sink = p.sink_logit[head] * kLog2e, ref = fmaxf(top, sink);
                scale = top == -INFINITY ? 1.f : fast_exp2(top - ref);
                sum = sum * scale + (sink == -INFINITY ? 0.f : fast_exp2(sink - ref));
                top = ref;
            }
            scale = sum == 0.f ? 0.f : scale / sum;
            f *= scale;
            fp *= scale;
            if (p.lse_out)
                p.lse_out[row] = sum == 0.f ? -INFINITY : ((top == -INFINITY ? 0.f : top) + log2f(sum)) * kLn2;
        } else {
            ml[sum_at] = make_float2(top, sum);
        }
#pragma unroll 1
        for (int col = 0; col < D; col += 4) {
            const float4 x = *reinterpret_cast<const float4*>(p.part_o + own * D + col);
            float o[4] = {x.x * f, x.y * f, x.z * f, x.w * f};
            float* at = p.part_o + sum_at * D + col;
            if (fp != 0.f) {
                const float4 y = *reinterpret_cast<const float4*>(at);
                o[0] = fmaf(y.x, fp, o[0]);
                o[1] = fmaf(y.y, fp, o[1]);
                o[2] = fmaf(y.z, fp, o[2]);
                o[3] = fmaf(y.w, fp, o[3]);
            }
            if (done)
                put_row<4>(static_cast<T*>(p.out) + row * D + col, o);
            else
                put_row<4>(at, o);
        }
    }
}

constexpr int kMergeRows = 8;  // blocks of a unit

inline int ctas() { return std::min(num_sms(), kMaxCtas); }

struct Plan {
    size_t off_ml, off_o, total;
};
inline Plan make_plan(int D) {
    const size_t n = static_cast<size_t>(ctas());
    Plan pl;
    pl.off_ml = (n * sizeof(PrefillHead) + 255) & ~static_cast<size_t>(255);
    pl.off_o = pl.off_ml + n * kSlots * 2 * kM * 8;
    pl.total = pl.off_o + n * kSlots * 2 * kM * D * 4;
    return pl;
}

// Launches the merge of a call whose main launch has been issued, unless none of its units can have been
// cut: there are few, and no unit walks many keys. U: tokens of a unit.
template <int D, typename T, int kN>
inline cudaError_t launch_merge(const PrefillParams& p, int U, cudaStream_t stream) {
    const long long units = static_cast<long long>(p.Hkv) * (p.T / U + std::min(p.B, p.T));
    // (a unit's length in the list: of the keys, or, with fewer keys than new tokens, of those)
    long long most = std::max<long long>(
        p.block_table ? static_cast<long long>(p.max_pages) << p.page_shift : p.Tk, p.T);
    if (p.window > 0) most = std::min(most, static_cast<long long>(p.window) + p.n_sink + 128);
    if (units <= p.n_cta && most + U + p.unit_cost <= p.flat_slack) return cudaSuccess;
    return launch_kernel(prefill_merge_kernel<D, T, kN>, dim3(static_cast<unsigned>(p.n_cta), kMergeRows),
                         dim3(128), 0, stream, p);
}

// The call's part of the parameters: workspace and how work is cut.
inline void set_plan(PrefillParams& p, int D, void* ws, int unit_cost, int flat_slack) {
    // A wait may be as long as the four pieces that are under way, of some 100 cycles a key and four times that
    // with values that are not finite in each tile, or as the look through all sequences' lengths.
    const long long keys = p.block_table ? static_cast<long long>(p.max_pages) << p.page_shift : p.Tk;
    p.wait_cycles = p.stall ? 4000000 : kWaitCycles + 4096 * keys + 256LL * p.B;
    const Plan pl = make_plan(D);
    uint8_t* base = static_cast<uint8_t*>(ws);
    p.head = reinterpret_cast<PrefillHead*>(base);
    p.part_ml = reinterpret_cast<float*>(base + pl.off_ml);
    p.part_o = reinterpret_cast<float*>(base + pl.off_o);
    p.n_cta = ctas();
    p.inv_cta = 1.0 / p.n_cta;
    p.unit_cost = unit_cost;
    p.flat_slack = flat_slack;
}

}  // namespace prefill
}  // namespace kvd
