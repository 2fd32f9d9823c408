// cache_read.cu -- what a paged, rolling or 4-bit cache holds, as packed rows.
//
// What is computed: the inverse of the appends. A sequence of length L holds positions 0 .. L - 1
// (paged), or, rolling, its first n_sink and its last W; row cu_seqlens[b] + j receives the j-th of
// them in the order of positions. Plain rows are copied as bytes; a 4-bit group of 64 channels is
// s * code + b (one multiply-add in float32: a code has 4 bits, s 11, so the product is exact),
// rounded once to the output's type.
//
// GB300: a stream. One warp takes the 16 slots of one block of a page for one head and one pool:
// their rows lie together (2 to 8 KB; 4 bits: one block of codes and its scales), so that each lane
// has all of its loads in flight at once, and the page is looked up once. Warps find their sequence
// without a scan: block k of sequence b is item cu[b] / 16 + b + k, which is unique and ascending, so
// a 32-way search over b (one round of loads up to 32 sequences, two up to 1024) inverts it.
//
// Bound by the bytes written, of which every SM can hand on 32 a cycle: 4 bits to bf16, 41,000 tokens of 8
// heads of 128 (48 MB read, 171 MB written) take 45.6 us, 4.8 TB/s, with that path busy 68 % of the time. But
// nearly half of what is on it is a copy of the arguments, which each thread writes to its stack, as they are
// indexed at run time: without it the same call takes 36.1 us, which is left for a change of its own. (Whole
// rows at a time for the keys as well, or codes turned to numbers without a conversion, did not change the
// time.) Plain rows of as many tokens 53.9 us, 6.3 TB/s. A short call, four contexts of 33 to 700 tokens,
// takes 3.5 us: four dependent reads (the search, offsets and length, the page, the rows).

#include <algorithm>

#include "kvd_device.cuh"
#include "kvd_host.h"
#include "kvd_q4.cuh"

namespace kvd {

namespace {

constexpr int kReadWarps = 8;

// The slots of one 16-slot block and where their tokens go.
struct ReadBlock {
    int held;        // tokens that the cache holds of the sequence
    int slot0;       // first slot of the block
    long long row0;  // first row of the sequence
    int first;       // rolling: window offset of the oldest token's slot
    int page;        // -1: nothing to read
};

// Row of the token in `slot`, -1 if there is none.
__device__ __forceinline__ long long row_of(const CacheReadParams& p, const ReadBlock& k, int slot) {
    int j = slot;
    if (p.window > 0 && slot >= p.n_sink) {
        j = slot - p.n_sink - k.first;
        j = p.n_sink + (j < 0 ? j + p.window : j);
        if (slot >= p.n_sink + p.window) return -1;
    }
    return j < k.held ? k.row0 + j : -1;
}

__device__ __forceinline__ ReadBlock find_block(const CacheReadParams& p, int item, int lane) {
    // largest b with cu[b] / 16 + b <= item, of those up to which offsets ascend: a sequence behind a bad offset
    // is given no block, so that it takes none of a sequence in front of it. (Of more than 32 sequences the
    // first round looks at every so many.)
    int lo = 0, n = p.B;  // the answer is in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int b = lo + lane * step;
        const int c = lane * step < n ? p.cu_seqlens[b] : 0, before = __shfl_up_sync(0xffffffffu, c, 1);
        const bool le = lane * step < n && (lane == 0 || c >= before) && (c >> 4) + b <= item;
        const unsigned m = __ballot_sync(0xffffffffu, le);
        const int k = max(__ffs(~m) - 2, m == 0xffffffffu ? 31 : 0);
        lo += k * step;
        n = min(step, n - k * step);
    }
    ReadBlock r;
    r.page = -1;
    const int c0 = p.cu_seqlens[lo], c1 = p.cu_seqlens[lo + 1];
    const int L = p.seq_lens[lo];
    if (c0 < 0 || c1 < c0 || c1 > p.T || (lo == 0 && c0 != 0)) return r;  // (recorded by the grid's first block)
    const long long cap = p.window > 0 ? static_cast<long long>(p.n_sink) + p.window
                                       : static_cast<long long>(p.max_pages) << p.page_shift;
    if (L < 0 || (p.window <= 0 && L > cap)) return r;
    r.first = p.window > 0 && L > cap ? static_cast<int>((L - cap) % p.window) : 0;
    r.held = static_cast<int>(min(static_cast<long long>(L), cap));
    r.slot0 = (item - ((c0 >> 4) + lo)) * 16;
    r.row0 = c0;
    if (r.slot0 < 0 || r.slot0 >= r.held || r.held > c1 - c0) return r;
    const int pg = p.block_table[static_cast<size_t>(lo) * p.max_pages +
                                 (r.slot0 >> p.page_shift)];
    if (pg < 0 || pg >= p.num_pages) {
        if (lane == 0) record_error(p.err, KVD_ERR_DEVICE_OOB);
        return r;
    }
    r.page = pg;
    return r;
}

// Offsets that do not ascend and lengths out of range, looked at once for every sequence.
__device__ __forceinline__ void check_sequences(const CacheReadParams& p) {
    const long long cap = p.window > 0 ? static_cast<long long>(p.n_sink) + p.window
                                       : static_cast<long long>(p.max_pages) << p.page_shift;
    for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
        const int c0 = p.cu_seqlens[b], c1 = p.cu_seqlens[b + 1], L = p.seq_lens[b];
        if (c0 < 0 || c1 < c0 || c1 > p.T || (b == 0 && c0 != 0) || L < 0 ||
            (p.window <= 0 && L > cap) || min(static_cast<long long>(L), cap) > c1 - c0)
            record_error(p.err, KVD_ERR_DEVICE_OOB);
    }
}

// kRow: 16-byte pieces of a row (D * element size / 16): 8, 16 or 32
template <int kRow>
__global__ void __launch_bounds__(kReadWarps * 32) cache_read_kernel(const CacheReadParams p) {
    griddep_wait();
    if (blockIdx.x == 0 && blockIdx.y == 0) check_sequences(p);
    const int lane = threadIdx.x % 32;
    const int unit = blockIdx.y * kReadWarps + threadIdx.x / 32;  // (pool, head)
    if (unit >= 2 * p.Hkv) return;
    const int h = unit >> 1, which = unit & 1;
    const ReadBlock k = find_block(p, blockIdx.x, lane);
    if (k.page < 0) return;
    const int off = k.slot0 & ((1 << p.page_shift) - 1);
    const uint4* src = static_cast<const uint4*>(p.pool[which]) +
                       (((static_cast<size_t>(k.page) * p.Hkv + h) << p.page_shift) + off) * kRow;
    constexpr int kLoads = 16 * kRow / 32;
    uint4 v[kLoads];
    long long row[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int at = i * 32 + lane;
        row[i] = row_of(p, k, k.slot0 + at / kRow);
        if (row[i] >= 0) v[i] = __ldcs(src + at);
    }
    uint4* dst = static_cast<uint4*>(p.out[which]);
    const long long stride = p.stride[which];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int c = (i * 32 + lane) % kRow;
        if (row[i] >= 0) dst[row[i] * stride + h * kRow + c] = v[i];
    }
}

// Eight consecutive channels, rounded to the output's type.
__device__ __forceinline__ void put8(__nv_bfloat16* dst, const float (&x)[8]) {
    uint4 v;
    v.x = pack_bf16(x[0], x[1]);
    v.y = pack_bf16(x[2], x[3]);
    v.z = pack_bf16(x[4], x[5]);
    v.w = pack_bf16(x[6], x[7]);
    *reinterpret_cast<uint4*>(dst) = v;
}
__device__ __forceinline__ void put8(float* dst, const float (&x)[8]) {
    reinterpret_cast<float4*>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

template <int D, typename T>
__global__ void __launch_bounds__(kReadWarps * 32) cache_read_q4_kernel(const CacheReadParams p) {
    griddep_wait();
    if (blockIdx.x == 0 && blockIdx.y == 0) check_sequences(p);
    const int lane = threadIdx.x % 32;
    const int unit = blockIdx.y * kReadWarps + threadIdx.x / 32;
    if (unit >= 2 * p.Hkv) return;
    const int h = unit >> 1, which = unit & 1;
    const ReadBlock k = find_block(p, blockIdx.x, lane);
    if (k.page < 0) return;
    using L = Q4<D>;
    const int blk = (k.slot0 & ((1 << p.page_shift) - 1)) / 16;
    const uint8_t* src = static_cast<const uint8_t*>(p.pool[which]) +
                         ((static_cast<size_t>(k.page) * p.Hkv + h) * ((1 << p.page_shift) / 16) +
                          blk) * L::kBlockBytes;
    const uint32_t* code = reinterpret_cast<const uint32_t*>(src);
    T* dst = static_cast<T*>(p.out[which]);
    const long long stride = p.stride[which];
    auto param = [&](int r, int grp) {
        return __half22float2(*reinterpret_cast<const __half2*>(src + L::param(r, grp)));
    };
    if (which == 0) {
        // keys: a lane takes eighth t of a token's words, 8 channels each
        constexpr int kW = D / 32;
        uint32_t w[2][kW];
        float2 sb[2][D / 64];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = i * 8 + lane / 4, t = lane % 4;
#pragma unroll
            for (int c = 0; c < kW; ++c) w[i][c] = code[L::k_word(r, c * 4 + t)];
#pragma unroll
            for (int g = 0; g < D / 64; ++g) sb[i][g] = param(r, g);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = i * 8 + lane / 4, t = lane % 4;
            const long long row = row_of(p, k, k.slot0 + r);
            if (row < 0) continue;
#pragma unroll
            for (int c = 0; c < kW; ++c) {
                const uint32_t x = __funnelshift_r(w[i][c], w[i][c], 3);
                float y[8];
#pragma unroll
                for (int n = 0; n < 8; ++n)
                    y[n] = fmaf(static_cast<float>((x >> (4 * n)) & 15u), sb[i][c / 2].x, sb[i][c / 2].y);
                put8(dst + row * stride + h * D + 32 * c + 8 * t, y);
            }
        }
    } else {
        // values: the 64 channels of a token's group lie in eight words, 8 channels 8j .. 8j + 7 in their
        // codes j. So the words go through shared memory: eight lanes take the group and write its 128
        // (float32: 256) bytes together. (A lane that takes a group alone writes 16 bytes of 32 lines at
        // a time: nine contexts of 1001 to 8191 tokens, 8 KV heads of 128, take 5 us more.)
        constexpr int kRows = 16 * L::kGroups, kPer = 8 * kRows / 32;  // groups; words that a lane fetches
        struct __align__(16) Group {
            uint32_t w[8];
            float2 sb;
            uint32_t pad[2];  // (rows 48 bytes apart: eight lanes' 16 bytes lie in different banks)
        };
        __shared__ Group groups[kReadWarps][kRows];
        Group* mine = groups[threadIdx.x / 32];
        {
            const int i = lane % kRows, r = i / L::kGroups, grp = i % L::kGroups, g0 = lane / kRows * kPer;
            uint32_t w[kPer];
#pragma unroll
            for (int g = 0; g < kPer; ++g) w[g] = code[L::v_word(r, g0 + g, grp)];
            const float2 sb = param(r, grp);
#pragma unroll
            for (int g = 0; g < kPer; g += 4)
                *reinterpret_cast<uint4*>(&mine[i].w[g0 + g]) = make_uint4(w[g], w[g + 1], w[g + 2], w[g + 3]);
            if (g0 == 0) mine[i].sb = sb;
        }
        __syncwarp();
        const int j = lane % 8;
#pragma unroll
        for (int i0 = 0; i0 < kRows; i0 += 4) {
            const int i = i0 + lane / 8, r = i / L::kGroups, grp = i % L::kGroups;
            const long long row = row_of(p, k, k.slot0 + r);
            if (row < 0) continue;
            const uint4 lo = *reinterpret_cast<const uint4*>(&mine[i].w[0]);
            const uint4 hi = *reinterpret_cast<const uint4*>(&mine[i].w[4]);
            const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
            const float2 sb = mine[i].sb;
            float y[8];
#pragma unroll
            for (int g = 0; g < 8; ++g)
                y[g] = fmaf(static_cast<float>((w[g] >> (4 * j)) & 15u), sb.x, sb.y);
            put8(dst + row * stride + h * D + 64 * grp + 8 * j, y);
        }
    }
}

}  // namespace

int cache_read_launch(const CacheReadParams& p, bool q4, int D, int dtype, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>(p.T / 16 + p.B),
                    static_cast<unsigned>((2 * p.Hkv + kReadWarps - 1) / kReadWarps));
    const dim3 block(kReadWarps * 32);
    cudaError_t e;
    if (q4) {
        if (dtype == KVD_F32)
            e = D == 64 ? launch_kernel(cache_read_q4_kernel<64, float>, grid, block, 0, stream, p)
                        : launch_kernel(cache_read_q4_kernel<128, float>, grid, block, 0, stream, p);
        else
            e = D == 64 ? launch_kernel(cache_read_q4_kernel<64, __nv_bfloat16>, grid, block, 0, stream, p)
                        : launch_kernel(cache_read_q4_kernel<128, __nv_bfloat16>, grid, block, 0, stream, p);
    } else {
        const int row = D * (dtype == KVD_F32 ? 4 : 2) / 16;
        e = row == 8    ? launch_kernel(cache_read_kernel<8>, grid, block, 0, stream, p)
            : row == 16 ? launch_kernel(cache_read_kernel<16>, grid, block, 0, stream, p)
                        : launch_kernel(cache_read_kernel<32>, grid, block, 0, stream, p);
    }
    if (e != cudaSuccess) return KVD_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? KVD_OK : KVD_ERR_CUDA;
}

}  // namespace kvd
