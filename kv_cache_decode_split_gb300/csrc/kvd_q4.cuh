// kvd_q4.cuh -- the 4-bit cache: layout of a pool page and the rule that makes its codes.
//
// A pool is bytes [num_pages, Hkv, page_bytes]. A page is page_size / 16 blocks of 16 tokens; a
// block is 16 * D / 2 bytes of codes, then 16 * D / 64 pairs (scale, minimum) in float16,
// [token][group of 64 channels]. One bulk copy moves whole blocks, codes and scales together,
// and a warp's 16-token step of the attention reads exactly one block.
//   K  word [token r][t < 4][w < D/32]: code n < 8 is channel 32w + 8t + n, at bits 4n + 3 of the
//      word taken as a ring of 32 bits
//   V  token r = 8f + 2t + o: word [f][g < 8][t][o][w < 2] (D = 128), [g][t][f][o] (D = 64, w = 0):
//      code j < 8 is channel 64w + 8j + g, at bits 4j
// so that lane (g, t) of the attention's matrix instructions finds its fragments with 16-byte
// (or, for D = 64 keys, 8-byte) reads that touch every shared-memory bank once. Every word
// belongs to one token: appends of different tokens never share a word.
//
// A group's code is clamp(rint((x - b) * (1 / s)), 0, 15) with b = f16(min), s = f16((max - min)
// * f32(1/15)), every step rounded to float32 (x clamped to the float16 range first); it stands
// for s * code + b. A group that holds a NaN or an infinity has b = NaN and reads back as NaN.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

namespace kvd {

template <int D>
struct Q4 {
    static constexpr int kGroups = D / 64;                  // scale groups of a row
    static constexpr int kCodeBytes = 16 * D / 2;           // codes of a 16-token block
    static constexpr int kBlockBytes = kCodeBytes + 16 * kGroups * 4;
    // word index, inside a block, of the keys' codes of channels 8c .. 8c + 7 of token r
    __host__ __device__ static constexpr int k_word(int r, int c) {
        return (r * 4 + (c & 3)) * (D / 32) + (c >> 2);
    }
    // word index of the values' codes of channels 64w + 8j + g (j < 8) of token r
    __host__ __device__ static constexpr int v_word(int r, int g, int w) {
        return D == 128 ? ((((r >> 3) * 8 + g) * 4 + ((r >> 1) & 3)) * 2 + (r & 1)) * 2 + w
                        : ((g * 4 + ((r >> 1) & 3)) * 2 + (r >> 3)) * 2 + (r & 1);
    }
    // byte offset, inside a block, of the (scale, minimum) pair of token r's group
    __host__ __device__ static constexpr int param(int r, int grp) {
        return kCodeBytes + (r * kGroups + grp) * 4;
    }
};

}  // namespace kvd
