// The 4-bit record of one 64-token chunk of one KV head, and how its codes are read.
//
// A record is 72 D bytes, K then V:
//   K codes  uint32 [64 tokens][D / 8], word w of a token: channels 8w .. 8w + 7
//   K grid   bf16 s[D], z[D]                    one pair per channel (64 tokens)
//   V codes  uint32 [D channels][8], word w of a channel: tokens 8w .. 8w + 7
//   V grid   bf16 s[D / 64][64], z[D / 64][64]  one pair per token and 64 channels
// Nibble j < 4 of a word is its element 2j, nibble 4 + j its element 2j + 1.  Code c
// stands for the bf16 value bf16(s (16 + c) + z), one rounding.
//
// Why this form: bf16 16 + c is 0x4180 with c in mantissa bits 3-6, so one shift and one
// three-input logic op give a pair of them and one bf16x2 FMA the pair of values -- the
// values of the definition bit for bit, 12 operations per 8 codes.  A pair runs along
// the channels in K and along the tokens in V, the directions that the two products of
// the attention contract, so a pair is a register of an MMA operand.  Keys share a grid
// along the tokens because a channel's offset and range persist over a chunk; values
// have no such axis and share one along 64 channels of a token.
#pragma once

#include "common.cuh"

namespace hga {

template <int D> struct Packed {
    static constexpr int kCodes = 32 * D;       // bytes of the K (or V) codes
    static constexpr int kGridOff = kCodes;     // s, then z kGridHalf bytes behind it
    static constexpr int kGridHalf = 2 * D;
    static constexpr int kPart = 36 * D;        // K part; V part behind it
    static constexpr int kRecord = 72 * D;
};

// s (16 + c) + z of pair J of a word (elements 2J, 2J + 1), bf16x2; s and z hold the
// two elements' grids.
template <int J> __device__ __forceinline__ uint32_t packed_pair(uint32_t w, uint32_t s, uint32_t z) {
    const uint32_t sh = J == 0 ? w << 3 : w >> (4 * J - 3);
    uint32_t m, r;
    // (sh & mask) | 16.0 pair: one instruction, with both constants in registers
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(m) : "r"(sh), "r"(0x00780078u), "r"(0x41804180u));
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(m), "r"(s), "r"(z));
    return r;
}

// The 8 values of a word as four bf16x2 in element order.
__device__ __forceinline__ void packed_octet(uint32_t w, const uint32_t (&s)[4], const uint32_t (&z)[4],
                                             uint32_t (&r)[4]) {
    r[0] = packed_pair<0>(w, s[0], z[0]);
    r[1] = packed_pair<1>(w, s[1], z[1]);
    r[2] = packed_pair<2>(w, s[2], z[2]);
    r[3] = packed_pair<3>(w, s[3], z[3]);
}

}  // namespace hga
