// The 4-bit key/value cache: its layout, shared by the kernels that write it and read it.
//
// A pool holds n_pages pages of page_size tokens for Hkv heads: [n_pages][Hkv][page_size / 16]
// records.  A record is 16 consecutive tokens of one head, 18 d bytes that one bulk copy brings in:
//   K codes    16 x d/2 bytes    token row t; channel i = 32 w + 8 c + j is nibble j % 2 of byte
//                                t d/2 + c d/8 + 4 w + j/2
//   K words    16 x d/64 words   [t][i / 64]: scale (bf16) | minimum (bf16) << 16
//   V codes    16 x d/2 bytes    channel i = 64 p + 16 u + 8 y + g, token t: nibble y of byte
//                                512 p + 16 (4 g + (t % 8) / 2) + 4 u + 2 (t % 2) + t / 8
//   V words    16 x d/64 words
// A code n stands for n * scale + minimum.  The order inside a record is that of the operand
// fragments of the attention: lane 4 g + c of a warp reads its 8 K channels of word w of token g
// and its V tokens 2c, 2c + 1, 2c + 8, 2c + 9 as whole 32-bit words without bank conflicts, and every
// byte belongs to one token, so tokens can be appended one at a time.
#pragma once

#include <cstdint>

namespace sparge {

constexpr int C4_TOKENS = 16;  // tokens of a record

template <int D>
struct Rec4 {
  static constexpr int NG = D / 64;                 // channel groups: scales and minima of a token
  static constexpr int CODES = C4_TOKENS * D / 2;   // bytes of K (or V) codes
  static constexpr int WORDS = C4_TOKENS * NG * 4;  // bytes of K (or V) scale words
  static constexpr int K = 0, KW = CODES, V = CODES + WORDS, VW = V + CODES;
  static constexpr int BYTES = 2 * (CODES + WORDS);
};

// Validated pool.
struct Cache4 {
  uint8_t *data;
  int64_t n_pages;
  int page_size, page_shift;  // page_size = 1 << page_shift tokens
  int H, d;
};

}  // namespace sparge
