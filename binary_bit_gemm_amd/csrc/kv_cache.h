// Layout of the paged cache of keys and values (lowbit_cache in include/lowbit.h), shared by the kernels that
// write and read it.
//
// A page holds page_size tokens (16 .. 256, a power of two) of every kv head: k and v [pages, kv_heads, page_size, row], a row
// being D elements at 16, 8 or 4 bits.  Inside a page's head the codes lie as the attention kernel's lanes take them
// (lane (q, l16): quarter q of a wave, lane l16 of it):
//   K  a token's row after the other.  16 and 8 bits: elements in order.  4 bits: four parts, part p holds elements
//      16 p .. 16 p + 15 of every group of 64 as two words of 8 codes, element e of a word at nibble e / 2 + 4 (e % 2):
//      masks then cut a word into pairs of neighbouring elements.  Lane (q, l16) reads part q of key l16's row.
//   V  blocks of kBlock tokens, [16 pieces][kBlock tokens][kPiece bytes].  Piece l holds elements l D / 16 .. of a row, at 4 bits
//      elements 4 l .. 4 l + 3 of every group of 64 (first in the low nibble).  Lane (q, l16) takes piece l16 of
//      keys 4q .. 4q + 3: its part of the matrix operand for all those columns, 16 bytes a load, with neighbouring lanes on
//      neighbouring 16 bytes; the transposition that the product needs is then byte permutes between a lane's own registers.
// Scales (bf16): 8 bits one per token [pages, kv_heads, page_size]; 4 bits (scale, smallest value) per token and group of 64,
// [pages, kv_heads, page_size, D / 64, 2].
#pragma once

#include <stdint.h>

namespace lowbit {

constexpr int kCacheGroup = 64;  // elements that share a scale at 4 bits

template <int D, int BITS>
struct CacheFmt {
    static constexpr int kRow = D * BITS / 8;      // bytes of a token's row
    static constexpr int kPiece = kRow / 16;       // bytes of a piece of V: 16, 8, 4 or 2
    static constexpr int kBlock = kPiece >= 16 ? 1 : kPiece == 8 ? 2 : 4;  // tokens of a block of V
    static constexpr int kGroups = BITS == 4 ? D / kCacheGroup : 1;
    static constexpr int kScaleBytes = BITS == 16 ? 0 : BITS == 8 ? 2 : 4 * kGroups;  // of a token
    static constexpr uint32_t v_offset(uint32_t token, uint32_t piece) {
        return token / kBlock * (kBlock * kRow) + piece * (kBlock * kPiece) + token % kBlock * kPiece;
    }
};

}  // namespace lowbit
