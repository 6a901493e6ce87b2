// The cross entropy's buffers, which lie one behind the other in one allocation.  Host code alone.
#pragma once
#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace are {

constexpr int kXentTile = 256;              // rows and columns of a tile
constexpr size_t kXentMinPairs = 4u << 20;  // bytes for a part of d or the forward pass's pairs, whatever M_max is: few pieces for few tokens

// Each a multiple of 256 bytes, so that every buffer begins where a tensor map, a copy or a vector access may.
struct XentSizes {
    size_t d_bytes;    // one of the two parts of a piece's d [M, piece], or the forward pass's pairs
    size_t sum_bytes;  // fp32 sums of dh
    size_t h_bytes;    // the hidden states of rows with a target
    size_t row_bytes;  // a running pair and a logit a row
    size_t sums_at() const { return 2 * d_bytes; }
    size_t h_at() const { return sums_at() + sum_bytes; }
    size_t rows_at() const { return h_at() + h_bytes; }
    size_t total() const { return rows_at() + row_bytes; }
};

// False for capacities whose buffers no device holds (the sizes stay below 2^48, and so do their products).
inline bool xent_sizes(int64_t M_max, int64_t K_max, int64_t piece, XentSizes& z) {
    const int64_t most = (int64_t)1 << 48, columns = (piece + kXentTile - 1) / kXentTile * kXentTile;
    if (M_max > most / (columns * 2) || M_max > most / 12 || K_max > most / (M_max * 4)) return false;
    auto up = [](size_t n) { return (n + 255) & ~(size_t)255; };
    z.d_bytes = up(std::max<size_t>((size_t)M_max * columns * 2, kXentMinPairs));
    // one set of sums for the longest call, or several for calls of few tiles that split the vocabulary over the pairs
    z.sum_bytes = up((size_t)M_max * K_max * 4 + (size_t)std::min<int64_t>(M_max, kXentTile) * kXentTile * 4 * 80);
    z.h_bytes = up((size_t)M_max * K_max * 2);
    z.row_bytes = up((size_t)M_max * 12);
    return true;
}

}  // namespace are
