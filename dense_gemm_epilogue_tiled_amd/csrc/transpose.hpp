// A 64 x 64 tile of 16-bit values on its way through LDS to its transpose: 16-byte chunk c of
// row r at slot c XOR (r / 8) mod 8, so that the eight lanes that gather a column's octets of
// rows meet eight distinct groups of banks.
#pragma once

#include "common.hpp"

namespace gr {
namespace train {

constexpr int THREADS = 256;
constexpr int TILE = 64;     // rows and columns of a tile

__device__ __forceinline__ uint32_t tile_off(uint32_t r, uint32_t chunk) {
    return r * (TILE * 2) + ((chunk ^ ((r >> 3) & 7u)) << 4);
}

// Eight rows 8 oct .. of column c of a staged tile.
__device__ __forceinline__ u32x4 column8(const uint8_t* tile, uint32_t c, uint32_t oct) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = *reinterpret_cast<const uint16_t*>(tile + tile_off(8 * oct + 2 * i, c >> 3) + 2 * (c & 7u));
        const uint32_t hi = *reinterpret_cast<const uint16_t*>(tile + tile_off(8 * oct + 2 * i + 1, c >> 3) + 2 * (c & 7u));
        v[i] = lo | (hi << 16);
    }
    return v;
}

}  // namespace train
}  // namespace gr
