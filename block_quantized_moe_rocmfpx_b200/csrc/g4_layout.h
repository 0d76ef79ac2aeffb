// g4_layout.h -- packed layout of 4-bit weights with group scales ("G4").
//
// W[n][c] = scale[n][c / G] * (code[n][c] - zero[n][c / G]), codes and zeros
// 0..15, binary16 scales, G = 32, 64 or 128 columns a group, cols % G == 0.
// Rows are padded to row-groups of 16; a row-group is one contiguous stream of
// chunks of 128 columns (the last one may be shorter).  A chunk of nc columns:
//   codes   ceil(nc / 64) slabs of 512 bytes; a slab holds two 32-column tiles,
//           lane L = 4g + t at L * 16: words [tile 0 row g][tile 0 row g + 8]
//           [tile 1 row g][tile 1 row g + 8]; half j (0, 1) of a word is
//           c0 | c1 << 4 | c2 << 8 | c3 << 12 turned left by 3 bits, ci the
//           code of column 8t + 2i + j of its tile
//   scales  [g][group] words: row g | row g + 8 << 16
//   zeros   (if any) [g][group] bytes: row g | row g + 8 << 4; padded to 16 bytes
// so that lane L's 16 bytes of a slab are its A operands of four m16n8k16
// products, and every section starts on a 16-byte boundary.
#pragma once
#include <stddef.h>
#include <stdint.h>

#define G4_CHUNK 128

#ifdef __CUDACC__
#define G4_HD __host__ __device__ __forceinline__ constexpr
#else
#define G4_HD static inline
#endif

G4_HD int g4_slabs(int nc) { return (nc + 63) / 64; }
G4_HD int g4_scale_off(int nc) { return g4_slabs(nc) * 512; }
G4_HD int g4_zero_off(int nc, int G) { return g4_scale_off(nc) + nc / G * 32; }
G4_HD int g4_chunk_bytes(int nc, int G, int zeros) {
    return g4_zero_off(nc, G) + (zeros ? (nc / G * 8 + 15) / 16 * 16 : 0);
}
G4_HD int64_t g4_rowgroup_bytes(int64_t K, int G, int zeros) {
    const int tail = (int)(K % G4_CHUNK);
    return K / G4_CHUNK * g4_chunk_bytes(G4_CHUNK, G, zeros) + (tail ? g4_chunk_bytes(tail, G, zeros) : 0);
}
G4_HD int64_t g4_matrix_bytes(int64_t N, int64_t K, int G, int zeros) {
    return (N + 15) / 16 * g4_rowgroup_bytes(K, G, zeros);
}
