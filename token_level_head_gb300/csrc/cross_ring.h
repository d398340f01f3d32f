// The rings of tc_cross_read_kernel, in a header of their own: the kernel and a host model of its waits compile the same
// numbers.
#pragma once

namespace mhla {

// Buffers that a block's tiles of queries lie in, one after another (d = 64: three blocks an SM).
constexpr int read_buffers(int d) { return d == 64 ? 3 : 4; }

// Places of the tiles' row sums (den), a sum in parts by the warps that share a row: one beside every buffer.  A warp writes
// its part with the features of a tile and reads all parts with that tile's results; what holds the others back is the copy
// into the tile's buffer, which waits for the results of the tile that lay there.  So a place is free when the buffer is, and
// with fewer places than buffers a warp a tile behind would read a later tile's sum.
constexpr int read_sums(int d) { return read_buffers(d); }

}  // namespace mhla
