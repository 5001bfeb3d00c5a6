// Which 16-byte pieces of packed rows may leave their array: plain integer
// arithmetic, the same on the host, where the tests enumerate it.
//
// Rows of `tokens` elements lie end to end, so a row that is no whole number of
// 16-byte vectors is staged in pieces from the boundary at or below its first
// token of a tile: up to vec - 1 elements early, and up to vec past the tile.
// Those elements belong to neighbouring rows, except at the array's two ends;
// with few tokens the overhang is longer than a row and passes several rows at once.
#pragma once

#ifdef __CUDACC__
#define SSCAN_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define SSCAN_HOST_DEVICE inline
#endif

namespace sscan {

// Of rows row0 .. row0 + rows - 1 in an array of dim rows, the last tile
// [t0, t0 + tile) whose pieces end inside the array (-1: none).
SSCAN_HOST_DEVICE int last_inner_tile(long long row0, int rows, long long dim, int tokens, int tile, int vec) {
    const long long room = (dim - row0 - rows + 1) * tokens;  // from the last row's start to the array's end
    const long long last = room - tile - vec;
    return last < -1 ? -1 : last < tokens ? (int)last : tokens;
}
// Whether pieces of the tile at t0 may lie outside the array.  At its front only
// a first tile can: any later one begins tile >= vec elements into its row.
SSCAN_HOST_DEVICE bool at_edge(int t0, int last_inner) { return t0 == 0 || t0 > last_inner; }
// The same for tiles that end before their rows do (t0 + tile < tokens), of
// rows from the first or from vec rows on: what they reach past a row's end is
// shorter than a further row, so only the array's first and last row matter.
SSCAN_HOST_DEVICE bool inner_at_edge(long long row0, int rows, long long dim, int tokens, int t0, int tile, int vec) {
    return (row0 == 0 && t0 == 0) || (row0 + rows >= dim && t0 + tile + vec > tokens);
}

}  // namespace sscan
