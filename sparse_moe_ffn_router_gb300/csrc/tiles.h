// tiles.h -- how the linear layers cut an expert's columns into tiles. Plain arithmetic, for the kernels and for a host
// compiler. Columns are rows of x (or of W), up to 2^31 - 2^16 of them: nothing here adds to their number.
#pragma once

#ifdef __CUDACC__
#define MOE_TILES_FN __host__ __device__ __forceinline__
#else
#define MOE_TILES_FN inline
#endif

namespace moe {

// Tiles of at most `most` columns.
MOE_TILES_FN int lin_tiles(int cols, int most) { return cols > 0 ? (cols - 1) / most + 1 : 0; }

// Columns of each of them (cols >= 1; the last has what is left): as even as steps of STEP allow, STEP a divisor of `most`.
template <int STEP>
MOE_TILES_FN int lin_width(int cols, int tiles) { return ((cols - 1) / tiles + STEP) / STEP * STEP; }

}  // namespace moe
