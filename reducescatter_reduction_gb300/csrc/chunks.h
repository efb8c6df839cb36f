// Which chunk of a schedule an element lies in, host and device.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define CCL_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define CCL_HOST_DEVICE inline
#endif

namespace ccl {

// The chunk of element e, walked to from chunk c, which does not begin behind e.  The walk ends in the table only for
// elements of the buffers, e < bound[p].
CCL_HOST_DEVICE int chunk_from(const uint64_t *bound, int c, uint64_t e)
{
    while (e >= bound[c + 1]) ++c;
    return c;
}

// The column that stands for a unit which begins at `column` when its chunk is looked up: rows narrower than a warp's
// columns leave lanes without any, whose elements may lie behind the last row.  They take the row's last column.
CCL_HOST_DEVICE uint32_t lookup_column(uint32_t column, uint32_t hidden) { return column < hidden ? column : hidden - 1; }

}  // namespace ccl
