// csrc/chunks.h for the host: the chunk of a unit that begins at `column` of the row that begins at element `base`.
#include "../../reducescatter_reduction_gb300/csrc/chunks.h"

extern "C" int chunk_of(const uint64_t *bound, int c, uint64_t base, uint32_t column, uint32_t hidden)
{
    return ccl::chunk_from(bound, c, base + ccl::lookup_column(column, hidden));
}
