// sage_paged_tiles_half.cu - the many-rows kernel's list of a tree's items with
// two lanes a row, a translation unit of its own.
#define SAGE_PAGED_TILES_TREE 2
#include "sage_paged_tiles.cu"
