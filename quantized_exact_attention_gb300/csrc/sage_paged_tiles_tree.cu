// sage_paged_tiles_tree.cu - the many-rows kernel's forms with a tree's mask, a
// translation unit of their own so that they compile beside the others.
#define SAGE_PAGED_TILES_TREE 1
#include "sage_paged_tiles.cu"
