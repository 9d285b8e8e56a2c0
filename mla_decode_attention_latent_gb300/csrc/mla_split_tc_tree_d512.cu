// Split-KV kernel with a draft tree's mask over the last rows of each sequence,
// for the 512-wide cached row.
#define MLA_SPLIT_D 512
#define MLA_SPLIT_TREE 1
#include "mla_split_tc_impl.cuh"
