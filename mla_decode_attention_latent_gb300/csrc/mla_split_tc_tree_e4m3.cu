// Split-KV kernel with a draft tree's mask over the last rows of each sequence,
// for the 576-wide latent cache stored as packed e4m3 pages.
#define MLA_SPLIT_D 576
#define MLA_SPLIT_FP8 1
#define MLA_SPLIT_TREE 1
#include "mla_split_tc_impl.cuh"
