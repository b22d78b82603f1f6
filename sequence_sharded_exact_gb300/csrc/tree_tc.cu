// tree_tc.cu -- the tensor-core attention over a cache for head dim 128 (the kernel is tree_tc_body.cuh).
#define RA_TREE_HD 128
#define RA_TREE_LAUNCH launch_tree_tc_d128
#define RA_TREE_WINDOW 0
#include "tree_tc_body.cuh"
