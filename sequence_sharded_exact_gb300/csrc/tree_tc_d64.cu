// tree_tc_d64.cu -- the tensor-core attention over a cache for head dim 64 (the kernel is tree_tc_body.cuh).
#define RA_TREE_HD 64
#define RA_TREE_LAUNCH launch_tree_tc_d64
#define RA_TREE_WINDOW 0
#include "tree_tc_body.cuh"
