// tree_window_tc_d64.cu -- the tensor-core path of the attention over a cache through a window, head dim 64 (tree_tc_body.cuh).
#define RA_TREE_HD 64
#define RA_TREE_LAUNCH launch_tree_window_tc_d64
#define RA_TREE_WINDOW 1
#include "tree_tc_body.cuh"
