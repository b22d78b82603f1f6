// tree_window_tc.cu -- the tensor-core path of the attention over a cache through a window, head dim 128 (tree_tc_body.cuh).
#define RA_TREE_HD 128
#define RA_TREE_LAUNCH launch_tree_window_tc_d128
#define RA_TREE_WINDOW 1
#include "tree_tc_body.cuh"
