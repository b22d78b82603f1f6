// window_bwd_tc.cu -- the tensor-core backward through a window for head dim 128 (the kernel is window_bwd_tc_body.cuh).
#define RA_WIN_HD 128
#define RA_WIN_BWD_LAUNCH launch_window_bwd_tc_d128
#include "window_bwd_tc_body.cuh"
