// window_bwd_tc_d64.cu -- the tensor-core backward through a window for head dim 64 (the kernel is window_bwd_tc_body.cuh).
#define RA_WIN_HD 64
#define RA_WIN_BWD_LAUNCH launch_window_bwd_tc_d64
#include "window_bwd_tc_body.cuh"
