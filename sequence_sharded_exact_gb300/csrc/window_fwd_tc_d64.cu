// window_fwd_tc_d64.cu -- the tensor-core forward through a window for head dim 64 (the kernel is window_fwd_tc_body.cuh).
#define RA_WIN_HD 64
#define RA_WIN_FWD_LAUNCH launch_window_fwd_tc_d64
#include "window_fwd_tc_body.cuh"
