// window_fwd_tc.cu -- the tensor-core forward through a window for head dim 128 (the kernel is window_fwd_tc_body.cuh).
#define RA_WIN_HD 128
#define RA_WIN_FWD_LAUNCH launch_window_fwd_tc_d128
#include "window_fwd_tc_body.cuh"
