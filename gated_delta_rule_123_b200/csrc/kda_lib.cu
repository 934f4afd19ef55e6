// The translation unit of libkda.so that holds every kernel with a bounded wait (one
// definition of the device status word that they share) and all entry points.  The
// mixer's kernels without waits are units of their own (kda_norm.cu, kda_conv.cu,
// kda_scan.cu, kda_scan_bwd.cu), compiled at the same time.
#include "kda_api.cu"
#include "kda_chunk.cu"
#include "kda_dplr.cu"
#include "kda_decode.cu"
#include "kda_backward.cu"
#include "kda_gemm.cu"
#include "kda_layer.cu"
#include "kda_noalloc.cu"
#include "kda_linear_act.cu"
#include "kda_mixer_api.cu"
