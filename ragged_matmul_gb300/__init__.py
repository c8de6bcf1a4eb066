"""GB300 (sm_103a) ragged grouped GEMM for mixture-of-experts layers.

The compute lives in libgmm.so (hand-written CUDA, C ABI in include/gmm.h);
this package holds its ctypes binding, the in-tree build step and the seeded
workload generators.  Importing the package does not load the library; the
first call does, and raises if the library is missing.
"""
from .binding import (EXPORTED, GMM_ERR_BAD_INPUT, GMM_ERR_CUDA, GMM_ERR_DEVICE_TIMEOUT,  # noqa: F401
                      GMM_ERR_INVALID_ARG, GMM_ERR_NO_DEVICE, GMM_ERR_UNSUPPORTED, GMM_OK, GmmError,
                      GMM_ACT_GELU_TANH, GMM_ACT_NONE, GMM_ACT_RELU, GMM_ACT_SILU,
                      Handle, gmm_create, gmm_destroy, gmm_error_string, gmm_query_status, gmm_run,
                      gmm_matmul_int4, gmm_run_ex, gmm_run_fp8, gmm_run_int4, gmm_run_planes, gmm_run_int4_ex, library_path,
                      load_library, GMM_DTYPE_BF16, GMM_DTYPE_FP16, GMM_DTYPE_FP32, GMM_FP4_MX, GMM_FP4_NV,
                      fp4_scale_pitch, gmm_combine, gmm_combine_grad, gmm_dequantize_fp4, gmm_dispatch,
                      gmm_quantize_fp4, gmm_run_fp4, GMM_SCORE_SIGMOID, GMM_SCORE_SOFTMAX, fp8_cols_pitch,
                      gmm_quantize_fp8, gmm_quantize_fp8_cols, gmm_quantize_fp8_tiles, gmm_route, gmm_route_grad,
                      gmm_weight_grad_fp8)
