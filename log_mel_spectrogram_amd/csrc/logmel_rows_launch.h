// Internal launchers of the row operators, shared with the C-ABI layer. Sizes
// and pointers have been checked by the caller; every kernel keeps its
// accesses inside [0, rows) of the row operands whatever the offsets hold.
#pragma once
#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "logmel.h"

// Bytes of workspace, and the call itself (cus: compute units of the device).
int64_t logmel_scan_workspace(const logmel_scan_input& in, int backward, int cus);
hipError_t logmel_launch_scan(const logmel_scan_input& in, void* h, int64_t h_stride,
                              float* state_out, float* checkpoints, void* ws, int cus,
                              hipStream_t stream);
hipError_t logmel_launch_scan_backward(const logmel_scan_input& in, const float* checkpoints,
                                       const logmel_scan_grad& grad, void* ws, int cus,
                                       hipStream_t stream);

int64_t logmel_norm_workspace(const logmel_norm_input& in, int cus);
hipError_t logmel_launch_norm(const logmel_norm_input& in, void* y, int64_t y_stride, void* z,
                              int64_t z_stride, int cus, hipStream_t stream);
hipError_t logmel_launch_norm_backward(const logmel_norm_input& in, const logmel_norm_grad& grad,
                                       void* ws, int cus, hipStream_t stream);

// out[c] = sum over g of part[g * stride + c], c < channels, in a fixed order
// (logmel_scan.hip).
hipError_t logmel_launch_part_sum(const double* part, int64_t parts, int64_t stride,
                                  int64_t channels, float* out, hipStream_t stream);
