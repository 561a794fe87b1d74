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

int64_t logmel_attention_workspace(const logmel_attention_input& in, int backward, int cus);
hipError_t logmel_launch_attention(const logmel_attention_input& in, void* o, int64_t o_stride,
                                   float* state_out, void* ws, int cus, hipStream_t stream);
hipError_t logmel_launch_attention_backward(const logmel_attention_input& in,
                                            const logmel_attention_grad& grad, void* ws, int cus,
                                            hipStream_t stream);

int64_t logmel_group_workspace(const logmel_group_norm_input& in, int backward, int cus);
hipError_t logmel_launch_group(const logmel_group_norm_input& in, void* y, int64_t y_stride,
                               float* stats, void* ws, int cus, hipStream_t stream);
hipError_t logmel_launch_group_backward(const logmel_group_norm_input& in, const float* stats,
                                        const logmel_group_norm_grad& grad, void* ws, int cus,
                                        hipStream_t stream);

// One sum of a launch: out[c] = factor[c] times the sum over g of
// part[g][which][c], part being [parts][sums][channels]; factor null: 1, out
// null: left out.
struct PartSums {
  float* out;
  int which;
  const float* factor;
};

// Three of them, each in a fixed order and in fp64 (logmel_scan.hip).
hipError_t logmel_launch_part_sums(const float* part, int64_t parts, int sums, int64_t channels,
                                   const PartSums out[3], hipStream_t stream);
