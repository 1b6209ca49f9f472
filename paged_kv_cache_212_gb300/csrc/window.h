// window.h -- internal interface of the rotary and windowed calls: host checks
// they share with the entry points of api.cu, and the windowed prefill's launch.
#pragma once

#include "launch.h"
#include "../../include/pagedkv_rope.h"

namespace pkv {

// Host checks (api.cu): PKV_OK or PKV_ERR_CUDA with the error recorded; 16-byte
// alignment; the SM count of the current device; the geometry every kernel supports.
int cuda_status(cudaError_t e);
bool aligned16(const void *p);
int num_sms_of_current_device(int *out);
constexpr int32_t kMaxBlockSize = 256;   // tokens; check_dims refuses larger blocks
int check_dims(const pkv_dims &d);

// Checks of a rotary turn for heads of head_dim elements, and of a stride between
// tokens of `heads` head rows (rope_write.cu).
int check_rope(const pkv_rope *rope, int32_t head_dim);
bool row_stride_ok(int64_t stride, int32_t heads, int32_t head_dim);

cudaError_t launch_prefill_window(const PrefillArgs &a, int32_t window, int32_t sinks, int num_sms, cudaStream_t stream);

}  // namespace pkv
