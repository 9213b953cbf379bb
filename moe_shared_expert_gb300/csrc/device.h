// Services of the C-ABI layer (api.cu) that the other translation units' entry points use.
#pragma once
#include <cuda.h>
#include <stdint.h>

#include "mse.h"

namespace mse {

struct DeviceView {
    int sm_count;
    uint32_t *err;      // device error word
};
// The current device, checked: MSE_ERR_UNSUPPORTED_DEVICE unless it is compute capability 10.3.
mse_status device_view(DeviceView *out);
// The kernel path of a call whose shape and alignment the tensor-core kernels serve or not
// (mse_set_kernel_path): *tensorcore is the choice, MSE_ERR_UNSUPPORTED_SHAPE when it is forced
// and cannot serve.
mse_status choose_tensorcore(bool tc_ok, bool *tensorcore);
bool pdl_enabled();
uint64_t wait_limit_ns();
// A call on `stream` whose outputs the early token loads do not track: the next call waits.
void begin_untracked_call(void *stream);
// [rows x cols] row-major bytes (row pitch ld, a multiple of 16; base 16-byte aligned), box of
// 128 bytes x box_rows rows with 128-byte swizzle; what lies outside reads zero.
mse_status map_bytes(CUtensorMap *m, const void *base, int64_t rows, int64_t cols, int64_t ld, int box_rows);

}  // namespace mse
