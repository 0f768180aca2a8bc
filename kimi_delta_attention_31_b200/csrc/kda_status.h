// kda_status.h -- error reporting shared by the library's translation units:
// the calling thread's message (kda_last_error) and the device error words.
#pragma once
#include <cuda_runtime_api.h>

#include "../../include/kda.h"

namespace kda {

// Records the calling thread's message and returns st; clear_status() empties it.
__attribute__((visibility("hidden"))) kda_status_t set_status(kda_status_t st, const char* fmt, ...)
    __attribute__((format(printf, 2, 3)));
__attribute__((visibility("hidden"))) void clear_status();

// Every translation unit with kernels has an error word of its own
// (g_device_error in kda_common.cuh); this one reads and clears the word of the
// kernels in kda_layer_api.cu on the current device.
__attribute__((visibility("hidden"))) cudaError_t take_layer_device_error(int* code);

}  // namespace kda
