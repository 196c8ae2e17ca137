// Host helpers shared by the translation units of the C ABI.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/litela.h"

namespace litela {

// records the calling thread's last failure (`msg` is copied) and returns `s`
litela_status host_fail(litela_status s, const char* msg);
litela_status host_cuda_fail(cudaError_t e, const char* what);
// forgets the calling thread's last failure
void host_ok();
// the current device, checked to be an sm_100 one: its index and SM count
litela_status host_device(int* dev, int* num_sms);

// The error word of the gated delta rule's kernels on device `dev` (litela_seq_abi.cu), or null
// before that device's first call.
int* delta_error_word(int dev);

}  // namespace litela
