// What the library's entry points share across translation units (host code).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace segtopk {

// Records a failed CUDA call for segtopk_last_cuda_error on this thread;
// returns SEGTOPK_ERROR_CUDA.
int record_cuda_error(cudaError_t e);

// Sets what segtopk_last_launch_count returns on this thread.
void record_launch_count(int launches);

// SEGTOPK_SUCCESS and the number of SMs if the current device is an sm_103
// GPU, else the status to return.
int check_device(int* sms);

// The bound of a wait in SM clock cycles, and the bytes that a test adds to
// what the first copies are expected to bring (segtopk_set_test_hooks; 0 in
// the ordinary build).
void test_hooks(long long* wait_limit, uint32_t* extra_bytes);

// Read and clear the device error words of the units that can set one
// (synchronous).
cudaError_t read_group_error(uint32_t* word);
cudaError_t read_embedding_error(uint32_t* word);
cudaError_t read_matmul_error(uint32_t* word);

} // namespace segtopk
