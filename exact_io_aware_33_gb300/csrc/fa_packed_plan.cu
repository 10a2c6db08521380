// The list of the forward's work (make_list in fa_packed.cuh; the backward's are
// made beside its row sums), as a kernel of one block.
//
// Bound by latency: 3.4 us for 8 sequences of up to 4096 tokens (198 entries of 64
// tokens), 12.7 us for 4096 of up to 16 (3941 entries).

#include "fa_packed.cuh"

namespace fa {
namespace {

constexpr int kThreads = 1024;

__global__ void __launch_bounds__(kThreads, 1) packed_plan_kernel(const __grid_constant__ PackedShape s,
                                                                 const __grid_constant__ PackedList list, int* status) {
  grid_dep_wait();
  grid_dep_launch();
  make_list<kThreads>(s, list, status);
}

}  // namespace

int launch_packed_plan(const PackedShape& s, const PackedList& list, cudaStream_t stream) {
  int* status = device_status_word();
  if (!status) return -3;
  const cudaError_t e = launch_overlapped(packed_plan_kernel, dim3(1), dim3(kThreads), 0, stream, s, list, status);
  return cudaGetLastError() == cudaSuccess && e == cudaSuccess ? 0 : -3;
}

}  // namespace fa
