// Probe of the bounded device waits (failure detection without a fault).
//
// Every mbarrier wait of the tensor-core kernels gives up after a time limit,
// flags DLITE_DEV_TIMEOUT in the status word and lets the kernel return; a
// kernel that starts while the flag is set skips its work. These two tiny
// kernels exercise exactly those helpers with a short, caller-chosen limit:
// the first waits on a barrier nobody arrives at (one warp through the
// warp-wide wait, one thread through the single-thread wait), the second
// makes the engines' entry check. A third walks the rows of a ring (row_ring.cuh) whose copies stop coming.
#include "tc_device.cuh"
#include "kernels.h"
#include "row_ring.cuh"

namespace dlite {
namespace {

__global__ void __launch_bounds__(64) wait_probe_kernel(uint64_t limit_ns, int* status, int32_t* result) {
  __shared__ __align__(8) uint64_t bar;
  const uint32_t b = tc::su32(&bar);
  if (threadIdx.x == 0) {
    tc::mbar_init(b, 1);  // one arrival expected; none comes
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const bool got = tc::mbar_wait_warp(b, 0, status, limit_ns);
    if (threadIdx.x == 0) result[0] = got ? 0 : 1;
  } else if (threadIdx.x == 32) {
    const bool got = tc::mbar_wait(b, 0, status, limit_ns);
    result[1] = got ? 0 : 1;
  }
}

__global__ void abort_probe_kernel(int* status, int32_t* result) {
  const bool aborted = status && (*(volatile int*)status & kDevTimeout);  // as the engines check
  if (threadIdx.x == 0) result[2] = aborted ? 1 : 0;
}

// Case blockIdx.x. 0: no row arrives. 1: rows 0 to 4 arrive. 2: all arrive, but thread 5 takes itself for late in turn 7 alone.
// What stands for a copy: an arrival, or, of a row that does not come, an arrival that expects 16 bytes which nobody sends.
__global__ void __launch_bounds__(64) ring_probe_kernel(uint64_t limit_ns, int* status, int32_t* result) {
  constexpr int kSlots = 3, kRows = 1000;
  __shared__ __align__(8) uint64_t full[kSlots];
  __shared__ int gave_up[2];
  const int which = blockIdx.x, comes = which == 0 ? 0 : which == 1 ? 5 : kRows;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) tc::mbar_init(tc::su32(full + i), 1);
    gave_up[0] = gave_up[1] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  const uint64_t t0 = tc::gtimer();
  RowRing r = {tc::su32(full), kSlots, gave_up, status, limit_ns};
  int ahead = 0, row = 0, stored = 0;
  auto copy = [&](int slot) {
    if (ahead++ < comes)
      tc::mbar_arrive(r.bar(slot));
    else
      tc::mbar_expect_tx(r.bar(slot), 16);
  };
  if (threadIdx.x == 0)
    for (; r.flying < kSlots; ++r.flying) copy(r.flying);
  for (; row < kRows; ++row) {
    r.wait();
    if (which == 2 && row == 7 && threadIdx.x == 5) gave_up[r.parity] = 1;
    __syncthreads();
    if (r.late()) break;
    if (threadIdx.x == 0) {
      if (ahead < kRows)
        copy(r.slot);
      else
        r.used();
    }
    ++stored;
    r.next();
  }
  if (threadIdx.x == 0) r.drain();
  const uint64_t limits = (tc::gtimer() - t0) / limit_ns;
  __shared__ int first;
  if (threadIdx.x == 0) first = stored;
  __syncthreads();
  const int same = __syncthreads_and(stored == first);
  if (threadIdx.x == 0) {
    result[4 * which] = stored;
    result[4 * which + 1] = same;
    result[4 * which + 2] = r.flying;
    result[4 * which + 3] = (int32_t)min(limits, (uint64_t)0x7fffffff);
  }
}

}  // namespace

cudaError_t launch_ring_probe(uint64_t limit_ns, int* status, int32_t* result, cudaStream_t s) {
  ring_probe_kernel<<<3, 64, 0, s>>>(limit_ns, status, result);
  return cudaGetLastError();
}

cudaError_t launch_wait_probe(uint64_t limit_ns, int* status, int32_t* result, cudaStream_t s) {
  wait_probe_kernel<<<1, 64, 0, s>>>(limit_ns, status, result);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  abort_probe_kernel<<<1, 32, 0, s>>>(status, result);
  return cudaGetLastError();
}

}  // namespace dlite
