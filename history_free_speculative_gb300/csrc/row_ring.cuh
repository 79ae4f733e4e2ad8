// Rows that a CTA takes in turn out of a ring of slots in shared memory, filled ahead of their use by one thread's bulk copies.
//
//   thread 0 fills slots and counts them in `flying`
//   while rows are left:
//     wait()               every thread, for the turn's slot; true: the row is there, whatever other threads say
//     .. reads it; a thread whose wait ran out stores nothing outside the CTA ..
//     a barrier of the CTA
//     if (late()) break    the same answer in every thread
//     thread 0: copies the next row into the slot, or used() where none is left
//     .. stores ..
//     next()
//   thread 0: drain()
//
// A wait that runs out (status flagged) takes the whole CTA out of the loop in the same turn, at its barrier; then the
// copies in flight have one more limit, all of them together. So a CTA ends within two limits of a row that does not come, however many it had left.
#pragma once

#include "tc_device.cuh"

namespace dlite {

struct RowRing {
  uint32_t full;  // the slots' barriers: the arrival of the copying thread and the bytes of its copies
  int slots;
  volatile int* gave_up;  // [2] in shared memory, 0 at first: of turns in turn, so that a thread may still read one turn's while another writes the next's
  int* status;
  uint64_t limit_ns = tc::kTimeoutNs;
  int slot = 0, parity = 0, flying = 0;
  uint32_t phase = 0;

  __device__ __forceinline__ uint32_t bar(int s) const { return full + 8 * s; }
  __device__ __forceinline__ bool wait() {
    const bool there = tc::mbar_wait_hint(bar(slot), phase, status, limit_ns);
    if (!there) gave_up[parity] = 1;
    return there;
  }
  __device__ __forceinline__ bool late() const { return gave_up[parity] != 0; }
  __device__ __forceinline__ void used() { --flying; }
  __device__ __forceinline__ void next() {
    parity ^= 1;
    if (++slot == slots) {
      slot = 0;
      phase ^= 1u;
    }
  }
  __device__ __forceinline__ void drain() {
    if (flying <= 0) return;
    const uint64_t t0 = tc::gtimer();
    for (; flying > 0; --flying, next()) {
      const uint64_t spent = tc::gtimer() - t0;
      tc::mbar_wait(bar(slot), phase, status, spent < limit_ns ? limit_ns - spent : 0);
    }
  }
};

}  // namespace dlite
