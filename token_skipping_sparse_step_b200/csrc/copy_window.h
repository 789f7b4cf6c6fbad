// Bookkeeping of a walk over chunks 0, 1, ... whose copies go through a ring of
// stages. Plain C++, so that it also compiles without CUDA.
#pragma once

#ifdef __CUDACC__
#define ESD_HOST_DEVICE __host__ __device__
#else
#define ESD_HOST_DEVICE
#endif

namespace esd {

// Copies start and land in the order of the chunks. When the walk gives up, chunks
// [landed, started) are in flight: each of them completes its barrier's phase, and
// nothing completes a phase of a chunk whose copy never started.
struct CopyWindow {
  int started = 0, landed = 0;
  ESD_HOST_DEVICE void start(int chunk) { started = chunk + 1; }
  ESD_HOST_DEVICE void land(int chunk) { landed = chunk + 1; }
  // f(chunk) for every chunk in flight
  template <typename F>
  ESD_HOST_DEVICE void drain(F f) const {
    for (int j = landed; j < started; ++j) f(j);
  }
};

}  // namespace esd
