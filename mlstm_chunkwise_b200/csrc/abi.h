// What the files that hold C entry points share (implemented in abi.cu).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <type_traits>

#include "common.cuh"

namespace mlstm {

// Device error word in the current context (nullptr if it cannot be looked up).
uint32_t* device_error_word();
// Spin limit of every bounded wait of the launches made from now on.
unsigned long long watchdog_polls();

// Runs fn(arg), which enqueues `n_launch` kernels of family `id` on `st`:
// counts them and, while profiling is on, brackets them with events.
mlstm_status run_family(int id, int n_launch, cudaStream_t st, cudaError_t (*fn)(void*),
                        void* arg);
template <typename Fn>
mlstm_status run_family(int id, int n_launch, cudaStream_t st, Fn&& fn) {
  return run_family(
      id, n_launch, st,
      [](void* f) -> cudaError_t { return (*static_cast<typename std::remove_reference<Fn>::type*>(f))(); },
      const_cast<void*>(static_cast<const void*>(&fn)));
}

inline bool is_aligned(const void* p, unsigned n) {
  return reinterpret_cast<uintptr_t>(p) % n == 0;
}

}  // namespace mlstm
