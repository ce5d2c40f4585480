// kivi_status.h - how the host takes a status word that kernels OR bits into.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace kivi {

// Waits for `stream`, reads the word that `words` begins with and, where it is set, clears `bytes`
// from there: the word, and the tickets behind it that a failed call may have left counting.  All of
// it runs on `stream` and is complete on return, so that a later call on any stream finds the words
// clear (the legacy stream would order neither: a non-blocking stream does not wait for it).
inline bool take_status(void* words, size_t bytes, cudaStream_t stream, uint32_t* code) {
  return cudaMemcpyAsync(code, words, sizeof *code, cudaMemcpyDeviceToHost, stream) ==
             cudaSuccess &&
         cudaStreamSynchronize(stream) == cudaSuccess &&
         (*code == 0 || (cudaMemsetAsync(words, 0, bytes, stream) == cudaSuccess &&
                         cudaStreamSynchronize(stream) == cudaSuccess));
}

}  // namespace kivi
