// sample.h -- host-side interface of the sampling kernel.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gemma {

struct SampleParams {
    const void* logits;  // [batch][vocab]
    const float* temperature;
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    const float* uniform;
    int32_t* token;
    int32_t* open;             // [batch] whether the short lists left the row undecided
    unsigned long long* mass;  // fp32 logits: [batch][65536] sums of weights, else unused
    uint32_t* err;
    int batch, vocab;
    float softcap;
};

constexpr int kSampleMaxVocab = 16 * 65535;  // 16 CTAs of a row, 16-bit counters
// row flags, then the sums
size_t sample_workspace(int batch, int fp32);
cudaError_t launch_sample(const SampleParams& p, int fp32, cudaStream_t st);

}  // namespace gemma
