// f4_pair.cuh -- entry of the CTA-pair kernel of f4_mm (f4_pair.cu).
#pragma once

#include "f4.cuh"

namespace f4 {

// Validated arguments of f4_mm.
struct PairArgs {
    const uint8_t* codes;
    const uint8_t* scales;
    const float* gw;
    int64_t N, K;
    const uint8_t* qa;
    const uint8_t* sa;
    const float* ga;
    int64_t M;
    void* y;
    int* err;
};

int launch_pair(const PairArgs& args, int format, int out_dtype, cudaStream_t stream);

}  // namespace f4
