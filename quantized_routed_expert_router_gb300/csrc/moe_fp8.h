// moe_fp8.h - arguments shared by the two forms of moe_fp8_matmul.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

struct Fp8Args {
    const uint8_t *x, *w;
    const float *xs, *ws;
    const int32_t *rows, *offsets;
    void *y;
    unsigned *status;
    int X, M, G, N, K, KB, NB;
    int ntn;       // column tiles
    int xbox;      // rows of an x copy (ungathered)
    int yalign;    // bytes that rows of y are aligned to: 32, 16 or less
};

// few rows: the weights straight into matrix instructions (moe_fp8_rows.cu)
bool fp8_few_rows(const Fp8Args &a);
cudaError_t launch_fp8_rows(const Fp8Args &a, int ydtype, cudaStream_t s);

}  // namespace moe
