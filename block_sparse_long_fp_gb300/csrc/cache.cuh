// The bf16 / e4m3 paged K/V cache and rotary positions as their kernels see them.
#pragma once

#include "qcache.cuh"

namespace fp {

struct Rotation {
    const unsigned long long *turns;           // [rot / 2]; null: none
    int rot;
    bool interleaved;
    float scale;                               // of cos, and of sin (negated there for the inverse)
    float sin_scale;
};

// `heads` vectors of kHeadDim elements a row: bf16 in, bf16 or (with scales) e4m3 out.
struct RowsPart {
    const __nv_bfloat16 *in;
    void *out;
    long long in_tok, in_head, out_tok, out_head;   // elements
    const float *scale;
    int heads;
};

struct RotateRows {
    Rotation rot;
    const int *positions;                      // null: nothing is rotated
    int rows;
    RowsPart q, k, v;                          // q and k are rotated; k and v go to row slots[i]
    const int *slots;
    long long num_slots;
    int *status;
};
cudaError_t launch_rotate_rows(const RotateRows &r, cudaStream_t st);

}  // namespace fp
