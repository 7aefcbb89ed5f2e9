// Low-rank adapters beside a shared projection (internal to the library).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace w4a16 {

struct LoraArgs {
    const uint16_t* x;
    int64_t ldx;
    int64_t m, n, k;
    const uint16_t* a;  // [adapters][rank][k]
    const uint16_t* b;  // [adapters][n][rank]
    int adapters, rank;
    const int32_t* index;
    const float* scales;  // may be null
    const uint16_t* y;
    int64_t ldy;
    uint16_t* out;
    int64_t ldo;
    void* workspace;
};

struct LoraPlan {
    bool one;          // a row or two: one launch, no workspace
    bool tall;         // many rows: the second launch takes tiles of 64 rows by 512 columns
    int tile;          // rows of the first launch's tiles (few rows: of both)
    int slots;         // workgroups that share a row tile's distinct adapters
    int splits;        // parts of K
    int64_t kspan;     // columns of one part (a multiple of 32 except the last)
    size_t workspace;  // after the header
};
LoraPlan plan_lora(int64_t m, int64_t n, int64_t k, int adapters, int rank);
hipError_t launch_lora(const LoraArgs& a, int act, hipStream_t stream);

}  // namespace w4a16
