// rr_logprob.h -- parameter blocks and launchers of the token log
// probabilities (rr_logprob.cu, host side rr_logprob_api.cu).  Not part of the
// C ABI.
#pragma once

#include "rr_internal.h"

namespace rr {

constexpr int kMaxTop = 32;  // alternatives per row: one per lane of a warp

struct LogprobParams {
    const void* x[kMaxRanksH];    // logits of each rank: T rows of V values, ld elements apart
    const void* ids[kMaxRanksH];  // T ids each
    uint64_t ld;
    uint32_t T, M;                // rows per rank, rows in all
    uint32_t V;
    int ids64;
    float scale;
    int k;                        // alternatives per row
    int split;                    // CTAs (one cluster) per row
    float* logprob;               // [M]
    float* lse;                   // [M]
    float* entropy;               // [M] or NULL
    float* top_logprob;           // [M, k]
    int32_t* top_id;
};

struct LogprobGradParams {
    const void* x[kMaxRanksH];
    const void* ids[kMaxRanksH];
    void* dx[kMaxRanksH];
    uint64_t ld, gld;             // elements from row to row: logits, gradients
    uint32_t T, M;
    uint32_t V;
    int ids64;
    float scale;
    const float* lse;             // [M]
    const float* entropy;         // [M] where dentropy is
    const float* dlogprob;        // [M]
    const float* dentropy;        // [M] or NULL
    uint32_t tiles;               // warp tiles per row
    uint64_t first;               // the launch's first warp tile
};

// CTAs per row a call takes (1, 2, 4 or 8), and whether a warp takes a row.
int logprob_split(uint64_t M, uint64_t V, int dtype);
cudaError_t launch_logprob(int dtype, const LogprobParams& p, cudaStream_t s);
cudaError_t launch_logprob_grad(int dtype, LogprobGradParams p, int* launches, cudaStream_t s);

}  // namespace rr
