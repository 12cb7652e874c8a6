// ssm_launch.h -- host launchers of the selective state space scan (ssm.cu,
// ssm_bwd.cu) behind the C ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

namespace rdm {

// Tokens between two saved states (forward to backward).
constexpr int kSsmChunk = 16;

struct SsmParams {
    int B, H, G, T, D, N, W;  // W = 0: no convolution
    int bf16;    // element type of x, dt, Bm, Cm, z, y, convolution states and their gradients
    int preact;  // delta = softplus(dt + dt_bias) instead of dt
    int silu;    // SiLU behind the convolution
    const void *x, *dt;      // [B,H,T,D]
    const void *Bm, *Cm;     // [B,G,T,N]
    const void* z;           // [B,H,T,D] or null
    const float* A;          // [H,D,N]
    const float* dt_bias;    // [H,D] or null
    const float* dfeed;      // [H,D] or null
    const float* cw;         // [H,D,W]
    const float* cb;         // [H,D] or null
    const void* cs_in;       // [B,H,W-1,D] or null
    const float* S0;         // [B,H,D,N] or null
    const int* lengths;      // [B] or null
    void* y;                 // [B,H,T,D]; null: states only
    float* ST;               // [B,H,D,N] or null
    void* cs_out;            // [B,H,W-1,D] or null
    float* saved;            // [B,H,ceil(T/16),D,N] state before each 16 tokens, or null
    void* ws;
    size_t ws_bytes;
    unsigned* err;           // device status word (a length out of range)
};

struct SsmBwdParams {
    SsmParams f;             // forward arguments (y, ST, cs_out unused; saved = its states, or null)
    const void* gy;          // [B,H,T,D]
    const float* gST;        // [B,H,D,N] or null
    const void* gcs;         // [B,H,W-1,D] gradient of the carried-out inputs, or null
    void *dx, *ddt, *dz;     // [B,H,T,D] (dz null without z)
    void *dB, *dC;           // [B,G,T,N]
    float* dA;               // [H,D,N]
    float *ddt_bias, *ddfeed, *dcw, *dcb;  // null = not asked for
    float* dS0;
    void* dcs;               // [B,H,W-1,D] or null
};

struct SsmStepParams {
    int B, H, G, D, N, W;
    int bf16, preact, silu;
    const void *x, *dt, *Bm, *Cm, *z;  // [B,H,D], [B,G,N]
    const float *A, *dt_bias, *dfeed, *cw, *cb;
    float* S;                // [B,H,D,N] in place
    void* cs;                // [B,H,W-1,D] in place
    void* y;                 // [B,H,D]
};

size_t ssm_fwd_workspace(const SsmParams& p);
cudaError_t launch_ssm_fwd(const SsmParams& p, cudaStream_t s);
size_t ssm_bwd_workspace(const SsmBwdParams& p);
cudaError_t launch_ssm_bwd(const SsmBwdParams& p, cudaStream_t s);
cudaError_t launch_ssm_step(const SsmStepParams& p, cudaStream_t s);

}  // namespace rdm
