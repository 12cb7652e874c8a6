// ska_q8_launch.h -- host launchers of shared-key attention over an 8-bit ring
// cache (ska_q8.cu) behind the C ABI.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

namespace rdm {

// The cache: position p of a sequence in slot p mod window, slots in blocks of
// `block` (the last one may be short); codes with a scale for each block and
// head, and the tokens of the block being written in bf16 beside them.
struct SkaQ8Cache {
    int B, H, dk, dv, window, block;
    int int8;              // codes are int8, else e4m3
    unsigned char* k;      // [B,window,dk]
    unsigned char* v;      // [B,H,window,dv]
    float* k_scale;        // [B,NB]
    float* v_scale;        // [B,H,NB]
    void* k_tail;          // [B,block,dk] bf16
    void* v_tail;          // [B,H,block,dv] bf16
    int* pos;              // [B]
};
struct SkaQ8FillParams {
    SkaQ8Cache c;
    int T;
    const void *k, *v;     // [B,T,dk], [B,H,T,dv] bf16
    const int* lengths;    // [B] or null
    unsigned* err;
};
struct SkaQ8DecodeParams {
    SkaQ8Cache c;
    float scale;
    const void *q, *k, *v; // [B,H,dk], [B,dk], [B,H,dv] bf16
    void* o;               // [B,H,dv] bf16
    int advance;
    void* ws;
    size_t ws_bytes;
    unsigned* err;
};
cudaError_t launch_ska_q8_fill(const SkaQ8FillParams& p, cudaStream_t s);
size_t ska_q8_decode_workspace(const SkaQ8DecodeParams& p);
cudaError_t launch_ska_q8_decode(const SkaQ8DecodeParams& p, cudaStream_t s);

}  // namespace rdm
