// kda_lin.h -- what the translation units of the decayed linear attention share (kda_lin_*.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_internal.h"

namespace kda {

// A decay below e^-120 is 0 in fp32, and so is every product with it: clamping the logarithm there leaves
// alpha as it is and keeps sums of logarithms finite (minus infinity and NaN become -120 too).
constexpr float kLinLogMin = -120.f;

constexpr int kLinSms = 148;   // SMs of a B200

// One segment of a sequence: what one CTA (of each head and slice) walks through, chunk by chunk.
struct __align__(16) LinItem {
    int seq;     // sequence
    int seg;     // segment within the sequence
    int n_seg;   // segments of the sequence
    int t0;      // first token, in the packed batch
    int n;       // tokens
    int pos;     // tokens of the sequence ahead of the segment (a multiple of kChunk)
    int z0;      // first boundary of the sequence: boundary z0 + s lies between its segments s and s + 1
    int pad;
};

// Workspace header, followed by the items, the sequences with more than one segment, and per boundary and
// head a state [dk, dv] and the decay of the segment ahead of it.
struct __align__(16) LinHead {
    int n_items;
    int n_multi;   // sequences with more than one segment
    int next[2];   // (item, head) pairs taken from behind the grid's own, in the full and the boundary pass
};

struct LinArgs {
    const void* q;
    const void* k;
    const void* v;
    const float* la;
    int la_t;                    // log_alpha of (token, head) is la[token * la_t + head]
    const float* initial_state;
    const int32_t* cu_seqlens;
    int n_seqs;
    int64_t total_tokens;
    int Hqk, H, dk, dv;
    int ckpt_stride;
    void* o;
    float* final_state;
    float* checkpoints;
    const int32_t* ckpt_cu;
    // workspace parts
    LinHead* head;
    LinItem* items;
    int2* multi;                 // {first item's sequence boundary z0, segments} of the sequences with several
    float* z;                    // [boundaries, H, dk, dv]
    float* zdecay;               // [boundaries, H]
    int max_items, max_bounds;   // bounds the host knows
    int* status;
};

// Tensor maps of q, k, v and o for the bf16 kernel, made once per call.
struct LinMaps {
    CUtensorMap q, k, v, o;
};
bool make_lin_maps(const LinArgs& a, LinMaps& m);

// One pass over all segments (kda_lin_simt.cu: fp32 on the fp32 units; kda_lin_bf16.cu: bf16 on the tensor cores).
// boundary_pass: only the segments with a successor, only their end states, into z and zdecay.
cudaError_t launch_lin_simt(const LinArgs& a, bool boundary_pass, cudaStream_t s);
cudaError_t launch_lin_bf16(const LinArgs& a, const LinMaps& m, bool boundary_pass, cudaStream_t s);

// Decode step (kda_lin_step.cu).
cudaError_t launch_lin_step(float* state, int64_t n_states, const int32_t* slots, int slot_stride, const void* q,
                            const void* k, const void* v, const float* la, int la_per_token, int n, int Hqk, int H,
                            int dk, int dv, bool bf16, void* o, int* status, cudaStream_t s);

}  // namespace kda
