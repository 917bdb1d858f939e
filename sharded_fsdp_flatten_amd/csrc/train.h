// train.h -- launchers of a training step's other operators (host-callable): rotary positions
// (rotary.hip), token log probabilities (logprob.hip), AdamW over many tensors (adam_tensors.hip).
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <vector>

#include "kernels.h"
#include "layer.h"

namespace fsdp {

// ---- rotary ----
struct Heads {
    void* p;
    int64_t batch, token, head;  // pitches, in elements
};
struct Rotary {
    int64_t batch, tokens, heads, kv_heads, start;
    int32_t head_dim, rot;
    int32_t bf16, interleaved;
    float scale, sign;           // sign: -1 turns the other way
    Heads q, q_out, k, k_out;    // k.p may be nullptr (kv_heads == 0)
    const int64_t* positions;    // nullptr: start + token
    const double* freqs;
};
hipError_t launch_rotary(const Rotary& a, hipStream_t stream);

// ---- log probabilities ----
constexpr int kMaxTop = 64;
struct LogprobFwd {
    int64_t rows, cols;
    int32_t bf16, top;
    float scale;
    RowsIn x;
    const int64_t* tokens;       // with logprob; else nullptr
    float *logprob, *max, *logsum;
    float* entropy;              // may be nullptr
    float* top_logprob;          // with top
    int64_t* top_token;
    float* workspace;
};
struct LogprobBwd {
    int64_t rows, cols;
    int32_t bf16;
    float scale;
    RowsIn x;
    RowsOut dx;
    const int64_t* tokens;       // with dl
    const float *dl, *dh;        // either may be nullptr
    const float *max, *logsum, *entropy;
};
int64_t logprob_workspace_floats(int64_t rows, int64_t cols, int32_t top);
hipError_t launch_logprob_forward(const LogprobFwd& a, hipStream_t stream);
hipError_t launch_logprob_backward(const LogprobBwd& a, hipStream_t stream);

// ---- AdamW over many tensors ----
constexpr int kAdamGroups = 16;
constexpr int kStateGroup = 32;  // elements of an 8-bit state that share a scale
struct AdamTensor {
    int64_t n;
    float* p;
    const void* g;
    void *m, *v;
    uint16_t* pb;                // may be nullptr
    uint32_t key;                // of its random numbers
    int32_t group;
};
// Bytes from the start of an 8-bit state of n elements to its scales.
inline int64_t state_scales(int64_t n) { return (n + 15) / 16 * 16; }
inline int64_t state_bytes(int64_t n) { return state_scales(n) + (n + kStateGroup - 1) / kStateGroup; }
hipError_t launch_adam_tensors(const std::vector<AdamTensor>& t, const AdamScalars* groups, int n_groups,
                               bool state8, bool grad_bf16, const float* grad_scale, const float* skip,
                               hipStream_t stream);
// One list's states in another format; the 8-bit ones are rounded with the tensors' keys.
enum class State { kF32, kBF16, k8Bit };
struct StateCopy {
    int64_t n;
    const void *m, *v;
    void *m_to, *v_to;
    uint32_t key;
};
hipError_t launch_adam_convert(const std::vector<StateCopy>& t, State from, State to, hipStream_t stream);
// Key of a tensor's random numbers: a 64-bit hash of seed, step and the tensor's place in its list.
uint32_t adam_key(uint64_t seed, int64_t step, int64_t tensor);

}  // namespace fsdp
