// layer.h -- launchers of the layer operators (host-callable, defined in layer.hip): 8-bit
// activation checkpoints, LayerNorm / RMSNorm and the MLP activation, forward and backward.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdint>

namespace fsdp {

constexpr int kCkptGroup = 32;  // columns that share one scale

// A rows x cols matrix of bf16 or fp32 whose rows start `pitch` elements apart.
struct RowsIn {
    const void* p;
    int64_t pitch;
};
struct RowsOut {
    void* p;
    int64_t pitch;
};
// 8-bit codes and their groups' scales; codes == nullptr: none.
struct CkptRows {
    uint8_t* codes;
    uint8_t* scales;
    int64_t code_pitch, scale_pitch;
    int32_t int8;  // 0: e4m3 codes, 1: integers
};

// Column sums of a backward pass: out = (accumulate ? out : 0) + sum.
struct ColOut {
    void* p;  // nullptr: not wanted
    int32_t bf16, accumulate;
};

struct NormFwd {
    int64_t rows, cols;
    int32_t bf16, param_bf16, rms;
    float eps;
    RowsIn x, residual;  // residual.p may be nullptr
    RowsOut sum, y;      // sum.p may be nullptr
    const void *weight, *bias;
    float *mean, *rstd;  // mean may be nullptr
    CkptRows ckpt;
};

struct NormBwd {
    int64_t rows, cols;
    int32_t bf16, param_bf16, rms;
    RowsIn dy, x, dres;  // x.p is nullptr where ckpt holds the input
    CkptRows ckpt;
    RowsOut dx, y;       // y.p may be nullptr
    const void *weight, *bias;
    const float *mean, *rstd;
    ColOut dweight, dbias;
    float* workspace;
};

// f: 0 none (a checkpoint only), 1 relu, 2 gelu, 3 gelu with tanh, 4 silu.
struct ActFwd {
    int64_t rows, cols;
    int32_t bf16, f;
    RowsIn x;
    RowsOut y;
    CkptRows ckpt;
};

struct ActBwd {
    int64_t rows, cols;
    int32_t bf16, f;
    RowsIn dy, x;
    CkptRows ckpt;
    RowsOut dx, y;
    ColOut dbias;
    float* workspace;
};

// Floats of workspace (16-byte aligned) of the backward passes; -1 if that overflows int64.
int64_t norm_workspace_floats(int64_t rows, int64_t cols);
int64_t act_workspace_floats(int64_t rows, int64_t cols);

hipError_t launch_act_forward(const ActFwd& a, hipStream_t stream);   // f == 0: pack
hipError_t launch_unpack(int64_t rows, int64_t cols, bool bf16, const CkptRows& q, RowsOut x,
                         hipStream_t stream);
hipError_t launch_act_backward(const ActBwd& a, hipStream_t stream);
hipError_t launch_norm_forward(const NormFwd& a, hipStream_t stream);
hipError_t launch_norm_backward(const NormBwd& a, hipStream_t stream);

// The kernels of the norms' backward pass that hold a row in registers, `threads` of them with
// `vectors` vectors of 4 columns each: they write the input's gradient and, for every workgroup, a
// partial row (2 x cols floats) of the weight's and the bias's.
struct BwdShape {
    int threads, vectors;
};
BwdShape norm_bwd_shape(int64_t cols);
// Workgroups of these kernels that a CU holds at once: two of 8 waves with 128 registers or one of 16
// waves; one of 8 waves with more registers where a row's three vectors and a residual gradient are fp32
// or come with codes (up to 150; held to 128 they spill up to 40).
constexpr int norm_bwd_resident(bool bf16, bool ckpt, bool residual, int threads, int vectors) {
    return threads > 512 || (vectors == 3 && residual && (!bf16 || ckpt)) ? 1 : 2;
}
void launch_norm_bwd_rows_bf16(const NormBwd& a, float* partial, uint32_t blocks, hipStream_t stream);
void launch_norm_bwd_rows_f32(const NormBwd& a, float* partial, uint32_t blocks, hipStream_t stream);
// the same with non-temporal loads
void launch_norm_bwd_rows_bf16_nt(const NormBwd& a, float* partial, uint32_t blocks, hipStream_t stream);
void launch_norm_bwd_rows_f32_nt(const NormBwd& a, float* partial, uint32_t blocks, hipStream_t stream);

}  // namespace fsdp
