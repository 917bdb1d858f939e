// logprob.hip -- log probabilities of given tokens with entropy and top alternatives, and the gradient of
// the logits.
//
// With z = scale x over a row of logits: one pass keeps, for every lane, the largest x so far, the sum of
// 2^(k (x - m)) and (for the entropy) of that times its exponent, k = scale log2 e; sums move to a new
// maximum by one factor.  The lanes' triples join in a fixed order.  Bound by HBM: forward reads every
// logit once, backward reads and writes each once.
#include <algorithm>

#include "layer_dev.h"
#include "train.h"

namespace fsdp {
namespace {

constexpr double kLog2e = 1.4426950408889634074, kLn2 = 0.69314718055994530942;

// Running sums of a part of a row, against its largest logit m: s = sum of e, t = sum of e u with
// u = k (x - m), e = 2^u.  A part without logits above -infinity has m = -infinity, s = t = 0.
struct Part {
    float m, s, t;
};
// Logits are taken against their difference from the maximum, not against k m: masks of the type's
// lowest value would overflow in the product.  -infinity as a maximum would make NaN of masked logits.
__device__ __forceinline__ float anchor(float m) { return m == -INFINITY ? 0.0f : m; }

// How far the exponents of sums against `from` move when they are taken against `to`, the larger one;
// never so far that 2^shift times a sum's weight could be infinity times 0.
__device__ __forceinline__ float shift(float from, float to, float k) {
    return from == to ? 0.0f : fmaxf((from - to) * k, -1000.0f);
}
__device__ __forceinline__ Part join(Part a, Part b, float k) {
    const float m = fmaxf(a.m, b.m);
    const float da = shift(a.m, m, k), db = shift(b.m, m, k);
    const float fa = __builtin_amdgcn_exp2f(da), fb = __builtin_amdgcn_exp2f(db);
    return Part{m, a.s * fa + b.s * fb, fa * (a.t + da * a.s) + fb * (b.t + db * b.s)};
}

// e u without 0 x infinity: far below -149 e is 0; a NaN stays one
__device__ __forceinline__ float weighted(float e, float u) { return e * fmaxf(u, -200.0f); }

// What the sums of a whole row come to.
struct Row {
    float max, logsum, entropy;
    __device__ bool empty() const { return max == -INFINITY && logsum == 0.0f; }
};
__device__ __forceinline__ Row finish(const Part& p, float scale) {
    Row r;
    r.max = p.m * scale;
    if (r.max == -INFINITY && p.s == p.s) return Row{-INFINITY, 0.0f, 0.0f};  // nothing above -infinity
    if (r.max == INFINITY) return Row{INFINITY, NAN, NAN};
    const float ls = logf(p.s);
    r.logsum = ls + fmaf(p.m, scale, -r.max);   // of the rounded maximum, so that the two add up
    r.entropy = ls - static_cast<float>(kLn2) * (p.t / p.s);
    return r;
}

__device__ __forceinline__ float value(const uint16_t* p) {
    return __builtin_bit_cast(float, static_cast<uint32_t>(*p) << 16);
}
__device__ __forceinline__ float value(const float* p) { return *p; }

// A logit's place in the order of alternatives: larger values first, then lower columns; NaN as
// -infinity.  Larger keys come first; no two are equal; 0 is below every key.
__device__ __forceinline__ uint64_t rank_key(float x, uint32_t col) {
    x = x == x ? x + 0.0f : -INFINITY;  // -0 as 0
    const uint32_t b = __builtin_bit_cast(uint32_t, x);
    const uint32_t o = b & 0x80000000u ? ~b : b | 0x80000000u;
    return static_cast<uint64_t>(o) << 32 | static_cast<uint32_t>(~col);
}

template <typename T, bool kEntropy>
__global__ void __launch_bounds__(kThreads) logprob_fwd_kernel(LogprobFwd a, int64_t row0) {
    __shared__ Part parts[kThreads / 64];
    __shared__ uint64_t keys[kThreads / 64];
    const int64_t row = row0 + blockIdx.x;
    const T* x = static_cast<const T*>(a.x.p) + row * a.x.pitch;
    const float k = static_cast<float>(a.scale * kLog2e);
    Part p = {-INFINITY, 0.0f, 0.0f};
    for (int64_t c = threadIdx.x * kV; c < a.cols; c += kThreads * kV) {
        const int n = static_cast<int>(min(a.cols - c, int64_t{kV}));
        Vec<T> t;
        vload<false>(t, x + c, n);
        float v[kV];
        t.get(v);
        Part q = {-INFINITY, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            if (j >= n) v[j] = -INFINITY;
            q.m = fmaxf(q.m, v[j]);
        }
        const float r = anchor(q.m);
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const float u = (v[j] - r) * k, e = __builtin_amdgcn_exp2f(u);
            q.s += e;
            if constexpr (kEntropy) q.t += weighted(e, u);
        }
        p = join(p, q, k);
    }
    // join the lanes, then the waves
    for (int d = 1; d < 64; d <<= 1) {
        Part q = {__shfl_xor(p.m, d), __shfl_xor(p.s, d), __shfl_xor(p.t, d)};
        // both sides of a pair join in the same order
        p = threadIdx.x & d ? join(q, p, k) : join(p, q, k);
    }
    if ((threadIdx.x & 63) == 0) parts[threadIdx.x >> 6] = p;
    __syncthreads();
    p = parts[0];
    for (int i = 1; i < kThreads / 64; ++i) p = join(p, parts[i], k);
    const Row r = finish(p, a.scale);
    const auto logprob = [&](float v) {
        return r.empty() ? -INFINITY : fmaf(v, a.scale, -r.max) - r.logsum;
    };
    if (threadIdx.x == 0) {
        a.max[row] = r.max;
        a.logsum[row] = r.logsum;
        if (a.entropy) a.entropy[row] = r.entropy;
        if (a.tokens) {
            const int64_t tok = a.tokens[row];
            a.logprob[row] = tok >= 0 && tok < a.cols ? logprob(value(x + tok)) : 0.0f;
        }
    }
    // alternatives one by one: the largest key below the last one
    uint64_t last = ~uint64_t{0};
    for (int i = 0; i < a.top; ++i) {
        uint64_t best = 0;
        for (int64_t c = threadIdx.x; c < a.cols; c += kThreads) {
            const uint64_t key = rank_key(value(x + c), static_cast<uint32_t>(c));
            if (key < last && key > best) best = key;
        }
        for (int d = 1; d < 64; d <<= 1) {
            const uint64_t o = static_cast<uint64_t>(__shfl_xor(static_cast<unsigned long long>(best), d));
            best = o > best ? o : best;
        }
        __syncthreads();
        if ((threadIdx.x & 63) == 0) keys[threadIdx.x >> 6] = best;
        __syncthreads();
        best = keys[0];
        for (int w = 1; w < kThreads / 64; ++w) best = keys[w] > best ? keys[w] : best;
        last = best;
        if (threadIdx.x == 0) {
            const int64_t col = static_cast<uint32_t>(~static_cast<uint32_t>(best));
            a.top_token[row * a.top + i] = col;
            a.top_logprob[row * a.top + i] = logprob(value(x + col));
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) logprob_bwd_kernel(LogprobBwd a, int64_t row0, uint32_t across) {
    const int64_t row = row0 + blockIdx.x / across;
    const int64_t c = (static_cast<int64_t>(blockIdx.x % across) * kThreads + threadIdx.x) * kV;
    const int n = static_cast<int>(max(min(a.cols - c, int64_t{kV}), int64_t{0}));
    const T* x = static_cast<const T*>(a.x.p) + row * a.x.pitch;
    T* y = static_cast<T*>(a.dx.p) + row * a.dx.pitch;
    const float mx = a.max[row], logsum = a.logsum[row];
    const int64_t tok = a.dl ? a.tokens[row] : -1;
    const float dl = tok >= 0 && tok < a.cols ? a.dl[row] : 0.0f, dh = a.dh ? a.dh[row] : 0.0f;
    float v[kV] = {};
    if ((dl != 0.0f || dh != 0.0f) && !(mx == -INFINITY && logsum == 0.0f)) {
        const float H = a.dh ? a.entropy[row] : 0.0f;
        Vec<T> t;
        vload<false>(t, x + c, n);
        t.get(v);
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const float lp = fmaf(v[j], a.scale, -mx) - logsum;
            const float p = __builtin_amdgcn_exp2f(lp * static_cast<float>(kLog2e));
            float d = -dl * p;
            if (a.dh) d -= dh * (weighted(p, lp) + p * H);
            if (c + j == tok) d += dl;
            v[j] = d * a.scale;
        }
    }
    put8(y + c, v, n);
}

constexpr int64_t kMaxBlocks = int64_t{1} << 22;  // of 256 threads: a grid's threads fit 32 bits

}  // namespace

int64_t logprob_workspace_floats(int64_t, int64_t, int32_t) { return 0; }

hipError_t launch_logprob_forward(const LogprobFwd& a, hipStream_t stream) {
    for (int64_t r0 = 0; r0 < a.rows; r0 += kMaxBlocks) {
        const dim3 grid(static_cast<uint32_t>(std::min(a.rows - r0, kMaxBlocks)));
        if (a.bf16) {
            if (a.entropy) logprob_fwd_kernel<uint16_t, true><<<grid, kThreads, 0, stream>>>(a, r0);
            else logprob_fwd_kernel<uint16_t, false><<<grid, kThreads, 0, stream>>>(a, r0);
        } else {
            if (a.entropy) logprob_fwd_kernel<float, true><<<grid, kThreads, 0, stream>>>(a, r0);
            else logprob_fwd_kernel<float, false><<<grid, kThreads, 0, stream>>>(a, r0);
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_logprob_backward(const LogprobBwd& a, hipStream_t stream) {
    const int64_t across = (a.cols + kThreads * kV - 1) / (kThreads * kV);
    const int64_t rows = std::max<int64_t>(1, kMaxBlocks / across);
    for (int64_t r0 = 0; r0 < a.rows; r0 += rows) {
        const dim3 grid(static_cast<uint32_t>(std::min(a.rows - r0, rows) * across));
        if (a.bf16) logprob_bwd_kernel<uint16_t><<<grid, kThreads, 0, stream>>>(a, r0, static_cast<uint32_t>(across));
        else logprob_bwd_kernel<float><<<grid, kThreads, 0, stream>>>(a, r0, static_cast<uint32_t>(across));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace fsdp
