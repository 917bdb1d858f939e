// norm_backward.h -- the norms' backward pass for rows that fit in registers; compiled for each
// activation type and load policy in norm_backward_*.hip.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "layer.h"
#include "layer_dev.h"

#pragma clang fp contract(fast)

namespace fsdp {
namespace {

// Vectors of 4 columns: the column sums, a row's values and the next row's loads are all in
// registers, and narrower vectors leave fewer of them unused.
constexpr int kQ = 4;
typedef uint32_t u1e __attribute__((aligned(1)));
typedef uint32_t u2h __attribute__((ext_vector_type(2), aligned(2)));
template <typename T> struct Quad;
template <> struct Quad<uint16_t> {
    u2 r;
    template <bool kNt> __device__ void load(const uint16_t* p) {
        r = kNt ? __builtin_nontemporal_load((const u2h*)p) : *(const u2h*)p;
    }
    // drops the first k elements, zeros behind the last
    __device__ void drop(int k) {
        r = __builtin_bit_cast(u2, __builtin_bit_cast(uint64_t, r) >> (16 * k));
    }
    __device__ void keep(bool inside) { r = inside ? r : u2{0u, 0u}; }
    __device__ void get(float* v) const {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            v[2 * j] = __builtin_bit_cast(float, r[j] << 16);
            v[2 * j + 1] = __builtin_bit_cast(float, r[j] & 0xFFFF0000u);
        }
    }
    __device__ static void put(uint16_t* p, const float* v, int n) {
        u2 r;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            r[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{v[2 * j], v[2 * j + 1]}), bf2));
        if (n >= kQ) {
            __builtin_nontemporal_store(r, (u2h*)p);
            return;
        }
#pragma unroll
        for (int j = 0; j < kQ; ++j)
            if (j < n) p[j] = static_cast<uint16_t>(r[j >> 1] >> (16 * (j & 1)));
    }
};
template <> struct Quad<float> {
    f4 r;
    template <bool kNt> __device__ void load(const float* p) {
        r = kNt ? __builtin_nontemporal_load((const f4e*)p) : *(const f4e*)p;
    }
    __device__ void drop(int k) {
        if (k & 1) r = f4{r[1], r[2], r[3], 0.0f};
        if (k & 2) r = f4{r[2], r[3], 0.0f, 0.0f};
    }
    __device__ void keep(bool inside) { r = inside ? r : f4{0.0f, 0.0f, 0.0f, 0.0f}; }
    __device__ void get(float* v) const {
#pragma unroll
        for (int j = 0; j < kQ; ++j) v[j] = r[j];
    }
    __device__ static void put(float* p, const float* v, int n) {
        if (n >= kQ) {
            __builtin_nontemporal_store(f4{v[0], v[1], v[2], v[3]}, (f4e*)p);
            return;
        }
#pragma unroll
        for (int j = 0; j < kQ; ++j)
            if (j < n) p[j] = v[j];
    }
};
// 4 values of a parameter, 0 outside its n.
__device__ __forceinline__ f4 param4(const void* w, bool bf16, int64_t c, int n) {
    f4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (bf16) {
        const uint16_t* p = static_cast<const uint16_t*>(w) + c;
        if (n >= kQ) {
            const u2 r = *(const u2h*)p;
            v = f4{__builtin_bit_cast(float, r[0] << 16), __builtin_bit_cast(float, r[0] & 0xFFFF0000u),
                   __builtin_bit_cast(float, r[1] << 16), __builtin_bit_cast(float, r[1] & 0xFFFF0000u)};
        } else {
            for (int j = 0; j < n; ++j) v[j] = __builtin_bit_cast(float, uint32_t{p[j]} << 16);
        }
    } else {
        const float* p = static_cast<const float*>(w) + c;
        if (n >= kQ) v = *(const f4e*)p;
        else
            for (int j = 0; j < n; ++j) v[j] = p[j];
    }
    return v;
}
// Partial sums, which the next kernel reads.
__device__ __forceinline__ void keep(float* p, const float* v, int n) {
    if (n >= kQ) {
        *(f4e*)p = f4{v[0], v[1], v[2], v[3]};
        return;
    }
#pragma unroll
    for (int j = 0; j < kQ; ++j)
        if (j < n) p[j] = v[j];
}

// p + i as a scalar address and an unsigned 32-bit offset, which the memory instructions add.
template <typename T>
__device__ __forceinline__ const T* from(const T* p, uint32_t i) {
    return reinterpret_cast<const T*>(reinterpret_cast<const char*>(p) + i * static_cast<uint32_t>(sizeof(T)));
}
template <typename T>
__device__ __forceinline__ T* from(T* p, uint32_t i) {
    return reinterpret_cast<T*>(reinterpret_cast<char*>(p) + i * static_cast<uint32_t>(sizeof(T)));
}

// Where the input comes from.
enum { kTensor = 0, kE4m3 = 1, kInt8 = 2 };

// What a row's backward pass reads, in flight.
template <typename T, int kSrc, bool kRes, bool kNt, int kN>
struct BwdRow {
    Quad<T> dy[kN], x[kSrc == kTensor ? kN : 1], r[kRes ? kN : 1];
    uint32_t q[kSrc == kTensor ? 1 : kN], byte[kSrc == kTensor ? 1 : kN];
    float mean, rstd;
    // at[i]: the column that vector i is read from, group[i]: its scale.  A row past the last
    // is not branched around, which would have the compiler wait for loads that it cannot count:
    // the last row's first columns are read instead, by all lanes at once.
    __device__ __forceinline__ void load(const NormBwd& a, int64_t row, const uint32_t* at, const uint32_t* group) {
        const uint32_t mask = row < a.rows ? ~0u : 0u;
        row = row < a.rows ? row : a.rows - 1;
        const T* dp = static_cast<const T*>(a.dy.p) + row * a.dy.pitch;
        const T* xp = static_cast<const T*>(a.x.p) + row * a.x.pitch;
        const T* rp = static_cast<const T*>(a.dres.p) + row * a.dres.pitch;
        const uint8_t* qp = a.ckpt.codes + row * a.ckpt.code_pitch;
        const uint8_t* sp = a.ckpt.scales + row * a.ckpt.scale_pitch;
        rstd = a.rstd[row];
        mean = (a.rms ? a.rstd : a.mean)[row];   // no branch between the loads either
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const uint32_t c = at[i] & mask;   // unsigned: added to a scalar address as it is
            dy[i].template load<kNt>(from(dp, c));
            if constexpr (kSrc != kTensor) {
                q[i] = *(const u1e*)from(qp, c);
                byte[i] = *from(sp, group[i] & mask);
            } else {
                x[i].template load<kNt>(from(xp, c));
            }
            if constexpr (kRes) r[i].template load<kNt>(from(rp, c));
        }
    }
    __device__ __forceinline__ void drop(int i, int k) {
        dy[i].drop(k);
        if constexpr (kSrc != kTensor) q[i] >>= 8 * k;
        else x[i].drop(k);
        if constexpr (kRes) r[i].drop(k);
    }
    // zeros where the vector lies outside its row
    __device__ __forceinline__ void keep(int i, bool inside) {
        dy[i].keep(inside);
        x[i].keep(inside);
    }
    __device__ __forceinline__ void input(int i, float* v) const {
        if constexpr (kSrc == kTensor) x[i].get(v);
        else decode4<kSrc == kInt8>(q[i], byte[i], v);
    }
};

// A workgroup is 8 waves, or the 16 of a row that takes as many.
template <int kT> constexpr int bwd_threads() { return kT < 512 ? 512 : kT; }
// Waves a SIMD (four of them a CU) of the workgroups that the launch counts on being resident.
template <typename T, int kSrc, bool kRes, int kT, int kN>
constexpr int bwd_waves() {
    return norm_bwd_resident(sizeof(T) == 2, kSrc != kTensor, kRes, kT, kN) * bwd_threads<kT>() / 256;
}

// Row groups of kT threads, kN vectors a thread, take rows g, g + groups, ... with the next row's
// loads in flight, and keep the column sums of all their rows in registers; a workgroup adds up
// its groups' sums and writes one partial row of each.  One pass over the data: dy and the input
// are read once, and dx (and y) written once, with the row's two means between.
// Bound by HBM, at the rate of a grid that stays resident (loads wait behind stores, and the
// workgroups read and write in step).  This kernel alone, in a kernel trace: 8192 x 12288 bf16 107 us and 604 MB,
// 5.6 TB/s; 32768 x 1024 from int8 with y 41 us and 236 MB, 5.7; 24 and 17 vector instructions an element take
// half that time at most.  More rows in flight do not help (two ahead: 2% slower at the latter
// size), nor do other orders of the rows over the XCDs (within 1%).  Weight and bias lie in LDS: read as
// memory, they would make a row wait for the next one's loads, which return in order.  kWhole:
// the columns are a multiple of 4; else the vector that the row's end cuts is read from the row's
// last 4 columns.  A vector outside the row reads its first columns, is left out of the sums
// and not stored.
template <typename T, int kSrc, bool kRes, bool kNt, int kT, int kN, bool kWhole>
__global__ void __launch_bounds__(bwd_threads<kT>(), (bwd_waves<T, kSrc, kRes, kT, kN>())) norm_bwd_kernel(NormBwd a, float* partial) {
    constexpr int kW = bwd_threads<kT>(), kRows = kW / kT;
    __shared__ f4 lw[kT * kN], lb[kT * kN];
    __shared__ float lds[2][2 * (kW / 64)];
    const int t = threadIdx.x % kT;
    const int mine = kRows > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / kT) : 0;
    const int64_t groups = static_cast<int64_t>(gridDim.x) * kRows;
    int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + mine;
    const int cols = static_cast<int>(a.cols);
    const float inv = 1.0f / static_cast<float>(cols);
    const bool again = a.y.p != nullptr;
    uint32_t at[kN], group[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        const int c = (t + i * kT) * kQ;
        at[i] = static_cast<uint32_t>(c < cols ? (kWhole ? c : min(c, cols - kQ)) : 0);
        group[i] = static_cast<uint32_t>(c < cols ? c / kCkptGroup : 0);
    }
    typedef BwdRow<T, kSrc, kRes, kNt, kN> Row;
    Row even, odd;
    even.load(a, row, at, group);
    for (int v = threadIdx.x; v < kT * kN; v += kW) {
        lw[v] = param4(a.weight, a.param_bf16, v * kQ, cols - v * kQ);
        if (again && a.bias) lb[v] = param4(a.bias, a.param_bf16, v * kQ, cols - v * kQ);
        else lb[v] = f4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    __syncthreads();
    float sw[kN][kQ] = {}, sb[kN][kQ] = {};
    // Only a thread's last vector can lie outside the row; what it read must not reach the row's sums (an
    // infinity times its weight of 0 is NaN).  The loads are cleared, or the sums from before it kept, by
    // what spills less in rows of four vectors: 4096 x 14336 with residual from the tensor 123 us cleared,
    // 150 kept; without 80 and 77, from e4m3 83 and 73, from int8 95 and 73.
    constexpr bool kClear = kSrc == kTensor && kRes;

    // One row of each group; `half` alternates, for a row's sums must not overwrite those that a
    // slower wave still reads for the row before.
    const auto step = [&](Row& now, int half) __attribute__((always_inline)) {
        // groups of several waves meet at the barrier also without a row
        const bool live = kT == 64 || kRows == 1 || row < a.rows;
        const float rstd = now.rstd, mean = a.rms ? 0.0f : now.mean;
        float s0 = 0.0f, s1 = 0.0f, xh[kN][kQ], gw[kN][kQ];
        if (live) {
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                const int c = (t + i * kT) * kQ;
                if constexpr (!kWhole) now.drop(i, c < cols ? c - static_cast<int>(at[i]) : 0);
                if constexpr (kClear) {
                    if (i + 1 == kN) now.keep(i, c < cols);
                }
                float g[kQ];
                now.input(i, xh[i]);
                now.dy[i].get(g);
                const f4 w = lw[t + i * kT];
                const float t0 = s0, t1 = s1;
#pragma unroll
                for (int j = 0; j < kQ; ++j) {
                    xh[i][j] = (xh[i][j] - mean) * rstd;
                    sw[i][j] += g[j] * xh[i][j];
                    sb[i][j] += g[j];
                    gw[i][j] = g[j] * w[j];
                    s0 += gw[i][j];
                    s1 += gw[i][j] * xh[i][j];
                }
                if (!kClear && i + 1 == kN) {
                    s0 = c < cols ? s0 : t0;
                    s1 = c < cols ? s1 : t1;
                }
            }
        } else {
            // Loads that nothing uses have to be waited for somewhere before their registers are
            // loaded again; left to the compiler, that is before every row's loads, where the wait
            // would be for the row's stores as well.
            __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0)
        }
        __builtin_amdgcn_s_setprio(2);
        s0 = wave_sum(s0);
        s1 = wave_sum(s1);
        if constexpr (kT > 64) {
            if ((threadIdx.x & 63) == 0) {
                lds[half][2 * (threadIdx.x >> 6)] = s0;
                lds[half][2 * (threadIdx.x >> 6) + 1] = s1;
            }
            __syncthreads();
            // every lane takes one wave's sums, and lanes next to each other add up
            constexpr int kWaves = kT / 64;
            const int l = 2 * (mine * kWaves + (threadIdx.x & (kWaves - 1)));
            s0 = add_lanes<kWaves>(lds[half][l]);
            s1 = add_lanes<kWaves>(lds[half][l + 1]);
        }
        if (!live) return;
        // dx = rstd gw - (rstd c2) xh - rstd c1
        const float c1 = a.rms ? 0.0f : s0 * inv * rstd, c2 = s1 * inv * rstd;
        T* dxp = static_cast<T*>(a.dx.p) + row * a.dx.pitch;
        T* yp = static_cast<T*>(a.y.p) + row * a.y.pitch;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int c = (t + i * kT) * kQ, n = kWhole ? kQ : cols - c;
            float d[kQ], r[kQ] = {};
            if constexpr (kRes) now.r[i].get(r);
#pragma unroll
            for (int j = 0; j < kQ; ++j) d[j] = gw[i][j] * rstd - (xh[i][j] * c2 + c1) + r[j];
            if (c < cols) Quad<T>::put(from(dxp, static_cast<uint32_t>(c)), d, n);
            if (again) {
                const f4 w = lw[t + i * kT], b = lb[t + i * kT];
#pragma unroll
                for (int j = 0; j < kQ; ++j) d[j] = xh[i][j] * w[j] + b[j];
                if (c < cols) Quad<T>::put(from(yp, static_cast<uint32_t>(c)), d, n);
            }
        }
    };
    // Groups of several waves all go on while the workgroup's first one has a row.  A wave at its loads
    // goes before the others, then those between a row's sums and its stores (1-2% on 148-400 MB).
    const int64_t behind = kT == 64 ? 0 : mine;
    while (row - behind < a.rows) {
        __builtin_amdgcn_s_setprio(3);
        odd.load(a, row + groups, at, group);
        __builtin_amdgcn_s_setprio(0);
        step(even, 0);
        row += groups;
        if (row - behind >= a.rows) break;
        __builtin_amdgcn_s_setprio(3);
        even.load(a, row + groups, at, group);
        __builtin_amdgcn_s_setprio(0);
        step(odd, 1);
        row += groups;
    }
    // the workgroup's row groups add up in LDS, one after another
    if constexpr (kRows > 1) {
        for (int v = 0; v < kRows; ++v) {
            __syncthreads();
            if (mine == v) {
#pragma unroll
                for (int i = 0; i < kN; ++i) {
                    const int l = t + i * kT;
                    f4 w = {sw[i][0], sw[i][1], sw[i][2], sw[i][3]}, b = {sb[i][0], sb[i][1], sb[i][2], sb[i][3]};
                    if (v) {
                        w += lw[l];
                        b += lb[l];
                    }
                    lw[l] = w;
                    lb[l] = b;
                }
            }
        }
        __syncthreads();
    }
    // and all of its threads write them
    float* out = partial + static_cast<int64_t>(blockIdx.x) * 2 * cols;
    if constexpr (kRows > 1) {
        for (int v = threadIdx.x; v < kT * kN; v += kW) {
            const f4 w = lw[v], b = lb[v];
            const float ws[kQ] = {w[0], w[1], w[2], w[3]}, bs[kQ] = {b[0], b[1], b[2], b[3]};
            const int n = cols - v * kQ;
            if (a.dweight.p) keep(out + v * kQ, ws, n);
            if (a.dbias.p) keep(out + cols + v * kQ, bs, n);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int c = (t + i * kT) * kQ;
            if (a.dweight.p) keep(out + c, sw[i], cols - c);
            if (a.dbias.p) keep(out + cols + c, sb[i], cols - c);
        }
    }
}

template <typename T, int kSrc, bool kRes, bool kNt, int kT, int kN>
void norm_bwd_run(const NormBwd& a, float* partial, uint32_t blocks, hipStream_t stream) {
    if (a.cols % kQ == 0) norm_bwd_kernel<T, kSrc, kRes, kNt, kT, kN, true><<<blocks, bwd_threads<kT>(), 0, stream>>>(a, partial);
    else norm_bwd_kernel<T, kSrc, kRes, kNt, kT, kN, false><<<blocks, bwd_threads<kT>(), 0, stream>>>(a, partial);
}
template <typename T, int kSrc, bool kRes, bool kNt>
void norm_bwd_shaped(const NormBwd& a, float* partial, uint32_t blocks, hipStream_t stream) {
    const BwdShape s = norm_bwd_shape(a.cols);
    switch (s.threads + s.vectors) {
#define FSDP_SHAPE(kT, kN) case kT + kN: return norm_bwd_run<T, kSrc, kRes, kNt, kT, kN>(a, partial, blocks, stream)
        FSDP_SHAPE(64, 1);
        FSDP_SHAPE(64, 2);
        FSDP_SHAPE(64, 3);
        FSDP_SHAPE(128, 2);
        FSDP_SHAPE(128, 3);
        FSDP_SHAPE(256, 2);
        FSDP_SHAPE(256, 3);
        FSDP_SHAPE(512, 2);
        FSDP_SHAPE(512, 3);
        FSDP_SHAPE(1024, 2);
        FSDP_SHAPE(1024, 3);
        FSDP_SHAPE(1024, 4);
#undef FSDP_SHAPE
    }
}
template <typename T, int kSrc, bool kNt>
void norm_bwd_res(const NormBwd& a, float* partial, uint32_t blocks, hipStream_t stream) {
    if (a.dres.p) norm_bwd_shaped<T, kSrc, true, kNt>(a, partial, blocks, stream);
    else norm_bwd_shaped<T, kSrc, false, kNt>(a, partial, blocks, stream);
}
template <typename T, bool kNt>
void norm_bwd_rows(const NormBwd& a, float* partial, uint32_t blocks, hipStream_t stream) {
    if (!a.ckpt.codes) norm_bwd_res<T, kTensor, kNt>(a, partial, blocks, stream);
    else if (a.ckpt.int8) norm_bwd_res<T, kInt8, kNt>(a, partial, blocks, stream);
    else norm_bwd_res<T, kE4m3, kNt>(a, partial, blocks, stream);
}

}  // namespace
}  // namespace fsdp
