// layer.hip -- HIP kernels of the layer operators for CDNA4 (gfx950): 8-bit activation
// checkpoints, LayerNorm / RMSNorm and the MLP activation, forward and backward.
//
// All of them stream their operands once; what bounds them is HBM.  Every lane owns vectors of
// 8 neighbouring columns (one 16-byte load of bf16, two of fp32, 8 bytes of codes), four lanes
// of a quad one group of 32 columns with one scale.  Rows may start at any element: global
// loads and stores of several dwords work at any address, so odd pitches and widths take the
// same path, and only the vector that the row's end cuts goes element by element.
// Sums, statistics and the arithmetic between load and store are binary32; a result is rounded
// once, when it is stored.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "layer.h"

// Nothing here is compared bit for bit with separately rounded steps (scaling by powers of two
// is exact either way), so multiply-adds may be fused.
#pragma clang fp contract(fast)

namespace fsdp {
namespace {

constexpr int kV = 8;           // columns of a lane's vector
constexpr int kThreads = 256;   // workgroup of the kernels that walk tiles

typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
// the same at any element's alignment
typedef uint32_t u4e __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u2e __attribute__((ext_vector_type(2), aligned(1)));
typedef float f4e __attribute__((ext_vector_type(4), aligned(4)));

// ---------------------------------------------------------------------------
// vectors of 8 columns: raw registers, and their values
// ---------------------------------------------------------------------------
template <typename T> struct Vec;
template <> struct Vec<uint16_t> {
    u4 r;
    __device__ void load(const uint16_t* p) { r = __builtin_nontemporal_load((const u4e*)p); }
    __device__ void load_part(const uint16_t* p, int n) {
        r = u4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int j = 0; j < kV; ++j)
            if (j < n) r[j >> 1] |= uint32_t{p[j]} << (16 * (j & 1));
    }
    __device__ void zero() { r = u4{0u, 0u, 0u, 0u}; }
    __device__ void get(float* v) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __builtin_bit_cast(float, r[j] << 16);
            v[2 * j + 1] = __builtin_bit_cast(float, r[j] & 0xFFFF0000u);
        }
    }
    // round to nearest even, NaN kept NaN (v_cvt_pk_bf16_f32)
    __device__ void set(const float* v) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            r[j] = __builtin_bit_cast(uint32_t,
                                      __builtin_convertvector((f2{v[2 * j], v[2 * j + 1]}), bf2));
    }
    __device__ void store(uint16_t* p) const { __builtin_nontemporal_store(r, (u4e*)p); }
    __device__ void store_part(uint16_t* p, int n) const {
#pragma unroll
        for (int j = 0; j < kV; ++j)
            if (j < n) p[j] = static_cast<uint16_t>(r[j >> 1] >> (16 * (j & 1)));
    }
};
template <> struct Vec<float> {
    f4 r[2];
    __device__ void load(const float* p) {
        r[0] = __builtin_nontemporal_load((const f4e*)p);
        r[1] = __builtin_nontemporal_load((const f4e*)(p + 4));
    }
    __device__ void load_part(const float* p, int n) {
        zero();
#pragma unroll
        for (int j = 0; j < kV; ++j)
            if (j < n) r[j >> 2][j & 3] = p[j];
    }
    __device__ void zero() { r[0] = r[1] = f4{0.0f, 0.0f, 0.0f, 0.0f}; }
    __device__ void get(float* v) const {
#pragma unroll
        for (int j = 0; j < kV; ++j) v[j] = r[j >> 2][j & 3];
    }
    __device__ void set(const float* v) {
#pragma unroll
        for (int j = 0; j < kV; ++j) r[j >> 2][j & 3] = v[j];
    }
    __device__ void store(float* p) const {
        __builtin_nontemporal_store(r[0], (f4e*)p);
        __builtin_nontemporal_store(r[1], (f4e*)(p + 4));
    }
    __device__ void store_part(float* p, int n) const {
#pragma unroll
        for (int j = 0; j < kV; ++j)
            if (j < n) p[j] = r[j >> 2][j & 3];
    }
};

// n: columns of this vector inside the row (8 or more: whole; 0 or less: none).
template <typename T>
__device__ __forceinline__ void vload(Vec<T>& v, const T* p, int n) {
    if (n >= kV) v.load(p);
    else if (n > 0) v.load_part(p, n);
    else v.zero();
}
template <typename T>
__device__ __forceinline__ void vstore(const Vec<T>& v, T* p, int n) {
    if (n >= kV) v.store(p);
    else if (n > 0) v.store_part(p, n);
}
template <typename T>
__device__ __forceinline__ void put8(T* p, const float* f, int n) {
    Vec<T> v;
    v.set(f);
    vstore(v, p, n);
}
// 8 values of a parameter (weight, bias): cached loads, every row reads them again.
__device__ __forceinline__ void param8(const void* w, bool bf16, int64_t c, int n, float* v) {
#pragma unroll
    for (int j = 0; j < kV; ++j) v[j] = 0.0f;
    if (n <= 0) return;
    if (bf16) {
        const uint16_t* p = static_cast<const uint16_t*>(w) + c;
        if (n >= kV) {
            Vec<uint16_t> t;
            t.r = *(const u4e*)p;
            t.get(v);
        } else {
            for (int j = 0; j < kV; ++j)
                if (j < n) v[j] = __builtin_bit_cast(float, uint32_t{p[j]} << 16);
        }
    } else {
        const float* p = static_cast<const float*>(w) + c;
        if (n >= kV) {
            const f4 a = *(const f4e*)p, b = *(const f4e*)(p + 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) { v[j] = a[j]; v[4 + j] = b[j]; }
        } else {
            for (int j = 0; j < kV; ++j)
                if (j < n) v[j] = p[j];
        }
    }
}

// ---------------------------------------------------------------------------
// 8-bit groups
// ---------------------------------------------------------------------------
// A group's scale is 2^s, held as the byte s + 127.  s is the smallest power at which the
// group's largest magnitude still rounds to a value the codes have: e4m3 up to 464 (448 is
// the largest code; 464, halfway to the next step, goes to the even one below), integers below
// 127.5.  With the magnitude 1.m x 2^e that is s = e - 8, one more where 1.m > 464/256, or
// s = e - 6, one more where 1.m >= 127.5/64; never below -124 (e4m3: its smallest step is then
// bf16's smallest) or -127 (integers, the byte's end).  Dividing by a power of two is exact, so
// a code is off by at most half its step, and every value a code stands for is a bf16 number.
// Byte 255: the group held an infinity or a NaN, and reads back as NaN throughout.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits, bool int8) {
    const uint32_t e = amax_bits >> 23, m = amax_bits & 0x7FFFFFu;
    if (e == 255u) return 255u;
    const int s = int8 ? static_cast<int>(e) - 6 + (m >= 0x7F0000u) : static_cast<int>(e) - 8 + (m > 0x680000u);
    return static_cast<uint32_t>(max(s, int8 ? 0 : 3));
}
__device__ __forceinline__ float scale_value(uint32_t b) {
    uint32_t bits = b << 23;
    if (b == 0u) bits = 0x00400000u;   // 2^-127, a subnormal
    if (b == 255u) bits = 0x7FC00000u;
    return __builtin_bit_cast(float, bits);
}
template <int kCtrl>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
    return __builtin_amdgcn_update_dpp(0u, x, kCtrl, 0xF, 0xF, true);
}
constexpr int kQuadXor1 = 0xB1, kQuadXor2 = 0x4E;   // quad_perm [1,0,3,2], [2,3,0,1]
constexpr int kHalfMirror = 0x141, kMirror = 0x140;

// Codes of 8 columns whose group is the calling lane's quad; every lane of the quad calls it.
__device__ __forceinline__ u2 encode8(const float* v, bool int8, uint32_t* byte) {
    uint32_t a = 0;
#pragma unroll
    for (int j = 0; j < kV; ++j) a = max(a, __builtin_bit_cast(uint32_t, v[j]) & 0x7FFFFFFFu);
    a = max(a, dpp<kQuadXor1>(a));
    a = max(a, dpp<kQuadXor2>(a));
    const uint32_t b = scale_byte(a, int8);
    *byte = b;
    u2 q = {0u, 0u};
    if (b == 255u) return q;
    const float inv = __builtin_bit_cast(float, (254u - b) << 23);   // 2^-s, a normal number
    if (int8) {
        // 1.5 x 2^23 + x 2^-s rounds to the nearest integer, ties to even, and its low byte is
        // that integer in two's complement
        uint32_t t[kV];
#pragma unroll
        for (int j = 0; j < kV; ++j)
            t[j] = __builtin_bit_cast(uint32_t, __builtin_fmaf(v[j], inv, 12582912.0f));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t lo = __builtin_amdgcn_perm(t[4 * h + 1], t[4 * h], 0x0C0C0400u);
            const uint32_t hi = __builtin_amdgcn_perm(t[4 * h + 3], t[4 * h + 2], 0x04000C0Cu);
            q[h] = lo | hi;
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            int w = 0;
            w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h] * inv, v[4 * h + 1] * inv, w, false);
            w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2] * inv, v[4 * h + 3] * inv, w, true);
            q[h] = static_cast<uint32_t>(w);
        }
    }
    return q;
}
__device__ __forceinline__ void decode8(u2 q, uint32_t byte, bool int8, float* v) {
    const float s = scale_value(byte);
    if (int8) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t u = q[h] ^ 0x80808080u;   // offset by 128
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[4 * h + j] = (static_cast<float>((u >> (8 * j)) & 0xFFu) - 128.0f) * s;
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const f2 a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(q[h]), false);
            const f2 b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(q[h]), true);
            v[4 * h] = a[0] * s;
            v[4 * h + 1] = a[1] * s;
            v[4 * h + 2] = b[0] * s;
            v[4 * h + 3] = b[1] * s;
        }
    }
}
__device__ __forceinline__ u2 code_load(const uint8_t* p, int n) {
    if (n >= kV) return __builtin_nontemporal_load((const u2e*)p);
    u2 q = {0u, 0u};
#pragma unroll
    for (int j = 0; j < kV; ++j)
        if (j < n) q[j >> 2] |= uint32_t{p[j]} << (8 * (j & 3));
    return q;
}
__device__ __forceinline__ void code_store(uint8_t* p, u2 q, int n) {
    if (n >= kV) {
        __builtin_nontemporal_store(q, (u2e*)p);
        return;
    }
#pragma unroll
    for (int j = 0; j < kV; ++j)
        if (j < n) p[j] = static_cast<uint8_t>(q[j >> 2] >> (8 * (j & 3)));
}
// Codes and scale of the vector at column c (n of its columns inside the row) of a row.
__device__ __forceinline__ void pack8(const CkptRows& q, int64_t row, int64_t c, int n,
                                      const float* v) {
    uint32_t byte;
    const u2 code = encode8(v, q.int8 != 0, &byte);
    code_store(q.codes + row * q.code_pitch + c, code, n);
    if (n > 0 && (threadIdx.x & 3) == 0)
        q.scales[row * q.scale_pitch + c / kCkptGroup] = static_cast<uint8_t>(byte);
}

// ---------------------------------------------------------------------------
// sums over a wave and a workgroup
// ---------------------------------------------------------------------------
__device__ __forceinline__ float wave_sum(float x) {
    const auto add = [](float a, uint32_t b) { return a + __builtin_bit_cast(float, b); };
    const auto bits = [](float a) { return __builtin_bit_cast(uint32_t, a); };
    x = add(x, dpp<kQuadXor1>(bits(x)));
    x = add(x, dpp<kQuadXor2>(bits(x)));
    x = add(x, dpp<kHalfMirror>(bits(x)));
    x = add(x, dpp<kMirror>(bits(x)));
    const auto r = __builtin_amdgcn_permlane16_swap(bits(x), bits(x), false, false);
    x = __builtin_bit_cast(float, static_cast<uint32_t>(r[0])) +
        __builtin_bit_cast(float, static_cast<uint32_t>(r[1]));
    const auto t = __builtin_amdgcn_permlane32_swap(bits(x), bits(x), false, false);
    return __builtin_bit_cast(float, static_cast<uint32_t>(t[0])) +
           __builtin_bit_cast(float, static_cast<uint32_t>(t[1]));
}
// Sum over the workgroup, the same in every thread.  `lds` holds one float per wave and is
// free again only after the next barrier.
template <int kT>
__device__ __forceinline__ float group_sum(float x, float* lds) {
    x = wave_sum(x);
    if constexpr (kT > 64) {
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
        __syncthreads();
        x = lds[0];
#pragma unroll
        for (int i = 1; i < kT / 64; ++i) x += lds[i];
    }
    return x;
}

// ---------------------------------------------------------------------------
// activations
// ---------------------------------------------------------------------------
enum { kNone = 0, kRelu = 1, kGelu = 2, kGeluTanh = 3, kSilu = 4 };

// e^x by the hardware's 2^x: off by |x| 2^-24 and one rounding, relative.
__device__ __forceinline__ float fast_exp(float x) {
    return __builtin_amdgcn_exp2f(x * 1.44269504088896341f);
}
// f(h) and f'(h).
template <int kF>
__device__ __forceinline__ void activate(float h, float* y, float* d) {
    if constexpr (kF == kNone) {
        *y = h;
        *d = 1.0f;
    } else if constexpr (kF == kRelu) {
        *y = h <= 0.0f ? 0.0f : h;                       // NaN stays NaN
        *d = h > 0.0f ? 1.0f : (h <= 0.0f ? 0.0f : h);
    } else if constexpr (kF == kSilu) {
        const float s = __builtin_amdgcn_rcpf(1.0f + fast_exp(-h));
        *y = h * s;
        *d = s * (1.0f + h * (1.0f - s));
    } else if constexpr (kF == kGeluTanh) {
        // (1 + tanh u) / 2 = 1 / (1 + e^-2u), u = sqrt(2/pi) (h + 0.044715 h^3)
        constexpr float a = 0.79788456080286536f, c = 0.044715f;
        // h^2 is capped where the logistic function is flat, so that no product overflows to 0 x inf;
        // a NaN comes through h
        const float h2 = __builtin_fminf(h * h, 1000.0f);
        const float s = __builtin_amdgcn_rcpf(1.0f + fast_exp(-2.0f * a * h * (1.0f + c * h2)));
        *y = h * s;
        *d = s + (s * (1.0f - s) * h) * (2.0f * a + 6.0f * a * c * h2);
    } else {
        // Phi(h) by Hastings' rational form of erfc (Abramowitz and Stegun 7.1.26, absolute error
        // 1.5e-7): erfc(z) = t (a1 + t (a2 + ...)) e^-z^2, t = 1 / (1 + p z), z = |h| / sqrt 2;
        // the exponential is also the density's, which f' needs.
        const float z = __builtin_fabsf(h) * 0.70710678118654752f;
        const float t = __builtin_amdgcn_rcpf(1.0f + 0.3275911f * z);
        const float e = fast_exp(-z * z);
        const float poly = t * (0.254829592f + t * (-0.284496736f + t * (1.421413741f + t * (-1.453152027f + t * 1.061405429f))));
        const float q = 0.5f * poly * e;                 // Phi(-|h|)
        const float phi = h < 0.0f ? q : 1.0f - q;
        *y = h * phi;
        *d = phi + h * e * 0.39894228040143268f;
    }
}

// ---------------------------------------------------------------------------
// tiles: 2^k vectors wide, kThreads >> k rows high
// ---------------------------------------------------------------------------
// A workgroup covers one tile (or walks down a column of them); wide rows give tiles of one
// row, narrow ones of many, so that a wave's loads stay whole lines either way.
struct Tiles {
    int32_t k;        // log2 of a tile's vectors
    uint32_t across;  // tiles across a row
    int64_t down;     // tiles down the rows
};
Tiles plan_tiles(int64_t rows, int64_t cols) {
    const int64_t nv = (cols + kCkptGroup - 1) / kCkptGroup * (kCkptGroup / kV);
    int best = 2;
    while (best < 5 && (int64_t{1} << best) < nv) ++best;
    if (best == 5) {
        // of 32, 64, 128 and 256 vectors the width that leaves the fewest lanes idle
        for (int k = 6; k <= 8; ++k) {
            const auto padded = [&](int b) { return (((nv - 1) >> b) + 1) << b; };
            if (padded(k) <= padded(best)) best = k;
        }
    }
    Tiles t;
    t.k = best;
    t.across = static_cast<uint32_t>(((nv - 1) >> best) + 1);
    const int64_t high = kThreads >> best;
    t.down = (rows + high - 1) / high;
    return t;
}

// y = f(x) and the checkpoint of x, one tile per workgroup.
template <typename T, int kF>
__global__ void __launch_bounds__(kThreads) act_fwd_kernel(ActFwd a, int k, uint32_t across) {
    const uint32_t down = blockIdx.x / across, tile = blockIdx.x - down * across;
    const int64_t row = static_cast<int64_t>(down) * (kThreads >> k) + (threadIdx.x >> k);
    if (row >= a.rows) return;  // whole quads leave together (k >= 2)
    const int64_t c = ((static_cast<int64_t>(tile) << k) + (threadIdx.x & ((1 << k) - 1))) * kV;
    const int n = static_cast<int>(min(a.cols - c, int64_t{kV}));
    Vec<T> x;
    vload(x, static_cast<const T*>(a.x.p) + row * a.x.pitch + c, n);
    float v[kV];
    x.get(v);
    if (a.ckpt.codes) pack8(a.ckpt, row, c, n, v);
    if constexpr (kF != kNone) {
        float y[kV], d;
#pragma unroll
        for (int j = 0; j < kV; ++j) activate<kF>(v[j], &y[j], &d);
        put8(static_cast<T*>(a.y.p) + row * a.y.pitch + c, y, n);
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
unpack_kernel(int64_t rows, int64_t cols, CkptRows q, RowsOut x, int k, uint32_t across) {
    const uint32_t down = blockIdx.x / across, tile = blockIdx.x - down * across;
    const int64_t row = static_cast<int64_t>(down) * (kThreads >> k) + (threadIdx.x >> k);
    if (row >= rows) return;
    const int64_t c = ((static_cast<int64_t>(tile) << k) + (threadIdx.x & ((1 << k) - 1))) * kV;
    const int n = static_cast<int>(min(cols - c, int64_t{kV}));
    if (n <= 0) return;
    float v[kV];
    decode8(code_load(q.codes + row * q.code_pitch + c, n),
            q.scales[row * q.scale_pitch + c / kCkptGroup], q.int8 != 0, v);
    put8(static_cast<T*>(x.p) + row * x.pitch + c, v, n);
}

// ---------------------------------------------------------------------------
// column sums: partial sums per workgroup, then their sum in a fixed order
// ---------------------------------------------------------------------------
// The lanes of a tile's rows add their 8 columns in LDS, row by row; the first row's lanes
// write the workgroup's partial sums.  Called by every thread.
__device__ __forceinline__ void tile_partial(const float* s, float* lds, int k, float* out, int n) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kV; ++j) lds[j * kThreads + threadIdx.x] = s[j];
    __syncthreads();
    if (threadIdx.x >> k) return;
#pragma unroll
    for (int j = 0; j < kV; ++j) {
        float t = lds[j * kThreads + threadIdx.x];
        for (int r = 1; r < (kThreads >> k); ++r) t += lds[j * kThreads + threadIdx.x + (r << k)];
        if (j < n) out[j] = t;
    }
}

constexpr int kSumCols = 64, kSumSlices = 16;   // sum kernel: columns and slices of a workgroup
// out[c] (+)= sum over g of partial[g][c]: each slice sums its part of the partial rows, then the
// slices are added in order.
__global__ void __launch_bounds__(kSumCols / 4 * kSumSlices)
col_sum_kernel(const float* partial, int64_t G, int64_t pitch, int64_t cols, ColOut o0, ColOut o1) {
    __shared__ f4 lds[kSumSlices][kSumCols / 4];
    const ColOut o = blockIdx.y ? o1 : o0;
    const float* p = partial + (blockIdx.y ? cols : 0);
    const int lane = threadIdx.x % (kSumCols / 4), slice = threadIdx.x / (kSumCols / 4);
    const int64_t c = static_cast<int64_t>(blockIdx.x) * kSumCols + 4 * lane;
    const int n = static_cast<int>(min(cols - c, int64_t{4}));
    f4 s = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t g = slice; g < G; g += kSumSlices) {
        const float* q = p + g * pitch + c;
        if (n == 4) {
            s += *(const f4e*)q;
        } else {
            for (int j = 0; j < 4; ++j)
                if (j < n) s[j] += q[j];
        }
    }
    lds[slice][lane] = s;
    __syncthreads();
    if (slice || n <= 0) return;
    for (int i = 1; i < kSumSlices; ++i) s += lds[i][lane];
    for (int j = 0; j < 4; ++j) {
        if (j >= n) break;
        if (o.bf16) {
            uint16_t* d = static_cast<uint16_t*>(o.p) + c + j;
            float t = s[j];
            if (o.accumulate) t += __builtin_bit_cast(float, uint32_t{*d} << 16);
            const uint32_t r = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{t, 0.0f}), bf2));
            *d = static_cast<uint16_t>(r);
        } else {
            float* d = static_cast<float*>(o.p) + c + j;
            *d = o.accumulate ? *d + s[j] : s[j];
        }
    }
}
hipError_t launch_col_sum(const float* partial, int64_t G, int64_t pitch, int64_t cols,
                          const ColOut& o0, const ColOut& o1, hipStream_t stream) {
    if (!o0.p && !o1.p) return hipSuccess;
    // one output only: its half of the partial sums is the first (see the callers) unless o0 is missing
    const int64_t blocks = (cols + kSumCols - 1) / kSumCols;
    const float* p = partial;
    ColOut a = o0, b = o1;
    if (!a.p) {
        a = b;
        b.p = nullptr;
        p += cols;
    }
    col_sum_kernel<<<dim3(static_cast<uint32_t>(blocks), b.p ? 2 : 1), kSumCols / 4 * kSumSlices, 0, stream>>>(
        p, G, pitch, cols, a, b);
    return hipGetLastError();
}

// How a backward pass that walks tiles cuts its rows: `chunks` runs of tiles down, about eight
// workgroups per CU, each run long enough that its partial sums stay small against its rows.
struct Walk {
    Tiles t;
    int64_t chunks, per;  // per: tiles down a chunk
};
Walk plan_walk(int64_t rows, int64_t cols) {
    Walk w;
    w.t = plan_tiles(rows, cols);
    int64_t want = std::max<int64_t>(1, 2048 / w.t.across);
    want = std::min(want, std::max<int64_t>(1, (w.t.down + 7) / 8));
    w.per = std::max<int64_t>(1, (w.t.down + want - 1) / want);
    w.chunks = w.t.down ? (w.t.down + w.per - 1) / w.per : 0;
    return w;
}

// dx = dy f'(h), optionally y = f(h) again, and the column sums of dx before its rounding.
template <typename T, int kF, bool kCkpt>
__global__ void __launch_bounds__(kThreads)
act_bwd_kernel(ActBwd a, int k, uint32_t across, int64_t per) {
    __shared__ float lds[kV * kThreads];
    const uint32_t chunk = blockIdx.x / across, tile = blockIdx.x - chunk * across;
    const int64_t c = ((static_cast<int64_t>(tile) << k) + (threadIdx.x & ((1 << k) - 1))) * kV;
    const int n = static_cast<int>(max(min(a.cols - c, int64_t{kV}), int64_t{0}));
    const int high = kThreads >> k;
    const int64_t r0 = chunk * per * high;
    const int64_t r1 = min(a.rows, r0 + per * high);
    float s[kV] = {};
    for (int64_t row = r0 + (threadIdx.x >> k); row < r1; row += high) {
        if (n == 0) break;
        Vec<T> dy;
        vload(dy, static_cast<const T*>(a.dy.p) + row * a.dy.pitch + c, n);
        float h[kV], g[kV], y[kV];
        if constexpr (kCkpt) {
            decode8(code_load(a.ckpt.codes + row * a.ckpt.code_pitch + c, n),
                    a.ckpt.scales[row * a.ckpt.scale_pitch + c / kCkptGroup], a.ckpt.int8 != 0, h);
        } else {
            Vec<T> x;
            vload(x, static_cast<const T*>(a.x.p) + row * a.x.pitch + c, n);
            x.get(h);
        }
        dy.get(g);
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            float d;
            activate<kF>(h[j], &y[j], &d);
            g[j] *= d;
            s[j] += g[j];
        }
        put8(static_cast<T*>(a.dx.p) + row * a.dx.pitch + c, g, n);
        if (a.y.p) put8(static_cast<T*>(a.y.p) + row * a.y.pitch + c, y, n);
    }
    if (a.dbias.p) tile_partial(s, lds, k, a.workspace + chunk * a.cols + c, n);
}

// ---------------------------------------------------------------------------
// norms, rows of any length: one workgroup per row, the row read again for each pass over it
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_fwd_long_kernel(NormFwd a) {
    __shared__ float lds[2][kThreads / 64];
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(a.x.p) + row * a.x.pitch;
    const T* res = a.residual.p ? static_cast<const T*>(a.residual.p) + row * a.residual.pitch : nullptr;
    T* sum = a.sum.p ? static_cast<T*>(a.sum.p) + row * a.sum.pitch : nullptr;
    // every pass adds x and the residual anew, to the same rounded sum
    const auto get = [&](int64_t c, int n, float* v, bool store) {
        Vec<T> t;
        vload(t, x + c, n);
        t.get(v);
        if (res) {
            Vec<T> r;
            vload(r, res + c, n);
            float w[kV];
            r.get(w);
#pragma unroll
            for (int j = 0; j < kV; ++j) v[j] += w[j];
            t.set(v);
            if (store && sum) vstore(t, sum + c, n);
            t.get(v);
        }
    };
    const float inv = 1.0f / static_cast<float>(a.cols);
    float mean = 0.0f;
    if (!a.rms) {
        float s = 0.0f;
        for (int64_t c = threadIdx.x * kV; c < a.cols; c += kThreads * kV) {
            float v[kV];
            get(c, static_cast<int>(min(a.cols - c, int64_t{kV})), v, false);
#pragma unroll
            for (int j = 0; j < kV; ++j) s += v[j];
        }
        mean = group_sum<kThreads>(s, lds[0]) * inv;
    }
    float s = 0.0f;
    for (int64_t c = threadIdx.x * kV; c < a.cols; c += kThreads * kV) {
        float v[kV];
        const int n = static_cast<int>(min(a.cols - c, int64_t{kV}));
        get(c, n, v, false);
#pragma unroll
        for (int j = 0; j < kV; ++j)
            if (j < n) s += (v[j] - mean) * (v[j] - mean);
    }
    const float rstd = 1.0f / __builtin_sqrtf(group_sum<kThreads>(s, lds[1]) * inv + a.eps);
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[row] = mean;
        a.rstd[row] = rstd;
    }
    const int64_t padded = (a.cols + kCkptGroup - 1) / kCkptGroup * kCkptGroup;  // whole quads
    for (int64_t c = threadIdx.x * kV; c < padded; c += kThreads * kV) {
        float v[kV], w[kV], b[kV] = {};
        const int n = static_cast<int>(min(a.cols - c, int64_t{kV}));
        get(c, n, v, true);
        if (a.ckpt.codes) pack8(a.ckpt, row, c, n, v);
        param8(a.weight, a.param_bf16, c, n, w);
        if (a.bias) param8(a.bias, a.param_bf16, c, n, b);
#pragma unroll
        for (int j = 0; j < kV; ++j) v[j] = (v[j] - mean) * rstd * w[j] + b[j];
        put8(static_cast<T*>(a.y.p) + row * a.y.pitch + c, v, n);
    }
}

// The input's vector, from the tensor or the checkpoint.
template <typename T, bool kCkpt>
__device__ __forceinline__ void input8(const NormBwd& a, int64_t row, int64_t c, int n, float* v) {
    if constexpr (kCkpt) {
        if (n <= 0) {
            for (int j = 0; j < kV; ++j) v[j] = 0.0f;
            return;
        }
        decode8(code_load(a.ckpt.codes + row * a.ckpt.code_pitch + c, n),
                a.ckpt.scales[row * a.ckpt.scale_pitch + c / kCkptGroup], a.ckpt.int8 != 0, v);
    } else {
        Vec<T> t;
        vload(t, static_cast<const T*>(a.x.p) + row * a.x.pitch + c, n);
        t.get(v);
    }
}

// stat[2 row] = mean of g, stat[2 row + 1] = mean of g xh, with g = dy w.
template <typename T, bool kCkpt>
__global__ void __launch_bounds__(kThreads) norm_bwd_stat_kernel(NormBwd a, float* stat) {
    __shared__ float lds[2][kThreads / 64];
    const int64_t row = blockIdx.x;
    const float mean = a.rms ? 0.0f : a.mean[row], rstd = a.rstd[row];
    float s0 = 0.0f, s1 = 0.0f;
    for (int64_t c = threadIdx.x * kV; c < a.cols; c += kThreads * kV) {
        const int n = static_cast<int>(min(a.cols - c, int64_t{kV}));
        float x[kV], g[kV], w[kV];
        input8<T, kCkpt>(a, row, c, n, x);
        Vec<T> dy;
        vload(dy, static_cast<const T*>(a.dy.p) + row * a.dy.pitch + c, n);
        dy.get(g);
        param8(a.weight, a.param_bf16, c, n, w);
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            if (j >= n) break;
            const float t = g[j] * w[j];
            s0 += t;
            s1 += t * ((x[j] - mean) * rstd);
        }
    }
    const float inv = 1.0f / static_cast<float>(a.cols);
    s0 = group_sum<kThreads>(s0, lds[0]);
    s1 = group_sum<kThreads>(s1, lds[1]);
    if (threadIdx.x == 0) {
        stat[2 * row] = a.rms ? 0.0f : s0 * inv;
        stat[2 * row + 1] = s1 * inv;
    }
}

template <typename T, bool kCkpt>
__global__ void __launch_bounds__(kThreads)
norm_bwd_tile_kernel(NormBwd a, const float* stat, float* partial, int k, uint32_t across, int64_t per) {
    __shared__ float lds[kV * kThreads];
    const uint32_t chunk = blockIdx.x / across, tile = blockIdx.x - chunk * across;
    const int64_t c = ((static_cast<int64_t>(tile) << k) + (threadIdx.x & ((1 << k) - 1))) * kV;
    const int n = static_cast<int>(max(min(a.cols - c, int64_t{kV}), int64_t{0}));
    const int high = kThreads >> k;
    const int64_t r0 = chunk * per * high;
    const int64_t r1 = min(a.rows, r0 + per * high);
    float w[kV], b[kV] = {}, sw[kV] = {}, sb[kV] = {};
    param8(a.weight, a.param_bf16, c, n, w);
    if (a.bias && a.y.p) param8(a.bias, a.param_bf16, c, n, b);
    for (int64_t row = r0 + (threadIdx.x >> k); row < r1; row += high) {
        if (n == 0) break;
        const float mean = a.rms ? 0.0f : a.mean[row], rstd = a.rstd[row];
        const float c1 = stat[2 * row], c2 = stat[2 * row + 1];
        float x[kV], g[kV], r[kV] = {};
        input8<T, kCkpt>(a, row, c, n, x);
        Vec<T> dy;
        vload(dy, static_cast<const T*>(a.dy.p) + row * a.dy.pitch + c, n);
        dy.get(g);
        if (a.dres.p) {
            Vec<T> t;
            vload(t, static_cast<const T*>(a.dres.p) + row * a.dres.pitch + c, n);
            t.get(r);
        }
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const float xh = (x[j] - mean) * rstd;
            sw[j] += g[j] * xh;
            sb[j] += g[j];
            x[j] = xh * w[j] + b[j];
            g[j] = rstd * (g[j] * w[j] - c1 - xh * c2) + r[j];
        }
        put8(static_cast<T*>(a.dx.p) + row * a.dx.pitch + c, g, n);
        if (a.y.p) put8(static_cast<T*>(a.y.p) + row * a.y.pitch + c, x, n);
    }
    float* out = partial + chunk * 2 * a.cols + c;
    if (a.dweight.p) tile_partial(sw, lds, k, out, n);
    if (a.dbias.p) tile_partial(sb, lds, k, out + a.cols, n);
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
// A launch takes at most 2^31 threads; longer inputs go in runs of rows.
constexpr int64_t kMaxBlocks = int64_t{1} << 22;

RowsIn skip(RowsIn m, int64_t rows, bool bf16) {
    if (m.p) m.p = static_cast<const char*>(m.p) + rows * m.pitch * (bf16 ? 2 : 4);
    return m;
}
RowsOut skip(RowsOut m, int64_t rows, bool bf16) {
    if (m.p) m.p = static_cast<char*>(m.p) + rows * m.pitch * (bf16 ? 2 : 4);
    return m;
}
CkptRows skip(CkptRows q, int64_t rows) {
    if (q.codes) {
        q.codes += rows * q.code_pitch;
        q.scales += rows * q.scale_pitch;
    }
    return q;
}

// body(first row, rows, tiles across, log2 of a tile's vectors, workgroups) for each run of rows.
template <typename F>
hipError_t for_tiles(int64_t rows, int64_t cols, F&& body) {
    const Tiles t = plan_tiles(rows, cols);
    const int64_t run = std::max<int64_t>(1, kMaxBlocks / t.across) * (kThreads >> t.k);
    for (int64_t r = 0; r < rows; r += run) {
        const int64_t n = std::min(run, rows - r);
        const int64_t high = kThreads >> t.k;
        body(r, n, t.across, t.k, static_cast<uint32_t>((n + high - 1) / high * t.across));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <typename T>
hipError_t act_forward_t(const ActFwd& a, hipStream_t stream) {
    return for_tiles(a.rows, a.cols, [&](int64_t r, int64_t n, uint32_t across, int k, uint32_t blocks) {
        ActFwd b = a;
        b.rows = n;
        b.x = skip(a.x, r, a.bf16);
        b.y = skip(a.y, r, a.bf16);
        b.ckpt = skip(a.ckpt, r);
        switch (a.f) {
            case kNone: act_fwd_kernel<T, kNone><<<blocks, kThreads, 0, stream>>>(b, k, across); break;
            case kRelu: act_fwd_kernel<T, kRelu><<<blocks, kThreads, 0, stream>>>(b, k, across); break;
            case kGelu: act_fwd_kernel<T, kGelu><<<blocks, kThreads, 0, stream>>>(b, k, across); break;
            case kGeluTanh: act_fwd_kernel<T, kGeluTanh><<<blocks, kThreads, 0, stream>>>(b, k, across); break;
            default: act_fwd_kernel<T, kSilu><<<blocks, kThreads, 0, stream>>>(b, k, across); break;
        }
    });
}

template <typename T, bool kCkpt>
void act_backward_t(const ActBwd& a, const Walk& w, hipStream_t stream) {
    const uint32_t blocks = static_cast<uint32_t>(w.chunks * w.t.across);
    switch (a.f) {
        case kRelu: act_bwd_kernel<T, kRelu, kCkpt><<<blocks, kThreads, 0, stream>>>(a, w.t.k, w.t.across, w.per); break;
        case kGelu: act_bwd_kernel<T, kGelu, kCkpt><<<blocks, kThreads, 0, stream>>>(a, w.t.k, w.t.across, w.per); break;
        case kGeluTanh: act_bwd_kernel<T, kGeluTanh, kCkpt><<<blocks, kThreads, 0, stream>>>(a, w.t.k, w.t.across, w.per); break;
        default: act_bwd_kernel<T, kSilu, kCkpt><<<blocks, kThreads, 0, stream>>>(a, w.t.k, w.t.across, w.per); break;
    }
}

template <typename T, bool kCkpt>
hipError_t norm_backward_t(const NormBwd& a, hipStream_t stream) {
    const Walk w = plan_walk(a.rows, a.cols);
    float* stat = a.workspace;
    float* partial = a.workspace + (2 * a.rows + 3) / 4 * 4;
    if (a.rows > 0) {
        for (int64_t r = 0; r < a.rows; r += kMaxBlocks) {
            NormBwd b = a;
            b.dy = skip(a.dy, r, a.bf16);
            b.x = skip(a.x, r, a.bf16);
            b.ckpt = skip(a.ckpt, r);
            if (a.mean) b.mean = a.mean + r;
            b.rstd = a.rstd + r;
            norm_bwd_stat_kernel<T, kCkpt><<<static_cast<uint32_t>(std::min(kMaxBlocks, a.rows - r)), kThreads, 0, stream>>>(b, stat + 2 * r);
        }
        norm_bwd_tile_kernel<T, kCkpt><<<static_cast<uint32_t>(w.chunks * w.t.across), kThreads, 0, stream>>>(
            a, stat, partial, w.t.k, w.t.across, w.per);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return launch_col_sum(partial, w.chunks, 2 * a.cols, a.cols, a.dweight, a.dbias, stream);
}

}  // namespace

int64_t norm_workspace_floats(int64_t rows, int64_t cols) {
    if (rows == 0 || cols == 0) return 0;
    int64_t n, r;
    if (__builtin_mul_overflow(2 * plan_walk(rows, cols).chunks, cols, &n)) return -1;
    if (__builtin_mul_overflow(rows, int64_t{2}, &r) || __builtin_add_overflow(r, 3, &r) ||
        __builtin_add_overflow(n, r / 4 * 4, &n))
        return -1;
    return n;
}
int64_t act_workspace_floats(int64_t rows, int64_t cols) {
    if (rows == 0 || cols == 0) return 0;
    int64_t n;
    return __builtin_mul_overflow(plan_walk(rows, cols).chunks, cols, &n) ? -1 : n;
}

hipError_t launch_act_forward(const ActFwd& a, hipStream_t stream) {
    return a.bf16 ? act_forward_t<uint16_t>(a, stream) : act_forward_t<float>(a, stream);
}

hipError_t launch_unpack(int64_t rows, int64_t cols, bool bf16, const CkptRows& q, RowsOut x,
                         hipStream_t stream) {
    return for_tiles(rows, cols, [&](int64_t r, int64_t n, uint32_t across, int k, uint32_t blocks) {
        if (bf16)
            unpack_kernel<uint16_t><<<blocks, kThreads, 0, stream>>>(n, cols, skip(q, r), skip(x, r, true), k, across);
        else
            unpack_kernel<float><<<blocks, kThreads, 0, stream>>>(n, cols, skip(q, r), skip(x, r, false), k, across);
    });
}

hipError_t launch_act_backward(const ActBwd& a, hipStream_t stream) {
    const Walk w = plan_walk(a.rows, a.cols);
    if (a.rows > 0) {
        if (a.bf16) {
            if (a.ckpt.codes) act_backward_t<uint16_t, true>(a, w, stream);
            else act_backward_t<uint16_t, false>(a, w, stream);
        } else {
            if (a.ckpt.codes) act_backward_t<float, true>(a, w, stream);
            else act_backward_t<float, false>(a, w, stream);
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return launch_col_sum(a.workspace, w.chunks, a.cols, a.cols, a.dbias, ColOut{nullptr, 0, 0}, stream);
}

hipError_t launch_norm_forward(const NormFwd& a, hipStream_t stream) {
    for (int64_t r = 0; r < a.rows; r += kMaxBlocks) {
        NormFwd b = a;
        b.rows = std::min(kMaxBlocks, a.rows - r);
        b.x = skip(a.x, r, a.bf16);
        b.residual = skip(a.residual, r, a.bf16);
        b.sum = skip(a.sum, r, a.bf16);
        b.y = skip(a.y, r, a.bf16);
        b.ckpt = skip(a.ckpt, r);
        if (a.mean) b.mean = a.mean + r;
        b.rstd = a.rstd + r;
        if (a.bf16) norm_fwd_long_kernel<uint16_t><<<static_cast<uint32_t>(b.rows), kThreads, 0, stream>>>(b);
        else norm_fwd_long_kernel<float><<<static_cast<uint32_t>(b.rows), kThreads, 0, stream>>>(b);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_norm_backward(const NormBwd& a, hipStream_t stream) {
    if (a.bf16)
        return a.ckpt.codes ? norm_backward_t<uint16_t, true>(a, stream) : norm_backward_t<uint16_t, false>(a, stream);
    return a.ckpt.codes ? norm_backward_t<float, true>(a, stream) : norm_backward_t<float, false>(a, stream);
}

}  // namespace fsdp
