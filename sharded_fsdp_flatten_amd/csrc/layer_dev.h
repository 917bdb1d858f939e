// layer_dev.h -- device code that the layer operators' kernels share: vectors of neighbouring
// columns, 8-bit groups, sums over a wave and a workgroup.
#pragma once

#include <hip/hip_runtime.h>

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
    template <bool kNt> __device__ void load(const uint16_t* p) {
        r = kNt ? __builtin_nontemporal_load((const u4e*)p) : *(const u4e*)p;
    }
    __device__ void load_part(const uint16_t* p, int n) {
        r = u4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int j = 0; j < kV; ++j)
            if (j < n) r[j >> 1] |= uint32_t{p[j]} << (16 * (j & 1));
    }
    __device__ void zero() { r = u4{0u, 0u, 0u, 0u}; }
    // drops the first k elements, zeros behind the last
    __device__ void drop(int k) {
        if (k & 4) r = u4{r[2], r[3], 0u, 0u};
        if (k & 2) r = u4{r[1], r[2], r[3], 0u};
        if (k & 1)
            r = u4{__builtin_amdgcn_alignbit(r[1], r[0], 16), __builtin_amdgcn_alignbit(r[2], r[1], 16),
                   __builtin_amdgcn_alignbit(r[3], r[2], 16), r[3] >> 16};
    }
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
    // cached in any case: each of the two loads reads half of every line, and a line dropped between
    // them is read twice (norm forward 32768 x 1024: nt 54.7, cached 51.0 us; stores, which the cache
    // joins either way, are better nt: unpack 8192 x 12288 110 us against 123)
    template <bool> __device__ void load(const float* p) {
        r[0] = *(const f4e*)p;
        r[1] = *(const f4e*)(p + 4);
    }
    __device__ void load_part(const float* p, int n) {
        zero();
#pragma unroll
        for (int j = 0; j < kV; ++j)
            if (j < n) r[j >> 2][j & 3] = p[j];
    }
    __device__ void zero() { r[0] = r[1] = f4{0.0f, 0.0f, 0.0f, 0.0f}; }
    __device__ void drop(int k) {
        const f4 z = {0.0f, 0.0f, 0.0f, 0.0f};
        if (k & 4) { r[0] = r[1]; r[1] = z; }
        if (k & 2) {
            r[0] = f4{r[0][2], r[0][3], r[1][0], r[1][1]};
            r[1] = f4{r[1][2], r[1][3], 0.0f, 0.0f};
        }
        if (k & 1) {
            r[0] = f4{r[0][1], r[0][2], r[0][3], r[1][0]};
            r[1] = f4{r[1][1], r[1][2], r[1][3], 0.0f};
        }
    }
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

// Loads are non-temporal (kNt) where a call's operands outgrow what the 256 MB Infinity Cache can
// keep, else cached: an activation was written just before it is read here.  kNtBytes: from that
// many bytes read and written on.  MI355X, nt against cached, operands rotating: norm forward 84 MB
// 17.1 / 14.6 us, with residual 403 MB 67.5 / 69.0 us; norm backward 148 MB 34.1 / 30.5 us, 201 MB
// 40.8 / 42.3 us, 604 MB 111 / 117 us, fp32 63 MB 20.6 / 17.6, 252 MB 53.9 / 57.2, 1.2 GB 214 / 228;
// GELU forward 105 MB 19.6 / 17.0 us, 675 MB 107 / 106 us.  The activation's backward pass finds the
// forward pass's matrices between its own and takes kActBwdNtBytes: behind the forward pass, three / six sets
// of operands rotating, 18 MB 13.9 / 13.3 and 14.0 / 13.2 us for both, 37 MB 18.8 / 17.7 and 18.8 / 17.8, 73 MB
// 29.2 / 26.4 and 29.4 / 31.6, 147 MB 49.9 / 52.7 and 53.1 / 53.6; alone, 147 MB 31.7 / 28.3 and 31.8 / 32.6, 472 MB
// 76.7 / 83.8.  Rows that start off a 16-byte boundary share lines
// between vectors and are always cached (norm forward 8192 x 5003: nt 47.0, cached 38.3 us; ReLU backward
// 8192 x 12289 133.3 / 128.4), but for a residual gradient beside aligned rows, which goes with them (norm
// backward 8192 x 12288 with an odd pitch there 151 / 158 us).  Codes are always cached too: a wave's vector is
// 256 or 512 bytes of them (unpack 8192 x 5003: nt 28.0, cached 20.8 us; aligned the same).
constexpr int64_t kNtBytes = int64_t{192} << 20, kActBwdNtBytes = int64_t{64} << 20;

// n: columns of this vector inside the row (8 or more: whole; 0 or less: none).
template <bool kNt, typename T>
__device__ __forceinline__ void vload(Vec<T>& v, const T* p, int n) {
    if (n >= kV) v.template load<kNt>(p);
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
constexpr int kHalfMirror = 0x141, kMirror = 0x140, kRowRor8 = 0x128;

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
// Four values of a word of codes.  gfx950's scaled conversion takes e4m3 codes and the scale's
// exponent field, which the byte is (255: NaN; e4m3 never has the byte 0).
template <bool kInt8>
__device__ __forceinline__ void decode4(uint32_t q, uint32_t byte, float* v) {
    if constexpr (kInt8) {
        const float s = scale_value(byte);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = static_cast<float>(static_cast<int8_t>(q >> (8 * j))) * s;
    } else {
        const float s = __builtin_bit_cast(float, byte << 23);
        const f2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q, s, false);
        const f2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q, s, true);
        v[0] = a[0];
        v[1] = a[1];
        v[2] = b[0];
        v[3] = b[1];
    }
}
__device__ __forceinline__ void decode8(u2 q, uint32_t byte, bool int8, float* v) {
    if (int8) {
        decode4<true>(q[0], byte, v);
        decode4<true>(q[1], byte, v + 4);
    } else {
        decode4<false>(q[0], byte, v);
        decode4<false>(q[1], byte, v + 4);
    }
}
__device__ __forceinline__ u2 code_load(const uint8_t* p, int n) {
    if (n >= kV) return *(const u2e*)p;
    u2 q = {0u, 0u};
#pragma unroll
    for (int j = 0; j < kV; ++j)
        if (j < n) q[j >> 2] |= uint32_t{p[j]} << (8 * (j & 3));
    return q;
}
// Codes are stored non-temporally (kNt) by a pass that writes nothing else, and through the cache
// beside a norm's or an activation's output (pack 8192 x 12288: nt 52.8, cached 55.9 us; norm forward
// and backward from int8 32768 x 1024: 77.7 / 73.6 us, ReLU 2048 x 65536: 267 / 259 us).
template <bool kNt>
__device__ __forceinline__ void code_store(uint8_t* p, u2 q, int n) {
    if (n >= kV) {
        if constexpr (kNt) __builtin_nontemporal_store(q, (u2e*)p);
        else *(u2e*)p = q;
        return;
    }
#pragma unroll
    for (int j = 0; j < kV; ++j)
        if (j < n) p[j] = static_cast<uint8_t>(q[j >> 2] >> (8 * (j & 3)));
}
// Codes and scale of the vector at column c (n of its columns inside the row) of a row.
template <bool kNt>
__device__ __forceinline__ void pack8(const CkptRows& q, int64_t row, int64_t c, int n,
                                      const float* v) {
    uint32_t byte;
    const u2 code = encode8(v, q.int8 != 0, &byte);
    code_store<kNt>(q.codes + row * q.code_pitch + c, code, n);
    if (n > 0 && (threadIdx.x & 3) == 0)
        q.scales[row * q.scale_pitch + c / kCkptGroup] = static_cast<uint8_t>(byte);
}

// ---------------------------------------------------------------------------
// sums over a wave and a workgroup
// ---------------------------------------------------------------------------
// Sum over the wave's four rows of 16 lanes, lane by lane.
__device__ __forceinline__ float sum_rows(float x) {
    const uint32_t a = __builtin_bit_cast(uint32_t, x);
    const auto r = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    const uint32_t b = __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, static_cast<uint32_t>(r[0])) +
                                                        __builtin_bit_cast(float, static_cast<uint32_t>(r[1])));
    const auto t = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    return __builtin_bit_cast(float, static_cast<uint32_t>(t[0])) +
           __builtin_bit_cast(float, static_cast<uint32_t>(t[1]));
}
// Sum over aligned groups of kLanes neighbouring lanes (2, 4, 8 or 16), the same in each of them.
template <int kLanes>
__device__ __forceinline__ float add_lanes(float x) {
    const auto add = [](float a, uint32_t b) { return a + __builtin_bit_cast(float, b); };
    const auto bits = [](float a) { return __builtin_bit_cast(uint32_t, a); };
    x = add(x, dpp<kQuadXor1>(bits(x)));
    if constexpr (kLanes >= 4) x = add(x, dpp<kQuadXor2>(bits(x)));
    if constexpr (kLanes >= 8) x = add(x, dpp<kHalfMirror>(bits(x)));
    if constexpr (kLanes >= 16) x = add(x, dpp<kMirror>(bits(x)));
    return x;
}
__device__ __forceinline__ float wave_sum(float x) { return sum_rows(add_lanes<16>(x)); }
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

}  // namespace
}  // namespace fsdp
