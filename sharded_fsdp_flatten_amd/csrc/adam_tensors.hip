// adam_tensors.hip -- AdamW over a list of tensors, states in fp32 or 8 bits, and the conversion between
// state formats.
//
// A launch carries a table of tensors in its arguments; a workgroup takes one tile of one tensor.  With
// fp32 states every element takes the operations of the single shard's step, each rounded on its own.
// 8-bit states (m: e4m3, v: e5m3, a power-of-two scale for 32 elements) are read, updated in fp32, and
// rounded at random to codes again.  Bound by HBM: 28 bytes an element with fp32 states and
// gradients, 16.1 with 8-bit states (2 less with bf16 gradients, 2 more with a bf16 copy).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "train.h"

#pragma clang fp contract(off)

namespace fsdp {
namespace {

constexpr int kThreads = 256;
// Elements of a workgroup: 14.2 M elements with fp32 states, tiles of 1024 / 2048 / 4096 72.1 / 74.0 / 73.9 us; 25 M with 8-bit
// ones and fp32 gradients 67.3 / 62.8 / 65.8.
template <State kState> constexpr int kTile = kThreads * (kState == State::kF32 ? 4 : 8);
constexpr int64_t kMaxTiles = int64_t{1} << 20;   // of a launch

typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef uint32_t u2e __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u1e __attribute__((aligned(1)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f4e __attribute__((ext_vector_type(4), aligned(4)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));

// ---------------------------------------------------------------------------
// 8-bit states
// ---------------------------------------------------------------------------
struct FormatM {   // e4m3, signed
    static constexpr int kMinExp = -6, kLowByte = 3, kTopExp = 8;
    static constexpr uint32_t kTopMant = 0x600000u;   // 448 = 1.75 x 2^8
    static constexpr bool kKeep = false;
};
struct FormatV {   // e5m3, unsigned: the 8 bits below the sign of a binary16 number
    static constexpr int kMinExp = -14, kLowByte = 11, kTopExp = 15;
    static constexpr uint32_t kTopMant = 0x700000u;   // 61440 = 1.875 x 2^15
    static constexpr bool kKeep = true;               // what is not 0 stays so
};

// The scale byte of a group with this largest magnitude: the smallest power of two at which it is not
// above the largest code.
template <typename F>
__device__ __forceinline__ uint32_t scale_byte(float amax) {
    const uint32_t b = __builtin_bit_cast(uint32_t, amax), e = b >> 23, m = b & 0x7FFFFFu;
    if (e == 255u) return 255u;
    return static_cast<uint32_t>(max(static_cast<int>(e) - F::kTopExp + (m > F::kTopMant), F::kLowByte));
}
__device__ __forceinline__ float scale_value(uint32_t byte) {
    // 2^(byte - 127); 255: NaN; 0 (a state of zeros): 0
    return __builtin_bit_cast(float, byte == 255u ? 0x7FC00000u : byte << 23);
}
// Four values, scaled by inv = 1 / 2^s and rounded at random to codes' values: n = floor(|y| / q + r / 2^16) of
// steps q, an eighth of the power of two below y, but no less than 2^(kMinExp - 3).  Above 2^kMinExp that is
// adding r below the three mantissa bits that stay and cutting off what is left of them (20 bits; the sum is
// exact either way); smaller values, and zeros, take the sum itself.  16 bits of odds, so that one hash gives both states'
// numbers: a rounding is low by 2^-17 of a step on average.
// A v above 0 takes the smallest code at least.  At 0 beside an m that is not, the next update would be m / eps: of
// gradients of 1 and 31 of 5e-6 in a group, as of an embedding's row that is seen once, those moved their parameters by 452 lr
// in the step after; now by 0.69, with fp32 states by 0.67.  The smallest codes' m / sqrt(v) is at most 2^-9 / 224 /
// sqrt(2^-17 / 61440) = 0.8 of that of the group's largest.
template <typename F>
__device__ __forceinline__ void round_codes(const float* x, float inv, const uint32_t* r16, float* c) {
    uint32_t y[4], low = 0xFFFFFFFFu;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        y[j] = __builtin_bit_cast(uint32_t, x[j] * inv);
        low = min(low, y[j] & 0x7FFFFFFFu);
        c[j] = __builtin_bit_cast(float, (y[j] + (r16[j] << 4)) & 0xFFF00000u);
    }
    constexpr uint32_t kNormal = static_cast<uint32_t>(F::kMinExp + 127) << 23;
    if (low < kNormal) {
        constexpr float q = __builtin_bit_cast(float, kNormal - (3u << 23)), iq = __builtin_bit_cast(float, (257u << 23) - kNormal);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float v = __builtin_bit_cast(float, y[j]);
            const float n = floorf(fabsf(v) * iq + static_cast<float>(r16[j]) * 0x1p-16f) * q;
            // (of x, for y may have vanished)
            const float kept = F::kKeep && n == 0.0f && x[j] != 0.0f ? q : n;
            if ((y[j] & 0x7FFFFFFFu) < kNormal) c[j] = copysignf(kept, v);
        }
    }
}
// Four codes of a word, and back.  Values that are codes convert exactly.
__device__ __forceinline__ uint32_t pack_m(const float* v) {
    int w = 0;
    w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], w, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], w, true);
    return static_cast<uint32_t>(w);
}
__device__ __forceinline__ uint32_t pack_v(const float* v) {
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        w |= static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<_Float16>(v[j])) >> 7 & 0xFFu) << (8 * j);
    return w;
}
__device__ __forceinline__ void unpack_m(uint32_t w, float scale, float* v) {
    const f2 a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), false);
    const f2 b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), true);
    v[0] = a[0] * scale;
    v[1] = a[1] * scale;
    v[2] = b[0] * scale;
    v[3] = b[1] * scale;
}
__device__ __forceinline__ void unpack_v(uint32_t w, float scale, float* v) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint16_t h = static_cast<uint16_t>(((w >> (8 * j)) & 255u) << 7);
        v[j] = static_cast<float>(__builtin_bit_cast(_Float16, h)) * scale;
    }
}
// Random bits of an element: a xor-shift-multiply hash of its number and the tensor's key (multipliers
// next to 2^32 times the golden ratio, and the square roots of 2 and 3); m takes the upper 16, v the lower.
__device__ __forceinline__ void random_bits(uint64_t element, uint32_t key, uint32_t* r) {
    // four neighbouring elements, the first a multiple of 4
    const uint32_t first = static_cast<uint32_t>(element) * 0x9E3779B1u + key + static_cast<uint32_t>(element >> 32) * 0xDDB3D743u;
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j) {
        uint32_t x = first + j * 0x9E3779B1u;
        x ^= x >> 15;
        x *= 0xB504F333u;
        x ^= x >> 13;
        x *= 0xDDB3D743u;
        r[j] = x ^ (x >> 16);
    }
}
// The largest of a group's eight lanes.
__device__ __forceinline__ float group_max(float x) {
    const auto dpp = [](float v, auto ctrl) {
        return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), decltype(ctrl)::value, 0xF, 0xF, true));
    };
    // magnitudes as bits, so that a NaN is the largest
    const auto top = [](float a, float b) {
        return __builtin_bit_cast(float, max(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)));
    };
    x = top(x, dpp(x, std::integral_constant<int, 0xB1>{}));   // lanes xor 1
    x = top(x, dpp(x, std::integral_constant<int, 0x4E>{}));   // xor 2
    return top(x, dpp(x, std::integral_constant<int, 0x141>{}));  // the half row mirrored
}
__device__ __forceinline__ float largest(const float* v) {
    uint32_t a = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) a = max(a, __builtin_bit_cast(uint32_t, v[j]) & 0x7FFFFFFFu);
    return __builtin_bit_cast(float, a);
}
template <bool kWhole>
__device__ __forceinline__ void put4(float* p, int n, const float* v) {
    if (kWhole || n >= 4) {
        __builtin_nontemporal_store((f4{v[0], v[1], v[2], v[3]}), (f4e*)p);
    } else {
#pragma unroll
        for (int j = 0; j < 3; ++j)
            if (j < n) p[j] = v[j];
    }
}
template <bool kWhole>
__device__ __forceinline__ void put4(uint16_t* p, int n, const float* v) {
    u2 w;
    w[0] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{v[0], v[1]}), bf2));
    w[1] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{v[2], v[3]}), bf2));
    if (kWhole || n >= 4) {
        __builtin_nontemporal_store(w, (u2e*)p);
    } else {
        for (int j = 0; j < 3; ++j)
            if (j < n) p[j] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
    }
}
// Arrays are read past the cache (kNt) where a call's operands outgrow it, as the layer operators' are.  Steps
// queued one after another over three sets of operands, cached / nt, us: fp32 states 75 MB 14.3 / 16.0, 150 MB 27.1 /
// 28.8, 425 MB 82.9 / 73.9, 900 MB 168 / 152; 8-bit ones 91 MB 18.6 / 18.9, 257 MB 51.6 / 44.6, 544 MB 103 / 86.  (Alone after a
// read of 1 GiB cached loads look better, 69.6 against 77.8 us for 425 MB: then up to 256 MB of what was written
// is still on its way when the kernel ends, and the next one pays.)  Codes and scales
// are always read through the cache (nt 8% slower).
constexpr int64_t kNtBytes = int64_t{192} << 20;

// Raw loads of four elements, n of them inside the tensor (kWhole: all), so that a tile's loads are all issued
// before the first is used.
template <bool kWhole>
__device__ __forceinline__ uint32_t raw_codes(const uint8_t* s, int64_t at, int n) {
    if (kWhole || n >= 4) return *(const u1e*)(s + at);
    uint32_t w = 0;
    for (int j = 0; j < 3; ++j)
        if (j < n) w |= static_cast<uint32_t>(s[at + j]) << (8 * j);
    return w;
}
template <bool kWhole>
__device__ __forceinline__ uint32_t raw_scale(const uint8_t* s, int64_t at, int n, int64_t scales) {
    return kWhole || n > 0 ? s[scales + at / kStateGroup] : 0u;
}
template <bool kWhole, bool kNt>
__device__ __forceinline__ f4 raw4(const float* p, int n) {
    if (kWhole || n >= 4) return kNt ? __builtin_nontemporal_load((const f4e*)p) : *(const f4e*)p;
    f4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 3; ++j)
        if (j < n) v[j] = p[j];
    return v;
}
template <bool kWhole, bool kNt>
__device__ __forceinline__ u2 raw4(const uint16_t* p, int n) {
    if (kWhole || n >= 4) return kNt ? __builtin_nontemporal_load((const u2e*)p) : *(const u2e*)p;
    u2 v = {0u, 0u};
    for (int j = 0; j < 3; ++j)
        if (j < n) v[j >> 1] |= static_cast<uint32_t>(p[j]) << (16 * (j & 1));
    return v;
}
__device__ __forceinline__ void values(f4 w, float* v) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = w[j];
}
__device__ __forceinline__ void values(u2 w, float* v) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __builtin_bit_cast(float, j & 1 ? w[j >> 1] & 0xFFFF0000u : w[j >> 1] << 16);
}
// A state in its format: raw words of four elements, their values, and the way back.
template <State kState, typename F> struct Held;
template <typename F> struct Held<State::k8Bit, F> {
    uint32_t codes, scale;
    template <bool kWhole, bool kNt> __device__ void load(const void* s, int64_t at, int n, int64_t scales) {
        codes = raw_codes<kWhole>(static_cast<const uint8_t*>(s), at, n);
        scale = raw_scale<kWhole>(static_cast<const uint8_t*>(s), at, n, scales);
    }
    __device__ void get(float* v) const {
        if constexpr (F::kTopExp == 8) unpack_m(codes, scale_value(scale), v);
        else unpack_v(codes, scale_value(scale), v);
    }
    // every lane of a group calls it; values behind the tensor's end are 0
    template <bool kWhole> __device__ static void put(void* to, int64_t at, int n, int64_t scales, const float* v, const uint32_t* r) {
        uint8_t* s = static_cast<uint8_t*>(to);
        const uint32_t byte = scale_byte<F>(group_max(largest(v)));
        const float inv = __builtin_bit_cast(float, (254u - byte) << 23);
        uint32_t r16[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) r16[j] = F::kTopExp == 8 ? r[j] >> 16 : r[j] & 0xFFFFu;
        float c[4];
        round_codes<F>(v, inv, r16, c);
        uint32_t w = F::kTopExp == 8 ? pack_m(c) : pack_v(c);
        if (byte == 255u) w = 0;
        if (kWhole || n >= 4) {
            __builtin_nontemporal_store(w, (u1e*)(s + at));   // 64.8 -> 62.3 us (25 M elements)
        } else {
            for (int j = 0; j < 3; ++j)
                if (j < n) s[at + j] = static_cast<uint8_t>(w >> (8 * j));
        }
        if ((kWhole || n > 0) && (threadIdx.x & 7) == 0) s[scales + at / kStateGroup] = static_cast<uint8_t>(byte);
    }
};
template <typename F> struct Held<State::kF32, F> {
    f4 raw;
    template <bool kWhole, bool kNt> __device__ void load(const void* s, int64_t at, int n, int64_t) {
        raw = raw4<kWhole, kNt>(static_cast<const float*>(s) + at, n);
    }
    __device__ void get(float* v) const { values(raw, v); }
    template <bool kWhole> __device__ static void put(void* to, int64_t at, int n, int64_t, const float* v, const uint32_t*) {
        put4<kWhole>(static_cast<float*>(to) + at, n, v);
    }
};
template <typename F> struct Held<State::kBF16, F> {
    u2 raw;
    template <bool kWhole, bool kNt> __device__ void load(const void* s, int64_t at, int n, int64_t) {
        raw = raw4<kWhole, kNt>(static_cast<const uint16_t*>(s) + at, n);
    }
    __device__ void get(float* v) const { values(raw, v); }
    template <bool kWhole> __device__ static void put(void* to, int64_t at, int n, int64_t, const float* v, const uint32_t*) {
        put4<kWhole>(static_cast<uint16_t*>(to) + at, n, v);
    }
};

// ---------------------------------------------------------------------------
// the step
// ---------------------------------------------------------------------------
// A tensor in a launch's table, in 32-bit words: addresses and sizes take 48 bits each.  Where no tensor has a copy,
// or the states need no key, those words are left out, so that more tensors go in a launch (96 short ones in one instead
// of two of 50: 10.9 -> 7.4 us; 144 with 8-bit states in two instead of three: 119 -> 109).
template <bool kKey, bool kCopy> struct Entry {
    uint32_t low[kCopy ? 6 : 5];   // of p, g, m, v, n and the copy
    uint32_t high[3];              // the upper 16 bits in pairs: p and g, m and v, n (with the group, from bit 12 on) and the copy
    uint32_t key[kKey ? 1 : 0];
};
constexpr int kArguments = 4096 - 64;   // bytes of a table: the budget of a kernel's arguments, less what launches add
constexpr int kTableHead = kAdamGroups * sizeof(AdamScalars) + 2 * sizeof(void*) + 8;
template <bool kKey, bool kCopy> struct Table {
    static constexpr int kLaunch = (kArguments - kTableHead) / (4 + sizeof(Entry<kKey, kCopy>));
    AdamScalars sc[kAdamGroups];
    const float *grad_scale, *skip;
    uint32_t bias;             // the first entry's tiles that earlier launches took
    uint32_t start[kLaunch];   // first tile of each entry; beyond the last entry: UINT32_MAX
    Entry<kKey, kCopy> e[kLaunch];
};
static_assert(sizeof(Table<true, true>) <= kArguments && sizeof(Table<false, false>) <= kArguments,
              "the table must fit one kernel argument block");
// The same, read by a kernel.
struct Tensor {
    float* p;
    const void* g;
    void *m, *v;
    uint16_t* pb;
    int64_t n;
    uint32_t key, group;
};
template <bool kKey, bool kCopy>
__device__ __forceinline__ Tensor tensor_of(const Entry<kKey, kCopy>& e) {
    const auto at = [](uint32_t low, uint32_t high) { return static_cast<uint64_t>(high & 0xFFFFu) << 32 | low; };
    Tensor t;
    t.p = reinterpret_cast<float*>(at(e.low[0], e.high[0]));
    t.g = reinterpret_cast<const void*>(at(e.low[1], e.high[0] >> 16));
    t.m = reinterpret_cast<void*>(at(e.low[2], e.high[1]));
    t.v = reinterpret_cast<void*>(at(e.low[3], e.high[1] >> 16));
    t.n = static_cast<int64_t>(at(e.low[4], e.high[2] & 0xFFFu));
    t.group = e.high[2] >> 12 & 15u;
    t.pb = nullptr;
    if constexpr (kCopy) t.pb = reinterpret_cast<uint16_t*>(at(e.low[5], e.high[2] >> 16));
    t.key = 0;
    if constexpr (kKey) t.key = e.key[0];
    return t;
}
template <bool kKey, bool kCopy>
Entry<kKey, kCopy> entry_of_tensor(const AdamTensor& a) {
    const auto word = [](const void* p) { return reinterpret_cast<uint64_t>(p); };
    const auto pair = [](uint64_t x, uint64_t y) { return static_cast<uint32_t>(x >> 32 & 0xFFFFu) | static_cast<uint32_t>(y >> 32 << 16); };
    const uint64_t size = static_cast<uint64_t>(a.n) | static_cast<uint64_t>(a.group) << 44;
    Entry<kKey, kCopy> e;
    e.low[0] = static_cast<uint32_t>(word(a.p));
    e.low[1] = static_cast<uint32_t>(word(a.g));
    e.low[2] = static_cast<uint32_t>(word(a.m));
    e.low[3] = static_cast<uint32_t>(word(a.v));
    e.low[4] = static_cast<uint32_t>(size);
    if constexpr (kCopy) e.low[5] = static_cast<uint32_t>(word(a.pb));
    e.high[0] = pair(word(a.p), word(a.g));
    e.high[1] = pair(word(a.m), word(a.v));
    e.high[2] = pair(size, word(a.pb));
    if constexpr (kKey) e.key[0] = a.key;
    return e;
}

// The moments, and the parameter's decay, as the single shard's step has them, bit for bit.
__device__ __forceinline__ void moments(float& p, float g, float& m, float& v, const AdamScalars& s) {
    p = p * s.decay;
    m = s.b1 * m + s.omb1 * g;
    const float gg = g * g;
    v = s.b2 * v + s.omb2 * gg;
}
// The update.  kExact: the single shard's, bit for bit.  Else (8-bit states) its square root and quotients are the
// hardware's, to one unit in the last place each, and it stays within 14 x 2^-24 of itself: 29.5 M elements 97 ->
// 86 us, where the exact ones' 45 more instruction slots an element bind the kernel.
template <bool kExact>
__device__ __forceinline__ float updated(float p, float m, float v, const AdamScalars& s, float inv_bc2s) {
    if constexpr (kExact) {
        const float den = sqrtf(v) / s.bc2s + s.eps;
        return p - s.step_size * (m / den);
    } else {
        const float den = __builtin_amdgcn_sqrtf(v) * inv_bc2s + s.eps;
        return p - s.step_size * (m * __builtin_amdgcn_rcpf(den));
    }
}
// The hardware's root takes a subnormal v as 0; its reciprocal takes a subnormal denominator as 0, and gives 0 for
// a subnormal result.  Where either can matter the exact path is taken: groups with such an eps (but for eps a denominator
// above 0 lies between 2^-75 and 2^91), and four elements with such a v where eps does not hide its root (at most 2^-63).
// With v = 0 and no eps both paths give an infinity or NaN.
__device__ __forceinline__ bool far_eps(float eps) { return eps != 0.0f && !(eps >= 0x1p-126f && eps <= 0x1p96f); }
__device__ __forceinline__ bool hides_roots(const AdamScalars& s) { return s.eps * s.bc2s >= 0x1p-38f; }
__device__ __forceinline__ bool any_subnormal(const float* v) {
    uint32_t low = 0xFFFFFFFFu;
#pragma unroll
    for (int j = 0; j < 4; ++j) low = min(low, __builtin_bit_cast(uint32_t, v[j]) - 1u);   // (0 comes last)
    return low < 0x7FFFFFu;
}

// The workgroup's entry, and which of the entry's tiles of this launch it takes.  Each XCD takes runs of 64
// neighbouring tiles (14.2 M elements with fp32 states 74.0 -> 72.6 us).
template <int kLaunch>
__device__ __forceinline__ uint32_t entry_of(const uint32_t (&start)[kLaunch], uint32_t* tile) {
    constexpr uint32_t kXcds = 8, kRun = 64, kPer = kXcds * kRun;
    uint32_t at = blockIdx.x;
    if (at < gridDim.x / kPer * kPer) at = at / kPer * kPer + at % kXcds * kRun + at % kPer / kXcds;
    // an entry a lane
    static_assert(kLaunch <= 128);
    const uint32_t l = threadIdx.x & 63u;
    const uint32_t k = __popcll(__ballot(start[min(l, kLaunch - 1u)] <= at && l < kLaunch)) +
                       (kLaunch > 64 ? __popcll(__ballot(start[min(l + 64u, kLaunch - 1u)] <= at && l + 64u < kLaunch)) : 0) - 1u;
    *tile = at - start[k];
    return k;
}

template <typename G, State kState, bool kWhole, bool kNt>
__device__ __forceinline__ void adam_tile(const AdamScalars& s, const float* grad_scale, const Tensor& e, int64_t base) {
    constexpr int kN = kTile<kState> / kThreads / 4;
    const float inv_bc2s = 1.0f / s.bc2s;
    const bool rare = kState != State::kF32 && far_eps(s.eps), hidden = hides_roots(s);
    const float gs = grad_scale ? *grad_scale : 1.0f;
    const int64_t scales = (e.n + 15) / 16 * 16;
    f4 p[kN];
    decltype(raw4<true, kNt>(static_cast<const G*>(nullptr), 0)) g[kN];
    Held<kState, FormatM> m[kN];
    Held<kState, FormatV> v[kN];
    const auto place = [&](int h, int64_t* at) {
        *at = base + 4 * (threadIdx.x + h * kThreads);
        return kWhole ? 4 : static_cast<int>(max(min(e.n - *at, int64_t{4}), int64_t{0}));
    };
#pragma unroll
    for (int h = 0; h < kN; ++h) {
        int64_t at;
        const int n = place(h, &at);
        p[h] = raw4<kWhole, kNt>(e.p + at, n);
        g[h] = raw4<kWhole, kNt>(static_cast<const G*>(e.g) + at, n);
        m[h].template load<kWhole, kNt>(e.m, at, n, scales);
        v[h].template load<kWhole, kNt>(e.v, at, n, scales);
    }
#pragma unroll
    for (int h = 0; h < kN; ++h) {
        int64_t at;
        const int n = place(h, &at);
        float pp[4], gg[4], mm[4], vv[4];
        values(p[h], pp);
        values(g[h], gg);
        m[h].get(mm);
        v[h].get(vv);
#pragma unroll
        for (int j = 0; j < 4; ++j) moments(pp[j], grad_scale ? gg[j] * gs : gg[j], mm[j], vv[j], s);
        if (kState == State::kF32 || rare || (!hidden && any_subnormal(vv))) {
#pragma unroll
            for (int j = 0; j < 4; ++j) pp[j] = updated<true>(pp[j], mm[j], vv[j], s, inv_bc2s);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) pp[j] = updated<false>(pp[j], mm[j], vv[j], s, inv_bc2s);
        }
        put4<kWhole>(e.p + at, n, pp);
        if (e.pb) put4<kWhole>(e.pb + at, n, pp);
        uint32_t r[4];
        if constexpr (kState == State::k8Bit) {
            random_bits(static_cast<uint64_t>(at), e.key, r);
            if constexpr (!kWhole) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j >= n) mm[j] = vv[j] = 0.0f;
            }
        }
        Held<kState, FormatM>::template put<kWhole>(e.m, at, n, scales, mm, r);
        Held<kState, FormatV>::template put<kWhole>(e.v, at, n, scales, vv, r);
    }
}

template <typename G, State kState, bool kCopy, bool kNt>
__global__ void __launch_bounds__(kThreads) adam_tensors_kernel(Table<kState == State::k8Bit, kCopy> t) {
    if (t.skip && *t.skip != 0.0f) return;
    uint32_t tile;
    const uint32_t k = entry_of(t.start, &tile);
    const Tensor e = tensor_of(t.e[k]);
    const AdamScalars s = t.sc[e.group];
    const int64_t base = (static_cast<int64_t>(tile) + (k == 0 ? t.bias : 0u)) * kTile<kState>;
    if (base + kTile<kState> <= e.n) adam_tile<G, kState, true, kNt>(s, t.grad_scale, e, base);
    else adam_tile<G, kState, false, kNt>(s, t.grad_scale, e, base);
}

struct CopyEntry {
    const void *m, *v;
    void *m_to, *v_to;
    int64_t n;
    uint32_t key, unused;
};
struct CopyTable {
    static constexpr int kLaunch = 75;
    uint32_t bias;
    uint32_t start[kLaunch];
    CopyEntry e[kLaunch];
};
static_assert(sizeof(CopyTable) <= kArguments, "the table must fit one kernel argument block");

template <State kFrom, State kTo, bool kWhole>
__device__ __forceinline__ void convert_tile(const CopyEntry& e, int64_t base) {
    constexpr int kN = kTile<State::k8Bit> / kThreads / 4;
    const int64_t scales = (e.n + 15) / 16 * 16;
    Held<kFrom, FormatM> m[kN];
    Held<kFrom, FormatV> v[kN];
    const auto place = [&](int h, int64_t* at) {
        *at = base + 4 * (threadIdx.x + h * kThreads);
        return kWhole ? 4 : static_cast<int>(max(min(e.n - *at, int64_t{4}), int64_t{0}));
    };
#pragma unroll
    for (int h = 0; h < kN; ++h) {
        int64_t at;
        const int n = place(h, &at);
        m[h].template load<kWhole, false>(e.m, at, n, scales);
        v[h].template load<kWhole, false>(e.v, at, n, scales);
    }
#pragma unroll
    for (int h = 0; h < kN; ++h) {
        int64_t at;
        const int n = place(h, &at);
        float mm[4], vv[4];
        m[h].get(mm);
        v[h].get(vv);
        uint32_t r[4];
        if constexpr (kTo == State::k8Bit) random_bits(static_cast<uint64_t>(at), e.key, r);
        Held<kTo, FormatM>::template put<kWhole>(e.m_to, at, n, scales, mm, r);
        Held<kTo, FormatV>::template put<kWhole>(e.v_to, at, n, scales, vv, r);
    }
}

template <State kFrom, State kTo>
__global__ void __launch_bounds__(kThreads) adam_convert_kernel(CopyTable t) {
    uint32_t tile;
    const uint32_t k = entry_of(t.start, &tile);
    const CopyEntry& e = t.e[k];
    const int64_t base = (static_cast<int64_t>(tile) + (k == 0 ? t.bias : 0u)) * kTile<State::k8Bit>;
    if (base + kTile<State::k8Bit> <= e.n) convert_tile<kFrom, kTo, true>(e, base);
    else convert_tile<kFrom, kTo, false>(e, base);
}

// Cuts a list into launches: fill(table slot, tensor) for every entry, then launch(tiles).  A tensor too long for one
// launch goes on as the first of the next.
template <typename TableT, typename List, typename Fill, typename Launch>
hipError_t in_launches(const List& list, int tile, TableT& t, Fill&& fill, Launch&& launch) {
    constexpr int kLaunch = TableT::kLaunch;
    int used = 0;
    int64_t tiles = 0;
    const auto flush = [&]() -> hipError_t {
        if (!used) return hipSuccess;
        for (int i = used; i < kLaunch; ++i) t.start[i] = UINT32_MAX;
        launch(static_cast<uint32_t>(tiles));
        used = 0;
        tiles = 0;
        return hipGetLastError();
    };
    for (size_t i = 0; i < list.size(); ++i) {
        const int64_t all = (list[i].n + tile - 1) / tile;
        for (int64_t done = 0; done < all;) {
            const int64_t now = std::min(all - done, kMaxTiles - tiles);
            t.start[used] = static_cast<uint32_t>(tiles);
            if (used == 0) t.bias = static_cast<uint32_t>(done);
            fill(used++, list[i]);
            done += now;
            tiles += now;
            if (used == kLaunch || tiles == kMaxTiles) {
                const hipError_t e = flush();
                if (e != hipSuccess) return e;
            }
        }
    }
    return flush();
}

template <typename G, State kState, bool kCopy, bool kNt>
hipError_t step(const std::vector<AdamTensor>& list, const AdamScalars* groups, int n_groups, const float* grad_scale,
                const float* skip, hipStream_t stream) {
    constexpr bool kKey = kState == State::k8Bit;
    Table<kKey, kCopy> t{};
    std::copy(groups, groups + n_groups, t.sc);
    t.grad_scale = grad_scale;
    t.skip = skip;
    return in_launches(
        list, kTile<kState>, t, [&](int i, const AdamTensor& a) { t.e[i] = entry_of_tensor<kKey, kCopy>(a); },
        [&](uint32_t tiles) { adam_tensors_kernel<G, kState, kCopy, kNt><<<dim3(tiles), kThreads, 0, stream>>>(t); });
}

template <State kFrom, State kTo>
hipError_t convert(const std::vector<StateCopy>& list, hipStream_t stream) {
    CopyTable t{};
    return in_launches(
        list, kTile<State::k8Bit>, t,
        [&](int i, const StateCopy& a) { t.e[i] = {a.m, a.v, a.m_to, a.v_to, a.n, a.key, 0}; },
        [&](uint32_t tiles) { adam_convert_kernel<kFrom, kTo><<<dim3(tiles), kThreads, 0, stream>>>(t); });
}

// The output function of SplitMix64 (Steele, Lea and Flood, 2014), with its published multipliers.
uint64_t mix64(uint64_t k) {
    k = (k ^ (k >> 30)) * 0xBF58476D1CE4E5B9ull;
    k = (k ^ (k >> 27)) * 0x94D049BB133111EBull;
    return k ^ (k >> 31);
}

}  // namespace

uint32_t adam_key(uint64_t seed, int64_t step, int64_t tensor) {
    constexpr uint64_t kGolden = 0x9E3779B97F4A7C15ull;
    return static_cast<uint32_t>(mix64(mix64(seed + kGolden * static_cast<uint64_t>(step)) +
                                       kGolden * (static_cast<uint64_t>(tensor) + 1)));
}

hipError_t launch_adam_tensors(const std::vector<AdamTensor>& list, const AdamScalars* groups, int n_groups,
                               bool state8, bool grad_bf16, const float* grad_scale, const float* skip,
                               hipStream_t stream) {
    // bytes of the whole list: the launches of a step follow one another
    int64_t bytes = 0;
    bool copy = false;
    for (const AdamTensor& a : list) {
        bytes += a.n * ((state8 ? 12 : 24) + (grad_bf16 ? 2 : 4) + (a.pb ? 2 : 0));
        copy |= a.pb != nullptr;
    }
    const auto go = [&](auto grad, auto state) {
        using G = decltype(grad);
        constexpr State kState = decltype(state)::value;
        const auto with = [&](auto c) {
            constexpr bool kCopy = decltype(c)::value;
            return bytes >= kNtBytes ? step<G, kState, kCopy, true>(list, groups, n_groups, grad_scale, skip, stream)
                                     : step<G, kState, kCopy, false>(list, groups, n_groups, grad_scale, skip, stream);
        };
        return copy ? with(std::true_type{}) : with(std::false_type{});
    };
    using Small = std::integral_constant<State, State::k8Bit>;
    using Full = std::integral_constant<State, State::kF32>;
    if (state8) return grad_bf16 ? go(uint16_t{}, Small{}) : go(0.0f, Small{});
    return grad_bf16 ? go(uint16_t{}, Full{}) : go(0.0f, Full{});
}

hipError_t launch_adam_convert(const std::vector<StateCopy>& list, State from, State to, hipStream_t stream) {
    if (from == State::k8Bit)
        return to == State::kBF16 ? convert<State::k8Bit, State::kBF16>(list, stream)
                                  : convert<State::k8Bit, State::kF32>(list, stream);
    return from == State::kBF16 ? convert<State::kBF16, State::k8Bit>(list, stream)
                                : convert<State::kF32, State::k8Bit>(list, stream);
}

}  // namespace fsdp
