// rotary.hip -- rotary positions of queries and keys, forward and backward.
//
// Pair i of a head at position x turns by w = x f_i: (a, b) -> (a cos w - b sin w, a sin w + b cos w).  The
// cosine and sine of a (token, pair) serve every head: a workgroup takes a few tokens, computes theirs once into
// LDS, one a thread, and then walks the tokens' heads of q and k with them.  Bound by HBM: every element is
// read and written once.
#include <algorithm>

#include "layer_dev.h"
#include "train.h"

namespace fsdp {
namespace {

constexpr double kTurn = 0.15915494309189533577;  // 1 / (2 pi)
constexpr int kPairs = 2048;                      // cosines and sines of a workgroup (16 KB of LDS)

// 16 bytes, at any element
template <typename T> constexpr int kE = 16 / sizeof(T);
template <bool kNt>
__device__ __forceinline__ u4 load16(const void* p) {
    return kNt ? __builtin_nontemporal_load(static_cast<const u4e*>(p)) : *static_cast<const u4e*>(p);
}
__device__ __forceinline__ void put16(void* p, u4 w) { __builtin_nontemporal_store(w, static_cast<u4e*>(p)); }
__device__ __forceinline__ void values(u4 w, float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[2 * j] = __builtin_bit_cast(float, w[j] << 16);
        v[2 * j + 1] = __builtin_bit_cast(float, w[j] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void values(u4 w, float (&v)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __builtin_bit_cast(float, static_cast<uint32_t>(w[j]));
}
__device__ __forceinline__ u4 packed(const float (&v)[8]) {
    u4 w;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        w[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{v[2 * j], v[2 * j + 1]}), bf2));
    return w;
}
__device__ __forceinline__ u4 packed(const float (&v)[4]) {
    u4 w;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = __builtin_bit_cast(uint32_t, v[j]);
    return w;
}
// the first n elements of a vector (kWhole: all of them)
template <bool kWhole, bool kNt, typename T>
__device__ __forceinline__ u4 load_some(const T* p, int n) {
    if (kWhole || n >= kE<T>) return load16<kNt>(p);
    u4 w = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 0; j < kE<T>; ++j) {
        if (j >= n) break;
        if constexpr (sizeof(T) == 2) w[j >> 1] |= static_cast<uint32_t>(p[j]) << (16 * (j & 1));
        else w[j] = __builtin_bit_cast(uint32_t, static_cast<float>(p[j]));
    }
    return w;
}
template <bool kWhole, typename T>
__device__ __forceinline__ void put_some(T* p, u4 w, int n) {
    if (kWhole || n >= kE<T>) return put16(p, w);
#pragma unroll
    for (int j = 0; j < kE<T>; ++j) {
        if (j >= n) break;
        if constexpr (sizeof(T) == 2) p[j] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
        else p[j] = __builtin_bit_cast(float, static_cast<uint32_t>(w[j]));
    }
}

// kP cosines or sines; kWhole: aligned to as many.
template <bool kWhole, int kP>
__device__ __forceinline__ void angles(const float* p, float (&v)[kP]) {
    if constexpr (kWhole && kP >= 4) {
#pragma unroll
        for (int j = 0; j < kP; j += 4) {
            const f4 w = *reinterpret_cast<const f4*>(p + j);
#pragma unroll
            for (int q = 0; q < 4; ++q) v[j + q] = w[q];
        }
    } else {
#pragma unroll
        for (int j = 0; j < kP; ++j) v[j] = p[j];
    }
}

// `lanes` threads take a head: first those of its pairs (kE pairs each in the half layout, whose two vectors lie
// half apart, kE / 2 in the interleaved one, whose pairs are one vector), then one a vector behind the rotated
// elements; `across` of them are there (a head may need more than a workgroup has).  `slots` heads go side by
// side.  A workgroup takes `per` tokens or, where there are many heads, one of `cuts` parts (<= heads) of them.
// About two heads a thread: queries and keys of 4096 tokens x 192 heads x 128 bf16, a token's heads in 1 / 2 / 3 parts
// 71.9 / 68.8 / 66.4 us; 16384 tokens x 40 x 64, 1 / 2 / 4 heads a thread 42.2 / 33.4 / 36.7 us.
struct RotaryShape {
    int pair_lanes, lanes, across, slots, per, cuts;
};

template <typename T, bool kInter, bool kWhole, bool kNt>
__global__ void __launch_bounds__(kThreads) rotary_kernel(Rotary a, RotaryShape s, int64_t token0) {
    constexpr int kV = kE<T>, kP = kInter ? kV / 2 : kV;   // elements of a vector, pairs of a lane
    __shared__ alignas(16) float cs[kPairs + 16], sn[kPairs + 16];
    const int half = a.rot / 2;
    // each XCD takes runs of 16 neighbouring workgroups (30.2 -> 29.4 us, 8192 tokens x 40 x 128 bf16 interleaved)
    constexpr uint32_t kXcds = 8, kRun = 16, kPer = kXcds * kRun;
    uint32_t block = blockIdx.x;
    if (block < gridDim.x / kPer * kPer) block = block / kPer * kPer + block % kXcds * kRun + block % kPer / kXcds;
    const uint32_t down = block / s.cuts, cut = block - down * s.cuts;
    const int64_t first = token0 + static_cast<int64_t>(down) * s.per;
    const int tokens = static_cast<int>(min(static_cast<int64_t>(s.per), a.batch * a.tokens - first));
    // sequence and token of the workgroup's first, the same in every lane; the others count on from it
    const int64_t b0 = first / a.tokens, t0 = first - b0 * a.tokens;
    for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
        const int tok = i / half, pair = i - tok * half;
        int64_t x;
        if (a.positions) {
            x = a.positions[first + tok];
        } else {
            for (x = t0 + tok; x >= a.tokens;) x -= a.tokens;
            x += a.start;
        }
        const double turns = static_cast<double>(x) * a.freqs[pair] * kTurn;
        float si, co;
        sincospif(2.0f * static_cast<float>(turns - __builtin_rint(turns)), &si, &co);
        cs[i] = co * a.scale;
        sn[i] = si * a.scale * a.sign;
    }
    __syncthreads();
    const int lane0 = threadIdx.x % s.across, slot = threadIdx.x / s.across;
    if (slot >= s.slots) return;
    // the workgroup's heads of q and then k, `low` to `low` + `all`
    const int heads = static_cast<int>(a.heads);
    const int64_t whole = a.heads + a.kv_heads;
    const int low = static_cast<int>(whole * cut / s.cuts), all = static_cast<int>(whole * (cut + 1) / s.cuts) - low;
    for (int lane = lane0; lane < s.lanes; lane += s.across) {
        const bool rotates = lane < s.pair_lanes;
        // where the lane's (first) vector starts, and how many pairs or elements are left from there
        const int pair = lane * kP;
        const int at = rotates ? (kInter ? 2 * pair : pair) : a.rot + (lane - s.pair_lanes) * kV;
        const int n = rotates ? min(half - pair, kP) : min(a.head_dim - at, kV);
        // one head's vectors ahead of the one that is rotated
        struct Item {
            const T* x;
            T* y;
            u4 u, w;
            int tok;
        };
        int tok = slot / all, h = low + slot - tok * all;
        int64_t b = b0, t = t0 + tok;
        const auto fetch = [&](Item& it) {
            for (; t >= a.tokens; t -= a.tokens) ++b;
            const Heads& from = h < heads ? a.q : a.k;
            const Heads& to = h < heads ? a.q_out : a.k_out;
            const int hh = h < heads ? h : h - heads;
            it.x = static_cast<const T*>(from.p) + b * from.batch + t * from.token + hh * from.head + at;
            it.y = static_cast<T*>(to.p) + b * to.batch + t * to.token + hh * to.head + at;
            it.tok = tok;
            if (rotates) {
                it.u = load_some<kWhole, kNt>(it.x, kInter ? 2 * n : n);
                if constexpr (!kInter) it.w = load_some<kWhole, kNt>(it.x + half, n);
            } else if (it.x != it.y) {
                it.u = load_some<kWhole, kNt>(it.x, n);
            }
            for (h += s.slots; h >= low + all; h -= all) {
                ++tok;
                ++t;
            }
        };
        const auto finish = [&](const Item& it) {
            if (!rotates) {
                if (it.x != it.y) put_some<kWhole>(it.y, it.u, n);
                return;
            }
            float c[kP], z[kP], p[kV];
            angles<kWhole>(cs + it.tok * half + pair, c);
            angles<kWhole>(sn + it.tok * half + pair, z);
            values(it.u, p);
            if constexpr (kInter) {
#pragma unroll
                for (int j = 0; j < kP; ++j) {
                    const float A = p[2 * j], B = p[2 * j + 1];
                    p[2 * j] = A * c[j] - B * z[j];
                    p[2 * j + 1] = A * z[j] + B * c[j];
                }
                put_some<kWhole>(it.y, packed(p), 2 * n);
            } else {
                float q[kV];
                values(it.w, q);
#pragma unroll
                for (int j = 0; j < kP; ++j) {
                    const float A = p[j], B = q[j];
                    p[j] = A * c[j] - B * z[j];
                    q[j] = A * z[j] + B * c[j];
                }
                put_some<kWhole>(it.y, packed(p), n);
                put_some<kWhole>(it.y + half, packed(q), n);
            }
        };
        if (tok >= tokens) continue;
        Item now;
        fetch(now);
        while (tok < tokens) {
            Item next;
            fetch(next);
            finish(now);
            now = next;
        }
        finish(now);
    }
}

constexpr int64_t kMaxBlocks = int64_t{1} << 20;  // of a launch

template <typename T, bool kInter>
hipError_t rotate(const Rotary& a, hipStream_t stream) {
    constexpr int kV = kE<T>, kP = kInter ? kV / 2 : kV;
    RotaryShape s;
    const int half = a.rot / 2, rest = a.head_dim - a.rot;
    s.pair_lanes = (half + kP - 1) / kP;
    s.lanes = s.pair_lanes + (rest + kV - 1) / kV;
    s.across = std::min(s.lanes, kThreads);
    s.slots = kThreads / s.across;
    const bool whole = half % kP == 0 && rest % kV == 0;
    const int64_t all = a.heads + a.kv_heads, tokens = a.batch * a.tokens;
    // (but workgroups for the whole device)
    int64_t per = std::max<int64_t>(1, 2 * kThreads / (all * s.lanes));
    s.cuts = static_cast<int>(std::min(all, std::max<int64_t>(1, all * s.lanes / (2 * kThreads))));
    per = std::min({per, std::max<int64_t>(1, tokens / 512), static_cast<int64_t>(kPairs / half)});
    s.per = static_cast<int>(per);
    const bool nt = 2 * tokens * all * a.head_dim * static_cast<int64_t>(sizeof(T)) >= kNtBytes;
    const int64_t most = std::max<int64_t>(1, kMaxBlocks / s.cuts) * per;
    for (int64_t t0 = 0; t0 < tokens; t0 += most) {
        const dim3 grid(static_cast<uint32_t>((std::min(tokens - t0, most) + per - 1) / per * s.cuts));
        if (whole) {
            if (nt) rotary_kernel<T, kInter, true, true><<<grid, kThreads, 0, stream>>>(a, s, t0);
            else rotary_kernel<T, kInter, true, false><<<grid, kThreads, 0, stream>>>(a, s, t0);
        } else {
            if (nt) rotary_kernel<T, kInter, false, true><<<grid, kThreads, 0, stream>>>(a, s, t0);
            else rotary_kernel<T, kInter, false, false><<<grid, kThreads, 0, stream>>>(a, s, t0);
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_rotary(const Rotary& a, hipStream_t stream) {
    if (a.bf16) return a.interleaved ? rotate<uint16_t, true>(a, stream) : rotate<uint16_t, false>(a, stream);
    return a.interleaved ? rotate<float, true>(a, stream) : rotate<float, false>(a, stream);
}

}  // namespace fsdp
