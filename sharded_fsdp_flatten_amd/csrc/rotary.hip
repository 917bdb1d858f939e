// rotary.hip -- rotary positions of queries and keys, forward and backward.
//
// Pair i of a head at position x turns by w = x f_i: (a, b) -> (a cos w - b sin w, a sin w + b cos w).
// The cosine and sine of a (token, pair) serve every head, so a lane owns eight pairs of a token and walks
// its heads with sixteen numbers in registers; q and k share them in one launch.  Bound by HBM: every
// element is read and written once.
#include <algorithm>

#include "layer_dev.h"
#include "train.h"

namespace fsdp {
namespace {

constexpr double kTurn = 0.15915494309189533577;  // 1 / (2 pi)

// Lanes of a workgroup: `lanes` of them own a head (its vectors of 8 pairs, then the vectors of 8
// elements behind the rotated ones), `slots` heads side by side, `per` tokens a workgroup.
struct RotaryShape {
    int pair_vecs, lanes, slots, per;
};

template <typename T, bool kInter>
__global__ void __launch_bounds__(kThreads) rotary_kernel(Rotary a, RotaryShape s, int64_t token0) {
    const int lane = threadIdx.x % s.lanes, slot = threadIdx.x / s.lanes;
    if (slot >= s.slots) return;
    const int all = static_cast<int>(a.heads + a.kv_heads);
    const int across = s.per > 1 ? slot / all : 0;           // which of the workgroup's tokens
    if (across >= s.per) return;
    const int64_t token = token0 + static_cast<int64_t>(blockIdx.x) * s.per + across;
    if (token >= a.batch * a.tokens) return;
    const int64_t b = token / a.tokens, t = token - b * a.tokens;
    const int half = a.rot / 2;
    const bool rotates = lane < s.pair_vecs;
    const int first = rotates ? lane * kV : a.rot + (lane - s.pair_vecs) * kV;  // pair, or element
    const int n = min(kV, rotates ? half - first : a.head_dim - first);
    float c[kV], sn[kV];
    if (rotates) {
        const double x = static_cast<double>(a.positions ? a.positions[token] : a.start + t);
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            c[j] = sn[j] = 0.0f;
            if (j < n) {
                const double turns = x * a.freqs[first + j] * kTurn;
                const float r = static_cast<float>(turns - __builtin_rint(turns));
                float si, co;
                sincospif(2.0f * r, &si, &co);
                c[j] = co * a.scale;
                sn[j] = si * a.scale * a.sign;
            }
        }
    }
    const int step = s.per > 1 ? all : s.slots;
    for (int h = s.per > 1 ? slot - across * all : slot; h < all; h += step) {
        const bool is_q = h < a.heads;
        const Heads& from = is_q ? a.q : a.k;
        const Heads& to = is_q ? a.q_out : a.k_out;
        const int64_t hh = is_q ? h : h - a.heads;
        const T* x = static_cast<const T*>(from.p) + b * from.batch + t * from.token + hh * from.head;
        T* y = static_cast<T*>(to.p) + b * to.batch + t * to.token + hh * to.head;
        if (!rotates) {
            if (x == y) continue;
            Vec<T> v;
            vload<false>(v, x + first, n);
            vstore(v, y + first, n);
            continue;
        }
        // a pair's elements are `half` apart, or next to each other
        Vec<T> u, w;
        float p[kV], q[kV];
        if constexpr (kInter) {
            vload<false>(u, x + 2 * first, 2 * n);
            vload<false>(w, x + 2 * first + kV, 2 * n - kV);
            float e[2 * kV];
            u.get(e);
            w.get(e + kV);
#pragma unroll
            for (int j = 0; j < kV; ++j) {
                const float A = e[2 * j], B = e[2 * j + 1];
                e[2 * j] = A * c[j] - B * sn[j];
                e[2 * j + 1] = A * sn[j] + B * c[j];
            }
            put8(y + 2 * first, e, 2 * n);
            put8(y + 2 * first + kV, e + kV, 2 * n - kV);
        } else {
            vload<false>(u, x + first, n);
            vload<false>(w, x + half + first, n);
            u.get(p);
            w.get(q);
#pragma unroll
            for (int j = 0; j < kV; ++j) {
                const float A = p[j], B = q[j];
                p[j] = A * c[j] - B * sn[j];
                q[j] = A * sn[j] + B * c[j];
            }
            put8(y + first, p, n);
            put8(y + half + first, q, n);
        }
    }
}

constexpr int64_t kMaxBlocks = int64_t{1} << 22;  // of 256 threads: a grid's threads fit 32 bits

}  // namespace

hipError_t launch_rotary(const Rotary& a, hipStream_t stream) {
    RotaryShape s;
    s.pair_vecs = (a.rot / 2 + kV - 1) / kV;
    s.lanes = s.pair_vecs + (a.head_dim - a.rot + kV - 1) / kV;
    // heads longer than a workgroup's lanes are cut by the caller's limit on head_dim
    s.slots = std::max(1, kThreads / s.lanes);
    const int64_t all = a.heads + a.kv_heads;
    s.per = static_cast<int>(std::max<int64_t>(1, s.slots / all));
    const int64_t tokens = a.batch * a.tokens;
    for (int64_t t0 = 0; t0 < tokens; t0 += kMaxBlocks * s.per) {
        const int64_t blocks = (std::min(tokens - t0, kMaxBlocks * s.per) + s.per - 1) / s.per;
        const dim3 grid(static_cast<uint32_t>(blocks));
        if (a.bf16) {
            if (a.interleaved) rotary_kernel<uint16_t, true><<<grid, kThreads, 0, stream>>>(a, s, t0);
            else rotary_kernel<uint16_t, false><<<grid, kThreads, 0, stream>>>(a, s, t0);
        } else {
            if (a.interleaved) rotary_kernel<float, true><<<grid, kThreads, 0, stream>>>(a, s, t0);
            else rotary_kernel<float, false><<<grid, kThreads, 0, stream>>>(a, s, t0);
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace fsdp
