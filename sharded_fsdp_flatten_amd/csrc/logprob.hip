// logprob.hip -- log probabilities of given tokens with entropy and top alternatives, and the gradient of
// the logits.
//
// With z = scale x over a row of logits: one pass keeps, for every lane, the largest x so far, the sum of
// 2^(k (x - m)) and (for the entropy) of that times its exponent, k = scale log2 e; sums move to a new
// maximum by one factor.  The lanes' triples join in a fixed order.  Bound by HBM: forward reads every
// logit once, backward reads and writes each once.
#include <algorithm>
#include <type_traits>

#include "layer_dev.h"
#include "train.h"

namespace fsdp {
namespace {

constexpr double kLog2e = 1.4426950408889634074, kLn2 = 0.69314718055994530942;

// Running sums of a part of a row with the largest logit m, against r = anchor(m): s = sum of e, t = sum of
// e u with u = k x - r (one rounding), e = 2^u.  A part without logits above -infinity has m = -infinity,
// s = t = 0.
struct Part {
    float m, s, t;
};
// k m, rounded, held within 2^24: against it -infinity gives e = 0 instead of NaN.  What its rounding
// lacks, at most a half, is made up once for a row (finish).  A run of a row whose own k m lies beyond (masks of the
// type's lowest value and nothing else, or logits as large as a scale's 2^24) is summed again, of differences from the
// maximum: its r is k m itself.
constexpr float kFar = 0x1p24f;
__device__ __forceinline__ float anchor(float m, float k) { return __builtin_amdgcn_fmed3f(m * k, -kFar, kFar); }
__device__ __forceinline__ bool beyond(float m, float k) {
    return m > -INFINITY && m < INFINITY && fabsf(anchor(m, k)) == kFar;
}
// k m less the r of a run's sums.
__device__ __forceinline__ float lacking(float m, float k) { return beyond(m, k) ? 0.0f : fmaf(m, k, -anchor(m, k)); }

// How far the exponents of sums against `from`'s anchor move when they are taken against that of `to`, the
// larger one; never so far that 2^shift times a sum's weight could be infinity times 0.  The anchors are what the sums
// of lanes and waves stand against, held or not: where their run's maximum lies beyond, the sums go.
__device__ __forceinline__ float shift(float from, float to, float k) {
    return fmaxf(anchor(from, k) - anchor(to, k), -1000.0f);
}
// The same between runs, where either may stand against its k m instead: (from - to) k is exact but for one rounding
// where the two are near each other.
__device__ __forceinline__ float run_shift(float from, float to, float k) {
    if (from == -INFINITY || !(beyond(from, k) || beyond(to, k))) return shift(from, to, k);
    return fmaxf((from - to) * k - lacking(from, k) + lacking(to, k), -1000.0f);
}
// e u without 0 x infinity: far below -149 e is 0; a NaN stays one
__device__ __forceinline__ float weighted(float e, float u) { return e * fmaxf(u, -200.0f); }

// What the sums of a whole row come to.
struct Row {
    float max, logsum, entropy;
    __device__ bool empty() const { return max == -INFINITY && logsum == 0.0f; }
    __device__ float logprob(float x, float scale) const {
        return empty() ? -INFINITY : fmaf(x, scale, -max) - logsum;
    }
};
__device__ __forceinline__ Row finish(const Part& p, float scale, float k) {
    Row r;
    r.max = p.m * scale;
    if (r.max == -INFINITY && p.s == p.s) return Row{-INFINITY, 0.0f, 0.0f};  // nothing above -infinity
    if (r.max == INFINITY) return Row{INFINITY, NAN, NAN};
    const float ls = logf(p.s), lacks = lacking(p.m, k);
    // against the exact k m, and then of the rounded maximum, so that the two add up
    r.logsum = ls - static_cast<float>(kLn2) * lacks + fmaf(p.m, scale, -r.max);
    r.entropy = ls - static_cast<float>(kLn2) * (p.t / p.s);
    return r;
}

__device__ __forceinline__ float value(const uint16_t* p) {
    return __builtin_bit_cast(float, static_cast<uint32_t>(*p) << 16);
}
__device__ __forceinline__ float value(const float* p) { return *p; }

// 16 bytes of logits: neighbouring lanes read neighbouring vectors, so that every load of a wave takes whole
// lines.
template <typename T> constexpr int kE = 16 / sizeof(T);
template <bool kNt>
__device__ __forceinline__ u4 load16(const void* p) {
    return kNt ? __builtin_nontemporal_load(static_cast<const u4*>(p)) : *static_cast<const u4*>(p);
}
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
// stores at any element
__device__ __forceinline__ void put16(void* p, u4 w) { __builtin_nontemporal_store(w, static_cast<u4e*>(p)); }
__device__ __forceinline__ void put1(uint16_t* p, float v) {
    *p = static_cast<uint16_t>(__builtin_bit_cast(uint32_t, __builtin_convertvector((f2{v, 0.0f}), bf2)));
}
__device__ __forceinline__ void put1(float* p, float v) { *p = v; }

// A logit's place in the order of alternatives: larger values first, then lower places; NaN as
// -infinity.  Larger keys come first; no two of a row are equal; 0 is below every key.
__device__ __forceinline__ uint32_t rank_bits(float x) {
    x = x == x ? x + 0.0f : -INFINITY;  // -0 as 0
    const uint32_t b = __builtin_bit_cast(uint32_t, x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float ranked_value(uint32_t o) {
    return __builtin_bit_cast(float, o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ uint64_t key_of(uint32_t bits, uint32_t place) {
    return static_cast<uint64_t>(bits) << 32 | static_cast<uint32_t>(~place);
}

// ---------------------------------------------------------------------------
// over a wave
// ---------------------------------------------------------------------------
__device__ __forceinline__ float wave_max(float x) {
    const auto bits = [](float a) { return __builtin_bit_cast(uint32_t, a); };
    const auto val = [](uint32_t a) { return __builtin_bit_cast(float, a); };
    x = fmaxf(x, val(dpp<kQuadXor1>(bits(x))));
    x = fmaxf(x, val(dpp<kQuadXor2>(bits(x))));
    x = fmaxf(x, val(dpp<kHalfMirror>(bits(x))));
    x = fmaxf(x, val(dpp<kMirror>(bits(x))));
    const auto r = __builtin_amdgcn_permlane16_swap(bits(x), bits(x), false, false);
    x = fmaxf(val(r[0]), val(r[1]));
    const auto t = __builtin_amdgcn_permlane32_swap(bits(x), bits(x), false, false);
    return fmaxf(val(t[0]), val(t[1]));
}
// Join of the wave's lanes, the same in each: moved to the common maximum, then added.  (A product fused
// into the first addition would round differently in the two lanes that exchange it.)
template <bool kRuns = false>
__device__ __forceinline__ Part wave_join(Part p, float k) {
#pragma clang fp contract(off)
    const float m = wave_max(p.m), d = kRuns ? run_shift(p.m, m, k) : shift(p.m, m, k), f = __builtin_amdgcn_exp2f(d);
    return Part{m, wave_sum(p.s * f), wave_sum(f * (p.t + d * p.s))};
}
// The largest key of the lane's quad.
__device__ __forceinline__ uint64_t quad_key(uint64_t key) {
    const auto swapped = [](uint64_t x, auto ctrl) {
        return static_cast<uint64_t>(dpp<decltype(ctrl)::value>(static_cast<uint32_t>(x >> 32))) << 32 |
               dpp<decltype(ctrl)::value>(static_cast<uint32_t>(x));
    };
    key = max(key, swapped(key, std::integral_constant<int, kQuadXor1>{}));
    return max(key, swapped(key, std::integral_constant<int, kQuadXor2>{}));
}
__device__ __forceinline__ uint64_t lane_key(uint64_t key, int l) {
    return static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(key >> 32), l))) << 32 |
           static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(key), l));
}
// The key that `want` of the wave's keys are larger than, of every kG-th lane; 0 where there are no more.
template <int kG>
__device__ __forceinline__ uint64_t wave_key(uint64_t key, int want) {
    int rank = 0;
#pragma unroll
    for (int l = 0; l < 64; l += kG) rank += lane_key(key, l) > key ? 1 : 0;
    const uint64_t has = __ballot(rank == want && key != 0);
    return has ? lane_key(key, __builtin_ctzll(has)) : 0;
}
// How many of the first n keys are larger; kL neighbouring lanes, which hold the same key, share the counting.
template <int kL>
__device__ __forceinline__ int larger(const uint64_t* keys, uint32_t n, uint64_t key) {
    const uint32_t l = threadIdx.x % kL;
    int place = 0;
    uint32_t j = 0;
    for (; j + 8 * kL <= n; j += 8 * kL) {
#pragma unroll
        for (int q = 0; q < 8; ++q) place += keys[j + q * kL + l] > key ? 1 : 0;
    }
    for (; j + l < n; j += kL) place += keys[j + l] > key ? 1 : 0;
    if constexpr (kL >= 4) {
        place += dpp<kQuadXor1>(place);
        place += dpp<kQuadXor2>(place);
    }
    if constexpr (kL == 16) {
        place += dpp<kHalfMirror>(place);
        place += dpp<kMirror>(place);
    }
    return place;
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
// Candidates for the alternatives that a workgroup of kT threads gathers (where there are more, the bound is
// found exactly), and the segments of its run (longer ones have larger segments).  A wave's own rows, of
// kShort columns at most, hold less, so that a compute unit holds more of them: top 20 with entropy of 16384 x 500 bf16
// 30 us, with as much as the others 47; of 16384 x 3000 41 and 68.
constexpr int64_t kShort = 4096;
template <int kT> constexpr int kCandidates = kT == 64 ? 512 : 1024;
template <typename T, int kT> constexpr uint32_t kSegments = kT == 64 ? kShort / kE<T> : 2048;

// A row in `parts` runs of `per` columns, one workgroup each; with more than one the runs' results meet
// in the workspace and logprob_join_kernel.
struct Split {
    uint32_t parts;
    int64_t per;
};
// What a run leaves in the workspace (then its `top` keys in falling order; a run is longer than that).
constexpr int kPartFloats = 4;

__device__ __forceinline__ float* part_at(const LogprobFwd& a, const Split& sp, int64_t row, uint32_t part) {
    return a.workspace + (row * sp.parts + part) * (kPartFloats + 2 * a.top);
}

// The row's given token (-1: none), and its logit.
__device__ __forceinline__ int64_t given(const LogprobFwd& a, int64_t row) {
    const int64_t tok = a.tokens ? a.tokens[row] : -1;
    return tok < a.cols ? tok : -1;
}
template <typename T>
__device__ __forceinline__ float logit(const LogprobFwd& a, int64_t row, int64_t tok) {
    return tok >= 0 ? value(static_cast<const T*>(a.x.p) + row * a.x.pitch + tok) : 0.0f;
}
// Statistics, and the given token's log probability, of a whole row.
__device__ __forceinline__ void put_row(const LogprobFwd& a, int64_t row, const Row& r, int64_t tok, float x) {
    a.max[row] = r.max;
    a.logsum[row] = r.logsum;
    if (a.entropy) a.entropy[row] = r.entropy;
    if (a.tokens) a.logprob[row] = tok >= 0 ? r.logprob(x, a.scale) : 0.0f;
}
__device__ __forceinline__ void put_top(const LogprobFwd& a, int64_t row, int i, uint64_t key, const Row& r) {
    a.top_token[row * a.top + i] = static_cast<uint32_t>(~static_cast<uint32_t>(key));
    a.top_logprob[row * a.top + i] = r.logprob(ranked_value(static_cast<uint32_t>(key >> 32)), a.scale);
}

// The k largest keys of a run of n > k logits in `keys` (in any order).  Every pass
// counts the next eight bits of the keys that begin as the k-th largest does.
template <typename T, int kT>
__device__ uint32_t select(const T* x, int64_t n, int64_t c0, int k, uint64_t* keys, uint32_t* count) {
    uint32_t* const hist = reinterpret_cast<uint32_t*>(keys);
    const int t = threadIdx.x;
    uint64_t prefix = 0;
    uint32_t left = static_cast<uint32_t>(k);   // the wanted key's place among those that begin with prefix
    for (int bit = 56; bit >= 0; bit -= 8) {
        for (int i = t; i < 256; i += kT) hist[i] = 0;
        __syncthreads();
        for (int64_t c = t; c < n; c += kT) {
            const uint64_t key = key_of(rank_bits(value(x + c)), static_cast<uint32_t>(c0 + c));
            if (bit == 56 || key >> (bit + 8) == prefix) atomicAdd(&hist[key >> bit & 255u], 1u);
        }
        __syncthreads();
        // every wave: four digits a lane, the largest digits in the first lane
        const int l = t & 63;
        uint32_t each[4], sum = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) sum += each[q] = hist[255 - 4 * l - q];
        uint32_t before = sum;
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t o = __shfl_up(before, d);
            if (l >= d) before += o;
        }
        before -= sum;
        uint32_t digit = 0, rest = 0;
        bool here = false;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (!here && before < left && left <= before + each[q]) {
                here = true;
                digit = 255u - 4u * l - q;
                rest = left - before;
            }
            if (!here) before += each[q];
        }
        const int from = __builtin_ctzll(__ballot(here));
        prefix = prefix << 8 | static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(digit), from));
        left = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(rest), from));
        __syncthreads();
    }
    if (t == 0) *count = 0;
    __syncthreads();
    for (int64_t c = t; c < n; c += kT) {
        const uint64_t key = key_of(rank_bits(value(x + c)), static_cast<uint32_t>(c0 + c));
        if (key >= prefix) keys[atomicAdd(count, 1u)] = key;
    }
    __syncthreads();
    return static_cast<uint32_t>(k);
}

// Lane t of a run takes its head's element t (the head ends at a 16-byte boundary, or where loads go past the cache at a
// whole line: 2048 x 50257 fp32 65.6 -> 62.4 us, 8192 x 50257 bf16 123.2 -> 121.1), vectors t, t + kT, ... of 16 bytes,
// and its tail's element t - kEdge.
//
// Alternatives: the pass over the logits also leaves the largest logit of every segment in LDS (kSeg
// neighbouring lanes' vectors, 128 bytes; one vector in short rows).  The k-th largest of them, with the lower
// segment first among equals, bounds the k-th largest logit from below, for they are different logits, and
// only the k best segments can hold one of the k.  A bound that takes no sorting across waves is the lowest over
// the waves of the (k / waves)-th best of their lanes' segments (of quads', where enough are left).  The
// segments that reach it are read again, all at once, what reaches it is gathered, and the place of a candidate is
// how many are larger.  Where too many reach it (rows that allow fewer than k tokens, rows whose largest
// logits meet in a few segments) the k-th largest key itself is found, eight bits a pass over the row.
// Measured, top 20 with entropy of 2048 x 50257 fp32: lanes that read all of their own logits again 107 us (they
// are 16 bytes in every 4 KB: as many lines as the row has), segments 78 (73 with what came after).
template <typename T, int kT, bool kEntropy, bool kTop, bool kNt>
__global__ void __launch_bounds__(kT) logprob_fwd_kernel(LogprobFwd a, Split sp, int64_t row0) {
    constexpr int kW = kT / 64, kV = kE<T>, kU = 32 / kV;
    constexpr uint32_t kSeg = kT == 64 ? 1 : 8, kAll = kSegments<T, kT>;
    constexpr int kMost = kCandidates<kT>;
    // Few rows: the last wave alone joins the waves' sums and writes the row, and it asks for the given token ahead, for all
    // instructions of the other fifteen share four SIMDs (16 x 50257 bf16 with 8 / 64 alternatives 11.0 / 14.8 -> 10.2 / 13.6
    // us).  Where rows fill the chip a wave's wait for the token costs more (16384 x 3001: 20.9 without and 22.0 with it).
    constexpr bool kLone = kT == 1024;
    __shared__ Part parts[kW], sums;
    __shared__ Row stats;
    __shared__ bool far;
    __shared__ uint64_t bound[kTop ? kW : 1];
    __shared__ alignas(16) uint64_t keys[kTop ? kMost : 2];
    __shared__ uint32_t segs[kTop ? kAll : 1];      // rank_bits of the segments' largest
    __shared__ uint16_t chosen[kTop ? kMost : 1];  // segments that reach the bound
    __shared__ uint32_t count, picked;
    const int64_t row = row0 + blockIdx.x / sp.parts;
    const uint32_t part = blockIdx.x % sp.parts;
    const int64_t c0 = part * sp.per;
    const int64_t n = min(a.cols - c0, sp.per);
    const T* x = static_cast<const T*>(a.x.p) + row * a.x.pitch + c0;
    const float k = static_cast<float>(a.scale * kLog2e);
    const int t = threadIdx.x;
    constexpr int kAlign = kNt ? 128 : 16, kEdge = kAlign / sizeof(T);
    static_assert(kEdge + kV <= kT);
    const int head = static_cast<int>(min(static_cast<int64_t>((kAlign - reinterpret_cast<uintptr_t>(x) % kAlign) % kAlign / sizeof(T)), n));
    const uint32_t nv = static_cast<uint32_t>((n - head) / kV);
    const int tail = static_cast<int>(n - head - static_cast<int64_t>(nv) * kV);
    const T* body = x + head;

    const bool last = t >> 6 == kW - 1, whole = sp.parts == 1;
    int64_t tok = kLone && last && whole ? given(a, row) : -1;

    Part p = {-INFINITY, 0.0f, 0.0f};
    // segments of kSeg << wide vectors
    const uint32_t all = (nv + kSeg - 1) / kSeg;
    const int wide = kTop && all > kAll ? 32 - __builtin_clz((all - 1) / kAll) : 0;
    if constexpr (kTop) {
        if (t == 0) count = picked = 0;
        for (uint32_t i = t; i < min(all, kAll); i += kT) segs[i] = 0;
        __syncthreads();
    }
    const auto one = [&](float v) {
        const float m = fmaxf(p.m, v), d = shift(p.m, m, k), f = __builtin_amdgcn_exp2f(d);
        const float u = fmaf(v, k, -anchor(m, k)), e = __builtin_amdgcn_exp2f(u);
        if (kEntropy) p.t = f * (p.t + d * p.s) + weighted(e, u);
        p.s = p.s * f + e;
        p.m = m;
    };
    const auto load = [&](uint32_t i) { return load16<kNt>(reinterpret_cast<const char*>(body) + i * 16u); };
    // kU vectors from place i on (those beyond the end were read from the last one)
    const auto take = [&](const u4* w, uint32_t i, auto full) {
        constexpr bool kWhole = decltype(full)::value;
        float v[kU][kV], g[kU], top = p.m;
#pragma unroll
        for (int j = 0; j < kU; ++j) {
            values(w[j], v[j]);
            // maxima that keep a NaN need no quieting of their operands
            g[j] = v[j][0];
#pragma unroll
            for (int q = 1; q < kV; ++q) g[j] = __builtin_elementwise_maximum(g[j], v[j][q]);
            if (!kWhole && i + j * kT >= nv) g[j] = -INFINITY;
            top = __builtin_elementwise_maximum(top, g[j]);
        }
        if (top != top) {   // and where there is one are taken again without it
            top = p.m;
#pragma unroll
            for (int j = 0; j < kU; ++j) {
                g[j] = -INFINITY;
#pragma unroll
                for (int q = 0; q < kV; ++q) g[j] = fmaxf(g[j], v[j][q]);
                if (!kWhole && i + j * kT >= nv) g[j] = -INFINITY;
                top = fmaxf(top, g[j]);
            }
        }
        if constexpr (kTop) {
#pragma unroll
            for (int j = 0; j < kU; ++j) {
                uint32_t b = __builtin_bit_cast(uint32_t, g[j] + 0.0f);
                b ^= static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u;   // as rank_bits; no NaN is left
                if constexpr (kSeg == 8) {
                    b = max(b, dpp<kQuadXor1>(b));
                    b = max(b, dpp<kQuadXor2>(b));
                    b = max(b, dpp<kHalfMirror>(b));
                }
                // a segment's first lane has it; lanes beyond the end hold -infinity
                if (t % kSeg == 0 && (kWhole || i + j * kT < nv)) atomicMax(&segs[(i + j * kT) / kSeg >> wide], b);
            }
        }
        const float r = anchor(top, k), d = fmaxf(anchor(p.m, k) - r, -1000.0f), f = __builtin_amdgcn_exp2f(d);
        // the step's own sums first: 32 terms, then one sum a step, instead of one long chain of roundings
        float sum = 0.0f, sum_u = 0.0f;
#pragma unroll
        for (int j = 0; j < kU; ++j) {
            if (!kWhole && i + j * kT >= nv) break;
#pragma unroll
            for (int q = 0; q < kV; ++q) {
                const float u = fmaf(v[j][q], k, -r), e = __builtin_amdgcn_exp2f(u);
                sum += e;
                if (kEntropy) sum_u += weighted(e, u);
            }
        }
        if (kEntropy) p.t = f * (p.t + d * p.s) + sum_u;
        p.s = p.s * f + sum;
        p.m = top;
    };
    // a segment's lanes go together, so that its maximum meets
    constexpr uint32_t kLast = kTop ? kSeg - 1 : 0;
    uint32_t i = t;
    if constexpr (kT < 1024) {   // (few rows take few steps: one path, for its instructions are fetched once)
        for (; (i | kLast) + (kU - 1) * kT < nv; i += kU * kT) {
            u4 w[kU];
#pragma unroll
            for (int j = 0; j < kU; ++j) w[j] = load(i + j * kT);
            take(w, i, std::true_type{});
        }
    }
    for (; (i & ~kLast) < nv; i += kU * kT) {
        u4 w[kU];
#pragma unroll
        for (int j = 0; j < kU; ++j) w[j] = load(min(i + j * kT, nv - 1));
        take(w, i, std::false_type{});
    }
    // head and tail
    const bool in_tail = t >= kEdge && t - kEdge < tail;
    const int64_t edge = t < head ? t : in_tail ? n - tail + (t - kEdge) : -1;
    if (edge >= 0) one(value(x + edge));

    // the lanes' sums, then the waves'
    float* ws = whole ? nullptr : part_at(a, sp, row, part);
    float x_tok = logit<T>(a, row, tok);
    const auto put_sums = [&](const Part& q, const Row& r) {
        if (whole) {
            put_row(a, row, r, tok, x_tok);
        } else {
            ws[0] = q.m;
            ws[1] = q.s;
            ws[2] = q.t;
        }
    };
    const auto meet = [&](Part q) {
        q = wave_join(q, k);
        if constexpr (kW > 1) {
            if ((t & 63) == 0) parts[t >> 6] = q;
        }
        __syncthreads();
        if constexpr (kW > 1) {
            if (!kLone || last) q = wave_join((t & 63) < kW ? parts[t & 63] : Part{-INFINITY, 0.0f, 0.0f}, k);
        }
        return q;
    };
    const auto again = [&](float m) {
        Part q = {m, 0.0f, 0.0f};
        for (int64_t c = t; c < n; c += kT) {
            const float u = (value(x + c) - m) * k, e = __builtin_amdgcn_exp2f(u);
            q.s += e;
            q.t += weighted(e, u);
        }
        return meet(q);
    };
    p = meet(p);
    Row r;
    if constexpr (kLone) {
        if (last) {
            r = finish(p, a.scale, k);
            if ((t & 63) == 0) {
                far = beyond(p.m, k);
                sums = p;
                stats = r;
                if (!beyond(p.m, k)) put_sums(p, r);
            }
        }
    } else {
        if (beyond(p.m, k)) {
            __syncthreads();
            p = again(p.m);
        }
        r = finish(p, a.scale, k);
        if (t == 0) {
            if (whole) {
                tok = given(a, row);
                x_tok = logit<T>(a, row, tok);
            }
            put_sums(p, r);
        }
    }
    const uint32_t n_segs = kTop && nv ? ((all - 1) >> wide) + 1 : 0;
    if constexpr (kTop) {
        // (the sums' meeting was a barrier: the segments are complete)
        uint64_t best = 0;
        for (uint32_t i = t; i < n_segs; i += kT) best = max(best, key_of(segs[i], i));
        // the first waves have a segment in each of their lanes
        const int full = max(1, static_cast<int>(min(n_segs / 64, static_cast<uint32_t>(kW))));
        const int share = (a.top + full - 1) / full - 1;
        uint64_t low = ~uint64_t{0};
        // ranks of quads where four times the alternatives are left of them, else of lanes
        if ((t >> 6) < full)
            low = 4 * a.top <= 16 * full ? wave_key<4>(quad_key(best), share) : wave_key<1>(best, share);
        if ((t & 63) == 0) bound[t >> 6] = low;
    }
    if constexpr (kTop || kLone) __syncthreads();
    if constexpr (kLone) {
        if (far) {
            p = again(sums.m);
            if (last) {
                r = finish(p, a.scale, k);
                if ((t & 63) == 0) {
                    stats = r;
                    put_sums(p, r);
                }
            }
        }
    }
    if constexpr (kTop) {
        uint64_t reach = bound[0];
#pragma unroll
        for (int i = 1; i < kW; ++i) reach = min(reach, bound[i]);
        for (uint32_t i = t; i < n_segs; i += kT) {
            if (key_of(segs[i], i) < reach) continue;
            const uint32_t slot = atomicAdd(&picked, 1u);
            if (slot < kMost) chosen[slot] = static_cast<uint16_t>(i);
        }
        __syncthreads();
        const auto put = [&](int i, uint64_t key) {
            if (whole) put_top(a, row, i, key, kLone ? stats : r);
            else reinterpret_cast<uint64_t*>(ws + kPartFloats)[i] = key;
        };
        // against the bound a logit counts as if it had its segment's place
        const auto gather = [&](float v, uint32_t seg, int64_t col) {
            const uint32_t bits = rank_bits(v);
            if (key_of(bits, seg) < reach) return;
            const uint32_t slot = atomicAdd(&count, 1u);
            if (slot < kMost) keys[slot] = key_of(bits, static_cast<uint32_t>(c0 + col));
        };
        const uint32_t taken = picked;
        if (taken <= kMost) {
            const int vecs = __builtin_ctz(kSeg) + wide;
            const uint32_t work = taken << vecs;
            // (one vector a thread reads what is usually chosen)
            for (uint32_t i = t; i < work; i += kT) {
                const uint32_t seg = chosen[i >> vecs], at = (seg << vecs) + (i & ((1u << vecs) - 1));
                if (at >= nv) continue;
                float v[kV];
                values(load16<false>(reinterpret_cast<const char*>(body) + at * 16u), v);
#pragma unroll
                for (int q = 0; q < kV; ++q) gather(v[q], seg, head + static_cast<int64_t>(at) * kV + q);
            }
            // the head comes before every segment, the tail behind all of them
            if (edge >= 0) gather(value(x + edge), in_tail ? n_segs : 0u, edge);
        } else if (t == 0) {
            count = kMost + 1;
        }
        __syncthreads();
        uint32_t got = count;
        if (got > kMost) {
            __syncthreads();
            got = select<T, kT>(x, n, c0, a.top, keys, &count);
        }
        constexpr int kL = kLone ? 16 : 1;   // lanes a key
        for (uint32_t i = t / kL; i < got; i += kT / kL) {
            const uint64_t key = keys[i];
            const int place_of = larger<kL>(keys, got, key);
            if (t % kL == 0 && place_of < a.top) put(place_of, key);
        }
    }
}

// The runs of a row joined, in their order; the alternatives from the runs' own.
constexpr int kMaxParts = 64;
template <typename T>
__global__ void __launch_bounds__(kThreads) logprob_join_kernel(LogprobFwd a, Split sp, int64_t row0) {
    __shared__ alignas(16) uint64_t keys[kMaxParts * kMaxTop];
    __shared__ uint32_t count;
    const int64_t row = row0 + blockIdx.x;
    const int t = threadIdx.x;
    const float k = static_cast<float>(a.scale * kLog2e);
    if (t == 0) count = 0;
    const int64_t tok = given(a, row);
    const float x_tok = logit<T>(a, row, tok);
    // every wave joins all of them
    const int l = t & 63;
    Part p = {-INFINITY, 0.0f, 0.0f};
    uint64_t least = ~uint64_t{0};
    if (l < static_cast<int>(sp.parts)) {
        const float* ws = part_at(a, sp, row, l);
        p = Part{ws[0], ws[1], ws[2]};
        // the runs' shares of the alternatives: all runs together have that many at least as large as the
        // lowest of these
        if (a.top) least = reinterpret_cast<const uint64_t*>(ws + kPartFloats)[(a.top + sp.parts - 1) / sp.parts - 1];
    }
    p = wave_join<true>(p, k);
    const Row r = finish(p, a.scale, k);
    if (t == 0) put_row(a, row, r, tok, x_tok);
    if (!a.top) return;
    for (int d = 1; d < 64; d <<= 1)
        least = min(least, static_cast<uint64_t>(__shfl_xor(static_cast<unsigned long long>(least), d)));
    __syncthreads();
    for (uint32_t i = t; i < sp.parts * a.top; i += kThreads) {
        const uint64_t key = reinterpret_cast<const uint64_t*>(part_at(a, sp, row, i / a.top) + kPartFloats)[i % a.top];
        if (key < least) continue;
        keys[atomicAdd(&count, 1u)] = key;
    }
    __syncthreads();
    const uint32_t got = count;
    constexpr int kL = 4;
    for (uint32_t i = t / kL; i < got; i += kThreads / kL) {
        const uint64_t key = keys[i];
        const int place = larger<kL>(keys, got, key);
        if (t % kL == 0 && place < a.top) put_top(a, row, place, key, r);
    }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// One shot: a workgroup takes two vectors a thread of one row (where rows are short a wave takes a row, four
// vectors a thread), aligned as the logits are, to whole lines where they go past the cache (126.7 -> 121.8 us, 4096 x 50257 bf16);
// block 0 of a row also takes its head and its tail.  A lane stores what it has read, so that the gradient may take the
// logits' place.
// Vectors a thread, 4096 x 50257 bf16 with a tenth of the rows padded: 1 / 2 / 3 / 4 / 8 163 / 127.5 / 133 / 137 / 147 us; 2048 x
// 50257 fp32 with entropy 181 / 132 / 138 / 138 / 406.  Cached loads 2-7% slower there, cached stores 5-20% everywhere.
template <int kT> constexpr int kBwdVecs = kT == 64 ? 4 : 2;
template <typename T, int kT, bool kEntropy, bool kNt>
__global__ void __launch_bounds__(kThreads) logprob_bwd_kernel(LogprobBwd a, int64_t row0, int64_t rows, uint32_t across) {
    constexpr int kV = kE<T>, kN = kBwdVecs<kT>;
    const int t = threadIdx.x % kT;
    // each XCD takes runs of 16 neighbouring blocks: 128.5 -> 126 us (4096 x 50257 bf16; runs of 64 / 128 / 256 / 512 126.0 /
    // 127.0 / 127.5 / 131)
    constexpr uint32_t kXcds = 8, kRunOf = 16, kPer = kXcds * kRunOf;
    uint32_t at = blockIdx.x;
    if (at < gridDim.x / kPer * kPer) at = at / kPer * kPer + at % kXcds * kRunOf + at % kPer / kXcds;
    const uint32_t unit = at * (kThreads / kT) + (kT < kThreads ? __builtin_amdgcn_readfirstlane(threadIdx.x / kT) : 0);
    const uint32_t down = unit / across, block = unit - down * across;
    if (down >= rows) return;
    const int64_t row = row0 + down;
    const T* x = static_cast<const T*>(a.x.p) + row * a.x.pitch;
    T* y = static_cast<T*>(a.dx.p) + row * a.dx.pitch;
    const float mx = a.max[row], logsum = a.logsum[row];
    const int64_t tok = a.dl ? a.tokens[row] : -1;
    const bool has = tok >= 0 && tok < a.cols;
    const float dl = has ? a.dl[row] : 0.0f, dh = kEntropy ? a.dh[row] : 0.0f;
    const bool zero = (dl == 0.0f && dh == 0.0f) || (mx == -INFINITY && logsum == 0.0f);
    const float H = kEntropy ? a.entropy[row] : 0.0f;
    constexpr float c2 = static_cast<float>(kLog2e);
    const float l2 = logsum * c2, base = dl + dh * H, back = -a.scale, up = dl * a.scale;
    const int64_t n = a.cols;
    constexpr int kAlign = kNt && kT > 64 ? 128 : 16, kEdge = kAlign / sizeof(T);
    const int head = static_cast<int>(min(static_cast<int64_t>((kAlign - reinterpret_cast<uintptr_t>(x) % kAlign) % kAlign / sizeof(T)), n));
    const int64_t nv = (n - head) / kV;
    const auto grad = [&](float v) {
        const float d = fmaf(v, a.scale, -mx), p = __builtin_amdgcn_exp2f(fmaf(d, c2, -l2));
        // log p far below its place in p is 0 times infinity
        if constexpr (kEntropy) return back * p * fmaf(dh, fmaxf(d - logsum, -1e4f), base);
        else return back * dl * p;
    };
    const int64_t first = static_cast<int64_t>(block) * (kT * kN) + t;
    if (zero) {
#pragma unroll
        for (int j = 0; j < kN; ++j) {
            const int64_t i = first + j * kT;
            if (i < nv) put16(y + head + i * kV, u4{0u, 0u, 0u, 0u});
        }
    } else {
        u4 w[kN];
#pragma unroll
        for (int j = 0; j < kN; ++j) {
            const int64_t i = first + j * kT;
            w[j] = u4{0u, 0u, 0u, 0u};
            if (i < nv) w[j] = load16<kNt>(x + head + i * kV);
        }
#pragma unroll
        for (int j = 0; j < kN; ++j) {
            const int64_t i = first + j * kT;
            if (i >= nv) break;
            float v[kV];
            values(w[j], v);
#pragma unroll
            for (int q = 0; q < kV; ++q) v[q] = grad(v[q]);
            const int64_t at = tok - (head + i * kV);
            if (has && at >= 0 && at < kV) {
#pragma unroll
                for (int q = 0; q < kV; ++q) v[q] += q == at ? up : 0.0f;
            }
            put16(y + head + i * kV, packed(v));
        }
    }
    if (block == 0) {
        const int64_t tail = n - head - nv * kV;
        const int64_t c = t < head ? t : t >= kEdge && t - kEdge < tail ? head + nv * kV + (t - kEdge) : -1;
        if (c >= 0) {
            const float g = zero ? 0.0f : grad(value(x + c)) + (has && c == tok ? up : 0.0f);
            put1(y + c, g);
        }
    }
}

constexpr int64_t kMaxBlocks = int64_t{1} << 22;  // of 256 threads: a grid's threads fit 32 bits

// Runs of a row: a few long rows leave most compute units idle, so that they are cut into runs of at
// least kRun columns, up to kFill workgroups; joining them costs a launch.  bf16 rows in runs and whole, us: 16 x 50257 7.4 and
// 5.4 (not cut), 16 x 131072 7.2 and 8.3, 16 x 262144 7.2 and 13.3, 64 x 262144 11.1 and 14.5.
constexpr int64_t kRun = 32768, kFill = 256;
Split plan_split(int64_t rows, int64_t cols) {
    int64_t parts = std::min<int64_t>({cols / kRun, kFill / std::max<int64_t>(rows, 1), kMaxParts});
    parts = std::max<int64_t>(parts, 1);
    const int64_t per = ((cols + parts - 1) / parts + kV - 1) / kV * kV;
    // runs differ by the last one's lack of up to 8 (parts - 1) columns: none is shorter than the alternatives wanted
    static_assert(kRun - 8 * (kMaxParts - 1) >= kMaxTop);
    return {static_cast<uint32_t>((cols + per - 1) / per), per};
}

template <typename T, int kT, bool kTop, bool kNt>
void launch(const LogprobFwd& a, const Split& sp, int64_t r0, uint32_t blocks, hipStream_t stream) {
    if (a.entropy) logprob_fwd_kernel<T, kT, true, kTop, kNt><<<blocks, kT, 0, stream>>>(a, sp, r0);
    else logprob_fwd_kernel<T, kT, false, kTop, kNt><<<blocks, kT, 0, stream>>>(a, sp, r0);
}
template <typename T, int kT, bool kNt>
void forward(const LogprobFwd& a, const Split& sp, int64_t r0, uint32_t blocks, hipStream_t stream) {
    if (a.top) launch<T, kT, true, kNt>(a, sp, r0, blocks, stream);
    else launch<T, kT, false, kNt>(a, sp, r0, blocks, stream);
}

template <typename T>
hipError_t forward_rows(const LogprobFwd& a, hipStream_t stream) {
    const Split sp = plan_split(a.rows, a.cols);
    const int64_t most = kMaxBlocks / 4 / sp.parts;   // of up to 1024 threads
    // Past the cache where a call's logits outgrow it, rows at any element: 4096 x 50257 bf16 (412 MB), 256 threads, cached 75.0,
    // nt 68.4 us (64 with 512 threads and whole lines); 2048 x 50257 fp32 72.1 and 66.7 (62).
    const bool nt = a.rows * a.cols * static_cast<int64_t>(sizeof(T)) >= kNtBytes;
    // Threads of a workgroup, each choice against 256 (us, its own time first; bf16 but where said):
    //   64, a wave a row, up to kShort columns: 16384 x 3000 19.6 / 32; x 6000 37.8 / 40.5, but 99 / 85 with 20 alternatives.
    //   512, from 2048 long rows past the cache: 4096 x 50257 64.2 / 65.0, 2560 x 50257 41.7 / 43.9, 8192 x 33000 84.1 / 88.1.  Not
    //     16384 x 20000, 119 / 103, 1024 x 131072, 47.0 / 43.7, or 4096 x 50257 with 20 alternatives, 91.5 / 86.7.  In fp32 at
    //     50257 columns it makes little difference on either side of the border: 1536 rows 47.5 / 47.7, 2048 61.8 / 62.0, 2560
    //     76.7 / 76.4; with 20 alternatives 57.2 / 55.7, 73.1 / 74.7, 87.8 / 87.2.
    //   128, short rows without alternatives: 16384 x 5001 34.8 / 41.7, x 10001 55.9 / 66.2, x 16001 86.8 / 89.3.  Not x 20001,
    //     103.2 / 102.7, x 6001 with 20 alternatives, 93.0 / 84.5, or fp32, x 8001 87.7 / 82.6.
    //   1024, under 512 workgroups of 16384 columns and more: 200 x 262144 21 / 33.7, 200 x 50257 7.1 / 8.2.  Not 600 x 50257, 14.6 /
    //     13.4 (27.6 / 22.6 with alternatives), or 200 x 12000 with alternatives, 9.5 / 8.8.
    const int64_t long_row = int64_t{a.top ? 128 : 64} << 10;
    const bool short_row = sizeof(T) == 2 && !a.top && sp.per <= 16384;
    for (int64_t r0 = 0; r0 < a.rows; r0 += most) {
        const int64_t rows = std::min(a.rows - r0, most);
        const uint32_t blocks = static_cast<uint32_t>(rows * sp.parts);
        if (sp.per <= kShort) forward<T, 64, false>(a, sp, r0, blocks, stream);
        else if (nt && blocks >= 2048 && sp.per * static_cast<int64_t>(sizeof(T)) >= long_row)
            forward<T, 512, true>(a, sp, r0, blocks, stream);
        else if (blocks >= 512 && short_row)
            nt ? launch<uint16_t, 128, false, true>(a, sp, r0, blocks, stream) : launch<uint16_t, 128, false, false>(a, sp, r0, blocks, stream);
        else if (blocks >= 512 || sp.per < 16384)
            nt ? forward<T, 256, true>(a, sp, r0, blocks, stream) : forward<T, 256, false>(a, sp, r0, blocks, stream);
        else forward<T, 1024, false>(a, sp, r0, blocks, stream);
        if (sp.parts > 1) logprob_join_kernel<T><<<static_cast<uint32_t>(rows), kThreads, 0, stream>>>(a, sp, r0);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

int64_t logprob_workspace_floats(int64_t rows, int64_t cols, int32_t top) {
    if (rows == 0 || cols == 0) return 0;
    const Split sp = plan_split(rows, cols);
    return sp.parts == 1 ? 0 : rows * sp.parts * (kPartFloats + 2 * top);
}

hipError_t launch_logprob_forward(const LogprobFwd& a, hipStream_t stream) {
    return a.bf16 ? forward_rows<uint16_t>(a, stream) : forward_rows<float>(a, stream);
}

namespace {

template <typename T, int kT>
hipError_t backward_rows(const LogprobBwd& a, hipStream_t stream) {
    constexpr int kRows = kThreads / kT;
    const int64_t across = std::max<int64_t>(1, (a.cols / kE<T> + kT * kBwdVecs<kT> - 1) / (kT * kBwdVecs<kT>));
    const int64_t most = std::max<int64_t>(1, kMaxBlocks / across) * kRows;
    const bool nt = a.rows * a.cols * static_cast<int64_t>(2 * sizeof(T)) >= kNtBytes;
    for (int64_t r0 = 0; r0 < a.rows; r0 += most) {
        const int64_t rows = std::min(a.rows - r0, most);
        const dim3 grid(static_cast<uint32_t>((rows * across + kRows - 1) / kRows));
        const uint32_t c = static_cast<uint32_t>(across);
        if (a.dh) {
            if (nt) logprob_bwd_kernel<T, kT, true, true><<<grid, kThreads, 0, stream>>>(a, r0, rows, c);
            else logprob_bwd_kernel<T, kT, true, false><<<grid, kThreads, 0, stream>>>(a, r0, rows, c);
        } else {
            if (nt) logprob_bwd_kernel<T, kT, false, true><<<grid, kThreads, 0, stream>>>(a, r0, rows, c);
            else logprob_bwd_kernel<T, kT, false, false><<<grid, kThreads, 0, stream>>>(a, r0, rows, c);
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_logprob_backward(const LogprobBwd& a, hipStream_t stream) {
    // a wave a row where its vectors are one shot of it
    if (a.bf16)
        return a.cols <= 64 * kBwdVecs<64> * kE<uint16_t> ? backward_rows<uint16_t, 64>(a, stream)
                                                      : backward_rows<uint16_t, kThreads>(a, stream);
    return a.cols <= 64 * kBwdVecs<64> * kE<float> ? backward_rows<float, 64>(a, stream)
                                               : backward_rows<float, kThreads>(a, stream);
}

}  // namespace fsdp
