// layer.hip -- HIP kernels of the layer operators for CDNA4 (gfx950): 8-bit activation
// checkpoints, LayerNorm / RMSNorm and the MLP activation, forward and backward.
//
// All of them read their operands once and write their results once (the norms of rows beyond
// 16384 columns read a row again for each pass over it); what bounds them is HBM.  Every lane owns
// vectors of 8 neighbouring columns (one 16-byte load of bf16, two of fp32, 8 bytes of codes), four
// lanes of a quad one group of 32 columns with one scale.  Rows may start at any element: global
// loads and stores of several dwords work at any address, so odd pitches and widths take the
// same path, and the vector that the row's end cuts is read from the row's last whole vector or
// element by element.  The norms' backward pass over rows in registers is in norm_backward.h.
// Sums, statistics and the arithmetic between load and store are binary32; a result is rounded
// once, when it is stored.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "layer.h"
#include "layer_dev.h"

// Nothing here is compared bit for bit with separately rounded steps (scaling by powers of two
// is exact either way), so multiply-adds may be fused.
#pragma clang fp contract(fast)

namespace fsdp {
namespace {

// ---------------------------------------------------------------------------
// activations
// ---------------------------------------------------------------------------
enum { kNone = 0, kRelu = 1, kGelu = 2, kGeluTanh = 3, kSilu = 4 };

// e^x by the hardware's 2^x: off by |x| 2^-24 and one rounding, relative.
__device__ __forceinline__ float fast_exp(float x) {
    return __builtin_amdgcn_exp2f(x * 1.44269504088896341f);
}
// 1 - s of s = 1 / (1 + e) as e s, whose error is relative: f' multiplies it by h, and the GELU's by up to
// 6 more.  The clamp (part of the product's instruction) makes inf x 0 a 0, where s is 0 too.
__device__ __forceinline__ float rest(float e, float s) { return __builtin_amdgcn_fmed3f(e * s, 0.0f, 1.0f); }
// f(h) and f'(h).
template <int kF>
__device__ __forceinline__ void activate(float h, float* y, float* d) {
    if constexpr (kF == kRelu) {
        *y = h <= 0.0f ? 0.0f : h;                       // NaN stays NaN
        *d = h > 0.0f ? 1.0f : (h <= 0.0f ? 0.0f : h);
    } else if constexpr (kF == kSilu) {
        const float e = fast_exp(-h), s = __builtin_amdgcn_rcpf(1.0f + e);
        *y = h * s;
        *d = s * (1.0f + h * rest(e, s));
    } else if constexpr (kF == kGeluTanh) {
        // (1 + tanh u) / 2 = 1 / (1 + e^-2u), u = sqrt(2/pi) (h + 0.044715 h^3).
        // h^2 is capped where the logistic function is flat, so that no product overflows to 0 x inf;
        // a NaN comes through h
        constexpr float a = 0.79788456080286536f, c = 0.044715f, l = -2.0f * a * 1.44269504088896341f;
        const float h2 = __builtin_fminf(h * h, 1000.0f);
        const float e = __builtin_amdgcn_exp2f(h * (l + l * c * h2)), s = __builtin_amdgcn_rcpf(1.0f + e);
        *y = h * s;
        *d = s + *y * rest(e, s) * (2.0f * a + 6.0f * a * c * h2);
    } else {
        // Q = Phi(-|h|) = e^(-h^2/2) R(|h|).  R, the scaled complementary error function's half, is analytic
        // in q = a / (a + 3), which takes a >= 0 to [0, 1): a polynomial of degree 9 in q, the minimax of the
        // relative error on [0, 14.6] (1.0e-8 with these coefficients, fitted to erfcx in binary64), with R(0)
        // = 1/2 held exactly, so that near 0 the reciprocal's error reaches Q only times q.  Q is within
        // 1e-7 and within (6 + 4|h| + h^2) 2^-24 of itself; a form of a bounded absolute error alone loses the
        // negative tail, where y is h Q.  The clamp (part of the product's instruction) turns an infinite h's
        // q into a number; the exponential is 0 there.  bf16 4096 x 5120 with checkpoint forward 23.5 us and
        // from it backward 35.2, fp32 36.4 and 58.0 (22.1, 34.9, 36.2 and 58.1 with five coefficients and Phi
        // off by 4e-7).
        const float a = __builtin_fabsf(h);
        const float q = __builtin_amdgcn_fmed3f(a * __builtin_amdgcn_rcpf(a + 3.0f), 0.0f, 1.0f);
        const float e = __builtin_amdgcn_exp2f(h * h * (-0.5f * 1.44269504088896341f));
        float r = 2.719713748e-02f;
        r = r * q - 9.296188504e-02f;
        r = r * q + 8.368366957e-02f;
        r = r * q + 9.343822487e-03f;
        r = r * q + 6.212504953e-02f;
        r = r * q - 1.587376297e-01f;
        r = r * q - 2.869739830e-01f;
        r = r * q + 1.053155661e+00f;
        r = r * q - 1.196826577e+00f;
        r = r * q + 0.5f;
        const float tail = r * e;
        const float phi = h < 0.0f ? tail : 1.0f - tail;
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
Tiles plan_tiles(int64_t rows, int64_t cols, int widest = 8) {
    const int64_t nv = (cols + kCkptGroup - 1) / kCkptGroup * (kCkptGroup / kV);
    int best = 2;
    while (best < 5 && (int64_t{1} << best) < nv) ++best;
    if (best == 5) {
        // of 32, 64, ... vectors the width that leaves the fewest lanes idle
        for (int k = 6; k <= widest; ++k) {
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

// The dispatcher deals workgroups to the eight XCDs in turn.  This hands each of them runs of
// `run` consecutive tiles instead (a bijection of the whole groups of 8 run; what is left over, and
// run == 0, stays as dealt), so that an XCD reads and writes longer stretches of memory.
__device__ __forceinline__ uint32_t xcd_order(uint32_t b, uint32_t blocks, uint32_t run) {
    const uint32_t span = 8u * run;
    if (b >= blocks / max(span, 1u) * span) return b;
    const uint32_t r = b % span;
    return b - r + (r & 7u) * run + (r >> 3);
}
// Pack 8192 x 12288 one row a lane: as dealt 58.2 us, runs of 16 / 64 / 256 tiles 53.6 / 53.4 /
// 55.5; unpack 54.7 as dealt, 52.9 with 64.  Below 4096 tiles a run is too large a part of the launch.
uint32_t xcd_run(uint32_t blocks) { return blocks >= 4096u ? 64u : 0u; }

// Rows of a lane where only a checkpoint is written or read: four from kLongTiles tiles on, all
// loads in flight before the first store (pack 8192 x 12288 bf16, 49152 tiles: 49.7 us against 54.4
// with one, unpack 51.0 against 53.7; 10240 tiles: 11.8 against 11.7 and 11.3 against 10.3).  An
// activation always takes one (ReLU 2048 x 65536: 106.6 us against 116.1 with four).
constexpr int kLongRows = 4;
constexpr int64_t kLongTiles = 32768;

// y = f(x) and the checkpoint of x, one tile of kRows rows a lane per workgroup.
template <typename T, int kF, bool kNt, int kRows>
__global__ void __launch_bounds__(kThreads) act_fwd_kernel(ActFwd a, int k, uint32_t across, uint32_t run) {
    const uint32_t block = xcd_order(blockIdx.x, gridDim.x, run);
    const uint32_t down = block / across, tile = block - down * across;
    const int high = kThreads >> k;
    const int64_t row = static_cast<int64_t>(down) * kRows * high + (threadIdx.x >> k);
    const int64_t c = ((static_cast<int64_t>(tile) << k) + (threadIdx.x & ((1 << k) - 1))) * kV;
    const int n = static_cast<int>(min(a.cols - c, int64_t{kV}));
    Vec<T> x[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u)
        vload<kNt>(x[u], static_cast<const T*>(a.x.p) + min(row + u * high, a.rows - 1) * a.x.pitch + c, n);
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        const int64_t r = row + u * high;
        if (r >= a.rows) return;  // whole quads leave together (k >= 2)
        float v[kV];
        x[u].get(v);
        if (a.ckpt.codes) pack8<kF == kNone>(a.ckpt, r, c, n, v);
        if constexpr (kF != kNone) {
            float y[kV], d;
#pragma unroll
            for (int j = 0; j < kV; ++j) activate<kF>(v[j], &y[j], &d);
            put8(static_cast<T*>(a.y.p) + r * a.y.pitch + c, y, n);
        }
    }
}

template <typename T, int kRows>
__global__ void __launch_bounds__(kThreads)
unpack_kernel(int64_t rows, int64_t cols, CkptRows q, RowsOut x, int k, uint32_t across, uint32_t run) {
    const uint32_t block = xcd_order(blockIdx.x, gridDim.x, run);
    const uint32_t down = block / across, tile = block - down * across;
    const int high = kThreads >> k;
    const int64_t row = static_cast<int64_t>(down) * kRows * high + (threadIdx.x >> k);
    const int64_t c = ((static_cast<int64_t>(tile) << k) + (threadIdx.x & ((1 << k) - 1))) * kV;
    const int n = static_cast<int>(min(cols - c, int64_t{kV}));
    if (n <= 0) return;
    u2 code[kRows];
    uint32_t byte[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        const int64_t r = min(row + u * high, rows - 1);
        code[u] = code_load(q.codes + r * q.code_pitch + c, n);
        byte[u] = q.scales[r * q.scale_pitch + c / kCkptGroup];
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        const int64_t r = row + u * high;
        if (r >= rows) return;
        float v[kV];
        decode8(code[u], byte[u], q.int8 != 0, v);
        put8(static_cast<T*>(x.p) + r * x.pitch + c, v, n);
    }
}

// ---------------------------------------------------------------------------
// column sums: partial sums per workgroup, then their sum in a fixed order
// ---------------------------------------------------------------------------
// The lanes of a tile's rows add their 8 columns in LDS, row by row; the first row's lanes
// write the workgroup's partial sums.  Called by every thread.
template <int kT>
__device__ __forceinline__ void tile_partial(const float* s, float* lds, int k, float* out, int n) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kV; ++j) lds[j * kT + threadIdx.x] = s[j];
    __syncthreads();
    // every thread adds up columns of its own
    for (int i = threadIdx.x; i < (kV << k); i += kT) {
        const int j = i >> k, l = i & ((1 << k) - 1);
        float t = lds[j * kT + l];
        for (int r = 1; r < (kT >> k); ++r) t += lds[j * kT + l + (r << k)];
        lds[j * kT + l] = t;   // of this column no other thread reads
    }
    __syncthreads();
    if (threadIdx.x >> k) return;
    if (n == kV) {
        *(f4e*)out = f4{lds[threadIdx.x], lds[kT + threadIdx.x], lds[2 * kT + threadIdx.x], lds[3 * kT + threadIdx.x]};
        *(f4e*)(out + 4) = f4{lds[4 * kT + threadIdx.x], lds[5 * kT + threadIdx.x], lds[6 * kT + threadIdx.x], lds[7 * kT + threadIdx.x]};
        return;
    }
#pragma unroll
    for (int j = 0; j < kV; ++j)
        if (j < n) out[j] = lds[j * kT + threadIdx.x];
}

// A workgroup sums 32 columns (one 128-byte line of a partial row): 8 lanes of 4 columns by
// kSumThreads / 8 slices of the partial rows, up to 8 of its slice's rows in flight a thread.  Each
// slice adds its rows in order, then the slices of a wave and the waves add up in a fixed tree.  16
// waves, or 4 up to kSumFew partial rows, where 16 have less than two loads a thread: 128 partial
// rows of 65536 columns 7.1 us against 12.4, 256 of 24576 6.4 against 8.4; 512 of 2560 4.6 either
// way.  A slice that went through its rows one load at a time took 9.3 us for the last.
constexpr int kSumCols = 32;
template <int kSumThreads>
__global__ void __launch_bounds__(kSumThreads)
col_sum_kernel(const float* partial, int64_t G, int64_t pitch, int64_t second, int64_t cols, ColOut o0, ColOut o1) {
    constexpr int kSumSlices = kSumThreads / (kSumCols / 4);
    __shared__ f4 lds[kSumThreads / 64][kSumCols / 4];
    const ColOut o = blockIdx.y ? o1 : o0;
    const float* p = partial + (blockIdx.y ? second : 0);
    const int lane = threadIdx.x % (kSumCols / 4), slice = threadIdx.x / (kSumCols / 4);
    const int64_t c = static_cast<int64_t>(blockIdx.x) * kSumCols + 4 * lane;
    const int n = static_cast<int>(min(cols - c, int64_t{4}));
    f4 s = {0.0f, 0.0f, 0.0f, 0.0f};
    constexpr int kAhead = 8;
    for (int64_t g = slice; g < G; g += kAhead * kSumSlices) {
        f4 v[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int64_t r = g + i * kSumSlices;
            v[i] = f4{0.0f, 0.0f, 0.0f, 0.0f};
            if (r < G) {
                const float* q = p + r * pitch + c;
                if (n == 4) {
                    v[i] = *(const f4e*)q;
                } else {
                    for (int j = 0; j < 4; ++j)
                        if (j < n) v[i][j] = q[j];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) s += v[i];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        // lanes 8, 16 and 32 apart hold the wave's other slices
        float x = s[j];
        x += __builtin_bit_cast(float, dpp<kRowRor8>(__builtin_bit_cast(uint32_t, x)));
        s[j] = sum_rows(x);
    }
    if ((threadIdx.x & 63) < kSumCols / 4) lds[threadIdx.x >> 6][lane] = s;
    __syncthreads();
    if (slice || n <= 0) return;
#pragma unroll
    for (int i = 1; i < kSumThreads / 64; ++i) s += lds[i][lane];
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
constexpr int64_t kSumFew = 256;
hipError_t launch_col_sum(const float* partial, int64_t G, int64_t pitch, int64_t cols, ColOut o0,
                          ColOut o1, hipStream_t stream) {
    int64_t second = cols;   // the second output's partial sums lie behind the first one's
    if (!o0.p) {
        o0 = o1;
        o1.p = nullptr;
        partial += cols;
    }
    if (!o0.p) return hipSuccess;
    const auto from = [](ColOut o, int64_t c) {
        if (o.p) o.p = static_cast<char*>(o.p) + c * (o.bf16 ? 2 : 4);
        return o;
    };
    constexpr int64_t kRun = int64_t{1} << 26;   // columns a launch takes at most
    for (int64_t c = 0; c < cols; c += kRun) {
        const int64_t n = std::min(kRun, cols - c);
        const dim3 grid(static_cast<uint32_t>((n + kSumCols - 1) / kSumCols), o1.p ? 2 : 1);
        const auto go = [&](auto kernel, int threads) {
            kernel<<<grid, threads, 0, stream>>>(partial + c, G, pitch, second, n, from(o0, c), from(o1, c));
        };
        if (G <= kSumFew) go(col_sum_kernel<256>, 256);
        else go(col_sum_kernel<1024>, 1024);
    }
    return hipGetLastError();
}

// What a lane reads of one row for the activation's backward pass.
template <typename T, bool kCkpt, bool kNt>
struct ActRow {
    Vec<T> dy, x;
    u2 q;
    uint32_t byte;
    __device__ __forceinline__ void load(const ActBwd& a, int64_t row, int64_t c, int64_t group) {
        dy.template load<kNt>(static_cast<const T*>(a.dy.p) + row * a.dy.pitch + c);
        if constexpr (kCkpt) {
            q = *(const u2e*)(a.ckpt.codes + row * a.ckpt.code_pitch + c);
            byte = a.ckpt.scales[row * a.ckpt.scale_pitch + group];
        } else {
            x.template load<kNt>(static_cast<const T*>(a.x.p) + row * a.x.pitch + c);
        }
    }
    // row of fewer than 8 columns
    __device__ __forceinline__ void load_part(const ActBwd& a, int64_t row, int n) {
        dy.load_part(static_cast<const T*>(a.dy.p) + row * a.dy.pitch, n);
        if constexpr (kCkpt) {
            q = code_load(a.ckpt.codes + row * a.ckpt.code_pitch, n);
            byte = a.ckpt.scales[row * a.ckpt.scale_pitch];
        } else {
            x.load_part(static_cast<const T*>(a.x.p) + row * a.x.pitch, n);
        }
    }
    __device__ __forceinline__ void drop(int k) {
        dy.drop(k);
        if constexpr (kCkpt) q = __builtin_bit_cast(u2, __builtin_bit_cast(uint64_t, q) >> (8 * k));
        else x.drop(k);
    }
};

// dx = dy f'(h), optionally y = f(h) again, and the column sums of dx before its rounding.  A
// workgroup takes one block of 2^k vectors across and kActThreads >> k lanes of kActRows rows
// each, all of whose loads are in flight at once, and ends: its lanes' sums add up in LDS to one
// partial row.  The vector that the row's end cuts is read from the row's last 8 columns (kNarrow:
// there are none); rows past the last read it once more, so that no branch stands between loads.
// Workgroups that walk down their columns with the sums in registers write fewer partial rows and are
// slower all the same: a load behind a store waits for the store, and the whole grid reads and writes
// in step (no sums, 2048 x 65536 from e4m3: one row a lane 146 us, walking 177).  16 waves of one row
// each, 512 columns wide, against 16 of two and 8 of four rows, from e4m3 with y: ReLU 2048 x 65536 166 / 168 /
// 166 us, 4096 x 5120 29.6 / 31.1 / 31.1, GELU (tanh) 8192 x 12288 131 / 126 / 127, 4096 x 5120 32.2 / 31.8 / 32.0,
// 128 x 5120 6.8 / 8.0 / 8.1, GELU 8192 x 12288 151 / 136 / 137 (bf16; fp32 252 / 268 / 264); 1024 columns wide
// 168, 30.6, 136, 33.6, 6.8 and 157.  The arithmetic of SiLU and the GELUs takes as long as the memory or
// longer: 33, 38 (tanh) and 48 vector instructions an element, two of them at a quarter of the rate; ReLU's 29.
// The blocks go to the XCDs as dealt: a line of scale bytes serves eight neighbouring blocks, and each
// XCD reads it (7% more bytes), but runs of 8 to 64 blocks an XCD are slower (ReLU 2048 x 65536 by 3-5%,
// GELU (tanh) 8192 x 12288 by 0-2%).
constexpr int kActThreads = 1024, kActRows = 1;
constexpr int kActWidest = 6;   // log2 of a block's vectors across, at most
template <typename T, int kF, bool kCkpt, bool kNarrow, bool kNt>
__global__ void __launch_bounds__(kActThreads)
act_bwd_kernel(ActBwd a, int k, uint32_t across) {
    __shared__ float lds[kV * kActThreads];
    const uint32_t down = blockIdx.x / across, tile = blockIdx.x - down * across;
    const int64_t c = ((static_cast<int64_t>(tile) << k) + (threadIdx.x & ((1 << k) - 1))) * kV;
    const int n = static_cast<int>(max(min(a.cols - c, int64_t{kV}), int64_t{0}));
    const int64_t at = n > 0 ? min(c, a.cols - kV) : 0, group = n > 0 ? c / kCkptGroup : 0;
    const int skip = n > 0 ? static_cast<int>(c - at) : 0;
    const int high = kActThreads >> k;
    const int64_t row = static_cast<int64_t>(down) * kActRows * high + (threadIdx.x >> k), last = a.rows - 1;
    ActRow<T, kCkpt, kNt> in[kActRows];
#pragma unroll
    for (int u = 0; u < kActRows; ++u) {
        const int64_t r = min(row + u * high, last);
        if constexpr (kNarrow) in[u].load_part(a, r, n);
        else in[u].load(a, r, at, group);
    }
    float s[kV] = {};
#pragma unroll
    for (int u = 0; u < kActRows; ++u) {
        const int64_t r = row + u * high;
        if (r > last || n == 0) continue;
        if (!kNarrow && skip) in[u].drop(skip);
        float h[kV], g[kV], y[kV];
        if constexpr (kCkpt) decode8(in[u].q, in[u].byte, a.ckpt.int8 != 0, h);
        else in[u].x.get(h);
        in[u].dy.get(g);
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            float d;
            activate<kF>(h[j], &y[j], &d);
            g[j] *= d;
            s[j] += g[j];
        }
        put8(static_cast<T*>(a.dx.p) + r * a.dx.pitch + c, g, n);
        if (a.y.p) put8(static_cast<T*>(a.y.p) + r * a.y.pitch + c, y, n);
    }
    if (a.dbias.p) tile_partial<kActThreads>(s, lds, k, a.workspace + static_cast<int64_t>(down) * a.cols + c, n);
}

// ---------------------------------------------------------------------------
// norms, rows of any length: one workgroup per row, the row read again for each pass over it
// ---------------------------------------------------------------------------
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
        vload<false>(t, x + c, n);
        t.get(v);
        if (res) {
            Vec<T> r;
            vload<false>(r, res + c, n);
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
        if (a.ckpt.codes) pack8<false>(a.ckpt, row, c, n, v);
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
        vload<false>(t, static_cast<const T*>(a.x.p) + row * a.x.pitch + c, n);
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
        vload<false>(dy, static_cast<const T*>(a.dy.p) + row * a.dy.pitch + c, n);
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
        vload<false>(dy, static_cast<const T*>(a.dy.p) + row * a.dy.pitch + c, n);
        dy.get(g);
        if (a.dres.p) {
            Vec<T> t;
            vload<false>(t, static_cast<const T*>(a.dres.p) + row * a.dres.pitch + c, n);
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
    if (a.dweight.p) tile_partial<kThreads>(sw, lds, k, out, n);
    if (a.dbias.p) tile_partial<kThreads>(sb, lds, k, out + a.cols, n);
}

// ---------------------------------------------------------------------------
// norms, a row in registers: kT threads (a wave, or a whole workgroup) own a row, kN vectors each
// ---------------------------------------------------------------------------
// Thread t of a row owns vectors t, t + kT, ...; with kWhole every vector is whole or outside, else
// the one that the row's end cuts is read from the row's last 8 columns, and no load is branched
// around.
template <int kT> constexpr int group_threads() { return kT == 64 ? kThreads : kT; }

template <bool kWhole, bool kNt, typename T>
__device__ __forceinline__ void rload(Vec<T>& v, const T* row, int c, int cols) {
    if constexpr (kWhole) {
        if (c < cols) v.template load<kNt>(row + c);
        else v.zero();
    } else {
        v.template load<kNt>(row + (c < cols ? min(c, cols - kV) : 0));
    }
}
// the same of a parameter, which other rows read too
template <bool kWhole>
__device__ __forceinline__ void pload(Vec<uint16_t>& v, const uint16_t* p, int c, int cols) {
    if constexpr (kWhole) {
        if (c < cols) v.r = *(const u4e*)(p + c);
        else v.zero();
    } else {
        v.r = *(const u4e*)(p + (c < cols ? min(c, cols - kV) : 0));
    }
}
// What a vector read from its row's last 8 columns, or outside of it, has to drop.
template <bool kWhole, typename T>
__device__ __forceinline__ void settle(Vec<T>& v, int c, int cols) {
    if constexpr (!kWhole) {
        if (c >= cols) v.zero();
        else if (c > cols - kV) v.drop(c - (cols - kV));
    }
}
template <bool kWhole, typename T>
__device__ __forceinline__ void rput(T* p, const float* f, int n) {
    Vec<T> v;
    v.set(f);
    if constexpr (kWhole) {
        if (n > 0) v.store(p);
    } else {
        vstore(v, p, n);
    }
}

// The parameters' loads are issued with the row's (kP16: bf16 parameters, held as they are; fp32
// ones would take twice the registers and are read when they are used).
template <typename T, bool kP16, int kT, int kN, bool kWhole, bool kNt>
__global__ void __launch_bounds__(group_threads<kT>()) norm_fwd_kernel(NormFwd a) {
    constexpr int kRows = group_threads<kT>() / kT;
    __shared__ float lds[2][kT / 64];
    const int t = threadIdx.x % kT;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows +
                        (kRows > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x / kT) : 0);
    if (kRows > 1 && row >= a.rows) return;
    const int cols = static_cast<int>(a.cols);
    float v[kN][kV];
    Vec<uint16_t> pw[kP16 ? kN : 1], pb[kP16 ? kN : 1];
    {
        Vec<T> x[kN];
        const T* xp = static_cast<const T*>(a.x.p) + row * a.x.pitch;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int c = (t + i * kT) * kV;
            rload<kWhole, kNt>(x[i], xp, c, cols);
        }
        if constexpr (kP16) {
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                const int c = (t + i * kT) * kV;
                pload<kWhole>(pw[i], static_cast<const uint16_t*>(a.weight), c, cols);
                if (a.bias) pload<kWhole>(pb[i], static_cast<const uint16_t*>(a.bias), c, cols);
                else pb[i].zero();
            }
        }
        if (a.residual.p) {
            Vec<T> r[kN];
            const T* rp = static_cast<const T*>(a.residual.p) + row * a.residual.pitch;
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                const int c = (t + i * kT) * kV;
                rload<kWhole, kNt>(r[i], rp, c, cols);
            }
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                float u[kV], w[kV];
                const int c = (t + i * kT) * kV;
                settle<kWhole>(x[i], c, cols);
                settle<kWhole>(r[i], c, cols);
                x[i].get(u);
                r[i].get(w);
#pragma unroll
                for (int j = 0; j < kV; ++j) u[j] += w[j];
                x[i].set(u);
            }
            if (a.sum.p) {
                T* sp = static_cast<T*>(a.sum.p) + row * a.sum.pitch;
#pragma unroll
                for (int i = 0; i < kN; ++i) {
                    const int c = (t + i * kT) * kV;
                    vstore(x[i], sp + c, cols - c);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < kN; ++i) settle<kWhole>(x[i], (t + i * kT) * kV, cols);
        }
#pragma unroll
        for (int i = 0; i < kN; ++i) x[i].get(v[i]);
    }
    const float inv = 1.0f / static_cast<float>(cols);
    float mean = 0.0f;
    if (!a.rms) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < kN; ++i)
#pragma unroll
            for (int j = 0; j < kV; ++j) s += v[i][j];
        mean = group_sum<kT>(s, lds[0]) * inv;
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        const int n = cols - (t + i * kT) * kV;
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const float d = v[i][j] - mean;
            if (kWhole ? n > 0 : n > j) s += d * d;
        }
    }
    const float rstd = 1.0f / __builtin_sqrtf(group_sum<kT>(s, lds[1]) * inv + a.eps);
    if (t == 0) {
        if (a.mean) a.mean[row] = mean;
        a.rstd[row] = rstd;
    }
    if (a.ckpt.codes) {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int c = (t + i * kT) * kV;
            pack8<false>(a.ckpt, row, c, cols - c, v[i]);
        }
    }
    T* yp = static_cast<T*>(a.y.p) + row * a.y.pitch;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        const int c = (t + i * kT) * kV;
        float w[kV], b[kV] = {};
        if constexpr (kP16) {
            settle<kWhole>(pw[i], c, cols);
            if (a.bias) settle<kWhole>(pb[i], c, cols);
            pw[i].get(w);
            pb[i].get(b);
        } else {
            param8(a.weight, false, c, cols - c, w);
            if (a.bias) param8(a.bias, false, c, cols - c, b);
        }
#pragma unroll
        for (int j = 0; j < kV; ++j) v[i][j] = (v[i][j] - mean) * rstd * w[j] + b[j];
        rput<kWhole>(yp + c, v[i], cols - c);
    }
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

// Whether a matrix's rows start on 16-byte boundaries.
bool aligned16(const void* p, int64_t pitch, bool bf16) {
    return (reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(pitch * (bf16 ? 2 : 4))) % 16 == 0;
}
// Whether a call that moves `units` elements for each of rows x cols loads non-temporally.
bool outgrows_cache(int64_t rows, int64_t cols, bool bf16, int units, int64_t bytes = kNtBytes) {
    return rows >= bytes / (bf16 ? 2 : 4) / units / cols;
}
bool norm_fwd_nt(const NormFwd& a) {
    return outgrows_cache(a.rows, a.cols, a.bf16, a.residual.p ? 4 : 2) && aligned16(a.x.p, a.x.pitch, a.bf16) &&
           (!a.residual.p || aligned16(a.residual.p, a.residual.pitch, a.bf16));
}

// body(first row, rows, tiles across, log2 of a tile's vectors, workgroups, whether a lane takes
// kLongRows rows) for each run of rows; `long_rows`: it may.
template <typename F>
hipError_t for_tiles(int64_t rows, int64_t cols, bool long_rows, F&& body) {
    const Tiles t = plan_tiles(rows, cols);
    const bool four = long_rows && t.down * t.across >= kLongTiles;
    const int64_t high = static_cast<int64_t>(kThreads >> t.k) * (four ? kLongRows : 1);
    const int64_t run = std::max<int64_t>(1, kMaxBlocks / t.across) * high;
    for (int64_t r = 0; r < rows; r += run) {
        const int64_t n = std::min(run, rows - r);
        body(r, n, t.across, t.k, static_cast<uint32_t>((n + high - 1) / high * t.across), four);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <typename T>
hipError_t act_forward_t(const ActFwd& a, hipStream_t stream) {
    constexpr bool kNt = sizeof(T) == 2;
    const bool stream_in = kNt && outgrows_cache(a.rows, a.cols, a.bf16, a.f == kNone ? 1 : 2) && aligned16(a.x.p, a.x.pitch, a.bf16);
    return for_tiles(a.rows, a.cols, a.f == kNone, [&](int64_t r, int64_t n, uint32_t across, int k, uint32_t blocks, bool four) {
        ActFwd b = a;
        b.rows = n;
        b.x = skip(a.x, r, a.bf16);
        b.y = skip(a.y, r, a.bf16);
        b.ckpt = skip(a.ckpt, r);
        const auto go = [&](auto cached, auto nt) {
            if (stream_in) nt<<<blocks, kThreads, 0, stream>>>(b, k, across, xcd_run(blocks));
            else cached<<<blocks, kThreads, 0, stream>>>(b, k, across, xcd_run(blocks));
        };
        switch (a.f) {
            case kNone:
                if (four) go(act_fwd_kernel<T, kNone, false, kLongRows>, act_fwd_kernel<T, kNone, kNt, kLongRows>);
                else go(act_fwd_kernel<T, kNone, false, 1>, act_fwd_kernel<T, kNone, kNt, 1>);
                break;
            case kRelu: go(act_fwd_kernel<T, kRelu, false, 1>, act_fwd_kernel<T, kRelu, kNt, 1>); break;
            case kGelu: go(act_fwd_kernel<T, kGelu, false, 1>, act_fwd_kernel<T, kGelu, kNt, 1>); break;
            case kGeluTanh: go(act_fwd_kernel<T, kGeluTanh, false, 1>, act_fwd_kernel<T, kGeluTanh, kNt, 1>); break;
            default: go(act_fwd_kernel<T, kSilu, false, 1>, act_fwd_kernel<T, kSilu, kNt, 1>); break;
        }
    });
}

// The blocks of the activation's backward pass: `t.down` partial rows.
Tiles act_tiles(int64_t rows, int64_t cols) {
    Tiles t = plan_tiles(rows, cols, kActWidest);
    const int64_t high = static_cast<int64_t>(kActThreads >> t.k) * kActRows;
    t.down = (rows + high - 1) / high;
    return t;
}
template <typename T, int kF, bool kCkpt>
void act_backward_f(const ActBwd& a, const Tiles& t, bool nt, hipStream_t stream) {
    constexpr bool kNt = sizeof(T) == 2;   // fp32 vectors are loaded through the cache in any case
    const auto go = [&](auto kernel) {
        kernel<<<static_cast<uint32_t>(t.down * t.across), kActThreads, 0, stream>>>(a, t.k, t.across);
    };
    if (a.cols < kV) go(act_bwd_kernel<T, kF, kCkpt, true, false>);
    else if (kNt && nt) go(act_bwd_kernel<T, kF, kCkpt, false, kNt>);
    else go(act_bwd_kernel<T, kF, kCkpt, false, false>);
}
template <typename T, bool kCkpt>
void act_backward_t(const ActBwd& a, const Tiles& w, bool nt, hipStream_t stream) {
    switch (a.f) {
        case kRelu: return act_backward_f<T, kRelu, kCkpt>(a, w, nt, stream);
        case kGelu: return act_backward_f<T, kGelu, kCkpt>(a, w, nt, stream);
        case kGeluTanh: return act_backward_f<T, kGeluTanh, kCkpt>(a, w, nt, stream);
        default: return act_backward_f<T, kSilu, kCkpt>(a, w, nt, stream);
    }
}

// Rows longer than this (and those shorter than a vector) take the kernels that read a row again
// for each pass.
constexpr int64_t kMaxRowCols = 16384;

// Threads of a row and vectors of a thread for the forward pass over rows in registers: a wave up to
// 2048 columns (no barrier; 16384 x 1280 18.4 us, as a workgroup's row 21.7), then 256 threads, which
// up to six vectors each hold 12288 columns in 193 registers (4096 x 12288 with residual: 67.0 us; 512
// threads of three 70.4), then 512.
struct RowShape {
    int threads, vectors;
};
RowShape fwd_shape(int64_t cols) {
    const int64_t nv = (cols + kV - 1) / kV;
    if (nv <= 256) return {64, static_cast<int>((nv + 63) / 64)};
    if (nv <= 1536) return {256, static_cast<int>((nv + 255) / 256)};
    return {512, 4};
}
// Whether the backward pass holds a row of these columns in registers.
bool bwd_in_registers(int64_t cols) { return cols >= 4 && cols <= kMaxRowCols; }
// Workgroups of the backward pass over rows in registers: each writes a partial row, so there are no
// more than the device holds at once (256 CUs with `resident` each), four rows a group where that
// leaves 64, and below that a row each, for latency.  777 x 5003: 195 workgroups 15.3 us, 389 17.7,
// 512 19.4; 128 x 1280: 32 workgroups 6.9 us, 8 9.7.  Two resident, 512 workgroups against 256: 32768 x 1024
// from int8 45.0 / 50.2 us, 16384 x 1280 from e4m3 29.7 / 28.6.  One resident (a residual gradient in each), 256
// against 512, and against 512 held to 128 registers: fp32 16384 x 704 37.8 / 40.2 / 52.8 us, 16384 x 1280
// 60.8 / 63.6 / 63.6, 4096 x 5120 63.3 / 68.3 / 74.8; bf16 from int8 8192 x 5003 101 / 109 / 115.
int64_t bwd_groups(int64_t rows, int64_t cols, int resident) {
    const int64_t high = std::max(1, 512 / norm_bwd_shape(cols).threads);
    const int64_t each = (rows + high - 1) / high;
    return std::min<int64_t>(256 * resident, std::max(std::min<int64_t>(each, 64), (each + 3) / 4));
}

template <typename T, int kT, int kN>
void norm_fwd_run(const NormFwd& a, hipStream_t stream) {
    constexpr int kRows = group_threads<kT>() / kT;
    const uint32_t blocks = static_cast<uint32_t>((a.rows + kRows - 1) / kRows);
    constexpr bool kNt = sizeof(T) == 2;   // fp32 vectors are loaded through the cache in any case
    const bool whole = a.cols % kV == 0, nt = kNt && whole && norm_fwd_nt(a);
    const auto go = [&](auto kernel) { kernel<<<blocks, group_threads<kT>(), 0, stream>>>(a); };
    if (a.param_bf16) {
        if (nt) go(norm_fwd_kernel<T, true, kT, kN, true, kNt>);
        else if (whole) go(norm_fwd_kernel<T, true, kT, kN, true, false>);
        else go(norm_fwd_kernel<T, true, kT, kN, false, false>);
    } else {
        if (nt) go(norm_fwd_kernel<T, false, kT, kN, true, kNt>);
        else if (whole) go(norm_fwd_kernel<T, false, kT, kN, true, false>);
        else go(norm_fwd_kernel<T, false, kT, kN, false, false>);
    }
}
template <typename T>
void norm_forward_t(const NormFwd& a, hipStream_t stream) {
    if (a.cols < kV || a.cols > kMaxRowCols) {
        norm_fwd_long_kernel<T><<<static_cast<uint32_t>(a.rows), kThreads, 0, stream>>>(a);
        return;
    }
    const RowShape s = fwd_shape(a.cols);
    switch (s.threads + s.vectors) {
#define FSDP_SHAPE(kT, kN) case kT + kN: return norm_fwd_run<T, kT, kN>(a, stream)
        FSDP_SHAPE(64, 1);
        FSDP_SHAPE(64, 2);
        FSDP_SHAPE(64, 3);
        FSDP_SHAPE(64, 4);
        FSDP_SHAPE(256, 2);
        FSDP_SHAPE(256, 3);
        FSDP_SHAPE(256, 4);
        FSDP_SHAPE(256, 5);
        FSDP_SHAPE(256, 6);
        FSDP_SHAPE(512, 4);
#undef FSDP_SHAPE
    }
}

template <typename T, bool kCkpt>
hipError_t norm_backward_t(const NormBwd& a, hipStream_t stream) {
    float* partial = a.workspace;
    int64_t G = 0;
    if (a.rows > 0 && bwd_in_registers(a.cols)) {
        const BwdShape shape = norm_bwd_shape(a.cols);
        G = bwd_groups(a.rows, a.cols, norm_bwd_resident(a.bf16, kCkpt, a.dres.p, shape.threads, shape.vectors));
        const bool nt = outgrows_cache(a.rows, a.cols, a.bf16, 3 + (a.dres.p != nullptr) + (a.y.p != nullptr)) &&
                        aligned16(a.dy.p, a.dy.pitch, a.bf16) && aligned16(a.x.p, a.x.pitch, a.bf16);
        const auto rows = a.bf16 ? (nt ? launch_norm_bwd_rows_bf16_nt : launch_norm_bwd_rows_bf16)
                                 : (nt ? launch_norm_bwd_rows_f32_nt : launch_norm_bwd_rows_f32);
        rows(a, partial, static_cast<uint32_t>(G), stream);
    } else if (a.rows > 0) {
        const Walk w = plan_walk(a.rows, a.cols);
        G = w.chunks;
        float* stat = a.workspace;
        partial = a.workspace + (2 * a.rows + 3) / 4 * 4;
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
    }
    if (a.rows > 0) {
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return launch_col_sum(partial, G, 2 * a.cols, a.cols, a.dweight, a.dbias, stream);
}

}  // namespace

// The fewest threads whose three vectors of 4 hold the row (four, beyond 1024 threads): two of a wave's
// own rows or a few waves' share a workgroup, and its registers allow two of 8 waves a CU.  Rows of
// 1024 and 1280 columns as one wave's, four and five vectors, leave one workgroup a CU, as fast on many
// rows (32768 x 1024 from int8 45.3 us, 16384 x 1280 from e4m3 29.8) and slower on few (128 x 1280 8.9 us
// against 7.0).
BwdShape norm_bwd_shape(int64_t cols) {
    const int64_t nq = (cols + 3) / 4;
    if (nq <= 64) return {64, 1};
    for (int threads = 64; threads < 1024; threads *= 2)
        if (nq <= 3 * threads) return {threads, static_cast<int>((nq + threads - 1) / threads)};
    return {1024, static_cast<int>((nq + 1023) / 1024)};
}

int64_t norm_workspace_floats(int64_t rows, int64_t cols) {
    if (rows == 0 || cols == 0) return 0;
    if (bwd_in_registers(cols)) {
        // the most that any type and source takes
        const BwdShape shape = norm_bwd_shape(cols);
        return 2 * bwd_groups(rows, cols, norm_bwd_resident(true, false, false, shape.threads, shape.vectors)) * cols;
    }
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
    return __builtin_mul_overflow(act_tiles(rows, cols).down, cols, &n) ? -1 : n;
}

hipError_t launch_act_forward(const ActFwd& a, hipStream_t stream) {
    return a.bf16 ? act_forward_t<uint16_t>(a, stream) : act_forward_t<float>(a, stream);
}

hipError_t launch_unpack(int64_t rows, int64_t cols, bool bf16, const CkptRows& q, RowsOut x,
                         hipStream_t stream) {
    return for_tiles(rows, cols, true, [&](int64_t r, int64_t n, uint32_t across, int k, uint32_t blocks, bool four) {
        const auto go = [&](auto kernel) {
            kernel<<<blocks, kThreads, 0, stream>>>(n, cols, skip(q, r), skip(x, r, bf16), k, across, xcd_run(blocks));
        };
        if (bf16) four ? go(unpack_kernel<uint16_t, kLongRows>) : go(unpack_kernel<uint16_t, 1>);
        else four ? go(unpack_kernel<float, kLongRows>) : go(unpack_kernel<float, 1>);
    });
}

hipError_t launch_act_backward(const ActBwd& a, hipStream_t stream) {
    const Tiles t = act_tiles(a.rows, a.cols);
    // runs of rows, as in the forward pass; each run's partial rows follow those before
    const int64_t high = static_cast<int64_t>(kActThreads >> t.k) * kActRows;
    const int64_t run = std::max<int64_t>(1, kMaxBlocks / 2 / t.across) * high;
    const bool nt = outgrows_cache(a.rows, a.cols, a.bf16, 3 + (a.y.p != nullptr), kActBwdNtBytes) &&
                    aligned16(a.dy.p, a.dy.pitch, a.bf16) && aligned16(a.x.p, a.x.pitch, a.bf16);
    for (int64_t r = 0; r < a.rows; r += run) {
        ActBwd b = a;
        b.rows = std::min(run, a.rows - r);
        b.dy = skip(a.dy, r, a.bf16);
        b.x = skip(a.x, r, a.bf16);
        b.ckpt = skip(a.ckpt, r);
        b.dx = skip(a.dx, r, a.bf16);
        b.y = skip(a.y, r, a.bf16);
        if (a.dbias.p) b.workspace = a.workspace + r / high * a.cols;
        Tiles u = t;
        u.down = (b.rows + high - 1) / high;
        if (a.bf16) {
            if (a.ckpt.codes) act_backward_t<uint16_t, true>(b, u, nt, stream);
            else act_backward_t<uint16_t, false>(b, u, nt, stream);
        } else {
            if (a.ckpt.codes) act_backward_t<float, true>(b, u, nt, stream);
            else act_backward_t<float, false>(b, u, nt, stream);
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return launch_col_sum(a.workspace, t.down, a.cols, a.cols, a.dbias, ColOut{nullptr, 0, 0}, stream);
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
        if (a.bf16) norm_forward_t<uint16_t>(b, stream);
        else norm_forward_t<float>(b, stream);
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
