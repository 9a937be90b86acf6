// norm.hip -- ep_rms_norm and ep_rms_norm_grad on gfx950.
//
// Bound by memory: a row is read once, held in registers over the sum of its squares
// (its dot product in the gradient) and written once, so 4,096 rows of 7,168 move
//   forward (x, residual; h, y, the 8-bit rows)  265 MB in 42.4 us, 6.2 TB/s
//     with a 32-bit stream                       382 MB in 68.6 us, 5.6 TB/s
//   gradient (h, dy, d_stream; d_h, d_gain)      235 MB in 45.1 us, 5.2 TB/s, and 4.9 us
//     to add the workgroups' parts of d_gain (14.7 MB, still in the caches)
//     with a 32-bit stream (and d_x)             470 MB in 90.0 us, 5.2 TB/s, and 4.8 us
// and one row of 7,168 takes 2.4 us, a launch's latency and two dependent loads.
// 201 rows of 2,056 with a 32-bit stream, gradient: 4.8 us in one launch.
// Vectors of eight values, as bf16 loads of 16 bytes; past 32,768 values (in the gradient of
// a 32-bit stream 16,384) a row does not fit the registers and is read twice.
#include <algorithm>
#include <cfloat>

#include "ep_internal.h"
#include "ep_mfma.h"
#include "ep_wave.h"

namespace ep {
namespace {

struct NormArgs {
    int T, H;
    int64_t row0;  // first row of this launch
    float eps;
    const uint16_t* x;
    const char* res;
    const uint16_t* gain;
    char* h;
    uint16_t* y;
    uint8_t* q;
    float* scales;
    float* rstd;
};

// Eight values of a bf16 or fp32 array.
__device__ __forceinline__ void unpack8(u32x4 v, float (&f)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[2 * j] = bf16_lo(v[j]), f[2 * j + 1] = bf16_hi(v[j]);
}
__device__ __forceinline__ u32x4 pack8(const float (&f)[8]) {
    u32x4 v;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = pack_bf16(f[2 * j], f[2 * j + 1]);
    return v;
}
template <bool WIDE>
struct Eight {  // as loaded
    u32x4 v[WIDE ? 2 : 1];
};
template <bool WIDE>
__device__ __forceinline__ Eight<WIDE> load8(const void* base, int64_t at) {
    Eight<WIDE> r;
    if constexpr (WIDE) {
        r.v[0] = ld16(static_cast<const float*>(base) + at);
        r.v[1] = ld16(static_cast<const float*>(base) + at + 4);
    } else {
        r.v[0] = ld16(static_cast<const uint16_t*>(base) + at);
    }
    return r;
}
template <bool WIDE>
__device__ __forceinline__ void floats8(const Eight<WIDE>& r, float (&f)[8]) {
    if constexpr (WIDE) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(r.v[j >> 2][j & 3]);
    } else {
        unpack8(r.v[0], f);
    }
}
template <bool WIDE>
__device__ __forceinline__ void store8(void* base, int64_t at, const float (&f)[8]) {
    if constexpr (WIDE) {
        u32x4 a, b;
#pragma unroll
        for (int j = 0; j < 4; ++j) a[j] = __float_as_uint(f[j]), b[j] = __float_as_uint(f[4 + j]);
        st16(static_cast<float*>(base) + at, a);
        st16(static_cast<float*>(base) + at + 4, b);
    } else {
        st16(static_cast<uint16_t*>(base) + at, pack8(f));
    }
}

// Sum over the LANES consecutive threads that share a row, in each of them.
template <int LANES>
__device__ __forceinline__ float share_sum(float v, float* scratch) {
    static_assert(LANES % kWave == 0, "whole waves");
    v = wave_sum(v);
    if constexpr (LANES == kWave) return v;
    constexpr int kWaves = LANES / kWave;
    const int wave = wave_in_block();
    if (lane_id() == 0) scratch[wave] = v;
    barrier_only();  // loads for later stay in flight
    const float* s = scratch + wave / kWaves * kWaves;
    v = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += s[w];
    return v;
}

// Added to a sum: the squares of a vector's values times `by`.
__device__ __forceinline__ void add_squares(const float (&h)[8], float by, float& sum) {
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(h[j] * by, h[j] * by, sum);
}
// The mean square of a row of H values from this thread's sum of squares. Where the row's
// passes 32 bits it is made again (`again`) of h * 2^-10: as H <= 2^20, that passes them
// only if the mean does.
template <int LANES, class Again>
__device__ __forceinline__ float mean_square(float sum, int H, float (&scratch)[2][LANES < 256 ? 4 : LANES / kWave],
                                             const Again& again) {
    sum = share_sum<LANES>(sum, scratch[0]);
    if (sum <= FLT_MAX) return sum / (float)H;  // the same in all of the row's threads
    return share_sum<LANES>(again(0x1p-10f), scratch[1]) / (float)H * 0x1p20f;
}

// One vector of eight: the normed values to the outputs.
__device__ __forceinline__ void put_normed(const NormArgs& a, int64_t t, int c, const float (&v)[8]) {
    if (a.y) st16(a.y + t * a.H + c, pack8(v));
    if (a.q) {
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));
        m = row_max(m);  // 16 lanes hold 128 channels
        const float s = m < 1e-33f ? 1.0f : m * (1.0f / 448.0f);
        const float inv = __builtin_amdgcn_rcpf(s);  // to 2^-23, beside e4m3's rounding of 2^-4
        u32x2 q;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            q[j] = pack_e4m3(v[4 * j] * inv, v[4 * j + 1] * inv, v[4 * j + 2] * inv, v[4 * j + 3] * inv);
        *reinterpret_cast<u32x2*>(a.q + t * a.H + c) = q;
        if (c % 128 == 0) a.scales[t * (a.H / 128) + c / 128] = s;
    }
}

// LANES threads to a row, NV vectors of eight values to a thread (0: as many as
// it takes, in two passes over the row).
template <int LANES, int NV, bool WIDE>
__global__ __launch_bounds__(LANES < 256 ? 256 : LANES) void norm_kernel(NormArgs a) {
    constexpr int kThreads = LANES < 256 ? 256 : LANES;
    __shared__ float scratch[2][kThreads / kWave];
    const int tid = threadIdx.x % LANES;
    const int64_t row = a.row0 + (int64_t)blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
    if (LANES <= kWave && row >= a.T) return;  // a workgroup with barriers has one row, which exists
    const int64_t base = row * a.H;
    // h of vector c: from memory, stored where it is asked for and the vector is there.
    auto add = [&](int c, bool in, const Eight<false>& xv, const Eight<WIDE>& rv, float(&h)[8]) {
        floats8<false>(xv, h);
        if (a.res) {
            float r[8];
            floats8<WIDE>(rv, r);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[j] += r[j];
            if constexpr (!WIDE) unpack8(pack8(h), h);
        }
        if (in && a.h) store8<WIDE>(a.h, base + c, h);
    };
    if constexpr (NV > 0) {
        float h[NV][8];
        Eight<false> xv[NV];
        Eight<WIDE> rv[NV];
        // Vectors past the row: its last again, and nothing is made of them. (Branches around
        // them made every row wait for its stores of h before its sum: 45.7 us instead of
        // 43.5 for 4,096 rows of 7,168.)
        auto at = [&](int n) { return min((n * LANES + tid) * 8, a.H - 8); };
        auto there = [&](int n) { return (n * LANES + tid) * 8 < a.H; };
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            xv[n] = load8<false>(a.x, base + at(n));
            if (a.res) rv[n] = load8<WIDE>(a.res, base + at(n));
        }
#pragma unroll
        for (int n = 0; n < NV; ++n) add(at(n), there(n), xv[n], rv[n], h[n]);
        auto squares = [&](float by) {
            float sum = 0.f;
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                float part = sum;
                add_squares(h[n], by, part);
                sum = there(n) ? part : sum;
            }
            return sum;
        };
        const float mean = mean_square<LANES>(squares(1.0f), a.H, scratch, squares);
        const float r = 1.0f / sqrtf(mean + a.eps);
        if (a.rstd && tid == 0) a.rstd[row] = r;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int c = (n * LANES + tid) * 8;
            if (c < a.H) {
                float g[8];
                unpack8(ld16(a.gain + c), g);
#pragma unroll
                for (int j = 0; j < 8; ++j) g[j] *= h[n][j] * r;
                put_normed(a, row, c, g);
            }
        }
    } else {
        auto read = [&](int c, bool stored, float(&h)[8]) {
            if (stored) {  // by this thread (residual may be gone)
                floats8<WIDE>(load8<WIDE>(a.h, base + c), h);
            } else {
                Eight<WIDE> rv;
                if (a.res) rv = load8<WIDE>(a.res, base + c);
                add(c, true, load8<false>(a.x, base + c), rv, h);
            }
        };
        auto squares = [&](bool stored, float by) {
            float sum = 0.f;
            for (int c = tid * 8; c < a.H; c += LANES * 8) {
                float h[8];
                read(c, stored, h);
                add_squares(h, by, sum);
            }
            return sum;
        };
        const float mean = mean_square<LANES>(squares(false, 1.0f), a.H, scratch,
                                              [&](float by) { return squares(a.h, by); });
        const float r = 1.0f / sqrtf(mean + a.eps);
        if (a.rstd && tid == 0) a.rstd[row] = r;
        for (int c = tid * 8; c < a.H; c += LANES * 8) {
            float h[8], g[8];
            read(c, a.h, h);
            unpack8(ld16(a.gain + c), g);
#pragma unroll
            for (int j = 0; j < 8; ++j) g[j] *= h[j] * r;
            put_normed(a, row, c, g);
        }
    }
}

struct NormGradArgs {
    int T, H;
    const char* h;
    const uint16_t* gain;
    const float* rstd;
    const uint16_t* dy;
    const char* ds;
    char* dh;
    uint16_t* dx;
    float* part;    // [groups][H]: each workgroup's rows' part of d_gain, or null
    float* d_gain;  // for gain_columns
    int groups;     // workgroups that take rows
};

constexpr int kGradThreads = 512;

// d_gain of 64 columns in one workgroup: a thread takes eight of them and every
// 64th row.
template <int THREADS, bool WIDE>
__device__ __forceinline__ void gain_columns(const NormGradArgs& a, int c0, float* sums) {
    const int c = c0 + (threadIdx.x & 7) * 8, slice = threadIdx.x >> 3;
    float dg[8] = {};
    if (c < a.H) {
#pragma unroll 4
        for (int64_t t = slice; t < a.T; t += THREADS / 8) {
            float dy[8], h[8];
            const float r = a.rstd[t];
            floats8<false>(load8<false>(a.dy, t * a.H + c), dy);
            floats8<WIDE>(load8<WIDE>(a.h, t * a.H + c), h);
#pragma unroll
            for (int j = 0; j < 8; ++j) dg[j] = fmaf(dy[j], h[j] * r, dg[j]);
        }
    }
    // Slices lie next to each other in a wave's rows of 16 lanes: two to a row, then
    // the rows, then the waves.
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        for (int d = 8; d < kWave; d <<= 1) dg[j] += __shfl_xor(dg[j], d);
        if (lane_id() < 8) sums[wave_in_block() * 64 + lane_id() * 8 + j] = dg[j];
    }
    __syncthreads();
    if (threadIdx.x < 64 && c0 + (int)threadIdx.x < a.H) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < THREADS / kWave; ++w) s += sums[w * 64 + threadIdx.x];
        a.d_gain[c0 + threadIdx.x] = s;
    }
}

// With v = h r, whose mean square is 1 at most, d = d_stream + r (a - v mean(a v)): each term
// is a number of 32 bits where d is (r^2 is none for a row of zeros with eps below 2^-128).
// LANES threads to a row, NV vectors of eight values to a thread. A workgroup takes
// every a.groups-th run of rows and keeps its part of d_gain in registers. The next
// rows' loads are in flight while these are summed and stored. Workgroups behind
// those of the rows, where there are any, make d_gain itself.
template <int LANES, int NV, bool WIDE>
__global__ __launch_bounds__(kGradThreads < LANES ? LANES : kGradThreads, 4) void norm_grad_kernel(NormGradArgs a) {
    constexpr int kThreads = kGradThreads < LANES ? LANES : kGradThreads, kRows = kThreads / LANES;
    __shared__ float scratch[2][kThreads / kWave];
    __shared__ float sums[kRows > 1 ? kThreads * 8 : kThreads];
    if ((int)blockIdx.x >= a.groups) {
        gain_columns<kThreads, WIDE>(a, ((int)blockIdx.x - a.groups) * 64, sums);
        return;
    }
    const int tid = threadIdx.x % LANES, sub = threadIdx.x / LANES;
    const float inv_h = 1.0f / (float)a.H;
    float dg[NV][8] = {};
    struct Row {
        Eight<false> dy[NV];
        Eight<WIDE> h[NV], s[NV];
        float r;
    };
    const int runs = (int)(((int64_t)a.T + kRows - 1) / kRows);
    // Rows past the last: the last again, and nothing is made of them.
    auto load = [&](int run, Row& g) {
        const int64_t row = min((int64_t)run * kRows + sub, (int64_t)a.T - 1), base = row * a.H;
        g.r = a.rstd[row];
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int c = min((n * LANES + tid) * 8, a.H - 8);
            g.dy[n] = load8<false>(a.dy, base + c);
            g.h[n] = load8<WIDE>(a.h, base + c);
            if (a.ds) g.s[n] = load8<WIDE>(a.ds, base + c);
        }
    };
    auto row = [&](int run, int turn, const Row& g) {
        const int64_t row = (int64_t)run * kRows + sub, base = row * a.H;
        const bool in = row < a.T;
        float dot = 0.f;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int c = (n * LANES + tid) * 8;
            if (in && c < a.H) {
                float dy[8], h[8], w[8];
                floats8<false>(g.dy[n], dy);
                floats8<WIDE>(g.h[n], h);
                unpack8(ld16(a.gain + c), w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float v = h[j] * g.r;
                    dot = fmaf(dy[j] * w[j], v, dot);
                    dg[n][j] = fmaf(dy[j], v, dg[n][j]);
                }
            }
        }
        if (!a.dh && !a.dx) return;
        // The other half of scratch next time: a wave may still read this one.
        dot = share_sum<LANES>(dot, scratch[turn]);
        const float k = dot * inv_h;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
            const int c = (n * LANES + tid) * 8;
            if (in && c < a.H) {
                float dy[8], h[8], w[8], s[8] = {};
                floats8<false>(g.dy[n], dy);
                floats8<WIDE>(g.h[n], h);
                if (a.ds) floats8<WIDE>(g.s[n], s);
                unpack8(ld16(a.gain + c), w);
#pragma unroll
                for (int j = 0; j < 8; ++j) s[j] = fmaf(g.r, fmaf(-k, h[j] * g.r, dy[j] * w[j]), s[j]);
                if (a.dh) store8<WIDE>(a.dh, base + c, s);
                if (a.dx) st16(a.dx + base + c, pack8(s));
            }
        }
    };
    Row g0, g1;
    if constexpr (NV > 2) {  // the rows of two turns would not fit the registers
        for (int run = blockIdx.x, turn = 0; run < runs; run += a.groups, turn ^= 1) {
            load(run, g0);
            row(run, turn, g0);
        }
    } else {
        load(blockIdx.x, g0);
    }
    for (int run = blockIdx.x; NV <= 2 && run < runs; run += 2 * a.groups) {
        load(run + a.groups, g1);
        __builtin_amdgcn_sched_barrier(0);
        row(run, 0, g0);
        __builtin_amdgcn_sched_barrier(0);
        load(run + 2 * a.groups, g0);
        __builtin_amdgcn_sched_barrier(0);
        row(run + a.groups, 1, g1);
        __builtin_amdgcn_sched_barrier(0);
    }
    if (!a.part) return;
    float* part = a.part + (int64_t)blockIdx.x * a.H;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const int c = (n * LANES + tid) * 8;
        if constexpr (kRows > 1) {  // the workgroup's rows together, in order
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; ++j) sums[j * kThreads + threadIdx.x] = dg[n][j];
            __syncthreads();
            if (sub == 0) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int s = 1; s < kRows; ++s) dg[n][j] += sums[j * kThreads + s * LANES + tid];
            }
        }
        if (sub == 0 && c < a.H) store8<true>(part, c, dg[n]);
    }
}

// Rows too long for registers: one row to a workgroup at a time, in two passes,
// without d_gain.
template <bool WIDE>
__global__ __launch_bounds__(1024) void norm_grad_long_kernel(NormGradArgs a) {
    __shared__ float scratch[16];
    const int64_t row = blockIdx.x, base = row * a.H;
    const float r = a.rstd[row];
    float dot = 0.f;
    for (int c = threadIdx.x * 8; c < a.H; c += 8192) {
        float dy[8], h[8], g[8];
        floats8<false>(load8<false>(a.dy, base + c), dy);
        floats8<WIDE>(load8<WIDE>(a.h, base + c), h);
        unpack8(ld16(a.gain + c), g);
#pragma unroll
        for (int j = 0; j < 8; ++j) dot = fmaf(dy[j] * g[j], h[j] * r, dot);
    }
    dot = share_sum<1024>(dot, scratch);
    const float k = dot / (float)a.H;
    for (int c = threadIdx.x * 8; c < a.H; c += 8192) {
        float dy[8], h[8], g[8], s[8] = {};
        floats8<false>(load8<false>(a.dy, base + c), dy);
        floats8<WIDE>(load8<WIDE>(a.h, base + c), h);
        unpack8(ld16(a.gain + c), g);
        if (a.ds) floats8<WIDE>(load8<WIDE>(a.ds, base + c), s);
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] = fmaf(r, fmaf(-k, h[j] * r, dy[j] * g[j]), s[j]);
        if (a.dh) store8<WIDE>(a.dh, base + c, s);
        if (a.dx) st16(a.dx + base + c, pack8(s));
    }
}

// Their d_gain: a thread takes eight columns and every gridDim.y-th row.
template <bool WIDE>
__global__ __launch_bounds__(256) void norm_gain_long_kernel(NormGradArgs a) {
    const int c = (blockIdx.x * 256 + threadIdx.x) * 8;
    if (c >= a.H) return;
    float dg[8] = {};
    for (int64_t t = blockIdx.y; t < a.T; t += gridDim.y) {
        float dy[8], h[8];
        const float r = a.rstd[t];
        floats8<false>(load8<false>(a.dy, t * a.H + c), dy);
        floats8<WIDE>(load8<WIDE>(a.h, t * a.H + c), h);
#pragma unroll
        for (int j = 0; j < 8; ++j) dg[j] = fmaf(dy[j], h[j] * r, dg[j]);
    }
    store8<true>(a.part + (int64_t)blockIdx.y * a.H, c, dg);
}

// d_gain from the parts: 64 columns to a workgroup, 16 threads of four columns
// by 64 runs of parts.
__global__ __launch_bounds__(1024) void norm_gain_kernel(const float* part, int parts, int H, float* d_gain) {
    __shared__ float4 sums[64][16];
    const int col = threadIdx.x & 15, run = threadIdx.x >> 4, c = blockIdx.x * 64 + col * 4;
    float4 s = {0.f, 0.f, 0.f, 0.f};
    if (c < H) {
        const int end = (run + 1) * parts / 64;
#pragma unroll 8
        for (int p = run * parts / 64; p < end; ++p) {
            const float4 v = *reinterpret_cast<const float4*>(part + (int64_t)p * H + c);
            s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
    }
    sums[run][col] = s;
    __syncthreads();
    if (threadIdx.x < 64 && blockIdx.x * 64 + (int)threadIdx.x < H) {
        const float* f = reinterpret_cast<const float*>(sums) + threadIdx.x;
        float v = 0.f;
#pragma unroll
        for (int n = 0; n < 64; ++n) v += f[n * 64];
        d_gain[blockIdx.x * 64 + threadIdx.x] = v;
    }
}

// Longest row held in registers. Up to it kernels of more than 8,192 values of a 32-bit
// stream and 16,384 of a bf16 one spill (52 and 80 bytes a lane: two vectors and more to
// each of 1,024 threads, at 128 registers); past it rows are read twice, d_gain in a launch of
// its own. us held and read twice: 32-bit stream, 2,048 rows of 16,384 127 148, 1,024 of
// 20,480 136 96.4, of 32,768 (208 bytes spilt) 194 158, 8 of 32,768 23.6 19.0; bf16, 1,024
// rows of 20,480 58.9 55.0, of 32,768 89.8 86.1, 8 of 32,768 11.4 17.2.
constexpr int long_h(bool wide) { return wide ? 16384 : 32768; }

// Threads to a row: with one vector of eight to a thread (a stream in 32 bits, whose
// rows take more registers) or two.
// In bf16 one, and two, us: 4,096 rows of 2,056 23.7 22.4, of 4,096 31.5 32.3, of 7,168
// 50.2 50.5; two for every length, within 3% of the better.
int grad_lanes(int H, bool wide) {
    int lanes = 64;
    while (lanes < 1024 && lanes * 8 * (wide ? 1 : 2) < H) lanes *= 2;
    return lanes;
}
// Workgroups of norm_grad_kernel that take rows: what the chip holds at once, 512 of 512
// threads or 256 of 1,024. us with 256 and 512: bf16, 4,096 rows of 2,056 (512 threads)
// 25.0 22.4, of 7,168 52.7 50.5; 2,048 of 16,384 (1,024 threads) 57.6 68.7; 32-bit
// stream, 4,096 of 7,168 (1,024) 95.4 101.
int grad_groups(int T, int H, bool wide) {
    if (H > long_h(wide)) return std::min(T, 64);
    const int lanes = grad_lanes(H, wide), rows = std::max(1, kGradThreads / lanes);
    return (int)std::min<int64_t>(((int64_t)T + rows - 1) / rows, lanes > kGradThreads ? 256 : 512);
}
// Whether d_gain is made beside the rows in the same launch, by workgroups that
// read dy and h once more, column by column, or from the rows' workgroups' parts in a
// second one. us a call, in one launch and in two:
//   bf16     128 x 512   1024 x 512   2048 x 512   4096 x 512   512 x 2056   1024 x 2056
//   one      11.1        11.2         11.5         20.7         11.3         12.1
//   two      14.1        13.9         14.4         14.1         14.1         14.1
//   bf16     1500 x 2056   128 x 7168   512 x 7168   1024 x 7168  2048 x 7168
//   one      16.3          10.9         11.7         19.9         33.2
//   two      14.0          13.8         17.0         22.2         31.4
//   32-bit   128 x 512   1024 x 512   2048 x 512   4096 x 512   512 x 2056   1024 x 2056
//   one      12.6        12.7         14.0         24.7         13.4         15.2
//   two      15.1        15.1         15.0         15.0         16.2         16.1
//   32-bit   1500 x 2056   128 x 7168   512 x 7168   1024 x 7168  512 x 16384
//   one      21.2          13.1         18.8         30.5         40.4
//   two      17.5          16.0         19.6         28.3         39.8
bool gain_beside(int T, int H, bool wide) {
    const int64_t values = (int64_t)T * H;
    return H <= long_h(wide) && (T <= 1024 ? values <= (wide ? 1 << 22 : 1 << 23) : T <= 2048 && values <= 1 << 20);
}

// Threads to a row: a wave up to 2,048 values (256 threads, with a barrier, are the same
// within 1%), then one vector to a thread, as far as a workgroup goes. us, 4,096 rows of
// 4,096, 5,120 and 7,168 with all outputs: 26.3 31.6 43.4; with 256 threads of two or
// four vectors 27.2 34.8 47.5; with a 32-bit stream of 7,168 69.6, 75.3. 2,048 rows of
// 16,384: 52.3, with 256 threads of eight vectors 61.4.
template <bool WIDE>
void launch_norm(NormArgs a, hipStream_t st) {
    const int vecs = (a.H + 7) / 8;
    auto go = [&](auto kernel, int lanes) {
        const int threads = std::max(lanes, 256), rows = threads / lanes;
        for (a.row0 = 0; a.row0 < a.T; a.row0 += kLaunchGroups * rows) {
            const int64_t groups = std::min((a.T - a.row0 + rows - 1) / rows, kLaunchGroups);
            hipLaunchKernelGGL(kernel, dim3((unsigned)groups), dim3(threads), 0, st, a);
        }
    };
    if (vecs <= 64) return go(norm_kernel<64, 1, WIDE>, 64);
    if (vecs <= 128) return go(norm_kernel<64, 2, WIDE>, 64);
    if (vecs <= 256) return go(norm_kernel<64, 4, WIDE>, 64);
    if (vecs <= 384) return go(norm_kernel<384, 1, WIDE>, 384);
    if (vecs <= 512) return go(norm_kernel<512, 1, WIDE>, 512);
    if (vecs <= 640) return go(norm_kernel<640, 1, WIDE>, 640);
    if (vecs <= 768) return go(norm_kernel<768, 1, WIDE>, 768);
    if (vecs <= 896) return go(norm_kernel<896, 1, WIDE>, 896);
    if (vecs <= 1024) return go(norm_kernel<1024, 1, WIDE>, 1024);
    if (vecs <= 2048) return go(norm_kernel<1024, 2, WIDE>, 1024);
    if (vecs <= 4096) return go(norm_kernel<1024, 4, WIDE>, 1024);
    go(norm_kernel<1024, 0, WIDE>, 1024);
}

template <bool WIDE>
void launch_norm_grad(const NormGradArgs& a, int parts, hipStream_t st) {
    const int vecs = (a.H + 7) / 8;
    if (a.H > long_h(WIDE)) {
        if (a.dh || a.dx) hipLaunchKernelGGL(norm_grad_long_kernel<WIDE>, dim3((unsigned)a.T), dim3(1024), 0, st, a);
        if (a.part)
            hipLaunchKernelGGL(norm_gain_long_kernel<WIDE>, dim3((unsigned)((vecs + 255) / 256), (unsigned)parts),
                               dim3(256), 0, st, a);
        return;
    }
    const int columns = a.d_gain ? (a.H + 63) / 64 : 0;
    auto go = [&](auto kernel, int lanes) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)(a.groups + columns)), dim3(std::max(lanes, kGradThreads)), 0, st, a);
    };
    const int lanes = grad_lanes(a.H, WIDE);
    if (vecs <= 64) return go(norm_grad_kernel<64, 1, WIDE>, lanes);
    if constexpr (WIDE) {
        if (lanes == 128) return go(norm_grad_kernel<128, 1, WIDE>, lanes);
        if (lanes == 256) return go(norm_grad_kernel<256, 1, WIDE>, lanes);
        if (lanes == 512) return go(norm_grad_kernel<512, 1, WIDE>, lanes);
        if (vecs <= 1024) return go(norm_grad_kernel<1024, 1, WIDE>, lanes);
    } else {
        if (lanes == 64) return go(norm_grad_kernel<64, 2, WIDE>, lanes);
        if (lanes == 128) return go(norm_grad_kernel<128, 2, WIDE>, lanes);
        if (lanes == 256) return go(norm_grad_kernel<256, 2, WIDE>, lanes);
        if (lanes == 512) return go(norm_grad_kernel<512, 2, WIDE>, lanes);
    }
    if (WIDE || vecs <= 2048) return go(norm_grad_kernel<1024, 2, WIDE>, lanes);
    if constexpr (!WIDE) go(norm_grad_kernel<1024, 4, WIDE>, lanes);
}

}  // namespace

size_t ws_norm(const ep_shape& s) {
    const int groups = std::max(grad_groups(s.T, s.H, false), grad_groups(s.T, s.H, true));
    return 256 + (sizeof(float) * (size_t)groups * s.H + 255) / 256 * 256;
}

hipError_t launch_rms_norm(const ep_shape& s, const uint16_t* x, const void* res, int stream_type,
                           const uint16_t* gain, float eps, const ep_norm_out& o, hipStream_t st) {
    if (s.T == 0) return hipSuccess;
    const NormArgs a = {s.T, s.H, 0, eps, x, static_cast<const char*>(res), gain, static_cast<char*>(o.h), o.y, o.y_fp8,
                        o.y_scales, o.rstd};
    if (stream_type == EP_STREAM_F32)
        launch_norm<true>(a, st);
    else
        launch_norm<false>(a, st);
    return hipGetLastError();
}

hipError_t launch_rms_norm_grad(const ep_shape& s, const void* h, int stream_type, const uint16_t* gain,
                                const float* rstd, const uint16_t* dy, const void* d_stream, void* d_h, uint16_t* d_x,
                                float* d_gain, char* ws, hipStream_t st) {
    const bool rows = s.T > 0 && (d_h || d_x), wide = stream_type == EP_STREAM_F32,
               beside = d_gain && s.T > 0 && gain_beside(s.T, s.H, wide);
    const int parts = grad_groups(s.T, s.H, wide);
    float* part = reinterpret_cast<float*>(ws + 256);
    const NormGradArgs a = {s.T, s.H, static_cast<const char*>(h), gain, rstd, dy, static_cast<const char*>(d_stream),
                            static_cast<char*>(d_h), d_x, d_gain && !beside ? part : nullptr, beside ? d_gain : nullptr,
                            beside && !rows ? 0 : parts};
    if (s.T > 0) {
        if (wide)
            launch_norm_grad<true>(a, parts, st);
        else
            launch_norm_grad<false>(a, parts, st);
    }
    if (d_gain && !beside)
        hipLaunchKernelGGL(norm_gain_kernel, dim3((unsigned)((s.H + 63) / 64)), dim3(1024), 0, st, part, parts, s.H, d_gain);
    return hipGetLastError();
}

}  // namespace ep
