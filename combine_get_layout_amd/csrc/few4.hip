// few4.hip -- ep_moe_few_w4 on gfx950: the expert layer for a few tokens with
// 4-bit weights, in the two launches of ep_moe_few.
//
// For token t and each used expert e, over the values w that codes and scales stand for:
//   gate, up = x[t] . w13[e],  act = gate / (1 + exp(-gate)) * up          (first launch)
//   out[t] = bf16(sum over e of (sum of t's weights for e) * act . w2[e])  (second launch)
// A code becomes bf16 exactly (four bits of magnitude at most), so the matrix
// instructions' products are those of the formula, summed in 32 bits. act goes to the
// second product as two bf16 values, the rounded one and the rest: 16 bits of it.
//
// What has to move is the used experts' weights once, 1.5 F H bytes each and a 32nd (int)
// or 16th (e2m1) of that in scales; products are few (32 tokens, top-8 of 64 experts
// of 7168 x 2048: 22 GFLOP for 1.48 GB). Medians on inputs that the caches do not hold:
//   1 token, top-8 of 64 experts of 7168 x 2048, int   27.3 + 22.0 us, 182 MB: 3.7 TB/s
//     e2m1                                             27.3 + 20.4 us, 187 MB: 3.9 TB/s
//   32 tokens, the same, e2m1                          202 + 131 us, 1.48 GB: 4.4 TB/s
//     int                                              219 + 136 us, 1.43 GB: 4.0 TB/s
//   13 tokens, top-3 of 40, 2080 x 736, e2m1           15.2 + 11.9 us, 58 MB: 2.2 TB/s
//   1 token, top-2 of 16, 256 x 512, int               5.6 + 5.2 us: two launches' latency
// The first launch of 32 tokens reads at 4.9 TB/s, as a copy does; the second is bound by
// latency: a wave waits for one unit of 256 values' fragments behind another, with the
// activations' (as many loads as the weights') between them. One token's launches end
// before the memory has come up to its rate. With many tokens to an expert both launches
// have a form whose workgroups hold the tokens' rows in LDS for four waves of different
// weights: 128 tokens, top-8 of 64 experts of 7168 x 2048, int, 233 + 243 us.
#include <algorithm>

#include "ep_internal.h"
#include "ep_mfma.h"
#include "few_route.h"

namespace ep {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kSpan = 256;  // contracted values per step (first launch) and per unit of work (second)
constexpr int kDownGroups = 512;  // workgroups of the second launch where they share outputs, two per CU

// The offset of a lane that loads nothing: past the end of x and, with kBufFar
// added, still past it.
constexpr uint32_t kBufNone = 0x40000000u;

struct Few4Args {
    int T, H, K, E, F;
    const uint16_t* x;
    const int64_t* topk;
    const float* topk_w;
    const uint8_t* w13;
    const char* s13;
    const uint8_t* w2;
    const char* s2;
    uint16_t* out;
    uint32_t* err;
    int* used;        // number of used experts, then expert | tokens << 16 of each
    Route* routes;    // [used][T], each expert's tokens in ascending order
    uint16_t* act;    // [T*K][2][F], row = first lane of (token, expert): values, rests
    int* joined;      // [H/16, rounded up]: workgroups of the second launch that have stored their part
    float* part;      // [splits][T][H]
    int splits;       // workgroups of the second launch that share values of h
};

__device__ __forceinline__ bf16x8 as_bf16(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

// What sums of products with codes are in units of: of EP_W4_INT, whose scales come after
// the sums of 128 columns, 2^-10, so that 128 products of |code - 8| <= 8 with the largest
// finite values stay finite whatever the scale makes of them.
template <int FORM>
constexpr float kUnit = FORM == EP_W4_INT ? 1024.0f : 1.0f;

// Eight codes (a byte holds two, the first in its low half) to bf16, exactly.
// EP_W4_E2M1: the instruction's own conversion, times a power of two.
// EP_W4_INT: code - 8 as the e4m3 byte of its sign and magnitude m, which stands for
// m * 2^-9 (below 8 as e4m3's denormals, 8 as the first number above them), times 2^-1.
// Signs and magnitudes of all eight at once: where bit 3 is clear (`less`, one in each
// four bits) the magnitude is 8 - code = ((code & 7) ^ 7) + 1, else code & 7. With SPLIT
// the even columns come first, then the odd ones, as the other operand then lies too
// (`split8`): two instructions less of 15. Codes as they are, in nine, and 8 times the
// other operand taken off the products by one more matrix instruction for every four, made
// infinities of finite values and NaN of infinite ones, and took (us, that and this) 50.1
// 50.0 (1 token, top-8 of 64 experts of 7168 x 2048), 351 359 (32 tokens), 495 476 (128).
template <int FORM, bool SPLIT>
__device__ __forceinline__ bf16x8 codes_to_bf16(uint32_t w, float scale) {
    bf16x2 a, b, c, d;
    if constexpr (FORM == EP_W4_E2M1) {
        a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
        b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
        d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
    } else {
        uint32_t sign = ~w & 0x88888888u;
        asm("" : "+v"(sign));  // knowing its bits the compiler makes 17 instructions of 13
        const uint32_t less = sign >> 3, seven = sign - less;
        uint32_t mag = ((w & 0x77777777u) ^ seven) + less;
        asm("" : "+v"(mag));
        const uint32_t even = (mag & 0x0F0F0F0Fu) | ((sign << 4) & 0xF0F0F0F0u);
        const uint32_t odd = ((mag >> 4) & 0x0F0F0F0Fu) | (sign & 0xF0F0F0F0u);
        const uint32_t lo = SPLIT ? even : __builtin_amdgcn_perm(odd, even, 0x05010400u);
        const uint32_t hi = SPLIT ? odd : __builtin_amdgcn_perm(odd, even, 0x07030602u);
        a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 0.5f, false);
        b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 0.5f, true);
        c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 0.5f, false);
        d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 0.5f, true);
    }
    bf16x8 r;
    r[0] = a[0], r[1] = a[1], r[2] = b[0], r[3] = b[1];
    r[4] = c[0], r[5] = c[1], r[6] = d[0], r[7] = d[1];
    return r;
}

// Eight bf16 values of an operand beside codes in SPLIT order; where column c of a row lies
// in that order.
template <int FORM>
__device__ __forceinline__ u32x4 split8(u32x4 v) {
    if constexpr (FORM != EP_W4_INT) return v;
    return u32x4{__builtin_amdgcn_perm(v[1], v[0], 0x05040100u), __builtin_amdgcn_perm(v[3], v[2], 0x05040100u),
                 __builtin_amdgcn_perm(v[1], v[0], 0x07060302u), __builtin_amdgcn_perm(v[3], v[2], 0x07060302u)};
}
template <int FORM>
__device__ __forceinline__ int split_place(int c) {
    return FORM == EP_W4_INT ? (c & ~7) | (c & 1) << 2 | (c & 7) >> 1 : c;
}

// Scales: of a row's blocks of 128 columns a bf16 each, or a byte for 32 of them.
// Loaded as they lie (past the descriptor's end: 0, beside codes of 0), made a
// float where they are used, so that no load is waited for before the others
// have been sent off.
template <int FORM>
struct ScaleRow {
    static constexpr int kShare = FORM == EP_W4_INT ? 128 : 32, kBytes = FORM == EP_W4_INT ? 2 : 1;
    static constexpr int kStep = kSpan / kShare * kBytes;  // bytes of a row's scales for one step
    static __host__ __device__ __forceinline__ uint32_t bytes(int cols) { return (uint32_t)(cols / kShare) * kBytes; }
    // Of a row's columns from 128 * p + 32 * q on, past the scalar offset's.
    static __device__ __forceinline__ uint32_t offset(int p, int q) {
        return FORM == EP_W4_INT ? p * 2u : p * 4u + q;
    }
    static __device__ __forceinline__ uint32_t load(__amdgpu_buffer_rsrc_t d, uint32_t off, uint32_t scalar_off) {
        if constexpr (FORM == EP_W4_INT)
            return __builtin_amdgcn_raw_buffer_load_b16(d, (int)off, (int)scalar_off, 0);
        else
            return __builtin_amdgcn_raw_buffer_load_b8(d, (int)off, (int)scalar_off, 0);
    }
    static __device__ __forceinline__ uint32_t from_lds(const uint8_t* p) {
        if constexpr (FORM == EP_W4_INT) return *reinterpret_cast<const uint16_t*>(p);
        return *p;
    }
    static __device__ __forceinline__ float value(uint32_t v) {
        return __uint_as_float(v << (FORM == EP_W4_INT ? 16 : 23));
    }
};

// Orders this wave's own LDS stores and loads of other lanes' values (LDS takes a
// wave's instructions in order; the compiler must not exchange them).
__device__ __forceinline__ void wave_lds_order() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Rows of 512 bytes (256 bf16 values) in LDS, their 16-byte chunks exchanged so that
// 16 rows read at the same chunk, as a fragment of the matrix instruction does, lie
// in different banks.
__device__ __forceinline__ uint32_t row_chunk(int row, int chunk) { return row * 512 + ((chunk ^ (row & 15)) << 4); }

// silu(gate) * up (__expf: |gate| 2^-24 of it, beside the 2^-16 that two bf16 values keep) as
// two bf16 values for the second product's matrix instruction, the
// rounded one (of a finite value bf16's largest at most) and, F values on, what it
// leaves (nothing of an infinity or NaN).
__device__ __forceinline__ void store_act(uint16_t* act, int F, float gate, float up) {
    const float r = gate / (1.0f + __expf(-gate)) * up;
    uint32_t hi = f32_to_bf16(r);
    if (__builtin_isfinite(r) && (hi & 0x7FFFu) == 0x7F80u) --hi;
    const float rest = __builtin_isfinite(r) ? r - __uint_as_float(hi << 16) : 0.f;
    act[0] = (uint16_t)hi;
    act[F] = (uint16_t)f32_to_bf16(rest);
}

// First launch: workgroup (x, y) computes RT / 2 * 16 values of f for the tokens
// of the y-th used expert, up to TT of them at a time; its waves share the contracted
// axis, a step of 256 columns each. Dynamic LDS: the scales (RT * 16 rows, if LDS),
// then the waves' copies of a step's tokens, kWaves * TT * 512 bytes, where their
// parts of the sums lie at the end.
typedef float Up4Part[4][16][17];

// What a wave loads for one step; the scales unless they lie in LDS.
template <int RT, int XL, bool LDS>
struct UpStage {
    u32x4 w[RT][2];
    uint32_t scale[LDS ? 1 : RT][2];
    u32x4 x[XL];
};

// Bytes of a row's scales at most for them to lie in LDS.
constexpr int kLdsScales = 512;

template <int FORM, int RT, int TT, bool LDS>
__device__ __forceinline__ void up4_tokens(const Few4Args& a, const Found& found, const FindShared& find, uint8_t* scales,
                                           uint8_t* area) {
    using Scale = ScaleRow<FORM>;
    const int tid = threadIdx.x, lane = lane_id(), wave = uniform_wave();
    const int i = lane & 15, q = lane >> 4;
    constexpr int GT = RT / 2, kCols = GT * 16, kLoads = TT / 2;
    using Stage = UpStage<RT, kLoads, LDS>;
    const int f0 = blockIdx.x * kCols, cols = min(kCols, a.F - f0);
    const uint32_t ld = (uint32_t)a.H / 2;
    const uint8_t* w = a.w13 + ((int64_t)found.expert * 2 * a.F + f0) * ld;
    // Gate rows, up rows and the tokens' rows; rows past F read as zeros.
    const auto d_gate = buf_resource(w, cols * ld), d_up = buf_resource(w + (int64_t)a.F * ld, cols * ld);
    const auto d_x = buf_resource(a.x, (uint32_t)a.T * a.H * 2);
    const uint32_t row0 = i * ld + q * 16;
    const uint32_t lds = Scale::bytes(a.H);
    const char* sc = a.s13 + ((int64_t)found.expert * 2 * a.F + f0) * lds;
    const auto s_gate = buf_resource(sc, cols * lds), s_up = buf_resource(sc + (int64_t)a.F * lds, cols * lds);
    const int steps = (a.H + kSpan - 1) / kSpan;

    for (int t0 = 0; t0 < found.tokens; t0 += TT) {
        // A step's values of a token are 512 bytes in a row: half a wave's load. (As the
        // fragments that the matrix instruction takes they would be eight loads of four
        // lanes a token each, which the L1 ran out of: one token 31 us instead of 25.)
        uint32_t xr[kLoads];
#pragma unroll
        for (int n = 0; n < kLoads; ++n) {
            const int at = t0 + 2 * n + (lane >> 5);
            xr[n] = at < found.tokens ? (uint32_t)find.token[at] * a.H * 2 + (lane & 31) * 16 : kBufNone;
        }
        uint8_t* const xs = area + wave * (TT * 512);
        f32x4 acc[RT][1] = {};  // as `settle` takes them
        auto load = [&](int s, Stage& g) {
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                // Columns past H: past the end, zeros.
                const uint32_t far = s * kSpan + p * 128 + q * 32 >= a.H ? kBufFar : 0u;
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    g.w[r][p] = buf_load16(r < GT ? d_gate : d_up, row0 + r % GT * 16 * ld + far, s * 128 + p * 64);
                    if constexpr (!LDS)
                        g.scale[r][p] = Scale::load(r < GT ? s_gate : s_up, (i + r % GT * 16) * lds + Scale::offset(p, q) + far,
                                                    s * Scale::kStep);
                }
            }
            const uint32_t far = s * kSpan + (lane & 31) * 8 >= a.H ? kBufFar : 0u;
#pragma unroll
            for (int n = 0; n < kLoads; ++n) g.x[n] = buf_load16(d_x, xr[n] + far, s * 512);
        };
        auto multiply = [&](const Stage& g, int s) {
#pragma unroll
            for (int n = 0; n < kLoads; ++n) st16(xs + row_chunk(2 * n + (lane >> 5), lane & 31), split8<FORM>(g.x[n]));
            wave_lds_order();
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                bf16x8 xf[4];
#pragma unroll
                for (int m = 0; m < 4; ++m)  // rows past TT: earlier ones again, of which nothing is kept
                    xf[m] = as_bf16(ld16(xs + row_chunk(i & (TT - 1), p * 16 + q * 4 + m)));
                const bool in = s * kSpan + p * 128 + q * 32 < a.H;  // else codes of 0, and no scale
                const uint32_t at = in ? s * Scale::kStep + Scale::offset(p, q) : 0u;
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    uint32_t bits;
                    if constexpr (LDS)
                        bits = in ? Scale::from_lds(scales + (r * 16 + i) * lds + at) : 0u;
                    else
                        bits = g.scale[r][p];
                    const float scale = Scale::value(bits);
                    bf16x8 wf[4];
#pragma unroll
                    for (int m = 0; m < 4; ++m) wf[m] = codes_to_bf16<FORM, true>(g.w[r][p][m], scale);
                    f32x4 c = {};
                    if constexpr (FORM != EP_W4_INT) c = acc[r][0];
#pragma unroll
                    for (int m = 0; m < 4; ++m) c = mfma_bf16(xf[m], wf[m], c);
                    if constexpr (FORM == EP_W4_INT) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[r][0][j] = fmaf(scale, c[j], acc[r][0][j]);
                    } else {
                        acc[r][0] = c;
                    }
                }
            }
            wave_lds_order();
        };
        // The next step's loads are in flight while this one is multiplied; those past
        // the last step find nothing (a branch around them would make the compiler
        // wait for everything).
        Stage g0, g1;
        if (LDS && t0 == 0) {
            // 16 rows' scales lie one after the other, in whole vectors. From memory each
            // step would take a line of 128 bytes for the 4 or 8 that it needs of a row.
            constexpr int kPasses = kCols * kLdsScales / 16 / kThreads;
            u32x4 v[2][kPasses];
#pragma unroll
            for (int n = 0; n < kPasses; ++n) {
                v[0][n] = buf_load16(s_gate, (n * kThreads + tid) * 16, 0);
                v[1][n] = buf_load16(s_up, (n * kThreads + tid) * 16, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
            load(wave, g0);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int n = 0; n < kPasses; ++n) {
                const uint32_t at = (n * kThreads + tid) * 16;
                if (at < kCols * lds) {
                    st16(scales + at, v[0][n]);
                    st16(scales + kCols * lds + at, v[1][n]);
                }
            }
            barrier_only();
        } else {
            load(wave, g0);
        }
        for (int s = wave; s < steps; s += 2 * kWaves) {
            load(s + kWaves, g1);
            __builtin_amdgcn_sched_barrier(0);
            multiply(g0, s);
            __builtin_amdgcn_sched_barrier(0);
            load(s + 2 * kWaves, g0);
            __builtin_amdgcn_sched_barrier(0);
            multiply(g1, s + kWaves);
            __builtin_amdgcn_sched_barrier(0);
        }
        settle(acc);
        // Sum the waves' parts, 32 values of f at a time.
        Up4Part* const part = reinterpret_cast<Up4Part*>(area);
        __syncthreads();
#pragma unroll
        for (int g = 0; g < GT; g += 2) {
            constexpr int kSub = GT < 2 ? 1 : 2;  // sub-tiles of 16 values in this pass
#pragma unroll
            for (int r = 0; r < 2 * kSub; ++r)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    part[wave][r / kSub * 2 + r % kSub][q * 4 + j][i] = acc[r / kSub * GT + g + r % kSub][0][j];
            __syncthreads();
#pragma unroll
            for (int c0 = 0; c0 < 16 * 32; c0 += kThreads) {
                const int tk = (c0 + tid) >> 5, c = tid & 31;
                const int at = t0 + tk, f = f0 + g * 16 + c;
                if (tk >= TT || at >= found.tokens || f >= a.F || c >= 16 * kSub) continue;
                float gate = 0.f, up = 0.f;
#pragma unroll
                for (int v = 0; v < kWaves; ++v) {
                    gate += part[v][c >> 4][tk][c & 15];
                    up += part[v][2 + (c >> 4)][tk][c & 15];
                }
                store_act(a.act + (int64_t)find.row[at] * 2 * a.F + split_place<FORM>(f), a.F, gate * kUnit<FORM>,
                          up * kUnit<FORM>);
            }
            __syncthreads();
        }
    }
}

template <int FORM, int RT, int TT, bool LDS>
__global__ __launch_bounds__(kThreads, 2) void few4_up_kernel(Few4Args a) {
    __shared__ FindShared find;
    extern __shared__ u32x4 lds_vectors[];
    uint8_t* const scales = reinterpret_cast<uint8_t*>(lds_vectors);
    uint8_t* const area = scales + (LDS ? RT * 16 * ScaleRow<FORM>::bytes(a.H) : 0u);
    const int tid = threadIdx.x;
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        if (tid == 0) a.err[0] = 0u;
        if (a.splits > 1)
            for (int n = tid; n * 16 < a.H; n += kThreads) a.joined[n] = 0;
    }
    const Found found = find_expert<kThreads>(a, find);
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) a.used[0] = found.used;
    if (found.expert < 0) return;
    up4_tokens<FORM, RT, TT, LDS>(a, found, find, scales, area);
}

// The same for experts with many tokens: 64 values of f to a workgroup, 16 of them (a
// gate and an up tile) to a wave, which goes over the whole contracted axis for all of
// the expert's tokens; steps of 128 columns, whose tokens' rows lie in LDS for all four
// waves, in two buffers. One barrier a step; the next step's rows and the next two's
// weights are in flight.
constexpr int kManyCols = 64, kManySpan = 128, kManyAhead = 2;

// Rows of 256 bytes in LDS; chunks exchanged as in row_chunk.
__device__ __forceinline__ uint32_t half_chunk(int row, int chunk) { return row * 256 + ((chunk ^ (row & 15)) << 4); }

template <int FORM, int NT>
__device__ __forceinline__ void up4_many_tokens(const Few4Args& a, const Found& found, const FindShared& find,
                                                const uint8_t* scales, uint8_t* rows, int t0) {
    using Scale = ScaleRow<FORM>;
    const int tid = threadIdx.x, lane = lane_id(), wave = uniform_wave();
    const int i = lane & 15, q = lane >> 4;
    const int f0 = blockIdx.x * kManyCols + wave * 16;
    // Into a scalar register: it would be found in a vector one, and each load be a loop.
    const int cols = __builtin_amdgcn_readfirstlane(max(min(16, a.F - f0), 0));
    const uint32_t ld = (uint32_t)a.H / 2, lds = Scale::bytes(a.H);
    const uint8_t* w = a.w13 + ((int64_t)found.expert * 2 * a.F + f0) * ld;
    const auto d_gate = buf_resource(w, cols * ld), d_up = buf_resource(w + (int64_t)a.F * ld, cols * ld);
    const auto d_x = buf_resource(a.x, (uint32_t)a.T * a.H * 2);
    const int steps = (a.H + kManySpan - 1) / kManySpan;
    uint32_t xr[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int at = t0 + n * 16 + (tid >> 4);
        xr[n] = at < found.tokens ? (uint32_t)find.token[at] * a.H * 2 + (tid & 15) * 16 : kBufNone;
    }
    f32x4 acc[2][NT] = {};
    u32x4 xv[NT], wv[kManyAhead][2];
    auto load_x = [&](int s) {
        const uint32_t far = s * kManySpan + (tid & 15) * 8 >= a.H ? kBufFar : 0u;
#pragma unroll
        for (int n = 0; n < NT; ++n) xv[n] = buf_load16(d_x, xr[n] + far, s * 256);
    };
    auto load_w = [&](int s, u32x4 (&v)[2]) {
        const uint32_t off = i * ld + q * 16 + (s * kManySpan + q * 32 >= a.H ? kBufFar : 0u);
        v[0] = buf_load16(d_gate, off, s * 64);
        v[1] = buf_load16(d_up, off, s * 64);
    };
    auto step = [&](int s, uint8_t* buf, u32x4 (&v)[2]) {
#pragma unroll
        for (int n = 0; n < NT; ++n) st16(buf + half_chunk(n * 16 + (tid >> 4), tid & 15), xv[n]);
        barrier_only();
        const bool in = s * kManySpan + q * 32 < a.H;  // else codes of 0, and no scale
        float scale[2];
        bf16x8 wf[2][4];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const uint32_t at = (g * kManyCols + wave * 16 + i) * lds + (in ? s * (Scale::kStep / 2) + Scale::offset(0, q) : 0u);
            uint32_t bits = Scale::from_lds(scales + at);
            asm volatile("" : "+v"(bits));  // read in any case, without a branch
            scale[g] = Scale::value(in ? bits : 0u);
#pragma unroll
            for (int m = 0; m < 4; ++m) wf[g][m] = codes_to_bf16<FORM, false>(v[g][m], scale[g]);
        }
        __builtin_amdgcn_sched_barrier(0);
        load_x(s + 1);
        load_w(s + kManyAhead, v);
        __builtin_amdgcn_sched_barrier(0);
        // One tile's fragments are read while the tile before is multiplied, and no more
        // (all of them at once would not fit the registers).
        bf16x8 tile[2][4];
        auto read = [&](int n) {
#pragma unroll
            for (int m = 0; m < 4; ++m) tile[n & 1][m] = as_bf16(ld16(buf + half_chunk(n * 16 + i, q * 4 + m)));
        };
        read(0);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (n + 1 < NT) read(n + 1);
            __builtin_amdgcn_sched_barrier(0);
            const bf16x8(&xf)[4] = tile[n & 1];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                f32x4 c = {};
                if constexpr (FORM != EP_W4_INT) c = acc[g][n];
#pragma unroll
                for (int m = 0; m < 4; ++m) c = mfma_bf16(xf[m], wf[g][m], c);
                if constexpr (FORM == EP_W4_INT) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[g][n][j] = fmaf(scale[g], c[j], acc[g][n][j]);
                } else {
                    acc[g][n] = c;
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    load_x(0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int k = 0; k < kManyAhead; ++k) load_w(k, wv[k]);
    for (int s = 0; s < steps; s += kManyAhead) {
#pragma unroll
        for (int k = 0; k < kManyAhead; ++k) step(s + k, rows + (k & 1) * NT * 4096, wv[k]);  // past the end: nothing
    }
    settle(acc);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int at = t0 + n * 16 + q * 4 + j;
            if (at < found.tokens && i < cols)
                store_act(a.act + (int64_t)find.row[at] * 2 * a.F + split_place<FORM>(f0 + i), a.F,
                          acc[0][n][j] * kUnit<FORM>, acc[1][n][j] * kUnit<FORM>);
        }
    __syncthreads();  // the buffers, before the next tokens
}

template <int FORM, int NT>
__global__ __launch_bounds__(kThreads, 2) void few4_up_many_kernel(Few4Args a) {
    __shared__ FindShared find;
    extern __shared__ u32x4 lds_vectors[];
    uint8_t* const scales = reinterpret_cast<uint8_t*>(lds_vectors);
    const uint32_t lds = ScaleRow<FORM>::bytes(a.H);
    uint8_t* const rows = scales + 2 * kManyCols * lds;
    const int tid = threadIdx.x;
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        if (tid == 0) a.err[0] = 0u;
        if (a.splits > 1)
            for (int n = tid; n * 16 < a.H; n += kThreads) a.joined[n] = 0;
    }
    const Found found = find_expert<kThreads>(a, find);
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) a.used[0] = found.used;
    if (found.expert < 0) return;
    const int f0 = blockIdx.x * kManyCols, vectors = min(kManyCols, a.F - f0) * lds / 16;
    const char* from = a.s13 + ((int64_t)found.expert * 2 * a.F + f0) * lds;
    for (int v = tid; v < vectors; v += kThreads) {
        st16(scales + v * 16, ld16(from + v * 16));
        st16(scales + kManyCols * lds + v * 16, ld16(from + (int64_t)a.F * lds + v * 16));
    }
    __syncthreads();
    for (int t0 = 0; t0 < found.tokens;) {
        const int left = found.tokens - t0;
        if (NT >= 8 && left > 64)
            up4_many_tokens<FORM, NT >= 8 ? 8 : 1>(a, found, find, scales, rows, t0), t0 += 128;
        else if (NT >= 4 && left > 32)
            up4_many_tokens<FORM, NT >= 4 ? 4 : 1>(a, found, find, scales, rows, t0), t0 += 64;
        else if (NT >= 2 && left > 16)
            up4_many_tokens<FORM, NT >= 2 ? 2 : 1>(a, found, find, scales, rows, t0), t0 += 32;
        else
            up4_many_tokens<FORM, 1>(a, found, find, scales, rows, t0), t0 += 16;
    }
}

__device__ __forceinline__ void look_over_ids(const Few4Args& a) {
    if (blockIdx.x != 0 || blockIdx.y != 0) return;
    bool bad = false;
    for (int n = threadIdx.x; n < a.T * a.K; n += kThreads) bad |= expert_bad(a.topk[n], a.E);
    if (__ballot(bad) && lane_id() == 0) report(a.err, EP_DEVERR_EXPERT_ID);
}

// The end of the second launch: COLS values of h for every token from the workgroup's
// SETS sums in LDS, [SETS][T][COLS + 1], and, where workgroups share outputs, from all
// of theirs by the last one to finish; in a fixed order.
template <int COLS, int SETS>
__device__ __forceinline__ void join(const Few4Args& a, const float* sums) {
    constexpr int kPairs = COLS / 2;  // two columns to a thread
    const int tid = threadIdx.x, h0 = blockIdx.x * COLS, cols = min(COLS, a.H - h0), pairs = a.T * kPairs;
    uint64_t* const part = reinterpret_cast<uint64_t*>(a.part);
    const int64_t set = (int64_t)a.T * a.H / 2;  // one workgroup's part, in pairs
    auto at = [&](int n) { return ((int64_t)(n / kPairs) * a.H + h0) / 2 + n % kPairs; };
    auto put = [&](int n, float v0, float v1) {
        *reinterpret_cast<uint32_t*>(a.out + 2 * at(n)) = pack_bf16(v0, v1);
    };
    __syncthreads();
    for (int n = tid; n < pairs; n += kThreads) {
        const int t = n / kPairs, c = n % kPairs * 2;
        if (c >= cols) continue;
        float v0 = 0.f, v1 = 0.f;
#pragma unroll
        for (int w = 0; w < SETS; ++w) {
            const float* s = sums + (w * a.T + t) * (COLS + 1) + c;
            v0 += s[0], v1 += s[1];
        }
        if (a.splits == 1)
            put(n, v0, v1);
        else
            __hip_atomic_store(part + blockIdx.y * set + at(n), (uint64_t)__float_as_uint(v1) << 32 | __float_as_uint(v0),
                               __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (a.splits == 1) return;
    __shared__ int before;
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this wave's stores are acknowledged
    __syncthreads();
    if (tid == 0)
        before = __hip_atomic_fetch_add(a.joined + blockIdx.x, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (before != a.splits - 1) return;
    // Eight parts of two pairs in flight: with four loads of one value, 128 tokens' sixteen
    // parts took 40 us.
    constexpr int kAtOnce = 8;
    for (int n0 = tid; n0 < pairs; n0 += 2 * kThreads) {
        float v[2][2] = {};
        int64_t from[2];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int n = min(n0 + g * kThreads, pairs - 1), c = n % kPairs * 2;
            from[g] = ((int64_t)(n / kPairs) * a.H + h0 + min(c, cols - 2)) / 2;
        }
        for (int p = 0; p < a.splits; p += kAtOnce) {
            uint64_t w[2][kAtOnce];
#pragma unroll
            for (int g = 0; g < 2; ++g)
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k)
                    w[g][k] = __hip_atomic_load(part + min(p + k, a.splits - 1) * set + from[g], __ATOMIC_RELAXED,
                                                __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
            for (int g = 0; g < 2; ++g)
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) {
                    v[g][0] += p + k < a.splits ? __uint_as_float((uint32_t)w[g][k]) : 0.f;
                    v[g][1] += p + k < a.splits ? __uint_as_float((uint32_t)(w[g][k] >> 32)) : 0.f;
                }
        }
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int n = n0 + g * kThreads;
            if (n < pairs && n % kPairs * 2 < cols) put(n, v[g][0], v[g][1]);
        }
    }
}

// What a wave loads for one unit; the scales as its own run of an expert's, where
// they lie in LDS.
template <int RT, int CAP, bool LDS>
struct DownStage {
    u32x4 w[RT][2];
    uint32_t scale[LDS ? 1 : RT][2];
    u32x4 act[CAP ? CAP : 8];
};

// Bytes of a row's scales at most for a wave to hold those of its rows in LDS.
constexpr int kLdsScales2 = 64;

// Second launch: workgroup x computes RT * 16 values of h for every token, or,
// where `splits` workgroups (grid y) share them, its part. Unit u = (used expert,
// span of 256 values of f); each wave takes a run of units. The matrix
// instruction's 16 rows are 8 tokens of the expert (CAP, where that is not 0), as
// rounded values (rows 0 to 7) and as what those leave (rows 8 to 15). Sums per token
// lie in LDS, one set a wave, and are added at the end in a fixed order.
template <int FORM, int RT, int CAP, bool LDS>
__global__ __launch_bounds__(kThreads, 2) void few4_down_kernel(Few4Args a) {
    using Scale = ScaleRow<FORM>;
    constexpr int kCols = RT * 16, kLd = kCols + 1, kTokens = CAP ? CAP : 8;
    extern __shared__ u32x4 lds_vectors[];
    // [kWaves][rows][bytes of a row's scales], [kWaves][2 * CAP][512] and [kWaves][T][kLd]
    const uint32_t lds = Scale::bytes(a.F), lds_block = LDS ? kCols * lds : 0u;
    uint8_t* const scales = reinterpret_cast<uint8_t*>(lds_vectors) + uniform_wave() * lds_block;
    uint8_t* const rows = reinterpret_cast<uint8_t*>(lds_vectors) + kWaves * lds_block + uniform_wave() * (CAP * 1024);
    float* const sums = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(lds_vectors) + kWaves * (lds_block + CAP * 1024));
    const int tid = threadIdx.x, lane = lane_id(), wave = uniform_wave();
    look_over_ids(a);
    const int i = lane & 15, q = lane >> 4;
    const int h0 = blockIdx.x * kCols, cols = min(kCols, a.H - h0);
    // The number of used experts and the first 63 of them, in one load (the array is
    // padded to 256 bytes).
    int entries = a.used[lane], entries_from = -1;
    const int spans = (a.F + kSpan - 1) / kSpan, used = readlane(entries, 0);
    const int units = used * spans;
    float* mine = sums + wave * a.T * kLd;
    for (int n = lane; n < a.T * kLd; n += kWave) mine[n] = 0.f;

    const uint32_t ld = (uint32_t)a.F / 2;
    const uint32_t w_off = i * ld + q * 16, w_bytes = (uint32_t)cols * ld;
    // A run of neighbouring units to each wave; dealt to a workgroup's waves in turn, which
    // then read 512 bytes of a row together, they took 348 us instead of 338 (32 tokens,
    // top-8 of 64 experts of 7168 x 2048), as each wave has every expert's scales to load.
    const int run = blockIdx.y * kWaves + wave, runs = a.splits * kWaves;
    int u = (int)((int64_t)units * run / runs);
    const int end = (int)((int64_t)units * (run + 1) / runs);
    int rank = u / spans, span = u % spans;

    // 64 experts' entries at a time.
    auto entry_of = [&](int r) {
        if (r < entries_from || r >= entries_from + 64) {
            entries_from = r;
            entries = a.used[1 + min(r + lane, used - 1)];
        }
        return readlane(entries, r - entries_from);
    };
    // As loads are what a wave runs out of, a tile's routes are read by one quarter of
    // it (lane i < 16: token t0 + i of the expert) and handed on between lanes, and
    // lanes without a token load no activations.
    auto load_route = [&](int rank, int tokens, int t0) {
        Route r = {0, 0.f};
        if (q == 0 && t0 + i < tokens) r = a.routes[(int64_t)rank * a.T + t0 + i];
        return r;
    };
    const auto d_act = buf_resource(a.act, (uint32_t)(a.T * a.K) * 4 * a.F);
    auto load_act = [&](const Route& route, int t0, int tokens, int span, auto& v) {
        if constexpr (CAP > 0) {
            // A token's values and their rests are 512 bytes each: a wave's load.
            const uint32_t off = (lane >> 5) * a.F * 2 + (lane & 31) * 16;
            const bool in = span * kSpan + (lane & 31) * 8 < a.F;
#pragma unroll
            for (int n = 0; n < CAP; ++n) {
                const int row = readlane(route.id, (t0 & 15) + n) & 0xFFFF;
                const uint32_t far = in && t0 + n < tokens ? row * 4u * a.F : kBufFar;
                v[n] = buf_load16(d_act, off + far, span * 512);
            }
        } else {
            const bool has = t0 + (i & 7) < tokens;
            const int id = __shfl(route.id, (t0 & 8) + (i & 7));
            const uint32_t off = has ? (uint32_t)((id & 0xFFFF) * 2 + (i >> 3)) * a.F * 2 + q * 64 : kBufFar;
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const uint32_t far = span * kSpan + p * 128 + q * 32 >= a.F ? kBufFar : off;
#pragma unroll
                for (int m = 0; m < 4; ++m) v[p * 4 + m] = buf_load16(d_act, far, span * 512 + p * 256 + m * 16);
            }
        }
    };
    auto load_weights = [&](int64_t e, int span, DownStage<RT, CAP, LDS>& g) {
        const auto d = buf_resource(a.w2 + (e * a.H + h0) * ld, w_bytes);
        const auto ds = buf_resource(a.s2 + (e * a.H + h0) * lds, cols * lds);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const uint32_t far = span * kSpan + p * 128 + q * 32 >= a.F ? kBufFar : 0u;
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                g.w[r][p] = buf_load16(d, w_off + r * 16 * ld + far, span * 128 + p * 64);
                if constexpr (!LDS)
                    g.scale[r][p] = Scale::load(ds, (i + r * 16) * lds + Scale::offset(p, q) + far, span * Scale::kStep);
            }
        }
    };
    // An expert's scales of these rows lie one after the other, in whole vectors.
    u32x4 block[RT];
    auto load_scales = [&](int64_t e, uint32_t far) {
        const auto ds = buf_resource(a.s2 + (e * a.H + h0) * lds, cols * lds);
#pragma unroll
        for (int v = 0; v < RT; ++v) block[v] = buf_load16(ds, (v * 64 + lane) * 16 + far, 0);
    };
    auto keep_scales = [&] {
#pragma unroll
        for (int v = 0; v < RT; ++v)
            if ((v * 64 + lane) * 16 < (int)(kCols * lds)) st16(scales + (v * 64 + lane) * 16, block[v]);
    };

    float acc[RT][4] = {};
    // kTokens tokens of one unit, whose loads are there.
    auto unit = [&](DownStage<RT, CAP, LDS>& g, int span, int t0, int tokens, const Route& route, bool flush) {
        uint32_t bits[RT][2];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const bool in = span * kSpan + p * 128 + q * 32 < a.F;  // else codes of 0, and no scale
            const uint32_t at = in ? span * Scale::kStep + Scale::offset(p, q) : 0u;
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                if constexpr (LDS)
                    bits[r][p] = in ? Scale::from_lds(scales + (r * 16 + i) * lds + at) : 0u;
                else
                    bits[r][p] = g.scale[r][p];
            }
        }
        bf16x8 v[8];
        if constexpr (CAP > 0) {
#pragma unroll
            for (int n = 0; n < CAP; ++n) st16(rows + row_chunk(2 * n + (lane >> 5), lane & 31), g.act[n]);
            wave_lds_order();
#pragma unroll
            for (int m = 0; m < 8; ++m)  // rows past CAP: earlier ones again, of which nothing is kept
                v[m] = as_bf16(ld16(rows + row_chunk((i & (CAP - 1)) * 2 + (i >> 3), (m >> 2) * 16 + q * 4 + (m & 3))));
            wave_lds_order();
        } else {
#pragma unroll
            for (int m = 0; m < 8; ++m) v[m] = as_bf16(g.act[m]);
        }
        f32x4 c[RT][2] = {};
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int p = 0; p < 2; ++p)
#pragma unroll
                for (int m = 0; m < 4; ++m)
                    c[r][p] = mfma_bf16(v[p * 4 + m],
                                        codes_to_bf16<FORM, true>(g.w[r][p][m], Scale::value(bits[r][p])), c[r][p]);
        settle(c);
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[r][j] += FORM == EP_W4_INT ? fmaf(Scale::value(bits[r][1]), c[r][1][j],
                                                      Scale::value(bits[r][0]) * c[r][0][j])
                                               : c[r][0][j] + c[r][1][j];
        if (!flush) return;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = (t0 & 15) + (((q & 1) * 4 + j) & (kTokens - 1));
            const int id = __shfl(route.id, n);
            const float weight = __shfl(route.w, n);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                // Rows 8 to 15: the rests' products. Where the value's is not finite the
                // rest's is no part of the sum.
                const float rest = __shfl_xor(acc[r][j], 32);
                const float dot = __builtin_isfinite(acc[r][j]) ? acc[r][j] + rest : acc[r][j];
                acc[r][j] = 0.f;
                if (q < 2 && q * 4 + j < kTokens && t0 + q * 4 + j < tokens) {
                    float* sum = mine + (id >> 16) * kLd + r * 16 + i;
                    *sum = fmaf(weight, dot * kUnit<FORM>, *sum);
                }
            }
        }
    };
    // The order of the work: the units of the run, the tokens of each in tiles of kTokens;
    // routes are kept for 16 tokens at a time.
    struct Tile {
        int rank, span, t0, entry;
    };
    auto behind = [&](const Tile& x, int step) {
        if (x.t0 + step < x.entry >> 16) return Tile{x.rank, x.span, x.t0 + step, x.entry};
        if (x.span + 1 < spans) return Tile{x.rank, x.span + 1, 0, x.entry};
        const int rank = min(x.rank + 1, used - 1);
        return Tile{rank, 0, 0, entry_of(rank)};
    };
    DownStage<RT, CAP, LDS> g0, g1;
    Tile now = {rank, span, 0, 0};
    Route route = {0, 0.f}, ahead = {0, 0.f};  // of this tile's 16 tokens, and of the 16 behind them
    if (u < end) {
        now.entry = entry_of(rank);
        route = load_route(rank, now.entry >> 16, 0);
        const Tile after = behind(now, 16);
        ahead = load_route(after.rank, after.entry >> 16, after.t0);
        load_weights(now.entry & 0xFFFF, span, g0);
        if constexpr (LDS) {
            load_scales(now.entry & 0xFFFF, 0u);
            keep_scales();
        }
        load_act(route, 0, now.entry >> 16, span, g0.act);
    }
    // The next tile's loads, and the routes of the 16 tokens behind its own, are in flight
    // while this one is multiplied; a unit's weights are asked for again with its next
    // tokens, and then lie near. All loads are made on every turn, behind the last one
    // past the row's end: a branch around them would make the compiler wait for
    // everything.
    auto turn = [&](DownStage<RT, CAP, LDS>& g, DownStage<RT, CAP, LDS>& gn) {
        const int tokens = now.entry >> 16;
        Tile next = behind(now, kTokens);
        const bool new_unit = next.t0 == 0, new_expert = new_unit && now.span + 1 == spans;
        const bool more = !new_unit || u + 1 < end;
        if (!more) next = {now.rank, spans, 0, now.entry};
        Route following = route;
        if (new_unit ? now.t0 >= 16 || new_expert : (next.t0 & 15) == 0) following = ahead;
        load_weights(next.entry & 0xFFFF, next.span, gn);
        if constexpr (LDS) load_scales(next.entry & 0xFFFF, more && new_expert ? 0u : kBufFar);
        load_act(following, next.t0, next.entry >> 16, next.span, gn.act);
        const Tile after = behind({next.rank, next.span, next.t0 & ~15, next.entry}, 16);
        ahead = load_route(after.rank, after.entry >> 16, after.t0);
        __builtin_amdgcn_sched_barrier(0);
        unit(g, now.span, now.t0, tokens, route, tokens > kTokens || !more || new_expert);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (LDS)
            if (more && new_expert) keep_scales();
        u += new_unit, now = next, route = following;
    };
    while (u < end) {
        turn(g0, g1);
        if (u < end) turn(g1, g0);
    }
    join<kCols, kWaves>(a, sums);
}

// The same for experts with many tokens: 64 values of h to a workgroup, 16 of them to a
// wave, for up to NT tiles of 16 tokens at a time, whose rows of act (rounded values, then
// rests) lie in LDS for all four waves, as in few4_up_many_kernel. The work of the
// workgroups that share outputs is cut into steps of 128 columns, over the used experts in
// order. A wave's sums are those of its own columns: one set of [T][65] in LDS.
struct DownManyShared {
    Route routes[EP_FEW_MAX_TOKENS];  // of the expert at hand
};

template <int FORM, int NT>
__device__ __forceinline__ void down4_many_tokens(const Few4Args& a, const DownManyShared& sh, const uint8_t* scales,
                                                  uint8_t* rows, float* sums, int expert, int tokens, int t0, int begin,
                                                  int end) {
    using Scale = ScaleRow<FORM>;
    const int tid = threadIdx.x, lane = lane_id(), wave = uniform_wave();
    const int i = lane & 15, q = lane >> 4;
    const int h0 = blockIdx.x * kManyCols + wave * 16;
    const int cols = __builtin_amdgcn_readfirstlane(max(min(16, a.H - h0), 0));
    const uint32_t ld = (uint32_t)a.F / 2, lds = Scale::bytes(a.F);
    const auto d_w = buf_resource(a.w2 + ((int64_t)expert * a.H + h0) * ld, cols * ld);
    const auto d_act = buf_resource(a.act, (uint32_t)(a.T * a.K) * 4 * a.F);
    uint32_t xr[2 * NT];  // tiles 0 to NT - 1: values, NT and on: rests
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int at = t0 + n * 16 + (tid >> 4);
        const uint32_t row = sh.routes[min(at, EP_FEW_MAX_TOKENS - 1)].id & 0xFFFF;
        xr[n] = at < tokens ? row * 4u * a.F + (tid & 15) * 16 : kBufFar;
        xr[NT + n] = at < tokens ? row * 4u * a.F + 2u * a.F + (tid & 15) * 16 : kBufFar;
    }
    f32x4 acc[1][2 * NT] = {};
    u32x4 xv[2 * NT], wv[kManyAhead];
    auto load_x = [&](int s) {
        const bool in = s < end && s * kManySpan + (tid & 15) * 8 < a.F;
#pragma unroll
        for (int n = 0; n < 2 * NT; ++n) xv[n] = buf_load16(d_act, in ? xr[n] : kBufFar, s * 256);
    };
    auto load_w = [&](int s, u32x4& v) {
        const bool in = s < end && s * kManySpan + q * 32 < a.F;
        v = buf_load16(d_w, in ? i * ld + q * 16 : kBufFar, s * 64);
    };
    auto step = [&](int s, uint8_t* buf, u32x4& v) {
#pragma unroll
        for (int n = 0; n < 2 * NT; ++n) st16(buf + half_chunk(n * 16 + (tid >> 4), tid & 15), xv[n]);
        barrier_only();
        const bool in = s < end && s * kManySpan + q * 32 < a.F;  // else codes of 0, and no scale
        const uint32_t at = (wave * 16 + i) * lds + (in ? s * (Scale::kStep / 2) + Scale::offset(0, q) : 0u);
        uint32_t bits = Scale::from_lds(scales + at);
        asm volatile("" : "+v"(bits));  // read in any case, without a branch
        const float scale = Scale::value(in ? bits : 0u);
        bf16x8 wf[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) wf[m] = codes_to_bf16<FORM, true>(v[m], scale);
        __builtin_amdgcn_sched_barrier(0);
        load_x(s + 1);
        load_w(s + kManyAhead, v);
        __builtin_amdgcn_sched_barrier(0);
        bf16x8 tile[2][4];
        auto read = [&](int n) {
#pragma unroll
            for (int m = 0; m < 4; ++m) tile[n & 1][m] = as_bf16(ld16(buf + half_chunk(n * 16 + i, q * 4 + m)));
        };
        read(0);
#pragma unroll
        for (int n = 0; n < 2 * NT; ++n) {
            if (n + 1 < 2 * NT) read(n + 1);
            __builtin_amdgcn_sched_barrier(0);
            const bf16x8(&xf)[4] = tile[n & 1];
            f32x4 c = {};
            if constexpr (FORM != EP_W4_INT) c = acc[0][n];
#pragma unroll
            for (int m = 0; m < 4; ++m) c = mfma_bf16(xf[m], wf[m], c);
            if constexpr (FORM == EP_W4_INT) {
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[0][n][j] = fmaf(scale, c[j], acc[0][n][j]);
            } else {
                acc[0][n] = c;
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    load_x(begin);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int k = 0; k < kManyAhead; ++k) load_w(begin + k, wv[k]);
    for (int s = begin; s < end; s += kManyAhead) {
#pragma unroll
        for (int k = 0; k < kManyAhead; ++k) step(s + k, rows + (k & 1) * NT * 8192, wv[k]);  // past the end: nothing
    }
    settle(acc);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int at = t0 + n * 16 + q * 4 + j;
            if (at >= tokens) continue;
            // The rests count where the values' product is finite.
            const float v = acc[0][n][j], dot = __builtin_isfinite(v) ? v + acc[0][NT + n][j] : v;
            const Route r = sh.routes[at];
            float* sum = sums + (r.id >> 16) * (kManyCols + 1) + wave * 16 + i;
            *sum = fmaf(r.w, dot * kUnit<FORM>, *sum);
        }
    __syncthreads();  // the buffers, before the next tokens
}

template <int FORM, int NT>
__global__ __launch_bounds__(kThreads, 2) void few4_down_many_kernel(Few4Args a) {
    __shared__ DownManyShared sh;
    extern __shared__ u32x4 lds_vectors[];
    // [64][bytes of a row's scales], two buffers of [2 * NT * 16][256] and [T][65]
    using Scale = ScaleRow<FORM>;
    const uint32_t lds = Scale::bytes(a.F);
    uint8_t* const scales = reinterpret_cast<uint8_t*>(lds_vectors);
    uint8_t* const rows = scales + kManyCols * kLdsScales2;
    float* const sums = reinterpret_cast<float*>(rows + NT * 16384);
    const int tid = threadIdx.x;
    look_over_ids(a);
    for (int n = tid; n < a.T * (kManyCols + 1); n += kThreads) sums[n] = 0.f;
    const int steps = (a.F + kManySpan - 1) / kManySpan, used = a.used[0];
    const int from = (int)((int64_t)used * steps * blockIdx.y / a.splits);
    const int to = (int)((int64_t)used * steps * (blockIdx.y + 1) / a.splits);
    const int h0 = blockIdx.x * kManyCols, vectors = min(kManyCols, a.H - h0) * (int)lds / 16;
    // An expert's scales and routes, in registers while the one before is worked on.
    u32x4 scale = {};
    Route route = {0, 0.f};
    auto load = [&](int rank) {
        if (rank * steps >= to) return;
        const int entry = __builtin_amdgcn_readfirstlane(a.used[1 + rank]);
        if (tid < vectors)
            scale = ld16(reinterpret_cast<const uint8_t*>(a.s2) + ((int64_t)(entry & 0xFFFF) * a.H + h0) * lds + tid * 16);
        if (tid < entry >> 16) route = a.routes[(int64_t)rank * a.T + tid];
    };
    int rank = from / steps;
    load(rank);
    for (int s = from; s < to; s = ++rank * steps) {
        const int entry = __builtin_amdgcn_readfirstlane(a.used[1 + rank]), expert = entry & 0xFFFF, tokens = entry >> 16;
        if (tid < vectors) st16(scales + tid * 16, scale);
        if (tid < tokens) sh.routes[tid] = route;
        __syncthreads();
        load(rank + 1);
        const int begin = s - rank * steps, end = min(to - rank * steps, steps);
        for (int t0 = 0; t0 < tokens;) {
            const int left = tokens - t0;
            if (NT >= 4 && left > 32)
                down4_many_tokens<FORM, NT >= 4 ? 4 : 1>(a, sh, scales, rows, sums, expert, tokens, t0, begin, end), t0 += 64;
            else if (NT >= 2 && left > 16)
                down4_many_tokens<FORM, NT >= 2 ? 2 : 1>(a, sh, scales, rows, sums, expert, tokens, t0, begin, end), t0 += 32;
            else
                down4_many_tokens<FORM, 1>(a, sh, scales, rows, sums, expert, tokens, t0, begin, end), t0 += 16;
        }
    }
    join<kManyCols, 1>(a, sums);
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Units of the second launch, at most (the used experts are known on the GPU alone).
int64_t down_units(const ep_shape& s, int F) {
    return std::min<int64_t>(s.E, (int64_t)s.T * s.K) * ((F + kSpan - 1) / kSpan);
}
// 16-value tiles of h per workgroup of the second launch: 4, which read the activations
// half as often, where each wave has many units (and LDS holds the sums), else 2, which
// keep more waves busy. Both launches with 4 and with 2 tiles, us:
//   32 tokens, top-8 of 64 experts of 7168 x 2048 (int, e2m1; 512 units)  360 372, 337 351
//   16 tokens, top-8 of 64, 7168 x 512 (int, e2m1; 128)      89.3 89.9, 82.7 82.8
//   8 tokens, top-4 of 64, 4096 x 1024 (int; 128)            51.6 49.3
//   13 tokens, top-3 of 40, 2080 x 736 (e2m1; 117)           32.6 30.6
//   1 token, top-8 of 64, 7168 x 2048 (int; 64)              52.9 49.8
int down_tiles(const ep_shape& s, int F) { return s.T <= 32 && down_units(s, F) >= 256 ? 4 : 2; }

// few4_down_many_kernel where an expert has more than four tokens on the average. Both
// launches without and with it, us:
//   128 tokens, top-8 of 64 experts of 7168 x 2048 (int)    676  476
//   128 tokens, top-4 of 32, 4096 x 1536 (e2m1)             154  111
//   128 tokens, top-8 of 64, 2048 x 768 (int)               94.4 82.6
//   64 tokens, top-6 of 13, 384 x 512 (int)                 34.9 28.2
//   48 tokens, top-4 of 32, 4096 x 2048 (int, e2m1)         146 135, 143 138
//   100 tokens, top-8 of 10, 512 x 1024 (e2m1)              46.0 46.5
//   64 tokens, top-2 of 16, 2048 x 1024 (int, e2m1)         37.0 36.6, 34.4 35.4
//   32 tokens, top-8 of 64, 7168 x 2048 (int, e2m1)         360 411, 337 401
//   16 tokens, top-4 of 16, 2048 x 1024 (int)               30.1 30.8
bool down_many(const ep_shape& s, int F, int form) {
    const uint32_t row = form == EP_W4_INT ? ScaleRow<EP_W4_INT>::bytes(F) : ScaleRow<EP_W4_E2M1>::bytes(F);
    return row <= kLdsScales2 && (int64_t)s.T * s.K > 4 * std::min<int64_t>(s.E, (int64_t)s.T * s.K);
}

// Workgroups of the second launch for the same values of h: as many as fill the chip
// (512; with 384, 768 and 1,024 50.0 us became 54.6, 49.2, 51.5 for 1 token, top-8 of 64
// experts of 7168 x 2048, int; 337 369, 347, 334 for 32 tokens, e2m1; 90.0 105, 90.7, 94.0
// for 16 tokens, 7168 x 512, int), with a unit for every wave. Of
// few4_down_many_kernel: eight steps to each, or four while there are fewer than 256.
// us with four always, and with eight (int): 74.6 61.8 (128 tokens, top-4 of 8 experts of 2048
// x 1024), 52.6 47.7 (128, top-2 of 8, 4096 x 512); 45.3 51.2 (128, top-2 of 4, 1024 x 1024),
// 28.1 33.2 (64, top-6 of 13, 384 x 512).
int down_splits(const ep_shape& s, int F, int form) {
    if (down_many(s, F, form)) {
        const int64_t cols = (s.H + kManyCols - 1) / kManyCols;
        const int64_t steps = std::min<int64_t>(s.E, (int64_t)s.T * s.K) * ((F + kManySpan - 1) / kManySpan);
        const int64_t eight = std::min(kDownGroups / cols, steps / 8), four = std::min(kDownGroups / 2 / cols, steps / 4);
        return (int)std::max<int64_t>({1, eight, four});
    }
    const int64_t width = 16 * down_tiles(s, F), cols = (s.H + width - 1) / width;
    return (int)std::max<int64_t>(1, std::min(kDownGroups / std::max<int64_t>(cols, 1), down_units(s, F) / kWaves));
}

typedef void (*Kernel)(Few4Args);
template <int FORM, int RT, int CAP>
Kernel down_kernel(bool lds) {
    return lds ? few4_down_kernel<FORM, RT, CAP, true> : few4_down_kernel<FORM, RT, CAP, false>;
}
// An instance of few4_up_kernel and the tokens (TT) that it takes at a time, by which the
// launch sizes its LDS.
struct UpForm {
    Kernel kernel;
    int tokens;
};
template <int FORM, int RT, int TT, bool LDS>
UpForm up_form() {
    return {few4_up_kernel<FORM, RT, TT, LDS>, TT};
}
// The smallest instance for `tokens` at a time. Few tokens take the wide form too, where
// their lanes repeat experts.
template <int FORM>
UpForm up_form(int tokens, bool narrow, bool lds_scales) {
    if (!lds_scales) return up_form<FORM, 2, 16, false>();
    if (!narrow) return tokens <= 8 ? up_form<FORM, 4, 8, true>() : up_form<FORM, 4, 16, true>();
    return tokens <= 2   ? up_form<FORM, 2, 2, true>()
           : tokens <= 4 ? up_form<FORM, 2, 4, true>()
           : tokens <= 8 ? up_form<FORM, 2, 8, true>()
                         : up_form<FORM, 2, 16, true>();
}

template <int FORM>
void launch(const Few4Args& a, const ep_shape& s, hipStream_t st) {
    const int64_t experts = std::min<int64_t>(s.E, (int64_t)s.T * s.K), lanes = (int64_t)s.T * s.K;
    const uint32_t row = ScaleRow<FORM>::bytes(a.H);
    const bool lds_scales = row <= kLdsScales;
    // Experts of many tokens: few4_up_many_kernel, if there are workgroups for most CUs.
    // Both launches without and with it, us (form; workgroups it has):
    //   128 tokens, top-8 of 64 experts of 7168 x 2048 (int, 2048) 631  475
    //   128 tokens, top-8 of 64, 2048 x 768 (int, 768)             116  82.7
    //   48 tokens, top-8 of 64, 7168 x 2048 (int, 2048)            463  417
    //   48 tokens, top-4 of 32, 4096 x 2048 (int, e2m1, 1024)      141 135, 135 138
    //   100 tokens, top-8 of 10, 512 x 1024 (e2m1, 160)            61.1 46.5
    //   128 tokens, top-1 of 8, 2048 x 2048 (int, 256)             51.1 49.3
    //   64 tokens, top-6 of 13, 384 x 512 (int, 104)               32.9 28.2
    //   128 tokens, top-4 of 8, 2048 x 1024 (e2m1, 128)            57.2 54.4
    //   64 tokens, top-2 of 8, 2048 x 1024 (int, 128)              29.9 32.4
    //   128 tokens, top-4 of 8, 2048 x 512 (int, 64)               47.4 55.7
    //   20 tokens, top-4 of 16, 4096 x 1024 (int, e2m1, 256)       45.5 52.2, 43.1 49.4
    //   32 tokens, top-8 of 64, 7168 x 2048 (int, e2m1, 2048)      360 351, 336 353
    //   32 tokens, top-4 of 32, 4096 x 2048 (int, e2m1, 1024)      128 132, 117 129
    // And of few tokens where rows are short, as a wave of the other form then has a step or
    // two, less than its workgroup's way to them (int, e2m1):
    //   24 tokens, top-8 of 64, 256 x 1024 (1024)                  57.5 36.8, 47.9 35.6
    //   1 token, top-4 of 16, 1024 x 8192 (512)                    31.2 26.4, 27.9 24.6
    //   20 tokens, top-4 of 64, 1024 x 1024 (1024)                 57.4 42.3, 50.0 39.9
    //   2 tokens, top-8 of 64, 2048 x 2048 (512)                   35.3 37.2, 33.1 33.4
    //   8 tokens, top-8 of 64, 2048 x 768 (768)                    43.7 41.6, 39.6 37.6
    //   24 tokens, top-8 of 64, 2048 x 768 (768)                   61.9 52.8, 55.7 49.3
    //   16 tokens, top-4 of 32, 2048 x 2048 (1024)                 67.9 65.9, 61.5 66.4
    //   24 tokens, top-8 of 64, 2816 x 1024 (1024)                 99.7 88.1, 87.8 92.8
    //   24 tokens, top-8 of 64, 4096 x 1024 (1024)                 113  116,  101  118
    const int64_t groups64 = (a.F + kManyCols - 1) / kManyCols * experts;
    const bool many = lds_scales && (lanes > 20 * experts  ? groups64 >= 96
                                     : lanes > 8 * experts ? groups64 >= 160
                                                           : groups64 >= 512 && (lanes > 4 * experts ||
                                                                                 a.H <= (s.T <= 4 ? 1024 : 2048)));
    // 16 or 32 values of f to a workgroup: 32 read the tokens half as often, 16 have more
    // waves to hide a step's latency. us with 16 and with 32 (form):
    //   1 token, top-8 of 64 experts of 7168 x 2048 (e2m1)    48.4 53.6
    //   2 tokens, top-6 of 64, 5120 x 1536 (int)              44.4 56.6
    //   8 tokens, top-4 of 64, 4096 x 1024 (int)              49.5 52.3
    //   16 tokens, top-4 of 16, 2048 x 1024 (int, e2m1)       30.1 28.5, 26.0 26.6
    //   32 tokens, top-8 of 64, 7168 x 2048 (int, e2m1)       359 364, 336 346
    //   20 tokens, top-4 of 16, 4096 x 1024 (e2m1)            46.3 43.1
    //   64 tokens, top-2 of 16, 2048 x 1024 (int, e2m1)       39.6 36.3, 38.2 35.2
    //   32 tokens, top-2 of 8, 1024 x 512 (int)               17.7 19.5
    const bool narrow = !lds_scales || lanes <= 4 * experts || (int64_t)((a.F + 31) / 32) * experts < 512;
    const int cols = many ? kManyCols : narrow ? 16 : 32;
    const dim3 up((a.F + cols - 1) / cols, (unsigned)experts);
    // Tokens at a time: those of most experts, as the weights are read again for more; no
    // more than these, as each is a load a step. us, and with 16 always (int): 49.9 64.5 (1
    // token, top-8 of 64 experts of 7168 x 2048), 35.9 41.5 (4 tokens, top-4 of 64, 4096 x
    // 1024), 360 426 (32 tokens, top-8 of 64, 7168 x 2048; e2m1 337 390).
    const int tt = s.T <= 2 ? 2 : s.T <= 4 ? 4 : s.T <= 8 || lanes <= 4 * experts ? 8 : 16;
    // Tiles of 16 tokens that few4_up_many_kernel multiplies at a time, at most: what fits
    // the registers decides how many waves there are. us with 2, this and 8: 82.6 82.8 107
    // (128 tokens, top-8 of 64, 2048 x 768), 417 417 561 (48 tokens, top-8 of 64, 7168 x
    // 2048), 49.0 46.4 46.4 (100 tokens, top-8 of 10), 63.3 54.4 54.4 (128 tokens, top-4
    // of 8, 2048 x 1024).
    const int tiles1 = s.T <= 32 || lanes <= 20 * experts ? 2 : s.T <= 64 || lanes <= 48 * experts ? 4 : 8;
    const UpForm form = up_form<FORM>(tt, narrow, lds_scales);
    const Kernel first = !many         ? form.kernel
                         : tiles1 == 8 ? few4_up_many_kernel<FORM, 8>
                         : tiles1 == 4 ? few4_up_many_kernel<FORM, 4>
                                       : few4_up_many_kernel<FORM, 2>;
    const size_t area = many ? 8192 * tiles1 : std::max<size_t>(sizeof(Up4Part) * kWaves, kWaves * 512 * form.tokens);
    hipLaunchKernelGGL(first, up, dim3(kThreads), area + (lds_scales ? 2 * cols * row : 0), st, a);
    if (down_many(s, a.F, FORM)) {
        // As tiles1. us with 2, this and 4: 82.4 82.4 101, 417 417 578, 47.9 46.4 46.4 and
        // 57.1 54.4 54.4 in the cases above.
        const int most = s.T <= 32 || lanes <= 20 * experts ? 2 : 4;
        const dim3 grid((s.H + kManyCols - 1) / kManyCols, (unsigned)a.splits);
        const size_t lds = kManyCols * kLdsScales2 + 16384 * most + sizeof(float) * (kManyCols + 1) * s.T;
        hipLaunchKernelGGL((most == 4 ? few4_down_many_kernel<FORM, 4> : few4_down_many_kernel<FORM, 2>), grid,
                           dim3(kThreads), lds, st, a);
        return;
    }
    const int tiles = down_tiles(s, a.F);
    const dim3 down((s.H + 16 * tiles - 1) / (16 * tiles), (unsigned)a.splits);
    const uint32_t row2 = ScaleRow<FORM>::bytes(a.F);
    const bool lds2 = row2 <= kLdsScales2;
    // One or two tokens' activations over LDS, in whole loads instead of fragments: 49.8
    // and 44.3 us instead of 52.0 and 46.1 (1 token, top-8 of 64 experts of 7168 x 2048; 2,
    // top-6 of 64 of 5120 x 1536; int), the same as fragments at 4 tokens, slower at more.
    const int cap = s.T <= 2 ? 2 : 0;
    const size_t lds = kWaves * (sizeof(float) * (16 * tiles + 1) * s.T + cap * 1024 + (lds2 ? 16 * tiles * row2 : 0));
    const Kernel second = tiles == 4 ? down_kernel<FORM, 4, 0>(lds2)
                          : cap == 2 ? down_kernel<FORM, 2, 2>(lds2)
                                     : down_kernel<FORM, 2, 0>(lds2);
    hipLaunchKernelGGL(second, down, dim3(kThreads), lds, st, a);
}

}  // namespace

WsFew ws_few_w4(const ep_shape& s, int F) {
    WsFew w;
    const size_t lanes = (size_t)s.T * s.K, used = std::min<size_t>(s.E, lanes);
    w.used = 256;
    w.routes = w.used + align256(4 * (1 + used));
    w.act = w.routes + align256(sizeof(Route) * used * s.T);
    w.joined = w.act + align256(4 * lanes * F);
    w.part = w.joined + align256(4 * (((size_t)s.H + 15) / 16));
    const size_t splits = std::max(down_splits(s, F, EP_W4_INT), down_splits(s, F, EP_W4_E2M1));
    w.total = w.part + (splits > 1 ? align256(4 * splits * s.T * s.H) : 0);
    return w;
}

hipError_t launch_moe_few_w4(const ep_shape& s, const ep_tokens& tk, const ep_experts_w4& x, uint16_t* out, char* ws,
                             hipStream_t st) {
    uint32_t* err = reinterpret_cast<uint32_t*>(ws);
    if (s.T == 0) {
        hipError_t e = launch_zero_words(err, 1, st);
        return e != hipSuccess ? e : hipGetLastError();
    }
    const WsFew l = ws_few_w4(s, x.F);
    const Few4Args a = {s.T, s.H, s.K, s.E, x.F, tk.x, tk.topk_idx, tk.topk_weights, x.w13,
                        static_cast<const char*>(x.w13_scales), x.w2, static_cast<const char*>(x.w2_scales), out, err,
                        reinterpret_cast<int*>(ws + l.used), reinterpret_cast<Route*>(ws + l.routes),
                        reinterpret_cast<uint16_t*>(ws + l.act), reinterpret_cast<int*>(ws + l.joined),
                        reinterpret_cast<float*>(ws + l.part), down_splits(s, x.F, x.form)};
    if (x.form == EP_W4_INT)
        launch<EP_W4_INT>(a, s, st);
    else
        launch<EP_W4_E2M1>(a, s, st);
    return hipGetLastError();
}

}  // namespace ep
