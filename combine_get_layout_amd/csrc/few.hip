// few.hip -- ep_moe_few on gfx950: the whole expert layer for a few tokens in
// two launches.
//
//   act[t][e] = silu(W13g[e] x[t]) * (W13u[e] x[t])          (first launch)
//   out[t]    = sum over the experts e of t of w[t][e] * W2[e] act[t][e]
//
// Bound: the used experts' weights are read once from HBM; every other array
// is small and stays in L2. One token, top-8 of 64 experts of 7168 x 2048: 89 +
// 50 us for 470 + 235 MB (5.3 and 4.7 TB/s, beside 5.0 of a large copy). 32
// tokens of the same with FP8 weights: 412 + 277 us for 1.94 + 0.97 GB (4.7 and
// 3.5 TB/s): the second launch has one unit's loads at a time in flight per
// wave, and with registers for more (a third of the waves less) it was slower;
// loads past the caches cost 18%, as a line is read in two halves.
// The smallest calls are bound by the launches: 4.4 + 4.3 us on the GPU for one
// token through 2 experts of 256 x 512.
#include <algorithm>

#include "ep_internal.h"
#include "ep_mfma.h"

namespace ep {
namespace {

constexpr int kFewThreads = 512;
constexpr int kFewWaves = kFewThreads / kWave;
constexpr int kDownCols = 16;  // values of h per workgroup of the second launch
constexpr int kDownSpan = 256; // contracted values per unit of work of the second launch
// Workgroups of the second launch where they share outputs, two per CU: 106 tokens,
// top-3 of 63 experts of 1536 x 896 take 87 us both launches together (256: 95);
// 46 tokens, top-6 of 62 experts of 896 x 640 49 (1024: 56).
constexpr int kDownGroups = 512;

// One token of a used expert: token << 16 | row of its inner activations (token
// * K + its first lane with that expert), and the sum of its lanes' weights.
struct Route {
    int id;
    float w;
};

struct FewArgs {
    int T, H, K, E, F;
    const uint16_t* x;
    const int64_t* topk;
    const float* topk_w;
    const char* w13;
    const float* s13;
    const char* w2;
    const float* s2;
    uint16_t* out;
    uint32_t* err;
    int* used;        // number of used experts, then expert | tokens << 16 of each
    Route* routes;    // [used][T], each expert's tokens in ascending order
    uint16_t* act;    // [T*K][2][F], row = first lane of (token, expert): values, rests
    int* joined;      // [H/16, rounded up]: workgroups of the second launch that have stored their part
    float* part;      // [splits][T][H]
    int splits;       // workgroups of the second launch that share 16 values of h
};

__device__ __forceinline__ bf16x8 as_bf16(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

// Eight e4m3 bytes to bf16, exactly.
__device__ __forceinline__ bf16x8 e4m3_to_bf16(uint32_t lo, uint32_t hi) {
    bf16x8 r;
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
    r[0] = a[0], r[1] = a[1], r[2] = b[0], r[3] = b[1];
    r[4] = c[0], r[5] = c[1], r[6] = d[0], r[7] = d[1];
    return r;
}

// The blockIdx.y-th used expert in ascending order (-1 if there are fewer)
// and its tokens in ascending order. Each workgroup finds them for itself:
// the ids are a few KB in L2.
struct Found {
    int expert, used, tokens;
};
__device__ __forceinline__ Found find_expert(const FewArgs& a, uint32_t* bits, short* token, int* scratch) {
    const int tid = threadIdx.x, lane = lane_id(), wave = wave_in_block();
    if (tid < EP_MAX_EXPERTS / 32) bits[tid] = 0u;
    __syncthreads();
    for (int i = tid; i < a.T * a.K; i += kFewThreads) {
        const int64_t e = a.topk[i];
        if (expert_ok(e, a.E)) atomicOr(&bits[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    const uint64_t word = (uint64_t)bits[2 * lane] | (uint64_t)bits[2 * lane + 1] << 32;
    const int n = __popcll(word);
    int sum = n;
    for (int d = 1; d < kWave; d <<= 1) {
        const int v = __shfl_up(sum, d);
        if (lane >= d) sum += v;
    }
    Found f;
    f.used = readlane(sum, kWave - 1);
    f.expert = -1;
    f.tokens = 0;
    const int want = blockIdx.y;
    const uint64_t in = __ballot(want >= sum - n && want < sum);
    if (!in) return f;
    const int src = __ffsll((unsigned long long)in) - 1;
    uint64_t w = (uint64_t)(uint32_t)readlane((int)word, src) | (uint64_t)(uint32_t)readlane((int)(word >> 32), src) << 32;
    for (int skip = want - readlane(sum - n, src); skip > 0; --skip) w &= w - 1;
    f.expert = src * 64 + __ffsll((unsigned long long)w) - 1;

    bool mine = false;
    Route r = {-1, 0.f};
    if (wave < 2) {
        if (tid < a.T) {
            for (int k = 0; k < a.K; ++k) {
                if (a.topk[tid * a.K + k] != f.expert) continue;
                if (r.id < 0) r.id = tid << 16 | (tid * a.K + k);
                r.w += a.topk_w[tid * a.K + k];
            }
        }
        mine = r.id >= 0;
        const uint64_t m = __ballot(mine);
        if (lane == 0) scratch[wave] = __popcll(m);
    }
    __syncthreads();
    f.tokens = scratch[0] + scratch[1];
    if (wave < 2 && mine) {
        const uint64_t m = __ballot(true);
        const int at = (wave ? scratch[0] : 0) + __popcll(m & ((1ull << lane) - 1));
        token[at] = (short)tid;
        scratch[2 + at] = r.id & 0xFFFF;
        if (blockIdx.x == 0) a.routes[(int64_t)want * a.T + at] = r;
    }
    if (blockIdx.x == 0 && tid == 0) a.used[1 + want] = f.expert | f.tokens << 16;
    __syncthreads();
    return f;
}

// First launch: workgroup (x, y) computes 32 values of f for the tokens of the
// y-th used expert: 64 weight rows (32 gate, 32 up) in four 16-row tiles, the
// contracted axis H cut into steps that the 8 waves take in turn. Weights go
// straight from memory into the registers of the matrix instruction (each is
// used once, so LDS would only add a trip); the tokens' values come from L2.
struct UpShared {
    uint32_t bits[EP_MAX_EXPERTS / 32];
    short token[128];
    int scratch[2 + 128];
    float part[kFewWaves][4][16][17];
};

// Tokens [t0, t0 + 16 * NT) of the expert's list, all NT tiles in use.
template <bool FP8, int RT, int NT>
__device__ __forceinline__ void up_tokens(const FewArgs& a, const Found& found, UpShared& sh, int t0) {
    constexpr int kStep = FP8 ? 128 : 64, kX = FP8 ? 4 : 2, kBytes = FP8 ? 1 : 2;
    const int tid = threadIdx.x, lane = lane_id(), wave = wave_in_block();
    const int i = lane & 15, q = lane >> 4;
    constexpr int GT = RT / 2, kCols = GT * 16;
    const int f0 = blockIdx.x * kCols, cols = min(kCols, a.F - f0);
    const uint32_t ld = (uint32_t)a.H * kBytes;
    const char* w = a.w13 + ((int64_t)found.expert * 2 * a.F + f0) * ld;
    // Gate rows, up rows and the tokens' rows; rows past F read as zeros.
    const auto d_gate = buf_resource(w, cols * ld), d_up = buf_resource(w + (int64_t)a.F * ld, cols * ld);
    const auto d_x = buf_resource(a.x, (uint32_t)a.T * a.H * 2);
    const uint32_t row0 = i * ld + q * 16;
    const int blocks = a.H / 128;
    uint32_t sc[RT];  // this lane's weight row's scales, from a.s13 + those of the expert
    const float* scales = FP8 ? a.s13 + (int64_t)found.expert * 2 * a.F * blocks : nullptr;
#pragma unroll
    for (int r = 0; r < RT; ++r) sc[r] = (uint32_t)(r / GT * a.F + min(f0 + r % GT * 16 + i, a.F - 1)) * blocks;
    const int steps = (a.H + kStep - 1) / kStep;
    // The L1 takes a 16-byte load four lanes at a time, whatever these have in
    // common, and that is what this kernel would run out of first: lanes
    // without a token load nothing, and one load of a scale serves four steps.
    uint32_t xr[NT];
    bool has[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        has[n] = t0 + n * 16 + i < found.tokens;
        xr[n] = has[n] ? (uint32_t)sh.token[t0 + n * 16 + i] * a.H * 2 + q * (FP8 ? 32 : 16) : 0u;
    }
    f32x4 acc[RT][NT] = {};
    float four[RT] = {};
    // One step's loads at a time: the other waves' loads (three or more to a
    // SIMD) cover the wait.
    for (int s = wave, it = 0; s < steps; s += kFewWaves, ++it) {
        u32x4 wv[RT][2], xv[NT][kX];
        float sv[RT];
        if (FP8 && it % 4 == 0) {
            // Lane (i, q) takes the scale of the q-th of the next four steps.
            const int mine = min(s + q * kFewWaves, steps - 1);
#pragma unroll
            for (int r = 0; r < RT; ++r) four[r] = scales[sc[r] + mine];
        }
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const uint32_t at = s * 128 + p * 64;  // bytes of a weight row
            // Values past H (the last step of a bf16 row): past the end.
            const uint32_t far = !FP8 && s * kStep + (p * 4 + q) * 8 >= a.H ? kBufFar : 0u;
#pragma unroll
            for (int r = 0; r < RT; ++r)
                wv[r][p] = buf_load16(r < GT ? d_gate : d_up, row0 + r % GT * 16 * ld + far, at);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int h = 0; h < kX / 2; ++h) {
                    u32x4 v = {0u, 0u, 0u, 0u};
                    if (has[n]) v = buf_load16(d_x, xr[n] + far, at * (FP8 ? 2 : 1) + h * 16);
                    xv[n][p * (kX / 2) + h] = v;
                }
        }
        if constexpr (FP8) {
#pragma unroll
            for (int r = 0; r < RT; ++r) sv[r] = __shfl(four[r], i + it % 4 * 16);
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            bf16x8 wf[kX];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                if constexpr (FP8) {
                    wf[2 * p] = e4m3_to_bf16(wv[r][p][0], wv[r][p][1]);
                    wf[2 * p + 1] = e4m3_to_bf16(wv[r][p][2], wv[r][p][3]);
                } else {
                    wf[p] = as_bf16(wv[r][p]);
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                f32x4 c = {};
                if constexpr (!FP8) c = acc[r][n];
#pragma unroll
                for (int p = 0; p < kX; ++p) c = mfma_bf16(as_bf16(xv[n][p]), wf[p], c);
                if constexpr (FP8) {
                    // The block's scale on the 32-bit sum: the products of
                    // e4m3 values themselves are not rounded.
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[r][n][j] = fmaf(sv[r], c[j], acc[r][n][j]);
                } else {
                    acc[r][n] = c;
                }
            }
        }
    }
    settle(acc);
    // Sum the waves' parts, 32 values of f at a time: thread -> (token of 16, f of 32).
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int g = 0; g < GT; g += 2) {
            constexpr int kSub = GT < 2 ? 1 : 2;  // sub-tiles of 16 values in this pass
#pragma unroll
            for (int r = 0; r < 2 * kSub; ++r)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sh.part[wave][r / kSub * 2 + r % kSub][q * 4 + j][i] = acc[r / kSub * GT + g + r % kSub][n][j];
            __syncthreads();
            const int tk = tid >> 5, c = tid & 31;
            const int at = t0 + n * 16 + tk, f = f0 + g * 16 + c;
            if (at < found.tokens && f < a.F && c < 16 * kSub) {
                float gate = 0.f, up = 0.f;
#pragma unroll
                for (int v = 0; v < kFewWaves; ++v) {
                    gate += sh.part[v][c >> 4][tk][c & 15];
                    up += sh.part[v][2 + (c >> 4)][tk][c & 15];
                }
                const float r = gate / (1.0f + __expf(-gate)) * up;
                // Two bf16 values for the second product's matrix instruction, the
                // rounded one (of a finite value bf16's largest at most) and what it
                // leaves (nothing of an infinity or NaN).
                uint32_t hi = f32_to_bf16(r);
                if (__builtin_isfinite(r) && (hi & 0x7FFFu) == 0x7F80u) --hi;
                const float rest = __builtin_isfinite(r) ? r - __uint_as_float(hi << 16) : 0.f;
                uint16_t* act = a.act + (int64_t)sh.scratch[2 + at] * 2 * a.F + f;
                act[0] = (uint16_t)hi;
                act[a.F] = (uint16_t)f32_to_bf16(rest);
            }
            __syncthreads();
        }
    }
}

template <bool FP8, int RT, int NT>
__global__ __launch_bounds__(kFewThreads, NT == 1 ? 4 : 2) void few_up_kernel(FewArgs a) {
    __shared__ UpShared sh;
    const int tid = threadIdx.x;
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        if (tid == 0) a.err[0] = 0u;
        if (a.splits > 1)
            for (int n = tid; n * kDownCols < a.H; n += kFewThreads) a.joined[n] = 0;
    }
    const Found found = find_expert(a, sh.bits, sh.token, sh.scratch);
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) a.used[0] = found.used;
    if (found.expert < 0) return;
    for (int t0 = 0; t0 < found.tokens; t0 += 16 * NT) {
        if (NT > 1 && found.tokens - t0 > 16)
            up_tokens<FP8, RT, NT>(a, found, sh, t0);
        else
            up_tokens<FP8, RT, 1>(a, found, sh, t0);
    }
}

// Second launch: workgroup x computes 16 values of h for every token. Unit u =
// (used expert, span of 256 values of f); each of the 8 waves takes a run of
// them. A unit's 16 weight rows and its expert's tokens' activations are loaded at once
// (the routes, which say where the latter are, a unit ahead) and multiplied. The
// spans of an expert add up in registers while it has one tile of tokens, and
// are then added, weighted, to the wave's sums of those tokens in LDS (a run of
// units rather than every 8th, each added there at once, took 2 to 6% off both
// launches together): an expert's infinities or NaN stay with its own tokens, and the matrix
// instruction's 16 rows are 8 tokens of the expert, however many others there
// are, as rounded values (rows 0 to 7) and as what those leave (rows 8 to 15).
// Rounded values alone, 16 tokens at a time, were 1 to 2% faster up to 64 tokens
// (10% at 128) and left 2.4e-3 of the output's norm as error instead of 1.7e-3,
// the output's own rounding. The waves' sums are added at the end in a fixed
// order.
//
// Where H / 16 workgroups leave CUs idle, `splits` of them (grid y) share the
// units; each stores its part of the sums, and the one that comes last adds the
// parts, in a fixed order. Stores and loads of parts are device-scope (the XCDs'
// L2s do not see each other's), acknowledged before the count goes up.
// 103 tokens, top-8 of 10 experts of 512 x 1024 (FP8): 128 -> 56 us; 13 tokens, 31
// experts of 448 x 1304: 63 -> 35; 102 tokens, 22 experts of 2752 x 184, whose two
// workgroups have 11 units each: 39 -> 43.
template <bool FP8>
__global__ __launch_bounds__(kFewThreads, 4) void few_down_kernel(FewArgs a) {
    constexpr int kLoads = FP8 ? 4 : 8, kBytes = FP8 ? 1 : 2;
    extern __shared__ float sums[];  // [kFewWaves][T][17]
    const int tid = threadIdx.x, lane = lane_id(), wave = uniform_wave();
    if (blockIdx.x == 0 && blockIdx.y == 0) {
        bool bad = false;
        for (int n = tid; n < a.T * a.K; n += kFewThreads) bad |= expert_bad(a.topk[n], a.E);
        if (__ballot(bad) && lane == 0) report(a.err, EP_DEVERR_EXPERT_ID);
    }
    const int i = lane & 15, q = lane >> 4;
    const int h0 = blockIdx.x * kDownCols, cols = min(kDownCols, a.H - h0);
    const int hr = min(h0 + i, a.H - 1);
    const int spans = (a.F + kDownSpan - 1) / kDownSpan;
    const int units = a.used[0] * spans;
    float* mine = sums + wave * a.T * 17;
    for (int n = lane; n < a.T * 17; n += kWave) mine[n] = 0.f;

    // As in the first launch, loads are spared: a tile's routes are read by one
    // quarter of the wave (lane i < 16: token t0 + i of the expert) and handed
    // on between lanes, and lanes without a token load no activations.
    auto load_route = [&](int rank, int tokens, int t0) {
        Route r = {0, 0.f};
        if (q == 0 && t0 + i < tokens) r = a.routes[(int64_t)rank * a.T + t0 + i];
        return r;
    };
    const uint32_t ld = (uint32_t)a.F * kBytes;
    const uint32_t w_off = i * ld + q * 16, w_bytes = (uint32_t)cols * ld;
    auto load_act = [&](int id, bool has, int span, u32x4 (&v)[8]) {
        const uint16_t* p = a.act + ((int64_t)(id & 0xFFFF) * 2 + (i >> 3)) * a.F + span * kDownSpan;
        const bool full = (span + 1) * kDownSpan <= a.F;
#pragma unroll
        for (int m = 0; m < 8; ++m) v[m] = u32x4{0u, 0u, 0u, 0u};
        if (has && full) {
#pragma unroll
            for (int m = 0; m < 8; ++m) v[m] = ld16(p + (FP8 ? ((m >> 1) * 4 + q) * 16 + (m & 1) * 8 : (m * 4 + q) * 8));
        } else if (has) {
#pragma unroll
            for (int m = 0; m < 8; ++m) {
                const int k = FP8 ? ((m >> 1) * 4 + q) * 16 + (m & 1) * 8 : (m * 4 + q) * 8;
                if (span * kDownSpan + k < a.F) v[m] = ld16(p + k);
            }
        }
    };
    const int run = blockIdx.y * kFewWaves + wave, runs = a.splits * kFewWaves;
    int u = (int)((int64_t)units * run / runs), entry = 0;
    const int end = (int)((int64_t)units * (run + 1) / runs);
    Route route = {0, 0.f};
    float acc[4] = {};
    if (u < end) {
        entry = __builtin_amdgcn_readfirstlane(a.used[1 + u / spans]);
        route = load_route(u / spans, entry >> 16, 0);
    }
    while (u < end) {
        const int rank = u / spans, span = u % spans, tokens = entry >> 16;
        const int64_t e = entry & 0xFFFF;
        u32x4 w[kLoads], v[8];
        float s0 = 0.f, s1 = 0.f;
        const auto d = buf_resource(a.w2 + (e * a.H + h0) * ld, w_bytes);
        const bool full = (span + 1) * kDownSpan <= a.F;
#pragma unroll
        for (int n = 0; n < kLoads; ++n) {
            const uint32_t far = !full && span * kDownSpan + (n * 4 + q) * (16 / kBytes) >= a.F ? kBufFar : 0u;
            w[n] = buf_load16(d, w_off + far, span * kDownSpan * kBytes + n * 64);
        }
        if constexpr (FP8) {  // lanes q = 0, 1: the span's two blocks
            float sv = 0.f;
            if (q < 2 && span * 2 + q < a.F / 128) sv = a.s2[(e * a.H + hr) * (a.F / 128) + span * 2 + q];
            s0 = __shfl(sv, i);
            s1 = __shfl(sv, i + 16);
        }
        load_act(__shfl(route.id, i & 7), (i & 7) < tokens, span, v);
        const int next = u + 1;
        int next_entry = entry;
        Route next_route = route;
        const bool last = next == end || span + 1 == spans;  // of the expert's spans here
        if (last && next < end) {
            next_entry = __builtin_amdgcn_readfirstlane(a.used[1 + next / spans]);
            next_route = load_route(next / spans, next_entry >> 16, 0);
        }
        for (int t0 = 0; t0 < tokens; t0 += 8) {
            f32x4 c[1][2] = {};
#pragma unroll
            for (int m = 0; m < 8; ++m) {
                bf16x8 wf;
                if constexpr (FP8)
                    wf = e4m3_to_bf16(w[m >> 1][(m & 1) * 2], w[m >> 1][(m & 1) * 2 + 1]);
                else
                    wf = as_bf16(w[m]);
                // FP8: the first four fragments are the span's first block of 128.
                f32x4& d = c[0][FP8 ? m >> 2 : 0];
                d = mfma_bf16(as_bf16(v[m]), wf, d);
            }
            settle(c);
            const Route now = route;
            if (t0 + 8 < tokens) {  // more than 8 tokens: the weights stay, the tokens change
                if (t0 & 8) route = load_route(rank, tokens, t0 + 8);
                const int n = (~t0 & 8) + (i & 7);
                load_act(__shfl(route.id, n), t0 + 8 + (i & 7) < tokens, span, v);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j] += FP8 ? fmaf(s1, c[0][1][j], s0 * c[0][0][j]) : c[0][0][j];
            if (tokens <= 8 && !last) break;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = (t0 & 8) + (q & 1) * 4 + j;
                const int id = __shfl(now.id, n);
                const float weight = __shfl(now.w, n);
                // Rows 8 to 15: the rests' products. Where the value's is not finite (an
                // infinite weight) the rest's, of either sign or 0 * infinity, is no part
                // of the sum.
                const float rest = __shfl_xor(acc[j], 32);
                const float dot = __builtin_isfinite(acc[j]) ? acc[j] + rest : acc[j];
                acc[j] = 0.f;
                if (q < 2 && t0 + q * 4 + j < tokens) {
                    float* sum = mine + (id >> 16) * 17 + i;
                    *sum = fmaf(weight, dot, *sum);
                }
            }
        }
        u = next, entry = next_entry, route = next_route;
    }
    __syncthreads();
    for (int n = tid; n < a.T * 16; n += kFewThreads) {
        const int t = n >> 4, h = h0 + (n & 15);
        if ((n & 15) >= cols) continue;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kFewWaves; ++w) v += sums[(w * a.T + t) * 17 + (n & 15)];
        if (a.splits == 1)
            a.out[(int64_t)t * a.H + h] = (uint16_t)f32_to_bf16(v);
        else
            __hip_atomic_store(a.part + ((int64_t)blockIdx.y * a.T + t) * a.H + h, v, __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
    }
    if (a.splits == 1) return;
    __shared__ int before;
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this wave's stores are acknowledged
    __syncthreads();
    if (tid == 0)
        before = __hip_atomic_fetch_add(a.joined + blockIdx.x, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (before != a.splits - 1) return;
    for (int n = tid; n < a.T * 16; n += kFewThreads) {
        const int t = n >> 4, h = h0 + (n & 15);
        if ((n & 15) >= cols) continue;
        float v = 0.f;
#pragma unroll 4
        for (int p = 0; p < a.splits; ++p)
            v += __hip_atomic_load(a.part + ((int64_t)p * a.T + t) * a.H + h, __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
        a.out[(int64_t)t * a.H + h] = (uint16_t)f32_to_bf16(v);
    }
}

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Workgroups of the second launch for each 16 values of h: as many as fill the
// chip, with a unit for every wave.
int down_splits(const ep_shape& s, int F) {
    const int64_t units = std::min<int64_t>(s.E, (int64_t)s.T * s.K) * ((F + kDownSpan - 1) / kDownSpan);
    const int64_t cols = (s.H + kDownCols - 1) / kDownCols;
    return (int)std::max<int64_t>(1, std::min(kDownGroups / std::max<int64_t>(cols, 1), units / kFewWaves));
}

}  // namespace

WsFew ws_few(const ep_shape& s, int F) {
    WsFew w;
    const size_t lanes = (size_t)s.T * s.K, used = std::min<size_t>(s.E, lanes);
    w.used = 256;
    w.routes = w.used + align256(4 * (1 + used));
    w.act = w.routes + align256(sizeof(Route) * used * s.T);
    w.joined = w.act + align256(4 * lanes * F);
    w.part = w.joined + align256(4 * (((size_t)s.H + kDownCols - 1) / kDownCols));
    const size_t splits = down_splits(s, F);
    w.total = w.part + (splits > 1 ? align256(4 * splits * s.T * s.H) : 0);
    return w;
}

hipError_t launch_moe_few(const ep_shape& s, const ep_tokens& tk, const ep_experts& x, uint16_t* out, char* ws,
                          hipStream_t st) {
    uint32_t* err = reinterpret_cast<uint32_t*>(ws);
    if (s.T == 0) {
        hipError_t e = launch_zero_words(err, 1, st);
        return e != hipSuccess ? e : hipGetLastError();
    }
    const WsFew l = ws_few(s, x.F);
    const bool fp8 = x.w13_fp8 != nullptr;
    const FewArgs a = {s.T, s.H, s.K, s.E, x.F, tk.x, tk.topk_idx, tk.topk_weights,
                       fp8 ? (const char*)x.w13_fp8 : (const char*)x.w13, x.w13_scales,
                       fp8 ? (const char*)x.w2_fp8 : (const char*)x.w2, x.w2_scales, out, err,
                       reinterpret_cast<int*>(ws + l.used), reinterpret_cast<Route*>(ws + l.routes),
                       reinterpret_cast<uint16_t*>(ws + l.act), reinterpret_cast<int*>(ws + l.joined),
                       reinterpret_cast<float*>(ws + l.part), down_splits(s, x.F)};
    const int64_t experts = std::min<int64_t>(s.E, (int64_t)s.T * s.K);
    // Values of f per workgroup of the first launch (x 2 = weight rows), by the
    // tokens that an expert has on the average. 64, and two token tiles at a time,
    // where these are more than 16, or where there are 1,024 workgroups and they
    // are more than 4, with FP8 weights (half the bytes beside the same tokens'
    // rows and twice the arithmetic) more than 8: the tokens' rows, which then
    // weigh, are read half as often. Top-8 of 64 experts, 64 against 32 values and
    // one tile, both launches, at 3, 4, 4.5, 6, 8, 12 and 16 tokens an expert:
    //   4096 x 1536        470 483 498 515 541 596 652, 442 486 531 540 574 648 779
    //   7168 x 2048        1041 1080 1101 1152 1228 1351 1490,
    //                      1049 1094 1119 1175 1254 1492 1824
    //   FP8, 7168 x 2048   672 697 716 769 832 965 1101, 650 678 701 763 847 1004 1252
    //   FP8, 2048 x 1024   114 121 123 132 143 166 179, 106 113 115 125 137 168 196
    // With fewer workgroups (top-3 of 63 experts of 1536 x 896) at 1.7, 4.6 and 6.1
    // tokens 96 140 144, 90 126 129. Else 32, or 16 where that gives fewer than 1,024
    // workgroups, which leave the memory idle (one token, top-8 of 4096 x 1536: 66
    // us with 16, 75 with 32; 13 tokens, 33 experts of 2056 x 712: 63.5 and 70).
    const int64_t lanes = (int64_t)s.T * s.K, wide = (x.F + 63) / 64 * experts;
    const bool many = s.T > 16 && (lanes > 16 * experts || (wide >= 1024 && lanes > (fp8 ? 8 : 4) * experts));
    const bool narrow = (int64_t)((x.F + 31) / 32) * experts < 1024;
    const int cols = many ? 64 : narrow ? 16 : 32;
    const dim3 up((x.F + cols - 1) / cols, (unsigned)experts);
    const dim3 down((s.H + kDownCols - 1) / kDownCols, (unsigned)a.splits);
    void (*const ups[2][3])(FewArgs) = {{few_up_kernel<false, 4, 1>, few_up_kernel<false, 8, 2>, few_up_kernel<false, 2, 1>},
                                        {few_up_kernel<true, 4, 1>, few_up_kernel<true, 8, 2>, few_up_kernel<true, 2, 1>}};
    hipLaunchKernelGGL(ups[fp8][many ? 1 : narrow ? 2 : 0], up, dim3(kFewThreads), 0, st, a);
    const size_t lds = sizeof(float) * kFewWaves * 17 * s.T;  // 69,632 bytes at most
    hipLaunchKernelGGL(fp8 ? few_down_kernel<true> : few_down_kernel<false>, down, dim3(kFewThreads), lds, st, a);
    return hipGetLastError();
}

}  // namespace ep
