// route.hip -- ep_route and ep_route_grad on gfx950.
#include <algorithm>

#include "ep_internal.h"
#include "ep_mfma.h"
#include "ep_wave.h"

namespace ep {
namespace {

constexpr float kNone = -__builtin_inff();
constexpr float kTiny = 1e-20f;  // beside the sum of the chosen scores

struct RouteArgs {
    int T, E, K;
    int groups, lanes, top_groups, group_top;  // groups that limit the choice (1: none), lanes that share one
    bool sigmoid, normalize;
    float scale;
    const float* logits;
    const float* bias;
    int64_t* topk;
    float* topk_w;
    uint32_t* err;
};

// exp(l - top) for a token's largest logit `top`: 1 where both are the same
// infinity, 0 for a masked expert.
__device__ __forceinline__ float relative_exp(float l, float top) { return l == kNone ? 0.f : l == top ? 1.f : __expf(l - top); }

// One wave per token. A group's experts lie in `lanes` neighbouring lanes, PER
// to a lane in ascending order, so that ties go to the lowest lane.
template <int PER, bool WIDE>
__global__ __launch_bounds__(kBlockThreads) void route_kernel(RouteArgs a) {
    using Key = std::conditional_t<WIDE, double, float>;
    const Key none = kNone;
    const int lane = lane_id();
    const int64_t t = (int64_t)blockIdx.x * kWavesPerBlock + wave_in_block();
    if (t >= a.T) return;
    const int size = a.E / a.groups, group = lane / a.lanes, at = lane % a.lanes * PER;
    const int first = group * size + at;  // this lane's first expert
    const int held = group < a.groups ? min(max(size - at, 0), PER) : 0;
    const float* l = a.logits + t * a.E;
    float v[PER];
    bool bad = false;
    float top = kNone;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        v[j] = j < held ? l[first + j] : kNone;
        if (v[j] != v[j]) bad = true, v[j] = kNone;
        top = fmaxf(top, v[j]);
    }
    float total = 1.f;
    if (!a.sigmoid) {
        top = wave_max(top);
        total = 0.f;
#pragma unroll
        for (int j = 0; j < PER; ++j) total += relative_exp(v[j], top);
        total = wave_sum(total);
    }
    Key key[PER];
    if constexpr (WIDE) {
        double sum = 1.0;
        if (a.sigmoid) {
#pragma unroll
            for (int j = 0; j < PER; ++j) key[j] = 1.0 / (1.0 + exp(-(double)v[j]));
        } else {
            sum = 0.0;
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                key[j] = v[j] == top ? 1.0 : exp((double)v[j] - (double)top);
                if (v[j] == kNone) key[j] = 0.0;
                sum += key[j];
            }
            sum = wave_sum(sum);
        }
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            if (!a.sigmoid) key[j] = key[j] / sum;
            if (a.bias && j < held) {
                const float b = a.bias[first + j];
                if (b != b) bad = true;
                key[j] += (double)b;
            }
            if (v[j] == kNone || !(key[j] > none)) key[j] = none;
        }
    } else {
#pragma unroll
        for (int j = 0; j < PER; ++j) key[j] = v[j];
    }
    if (__ballot(bad) && lane == 0) report(a.err, EP_DEVERR_LOGIT);

    if (a.groups > 1) {
        Key m1 = none, m2 = none;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            m2 = larger(m2, key[j] < m1 ? key[j] : m1);
            m1 = larger(m1, key[j]);
        }
        for (int d = 1; d < a.lanes; d <<= 1) {
            const Key o1 = __shfl_xor(m1, d), o2 = __shfl_xor(m2, d);
            m2 = larger(m1 < o1 ? m1 : o1, larger(m2, o2));
            m1 = larger(m1, o1);
        }
        const Key mine = a.group_top == 2 && m2 > none ? m1 + m2 : m1;
        int rank = 0;  // groups before this lane's
        for (int g = 0; g < a.groups; ++g) {
            const Key other = readlane_f(mine, g * a.lanes);
            rank += other > mine || (other == mine && g < group);
        }
        if (rank >= a.top_groups) {
#pragma unroll
            for (int j = 0; j < PER; ++j) key[j] = none;
        }
    }

    int mine = -1;  // lane k: the k-th chosen expert
    for (int k = 0; k < a.K; ++k) {
        Key best = key[0];
        int j_best = 0;
#pragma unroll
        for (int j = 1; j < PER; ++j)
            if (key[j] > best) best = key[j], j_best = j;
        const Key most = wave_max(best);
        if (!(most > none)) break;
        const int src = __ffsll((unsigned long long)__ballot(best == most)) - 1;
        const int e = readlane(first + j_best, src);
        if (lane == k) mine = e;
        if (lane == src) {
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (j == j_best) key[j] = none;
        }
    }
    float s = 0.f;
    if (mine >= 0) {
        const float lv = l[mine];
        s = a.sigmoid ? 1.0f / (1.0f + __expf(-lv)) : relative_exp(lv, top) / total;
    }
    float w = a.scale * s;
    if (a.normalize) w = w / (wave_sum(s) + kTiny);
    if (lane < a.K) {
        a.topk[t * a.K + lane] = mine;
        if (a.topk_w) a.topk_w[t * a.K + lane] = w;
    }
}

struct RouteGradArgs {
    int T, E, K;
    bool sigmoid, normalize, wide;
    float scale;
    const float* logits;
    const int64_t* topk;
    const float* d_w;
    void* d_logits;
    uint32_t* err;
};

__device__ __forceinline__ float unmasked(float l) { return l != l ? kNone : l; }

// One wave per token: lane k holds lane k of the token's choice.
__global__ __launch_bounds__(kBlockThreads) void route_grad_kernel(RouteGradArgs a) {
    const int lane = lane_id();
    const int64_t t = (int64_t)blockIdx.x * kWavesPerBlock + wave_in_block();
    if (t >= a.T) return;
    const float* l = a.logits + t * a.E;
    float top = kNone, total = 1.f;
    if (!a.sigmoid) {
        for (int e = lane; e < a.E; e += kWave) top = fmaxf(top, unmasked(l[e]));
        top = wave_max(top);
        total = 0.f;
        for (int e = lane; e < a.E; e += kWave) total += relative_exp(unmasked(l[e]), top);
        total = wave_sum(total);
        if (total == 0.f) total = 1.f;  // nothing but masked experts: scores of 0
    }
    int id = -1;
    float s = 0.f, not_s = 0.f, g = 0.f;
    bool bad = false;
    if (lane < a.K) {
        const int64_t e = a.topk[t * a.K + lane];
        bad = expert_bad(e, a.E);
        if (expert_ok(e, a.E)) {
            id = (int)e;
            g = a.scale * a.d_w[t * a.K + lane];
            const float lv = unmasked(l[id]);
            if (a.sigmoid) {
                const float p = __expf(-fabsf(lv)), q = 1.0f / (1.0f + p);
                s = lv >= 0.f ? q : p * q;
                not_s = lv >= 0.f ? p * q : q;
            } else {
                s = relative_exp(lv, top) / total;
            }
        }
    }
    if (__ballot(bad) && lane == 0) report(a.err, EP_DEVERR_EXPERT_ID);
    if (s == 0.f) g = 0.f;  // a masked expert or no lane
    float ds = g, mean = wave_sum(g * s);  // sum of d_s s
    if (a.normalize) {
        const float S = wave_sum(s) + kTiny;
        ds = s == 0.f ? 0.f : (g - mean / S) / S;
        mean = mean / S * (kTiny / S);
    }
    if (a.sigmoid) ds *= s * not_s, mean = 0.f;
    for (int e0 = 0; e0 < a.E; e0 += kWave) {
        const int e = e0 + lane;
        float d = 0.f;
        for (int k = 0; k < a.K; ++k) {
            const int ek = readlane(id, k);
            const float dk = readlane_f(ds, k);
            if (e == ek) d += dk;
        }
        if (e < a.E) {
            if (!a.sigmoid) d = relative_exp(unmasked(l[e]), top) / total * (d - mean);
            if (a.wide)
                static_cast<float*>(a.d_logits)[t * a.E + e] = d;
            else
                static_cast<uint16_t*>(a.d_logits)[t * a.E + e] = (uint16_t)f32_to_bf16(d);
        }
    }
}

}  // namespace

hipError_t launch_route(const ep_shape& s, const float* logits, const ep_router& r, int64_t* topk, float* w, char* ws,
                        hipStream_t st) {
    if (s.T == 0) return hipSuccess;
    const int groups = r.top_groups < s.G ? s.G : 1;
    int lanes = kWave;
    while (lanes * groups > kWave) lanes >>= 1;
    const RouteArgs a = {s.T, s.E, s.K, groups, lanes, r.top_groups, r.group_top, r.score == EP_SCORE_SIGMOID,
                         r.normalize != 0, r.scale, logits, r.bias, topk, w, reinterpret_cast<uint32_t*>(ws)};
    const bool wide = r.bias || (groups > 1 && r.group_top > 1);
    const int need = (s.E / groups + lanes - 1) / lanes;  // at most 124 (groups <= 64)
    void (*const kernels[2][8])(RouteArgs) = {
        {route_kernel<1, false>, route_kernel<2, false>, route_kernel<4, false>, route_kernel<8, false>,
         route_kernel<16, false>, route_kernel<32, false>, route_kernel<64, false>, route_kernel<128, false>},
        {route_kernel<1, true>, route_kernel<2, true>, route_kernel<4, true>, route_kernel<8, true>,
         route_kernel<16, true>, route_kernel<32, true>, route_kernel<64, true>, route_kernel<128, true>}};
    int which = 0;
    while (1 << which < need) ++which;
    hipLaunchKernelGGL(kernels[wide][which], dim3((unsigned)((s.T + kWavesPerBlock - 1) / kWavesPerBlock)),
                       dim3(kBlockThreads), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_route_grad(const ep_shape& s, const float* logits, const ep_router& r, const int64_t* topk,
                             const float* d_w, void* d_logits, int dtype, char* ws, hipStream_t st) {
    if (s.T == 0) return hipSuccess;
    const RouteGradArgs a = {s.T, s.E, s.K, r.score == EP_SCORE_SIGMOID, r.normalize != 0, dtype == EP_GRAD_F32,
                             r.scale, logits, topk, d_w, d_logits, reinterpret_cast<uint32_t*>(ws)};
    hipLaunchKernelGGL(route_grad_kernel, dim3((unsigned)((s.T + kWavesPerBlock - 1) / kWavesPerBlock)),
                       dim3(kBlockThreads), 0, st, a);
    return hipGetLastError();
}

}  // namespace ep
