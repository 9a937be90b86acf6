// route.hip -- ep_route and ep_route_grad on gfx950.
//
// A token's experts are spread over a wave, so that the softmax's maximum and sum, the
// groups and each of the K choices take lane-to-lane moves alone, without LDS or barriers.
// Bytes are few (4,096 tokens of 256 experts: 4.5 MB, 0.9 us at the memory's rate); what
// bounds it is the chain of K rounds, each a maximum over the wave that the next waits for,
// and the keys' arithmetic:
//   4,096 tokens, top-8 of 256, 4 of 8 groups by sums of two, bias (64-bit keys)  10.1 us
//   the same without groups, softmax                                              10.1 us
//   the same without bias (keys are the logits): softmax, sigmoid             6.8, 6.2 us
//   13 tokens, top-6 of 72, softmax (keys are the logits)                          3.4 us
//   1,024 tokens, top-8 of 4,092 in 33 groups: 124 experts in a lane's registers, of which
//     944 bytes spill (64-bit keys, where more than 64 fall to a lane)             140 us
//   gradients: 4,096 tokens of 256 experts, sigmoid, softmax                  5.0, 7.3 us
//              333 tokens of 48 experts, softmax                                   4.2 us
// Choices are made by keys in 64 bits
// where scores and biases are added: rounded to 32 bits, sums that differ would tie.
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
    int64_t token0;  // first token of this launch
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
// infinity, 0 for a masked expert. __expf scales its argument to base 2 in 32 bits, which
// puts |l - top| 2^-24 on the value, as much as the difference itself has lost: 5e-6 of a
// score of e^-80, nothing that counts in a sum with the largest's 1. No id depends on it.
__device__ __forceinline__ float relative_exp(float l, float top) { return l == kNone ? 0.f : l == top ? 1.f : __expf(l - top); }

// Keys as unsigned numbers of the same order: 0 for a masked expert (below every
// number's), the same for both zeros.
template <class Key>
__device__ __forceinline__ Key ordered(std::conditional_t<sizeof(Key) == 8, double, float> v) {
    constexpr Key kTop = (Key)1 << (8 * sizeof(Key) - 1);
    if (!(v > kNone)) return 0;
    const Key u = __builtin_bit_cast(Key, v + 0);
    return u & kTop ? ~u : u | kTop;
}
__device__ __forceinline__ uint32_t upper(uint32_t k) { return k; }
__device__ __forceinline__ uint32_t upper(uint64_t k) { return (uint32_t)(k >> 32); }
__device__ __forceinline__ uint32_t readlane_u(uint32_t v, int lane) { return (uint32_t)readlane((int)v, lane); }
__device__ __forceinline__ uint64_t readlane_u(uint64_t v, int lane) {
    return (uint64_t)readlane_u((uint32_t)(v >> 32), lane) << 32 | readlane_u((uint32_t)v, lane);
}
// The lowest lane with the largest key, -1 if all are masked. The upper halves
// decide nearly always.
template <class Key>
__device__ __forceinline__ int first_largest(Key key) {
    const uint32_t most = wave_max(upper(key));
    if (most == 0u) return -1;
    uint64_t lanes = __ballot(upper(key) == most);
    if constexpr (sizeof(Key) == 8) {
        if (lanes & (lanes - 1)) {
            const uint32_t low = upper(key) == most ? (uint32_t)key : 0u, most_low = wave_max(low);
            lanes = __ballot(upper(key) == most && low == most_low);
        }
    }
    return __ffsll((unsigned long long)lanes) - 1;
}

// One wave per token. A group's experts lie in `lanes` neighbouring lanes, PER
// to a lane in ascending order, so that ties go to the lowest lane. WIDE: keys
// are scores and biases in 64 bits, else the logits.
template <int PER, bool WIDE>
__global__ __launch_bounds__(kBlockThreads) void route_kernel(RouteArgs a) {
    using Number = std::conditional_t<WIDE, double, float>;
    using Key = std::conditional_t<WIDE, uint64_t, uint32_t>;
    const int lane = lane_id();
    const int64_t t = a.token0 + (int64_t)blockIdx.x * kWavesPerBlock + wave_in_block();
    if (t >= a.T) return;
    const int size = a.E / a.groups, group = lane / a.lanes, at = lane % a.lanes * PER;
    const int first = group * size + at;  // this lane's first expert
    const int held = group < a.groups ? min(max(size - at, 0), PER) : 0;
    const float* l = a.logits + t * a.E;
    float v[PER];
    Number key[PER];
    bool bad = false;
    float top = kNone;
#pragma unroll
    for (int j = 0; j < PER; ++j) v[j] = j < held ? l[first + j] : kNone;
    if constexpr (WIDE) {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const float b = a.bias && j < held ? a.bias[first + j] : 0.f;
            if (b != b) bad = true;
            key[j] = b;
        }
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        if (v[j] != v[j]) bad = true, v[j] = kNone;
        top = fmaxf(top, v[j]);
    }
    if (__ballot(bad) && lane == 0) report(a.err, EP_DEVERR_LOGIT);
    float total = 1.f;
    if (!a.sigmoid) {
        top = wave_max(top);
        total = 0.f;
#pragma unroll
        for (int j = 0; j < PER; ++j) total += relative_exp(v[j], top);
        total = wave_sum(total);
    }
    if constexpr (WIDE) {
        if (a.sigmoid) {
#pragma unroll
            for (int j = 0; j < PER; ++j) key[j] += 1.0 / (1.0 + exp(-(double)v[j]));
        } else {
            double p[PER], sum = 0.0;
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                p[j] = v[j] == top ? 1.0 : exp((double)v[j] - (double)top);
                if (v[j] == kNone) p[j] = 0.0;
                sum += p[j];
            }
            sum = wave_sum(sum);
#pragma unroll
            for (int j = 0; j < PER; ++j) key[j] = p[j] / sum + key[j];
        }
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (v[j] == kNone || !(key[j] > kNone)) key[j] = kNone;
    } else {
#pragma unroll
        for (int j = 0; j < PER; ++j) key[j] = v[j];
    }

    if (a.groups > 1) {
        Number m1 = kNone, m2 = kNone;  // this lane's two largest, then the group's
        auto more = [&](Number k) {
            const bool above = k > m1;
            m2 = above ? m1 : k > m2 ? k : m2;
            m1 = above ? k : m1;
        };
        auto merge = [&](Number o1, Number o2) {
            more(o1);
            more(o2);
        };
#pragma unroll
        for (int j = 0; j < PER; ++j) more(key[j]);
        // Lanes whose halves of the group hold the same two change places by a mirror too.
        if (a.lanes > 1) merge(dpp<kDppSwap1>(m1), dpp<kDppSwap1>(m2));
        if (a.lanes > 2) merge(dpp<kDppSwap2>(m1), dpp<kDppSwap2>(m2));
        if (a.lanes > 4) merge(dpp<kDppMirror8>(m1), dpp<kDppMirror8>(m2));
        if (a.lanes > 8) merge(dpp<kDppMirror16>(m1), dpp<kDppMirror16>(m2));
        if (a.lanes > 16) merge(__shfl_xor(m1, 16), __shfl_xor(m2, 16));
        const Key mine = ordered<Key>(a.group_top == 2 && m2 > kNone ? m1 + m2 : m1);
        int rank = 0;  // groups before this lane's
        for (int g = 0; g < a.groups; ++g) {
            const Key other = readlane_u(mine, g * a.lanes);
            rank += other > mine || (other == mine && g < group);
        }
        if (rank >= a.top_groups) {
#pragma unroll
            for (int j = 0; j < PER; ++j) key[j] = kNone;
        }
    }

    struct Expert {
        Key key;
        int id;
        float logit;
    };
    Expert left[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) left[j] = {ordered<Key>(key[j]), first + j, v[j]};
    // Few to a lane: each lane's in order once, then the first of each is all that a
    // round looks at. Else the lane's largest is looked for every time.
    constexpr bool kSorted = PER <= 8;
    if constexpr (kSorted) {
#pragma unroll
        for (int n = 1; n < PER; ++n)  // equal keys keep their order
#pragma unroll
            for (int j = n; j > 0; --j) {
                const Expert x = left[j - 1], y = left[j];
                const bool swap = y.key > x.key;
                left[j - 1] = {swap ? y.key : x.key, swap ? y.id : x.id, swap ? y.logit : x.logit};
                left[j] = {swap ? x.key : y.key, swap ? x.id : y.id, swap ? x.logit : y.logit};
            }
    }
    int mine = -1;  // lane k: the k-th chosen expert and its logit
    float lv = 0.f;
    for (int k = 0; k < a.K; ++k) {
        Expert best = left[0];
        int which = 0;
        if constexpr (!kSorted) {
#pragma unroll
            for (int j = 1; j < PER; ++j)
                if (left[j].key > best.key) best = left[j], which = j;
        }
        const int src = first_largest(best.key);
        if (src < 0) break;
        const int e = readlane(best.id, src);
        const float chosen = readlane_f(best.logit, src);
        if (lane == k) mine = e, lv = chosen;
        if (lane == src) {
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                if constexpr (kSorted) {
                    if (j + 1 < PER)
                        left[j] = left[j + 1 < PER ? j + 1 : 0];
                    else
                        left[j].key = 0;
                } else if (j == which) {
                    left[j].key = 0;
                }
            }
        }
    }
    float s = 0.f;
    if (mine >= 0) s = a.sigmoid ? 1.0f / (1.0f + __expf(-lv)) : relative_exp(lv, top) / total;
    float w = a.scale * s;
    if (a.normalize) w = w / (wave_sum(s) + kTiny);
    if (lane < a.K) {
        a.topk[t * a.K + lane] = mine;
        if (a.topk_w) a.topk_w[t * a.K + lane] = w;
    }
}

struct RouteGradArgs {
    int T, E, K;
    int64_t token0;
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
template <int VEC>
__global__ __launch_bounds__(kBlockThreads) void route_grad_kernel(RouteGradArgs a) {
    const int lane = lane_id();
    const int64_t t = a.token0 + (int64_t)blockIdx.x * kWavesPerBlock + wave_in_block();
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
    // VEC experts to a lane at a time.
    for (int e0 = 0; e0 < a.E; e0 += kWave * VEC) {
        const int e = e0 + lane * VEC;
        float d[VEC] = {};
        for (int k = 0; k < a.K; ++k) {
            const int ek = readlane(id, k) - e;
            const float dk = readlane_f(ds, k);
#pragma unroll
            for (int j = 0; j < VEC; ++j) d[j] += ek == j ? dk : 0.f;
        }
        if (e >= a.E) continue;
        if (!a.sigmoid) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) d[j] = relative_exp(unmasked(l[e + j]), top) / total * (d[j] - mean);
        }
        if constexpr (VEC == 4) {
            if (a.wide) {
                st16(static_cast<float*>(a.d_logits) + t * a.E + e, u32x4{__float_as_uint(d[0]), __float_as_uint(d[1]),
                                                                          __float_as_uint(d[2]), __float_as_uint(d[3])});
            } else {
                *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.d_logits) + t * a.E + e) =
                    u32x2{pack_bf16(d[0], d[1]), pack_bf16(d[2], d[3])};
            }
        } else if (a.wide) {
            static_cast<float*>(a.d_logits)[t * a.E + e] = d[0];
        } else {
            static_cast<uint16_t*>(a.d_logits)[t * a.E + e] = (uint16_t)f32_to_bf16(d[0]);
        }
    }
}

// One wave to a token, in launches of kLaunchGroups workgroups.
template <class Args>
hipError_t launch_tokens(void (*kernel)(Args), Args& a, hipStream_t st) {
    for (a.token0 = 0; a.token0 < a.T; a.token0 += kLaunchGroups * kWavesPerBlock) {
        const int64_t groups = std::min((a.T - a.token0 + kWavesPerBlock - 1) / kWavesPerBlock, kLaunchGroups);
        hipLaunchKernelGGL(kernel, dim3((unsigned)groups), dim3(kBlockThreads), 0, st, a);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const ep_shape& s, const float* logits, const ep_router& r, int64_t* topk, float* w, char* ws,
                        hipStream_t st) {
    if (s.T == 0) return hipSuccess;
    const int groups = r.top_groups < s.G ? s.G : 1;
    int lanes = kWave;
    while (lanes * groups > kWave) lanes >>= 1;
    RouteArgs a = {s.T, s.E, s.K, 0, groups, lanes, r.top_groups, r.group_top, r.score == EP_SCORE_SIGMOID,
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
    return launch_tokens(kernels[wide][which], a, st);
}

hipError_t launch_route_grad(const ep_shape& s, const float* logits, const ep_router& r, const int64_t* topk,
                             const float* d_w, void* d_logits, int dtype, char* ws, hipStream_t st) {
    if (s.T == 0) return hipSuccess;
    RouteGradArgs a = {s.T, s.E, s.K, 0, r.score == EP_SCORE_SIGMOID, r.normalize != 0, dtype == EP_GRAD_F32,
                             r.scale, logits, topk, d_w, d_logits, reinterpret_cast<uint32_t*>(ws)};
    return launch_tokens(s.E % 4 == 0 ? route_grad_kernel<4> : route_grad_kernel<1>, a, st);
}

}  // namespace ep
