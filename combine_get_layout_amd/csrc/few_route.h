// few_route.h -- what the few-token layers share: which experts the tokens use,
// and which tokens each of these has.
#pragma once

#include "ep_device.h"

namespace ep {
namespace {

// One token of a used expert: token << 16 | row of its inner activations (token
// * K + its first lane with that expert), and the sum of its lanes' weights.
struct Route {
    int id;
    float w;
};

// The blockIdx.y-th used expert in ascending order (-1 if there are fewer)
// and its tokens in ascending order. Each workgroup finds them for itself: it reads
// the ids once and keeps them in LDS; the routes, which take the weights too, are
// made by the workgroups with blockIdx.x = 0.
struct Found {
    int expert, used, tokens;
};
constexpr int kNoExpert = 0xFFFF;
struct FindShared {
    uint32_t bits[EP_MAX_EXPERTS / 32];
    short token[EP_FEW_MAX_TOKENS];         // the expert's tokens
    short row[EP_FEW_MAX_TOKENS];           // and the rows of their inner activations
    int scratch[2];
    uint16_t ids[EP_FEW_MAX_TOKENS * EP_MAX_TOPK];
};
template <int THREADS, class Args>
__device__ __forceinline__ Found find_expert(const Args& a, FindShared& sh) {
    const int tid = threadIdx.x, lane = lane_id(), wave = wave_in_block();
    if (tid < EP_MAX_EXPERTS / 32) sh.bits[tid] = 0u;
    __syncthreads();
    for (int i = tid; i < a.T * a.K; i += THREADS) {
        const int64_t e = a.topk[i];
        const bool ok = expert_ok(e, a.E);
        sh.ids[i] = (uint16_t)(ok ? (int)e : kNoExpert);
        if (ok) atomicOr(&sh.bits[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    const uint64_t word = (uint64_t)sh.bits[2 * lane] | (uint64_t)sh.bits[2 * lane + 1] << 32;
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
                if (sh.ids[tid * a.K + k] != f.expert) continue;
                if (r.id < 0) r.id = tid << 16 | (tid * a.K + k);
                if (blockIdx.x == 0) r.w += a.topk_w[tid * a.K + k];
            }
        }
        mine = r.id >= 0;
        const uint64_t m = __ballot(mine);
        if (lane == 0) sh.scratch[wave] = __popcll(m);
    }
    __syncthreads();
    f.tokens = sh.scratch[0] + sh.scratch[1];
    if (wave < 2 && mine) {
        const uint64_t m = __ballot(true);
        const int at = (wave ? sh.scratch[0] : 0) + __popcll(m & ((1ull << lane) - 1));
        sh.token[at] = (short)tid;
        sh.row[at] = (short)(r.id & 0xFFFF);
        if (blockIdx.x == 0) a.routes[(int64_t)want * a.T + at] = r;
    }
    if (blockIdx.x == 0 && tid == 0) a.used[1 + want] = f.expert | f.tokens << 16;
    __syncthreads();
    return f;
}

}  // namespace
}  // namespace ep
