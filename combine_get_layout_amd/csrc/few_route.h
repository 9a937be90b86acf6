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
// and its tokens in ascending order. Each workgroup finds them for itself:
// the ids are a few KB in L2.
struct Found {
    int expert, used, tokens;
};
template <int THREADS, class Args>
__device__ __forceinline__ Found find_expert(const Args& a, uint32_t* bits, short* token, int* scratch) {
    const int tid = threadIdx.x, lane = lane_id(), wave = wave_in_block();
    if (tid < EP_MAX_EXPERTS / 32) bits[tid] = 0u;
    __syncthreads();
    for (int i = tid; i < a.T * a.K; i += THREADS) {
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

}  // namespace
}  // namespace ep
