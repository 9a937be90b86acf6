// swiglu.hip -- ep_swiglu_grad on gfx950: the gradient of act = silu(g) * u from
// the 8-bit checkpoint of g and u.
//
// With s = 1 / (1 + exp(-g)), d the gradient of the expert's output taken back
// through W2 (before the routing weight w) and a = g s u:
//   d_g = w d u s (1 + g (1 - s)),  d_u = w d g s,  act_w = w a,  d_w = <d, a>.
//
// 32 bits throughout, rounded once at the end; the reciprocal is the
// instruction's own, within one unit in the last place.
//
// Bound: one pass over the row, 10 F bytes and its scales. 32,768 rows of F = 2048
// (676 MB): 129 us, 5.2 TB/s, beside 5.0 of a large copy.
#include "ep_internal.h"
#include "ep_mfma.h"

namespace ep {
namespace {

struct SwigluGradArgs {
    int64_t lanes;
    int F, rows;
    const int32_t* slot;
    const float* w;
    const uint8_t* gu;
    const float* scales;
    const uint16_t* d_act;
    uint16_t* d_gu;
    uint16_t* act_w;
    float* d_w;
    uint32_t* err;
};

// One wave per (token, lane): its row in passes of 512 values, 8 per thread, so
// that the row's sum <d, a> needs no atomics and no second launch.
__global__ __launch_bounds__(kBlockThreads) void swiglu_grad_kernel(SwigluGradArgs a) {
    const int lane = lane_id();
    const int64_t n = (int64_t)blockIdx.x * kWavesPerBlock + wave_in_block();
    if (n >= a.lanes) return;
    const int row = a.slot[n];
    const float w = a.w[n];
    if (row < 0 || row >= a.rows) {
        if (lane == 0) {
            if (row >= 0) report(a.err, EP_DEVERR_CAPACITY);
            if (a.d_w) a.d_w[n] = 0.f;
        }
        return;
    }
    const uint8_t* q = a.gu + (int64_t)row * 2 * a.F;
    const float* sc = a.scales + (int64_t)row * (2 * a.F / 128);
    const uint16_t* dr = a.d_act + (int64_t)row * a.F;
    uint16_t* o = a.d_gu + (int64_t)row * 2 * a.F;
    float sum = 0.f;
#pragma unroll 4
    for (int f = lane * 8; f < a.F; f += 512) {
        const u32x2 qg = *reinterpret_cast<const u32x2*>(q + f);
        const u32x2 qu = *reinterpret_cast<const u32x2*>(q + a.F + f);
        const u32x4 dv = ld16(dr + f);
        const float sg = sc[f / 128], su = sc[(a.F + f) / 128];
        u32x4 og, ou, oa;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const auto g2 = (p & 1) ? __builtin_amdgcn_cvt_pk_f32_fp8((int)qg[p >> 1], true)
                                    : __builtin_amdgcn_cvt_pk_f32_fp8((int)qg[p >> 1], false);
            const auto u2 = (p & 1) ? __builtin_amdgcn_cvt_pk_f32_fp8((int)qu[p >> 1], true)
                                    : __builtin_amdgcn_cvt_pk_f32_fp8((int)qu[p >> 1], false);
            float rg[2], ru[2], ra[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float g = g2[j] * sg, u = u2[j] * su;
                const float d = j ? bf16_hi(dv[p]) : bf16_lo(dv[p]);
                const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-g));
                const float gs = g * s, act = gs * u, dw = d * w;
                sum = fmaf(d, act, sum);
                rg[j] = dw * u * (s * fmaf(g, 1.0f - s, 1.0f));
                ru[j] = dw * gs;
                ra[j] = w * act;
            }
            og[p] = pack_bf16(rg[0], rg[1]);
            ou[p] = pack_bf16(ru[0], ru[1]);
            oa[p] = pack_bf16(ra[0], ra[1]);
        }
        st16_stream(o + f, og);
        st16_stream(o + a.F + f, ou);
        if (a.act_w) st16_stream(a.act_w + (int64_t)row * a.F + f, oa);
    }
    if (a.d_w) {
        for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
        if (lane == 0) a.d_w[n] = sum;
    }
}

}  // namespace

hipError_t launch_swiglu_grad(const ep_shape& s, const ep_layout& L, int F, const uint8_t* gu, const float* scales,
                              const uint16_t* d_act, int64_t rows, const float* w, uint16_t* d_gu, uint16_t* act_w,
                              float* d_w, char* ws, hipStream_t st) {
    const int64_t lanes = (int64_t)s.T * s.K;
    if (lanes == 0) return hipSuccess;
    const SwigluGradArgs a = {lanes, F, (int)rows, L.expert_slot, w, gu, scales, d_act, d_gu, act_w, d_w,
                              reinterpret_cast<uint32_t*>(ws)};
    hipLaunchKernelGGL(swiglu_grad_kernel, dim3((unsigned)((lanes + kWavesPerBlock - 1) / kWavesPerBlock)),
                       dim3(kBlockThreads), 0, st, a);
    return hipGetLastError();
}

}  // namespace ep
