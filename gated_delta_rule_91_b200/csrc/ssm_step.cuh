// ssm_step.cuh -- one token of the selective scan (gdr_ssm_step), the fp32
// state updated in place.  Row p of a head's state evolves on its own:
//     S_p <- a S_p + (Delta x_p) B,   y_p = S_p(new) . C + D x_p
// so the state is read once and written once, which is the whole cost
// (2 P N * 4 bytes per head): the step is HBM-bound.  A row of N fp32 is N/4
// lanes x float4; a warp keeps kSsmStepLoads float4 loads per lane in flight
// before any use, as in gdr_step.  B=256 H=16 P=N=128: 84 us, 6.4 TB/s.
#pragma once
#include "ssm_common.cuh"

namespace gdr {

constexpr int kSsmStepWarps = 4, kSsmStepLoads = 8;

template <typename T, int N>
__global__ void __launch_bounds__(kSsmStepWarps * 32) ssm_step_kernel(SsmArgs a) {
    constexpr int kLanes = N / 4, kSub = 32 / kLanes, kRows = kSsmStepLoads * kSub * kSsmStepWarps;
    const int nblk = a.P / kRows;
    const int bh = blockIdx.x / nblk, b = bh / a.H, h = bh % a.H, g = h / (a.H / a.G);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = (lane % kLanes) * 4, sub = lane / kLanes;
    const int row0 = (blockIdx.x % nblk) * kRows + warp * kSsmStepLoads * kSub + sub;
    float *S = a.S_T + (size_t)bh * a.P * N;
    float4 s[kSsmStepLoads];
#pragma unroll
    for (int l = 0; l < kSsmStepLoads; ++l)
        s[l] = __ldcs(reinterpret_cast<const float4 *>(S + (size_t)(row0 + l * kSub) * N + col));
    const float4 bb = load4(static_cast<const T *>(a.Bm) + (size_t)b * a.ldb + (size_t)g * N + col);
    const float4 cc = load4(static_cast<const T *>(a.Cm) + (size_t)b * a.ldc + (size_t)g * N + col);
    const T *x = static_cast<const T *>(a.x) + (size_t)b * a.ldx + (size_t)h * a.P;
    const float dt = ssm_step_size(a, b, 0, h);
    const float al = expf(a.A[h] * dt), D = a.D ? a.D[h] : 0.f;
    T *y = static_cast<T *>(a.y) + (size_t)bh * a.P;
#pragma unroll
    for (int l = 0; l < kSsmStepLoads; ++l) {
        const int row = row0 + l * kSub;
        const float xv = to_f32(x[row]), u = dt * xv;
        float4 n;
        n.x = fmaf(al, s[l].x, u * bb.x);
        n.y = fmaf(al, s[l].y, u * bb.y);
        n.z = fmaf(al, s[l].z, u * bb.z);
        n.w = fmaf(al, s[l].w, u * bb.w);
        __stcs(reinterpret_cast<float4 *>(S + (size_t)row * N + col), n);
        const float o = warp_sum(n.x * cc.x + n.y * cc.y + n.z * cc.z + n.w * cc.w, kLanes);
        if (lane % kLanes == 0) y[row] = from_f32<T>(a.D ? fmaf(D, xv, o) : o);
    }
}

template <typename T, int N>
cudaError_t ssm_step_launch(const SsmArgs &a, cudaStream_t s) {
    constexpr int kRows = kSsmStepLoads * (32 / (N / 4)) * kSsmStepWarps;  // 32 or 64: divides P
    ssm_step_kernel<T, N><<<(unsigned)(a.B * a.H) * (unsigned)(a.P / kRows), kSsmStepWarps * 32, 0, s>>>(a);
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return cudaGetLastError();
}

}  // namespace gdr
