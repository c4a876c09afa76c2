// kda_lin_step.cu -- decayed linear attention, one token per row:  S <- a S + k v^T,  o = S^T q.
//
// HBM-bound: a CTA streams one (row, head) state once in and once out, 16 bytes a load, all loads of a thread in
// flight before the first use; the column sums of S^T q are joined over the row groups in shared memory.
// 250 rows x 32 heads of 128 (1057 MB): 161 us = 6.56 TB/s, the rate of a plain copy.  One row: 8.4 us, the host's call.
#include "kda_device.cuh"
#include "kda_lin.h"

namespace kda {

namespace {

template <typename T, int DK, int DV, int NT>
__global__ void __launch_bounds__(NT) lin_step_kernel(float* __restrict__ state, long long n_states, const int32_t* slots,
                                                      int slot_stride, const T* q, const T* k, const T* v, const float* la,
                                                      int la_n, int n, int Hqk, int H, T* __restrict__ o, int* status) {
    constexpr int CG = DV / 4, RG = NT / CG, RPT = DK / RG;
    static_assert(RG * CG == NT && RPT * RG == DK && DV <= NT && DK <= NT, "tiling");
    __shared__ float sq[DK], sk[DK];
    __shared__ float4 red[RG][CG];
    const int t = threadIdx.x, cg = t % CG, rg = t / CG;
    const int i = blockIdx.x / H, h = blockIdx.x % H, hq = h / (H / Hqk);
    grid_launch_dependents();
    grid_dependency_wait();
    long long slot = i;
    if (slots) {
        slot = slots[static_cast<size_t>(i) * slot_stride];
        if (slot < 0) return;
        if (slot >= n_states) {
            if (t == 0) set_status(status, KDA_ERR_DEVICE_INPUT);
            return;
        }
    }
    float4* S = reinterpret_cast<float4*>(state + (slot * H + h) * (DK * DV));
    float4 s[RPT];
#pragma unroll
    for (int r = 0; r < RPT; ++r) s[r] = __ldcs(S + (rg * RPT + r) * (DV / 4) + cg);
    const float a = expf(fmaxf(la[static_cast<size_t>(i) * la_n + h], kLinLogMin));
    if (t < DK) {
        sq[t] = to_f32(q[(static_cast<size_t>(i) * Hqk + hq) * DK + t]);
        sk[t] = to_f32(k[(static_cast<size_t>(i) * Hqk + hq) * DK + t]);
    }
    const size_t vo = (static_cast<size_t>(i) * H + h) * DV;
    float x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = to_f32(v[vo + 4 * cg + e]);
    if (slots) {   // a state that two rows name is nobody's
        bool twice = false;
        for (int j = t; j < n; j += NT) twice |= j != i && slots[static_cast<size_t>(j) * slot_stride] == slot;
        if (__syncthreads_or(twice)) {
            if (t == 0) set_status(status, KDA_ERR_DEVICE_INPUT);
            return;
        }
    } else {
        __syncthreads();
    }
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
        const float kk = sk[rg * RPT + r], qq = sq[rg * RPT + r];
        s[r] = make_float4(fmaf(a, s[r].x, kk * x[0]), fmaf(a, s[r].y, kk * x[1]), fmaf(a, s[r].z, kk * x[2]),
                           fmaf(a, s[r].w, kk * x[3]));
        __stcs(S + (rg * RPT + r) * (DV / 4) + cg, s[r]);
        y = make_float4(fmaf(qq, s[r].x, y.x), fmaf(qq, s[r].y, y.y), fmaf(qq, s[r].z, y.z), fmaf(qq, s[r].w, y.w));
    }
    red[rg][cg] = y;
    __syncthreads();
    if (t < DV) {
        const float* p = reinterpret_cast<const float*>(red);
        float sum = 0.f;
#pragma unroll
        for (int g = 0; g < RG; ++g) sum += p[g * DV + t];
        o[vo + t] = from_f32<T>(sum);
    }
}

template <typename T, int DK, int DV>
cudaError_t launch(float* state, int64_t n_states, const int32_t* slots, int slot_stride, const void* q, const void* k,
                   const void* v, const float* la, int la_n, int n, int Hqk, int H, void* o, int* status,
                   cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(n) * H);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, lin_step_kernel<T, DK, DV, 256>, state, static_cast<long long>(n_states), slots, slot_stride,
                              static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v), la, la_n, n,
                              Hqk, H, static_cast<T*>(o), status);
}

template <typename T>
cudaError_t launch_t(float* state, int64_t n_states, const int32_t* slots, int slot_stride, const void* q,
                     const void* k, const void* v, const float* la, int la_n, int n, int Hqk, int H, int dk, int dv,
                     void* o, int* status, cudaStream_t s) {
    auto go = [&](auto f) { return f(state, n_states, slots, slot_stride, q, k, v, la, la_n, n, Hqk, H, o, status, s); };
    if (dk == 64) return dv == 64 ? go(launch<T, 64, 64>) : go(launch<T, 64, 128>);
    return dv == 64 ? go(launch<T, 128, 64>) : go(launch<T, 128, 128>);
}

}  // namespace

cudaError_t launch_lin_step(float* state, int64_t n_states, const int32_t* slots, int slot_stride, const void* q,
                            const void* k, const void* v, const float* la, int la_per_token, int n, int Hqk, int H,
                            int dk, int dv, bool bf16, void* o, int* status, cudaStream_t s) {
    const int la_n = la_per_token ? H : 0;
    return bf16 ? launch_t<__nv_bfloat16>(state, n_states, slots, slot_stride, q, k, v, la, la_n, n, Hqk, H, dk, dv, o, status, s)
                : launch_t<float>(state, n_states, slots, slot_stride, q, k, v, la, la_n, n, Hqk, H, dk, dv, o, status, s);
}

}  // namespace kda
