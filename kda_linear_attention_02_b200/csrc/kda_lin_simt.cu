// kda_lin_simt.cu -- decayed linear attention, chunked form, fp32 on the fp32 units.
//
// A CTA walks one segment of one (sequence, head) in chunks of C = 32 tokens and holds 32 of the state's dv
// columns.  With g_t = sum of log_alpha over tokens 1..t of the chunk,
//
//     A_tj = e^{g_t - g_j} (q_t . k_j)  (j <= t),
//     o_t  = e^{g_t} S^T q_t + sum_j A_tj v_j,
//     S   <- e^{g_C} S + sum_j e^{g_C - g_j} k_j v_j^T.
//
// The sums g are kept in 64 bits, and the differences rounded once, so that pairs behind a strong decay keep
// their precision; e^{g_C - g_j} comes from sums that start at the chunk's end.  Everything else is fp32 FMA.
#include "kda_device.cuh"
#include "kda_lin.h"

namespace kda {

namespace {

constexpr int kC = 32, kDvs = 32, kNt = 256;

template <int DK>
struct SimtSmem {
    float q[kC][DK + 4], k[kC][DK + 4], v[kC][kDvs], a[kC][kC + 1], s[DK][kDvs + 4];
    double g[kC];
    float eg[kC], w[kC];
};

// rows 0..n-1 of a [C, COLS] tile (row pitch in elements), zeros behind them
template <int COLS, int PITCH>
__device__ __forceinline__ void load_tile(float (*dst)[PITCH], const float* src, size_t pitch, int n) {
    constexpr int V = COLS / 4;
    for (int i = threadIdx.x; i < kC * V; i += kNt) {
        const int r = i / V, c = i % V * 4;
        *reinterpret_cast<float4*>(&dst[r][c]) =
            r < n ? *reinterpret_cast<const float4*>(src + r * pitch + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
}

template <int DK, bool BOUNDARY>
__global__ void __launch_bounds__(kNt) lin_simt_kernel(const LinArgs a) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    SimtSmem<DK>& sh = *reinterpret_cast<SimtSmem<DK>*>(smem_raw);
    grid_launch_dependents();
    grid_dependency_wait();
    const int item = blockIdx.x / a.H, h = blockIdx.x % a.H, j0 = blockIdx.y * kDvs;
    if (item >= a.head->n_items) return;
    const LinItem it = a.items[item];
    if (BOUNDARY && it.seg + 1 == it.n_seg) return;
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    const int hq = h / (a.H / a.Hqk), dv = a.dv;
    const size_t st_elems = static_cast<size_t>(DK) * dv;
    constexpr int R = DK / 32;            // state rows of a thread: R consecutive ones, four columns
    const int r0 = (t >> 3) * R, c0 = (t & 7) * 4;

    float4 S[R];
    const float* start = nullptr;
    if (it.seg == 0) {
        if (a.initial_state) start = a.initial_state + (static_cast<size_t>(it.seq) * a.H + h) * st_elems;
    } else if (!BOUNDARY) {
        start = a.z + (static_cast<size_t>(it.z0 + it.seg - 1) * a.H + h) * st_elems;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        S[r] = start ? *reinterpret_cast<const float4*>(start + (r0 + r) * dv + j0 + c0) : make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4*>(&sh.s[r0 + r][c0]) = S[r];
    }
    auto store_state = [&](float* dst) {
#pragma unroll
        for (int r = 0; r < R; ++r) *reinterpret_cast<float4*>(dst + (r0 + r) * dv + j0 + c0) = S[r];
    };

    const float* Q = static_cast<const float*>(a.q);
    const float* K = static_cast<const float*>(a.k);
    const float* V = static_cast<const float*>(a.v);
    float* O = static_cast<float*>(a.o);
    const size_t pq = static_cast<size_t>(a.Hqk) * DK, pv = static_cast<size_t>(a.H) * dv;
    double total = 0.0;   // sum of log_alpha over the segment (warp 0)
    for (int c = 0; c < it.n; c += kC) {
        const size_t tok = static_cast<size_t>(it.t0) + c;
        const int n = min(kC, it.n - c);
        if (!BOUNDARY) load_tile<DK>(sh.q, Q + tok * pq + static_cast<size_t>(hq) * DK, pq, n);
        load_tile<DK>(sh.k, K + tok * pq + static_cast<size_t>(hq) * DK, pq, n);
        load_tile<kDvs>(sh.v, V + tok * pv + static_cast<size_t>(h) * dv + j0, pv, n);
        if (w == 0) {
            const double x = lane < n ? static_cast<double>(fmaxf(a.la[(tok + lane) * a.la_t + static_cast<size_t>(h) * a.la_h], kLinLogMin)) : 0.0;
            double g = x, r = x;   // inclusive sums from the start and from the end
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const double y = __shfl_up_sync(0xffffffffu, g, off), z = __shfl_down_sync(0xffffffffu, r, off);
                if (lane >= off) g += y;
                if (lane + off < 32) r += z;
            }
            sh.g[lane] = g;
            sh.eg[lane] = expf(static_cast<float>(g));
            sh.w[lane] = expf(static_cast<float>(r - x));
            total += __shfl_sync(0xffffffffu, g, 31);
        }
        __syncthreads();
        if (!BOUNDARY) {
            // scores: a 2 x 2 block for each thread
            const int tr = (t >> 4) * 2, tc = (t & 15) * 2;
            float x00 = 0.f, x01 = 0.f, x10 = 0.f, x11 = 0.f;
            if (tc <= tr + 1) {
#pragma unroll 8
                for (int d = 0; d < DK; d += 4) {
                    const float4 qa = *reinterpret_cast<const float4*>(&sh.q[tr][d]);
                    const float4 qb = *reinterpret_cast<const float4*>(&sh.q[tr + 1][d]);
                    const float4 ka = *reinterpret_cast<const float4*>(&sh.k[tc][d]);
                    const float4 kb = *reinterpret_cast<const float4*>(&sh.k[tc + 1][d]);
                    x00 = fmaf(qa.x, ka.x, fmaf(qa.y, ka.y, fmaf(qa.z, ka.z, fmaf(qa.w, ka.w, x00))));
                    x01 = fmaf(qa.x, kb.x, fmaf(qa.y, kb.y, fmaf(qa.z, kb.z, fmaf(qa.w, kb.w, x01))));
                    x10 = fmaf(qb.x, ka.x, fmaf(qb.y, ka.y, fmaf(qb.z, ka.z, fmaf(qb.w, ka.w, x10))));
                    x11 = fmaf(qb.x, kb.x, fmaf(qb.y, kb.y, fmaf(qb.z, kb.z, fmaf(qb.w, kb.w, x11))));
                }
            }
            const double ga = sh.g[tr], gb = sh.g[tr + 1], ha = sh.g[tc], hb = sh.g[tc + 1];
            sh.a[tr][tc] = tc <= tr ? x00 * expf(static_cast<float>(ga - ha)) : 0.f;
            sh.a[tr][tc + 1] = tc + 1 <= tr ? x01 * expf(static_cast<float>(ga - hb)) : 0.f;
            sh.a[tr + 1][tc] = tc <= tr + 1 ? x10 * expf(static_cast<float>(gb - ha)) : 0.f;
            sh.a[tr + 1][tc + 1] = tc <= tr ? x11 * expf(static_cast<float>(gb - hb)) : 0.f;
            __syncthreads();
            const int row = t >> 3;
            if (row < n) {
                float4 y = make_float4(0.f, 0.f, 0.f, 0.f), x = y;
#pragma unroll 8
                for (int d = 0; d < DK; ++d) {
                    const float qd = sh.q[row][d];
                    const float4 s = *reinterpret_cast<const float4*>(&sh.s[d][c0]);
                    y = make_float4(fmaf(qd, s.x, y.x), fmaf(qd, s.y, y.y), fmaf(qd, s.z, y.z), fmaf(qd, s.w, y.w));
                }
                for (int j = 0; j <= row; ++j) {
                    const float p = sh.a[row][j];
                    const float4 vv = *reinterpret_cast<const float4*>(&sh.v[j][c0]);
                    x = make_float4(fmaf(p, vv.x, x.x), fmaf(p, vv.y, x.y), fmaf(p, vv.z, x.z), fmaf(p, vv.w, x.w));
                }
                const float e = sh.eg[row];
                *reinterpret_cast<float4*>(O + (tok + row) * pv + static_cast<size_t>(h) * dv + j0 + c0) =
                    make_float4(fmaf(e, y.x, x.x), fmaf(e, y.y, x.y), fmaf(e, y.z, x.z), fmaf(e, y.w, x.w));
            }
        }
        // rows behind the sequence's end have log_alpha 0 and k, v of zeros
        const float eC = sh.eg[kC - 1];
#pragma unroll
        for (int r = 0; r < R; ++r) S[r] = make_float4(eC * S[r].x, eC * S[r].y, eC * S[r].z, eC * S[r].w);
#pragma unroll 4
        for (int j = 0; j < kC; ++j) {
            const float4 vv = *reinterpret_cast<const float4*>(&sh.v[j][c0]);
            const float wj = sh.w[j];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float kk = wj * sh.k[j][r0 + r];
                S[r] = make_float4(fmaf(kk, vv.x, S[r].x), fmaf(kk, vv.y, S[r].y), fmaf(kk, vv.z, S[r].z),
                                   fmaf(kk, vv.w, S[r].w));
            }
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < R; ++r) *reinterpret_cast<float4*>(&sh.s[r0 + r][c0]) = S[r];
        const int pos = it.pos + c + kC;
        if (!BOUNDARY && a.ckpt_stride && n == kC && pos % a.ckpt_stride == 0) {
            const long long slot = static_cast<long long>(a.ckpt_cu[it.seq]) + pos / a.ckpt_stride - 1;
            if (slot >= 0 && slot < a.ckpt_cu[it.seq + 1])
                store_state(a.checkpoints + (static_cast<size_t>(slot) * a.H + h) * st_elems);
            else if (t == 0)
                set_status(a.status, KDA_ERR_DEVICE_INPUT);
        }
    }
    if (BOUNDARY) {
        const size_t b = static_cast<size_t>(it.z0 + it.seg) * a.H + h;
        store_state(a.z + b * st_elems);
        if (t == 0 && blockIdx.y == 0) a.zdecay[b] = expf(static_cast<float>(total));
    } else if (a.final_state && it.seg + 1 == it.n_seg) {
        store_state(a.final_state + (static_cast<size_t>(it.seq) * a.H + h) * st_elems);
    }
}

template <int DK, bool BOUNDARY>
cudaError_t launch(const LinArgs& a, cudaStream_t s) {
    constexpr int smem = sizeof(SimtSmem<DK>);
    cudaError_t e = cudaFuncSetAttribute(lin_simt_kernel<DK, BOUNDARY>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.max_items * a.H), a.dv / kDvs);
    cfg.blockDim = dim3(kNt);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, lin_simt_kernel<DK, BOUNDARY>, a);
}

}  // namespace

cudaError_t launch_lin_simt(const LinArgs& a, bool boundary_pass, cudaStream_t s) {
    if (a.dk == 64) return boundary_pass ? launch<64, true>(a, s) : launch<64, false>(a, s);
    return boundary_pass ? launch<128, true>(a, s) : launch<128, false>(a, s);
}

}  // namespace kda
