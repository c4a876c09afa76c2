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
// The products are bound by shared-memory reads: a thread forms 4 x 4 outputs over a quarter of the inner
// dimension (8 16-byte reads for 64 FMAs; its rows are eight apart, so that neighbouring lanes read neighbouring
// rows), and the quarters are joined in shared memory.  While a chunk is worked on, the next one's rows are
// copied (cp.async) and a ninth warp forms the next one's decays.
//
// 3 sequences of up to 256 tokens x 2 heads of 64: 29 us for a call, 18 of them in the full pass: a chain of chunks on
// 40 blocks.  4 x 4096 tokens x 8 heads of 128: 581 us, bound by the
// shared-memory reads of one block of nine warps on an SM, all of which wait at its barriers (one output a thread: 1223).
// Both figures with segments of half a share of the SMs (see segment_rule).
#include "kda_device.cuh"
#include "kda_lin.h"

namespace kda {

namespace {

constexpr int kC = 32, kDvs = 32, kNt = 256;   // and a warp for the decays
constexpr int kPart = kDvs + 8;                // pitch that keeps four rows of eight columns in different banks

// DK = 64: 77 KB, two blocks on an SM (96 registers x 288 threads); DK = 128: 118 KB, one.
template <int DK>
struct SimtSmem {
    float q[2][kC][DK + 4], k[2][kC][DK + 4], v[2][kC][kDvs];
    float part[4][kC][kPart];   // partial products of the four quarters
    float a[kC][kC + 4], s[DK][kDvs];
    double g[2][kC];
    float eg[2][kC], w[2][kC];
};

// 16 bytes global -> shared by an asynchronous copy, zeros when not `valid` (nothing is read then)
__device__ __forceinline__ void cp_async16z(void* dst, const float* src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(valid ? 16 : 0)
                 : "memory");
}

// rows 0..n-1 of a [C, COLS] tile (row pitch in elements), zeros behind them
template <int COLS, int PITCH>
__device__ __forceinline__ void fetch_tile(float (*dst)[PITCH], const float* src, size_t pitch, int n) {
    constexpr int V = COLS / 4;
#pragma unroll
    for (int i = threadIdx.x; i < kC * V; i += kNt) {
        const int r = i / V, c = i % V * 4;
        cp_async16z(&dst[r][c], r < n ? src + r * pitch + c : src, r < n);
    }
}

template <int DK, bool BOUNDARY>
__global__ void __launch_bounds__(kNt + 32) lin_simt_kernel(const LinArgs a) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    SimtSmem<DK>& sh = *reinterpret_cast<SimtSmem<DK>*>(smem_raw);
    grid_launch_dependents();
    grid_dependency_wait();
    const int item = blockIdx.x / a.H, h = blockIdx.x % a.H, j0 = blockIdx.y * kDvs;
    if (item >= a.head->n_items) return;
    const LinItem it = a.items[item];
    if (BOUNDARY && it.seg + 1 == it.n_seg) return;
    const int t = threadIdx.x;
    const int hq = h / (a.H / a.Hqk), dv = a.dv;
    if (t >= kNt) {
        // ---------------- decays of chunk c into buffer (c / C) % 2, one chunk ahead of the other warps
        const int lane = t & 31;
        const float* la = a.la + h;
        auto load = [&](int c) {
            return c + lane < it.n ? fmaxf(la[(static_cast<size_t>(it.t0) + c + lane) * a.la_t], kLinLogMin) : 0.f;
        };
        double total = 0.0;
        float next = load(0);
        for (int c = 0; c < it.n + kC; c += kC) {
            if (c < it.n) {
                const double x = next;
                next = load(c + kC);
                double g = x, r = x;   // inclusive sums from the start and from the end
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const double y = __shfl_up_sync(0xffffffffu, g, off), z = __shfl_down_sync(0xffffffffu, r, off);
                    if (lane >= off) g += y;
                    if (lane + off < 32) r += z;
                }
                const int b = (c / kC) & 1;
                sh.g[b][lane] = g;
                sh.eg[b][lane] = expf(static_cast<float>(g));
                sh.w[b][lane] = expf(static_cast<float>(r - x));
                total += __shfl_sync(0xffffffffu, g, 31);
            }
            // the other warps' barriers: one before a chunk, and those within the chunk before
            if (c > 0)
                for (int i = 0; i < (BOUNDARY ? 1 : 3); ++i) __syncthreads();
            if (c < it.n) __syncthreads();
        }
        if (BOUNDARY && lane == 0 && blockIdx.y == 0)
            a.zdecay[static_cast<size_t>(it.z0 + it.seg) * a.H + h] = expf(static_cast<float>(total));
        return;
    }
    const size_t st_elems = static_cast<size_t>(DK) * dv;
    constexpr int R = DK / 32;            // state rows of a thread: R consecutive ones, four columns
    const int r0 = (t >> 3) * R, c0 = (t & 7) * 4;
    // products: quarter pk of the inner dimension, rows p8 + 8 i, columns c0 .. c0 + 3 (scores: t % 8 + 8 j)
    const int pk = t >> 6, p8 = (t & 63) >> 3, s8 = t & 7;

    const size_t pq = static_cast<size_t>(a.Hqk) * DK, pv = static_cast<size_t>(a.H) * dv;
    const float* Q = static_cast<const float*>(a.q) + static_cast<size_t>(hq) * DK;
    const float* K = static_cast<const float*>(a.k) + static_cast<size_t>(hq) * DK;
    const float* V = static_cast<const float*>(a.v) + static_cast<size_t>(h) * dv + j0;
    float* O = static_cast<float*>(a.o) + static_cast<size_t>(h) * dv + j0;
    auto fetch = [&](int c) {
        if (c < it.n) {
            const size_t tok = static_cast<size_t>(it.t0) + c;
            const int n = min(kC, it.n - c), b = (c / kC) & 1;
            if (!BOUNDARY) fetch_tile<DK>(sh.q[b], Q + tok * pq, pq, n);
            fetch_tile<DK>(sh.k[b], K + tok * pq, pq, n);
            fetch_tile<kDvs>(sh.v[b], V + tok * pv, pv, n);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    fetch(0);

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
    // tokens to the next checkpoint, and its place
    int to_ck = 0x7fffffff, ck = 0;
    if (!BOUNDARY && a.ckpt_stride) {
        to_ck = a.ckpt_stride - it.pos % a.ckpt_stride;
        ck = a.ckpt_cu[it.seq] + it.pos / a.ckpt_stride;
    }

    for (int c = 0; c < it.n; c += kC) {
        const size_t tok = static_cast<size_t>(it.t0) + c;
        const int n = min(kC, it.n - c), b = (c / kC) & 1;
        fetch(c + kC);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();
        if (!BOUNDARY) {
            float acc[4][4] = {};
#pragma unroll 2
            for (int d = pk * (DK / 4); d < (pk + 1) * (DK / 4); d += 4) {
                float4 x[4], y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(&sh.q[b][p8 + 8 * i][d]);
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(&sh.k[b][s8 + 8 * j][d]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j <= i; ++j)
                        acc[i][j] = fmaf(x[i].x, y[j].x, fmaf(x[i].y, y[j].y, fmaf(x[i].z, y[j].z, fmaf(x[i].w, y[j].w, acc[i][j]))));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j <= i; ++j) sh.part[pk][p8 + 8 * i][s8 + 8 * j] = acc[i][j];
            // q S, in registers until the scores are there
            float qs[4][4] = {};
#pragma unroll 2
            for (int d = pk * (DK / 4); d < (pk + 1) * (DK / 4); d += 4) {
                float4 x[4], y[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(&sh.q[b][p8 + 8 * i][d]);
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(&sh.s[d + j][c0]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float xv[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        qs[i][0] = fmaf(xv[e], y[e].x, qs[i][0]);
                        qs[i][1] = fmaf(xv[e], y[e].y, qs[i][1]);
                        qs[i][2] = fmaf(xv[e], y[e].z, qs[i][2]);
                        qs[i][3] = fmaf(xv[e], y[e].w, qs[i][3]);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float e = sh.eg[b][p8 + 8 * i];
#pragma unroll
                for (int j = 0; j < 4; ++j) qs[i][j] *= e;
            }
            __syncthreads();
            {   // scores: row t / 8, columns 4 (t % 8) ..
                const int row = t >> 3;
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = c0 + e;
                    y[e] = 0.f;
                    if (j <= row)
                        y[e] = ((sh.part[0][row][j] + sh.part[1][row][j]) + (sh.part[2][row][j] + sh.part[3][row][j])) *
                               expf(static_cast<float>(sh.g[b][row] - sh.g[b][j]));
                }
                *reinterpret_cast<float4*>(&sh.a[row][c0]) = make_float4(y[0], y[1], y[2], y[3]);
            }
            __syncthreads();
            // tokens 8 pk .. 8 pk + 7; a token behind a row's own is left out, not multiplied by zero
#pragma unroll
            for (int d = 0; d < kC / 4; ++d) {
                const int j = pk * (kC / 4) + d;
                const float4 vv = *reinterpret_cast<const float4*>(&sh.v[b][j][c0]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (j > p8 + 8 * i) continue;
                    const float p = sh.a[p8 + 8 * i][j];
                    qs[i][0] = fmaf(p, vv.x, qs[i][0]);
                    qs[i][1] = fmaf(p, vv.y, qs[i][1]);
                    qs[i][2] = fmaf(p, vv.z, qs[i][2]);
                    qs[i][3] = fmaf(p, vv.w, qs[i][3]);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<float4*>(&sh.part[pk][p8 + 8 * i][c0]) = make_float4(qs[i][0], qs[i][1], qs[i][2], qs[i][3]);
        }
        // rows behind the sequence's end have log_alpha 0 and k, v of zeros
        const float eC = sh.eg[b][kC - 1];
#pragma unroll
        for (int r = 0; r < R; ++r) S[r] = make_float4(eC * S[r].x, eC * S[r].y, eC * S[r].z, eC * S[r].w);
#pragma unroll 8
        for (int j = 0; j < kC; ++j) {
            const float4 vv = *reinterpret_cast<const float4*>(&sh.v[b][j][c0]);
            const float wj = sh.w[b][j];
            float kk[R];
            if constexpr (R == 4) {
                const float4 k4 = *reinterpret_cast<const float4*>(&sh.k[b][j][r0]);
                kk[0] = k4.x; kk[1] = k4.y; kk[2] = k4.z; kk[3] = k4.w;
            } else {
                const float2 k2 = *reinterpret_cast<const float2*>(&sh.k[b][j][r0]);
                kk[0] = k2.x; kk[1] = k2.y;
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float x = wj * kk[r];
                S[r] = make_float4(fmaf(x, vv.x, S[r].x), fmaf(x, vv.y, S[r].y), fmaf(x, vv.z, S[r].z), fmaf(x, vv.w, S[r].w));
            }
        }
        __syncthreads();
        if (!BOUNDARY) {
            const int row = t >> 3;
            if (row < n) {
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    y[e] = (sh.part[0][row][c0 + e] + sh.part[1][row][c0 + e]) + (sh.part[2][row][c0 + e] + sh.part[3][row][c0 + e]);
                *reinterpret_cast<float4*>(O + (tok + row) * pv + c0) = make_float4(y[0], y[1], y[2], y[3]);
            }
#pragma unroll
            for (int r = 0; r < R; ++r) *reinterpret_cast<float4*>(&sh.s[r0 + r][c0]) = S[r];
            to_ck -= kC;
            if (to_ck == 0 && n == kC) {
                to_ck = a.ckpt_stride;
                if (ck >= 0 && a.checkpoints && ck < a.ckpt_cu[it.seq + 1])
                    store_state(a.checkpoints + (static_cast<size_t>(ck) * a.H + h) * st_elems);
                else if (t == 0)
                    set_status(a.status, KDA_ERR_DEVICE_INPUT);
                ++ck;
            }
        }
    }
    cp_async_wait_all();
    if (BOUNDARY) store_state(a.z + (static_cast<size_t>(it.z0 + it.seg) * a.H + h) * st_elems);
    else if (a.final_state && it.seg + 1 == it.n_seg)
        store_state(a.final_state + (static_cast<size_t>(it.seq) * a.H + h) * st_elems);
}

template <int DK, bool BOUNDARY>
cudaError_t launch(const LinArgs& a, cudaStream_t s) {
    constexpr int smem = sizeof(SimtSmem<DK>);
    static SmemLimit limit;
    cudaError_t e = limit.raise(reinterpret_cast<const void*>(&lin_simt_kernel<DK, BOUNDARY>), smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.max_items * a.H), a.dv / kDvs);
    cfg.blockDim = dim3(kNt + 32);
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
