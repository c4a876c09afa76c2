// kda_lin_bf16.cu -- decayed linear attention, chunked form, bf16 on the 5th-generation tensor cores.
//
// One CTA walks a segment of one (sequence, head) in chunks of 64 tokens.  With g_t the sum of log_alpha over
// tokens 1..t of the chunk, all products are written transposed, channels of v in the accumulator's lanes:
//
//     scores   s_tj = q_t . k_j                                   (SP, tokens t in lanes)
//     P_tj     = e^{g_t - g_j} s_tj  (j <= t), rounded to bf16
//     o_t      = e^{g_t} (S^T q_t)  +  sum_j P_tj v_j             (O1 = Sb Q^T, O2 = V^T P^T)
//     S^T     <- e^{g_C} S^T + sum_j (e^{g_C - g_j} v_j) k_j^T    (Z = W K, W_j = e^{g_C - g_j} v_j)
//
// S^T stays in fp32 registers (thread = channel of v, register = channel of k); its bf16 copy Sb goes to
// tensor memory as O1's A operand, in the lane layout the registers already have, and W takes the same way.
// What reaches o is rounded once in each path (P, and the copy of S).  What reaches the state is not: k and v
// are bf16 already, and W is split into three bf16 parts, which hold all 24 bits of the fp32 product, so Z is
// an fp32 sum of exact products.  Z starts from zero in every chunk and joins S by one rounded FMA: an
// accumulator that lived on in tensor memory would collect the truncation of its additions over the length of
// the sequence.
//
// The warps are specialised and meet at mbarriers: a producer (TMA tiles of q, k, v, and the chunk's decays),
// an issuer (all MMAs, in an order that keeps Z of one chunk ahead of the scores of the next), two warps for
// P, four that split W and write o, four that hold the state.
#include <string.h>

#include "kda_device.cuh"
#include "kda_lin.h"

namespace kda {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <int DK, int DV, bool BOUNDARY>
struct Cfg {
    static constexpr int C = kChunk;
    static constexpr uint32_t HALF = C * 128;                        // a 64-channel half tile: 64 rows of 128 B
    static constexpr uint32_t QB = BOUNDARY ? 0 : DK / 64 * HALF, KB = DK / 64 * HALF, VB = DV / 64 * HALF;
    static constexpr uint32_t STAGE = QB + KB + VB;
    static constexpr int NST = BOUNDARY ? 5 : (STAGE > 40960 ? 3 : 4);
    static constexpr uint32_t PB = C * 128;                          // P: 64 rows of 64 bf16
    static constexpr uint32_t P0 = NST * STAGE, O0 = P0 + (BOUNDARY ? 0 : 2 * PB);
    // the A operands of 128 rows read past 64-row tiles (their results are not used): the tiles behind exist
    static constexpr uint32_t BYTES = O0 + (BOUNDARY ? HALF : 2 * VB);
    // tensor memory columns
    static constexpr uint32_t SP = 0, O1 = 64, O2 = 128, Z = 192, SB = 320, W = 384, COLS = 512;
    static_assert(BYTES + 1024 + 4096 <= 227 * 1024, "shared memory");
};
constexpr int kThreads = 384;
constexpr int kPWarps = 2, kVWarps = 4, kSWarps = 4;

struct Decays {            // of one chunk
    float g2[kChunk];      // g_t log2(e)
    float eg[kChunk];      // e^{g_t}
    float w[kChunk];       // e^{g_C - g_t}
    float eC;              // e^{g_C}
    float pad[3];
};

// fp32 pair -> packed bf16 pair, and back
__device__ __forceinline__ float lo_f32(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f32(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// One lane of a converged warp, always the same one.  The MMAs are issued under this predicate by a warp whose
// addresses are warp-uniform values: issued by a lane chosen with threadIdx, from values the compiler cannot
// see to be uniform, each costs about 96 cycles; so, 32 to 64 (M = 128, K = 16, N = 64 to 128).
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t (&v)[16]) {
    tmem_st16(taddr, reinterpret_cast<const float(&)[16]>(v));
}

template <int DK, int DV, bool BOUNDARY>
__global__ void __launch_bounds__(kThreads, 1)
lin_bf16_kernel(const LinArgs a, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo) {
    using F = Cfg<DK, DV, BOUNDARY>;
    constexpr int NST = F::NST, C = F::C;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ Decays decays[NST];
    __shared__ __align__(8) uint64_t full[NST], empty[NST], sp_full, sp_free, p_ready[2], p_free[2], w_ready, z_full,
        z_free, sb_ready, sb_free, o_full, o_free, done;
    __shared__ uint32_t tmem_slot;
    const int t = threadIdx.x, w = __shfl_sync(0xffffffffu, t >> 5, 0), lane = t & 31;
    if (t == 0) {
        for (int s = 0; s < NST; ++s) {
            mbar_init(&full[s], 2);
            mbar_init(&empty[s], 1 + (BOUNDARY ? 0 : kPWarps) + kVWarps + kSWarps);
        }
        mbar_init(&sp_full, 1);
        mbar_init(&sp_free, kPWarps);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&p_ready[b], kPWarps);
            mbar_init(&p_free[b], 1);
        }
        mbar_init(&w_ready, kVWarps);
        mbar_init(&z_full, 1);
        mbar_init(&z_free, kSWarps);
        mbar_init(&sb_ready, kSWarps);
        mbar_init(&sb_free, 1);
        mbar_init(&o_full, 1);
        mbar_init(&o_free, kVWarps);
        mbar_init(&done, 1);
        fence_barrier_init();
    }
    grid_dependency_wait();
    const int item = blockIdx.x / a.H, h = blockIdx.x % a.H;
    if (item >= a.head->n_items) return;
    const LinItem it = a.items[item];
    if (BOUNDARY && it.seg + 1 == it.n_seg) return;
    if (w == 3) {
        tmem_alloc(&tmem_slot, F::COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_slot;
    const int nch = (it.n + C - 1) / C, hq = h / (a.H / a.Hqk);
    int* const status = a.status;

    if (w == 2) {
        // ---------------- producer
        const float* la = a.la + static_cast<size_t>(h) * a.la_h;
        auto log_alpha = [&](int c, float& x0, float& x1) {
            const int i = c * C + 2 * lane;
            const size_t tok = static_cast<size_t>(it.t0) + i;
            x0 = i < it.n ? fmaxf(la[tok * a.la_t], kLinLogMin) : 0.f;
            x1 = i + 1 < it.n ? fmaxf(la[(tok + 1) * a.la_t], kLinLogMin) : 0.f;
        };
        float x0, x1, total = 0.f;
        if (nch > 0) log_alpha(0, x0, x1);
        int issued = 0;
        for (int c = 0; c < nch; ++c) {
            const int s = c % NST;
            if (!mbar_wait(&empty[s], ((c / NST) & 1) ^ 1, status)) break;
            uint8_t* sb = sm + s * F::STAGE;
            if (lane == 0) {
                mbar_arrive_expect_tx(&full[s], F::STAGE);
                const int tok = it.t0 + c * C;
                if (!BOUNDARY)
                    for (int b = 0; b < DK / 64; ++b) tma_load_2d(sb + b * F::HALF, &mq, hq * DK + 64 * b, tok, &full[s]);
                for (int b = 0; b < DK / 64; ++b) tma_load_2d(sb + F::QB + b * F::HALF, &mk, hq * DK + 64 * b, tok, &full[s]);
                for (int b = 0; b < DV / 64; ++b)
                    tma_load_2d(sb + F::QB + F::KB + b * F::HALF, &mv, h * DV + 64 * b, tok, &full[s]);
            }
            issued = c + 1;
            // inclusive sums of the lanes' pairs, from the chunk's start and from its end
            float y0 = 0.f, y1 = 0.f;
            if (c + 1 < nch) log_alpha(c + 1, y0, y1);
            float f = x0 + x1, r = f;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const float u = __shfl_up_sync(0xffffffffu, f, off), v = __shfl_down_sync(0xffffffffu, r, off);
                if (lane >= off) f += u;
                if (lane + off < 32) r += v;
            }
            float before = __shfl_up_sync(0xffffffffu, f, 1), after = __shfl_down_sync(0xffffffffu, r, 1);
            if (lane == 0) before = 0.f;
            if (lane == 31) after = 0.f;
            const float sum = __shfl_sync(0xffffffffu, f, 31);
            Decays& d = decays[s];
            const float g0 = before + x0, g1 = f;
            *reinterpret_cast<float2*>(&d.g2[2 * lane]) = make_float2(g0 * kLog2e, g1 * kLog2e);
            *reinterpret_cast<float2*>(&d.eg[2 * lane]) = make_float2(expf(g0), expf(g1));
            *reinterpret_cast<float2*>(&d.w[2 * lane]) = make_float2(expf(after + x1), expf(after));
            if (lane == 0) d.eC = expf(sum);
            total += sum;
            x0 = y0;
            x1 = y1;
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[s]);
        }
        if (BOUNDARY && lane == 0) a.zdecay[static_cast<size_t>(it.z0 + it.seg) * a.H + h] = expf(total);
        // no copy stays in flight behind the CTA: wait (bounded, quietly) for the last fill of every stage
        for (int c = issued > NST ? issued - NST : 0; c < issued; ++c) mbar_wait(&full[c % NST], (c / NST) & 1, nullptr);
    } else if (w == 3) {
        // ---------------- issuer
        constexpr uint32_t id_sp = idesc_bf16(128, C), id_o1 = idesc_bf16(128, C),
                           id_o2 = idesc_bf16(128, C, false, false, true), id_z = idesc_bf16(128, DK, false, true);
        const uint32_t tmu = __shfl_sync(0xffffffffu, tm, 0), base = __shfl_sync(0xffffffffu, smem_u32(sm), 0);
        auto scores = [&](int s) {
            const uint32_t q = base + s * F::STAGE, k = q + F::QB;
            const uint64_t qd = sdesc_k_sw128(q), kd = sdesc_k_sw128(k);
            if (elect_one()) {
#pragma unroll
                for (int i = 0; i < DK / 16; ++i) {
                    const uint32_t off = ((i / 4) * F::HALF + (i % 4) * 32) >> 4;
                    umma_f16(tmu + F::SP, qd + off, kd + off, id_sp, i > 0);
                }
                umma_commit(&sp_full);
            }
            __syncwarp();
        };
        if (!BOUNDARY && nch > 0 && mbar_wait(&full[0], 0, status)) scores(0);
        int s = 0, ph = 0;   // stage of chunk c, and the parity of its use
        for (int c = 0; c < nch; ++c) {
            const uint32_t q = base + s * F::STAGE, k = q + F::QB, v = k + F::KB;
            const int s1 = s + 1 == NST ? 0 : s + 1, ph1 = s + 1 == NST ? ph ^ 1 : ph;
            if (!mbar_wait(&full[s], ph, status)) break;
            if (!mbar_wait(&w_ready, c & 1, status)) break;
            if (c > 0 && !mbar_wait(&z_free, (c - 1) & 1, status)) break;
            tc_fence_after();
            if (elect_one()) {
                const uint64_t kd = sdesc_mn_sw128(k, F::HALF);
#pragma unroll
                for (int p = 0; p < 3; ++p)
#pragma unroll
                    for (int i = 0; i < C / 16; ++i)
                        umma_f16_ts(tmu + F::Z, tmu + F::W + 32 * p + 8 * i, kd + i * (2048 >> 4), id_z, p > 0 || i > 0);
                umma_commit(&z_full);
            }
            __syncwarp();
            if (!BOUNDARY) {
                if (c + 1 < nch) {
                    if (!mbar_wait(&full[s1], ph1, status)) break;
                    if (!mbar_wait(&sp_free, c & 1, status)) break;
                    tc_fence_after();
                    scores(s1);
                }
                if (!mbar_wait(&sb_ready, c & 1, status)) break;
                if (c > 0 && !mbar_wait(&o_free, (c - 1) & 1, status)) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t qd = sdesc_k_sw128(q);
#pragma unroll
                    for (int i = 0; i < DK / 16; ++i)
                        umma_f16_ts(tmu + F::O1, tmu + F::SB + 8 * i, qd + (((i / 4) * F::HALF + (i % 4) * 32) >> 4), id_o1,
                                    i > 0);
                    umma_commit(&sb_free);
                }
                __syncwarp();
                if (!mbar_wait(&p_ready[c & 1], (c >> 1) & 1, status)) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t vd = sdesc_mn_sw128(v, F::HALF), pd = sdesc_k_sw128(base + F::P0 + (c & 1) * F::PB);
#pragma unroll
                    for (int i = 0; i < C / 16; ++i)
                        umma_f16(tmu + F::O2, vd + i * (2048 >> 4), pd + i * (32 >> 4), id_o2, i > 0);
                    umma_commit(&o_full);
                    umma_commit(&p_free[c & 1]);
                }
                __syncwarp();
            }
            if (elect_one()) umma_commit(&empty[s]);
            __syncwarp();
            s = s1;
            ph = ph1;
        }
        if (elect_one()) umma_commit(&done);
        __syncwarp();
        mbar_wait(&done, 0, nullptr);   // no product stays in flight behind the CTA
    } else if (w < 2) {
        // ---------------- P: warp w has rows 32 w .. 32 w + 31; columns above the diagonal blocks stay zero
        if (!BOUNDARY) {
            const int row = 32 * w + lane;
            uint8_t* p0 = sm + F::P0 + row * 128;
            if (w == 0)
                for (int b = 0; b < 2; ++b)
                    for (int i = 4; i < 8; ++i)
                        *reinterpret_cast<uint4*>(p0 + b * F::PB + ((i ^ (row & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
            for (int c = 0; c < nch; ++c) {
                const int s = c % NST;
                if (!mbar_wait(&full[s], (c / NST) & 1, status)) break;
                if (!mbar_wait(&sp_full, c & 1, status)) break;
                tc_fence_after();
                const Decays& d = decays[s];
                const float gr = d.g2[row];
                if (c >= 2 && !mbar_wait(&p_free[c & 1], ((c >> 1) - 1) & 1, status)) break;
                uint8_t* p = p0 + (c & 1) * F::PB;
#pragma unroll 1
                for (int j0 = 0; j0 < 32 * (w + 1); j0 += 16) {
                    float x[16];
                    tmem_ld16(tm + F::SP + (static_cast<uint32_t>(32 * w) << 16) + j0, x);
                    tmem_wait_ld_regs<16>(x);
                    uint32_t u[8];
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        const float4 g = *reinterpret_cast<const float4*>(&d.g2[j0 + j]);
                        const int k = row - j0 - j;   // columns up to k are on or under the diagonal
                        u[j / 2] = pack_bf16x2(k >= 0 ? x[j] * ex2_approx(gr - g.x) : 0.f,
                                               k >= 1 ? x[j + 1] * ex2_approx(gr - g.y) : 0.f);
                        u[j / 2 + 1] = pack_bf16x2(k >= 2 ? x[j + 2] * ex2_approx(gr - g.z) : 0.f,
                                                   k >= 3 ? x[j + 3] * ex2_approx(gr - g.w) : 0.f);
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        *reinterpret_cast<uint4*>(p + (((j0 / 8 + i) ^ (row & 7)) << 4)) =
                            make_uint4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&sp_free);
                    mbar_arrive(&empty[s]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_ready[c & 1]);
            }
        }
    } else if (w < 8) {
        // ---------------- W and o: thread = channel of v
        const int q4 = w & 3, ch = 32 * q4 + lane, tv = t - 128;
        const bool mine = ch < DV;
        const uint32_t lanes = static_cast<uint32_t>(32 * q4) << 16;
        uint32_t off[8];   // of (row j, this channel) in an eight-row group of a swizzled half tile
#pragma unroll
        for (int j = 0; j < 8; ++j) off[j] = (ch >> 6) * F::HALF + j * 128 + ((((ch & 63) >> 3) ^ j) << 4) + (ch & 7) * 2;
        // A wait that runs out ends this warp's work, but not its part in the four warps' own barrier.
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) { ok = ok && mbar_wait(bar, parity, status); };
        auto split = [&](int c) {
            const int s = c % NST;
            wait(&full[s], (c / NST) & 1);
            uint8_t* kt = sm + s * F::STAGE + F::QB;
            uint8_t* vt = kt + F::KB;
            const int n = it.n - c * C;
            if (n < C) {
                // rows behind the sequence belong to others: they must not reach a sum, not even times zero
                for (int i = tv; ok && i < (C - n) * 8; i += 128) {
                    const int r = n + i / 8, x = r * 128 + (i & 7) * 16;
#pragma unroll
                    for (int b = 0; b < DK / 64; ++b) *reinterpret_cast<uint4*>(kt + b * F::HALF + x) = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                    for (int b = 0; b < DV / 64; ++b) *reinterpret_cast<uint4*>(vt + b * F::HALF + x) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                named_bar_sync(1, 128);
            }
            if (c > 0) wait(&z_full, (c - 1) & 1);   // W of the chunk before has been read
            if (mine && ok) {
                tc_fence_after();
                const Decays& d = decays[s];
#pragma unroll 1
                for (int b = 0; b < C; b += 16) {   // 16 tokens: 8 packed columns of each part
                    uint32_t u[3][8];
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        const float4 wt = *reinterpret_cast<const float4*>(&d.w[b + j]);
                        const float wv[4] = {wt.x, wt.y, wt.z, wt.w};
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            const int r = j + e;   // its eight-row group starts at token b + (r & 8)
                            const uint8_t* p = vt + (b + (r & 8)) * 128;
                            const uint32_t v0 = *reinterpret_cast<const unsigned short*>(p + off[r & 7]);
                            const uint32_t v1 = *reinterpret_cast<const unsigned short*>(p + off[(r + 1) & 7]);
                            float f0 = wv[e] * lo_f32(v0), f1 = wv[e + 1] * lo_f32(v1);
#pragma unroll
                            for (int k = 0; k < 3; ++k) {
                                const uint32_t x = pack_bf16x2(f0, f1);
                                u[k][r / 2] = x;
                                f0 -= lo_f32(x);
                                f1 -= hi_f32(x);
                            }
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 3; ++k) tmem_st8(tm + lanes + F::W + 32 * k + b / 2, u[k]);
                }
                tmem_wait_st();
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0 && ok) {
                mbar_arrive(&w_ready);
                if (BOUNDARY) mbar_arrive(&empty[s]);
            }
        };
        auto out = [&](int c) {
            const int s = c % NST, n = it.n - c * C;
            wait(&o_full, c & 1);
            uint8_t* ob = sm + F::O0 + (c & 1) * F::VB;
            // the store that read this buffer two chunks ago is done with it
            if (tv == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
            named_bar_sync(1, 128);
            if (mine && ok) {
                tc_fence_after();
                const Decays& d = decays[s];
#pragma unroll 1
                for (int b = 0; b < C; b += 16) {
                    float x[16], y[16];
                    tmem_ld16(tm + lanes + F::O1 + b, x);
                    tmem_ld16(tm + lanes + F::O2 + b, y);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i) asm volatile("" : "+f"(x[i]), "+f"(y[i]));
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        const float4 e = *reinterpret_cast<const float4*>(&d.eg[b + j]);
                        const float ev[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            *reinterpret_cast<__nv_bfloat16*>(ob + (b + ((j + i) & 8)) * 128 + off[(j + i) & 7]) =
                                __float2bfloat16_rn(fmaf(ev[i], x[j + i], y[j + i]));
                    }
                }
                tc_fence_before();
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && ok) {
                mbar_arrive(&o_free);
                mbar_arrive(&empty[s]);
            }
            named_bar_sync(1, 128);
            if (n >= C) {
                if (tv == 0 && ok) {
#pragma unroll
                    for (int b = 0; b < DV / 64; ++b) tma_store_2d(&mo, h * DV + 64 * b, it.t0 + c * C, ob + b * F::HALF);
                    bulk_commit();
                }
            } else {   // the rows behind the sequence are not this one's to write
                __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.o) +
                                     (static_cast<size_t>(it.t0) + c * C) * a.H * DV + static_cast<size_t>(h) * DV;
                for (int i = tv; ok && i < n * (DV / 8); i += 128) {
                    const int r = i / (DV / 8), k8 = i % (DV / 8);
                    st_global_v4(dst + static_cast<size_t>(r) * a.H * DV + 8 * k8,
                                 *reinterpret_cast<const uint4*>(ob + (k8 >> 3) * F::HALF + r * 128 + (((k8 & 7) ^ (r & 7)) << 4)));
                }
            }
        };
        for (int c = 0; c < nch; ++c) {
            split(c);
            if (!BOUNDARY && c > 0) out(c - 1);
        }
        if (!BOUNDARY && nch > 0) out(nch - 1);
        if (!BOUNDARY && tv == 0) bulk_wait0();
    } else {
        // ---------------- state: thread = channel of v, S[i] = channel i of k
        const int q4 = w & 3, ch = 32 * q4 + lane;
        const bool mine = ch < DV;
        const uint32_t lanes = static_cast<uint32_t>(32 * q4) << 16;
        float S[DK];
        const float* start = nullptr;
        if (it.seg == 0) {
            if (a.initial_state) start = a.initial_state + (static_cast<size_t>(it.seq) * a.H + h) * DK * DV;
        } else if (!BOUNDARY) {
            start = a.z + (static_cast<size_t>(it.z0 + it.seg - 1) * a.H + h) * DK * DV;
        }
#pragma unroll
        for (int i = 0; i < DK; ++i) S[i] = start && mine ? start[i * DV + ch] : 0.f;
        auto publish = [&]() {   // the bf16 copy that O1 multiplies q with
            if (mine) {
#pragma unroll
                for (int b = 0; b < DK; b += 32) {
                    uint32_t u[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) u[i] = pack_bf16x2(S[b + 2 * i], S[b + 2 * i + 1]);
                    tmem_st16u(tm + lanes + F::SB + b / 2, u);
                }
                tmem_wait_st();
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sb_ready);
        };
        auto store_state = [&](float* dst) {
            if (mine)
#pragma unroll
                for (int i = 0; i < DK; ++i) dst[i * DV + ch] = S[i];
        };
        if (!BOUNDARY && nch > 0) publish();
        for (int c = 0; c < nch; ++c) {
            const int s = c % NST;
            if (!mbar_wait(&full[s], (c / NST) & 1, status)) break;
            const float eC = decays[s].eC;
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
            if (!mbar_wait(&z_full, c & 1, status)) break;
            if (mine) {
                tc_fence_after();
#pragma unroll
                for (int b = 0; b < DK; b += 16) {
                    float z[16];
                    tmem_ld16(tm + lanes + F::Z + b, z);
                    tmem_wait_ld_regs<16>(z);
#pragma unroll
                    for (int i = 0; i < 16; ++i) S[b + i] = fmaf(eC, S[b + i], z[i]);
                }
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&z_free);
            if (!BOUNDARY && c + 1 < nch) {
                if (!mbar_wait(&sb_free, c & 1, status)) break;
                tc_fence_after();
                publish();
            }
            const int pos = it.pos + (c + 1) * C;
            if (!BOUNDARY && a.ckpt_stride && (c + 1) * C <= it.n && pos % a.ckpt_stride == 0) {
                const long long slot = static_cast<long long>(a.ckpt_cu[it.seq]) + pos / a.ckpt_stride - 1;
                if (slot >= 0 && slot < a.ckpt_cu[it.seq + 1])
                    store_state(a.checkpoints + (static_cast<size_t>(slot) * a.H + h) * DK * DV);
                else if (lane == 0)
                    set_status(status, KDA_ERR_DEVICE_INPUT);
            }
        }
        if (BOUNDARY) store_state(a.z + (static_cast<size_t>(it.z0 + it.seg) * a.H + h) * DK * DV);
        else if (a.final_state && it.seg + 1 == it.n_seg)
            store_state(a.final_state + (static_cast<size_t>(it.seq) * a.H + h) * DK * DV);
    }
    tc_fence_before();
    __syncthreads();
    if (w == 3) tmem_dealloc(tm, F::COLS);
}

// [T, cols] bf16, boxes of 64 tokens x 64 columns with the 128-byte swizzle
bool make_map(CUtensorMap* m, const void* base, long long cols, long long T) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(T)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * 2};
    const cuuint32_t box[2] = {64u, 64u}, estr[2] = {1u, 1u};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK, int DV, bool BOUNDARY>
cudaError_t launch(const LinArgs& a, cudaStream_t s) {
    using F = Cfg<DK, DV, BOUNDARY>;
    CUtensorMap mq, mk, mv, mo;
    memset(&mq, 0, sizeof(mq));
    memset(&mk, 0, sizeof(mk));
    memset(&mv, 0, sizeof(mv));
    memset(&mo, 0, sizeof(mo));
    if (a.total_tokens > 0) {   // without tokens no tile is loaded or stored
        const long long cq = static_cast<long long>(a.Hqk) * DK, cv = static_cast<long long>(a.H) * DV;
        if (!make_map(&mq, a.q, cq, a.total_tokens) || !make_map(&mk, a.k, cq, a.total_tokens) ||
            !make_map(&mv, a.v, cv, a.total_tokens) || !make_map(&mo, a.o, cv, a.total_tokens))
            return cudaErrorInvalidValue;
    }
    const int smem = static_cast<int>(F::BYTES) + 1024;
    cudaError_t e = cudaFuncSetAttribute(lin_bf16_kernel<DK, DV, BOUNDARY>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.max_items * a.H));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, lin_bf16_kernel<DK, DV, BOUNDARY>, a, mq, mk, mv, mo);
}

template <int DK, int DV>
cudaError_t launch_b(const LinArgs& a, bool boundary_pass, cudaStream_t s) {
    return boundary_pass ? launch<DK, DV, true>(a, s) : launch<DK, DV, false>(a, s);
}

}  // namespace

cudaError_t launch_lin_bf16(const LinArgs& a, bool boundary_pass, cudaStream_t s) {
    if (a.dk == 64) return a.dv == 64 ? launch_b<64, 64>(a, boundary_pass, s) : launch_b<64, 128>(a, boundary_pass, s);
    return a.dv == 64 ? launch_b<128, 64>(a, boundary_pass, s) : launch_b<128, 128>(a, boundary_pass, s);
}

}  // namespace kda
