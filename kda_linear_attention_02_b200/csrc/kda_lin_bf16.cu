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
// tensor memory as O1's A operand, in the lane layout the registers already have, and W is an A operand there
// too.  What reaches o is rounded once in each path (P, and the copy of S).  What reaches the state is not: k
// and v are bf16 already, and W goes in as four bf16 parts that add up to w v to 24 bits, so Z is an fp32 sum
// of exact products.  With w = w1 + w2 + w3 in bf16 parts, packed bf16 FMAs give them two tokens at a time,
//     h = rn(w1 v),  -e = h - w1 v (exact: eight bits are left),  m = rn(w2 v),  -l = rn((m - w2 v) - w3 v),
// five instructions a pair (splitting the fp32 products w v takes seventeen); the MMAs negate -e and -l.  Z starts from zero in every chunk and joins S by one rounded FMA: an
// accumulator that lived on in tensor memory would collect the truncation of its additions over the length of
// the sequence.
//
// The warps are specialised and meet at mbarriers: a producer (TMA tiles of q, k, v, and the chunk's decays),
// an issuer (all MMAs, in an order that keeps Z of one chunk ahead of the scores of the next), two warps for
// P, eight that split W and write o, four that hold the state.
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
    static constexpr int ZN = DK;   // channels of k that one piece of Z has
    // tensor memory columns
    static constexpr uint32_t SP = 0, O1 = 64, O2 = 128, Z = 192, SB = 320, W = 384, COLS = 512;   // W: 4 x 32
    static_assert(BYTES + 1024 + 4096 <= 227 * 1024, "shared memory");
};
constexpr int kThreads = 512;
constexpr int kPWarps = 2, kVWarps = 8, kSWarps = 4;
// Registers of a thread: 128 at launch; the warps that hold the state take 176, the others give theirs
// (3 x 112 + 176 = 512, what four threads of the four groups were launched with).
constexpr int kRegsState = 176, kRegsOther = 112;

struct Decays {            // of one chunk
    float g2[kChunk];      // g_t log2(e)
    float eg[kChunk];      // e^{g_t}
    uint4 w[kChunk / 2];   // of tokens 2 i, 2 i + 1: the bf16 parts w1, w2, -w3 of e^{g_C - g_t}, packed pairs
    float m[kChunk / 2];   // e^{g_32 - g_t} of the chunk's first half
    float g2m;             // g_32 log2(e)
    float eC;              // e^{g_C}
    float pad[2];
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

// 32 consecutive columns of this warp's lanes
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&r)[32]) {
    uint32_t* u = reinterpret_cast<uint32_t*>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
          "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
          "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
          "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t (&v)[16]) {
    tmem_st16(taddr, reinterpret_cast<const float(&)[16]>(v));
}

// packed bf16 a b + c, one rounding
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
// 16 lanes x 32 columns of 32 bits, four columns a block: thread t has, of block b, column t % 4 of lanes t / 4
// (register 2 b) and t / 4 + 8 (2 b + 1).  For packed pairs of a K-adjacent operand this is the fragment that a
// transposed matrix load gives: rows = channels, columns = pairs of tokens.
__device__ __forceinline__ void tmem_st_16x128b_x4(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
// The accumulator fragment (see tmem_ld_16x256b_x2) of four blocks of 8 columns.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, float* r) {
    uint32_t* u = reinterpret_cast<uint32_t*>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
          "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
        : "r"(taddr));
}

// mbar_wait in few instructions, since the roles' code together has to fit the SM's instruction caches: polls
// that let the warp sleep (the polls of a tight loop were a quarter of all instructions issued), bounded by their
// number, at most about two seconds; the caller records a wait that ran out.
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity) {
    const uint32_t addr = smem_u32(bar);
#pragma unroll 1
    for (int i = 0; i < (1 << 20); ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(addr), "r"(parity), "r"(2000u)   // up to two microseconds
            : "memory");
        if (ok) return true;
    }
    return false;
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
    __shared__ __align__(8) uint64_t full[NST], empty[NST], sp_full, sp_free, p_ready[2], p_free[2], w_ready, z_full[2],
        z_free[2], sb_ready, sb_free, o_full, o_free, done;
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
            mbar_init(&z_full[b], 1);
            mbar_init(&z_free[b], kSWarps);
        }
        mbar_init(&w_ready, kVWarps);
        mbar_init(&sb_ready, kSWarps);
        mbar_init(&sb_free, 1);
        mbar_init(&o_full, 1);
        mbar_init(&o_free, kVWarps);
        mbar_init(&done, 1);
        fence_barrier_init();
    }
    grid_launch_dependents();
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
    bool ok = true;   // no wait of this warp has run out

    if (w < 4) {
        // every warp of a group of four changes its registers by the same instruction
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
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
                if (!(ok = bar_wait(&empty[s], ((c / NST) & 1) ^ 1))) break;
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
                const float g0 = before + x0, g1 = f, gm = __shfl_sync(0xffffffffu, f, 15);
                *reinterpret_cast<float2*>(&d.g2[2 * lane]) = make_float2(g0 * kLog2e, g1 * kLog2e);
                *reinterpret_cast<float2*>(&d.eg[2 * lane]) = make_float2(expf(g0), expf(g1));
                float w0 = expf(after + x1), w1 = expf(after);
                uint32_t part[3];
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    part[k] = pack_bf16x2(w0, w1);
                    w0 -= lo_f32(part[k]);
                    w1 -= hi_f32(part[k]);
                }
                d.w[lane] = make_uint4(part[0], part[1], part[2] ^ 0x80008000u, 0u);
                if (lane < 16) *reinterpret_cast<float2*>(&d.m[2 * lane]) = make_float2(expf(gm - g0), expf(gm - g1));
                if (lane == 0) {
                    d.g2m = gm * kLog2e;
                    d.eC = expf(sum);
                }
                total += sum;
                x0 = y0;
                x1 = y1;
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[s]);
            }
            if (BOUNDARY && lane == 0) a.zdecay[static_cast<size_t>(it.z0 + it.seg) * a.H + h] = expf(total);
            // no copy stays in flight behind the CTA: wait (bounded, quietly) for the last fill of every stage
    #pragma unroll 1
        for (int c = issued > NST ? issued - NST : 0; c < issued; ++c) bar_wait(&full[c % NST], (c / NST) & 1);
        } else if (w == 3) {
            // ---------------- issuer
            constexpr uint32_t id_sp = idesc_bf16(128, C), id_o1 = idesc_bf16(128, C),
                               id_o2 = idesc_bf16(128, C, false, false, true), id_z = idesc_bf16(128, F::ZN, false, true),
                               id_zn = idesc_bf16(128, F::ZN, true, true);
            const uint32_t tmu = __shfl_sync(0xffffffffu, tm, 0), base = __shfl_sync(0xffffffffu, smem_u32(sm), 0);
            auto scores = [&](int s) {
                const uint32_t q = base + s * F::STAGE, k = q + F::QB;
                const uint64_t qd = sdesc_k_sw128(q), kd = sdesc_k_sw128(k);
                if (elect_one()) {
#pragma unroll 1
                    for (int b = 0; b < DK / 64; ++b)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t off = (b * F::HALF + i * 32) >> 4;
                            umma_f16(tmu + F::SP, qd + off, kd + off, id_sp, b + i > 0);
                        }
                    umma_commit(&sp_full);
                }
                __syncwarp();
            };
            if (!BOUNDARY && nch > 0 && (ok = bar_wait(&full[0], 0))) scores(0);
            int s = 0, ph = 0;   // stage of chunk c, and the parity of its use
            for (int c = 0; c < nch; ++c) {
                const uint32_t q = base + s * F::STAGE, k = q + F::QB, v = k + F::KB;
                const int s1 = s + 1 == NST ? 0 : s + 1, ph1 = s + 1 == NST ? ph ^ 1 : ph;
                if (!(ok = bar_wait(&full[s], ph))) break;
                if (!(ok = bar_wait(&w_ready, c & 1))) break;
                tc_fence_after();
                // 64 channels of k at a time, so that the state warps read one half while the other is formed
#pragma unroll
                for (int z = 0; z < DK / F::ZN; ++z) {
                    if (c > 0) ok = ok && bar_wait(&z_free[z], (c - 1) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
                        const uint64_t kd = sdesc_mn_sw128(k + z * (F::ZN / 64) * F::HALF, F::HALF);
#pragma unroll 1
                        for (int p = 0; p < 4; ++p)
#pragma unroll
                            for (int i = 0; i < C / 16; ++i)
                                umma_f16_ts(tmu + F::Z + F::ZN * z, tmu + F::W + 32 * p + 8 * i, kd + i * (2048 >> 4),
                                            p & 1 ? id_zn : id_z, p > 0 || i > 0);
                        umma_commit(&z_full[z]);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (!BOUNDARY) {
                    if (c + 1 < nch) {
                        if (!(ok = bar_wait(&full[s1], ph1))) break;
                        if (!(ok = bar_wait(&sp_free, c & 1))) break;
                        tc_fence_after();
                        scores(s1);
                    }
                    if (!(ok = bar_wait(&sb_ready, c & 1))) break;
                    if (c > 0 && !(ok = bar_wait(&o_free, (c - 1) & 1))) break;
                    tc_fence_after();
                    if (elect_one()) {
                        const uint64_t qd = sdesc_k_sw128(q);
#pragma unroll 1
                        for (int b = 0; b < DK / 64; ++b)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                umma_f16_ts(tmu + F::O1, tmu + F::SB + 32 * b + 8 * i, qd + ((b * F::HALF + i * 32) >> 4), id_o1,
                                            b + i > 0);
                        umma_commit(&sb_free);
                    }
                    __syncwarp();
                    if (!(ok = bar_wait(&p_ready[c & 1], (c >> 1) & 1))) break;
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
            bar_wait(&done, 0);   // no product stays in flight behind the CTA
        } else {
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
                    if (!(ok = bar_wait(&full[s], (c / NST) & 1))) break;
                    if (!(ok = bar_wait(&sp_full, c & 1))) break;
                    tc_fence_after();
                    const Decays& d = decays[s];
                    const float gr = d.g2[row];
                    const uint32_t at = tm + F::SP + (static_cast<uint32_t>(32 * w) << 16);
                    float x[2][32];
                    if (w == 1) tmem_ld32(at, x[1]);
                    tmem_ld32(at + 32 * w, x[0]);
                    if (w == 1) tmem_wait_ld_regs<32>(x[1]);
                    tmem_wait_ld_regs<32>(x[0]);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sp_free);
                    if (c >= 2 && !(ok = bar_wait(&p_free[c & 1], ((c >> 1) - 1) & 1))) break;
                    uint8_t* p = p0 + (c & 1) * F::PB;
                    auto put = [&](int j0, const uint32_t (&u)[16]) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            *reinterpret_cast<uint4*>(p + (((j0 / 8 + i) ^ (row & 7)) << 4)) =
                                make_uint4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
                    };
                    uint32_t u[16];
                    if (w == 1) {
                        // left of the diagonal block the factor is a product of two, each at most 1, about g_32
                        const float er = ex2_approx(gr - d.g2m);
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            const float4 m = *reinterpret_cast<const float4*>(&d.m[j]);
                            u[j / 2] = pack_bf16x2(x[1][j] * (er * m.x), x[1][j + 1] * (er * m.y));
                            u[j / 2 + 1] = pack_bf16x2(x[1][j + 2] * (er * m.z), x[1][j + 3] * (er * m.w));
                        }
                        put(0, u);
                    }
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 g = *reinterpret_cast<const float4*>(&d.g2[32 * w + j]);
                        u[j / 2] = pack_bf16x2(j <= lane ? x[0][j] * ex2_approx(gr - g.x) : 0.f,
                                               j + 1 <= lane ? x[0][j + 1] * ex2_approx(gr - g.y) : 0.f);
                        u[j / 2 + 1] = pack_bf16x2(j + 2 <= lane ? x[0][j + 2] * ex2_approx(gr - g.z) : 0.f,
                                                   j + 3 <= lane ? x[0][j + 3] * ex2_approx(gr - g.w) : 0.f);
                    }
                    put(32 * w, u);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&empty[s]);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_ready[c & 1]);
                }
            }
        }
    } else if (w < 12) {
        // ---------------- W and o: thread = channel of v, and one half of the chunk's tokens
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        const int q4 = w & 3, ch = 32 * q4 + lane, tv = t - 128, half = (w - 4) / 4 * (C / 2);
        constexpr int NV = 32 * kVWarps;
        const bool mine = ch < DV;
        const uint32_t lanes = static_cast<uint32_t>(32 * q4) << 16;
        // Of a 16-token x 16-channel tile (tokens t0.., channels 32 q4 + 16 lh ..) as four 8 x 8 matrices, channels
        // first: the row that this lane addresses, in a swizzled 64-channel half tile.
        auto tile_row = [&](int t0, int lh) {
            const int tok = t0 + ((lane >> 4) << 3) + (lane & 7), c8 = 32 * q4 + 16 * lh + (lane & 8);
            return (c8 >> 6) * F::HALF + tok * 128 + ((((c8 & 63) >> 3) ^ (tok & 7)) << 4);
        };
        // A wait that runs out ends this warp's work, but not its part in the four warps' own barrier.
        auto wait = [&](uint64_t* bar, uint32_t parity) { ok = ok && bar_wait(bar, parity); };
        auto split = [&](int c) {
            const int s = c % NST;
            wait(&full[s], (c / NST) & 1);
            uint8_t* kt = sm + s * F::STAGE + F::QB;
            uint8_t* vt = kt + F::KB;
            const int n = it.n - c * C;
            if (n < C) {
                // rows behind the sequence belong to others: they must not reach a sum, not even times zero
#pragma unroll 1
                for (int i = tv; ok && i < (C - n) * 8; i += NV) {
                    const int r = n + i / 8, x = r * 128 + (i & 7) * 16;
#pragma unroll
                    for (int b = 0; b < DK / 64; ++b) *reinterpret_cast<uint4*>(kt + b * F::HALF + x) = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                    for (int b = 0; b < DV / 64; ++b) *reinterpret_cast<uint4*>(vt + b * F::HALF + x) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                named_bar_sync(1, NV);
            }
            uint32_t u[2][4][8];
            if (mine && ok) {
                const Decays& d = decays[s];
                uint4 wt[4];   // of this thread's token pair in each block of eight: w1, w2, -w3
#pragma unroll
                for (int b = 0; b < 4; ++b) wt[b] = d.w[half / 2 + 4 * b + (lane & 3)];
#pragma unroll
                for (int lh = 0; lh < 2; ++lh) {
                    uint32_t v[2][4];
                    ldsm_x4_trans(smem_u32(vt) + tile_row(half, lh), v[0]);
                    ldsm_x4_trans(smem_u32(vt) + tile_row(half + 16, lh), v[1]);
#pragma unroll
                    for (int r = 0; r < 8; ++r) {   // block r / 2, channels 8 (r % 2) + lane / 4 of the sixteen
                        const uint32_t x = v[r >> 2][r & 3];
                        const uint4 wb = wt[r >> 1];
                        u[lh][0][r] = fma_bf16x2(x, wb.x, 0x80008000u);
                        u[lh][1][r] = fma_bf16x2(x, wb.x ^ 0x80008000u, u[lh][0][r]);
                        u[lh][2][r] = fma_bf16x2(x, wb.y, 0x80008000u);
                        u[lh][3][r] = fma_bf16x2(x, wb.z, fma_bf16x2(x, wb.y ^ 0x80008000u, u[lh][2][r]));
                    }
                }
            }
            if (c > 0) wait(&z_full[DK / F::ZN - 1], (c - 1) & 1);   // W of the chunk before has been read
            if (mine && ok) {
                tc_fence_after();
#pragma unroll
                for (int lh = 0; lh < 2; ++lh)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tmem_st_16x128b_x4(tm + lanes + (static_cast<uint32_t>(16 * lh) << 16) + F::W + 32 * k + half / 2, u[lh][k]);
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
            named_bar_sync(1, NV);
            if (mine && ok) {
                tc_fence_after();
                const Decays& d = decays[s];
                float x[2][16], y[2][16];
#pragma unroll
                for (int lh = 0; lh < 2; ++lh) {
                    const uint32_t at = tm + lanes + (static_cast<uint32_t>(16 * lh) << 16) + half;
                    tmem_ld_16x256b_x4(at + F::O1, x[lh]);
                    tmem_ld_16x256b_x4(at + F::O2, y[lh]);
                }
                float2 e[4];
#pragma unroll
                for (int b = 0; b < 4; ++b) e[b] = *reinterpret_cast<const float2*>(&d.eg[half + 8 * b + 2 * (lane & 3)]);
#pragma unroll
                for (int lh = 0; lh < 2; ++lh) {
                    tmem_wait_ld_regs<16>(x[lh]);
                    tmem_wait_ld_regs<16>(y[lh]);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t u[4];
#pragma unroll
                        for (int r = 0; r < 4; ++r) {   // block 2 i + r / 2, channels 8 (r % 2) + lane / 4
                            const int k = 8 * i + 2 * r;
                            const float2 eb = e[2 * i + (r >> 1)];
                            u[r] = pack_bf16x2(fmaf(eb.x, x[lh][k], y[lh][k]), fmaf(eb.y, x[lh][k + 1], y[lh][k + 1]));
                        }
                        stsm_x4_trans(smem_u32(ob) + tile_row(half + 16 * i, lh), u);
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
            named_bar_sync(1, NV);
            if (n >= C) {
                if (tv == 0 && ok) {
#pragma unroll
                    for (int b = 0; b < DV / 64; ++b) tma_store_2d(&mo, h * DV + 64 * b, it.t0 + c * C, ob + b * F::HALF);
                    bulk_commit();
                }
            } else {   // the rows behind the sequence are not this one's to write
                __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.o) +
                                     (static_cast<size_t>(it.t0) + c * C) * a.H * DV + static_cast<size_t>(h) * DV;
#pragma unroll 1
                for (int i = tv; ok && i < n * (DV / 8); i += NV) {
                    const int r = i / (DV / 8), k8 = i % (DV / 8);
                    st_global_v4(dst + static_cast<size_t>(r) * a.H * DV + 8 * k8,
                                 *reinterpret_cast<const uint4*>(ob + (k8 >> 3) * F::HALF + r * 128 + (((k8 & 7) ^ (r & 7)) << 4)));
                }
            }
        };
        for (int c = 0; c <= nch; ++c) {
            if (c < nch) split(c);
            if (!BOUNDARY && c > 0) out(c - 1);
        }
        if (!BOUNDARY && tv == 0) bulk_wait0();
    } else {
        // ---------------- state: thread = channel of v, S[i] = channel i of k
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsState));
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
        float* end = nullptr;
        if (BOUNDARY) end = a.z + (static_cast<size_t>(it.z0 + it.seg) * a.H + h) * DK * DV;
        else if (a.final_state && it.seg + 1 == it.n_seg)
            end = a.final_state + (static_cast<size_t>(it.seq) * a.H + h) * DK * DV;
        if (nch == 0 && end && mine)   // no tokens: the state stays as it was
#pragma unroll 1
            for (int i = 0; i < DK; ++i) end[i * DV + ch] = start ? start[i * DV + ch] : 0.f;
        for (int c = 0; c < nch; ++c) {
            const int s = c % NST;
            if (!BOUNDARY) {
                if (c > 0 && !(ok = bar_wait(&sb_free, (c - 1) & 1))) break;   // the copy of the chunk before has been read
                tc_fence_after();
                publish();
            }
            if (!(ok = bar_wait(&full[s], (c / NST) & 1))) break;
            const float eC = decays[s].eC;
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
#pragma unroll
            for (int zh = 0; zh < DK / F::ZN; ++zh) {
                ok = ok && bar_wait(&z_full[zh], c & 1);
                if (!ok) break;
                if (mine) {
                    tc_fence_after();
#pragma unroll
                    for (int b = F::ZN * zh; b < F::ZN * (zh + 1); b += 32) {
                        float z[32];
                        tmem_ld32(tm + lanes + F::Z + b, z);
                        tmem_wait_ld_regs<32>(z);
#pragma unroll
                        for (int i = 0; i < 32; ++i) S[b + i] = fmaf(eC, S[b + i], z[i]);
                    }
                    tc_fence_before();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&z_free[zh]);
            }
            if (!ok) break;
            // a checkpoint, and the state at the segment's end
            float* dst = nullptr;
            const int pos = it.pos + (c + 1) * C;
            if (!BOUNDARY && a.ckpt_stride && (c + 1) * C <= it.n && pos % a.ckpt_stride == 0) {
                const long long slot = static_cast<long long>(a.ckpt_cu[it.seq]) + pos / a.ckpt_stride - 1;
                if (slot >= 0 && slot < a.ckpt_cu[it.seq + 1])
                    dst = a.checkpoints + (static_cast<size_t>(slot) * a.H + h) * DK * DV;
                else if (lane == 0)
                    set_status(a.status, KDA_ERR_DEVICE_INPUT);
            }
            if (mine && (dst || (end && c + 1 == nch))) {
#pragma unroll 1
                for (int k = 0; k < 2; ++k) {
                    float* p = k == 0 ? dst : c + 1 == nch ? end : nullptr;
                    if (p)
#pragma unroll
                        for (int i = 0; i < DK; ++i) p[i * DV + ch] = S[i];
                }
            }
        }
    }
    if (!ok && lane == 0) set_status(a.status, KDA_ERR_TIMEOUT);
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
