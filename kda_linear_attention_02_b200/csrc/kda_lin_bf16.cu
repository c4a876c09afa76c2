// kda_lin_bf16.cu -- decayed linear attention, chunked form, bf16 on the 5th-generation tensor cores.
//
// One CTA walks a segment of one (sequence, head) in chunks of 64 tokens.  With g_t the sum of log_alpha over
// tokens 1..t of the chunk, all products are written transposed, channels of v in the accumulator's lanes:
//
//     scores   s_tj = q_t . k_j                                   (SP, tokens t in lanes)
//     P_tj     = e^{g_t - g_j} s_tj  (j <= t), in two bf16 parts
//     o_t      = e^{g_t} (S^T q_t)  +  sum_j P_tj v_j             (O1 = Sb Q^T, O2 = V^T P^T)
//     S^T     <- e^{g_C} S^T + sum_j (e^{g_C - g_j} v_j) k_j^T    (Z = W K, W_j = e^{g_C - g_j} v_j)
//
// S^T stays in fp32 registers (thread = channel of v, register = channel of k); its bf16 copy Sb goes to tensor
// memory as O1's A operand, in the lane layout the registers already have, and W is an A operand there too.  On the
// way to o the copy of S is rounded once, channel by channel, and such errors average out over the sum: o is off by
// 0.0018 to 0.0021 of its norm, 0.0017 of it o's own rounding.  (With a second part of the copy that is all of it,
// but tensor memory has room for both parts of 64 channels at a time: 4 x 4096 x 32 heads 157 -> 198 us, 32768 x 32
// heads 411 -> 489 us.)  P's would not: one P_tj weighs all of v_j, so with a single bf16 part an output that one
// token dominates would be off by up to 2^-8 in every channel; a second part leaves 2^-16 and costs 2 % of the
// time.  For the same 16 bits the exponents g_t - g_j are differences of numbers in two parts (Log2, below), 1 to 4
// % of the time.  What reaches the state is not rounded: k and v are bf16 already, and W goes in as four bf16 parts
// that add up to w v to 24 bits, so Z is an fp32 sum of exact products.  With w = w1 + w2 + w3 in bf16 parts,
// packed bf16 FMAs give them two tokens at a time,
//     h = rn(w1 v),  -e = h - w1 v (exact: eight bits are left),  m = rn(w2 v),  -l = rn((m - w2 v) - w3 v),
// five instructions a pair (splitting the fp32 products w v takes seventeen); the MMAs negate -e and
// -l.  Z starts from zero in every chunk and joins S by one rounded FMA: an accumulator that lived on in tensor
// memory would collect the truncation of its additions over the length of the sequence.
//
// The grid has a CTA per SM; each takes (segment, head) pairs from a counter, longest first, until none is left,
// and its copies run ahead into the next pair while the last chunks of one are worked on.
//
// The warps are specialised and meet at mbarriers: a producer (TMA tiles of q, k, v, and the chunk's decays),
// an issuer (all MMAs, in an order that keeps Z of one chunk ahead of the scores of the next), two warps for
// P, four that split W, four that write o, four that hold the state.
//
// What bounds it (4 x 4096 tokens x 32 heads of 128, 614 MB): 147-160 us = 3.8-4.2 TB/s, 135 us of it this kernel.  A
// chunk takes 2900 cycles: the products about 2050 of the tensor pipe (57 % busy), with shared memory and W's warps
// close behind.  M = 128 for the channels of v leaves one product shape for all sizes of dv; chunks of 64 keep P at
// one N = 64 operand, and three 48 KB stages beside it in shared memory.  Before: bf16 P in one part 147 us, W as
// three parts of the fp32 products 201 us, fp32 units 4840 us.
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
    // Decays outlive their chunk's tiles, and are written before the stage is free: when those of chunk c are, the
    // products of chunk c - 1 - NST are known to be done, so that o of chunk c - 2 - NST has been written (and in the
    // boundary pass Z of it taken).
    static constexpr int ND = NST + 2;
    static constexpr uint32_t PB = C * 128;                          // P: 64 rows of 64 bf16
    static constexpr uint32_t P0 = NST * STAGE, O0 = P0 + (BOUNDARY ? 0 : 4 * PB);   // two places of two parts
    // the A operands of 128 rows read past 64-row tiles (their results are not used): the tiles behind exist
    static constexpr uint32_t BYTES = O0 + (BOUNDARY ? HALF : 2 * VB);
    // tensor memory columns
    // (W: 4 x 32; the boundary pass has room for Z twice: chunk c uses place c % NZ)
    static constexpr uint32_t SP = 0, O1 = 64, O2 = 128, SB = 320, W = 384, COLS = 512;
    static constexpr int NZ = BOUNDARY ? 2 : 1;
    static constexpr uint32_t Z = BOUNDARY ? 0 : 192;
};
constexpr int kThreads = 512;
constexpr int kPWarps = 2, kWWarps = 4, kOWarps = 4, kSWarps = 4;
// Registers of a thread: 128 at launch; the warps that hold the state take 176, the others give theirs
// (3 x 112 + 176 = 512, what four threads of the four groups were launched with).
constexpr int kRegsState = 176, kRegsOther = 112;

struct __align__(16) Job {   // a segment of one (sequence, head)
    LinItem it;
    int h;   // -1: there are no more
    int pad[3];
};

struct Decays {            // of one chunk
    float g2[kChunk];      // g_t log2(e), as two numbers (see Log2)
    float g2l[kChunk];
    float eg[kChunk];      // e^{g_t}
    uint4 w[kChunk / 2];   // of tokens 2 i, 2 i + 1: the bf16 parts w1, w2, -w3 of e^{g_C - g_t}, packed pairs
    float m[kChunk / 2];   // e^{g_32 - g_t} of the chunk's first half
    float g2m, g2ml;       // g_32 log2(e), likewise
    float eC;              // e^{g_C}
    float pad;
};

// fp32 pair -> packed bf16 pair, and back
__device__ __forceinline__ float lo_f32(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f32(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// MMAs for a whole converged warp, issued by its elected lane, with warp-uniform operands.  Issued by a lane
// chosen with threadIdx, from values the compiler cannot see to be uniform, each costs about 96 cycles; so, 32 to
// 64 (M = 128, K = 16, N = 64 to 128).
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Two products with the same A, one behind the other: the first leaves A in the collector buffer for the second.
__device__ __forceinline__ void mma_ss_keep(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16.collector::a::fill [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
        "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_ss_kept(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16.collector::a::lastuse [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
        "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Commits what the elected lane has issued.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
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

// mbar_wait in few instructions, since the roles' code together has to fit the SM's instruction cache: polls that
// let the warp sleep (two microseconds each, measured), bounded by their number, so about two seconds; the caller
// records a wait that ran out.
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\tmov.u32 n, 0;\n"
        "POLL:\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t@p bra DONE;\n\t"
        "add.u32 n, n, 1;\n\tsetp.lt.u32 q, n, 1048576;\n\t@q bra POLL;\n"
        "DONE:\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// One arrival for the warp, once all its lanes are here.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, bool yes = true) {
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 st;\n\tsetp.ne.u32 p, %1, 0;\n\t@p mbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" ::"r"(
            smem_u32(bar)),
        "r"(static_cast<uint32_t>(yes && (threadIdx.x & 31) == 0))
        : "memory");
}

// 4 bytes global -> shared by an asynchronous copy, zero when not `valid` (nothing is read then)
__device__ __forceinline__ void cp_async4(uint32_t dst, const float* src, bool valid) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(valid ? 4 : 0) : "memory");
}

// A logarithm to base 2 as h + l, h a multiple of 2^-10, |l| about 2^-11 at most for one token.  What counts are
// differences of a chunk's sums, and a token that forgets everything moves all later sums by 173: as plain fp32
// numbers, forty of them would leave the differences behind them 10 bits.  The sums of h (below 2^14) are exact in
// fp32, in any order, and those of l, below 2^-4, off by less than 2^-26, so that a difference is rounded once.
struct Log2 {
    float h, l;
};
__device__ __forceinline__ Log2 operator+(Log2 a, Log2 b) { return {a.h + b.h, a.l + b.l}; }
__device__ __forceinline__ Log2 operator-(Log2 a, Log2 b) { return {a.h - b.h, a.l - b.l}; }
__device__ __forceinline__ Log2 log2_of(float x) {   // of e^x
    const float y = x * kLog2e, r = fmaf(x, kLog2e, -y) + x * 1.9259629e-8f;   // log2(e) - kLog2e
    const float h = __fadd_rn(__fadd_rn(y, 12288.f), -12288.f);                // ulp(12288 - 174) = 2^-10
    return {h, (y - h) + r};
}
// 2^(h + l) to about one unit in the last place: the rounding of the sum is put back.
__device__ __forceinline__ float exp2_of(Log2 x) {
    const float y = x.h + x.l, r = (x.h - y) + x.l, e = ex2_approx(y);
    return fmaf(e, r * 0.69314718f, e);
}

// One warp's walk over the log_alpha of a segment: the decays of its chunks, in order.  Lane i has tokens 2 i and
// 2 i + 1 of a chunk, and fetches theirs three chunks ahead (a load takes longer than a chunk), to shared memory,
// since moving a value on in registers would wait for its load.
// FULL: and what o needs of them.
template <bool FULL>
struct DecayWalk {
    const float* la;
    const float* any;      // a valid address for copies that read nothing
    int la_t, n, left, lane;
    float* ring;           // this lane's pair in the first of four slots of kChunk
    Log2 total;            // sum over the chunks so far

    __device__ __forceinline__ void fetch(int c) {
        const uint32_t at = smem_u32(ring + (c & 3) * kChunk);
        cp_async4(at, left > 0 ? la : any, left > 0);
        cp_async4(at + 4, left > 1 ? la + la_t : any, left > 1);
        asm volatile("cp.async.commit_group;" ::: "memory");
        la += kChunk * static_cast<size_t>(la_t);
        left -= kChunk;
    }
    __device__ __forceinline__ void start(const LinArgs& a, const LinItem& it, int h, float* slots) {
        lane = threadIdx.x & 31;
        cp_async_wait_all();   // before the ring is filled anew
        any = a.la;
        la_t = a.la_t;
        la = a.la + (static_cast<size_t>(it.t0) + 2 * lane) * la_t + h;
        n = it.n;
        left = n - 2 * lane;
        ring = slots + 2 * lane;
        total = {0.f, 0.f};
        if (n > 0)
#pragma unroll 1
            for (int c = 0; c < 3; ++c) fetch(c);
    }
    __device__ __forceinline__ void chunk(int c, Decays& d) {
        fetch(c + 3);
        asm volatile("cp.async.wait_group 3;" ::: "memory");
        const float2 x = *reinterpret_cast<const float2*>(ring + (c & 3) * kChunk);
        const bool in0 = c * kChunk + 2 * lane < n, in1 = c * kChunk + 2 * lane + 1 < n;
        const Log2 x0 = log2_of(in0 ? fmaxf(x.x, kLinLogMin) : 0.f), x1 = log2_of(in1 ? fmaxf(x.y, kLinLogMin) : 0.f);
        Log2 f = x0 + x1;   // inclusive sums of the lanes' pairs
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const Log2 u = {__shfl_up_sync(0xffffffffu, f.h, off), __shfl_up_sync(0xffffffffu, f.l, off)};
            if (lane >= off) f = f + u;
        }
        auto of_lane = [&](int i) { return Log2{__shfl_sync(0xffffffffu, f.h, i), __shfl_sync(0xffffffffu, f.l, i)}; };
        const Log2 sum = of_lane(31), g0 = f - x1;
        float w0 = exp2_of(sum - g0), w1 = exp2_of(sum - f);
        if (FULL) {
            const Log2 gm = of_lane(15);
            *reinterpret_cast<float2*>(&d.g2[2 * lane]) = make_float2(g0.h, f.h);
            *reinterpret_cast<float2*>(&d.g2l[2 * lane]) = make_float2(g0.l, f.l);
            *reinterpret_cast<float2*>(&d.eg[2 * lane]) = make_float2(exp2_of(g0), exp2_of(f));
            if (lane < 16) {
                const Log2 m0 = gm - g0, m1 = gm - f;
                *reinterpret_cast<float2*>(&d.m[2 * lane]) = make_float2(ex2_approx(m0.h + m0.l), ex2_approx(m1.h + m1.l));
            }
            if (lane == 0) {
                d.g2m = gm.h;
                d.g2ml = gm.l;
            }
        }
        if (lane == 0) d.eC = exp2_of(sum);
        uint32_t part[3];
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            part[p] = pack_bf16x2(w0, w1);
            w0 -= lo_f32(part[p]);
            w1 -= hi_f32(part[p]);
        }
        d.w[lane] = make_uint4(part[0], part[1], part[2] ^ 0x80008000u, 0u);
        total = total + sum;
    }
};

template <int DK, int DV, bool BOUNDARY>
__global__ void __launch_bounds__(kThreads, 1)
lin_bf16_kernel(const LinArgs a, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo) {
    using F = Cfg<DK, DV, BOUNDARY>;
    constexpr int NST = F::NST, C = F::C;
    static_assert(F::BYTES + 1024 + F::ND * sizeof(Decays) + 2048 <= 227 * 1024, "shared memory, with 2 KB for barriers, pairs and the ring");
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ Decays decays[F::ND];
    __shared__ __align__(8) float la_ring[4 * C];
    __shared__ __align__(8) uint64_t full[NST], empty[NST], sp_full, sp_free, w_go[2], w_free, z_free[2],
        z_full[2], o_go[2], o_full[2], done, job_full[2], job_free[2], w_sync, o_sync;
    __shared__ Job jobs[2];
    __shared__ uint32_t tmem_slot;
    const int t = threadIdx.x, w = __shfl_sync(0xffffffffu, t >> 5, 0), lane = t & 31;
    if (t == 0) {
        for (int s = 0; s < NST; ++s) {
            mbar_init(&full[s], 2);
            // the chunk's last product is done, and with it all that read its tiles (in the boundary pass nothing of a
            // chunk waits for the state warps, which therefore say themselves that they have seen the filling)
            mbar_init(&empty[s], 1 + (BOUNDARY ? kSWarps : 0));
        }
        mbar_init(&sp_full, 1);
        mbar_init(&sp_free, kPWarps);
        // The issuer's waits and commits are what a chunk's time is made of, so there are few.
        for (int b = 0; b < 2; ++b) {
            // the tokens' half of W is in place (b = 0 of the full pass: and Z of the chunk before has been read)
            mbar_init(&w_go[b], kWWarps + (BOUNDARY || b ? 0 : kSWarps));
            mbar_init(&z_free[b], kSWarps);   // boundary pass
            mbar_init(&z_full[b], 1);         // Z is there, and W's second half free again
            // Sb and P are in place, and O1, O2 of the chunk before have been read
            mbar_init(&o_go[b], kOWarps + kSWarps + kPWarps);
            mbar_init(&o_full[b], 1);         // O1 and O2 are there, and Sb and this P free again
        }
        mbar_init(&w_free, 1);                // W's first half
        mbar_init(&done, 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&job_full[b], 1);
            mbar_init(&job_free[b], 1 + kWWarps + kSWarps + kOWarps + (BOUNDARY ? 1 : kPWarps));
        }
        mbar_init(&w_sync, kWWarps);
        mbar_init(&o_sync, kOWarps);
        fence_barrier_init();
    }
    grid_launch_dependents();
    grid_dependency_wait();
    const int n_jobs = a.head->n_items * a.H;
    if (BOUNDARY ? a.head->n_multi == 0 : static_cast<int>(blockIdx.x) >= n_jobs) return;
    if (w == 3) {
        tmem_alloc(&tmem_slot, F::COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_slot;
    bool ok = true;   // no wait of this warp has run out
    // The k-th pair of this CTA, for every warp but the producer; false behind the last.
    auto next_job = [&](int k, LinItem& it, int& h) {
        ok = ok && bar_wait(&job_full[k & 1], (k >> 1) & 1);
        if (!ok) return false;
        const Job& j = jobs[k & 1];
        it = j.it;
        h = j.h;
        warp_arrive(&job_free[k & 1]);
        return h >= 0;
    };
    // Four warps meet (bounded, as all waits are; a named barrier would not be).
    auto meet = [&](uint64_t* bar, int& n) {
        warp_arrive(bar);
        ok = ok && bar_wait(bar, n & 1);
        ++n;
    };

    if (w < 4) {
        // every warp of a group of four changes its registers by the same instruction
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (w == 2) {
            // ---------------- producer
            // Claims a pair: the CTA's own number first, then from the counter; lane 0.
            auto claim = [&](bool first, Job& j) {
                auto count = [&]() { return static_cast<int>(gridDim.x) + atomicAdd(&a.head->next[BOUNDARY], 1); };
                for (int x = first ? static_cast<int>(blockIdx.x) : count();; x = count()) {
                    j.h = -1;
                    if (x >= n_jobs) return;
                    j.it = a.items[x / a.H];
                    if (BOUNDARY && j.it.seg + 1 == j.it.n_seg) continue;
                    j.h = x % a.H;
                    return;
                }
            };
            DecayWalk<true> walk;
            Job next;
            if (lane == 0) claim(true, next);
            int s = 0, ph = 1, g = 0;   // stage and its parity, chunks so far
#pragma unroll 1
            for (int k = 0; ok; ++k) {
                if (k >= 2 && !(ok = bar_wait(&job_free[k & 1], ((k >> 1) - 1) & 1))) break;
                if (lane == 0) jobs[k & 1] = next;
                __syncwarp();
                const LinItem it = jobs[k & 1].it;
                const int h = jobs[k & 1].h;
                if (lane == 0) mbar_arrive(&job_full[k & 1]);
                if (h < 0) break;
                const int nch = (it.n + C - 1) / C, hq = h / (a.H / a.Hqk);
                if (!BOUNDARY) walk.start(a, it, h, la_ring);
#pragma unroll 1
                for (int c = 0; c < nch; ++c, ++g) {
                    // the decays ahead of the wait for the stage
                    if (!BOUNDARY) walk.chunk(c, decays[g % F::ND]);
                    // the tiles: halves of q, k and v lie one behind another in the stage, a lane issues each
                    if (!(ok = bar_wait(&empty[s], ph))) break;
                    if (lane == 0) mbar_arrive_expect_tx(&full[s], F::STAGE);
                    __syncwarp();
                    constexpr int NQ = F::QB / F::HALF, NK = NQ + DK / 64, NV = NK + DV / 64;
                    if (lane < NV)
                        tma_load_2d(sm + s * F::STAGE + lane * F::HALF, lane < NQ ? &mq : lane < NK ? &mk : &mv,
                                    lane < NK ? hq * DK + 64 * (lane < NQ ? lane : lane - NQ) : h * DV + 64 * (lane - NK),
                                    it.t0 + c * C, &full[s]);
                    if (!BOUNDARY) warp_arrive(&full[s]);   // (written ahead of the barrier above)
                    if (++s == NST) {
                        s = 0;
                        ph ^= 1;
                    }
                    // late, so that a CTA with a long pair does not sit on another
                    if (c == max(nch - 2, 0) && lane == 0) claim(false, next);
                }
                if (nch == 0 && lane == 0) claim(false, next);
            }
            cp_async_wait_all();
            // no copy stays in flight behind the CTA: wait (bounded, quietly) for the last fill of every stage
#pragma unroll 1
            for (int c = g > NST ? g - NST : 0; c < g; ++c) bar_wait(&full[c % NST], (c / NST) & 1);
        } else if (w == 3) {
            // ---------------- issuer
            constexpr uint32_t id_o = idesc_bf16(128, C), id_o2 = idesc_bf16(128, C, false, false, true),
                               id_z = idesc_bf16(128, DK, false, true), neg_a = 1u << 13;
            const uint32_t tmu = __shfl_sync(0xffffffffu, tm, 0), base = __shfl_sync(0xffffffffu, smem_u32(sm), 0);
            // K-major tiles: halves of 64 channels, 32 bytes (2 in a descriptor) for each 16
            auto scores = [&](int s) {
                const uint32_t q = base + s * F::STAGE, k = q + F::QB;
                const uint64_t qd = sdesc_k_sw128(q), kd = sdesc_k_sw128(k);
#pragma unroll 1
                for (uint32_t b = 0; b < DK / 64; ++b)
#pragma unroll
                    for (uint32_t i = 0; i < 4; ++i)
                        mma_ss(tmu + F::SP, qd + b * (F::HALF >> 4) + 2 * i, kd + b * (F::HALF >> 4) + 2 * i, id_o, b + i > 0);
                mma_commit(&sp_full);
            };
            int s = 0, ph = 0, g = 0;   // stage and its parity, chunks so far
            LinItem it;
            int h;
#pragma unroll 1
            for (int job = 0; ok && next_job(job, it, h); ++job) {
                const int nch = (it.n + C - 1) / C;
                // the scores are formed a chunk ahead, but not ahead of the pair
                if (!BOUNDARY && nch > 0) {
                    if (!(ok = bar_wait(&full[s], ph) && (g == 0 || bar_wait(&sp_free, (g - 1) & 1)))) break;
                    tc_fence_after();
                    scores(s);
                }
#pragma unroll 1
                for (int c = 0; c < nch; ++c, ++g) {
                    const uint32_t q = base + s * F::STAGE, k = q + F::QB, v = k + F::KB;
                    const int s1 = s + 1 == NST ? 0 : s + 1, ph1 = s + 1 == NST ? ph ^ 1 : ph;
                    if (BOUNDARY && !(ok = bar_wait(&full[s], ph))) break;
                    // Z in two halves of the chunk's tokens, so that the warps of W fill one half while the other is used
                    const uint64_t kd = sdesc_mn_sw128(k, F::HALF);
                    const uint32_t zcol = tmu + F::Z + (g % F::NZ) * 128;
                    auto z_half = [&](int half) {
                        tc_fence_after();
#pragma unroll 2
                        for (int i = 0; i < 8; ++i) {   // part i / 2, tokens 32 half + 16 (i % 2) ..; odd parts are negated
                            const int sl = 2 * half + (i & 1);
                            mma_ts(zcol, tmu + F::W + 32 * (i >> 1) + 8 * sl, kd + sl * (2048 >> 4), id_z | ((i & 2) ? neg_a : 0u),
                                   half + i > 0);
                        }
                    };
                    if (!(ok = bar_wait(&w_go[0], g & 1) &&
                               (!BOUNDARY || g < F::NZ || bar_wait(&z_free[g % F::NZ], (g / F::NZ - 1) & 1))))
                        break;
                    z_half(0);
                    mma_commit(&w_free);
                    if (!BOUNDARY && c + 1 < nch) {
                        if (!(ok = bar_wait(&full[s1], ph1) && bar_wait(&sp_free, g & 1))) break;
                        tc_fence_after();
                        scores(s1);
                    }
                    if (!(ok = bar_wait(&w_go[1], g & 1))) break;
                    z_half(1);
                    mma_commit(&z_full[g & 1]);
                    if (!BOUNDARY) {
                        if (!(ok = bar_wait(&o_go[g & 1], (g >> 1) & 1))) break;
                        tc_fence_after();
                        const uint64_t qd = sdesc_k_sw128(q);
#pragma unroll 1
                        for (uint32_t b = 0; b < DK / 64; ++b)
#pragma unroll
                            for (uint32_t i = 0; i < 4; ++i)
                                mma_ts(tmu + F::O1, tmu + F::SB + 32 * b + 8 * i, qd + b * (F::HALF >> 4) + 2 * i, id_o, b + i > 0);
                        const uint64_t vd = sdesc_mn_sw128(v, F::HALF), pd = sdesc_k_sw128(base + F::P0 + (g & 1) * 2 * F::PB);
#pragma unroll
                        for (int i = 0; i < C / 16; ++i) {
                            mma_ss_keep(tmu + F::O2, vd + i * (2048 >> 4), pd + i * 2, id_o2, i > 0);
                            mma_ss_kept(tmu + F::O2, vd + i * (2048 >> 4), pd + (F::PB >> 4) + i * 2, id_o2, 1u);
                        }
                        mma_commit(&o_full[g & 1]);
                    }
                    mma_commit(&empty[s]);
                    s = s1;
                    ph = ph1;
                }
            }
            mma_commit(&done);
            ok = bar_wait(&done, 0) && ok;   // no product stays in flight behind the CTA
        } else if (BOUNDARY) {
            // ---------------- decays, where a chunk takes less time than forming them and issuing its copies
            if (w == 1) {
                DecayWalk<false> walk;
                LinItem it;
                int h, s = 0, ph = 1, g = 0;
#pragma unroll 1
                for (int job = 0; ok && next_job(job, it, h); ++job) {
                    walk.start(a, it, h, la_ring);
                    const int nch = (it.n + C - 1) / C;
#pragma unroll 1
                    for (int c = 0; c < nch; ++c, ++g) {
                        if (!(ok = bar_wait(&empty[s], ph))) break;
                        walk.chunk(c, decays[g % F::ND]);
                        warp_arrive(&full[s]);
                        if (++s == NST) {
                            s = 0;
                            ph ^= 1;
                        }
                    }
                    if (lane == 0) a.zdecay[static_cast<size_t>(it.z0 + it.seg) * a.H + h] = exp2_of(walk.total);
                }
                cp_async_wait_all();
            }
        } else {
            // ---------------- P: warp w has rows 32 w .. 32 w + 31; columns above the diagonal blocks stay zero
            {
                const int row = 32 * w + lane;
                uint8_t* p0 = sm + F::P0 + row * 128;
                if (w == 0)
                    for (int b = 0; b < 4; ++b)
                        for (int i = 4; i < 8; ++i)
                            *reinterpret_cast<uint4*>(p0 + b * F::PB + ((i ^ (row & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
                // 32 columns from 8 b on, as two bf16 parts: x, and what its rounding left
                auto put = [&](uint8_t* p, int b, const float (&x)[32]) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t u[4], r[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float x0 = x[8 * i + 2 * j], x1 = x[8 * i + 2 * j + 1];
                            u[j] = pack_bf16x2(x0, x1);
                            r[j] = pack_bf16x2(x0 - lo_f32(u[j]), x1 - hi_f32(u[j]));
                        }
                        uint8_t* at = p + (((b + i) ^ (row & 7)) << 4);
                        *reinterpret_cast<uint4*>(at) = make_uint4(u[0], u[1], u[2], u[3]);
                        *reinterpret_cast<uint4*>(at + F::PB) = make_uint4(r[0], r[1], r[2], r[3]);
                    }
                };
                int s = 0, ph = 0, g = 0;
                LinItem it;
                int h;
#pragma unroll 1
                for (int job = 0; ok && next_job(job, it, h); ++job)
#pragma unroll 1
                for (int c = (it.n + C - 1) / C; c > 0; --c, ++g) {
                    if (!(ok = bar_wait(&full[s], ph) && bar_wait(&sp_full, g & 1))) break;
                    tc_fence_after();
                    // the scores first, so that the next ones can be formed: the diagonal block's 32 columns, and those
                    // left of it (second warp)
                    const uint32_t at = tm + F::SP + (static_cast<uint32_t>(32 * w) << 16);
                    float xd[32], xl[32];
                    tmem_ld32(at + 32 * w, xd);
                    if (w == 1) tmem_ld32(at, xl);
                    tmem_wait_ld_regs<32>(xd);
                    if (w == 1) tmem_wait_ld_regs<32>(xl);
                    tc_fence_before();
                    warp_arrive(&sp_free);
                    const Decays& d = decays[g % F::ND];
                    const float gr = d.g2[row], gl = d.g2l[row];
                    if (g >= 2 && !(ok = bar_wait(&o_full[g & 1], ((g >> 1) - 1) & 1))) break;
                    uint8_t* p = p0 + (g & 1) * 2 * F::PB;
                    if (w == 1) {   // a factor of two parts, each at most 1, about g_32
                        const float er = ex2_approx((gr - d.g2m) + (gl - d.g2ml));
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            const float4 m = *reinterpret_cast<const float4*>(&d.m[j]);
                            xl[j] *= er * m.x;
                            xl[j + 1] *= er * m.y;
                            xl[j + 2] *= er * m.z;
                            xl[j + 3] *= er * m.w;
                        }
                        put(p, 0, xl);
                    }
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {   // what lies behind the row's own column is cut off
                        const float4 gj = *reinterpret_cast<const float4*>(&d.g2[32 * w + j]);
                        const float4 lj = *reinterpret_cast<const float4*>(&d.g2l[32 * w + j]);
                        const float2 m1 = make_float2(-1.f, -1.f), gr2 = make_float2(gr, gr), gl2 = make_float2(gl, gl);
                        auto diff = [&](float h0, float h1, float l0, float l1) {
                            return __fadd2_rn(__ffma2_rn(m1, make_float2(h0, h1), gr2), __ffma2_rn(m1, make_float2(l0, l1), gl2));
                        };
                        const float2 e0 = diff(gj.x, gj.y, lj.x, lj.y), e1 = diff(gj.z, gj.w, lj.z, lj.w);
                        xd[j] = j <= lane ? xd[j] * ex2_approx(e0.x) : 0.f;
                        xd[j + 1] = j + 1 <= lane ? xd[j + 1] * ex2_approx(e0.y) : 0.f;
                        xd[j + 2] = j + 2 <= lane ? xd[j + 2] * ex2_approx(e1.x) : 0.f;
                        xd[j + 3] = j + 3 <= lane ? xd[j + 3] * ex2_approx(e1.y) : 0.f;
                    }
                    put(p, 4 * w, xd);
                    fence_proxy_async_smem();
                    warp_arrive(&o_go[g & 1]);
                    if (++s == NST) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
        }
    } else if (w < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        const int q4 = w & 3, tg = t & 127;   // channels of v 32 q4 .. 32 q4 + 31, thread of the group
        const bool mine = 32 * q4 < DV;
        const uint32_t lanes = static_cast<uint32_t>(32 * q4) << 16;
        // Of a 16-token x 16-channel tile (channels 32 q4 + 16 lh ..) as four 8 x 8 matrices, channels first: the row
        // that this lane addresses in a swizzled 64-channel half tile, for the chunk's first tokens (128 bytes on for
        // each further token; the swizzle repeats every eight).
        auto tile_row = [&](int lh) {
            const int tok = ((lane >> 4) << 3) + (lane & 7), c8 = 32 * q4 + 16 * lh + (lane & 8);
            return (c8 >> 6) * F::HALF + tok * 128 + ((((c8 & 63) >> 3) ^ (tok & 7)) << 4);
        };
        const uint32_t row0 = tile_row(0), row1 = tile_row(1);
        auto wait = [&](uint64_t* bar, uint32_t parity) { ok = ok && bar_wait(bar, parity); };
        int s = 0, ph = 0, g = 0, met = 0;
        LinItem it;
        int h;
        if (w < 8 || BOUNDARY) {
            // ---------------- W: all tokens, or in the boundary pass, where there is no o to write, 32 for each four
            // warps
            const int from = BOUNDARY && w >= 8 ? 32 : 0, to = BOUNDARY ? from + 32 : C;
            uint64_t* const sync = BOUNDARY && w >= 8 ? &o_sync : &w_sync;
#pragma unroll 1
            for (int job = 0; ok && next_job(job, it, h); ++job)
#pragma unroll 1
            for (int left = it.n; left > 0 && ok; left -= C, ++g) {
                wait(&full[s], ph);
                uint8_t* kt = sm + s * F::STAGE + F::QB;
                uint8_t* vt = kt + F::KB;
                if (left < C) {
                    // rows behind the sequence belong to others: they must not reach a sum, not even times zero
#pragma unroll 1
                    for (int i = tg; ok && i < (C - left) * 8; i += 128) {
                        const int r = left + i / 8, x = r * 128 + (i & 7) * 16;
#pragma unroll
                        for (int b = 0; b < DK / 64; ++b)
                            *reinterpret_cast<uint4*>(kt + b * F::HALF + x) = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                        for (int b = 0; b < DV / 64; ++b)
                            *reinterpret_cast<uint4*>(vt + b * F::HALF + x) = make_uint4(0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                    meet(sync, met);
                }
                const Decays& d = decays[g % F::ND];
                uint32_t v[2][4];
                uint4 wb[4];   // w1, w2, -w3 of this thread's pair of tokens in each block of eight
                auto load_v = [&](uint32_t row, int half) {
                    ldsm_x4_trans(smem_u32(vt) + row + half * 128, v[0]);
                    ldsm_x4_trans(smem_u32(vt) + row + half * 128 + 16 * 128, v[1]);
                };
                if (mine) load_v(row0, from);
#pragma unroll 1
                for (int half = from; half < to; half += 32) {
#pragma unroll
                    for (int b = 0; b < 4; ++b) wb[b] = d.w[half / 2 + 4 * b + (lane & 3)];
                    uint32_t u[2][4][8];   // 32 tokens, 16 channels each
                    if (mine) {
#pragma unroll
                        for (int lh = 0; lh < 2; ++lh) {
#pragma unroll
                            for (int r = 0; r < 8; ++r) {   // block r / 2, channels 8 (r % 2) + lane / 4 of the sixteen
                                const uint32_t x = v[r >> 2][r & 3];
                                const uint4 w4 = wb[r >> 1];
                                u[lh][0][r] = fma_bf16x2(x, w4.x, 0x80008000u);
                                u[lh][1][r] = fma_bf16x2(x, w4.x ^ 0x80008000u, u[lh][0][r]);
                                u[lh][2][r] = fma_bf16x2(x, w4.y, 0x80008000u);
                                u[lh][3][r] = fma_bf16x2(x, w4.z, fma_bf16x2(x, w4.y ^ 0x80008000u, u[lh][2][r]));
                            }
                            if (lh == 0) load_v(row1, half);
                            else if (half + 32 < to) load_v(row0, half + 32);
                        }
                    }
                    if (g > 0) {
                        if (half == 0) wait(&w_free, (g - 1) & 1);
                        else wait(&z_full[(g - 1) & 1], ((g - 1) >> 1) & 1);
                    }
                    if (mine && ok) {
                        tc_fence_after();
#pragma unroll
                        for (int lh = 0; lh < 2; ++lh)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                tmem_st_16x128b_x4(tm + lanes + (static_cast<uint32_t>(16 * lh) << 16) + F::W + 32 * k + half / 2,
                                                   u[lh][k]);
                    }
                    if (mine && ok) tmem_wait_st();
                    tc_fence_before();
                    warp_arrive(&w_go[half >> 5], ok);
                }
                if (++s == NST) {
                    s = 0;
                    ph ^= 1;
                }
            }
        } else {
            // ---------------- o
            // Leave for o of chunk c is given with the chunk's decays in sight: a stage is filled anew as soon as its
            // products are done, so nobody may look for a filling after it has let those go ahead.
            auto leave = [&](int n) {
                wait(&full[s], ph);
                if (++s == NST) {
                    s = 0;
                    ph ^= 1;
                }
                warp_arrive(&o_go[n & 1], ok);
            };
#pragma unroll 1
            for (int job = 0; ok && next_job(job, it, h); ++job) {
            if (it.n > 0) leave(g);
#pragma unroll 1
            for (int left = it.n; left > 0 && ok; left -= C, ++g) {
                const int tok = it.t0 + it.n - left;
                wait(&o_full[g & 1], (g >> 1) & 1);
                uint8_t* ob = sm + F::O0 + (g & 1) * F::VB;
                // the store that read this buffer two chunks ago is done with it
                if (tg == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
                meet(&o_sync, met);
                if (mine && ok) {
                    tc_fence_after();
                    const Decays& d = decays[g % F::ND];
#pragma unroll 1
                    for (int u4 = 0; u4 < 4; ++u4) {   // 16 channels, 32 tokens
                        const int lh = u4 & 1, half = (u4 >> 1) * 32;
                        float x[16], y[16];
                        const uint32_t at = tm + lanes + (static_cast<uint32_t>(16 * lh) << 16) + half;
                        tmem_ld_16x256b_x4(at + F::O1, x);
                        tmem_ld_16x256b_x4(at + F::O2, y);
                        float2 e[4];
#pragma unroll
                        for (int b = 0; b < 4; ++b) e[b] = *reinterpret_cast<const float2*>(&d.eg[half + 8 * b + 2 * (lane & 3)]);
                        tmem_wait_ld_regs<16>(x);
                        tmem_wait_ld_regs<16>(y);
                        if (u4 == 3) {   // O1 and O2 have been read
                            tc_fence_before();
                            if (left > C) leave(g + 1);
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t u[4];
#pragma unroll
                            for (int r = 0; r < 4; ++r) {   // block 2 i + r / 2, channels 8 (r % 2) + lane / 4
                                const int k = 8 * i + 2 * r;
                                const float2 eb = e[2 * i + (r >> 1)];
                                u[r] = pack_bf16x2(fmaf(eb.x, x[k], y[k]), fmaf(eb.y, x[k + 1], y[k + 1]));
                            }
                            stsm_x4_trans(smem_u32(ob) + (lh ? row1 : row0) + (half + 16 * i) * 128, u);
                        }
                    }
                } else if (left > C) {
                    leave(g + 1);
                }
                fence_proxy_async_smem();
                meet(&o_sync, met);
                if (left >= C) {
                    if (tg == 0 && ok) {
#pragma unroll
                        for (int b = 0; b < DV / 64; ++b) tma_store_2d(&mo, h * DV + 64 * b, tok, ob + b * F::HALF);
                        bulk_commit();
                    }
                } else {   // the rows behind the sequence are not this one's to write
                    if (tg == 0) bulk_commit();   // an empty group: the wait above counts one for every chunk
                    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.o) + (static_cast<size_t>(tok) * a.H + h) * DV;
#pragma unroll 1
                    for (int i = tg; ok && i < left * (DV / 8); i += 128) {
                        const int r = i / (DV / 8), k8 = i % (DV / 8);
                        st_global_v4(dst + static_cast<size_t>(r) * a.H * DV + 8 * k8,
                                     *reinterpret_cast<const uint4*>(ob + (k8 >> 3) * F::HALF + r * 128 + (((k8 & 7) ^ (r & 7)) << 4)));
                    }
                }
            }
            }
            if (tg == 0) bulk_wait0();
        }
    } else {
        // ---------------- state: thread = channel of v, S[i] = channel i of k
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsState));
        const int q4 = w & 3, ch = 32 * q4 + lane;
        const bool mine = ch < DV;
        const uint32_t lanes = static_cast<uint32_t>(32 * q4) << 16;
        float S[DK];
        int s = 0, ph = 0, g = 0;
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
            warp_arrive(&o_go[g & 1]);
        };
        if (!BOUNDARY) warp_arrive(&w_go[0]);   // there is no Z yet
        LinItem it;
        int h;
#pragma unroll 1
        for (int job = 0; ok && next_job(job, it, h); ++job) {
            const float* start = nullptr;
            if (it.seg == 0) {
                if (a.initial_state) start = a.initial_state + (static_cast<size_t>(it.seq) * a.H + h) * DK * DV;
            } else if (!BOUNDARY) {
                start = a.z + (static_cast<size_t>(it.z0 + it.seg - 1) * a.H + h) * DK * DV;
            }
            float* end = nullptr;
            if (BOUNDARY) end = a.z + (static_cast<size_t>(it.z0 + it.seg) * a.H + h) * DK * DV;
            else if (a.final_state && it.seg + 1 == it.n_seg)
                end = a.final_state + (static_cast<size_t>(it.seq) * a.H + h) * DK * DV;
#pragma unroll
            for (int i = 0; i < DK; ++i) S[i] = start && mine ? start[i * DV + ch] : 0.f;
            // tokens to the next checkpoint, its place, and how many places the table has from there
            int to_ck = 0, ck_room = 0;
            float* ck = nullptr;
            if (!BOUNDARY && a.ckpt_stride) {
                const int first = a.ckpt_cu[it.seq] + it.pos / a.ckpt_stride;
                to_ck = a.ckpt_stride - it.pos % a.ckpt_stride;
                ck_room = first >= 0 && a.checkpoints ? a.ckpt_cu[it.seq + 1] - first : 0;
                ck = a.checkpoints + (static_cast<long long>(first) * a.H + h) * (DK * DV);
            }
            // A chunk's checkpoint and the segment's end are written once the next chunk's products have their copy of
            // the state; without tokens the state stays as it was.
            float *dst = nullptr, *last = it.n > 0 ? nullptr : end;
#pragma unroll 1
            for (int left = it.n;; left -= C) {
                float eC = 0.f;
                if (left > 0) {
                    if (!(ok = bar_wait(&full[s], ph))) break;   // before Sb lets the chunk's products go ahead (see `leave`)
                    eC = decays[g % F::ND].eC;
                    if (BOUNDARY) {
                        warp_arrive(&empty[s]);
                    } else {
                        // the copy before has been read
                        if (g > 0 && !(ok = bar_wait(&o_full[(g - 1) & 1], ((g - 1) >> 1) & 1))) break;
                        tc_fence_after();
                        publish();
                    }
                }
                if (mine && (dst || last)) {
#pragma unroll 1
                    for (int k = 0; k < 2; ++k) {
                        float* p = k == 0 ? dst : last;
                        if (p)
#pragma unroll
                            for (int i = 0; i < DK; ++i) p[i * DV + ch] = S[i];
                    }
                }
                if (left <= 0) break;
                {
                    if (!(ok = bar_wait(&z_full[g & 1], (g >> 1) & 1))) break;
                    if (mine) {
                        tc_fence_after();
#pragma unroll
                        for (int b = 0; b < DK; b += 32) {
                            float z[32];
                            tmem_ld32(tm + lanes + F::Z + (g % F::NZ) * 128 + b, z);
                            tmem_wait_ld_regs<32>(z);
#pragma unroll
                            for (int i = 0; i < 32; i += 2) {
                                const float2 y = __ffma2_rn(make_float2(eC, eC), make_float2(S[b + i], S[b + i + 1]),
                                                            make_float2(z[i], z[i + 1]));
                                S[b + i] = y.x;
                                S[b + i + 1] = y.y;
                            }
                        }
                        tc_fence_before();
                    }
                    warp_arrive(BOUNDARY ? &z_free[g % F::NZ] : &w_go[0]);
                    if (++s == NST) {
                        s = 0;
                        ph ^= 1;
                    }
                    ++g;
                    to_ck -= C;
                    dst = nullptr;
                    if (!BOUNDARY && to_ck == 0 && left >= C) {
                        to_ck = a.ckpt_stride;
                        if (ck_room > 0) dst = ck;
                        else if (lane == 0) set_status(a.status, KDA_ERR_DEVICE_INPUT);
                        --ck_room;
                        ck += static_cast<size_t>(a.H) * (DK * DV);
                    }
                }
                last = left <= C ? end : nullptr;
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
cudaError_t launch(const LinArgs& a, const LinMaps& m, cudaStream_t s) {
    using F = Cfg<DK, DV, BOUNDARY>;
    const int smem = static_cast<int>(F::BYTES) + 1024;
    static SmemLimit limit;
    cudaError_t e = limit.raise(reinterpret_cast<const void*>(&lin_bf16_kernel<DK, DV, BOUNDARY>), smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    const long long jobs = static_cast<long long>(BOUNDARY ? a.max_bounds : a.max_items) * a.H;
    cfg.gridDim = dim3(static_cast<unsigned>(jobs < kLinSms ? jobs : kLinSms));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, lin_bf16_kernel<DK, DV, BOUNDARY>, a, m.q, m.k, m.v, m.o);
}

template <int DK, int DV>
cudaError_t launch_b(const LinArgs& a, const LinMaps& m, bool boundary_pass, cudaStream_t s) {
    return boundary_pass ? launch<DK, DV, true>(a, m, s) : launch<DK, DV, false>(a, m, s);
}

}  // namespace

bool make_lin_maps(const LinArgs& a, LinMaps& m) {
    memset(&m, 0, sizeof(m));
    if (a.total_tokens == 0) return true;   // without tokens no tile is loaded or stored
    const long long cq = static_cast<long long>(a.Hqk) * a.dk, cv = static_cast<long long>(a.H) * a.dv;
    return make_map(&m.q, a.q, cq, a.total_tokens) && make_map(&m.k, a.k, cq, a.total_tokens) &&
           make_map(&m.v, a.v, cv, a.total_tokens) && make_map(&m.o, a.o, cv, a.total_tokens);
}

cudaError_t launch_lin_bf16(const LinArgs& a, const LinMaps& m, bool boundary_pass, cudaStream_t s) {
    if (a.dk == 64) return a.dv == 64 ? launch_b<64, 64>(a, m, boundary_pass, s) : launch_b<64, 128>(a, m, boundary_pass, s);
    return a.dv == 64 ? launch_b<128, 64>(a, m, boundary_pass, s) : launch_b<128, 128>(a, m, boundary_pass, s);
}

}  // namespace kda
