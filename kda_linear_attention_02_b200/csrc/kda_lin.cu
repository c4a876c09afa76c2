// kda_lin.cu -- decayed linear attention, host side and bookkeeping: argument checks, the split of the batch
// into segments, and the pass that joins the segments' states.
//
// A sequence is walked chunk by chunk, and the state passes from chunk to chunk, so one (sequence, head)
// occupies one SM at a time.  A batch with few long sequences would leave SMs idle; its sequences are cut
// into segments.  Since a segment acts on the state it starts from by one factor alone,
//
//     S_end = e^{sum of log_alpha} S_start + Z,
//
// every segment with a successor is walked once from a zero state for its Z (reading k and v only), the
// starts of all segments follow from a short scan, and the segments are then walked in full side by side.
#include <algorithm>

#include "kda_device.cuh"
#include "kda_lin.h"

namespace kda {

namespace {

// Splits the sequences of more than `whole` tokens into segments of seg_len tokens and validates cu_seqlens
// (cu[0] = 0, non-decreasing, cu[N] = total); a bad table gives no items, so that the kernels behind do
// nothing.  When all items fit one block they are ordered by length, longest first: blocks start in that order,
// and a long sequence that started last would run on alone at the end.
__global__ void __launch_bounds__(1024) lin_index_kernel(const int32_t* cu, int n_seqs, int total,
                                                         int whole, int seg_len, LinHead* head, LinItem* items,
                                                         int2* multi, int* status) {
    __shared__ long long warp_sums[32];
    __shared__ int lens[1024];
    __shared__ int s_multi;
    grid_launch_dependents();
    grid_dependency_wait();
    const int t = threadIdx.x, lane = t & 31, w = t >> 5;
    if (t == 0) s_multi = 0;
    bool bad = t == 0 && (cu[0] != 0 || cu[n_seqs] != total);
    for (int i = t; i < n_seqs; i += 1024) bad |= cu[i + 1] < cu[i];
    if (__syncthreads_or(bad)) {
        if (t == 0) {
            *head = LinHead{0, 0, {0, 0}};
            set_status(status, KDA_ERR_DEVICE_INPUT);
        }
        return;
    }
    long long carry = 0;   // items in the low half, boundaries in the high half
    for (int base = 0; base < n_seqs; base += 1024) {
        const int i = base + t;
        int t0 = 0, len = 0, ns = 0;
        if (i < n_seqs) {
            t0 = cu[i];
            len = cu[i + 1] - t0;
            ns = len > whole ? (len - 1) / seg_len + 1 : 1;
        }
        const long long c = ns ? (static_cast<long long>(ns - 1) << 32) | ns : 0;
        long long x = c;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, off);
            if (lane >= off) x += y;
        }
        if (lane == 31) warp_sums[w] = x;
        __syncthreads();
        if (w == 0) {
            long long s = warp_sums[lane];
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, s, off);
                if (lane >= off) s += y;
            }
            warp_sums[lane] = s;
        }
        __syncthreads();
        const long long first = carry + x - c + (w ? warp_sums[w - 1] : 0);
        const int item0 = static_cast<int>(first & 0xffffffff), z0 = static_cast<int>(first >> 32);
        for (int s = 0; s < ns; ++s)
            items[item0 + s] = LinItem{i, s, ns, t0 + s * seg_len, ns == 1 ? len : min(seg_len, len - s * seg_len), s * seg_len, z0, 0};
        if (ns > 1) multi[atomicAdd(&s_multi, 1)] = make_int2(z0, ns);   // their order has no effect
        carry += warp_sums[31];
        __syncthreads();
    }
    const int n_items = static_cast<int>(carry & 0xffffffff);
    if (t == 0) *head = LinHead{n_items, s_multi, {0, 0}};
    if (n_items <= 1024) {
        LinItem it{};
        if (t < n_items) {
            it = items[t];
            lens[t] = it.n;
        }
        __syncthreads();
        if (t < n_items) {
            int rank = 0;
            for (int j = 0; j < n_items; ++j) rank += lens[j] > it.n || (lens[j] == it.n && j < t);
            items[rank] = it;
        }
    }
}

// Starts of the segments: z[s] holds the end state of segment s from a zero state (segment 0: from the
// sequence's own start), and becomes the state at the start of segment s + 1.  A thread carries four
// elements of one state through the boundaries of its sequence.
__global__ void __launch_bounds__(256) lin_join_kernel(const LinHead* head, const int2* multi,
                                                       float* __restrict__ z, const float* zdecay, int H,
                                                       int elems) {
    grid_launch_dependents();
    grid_dependency_wait();
    const long long e4 = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) * 4;
    const int h = static_cast<int>(e4 / elems);
    if (h >= H) return;
    for (int m = blockIdx.y; m < head->n_multi; m += gridDim.y) {
        const int z0 = multi[m].x, nb = multi[m].y - 1;
        float4* p = reinterpret_cast<float4*>(z + static_cast<size_t>(z0) * H * elems + e4);
        const size_t pitch = static_cast<size_t>(H) * elems / 4;
        const float* d = zdecay + static_cast<size_t>(z0) * H + h;
        float4 x = p[0];
#pragma unroll 4
        for (int s = 1; s < nb; ++s) {
            const float a = d[static_cast<size_t>(s) * H];
            const float4 y = p[s * pitch];
            x = make_float4(fmaf(a, x.x, y.x), fmaf(a, x.y, y.y), fmaf(a, x.z, y.z), fmaf(a, x.w, y.w));
            p[s * pitch] = x;
        }
    }
}

// A launch that may start while the kernel before it, which lets it, still writes: the kernels launched so wait before
// they read, and declare nothing const and __restrict__ (which would let them read by the non-coherent path).
template <typename... KArgs, typename... Args>
cudaError_t launch_chained(void (*kernel)(KArgs...), dim3 grid, dim3 block, cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

struct Span {
    const void* p;
    size_t n;
};
bool overlap(Span a, Span b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && a.n && b.n && x < y + b.n && y < x + a.n;
}
// Outputs are written while other heads and sequences are still read: none may lie over an input or over another output.
template <size_t NO, size_t NI>
bool clash(const Span (&outs)[NO], const Span (&ins)[NI]) {
    for (size_t i = 0; i < NO; ++i) {
        for (size_t j = i + 1; j < NO; ++j)
            if (overlap(outs[i], outs[j])) return true;
        for (const Span& in : ins)
            if (overlap(outs[i], in)) return true;
    }
    return false;
}
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
bool dims_ok(int dk, int dv) { return (dk == 64 || dk == 128) && (dv == 64 || dv == 128); }

// Which sequences are cut, and into segments of how many tokens.  A sequence stays whole when it has at most a
// quarter more than a fair share of the batch's (token, head) pairs over the SMs: the cut costs a second
// reading of k and v.  Else its segments have a little more than a share (bf16), so that the full ones fit the SMs
// once and what is left over fills the rest, but at least `least` tokens, below which a segment's set-up and the
// extra pass cost more than they give.  Measured, bf16, segments of half a share and of a share, each with 1/32
// more: 32768 tokens x 4 heads 110 and 76 us, 16384 x 16 heads 112 and 99 us, 3 x 10000 x 16 heads 174 and 158 us;
// of a share without more, or with 1/16: up to 10 % slower.
// fp32 keeps half a share: at dk = 64 two blocks share an SM (half and whole: 16384 tokens x 4 heads 133 and 223 us,
// 4 x 4096 x 8 heads 221 and 415); at dk = 128 one fits, and the choice matters little (392 and 376, 585 and 584 us;
// dv = 64, 3 heads of 5 x 3000: 163 and 172).
struct SegRule {
    int whole, len;
};
SegRule segment_rule(int64_t total_tokens, int H, int dv, bool bf16) {
    // fp32: a CTA has 32 columns of a state, and walks about five times as slowly
    const int64_t per_token = bf16 ? H : static_cast<int64_t>(H) * (dv / 32), least = bf16 ? 512 : 64;
    const int64_t share = (total_tokens * per_token + kLinSms - 1) / kLinSms;
    auto chunks = [](int64_t tokens) { return (tokens + kChunk - 1) / kChunk * kChunk; };
    SegRule r{};
    const int64_t part = bf16 ? share : share / 2;
    r.len = static_cast<int>(std::min<int64_t>(std::max<int64_t>(least, chunks(part + share / 32)), 0x40000000));
    r.whole = static_cast<int>(std::min<int64_t>(std::max<int64_t>(2 * least, share + share / 4), 0x40000000));
    return r;
}

struct LinLayout {
    SegRule seg;
    int max_items, max_bounds;
    size_t items, multi, z, zdecay, total;
};
LinLayout layout(int64_t total_tokens, int n_seqs, int H, int dk, int dv, bool bf16) {
    LinLayout l{};
    l.seg = segment_rule(total_tokens, H, dv, bf16);
    // a sequence that is cut has more than `whole` tokens, and every segment with a successor is full
    l.max_bounds = total_tokens > l.seg.whole ? static_cast<int>(total_tokens / l.seg.len) : 0;
    l.max_items = n_seqs + l.max_bounds;
    size_t at = round256(sizeof(LinHead));
    auto take = [&](size_t bytes) {
        const size_t p = at;
        at += round256(bytes);
        return p;
    };
    l.items = take(sizeof(LinItem) * static_cast<size_t>(l.max_items));
    l.multi = take(sizeof(int2) * static_cast<size_t>(l.max_bounds));
    l.z = take(sizeof(float) * static_cast<size_t>(l.max_bounds) * H * dk * dv);
    l.zdecay = take(sizeof(float) * static_cast<size_t>(l.max_bounds) * H);
    l.total = at;
    return l;
}

}  // namespace

}  // namespace kda

using namespace kda;

extern "C" {

size_t kda_lin_chunk_fwd_workspace_bytes(int64_t total_tokens, int n_seqs, int H, int dk, int dv, kda_dtype_t dtype) {
    if (total_tokens < 0 || total_tokens > 0x7fffffffLL || n_seqs < 0 || H <= 0 || !dims_ok(dk, dv)) return 0;
    if (dtype != KDA_BF16 && dtype != KDA_F32) return 0;
    if (n_seqs > 0x3fffffff) return 0;
    return layout(total_tokens, n_seqs, H, dk, dv, dtype == KDA_BF16).total;
}

kda_status_t kda_lin_chunk_fwd(const void* q, const void* k, const void* v, const float* log_alpha, int la_per_token,
                               const float* initial_state, const int32_t* cu_seqlens, int n_seqs,
                               int64_t total_tokens, int Hqk, int H, int dk, int dv, kda_dtype_t dtype,
                               int ckpt_stride, void* o, float* final_state, float* checkpoints,
                               const int32_t* ckpt_cu, void* workspace, size_t ws_bytes, kda_stream_t stream) {
    if (n_seqs < 0 || n_seqs > 0x3fffffff || total_tokens < 0 || H <= 0 || Hqk <= 0 || H % Hqk != 0 || ckpt_stride < 0 ||
        (la_per_token != 0 && la_per_token != 1))
        return KDA_ERR_ARG;
    if (total_tokens > 0x7fffffffLL) return KDA_ERR_ARG;   // cu_seqlens is int32
    if (dtype != KDA_BF16 && dtype != KDA_F32) return KDA_ERR_ARG;
    if (!dims_ok(dk, dv)) return KDA_ERR_UNSUPPORTED;
    if (ckpt_stride > 0 && (ckpt_stride % kChunk != 0 || !ckpt_cu)) return KDA_ERR_ARG;
    if (n_seqs == 0) return total_tokens == 0 ? KDA_OK : KDA_ERR_ARG;
    if (!cu_seqlens || !workspace) return KDA_ERR_ARG;
    if (total_tokens > 0 && (!q || !k || !v || !log_alpha || !o)) return KDA_ERR_ARG;
    const void* ptrs[] = {q, k, v, initial_state, o, final_state, checkpoints};
    for (const void* p : ptrs)
        if (p && !aligned(p, 16)) return KDA_ERR_ALIGN;
    if ((log_alpha && !aligned(log_alpha, 4)) || !aligned(cu_seqlens, 4) || (ckpt_cu && !aligned(ckpt_cu, 4)))
        return KDA_ERR_ALIGN;
    if (!aligned(workspace, 256)) return KDA_ERR_ALIGN;
    // (a later segment of a sequence may be done, and the final state written, before an earlier one starts)
    const size_t st_bytes = static_cast<size_t>(n_seqs) * H * dk * dv * sizeof(float);
    if (overlap({initial_state, st_bytes}, {final_state, st_bytes})) return KDA_ERR_ARG;
    const bool bf16 = dtype == KDA_BF16;
    const LinLayout l = layout(total_tokens, n_seqs, H, dk, dv, bf16);
    if (ws_bytes < l.total) return KDA_ERR_WORKSPACE;
    const size_t row = static_cast<size_t>(total_tokens) * (bf16 ? 2 : 4), nq = row * Hqk * dk, nv = row * H * dv,
                 table = (static_cast<size_t>(n_seqs) + 1) * 4;
    const Span outs[] = {{o, nv}, {final_state, st_bytes}, {workspace, l.total}};
    const Span ins[] = {{q, nq}, {k, nq}, {v, nv}, {log_alpha, (la_per_token ? static_cast<size_t>(total_tokens) : 1) * H * 4},
                        {initial_state, st_bytes}, {cu_seqlens, table}, {ckpt_stride ? ckpt_cu : nullptr, table}};
    if (clash(outs, ins)) return KDA_ERR_ARG;
    if (static_cast<long long>(l.max_items) * H > 0x7fffffffLL) return KDA_ERR_ARG;

    char* ws = static_cast<char*>(workspace);
    LinArgs a{};
    a.q = q; a.k = k; a.v = v; a.la = log_alpha; a.la_t = la_per_token ? H : 0;
    a.initial_state = initial_state; a.cu_seqlens = cu_seqlens; a.n_seqs = n_seqs; a.total_tokens = total_tokens;
    a.Hqk = Hqk; a.H = H; a.dk = dk; a.dv = dv; a.ckpt_stride = ckpt_stride; a.o = o; a.final_state = final_state;
    a.checkpoints = checkpoints; a.ckpt_cu = ckpt_cu;
    a.head = reinterpret_cast<LinHead*>(ws);
    a.items = reinterpret_cast<LinItem*>(ws + l.items);
    a.multi = reinterpret_cast<int2*>(ws + l.multi);
    a.z = reinterpret_cast<float*>(ws + l.z);
    a.zdecay = reinterpret_cast<float*>(ws + l.zdecay);
    a.max_items = l.max_items; a.max_bounds = l.max_bounds;
    a.status = status_ptr();
    if (!a.status) return KDA_ERR_CUDA;

    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    LinMaps maps;
    if (bf16 && !make_lin_maps(a, maps)) return KDA_ERR_CUDA;
    if (launch_chained(lin_index_kernel, dim3(1), dim3(1024), s, cu_seqlens, n_seqs, static_cast<int>(total_tokens),
                       l.seg.whole, l.seg.len, a.head, a.items, a.multi, a.status) != cudaSuccess)
        return KDA_ERR_CUDA;
    if (l.max_bounds > 0) {
        if ((bf16 ? launch_lin_bf16(a, maps, true, s) : launch_lin_simt(a, true, s)) != cudaSuccess) return KDA_ERR_CUDA;
        const int elems = dk * dv;
        const unsigned bx = static_cast<unsigned>((static_cast<size_t>(H) * elems / 4 + 255) / 256);
        const dim3 grid(bx, std::min(static_cast<unsigned>(l.max_bounds), std::max(1u, 4u * kLinSms / bx)));
        if (launch_chained(lin_join_kernel, grid, dim3(256), s, a.head, a.multi, a.z, a.zdecay, H, elems) != cudaSuccess)
            return KDA_ERR_CUDA;
    }
    return (bf16 ? launch_lin_bf16(a, maps, false, s) : launch_lin_simt(a, false, s)) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status_t kda_lin_recurrent_step(float* state, int64_t n_states, const int32_t* slots, int slot_stride,
                                    const void* q, const void* k, const void* v, const float* log_alpha,
                                    int la_per_token, int n, int Hqk, int H, int dk, int dv, kda_dtype_t dtype,
                                    void* o, kda_stream_t stream) {
    if (n < 0 || n > 0x40000000 || H <= 0 || Hqk <= 0 || H % Hqk != 0 || n_states < 0 || (la_per_token != 0 && la_per_token != 1))
        return KDA_ERR_ARG;
    if (slots ? slot_stride <= 0 : n > n_states) return KDA_ERR_ARG;
    if (dtype != KDA_BF16 && dtype != KDA_F32) return KDA_ERR_ARG;
    if (!dims_ok(dk, dv)) return KDA_ERR_UNSUPPORTED;
    if (n == 0) return KDA_OK;
    if (!q || !k || !v || !log_alpha || !o || (!state && n_states > 0)) return KDA_ERR_ARG;
    const size_t es = dtype == KDA_BF16 ? 2 : 4;
    if (!aligned(state, 16) || !aligned(q, es) || !aligned(k, es) || !aligned(v, es) || !aligned(o, es) ||
        !aligned(log_alpha, 4) || (slots && !aligned(slots, 4)))
        return KDA_ERR_ALIGN;
    if (static_cast<long long>(n) * H > 0x7fffffffLL) return KDA_ERR_ARG;
    const size_t nq = es * n * Hqk * dk, nv = es * n * H * dv;
    const Span outs[] = {{o, nv}, {state, static_cast<size_t>(n_states) * H * dk * dv * 4}};
    const Span ins[] = {{q, nq}, {k, nq}, {v, nv}, {log_alpha, (la_per_token ? static_cast<size_t>(n) : 1) * H * 4},
                        {slots, (static_cast<size_t>(n - 1) * slot_stride + 1) * 4}};
    if (clash(outs, ins)) return KDA_ERR_ARG;
    int* st = status_ptr();
    if (!st) return KDA_ERR_CUDA;
    return launch_lin_step(state, n_states, slots, slot_stride, q, k, v, log_alpha, la_per_token, n, Hqk, H, dk, dv,
                           dtype == KDA_BF16, o, st, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
               ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
