// Attention of whole prompts packed one behind the other, grouped heads.
//
// This form: a warp per (query, head) row, walking the visible keys one at a
// time with the running (m, l) softmax in fp32.
#include "common.cuh"
#include "serving.h"

namespace rwsm {

__device__ unsigned g_error_attention_packed = 0;

namespace {

constexpr int kTileTokens = 16;                    // query rows of a CTA's tile
constexpr int kThreads = 128;

// Rows of sequence s: false when its bounds fall or leave the tensor.
__device__ __forceinline__ bool bounds_of(const int32_t* cu, int64_t s, int64_t total, int64_t& a,
                                          int64_t& n)
{
    a = __ldg(cu + s);
    const int64_t b = __ldg(cu + s + 1);
    const bool ok = a >= 0 && b >= a && b <= total;
    n = ok ? b - a : 0;
    return ok;
}

__device__ __forceinline__ bool sequence_of(const PackedProblem& p, int64_t s, int64_t& q0,
                                            int64_t& n_q, int64_t& k0, int64_t& n_k)
{
    const bool ok_q = bounds_of(p.cu_q, s, p.total_q, q0, n_q);
    const bool ok_k = bounds_of(p.cu_k, s, p.total_k, k0, n_k);
    if (!(ok_q && ok_k))
        n_q = n_k = 0;
    return ok_q && ok_k;
}

// One query row against keys [0, n) of its sequence, on a warp; every lane
// holds D / 32 consecutive elements of the result.
template <typename T, int D>
__device__ void attend_row(const PackedProblem& p, const unsigned short* q,
                           const unsigned short* k, const unsigned short* v, int64_t n,
                           float scale_log2, float (&o)[D / 32], float& m, float& l)
{
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    auto load = [&](const unsigned short* row, float (&x)[E]) {
#pragma unroll
        for (int e = 0; e < E; e += 2)
            Elem<T>::unpack2(__ldg(reinterpret_cast<const unsigned*>(row + lane * E + e)), x[e],
                             x[e + 1]);
    };
    float qx[E];
    load(q, qx);
    m = kNegInf;
    l = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e)
        o[e] = 0.0f;
    for (int64_t j = 0; j < n; ++j) {
        float x[E], dot = 0.0f;
        load(k + j * p.k.row, x);
#pragma unroll
        for (int e = 0; e < E; ++e)
            dot = fmaf(qx[e], x[e], dot);
        dot = warp_sum(dot) * scale_log2;
        const float mn = fmaxf(m, dot), ref = mn == kNegInf ? 0.0f : mn;
        const float alpha = ex2_ftz(m - ref), w = ex2_ftz(dot - ref);
        m = mn;
        l = l * alpha + w;
        load(v + j * p.v.row, x);
#pragma unroll
        for (int e = 0; e < E; ++e)
            o[e] = fmaf(w, x[e], o[e] * alpha);
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
attention_packed_rows_kernel(const PackedProblem p, float scale_log2)
{
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int head = blockIdx.y;
    const int kvh = head / (p.n_heads / p.n_kv_heads);
    pdl_launch_dependents();
    pdl_wait();
    int64_t tile = blockIdx.x;
    for (int64_t s = 0; s < p.n_seqs; ++s) {
        int64_t q0, n_q, k0, n_k;
        if (!sequence_of(p, s, q0, n_q, k0, n_k)) {
            if (threadIdx.x == 0)
                atomicOr(&g_error_attention_packed, kErrBadIndex);
            continue;
        }
        const int64_t tiles = (n_q + kTileTokens - 1) / kTileTokens;
        if (tile >= tiles) {
            tile -= tiles;
            continue;
        }
        for (int r = warp; r < kTileTokens; r += kThreads / 32) {
            const int64_t i = tile * kTileTokens + r;
            if (i >= n_q)
                break;
            int64_t n = p.causal ? i + n_k - n_q + 1 : n_k;
            n = n < 0 ? 0 : n;
            float o[E], m, l;
            attend_row<T, D>(
                p, static_cast<const unsigned short*>(p.q.data) + (q0 + i) * p.q.row + head * p.q.head,
                static_cast<const unsigned short*>(p.k.data) + k0 * p.k.row + kvh * p.k.head,
                static_cast<const unsigned short*>(p.v.data) + k0 * p.v.row + kvh * p.v.head, n,
                scale_log2, o, m, l);
            const float inv = 1.0f / l;
            unsigned short* dst = static_cast<unsigned short*>(p.o.data) + (q0 + i) * p.o.row +
                                  head * p.o.head + lane * E;
#pragma unroll
            for (int e = 0; e < E; e += 2)
                *reinterpret_cast<unsigned*>(dst + e) = Elem<T>::pack2(o[e] * inv, o[e + 1] * inv);
            if (p.lse && lane == 0)
                p.lse[(q0 + i) * p.n_heads + head] =
                    l == 0.0f ? kNegInf : (m + __log2f(l)) * 0.69314718055994531f;
        }
        return;
    }
}

template <typename T, int D>
cudaError_t launch(const PackedProblem& p, cudaStream_t s)
{
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.total_q / kTileTokens + p.n_seqs),
                       static_cast<unsigned>(p.n_heads), 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = static_cast<unsigned>(launch_attrs(attr, 1));
    const float scale_log2 = static_cast<float>(static_cast<double>(p.scale) * 1.4426950408889634);
    const cudaError_t err = cudaLaunchKernelEx(&cfg, attention_packed_rows_kernel<T, D>, p,
                                               scale_log2);
    note_launch();
    return err;
}

}  // namespace

cudaError_t launch_attention_packed(const PackedProblem& p, cudaStream_t s)
{
    if (p.dtype == SOFTMAX_BF16)
        return p.head_dim == 64 ? launch<BF16Bits, 64>(p, s) : launch<BF16Bits, 128>(p, s);
    return p.head_dim == 64 ? launch<F16Bits, 64>(p, s) : launch<F16Bits, 128>(p, s);
}

unsigned read_error_attention_packed(bool clear)
{
    unsigned v = 0;
    if (cudaMemcpyFromSymbol(&v, g_error_attention_packed, sizeof v) != cudaSuccess)
        return 0;
    if (clear && v) {
        const unsigned zero = 0;
        cudaMemcpyToSymbol(g_error_attention_packed, &zero, sizeof zero);
    }
    return v;
}

}  // namespace rwsm
