// Cache append: rotate new tokens' queries and keys by their positions and
// put keys and values into the paged cache, in one pass over the data.
//
//   (a, b) -> (a cos t - b sin t, a sin t + b cos t),  t = pos * inv_freq[i].
//
// Angles.  A position times a frequency in fp32 loses the angle at far
// positions (2^20 * 2^-24 is a sixteenth of a radian).  Here a frequency is
// kept as the fraction of a turn it adds per position, in 64-bit fixed point:
// pos * f in wrapping integer arithmetic is the angle modulo a full turn,
// exactly for that f (f itself is the double inv_freq / 2 pi, off by 2^-53 of
// itself).  The upper 32 bits, read as a signed number of 2^-31 half turns,
// go to sincospif in fp32 (off by 2^-25 of the angle).
//
// Bound by bytes: every element is read and written once (16-byte vectors),
// against a few multiply-adds each.  A CTA computes its tokens' cosines and
// sines once, into shared memory, for all of their heads.  Measured (32 query
// heads, 8 key/value heads of 128, bf16): 16001 tokens 64.7 us with inputs not
// in L2 (6.1 TB/s, a plain copy runs at 6.7); 256 tokens 4.1 us and 8 tokens 3.2,
// which is the launch, the index reads one behind the other, and the angles.
#include "common.cuh"
#include "serving.h"

namespace rwsm {

__device__ unsigned g_error_kv_append = 0;

namespace {

constexpr int kThreads = 256;
constexpr int kMaxHalf = 64;                       // rot_dim / 2 at most

// Fraction of a turn per position, in units of 2^-64 of a turn.
__device__ __forceinline__ uint64_t turn_fraction(double inv_freq)
{
    double t = inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
    t -= floor(t);
    return static_cast<uint64_t>(t * 18446744073709551616.0);   // saturates, NaN: 0
}

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8])
{
    Elem<T>::unpack2(w.x, x[0], x[1]);
    Elem<T>::unpack2(w.y, x[2], x[3]);
    Elem<T>::unpack2(w.z, x[4], x[5]);
    Elem<T>::unpack2(w.w, x[6], x[7]);
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    uint4 w;
    w.x = Elem<T>::pack2(x[0], x[1]);
    w.y = Elem<T>::pack2(x[2], x[3]);
    w.z = Elem<T>::pack2(x[4], x[5]);
    w.w = Elem<T>::pack2(x[6], x[7]);
    return w;
}

// TT tokens per CTA.  A work unit is two 16-byte vectors of one head: with
// D / 16 units to a head, unit u holds vectors (u, u + rot / 16) of the
// rotated part (halves), or (2u, 2u + 1) (interleaved, and past the rotated
// part); either way its pairs are the frequencies 8u .. 8u + 7.
template <typename T, int D, int TT>
__global__ void __launch_bounds__(kThreads)
kv_append_kernel(const AppendProblem p)
{
    constexpr int U = D / 16;
    constexpr int kBatch = TT == 1 ? 1 : 2;        // units that a thread has under way
    __shared__ float2 turn[TT][kMaxHalf];
    __shared__ int64_t k_at[TT], v_at[TT];         // cache element of the token, < 0: none
    __shared__ int32_t pos_of[TT];
    const int tid = threadIdx.x;
    const int half = p.rot_dim / 2;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * TT;
    const int tokens = p.n_tokens - t0 < TT ? static_cast<int>(p.n_tokens - t0) : TT;

    pdl_launch_dependents();
    pdl_wait();
    if (tid < tokens) {
        const int32_t pos = p.positions[t0 + tid];
        pos_of[tid] = pos;
        int64_t ka = -1, va = -1;
        if (pos >= 0) {
            const int64_t seq = p.seq_ids ? p.seq_ids[t0 + tid] : t0 + tid;
            int32_t page = -1;
            if (seq >= 0 && seq < p.cache.n_seqs && pos < p.cache.capacity)
                page = p.cache.table[seq * p.cache.table_stride + divide(pos, p.cache.page)];
            if (page >= 0 && page < p.cache.n_pages) {
                const int64_t row = pos - divide(pos, p.cache.page) * p.cache.page.d;
                ka = page * p.cache.k_page + row * p.cache.k_row;
                va = page * p.cache.v_page + row * p.cache.v_row;
            } else {
                atomicOr(&g_error_kv_append, kErrBadIndex);
            }
        }
        k_at[tid] = ka;
        v_at[tid] = va;
    }
    for (int i = tid; i < half * tokens; i += kThreads) {
        const int t = i / half, f = i - t * half;
        const int32_t pos = p.positions[t0 + t];
        const double w = p.inv_freq[f];
        const uint64_t angle = turn_fraction(w) * static_cast<uint64_t>(pos < 0 ? 0 : pos);
        float s, c;
        sincospif(static_cast<float>(static_cast<int32_t>(angle >> 32)) * 0x1p-31f, &s, &c);
        if (!(fabs(w) < 1e300))                    // an infinite or NaN frequency has no angle
            s = c = __int_as_float(0x7fc00000);
        turn[t][f] = make_float2(c, s);
    }
    __syncthreads();

    const int nq = p.q.data ? p.n_heads : 0, nk = p.cache.n_kv_heads;
    const int per_token = (nq + 2 * nk) * U, units = per_token * tokens;
    // kBatch units at a time: all of their loads are under way before the
    // first is used.
    for (int i0 = tid; i0 < units; i0 += kThreads * kBatch) {
        unsigned short* dst[kBatch];               // null: nothing to do
        uint4 w0[kBatch], w1[kBatch];
        int c0[kBatch], c1[kBatch], turn_at[kBatch];   // turn_at < 0: copied as it is
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int i = i0 + b * kThreads;
            dst[b] = nullptr;
            if (i >= units)
                continue;
            const int t = TT == 1 ? 0 : i / per_token, r = (i - t * per_token) / U, u = i % U;
            if (pos_of[t] < 0)
                continue;
            // Which tensor this head row belongs to.
            const int64_t token = t0 + t;
            const unsigned short* src;
            if (r < nq) {
                src = static_cast<const unsigned short*>(p.q.data) + token * p.q.row + r * p.q.head;
                dst[b] = static_cast<unsigned short*>(p.q_out.data) + token * p.q_out.row +
                         r * p.q_out.head;
            } else if (r < nq + nk) {
                if (k_at[t] < 0)
                    continue;
                src = static_cast<const unsigned short*>(p.k.data) + token * p.k.row +
                      (r - nq) * p.k.head;
                dst[b] = static_cast<unsigned short*>(p.cache.k) + k_at[t] +
                         (r - nq) * p.cache.k_head;
            } else {
                if (v_at[t] < 0)
                    continue;
                src = static_cast<const unsigned short*>(p.v.data) + token * p.v.row +
                      (r - nq - nk) * p.v.head;
                dst[b] = static_cast<unsigned short*>(p.cache.v) + v_at[t] +
                         (r - nq - nk) * p.cache.v_head;
            }
            const bool turns = r < nq + nk && u * 16 < p.rot_dim;
            const bool apart = turns && !p.interleaved;
            turn_at[b] = turns ? t * kMaxHalf + u * 8 : -1;
            c0[b] = apart ? u : 2 * u;
            c1[b] = apart ? u + p.rot_dim / 16 : 2 * u + 1;
            w0[b] = *reinterpret_cast<const uint4*>(src + c0[b] * 8);
            w1[b] = *reinterpret_cast<const uint4*>(src + c1[b] * 8);
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (!dst[b])
                continue;
            if (turn_at[b] >= 0) {
                float x[8], y[8];
                unpack8<T>(w0[b], x);
                unpack8<T>(w1[b], y);
                const float2* cs = &turn[0][0] + turn_at[b];
                if (p.interleaved) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 f = cs[j], g = cs[j + 4];
                        const float x0 = x[2 * j], x1 = x[2 * j + 1];
                        const float y0 = y[2 * j], y1 = y[2 * j + 1];
                        x[2 * j] = x0 * f.x - x1 * f.y;
                        x[2 * j + 1] = x0 * f.y + x1 * f.x;
                        y[2 * j] = y0 * g.x - y1 * g.y;
                        y[2 * j + 1] = y0 * g.y + y1 * g.x;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 f = cs[j];
                        const float x0 = x[j], y0 = y[j];
                        x[j] = x0 * f.x - y0 * f.y;
                        y[j] = x0 * f.y + y0 * f.x;
                    }
                }
                w0[b] = pack8<T>(x);
                w1[b] = pack8<T>(y);
            }
            *reinterpret_cast<uint4*>(dst[b] + c0[b] * 8) = w0[b];
            *reinterpret_cast<uint4*>(dst[b] + c1[b] * 8) = w1[b];
        }
    }
}

template <typename T, int D>
cudaError_t launch(const AppendProblem& p, cudaStream_t s)
{
    // A CTA per token spreads few tokens wide, one per four computes the angles
    // of many with every thread at work: 8 tokens 3.2 against 5.4 us, 256 4.1
    // against 5.6, 1024 8.2 against 8.8, 2048 12.5 against 13.5, 4096 26.3
    // against 22.0, 16001 96 against 70 (outputs in L2).
    constexpr int TT = 4;
    const bool few = p.n_tokens <= 1024;
    auto* kern = few ? kv_append_kernel<T, D, 1> : kv_append_kernel<T, D, TT>;
    const int64_t grid = few ? p.n_tokens : (p.n_tokens + TT - 1) / TT;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = static_cast<unsigned>(launch_attrs(attr, 1));
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kern, p);
    note_launch();
    return err;
}

}  // namespace

cudaError_t launch_kv_append(const AppendProblem& p, cudaStream_t s)
{
    if (p.dtype == SOFTMAX_BF16)
        return p.head_dim == 64 ? launch<BF16Bits, 64>(p, s) : launch<BF16Bits, 128>(p, s);
    return p.head_dim == 64 ? launch<F16Bits, 64>(p, s) : launch<F16Bits, 128>(p, s);
}

unsigned read_error_kv_append(bool clear)
{
    unsigned v = 0;
    if (cudaMemcpyFromSymbol(&v, g_error_kv_append, sizeof v) != cudaSuccess)
        return 0;
    if (clear && v) {
        const unsigned zero = 0;
        cudaMemcpyToSymbol(g_error_kv_append, &zero, sizeof zero);
    }
    return v;
}

}  // namespace rwsm
