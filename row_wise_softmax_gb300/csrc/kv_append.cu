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
// heads, 8 key/value heads of 128, bf16): 16001 tokens 64.2 us with inputs not
// in L2 (6.1 TB/s, a plain copy runs at 6.7); 256 tokens 4.2 us and 8 tokens 3.1,
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

// (a, b) turned by the angle of cosine c and sine s.
__device__ __forceinline__ void rotate(float& a, float& b, float c, float s)
{
    const float x = a, y = b;
    a = x * c - y * s;
    b = x * s + y * c;
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
    // Units that a thread has under way: with few CTAs on the device two keep
    // more bytes in flight (1024 tokens 8.5 -> 7.8 us), with many the registers
    // cost more than they bring (16001 tokens 64 -> 73 us).
    constexpr int kBatch = TT == 1 ? 2 : 1;
    __shared__ __align__(16) float2 turn[TT][kMaxHalf];
    __shared__ int64_t k_at[TT], v_at[TT];         // cache element of the token, < 0: none
    __shared__ int32_t pos_of[TT];
    const int tid = threadIdx.x;
    const int half = p.rot_dim / 2;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * TT;
    const int tokens = p.n_tokens - t0 < TT ? static_cast<int>(p.n_tokens - t0) : TT;

    pdl_launch_dependents();
    pdl_wait();
    const int nq = p.q.data ? p.n_heads : 0, nk = p.cache.n_kv_heads;
    const int per_token = (nq + 2 * nk) * U, units = per_token * tokens;
    // A thread's units, kBatch at a time: all of their loads are under way
    // before the first is used, those of the first batch before the tokens'
    // places and angles are known (a token that turns out to be padding is
    // read in vain).
    uint4 w0[kBatch], w1[kBatch];
    auto place = [&](int i, int& t, int& r, int& u) {
        t = TT == 1 ? 0 : i / per_token;
        r = (i - t * per_token) / U;
        u = i % U;
    };
    auto load = [&](int i0) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int i = i0 + b * kThreads;
            if (i >= units)
                continue;
            int t, r, u;
            place(i, t, r, u);
            // Which tensor this head row belongs to.
            const Heads& x = r < nq ? p.q : r < nq + nk ? p.k : p.v;
            const int head = r < nq ? r : r < nq + nk ? r - nq : r - nq - nk;
            const unsigned short* src = static_cast<const unsigned short*>(x.data) +
                                        (t0 + t) * x.row + head * x.head;
            const bool apart = r < nq + nk && u * 16 < p.rot_dim && !p.interleaved;
            w0[b] = *reinterpret_cast<const uint4*>(src + (apart ? u : 2 * u) * 8);
            w1[b] = *reinterpret_cast<const uint4*>(
                src + (apart ? u + p.rot_dim / 16 : 2 * u + 1) * 8);
        }
    };
    load(tid);
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

    for (int i0 = tid; i0 < units; i0 += kThreads * kBatch) {
        if (i0 != tid)
            load(i0);
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int i = i0 + b * kThreads;
            if (i >= units)
                continue;
            int t, r, u;
            place(i, t, r, u);
            if (pos_of[t] < 0)
                continue;
            unsigned short* dst;
            if (r < nq) {
                dst = static_cast<unsigned short*>(p.q_out.data) + (t0 + t) * p.q_out.row +
                      r * p.q_out.head;
            } else if (r < nq + nk) {
                if (k_at[t] < 0)
                    continue;
                dst = static_cast<unsigned short*>(p.cache.k) + k_at[t] +
                      (r - nq) * p.cache.k_head;
            } else {
                if (v_at[t] < 0)
                    continue;
                dst = static_cast<unsigned short*>(p.cache.v) + v_at[t] +
                      (r - nq - nk) * p.cache.v_head;
            }
            const bool turns = r < nq + nk && u * 16 < p.rot_dim;
            const bool apart = turns && !p.interleaved;
            if (turns) {
                float x[8], y[8];
                unpack8<T>(w0[b], x);
                unpack8<T>(w1[b], y);
                const float4* cs = reinterpret_cast<const float4*>(&turn[t][u * 8]);
                if (p.interleaved) {
#pragma unroll
                    for (int j = 0; j < 4; j += 2) {
                        const float4 f = cs[j / 2], g = cs[j / 2 + 2];
                        rotate(x[2 * j], x[2 * j + 1], f.x, f.y);
                        rotate(x[2 * j + 2], x[2 * j + 3], f.z, f.w);
                        rotate(y[2 * j], y[2 * j + 1], g.x, g.y);
                        rotate(y[2 * j + 2], y[2 * j + 3], g.z, g.w);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        const float4 f = cs[j / 2];
                        rotate(x[j], y[j], f.x, f.y);
                        rotate(x[j + 1], y[j + 1], f.z, f.w);
                    }
                }
                w0[b] = pack8<T>(x);
                w1[b] = pack8<T>(y);
            }
            *reinterpret_cast<uint4*>(dst + (apart ? u : 2 * u) * 8) = w0[b];
            *reinterpret_cast<uint4*>(dst + (apart ? u + p.rot_dim / 16 : 2 * u + 1) * 8) = w1[b];
        }
    }
}

template <typename T, int D>
cudaError_t launch(const AppendProblem& p, cudaStream_t s)
{
    // A CTA per token spreads few tokens wide (8 tokens 3.1 us; one per four
    // 5.4), one per two or four computes the angles of many with every thread
    // at work and ends in fewer waves: with 1, 2 and 4 tokens to a CTA, 2048
    // tokens take 13.9, 11.6 and 15.0 us, 4096 28.0, 20.8 and 22.5, 16001 95,
    // 67 and 64.
    const int64_t n = p.n_tokens;
    const int tt = n <= 1024 ? 1 : n <= 4096 ? 2 : 4;
    auto* kern = tt == 1   ? kv_append_kernel<T, D, 1>
                 : tt == 2 ? kv_append_kernel<T, D, 2>
                           : kv_append_kernel<T, D, 4>;
    const int64_t grid = (n + tt - 1) / tt;
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
