// Attention of whole prompts packed one behind the other, grouped heads:
// o_i = sum_j p_ij v_j, p = softmax over a query's visible keys of
// scale q_i . k_j, with the running softmax over key tiles: for each tile
//   m' = max(m, max_j s_j), l = l 2^(m - m') + sum_j 2^(s_j - m'),
//   O = O 2^(m - m') + P V,   s = scale log2(e) q . k,   o = O / l.
//
//   unit     two query tiles of 128 rows per CTA against all of their keys.
//            Rows are tokens x heads of one group (as many heads as the
//            largest power of two in it, at most 32), so that one K/V tile
//            serves them all.  At D = 128 a cluster of two CTAs shares each
//            product (cta_group::2: 256 rows, half of K's rows and of V's
//            columns in each CTA), which halves the shared memory per key and
//            leaves room for three tiles of 128 keys on the way.  At D = 64 a
//            CTA's own products are as fast and units half as large.
//   warps    one copies (tensor maps, a ring of K and V tiles), two issue the
//            products (one per query tile: what one waits, the other fills),
//            sixteen compute the softmax: two per row of each tile, 64 keys
//            each.  S of both tiles goes through one region of tensor memory
//            in turn, which keeps the tiles out of phase, so that one's
//            exponentials run beside the other's products; P has its own
//            columns and is the product's A operand from there, O stays there
//            (rescaled only when a maximum moves by more than 2^8).
//   order    CTAs (pairs) stay and take their next unit from the grid itself
//            by cluster launch control, the units with most key tiles first;
//            it is found while the one before is computed.  Lengths are on
//            the device, so a unit is found from the bounds there; the grid
//            is as large as the sizes allow, units past the last do nothing.
//   parts    when units are few and sequences long, a unit's keys are cut into
//            equal parts, computed side by side; a second kernel joins their
//            (m, l, O) in order.
//   output   O / l through shared memory by tensor-map copies (a warp's 32 rows x 32
//            columns), or 16-byte stores where rows of the tile belong to
//            no query of the sequence.
//
// Long prompts are bound by the tensor cores: 4 D operations per visible pair
// and head.  Measured (bf16, D = 128): 16384 tokens of 16 heads over 2, full
// 1284 us (1712 TFLOP/s, near the board's power limit), causal 648 us (1697);
// 4 x 4096 tokens of 16 heads, causal 208 us (1320); 16 ragged prompts up to
// 4096 of 32 heads over 8, 231 us (1246).  D = 64 has half the products per
// exponential: 4 x 4096 tokens full 300 us (917 TFLOP/s), causal 175 (785); the
// tensor pipe is 21% and the exponential pipe 21% busy at 24 x 500 tokens, and
// what warps wait for is each other (a tile's maxima, its product).  A unit's
// beginning and end cost 2.7 us beside its tiles, which is what short
// sequences pay: 24 x 500 tokens of 12 heads 37 us (four tiles of 1.4 us a
// unit, four units a CTA).  Calls of one unit: 90 tokens 9.6 us.
#include "cluster_ring.cuh"
#include "common.cuh"
#include "serving.h"
#include "tensor_map.h"
#include "cta_pair.cuh"

#include <atomic>
#include <type_traits>

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

// attend_row for query row `qrow`, head `head` over keys k0 .. k0 + n - 1, and
// its output and logsumexp.
template <typename T, int D>
__device__ __forceinline__ void attend_row_store(const PackedProblem& p, int64_t qrow, int head,
                                              int kvh, int64_t k0, int64_t n, float scale_log2)
{
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    float o[E], m, l;
    attend_row<T, D>(
        p, static_cast<const unsigned short*>(p.q.data) + qrow * p.q.row + head * p.q.head,
        static_cast<const unsigned short*>(p.k.data) + k0 * p.k.row + kvh * p.k.head,
        static_cast<const unsigned short*>(p.v.data) + k0 * p.v.row + kvh * p.v.head, n,
        scale_log2, o, m, l);
    const float inv = 1.0f / l;
    unsigned short* dst =
        static_cast<unsigned short*>(p.o.data) + qrow * p.o.row + head * p.o.head + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2)
        *reinterpret_cast<unsigned*>(dst + e) = Elem<T>::pack2(o[e] * inv, o[e + 1] * inv);
    if (p.lse && lane == 0)
        p.lse[qrow * p.n_heads + head] =
            l == 0.0f ? kNegInf : (m + __log2f(l)) * 0.69314718055994531f;
}

// The form for operands that have no tensor map (repeated rows, no key at
// all): a warp per (query, head) row.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
attention_packed_rows_kernel(const PackedProblem p, float scale_log2)
{
    const int warp = threadIdx.x >> 5;
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
            attend_row_store<T, D>(p, q0 + i, head, kvh, k0, n, scale_log2);
        }
        return;
    }
}

// ------------------------------------------------------- the tensor core kernel
constexpr int kBM = 128;                           // rows of a query tile (TMEM lanes)
constexpr float kLazyRescaleLog2 = 8.0f;           // p <= 2^8 between rescales
constexpr float kInf = __builtin_inff();

// CTAs that share each product, keys per tile, ring slots of K and of V.
template <int D> struct Shape;
template <> struct Shape<128> {
    static constexpr int CG = 2, BN = 128, KVS = 3;
};
template <> struct Shape<64> {
    static constexpr int CG = 1, BN = 128, KVS = 4;
};
constexpr int kHS = 2;                             // warps that share a row of S
constexpr int kSoftWarps = 2 * 4 * kHS;            // two query tiles of four TMEM lane groups
constexpr int kStageBytes = 32 * 64;               // a warp's place for 32 x 32 outputs

// Key tiles of a part, at least (of the middle query's keys: a causal prompt
// without context has half as many).  With 2, 4 and 8: 128 queries of 32 heads
// over 8 after 1920 keys 18.8, 22.4 and 24.0 us (31.3 whole), 4000 tokens of 2
// heads 25.0, 30.7 and 30.5 (53.1 whole).
constexpr int kPartTiles = 2;

constexpr int kPackedThreads = (kSoftWarps + 3) * 32;    // softmax, two MMA warps, copy

template <int D>
constexpr int packed_smem()
{
    using S = Shape<D>;
    return (2 * kBM * D + 2 * S::KVS * (S::BN / S::CG) * D) * 2 + kSoftWarps * kStageBytes + 1024;
}

// The unit of work of a CTA (pair): `tokens` query tokens of one sequence,
// for the GP heads of one block.
struct Unit {
    int32_t q0, n_q, k0, n_k;
    int32_t tile, head;                            // head: first of the block
    int32_t ok;
};

// A part of a unit: its key tiles [lo, hi), its sum's place.
struct UnitPart : Unit {
    int32_t lo, hi, slot;
};

// What the kernel does with a unit: all of its keys, all of them with the
// causal mask, or (either mask) one of the equal parts that its key tiles are
// cut into, whose unnormalised sum goes to the workspace for the join kernel.
enum : int { kFull = 0, kCausal = 1, kParts = 2 };

// A part's sum over a query tile, in the workspace: O as [D / 4][128 rows] of
// four columns (a warp's rows side by side), then (m, l) of each row.
template <int D>
struct PartSum {
    float4 o[D / 4][kBM];
    float2 ml[kBM];
};

// Number of a sequence's units (of 2^tok_log2 query tokens) that visit at least
// x key tiles of BN keys, and through `first` the first of them.
template <int BN>
__device__ __forceinline__ int32_t units_with(int32_t n_q, int32_t n_k, int tok_log2, bool causal,
                                              int32_t x, int32_t& first)
{
    const int32_t last = (1 << tok_log2) - 1;
    const int32_t units = static_cast<int32_t>((static_cast<uint32_t>(n_q) + last) >> tok_log2);
    first = 0;
    if (x <= 0)
        return units;
    if (units == 0 || (x - 1) * static_cast<int64_t>(BN) >= n_k)
        return 0;
    if (causal) {
        // Unit i's last query min((i + 1) tokens, n_q) - 1 sees key (x - 1) BN.
        const int64_t need = static_cast<int64_t>(x - 1) * BN - (n_k - n_q) + 1;
        if (need > last + 1)
            first = static_cast<int32_t>((need + last) >> tok_log2) - 1;
        if (first > units - 1)
            first = units - 1;
    }
    return units - first;
}

// Finds unit number `rank` in the order in which units are handed out, by a
// warp: the units that visit most key tiles first, so that the ones dispatched
// last are short.  The sequences' bounds are read once and kept in shared
// memory (in registers they made the copy warp spill); above kRanked sequences
// the order is that of the sequences instead, and the walk goes on from where
// the last one ended.
constexpr int kRanked = 128;

struct Bounds {
    int32_t q0[kRanked], n_q[kRanked], k0[kRanked], n_k[kRanked];
};

// Reports sequences with bad bounds, by a warp.
__device__ __forceinline__ void report_bounds(const PackedProblem& p)
{
    int64_t q, nq, k, nk;
    for (int64_t s = threadIdx.x & 31; s < p.n_seqs; s += 32)
        if (!sequence_of(p, s, q, nq, k, nk))
            atomicOr(&g_error_attention_packed, kErrBadIndex);
}

template <int BN>
struct UnitFinder {
    Bounds* b;
    bool ranked;
    int32_t most;                                  // most key tiles of a unit
    int64_t total;                                 // units (ranked), or past the end
    int64_t at, before;                            // unranked: sequence block, units before it

    // Bounds of sequence s into place i (of this lane).
    __device__ __forceinline__ void lengths(const PackedProblem& p, int64_t s, int i)
    {
        int64_t q = 0, nq = 0, k = 0, nk = 0;
        if (s < p.n_seqs)
            sequence_of(p, s, q, nq, k, nk);
        b->q0[i] = static_cast<int32_t>(q);
        b->n_q[i] = static_cast<int32_t>(nq);
        b->k0[i] = static_cast<int32_t>(k);
        b->n_k[i] = static_cast<int32_t>(nk);
    }

    // Units that visit at least x key tiles.
    __device__ __forceinline__ int32_t count(const PackedProblem& p, int tok_log2, int32_t x) const
    {
        int32_t n = 0, first;
        for (int i = threadIdx.x & 31; i < p.n_seqs; i += 32)
            n += units_with<BN>(b->n_q[i], b->n_k[i], tok_log2, p.causal, x, first);
        return static_cast<int32_t>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(n)));
    }

    __device__ void init(const PackedProblem& p, Bounds* bounds, int tok_log2, bool by_length)
    {
        const int lane = threadIdx.x & 31;
        b = bounds;
        ranked = by_length && p.n_seqs <= kRanked;
        at = before = 0;
        total = INT64_MAX;
        if (!ranked)
            return;
        int32_t longest = 0;
        for (int i = lane; i < kRanked; i += 32) {
            lengths(p, i, i);
            if (b->n_q[i] > 0)
                longest = max(longest, static_cast<int32_t>((b->n_k[i] + BN - 1u) / BN));
        }
        __syncwarp();
        most = __reduce_max_sync(0xffffffffu, longest);
        total = count(p, tok_log2, 0);
    }

    // The first of the 32 sequences in slot i whose units, n to a lane, hold
    // unit number `left`; subtracts the units passed from `left`.
    __device__ __forceinline__ int pick(int32_t n, int64_t& left, int64_t& passed)
    {
        const int lane = threadIdx.x & 31;
        int32_t upto = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t up = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o)
                upto += up;
        }
        const unsigned past = __ballot_sync(0xffffffffu, upto > left);
        passed = __shfl_sync(0xffffffffu, upto, 31);
        if (!past) {
            left -= passed;
            return -1;
        }
        const int lane_of = __ffs(past) - 1;
        left -= __shfl_sync(0xffffffffu, upto - n, lane_of);
        return lane_of;
    }

    __device__ __forceinline__ Unit unit(int i, int32_t tile) const
    {
        return Unit{b->q0[i], b->n_q[i], b->k0[i], b->n_k[i], tile, 0, 1};
    }

    __device__ Unit find(const PackedProblem& p, int64_t rank, int tok_log2)
    {
        const int lane = threadIdx.x & 31;
        Unit none = {};
        if (rank >= total)
            return none;
        int64_t passed;
        if (!ranked) {
            if (rank < before)
                at = before = 0;
            for (; at < p.n_seqs; at += 32) {
                __syncwarp();
                lengths(p, at + lane, lane);
                __syncwarp();
                int64_t left = rank - before;
                int32_t first;
                const int32_t n =
                    units_with<BN>(b->n_q[lane], b->n_k[lane], tok_log2, p.causal, 0, first);
                const int l = pick(n, left, passed);
                if (l >= 0)                        // longest first within the sequence
                    return unit(l, __shfl_sync(0xffffffffu, n, l) - 1 - static_cast<int32_t>(left));
                before += passed;
            }
            total = rank;
            at = before = 0;
            return none;
        }
        int32_t lo = 0, hi = most + 1, above = 0;  // count(lo) > rank >= count(hi) = above
        while (lo + 1 < hi) {
            const int32_t x = lo + (hi - lo) / 2, n = count(p, tok_log2, x);
            if (n > rank) {
                lo = x;
            } else {
                hi = x;
                above = n;
            }
        }
        int64_t left = rank - above;
        for (int i = lane; i - lane < p.n_seqs; i += 32) {
            int32_t first, next;
            int32_t n = units_with<BN>(b->n_q[i], b->n_k[i], tok_log2, p.causal, lo, first);
            n -= units_with<BN>(b->n_q[i], b->n_k[i], tok_log2, p.causal, lo + 1, next);
            const int l = pick(n, left, passed);
            if (l >= 0)
                return unit(i - lane + l,
                            __shfl_sync(0xffffffffu, first, l) + static_cast<int32_t>(left));
        }
        return none;
    }
};

template <typename T, int D, int MODE>
__global__ void __launch_bounds__(kPackedThreads, 1)
attention_packed_kernel(const __grid_constant__ CUtensorMap map_q,
                        const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ CUtensorMap map_v,
                        const __grid_constant__ CUtensorMap map_o,
                        const __grid_constant__ PackedProblem p, float scale_log2, int gp_log2,
                        int n_parts, int by_length)
{
    using S = Shape<D>;
    using Work = std::conditional_t<MODE == kParts, UnitPart, Unit>;
    const bool causal = MODE == kParts ? p.causal != 0 : MODE == kCausal;
    constexpr int CG = S::CG, BN = S::BN, KVS = S::KVS, HS = kHS;
    constexpr bool kBF16 = Elem<T>::kNegInfBits == 0xff80u;
    constexpr uint32_t QT_BYTES = kBM * D * 2;               // a query tile
    constexpr uint32_t KV_BYTES = BN / CG * D * 2;           // this CTA's part of a key tile
    constexpr int KR = BN / CG;                              // K rows of this CTA's part
    constexpr int VD = D / CG;                               // V columns of this CTA's part
    static_assert(VD == 64, "a V part is one 128-byte swizzle atom wide");
    constexpr uint32_t IDESC_S = umma_idesc(kBM * CG, BN, kBF16, false);
    constexpr uint32_t IDESC_PV = umma_idesc(kBM * CG, D, kBF16, true);
    // Tensor memory: S of either query tile (BN columns), P of each (BN / 2),
    // O of each (D).
    constexpr uint32_t P_COL = BN, O_COL = 2 * BN, TMEM_COLS = 512;
    static_assert(O_COL + 2 * D <= TMEM_COLS, "all of tensor memory");
    constexpr int CW = BN / HS;                              // keys of S per softmax warp
    constexpr int NCH = CW / 32;                             // 32-column chunks per warp
    constexpr int OW = D / HS;                               // O columns per softmax warp
    constexpr int SOFT = kSoftWarps, CTRL = SOFT, LOADW = CTRL + 2;    // first MMA warp, copy warp
    extern __shared__ __align__(128) unsigned char pk_smem[];
    __shared__ __align__(8) unsigned long long bar_s[2], bar_ld[2], bar_p[2], bar_pv[2];
    __shared__ __align__(8) unsigned long long o_free[2], bar_end, bar_drain[2];
    __shared__ __align__(8) unsigned long long q_full, q_free, k_full[KVS], v_full[KVS];
    __shared__ __align__(8) unsigned long long k_free[KVS], v_free[KVS];
    __shared__ __align__(8) unsigned long long unit_full[2], unit_free[2];
    __shared__ __align__(8) unsigned long long next_full[2], next_free[2];
    __shared__ __align__(16) uint4 s_next[2];                // answers of cluster launch control
    __shared__ Work s_unit[2];
    __shared__ Bounds s_bounds;
    __shared__ uint32_t tmem_slot;
    __shared__ int s_failed;
    __shared__ int s_stop[2][2];
    // Row maxima (by tile parity) and final sums of the warps sharing a row,
    // and their rows to be done again.
    __shared__ float xmax[2][2][HS][kBM];
    __shared__ float xsum[2][HS][kBM];
    __shared__ unsigned xredo[2][HS][4];

    const uint32_t base = (smem_addr(pk_smem) + 1023u) & ~1023u;   // swizzle atoms
    const uint32_t sQ = base, sK = sQ + 2 * QT_BYTES, sV = sK + KVS * KV_BYTES;
    const uint32_t sO = sV + KVS * KV_BYTES;                 // kStageBytes per softmax warp
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cta_rank<CG>();
    const int gp = 1 << gp_log2;
    const int tile_tokens = kBM >> gp_log2;                  // tokens of a query tile
    const int tokens = 2 * CG * tile_tokens;                 // of the unit

    if (warp == CTRL)
        tmem_alloc_group<CG>(smem_addr(&tmem_slot), TMEM_COLS);
    if (tid == 0) {
        for (int x = 0; x < 2; ++x) {
            mbar_init(smem_addr(&bar_s[x]), 1);
            mbar_init(smem_addr(&bar_p[x]), 4 * HS * CG);
            mbar_init(smem_addr(&bar_ld[x]), 4 * HS * CG);
            mbar_init(smem_addr(&bar_pv[x]), 1);
            mbar_init(smem_addr(&o_free[x]), 4 * HS * CG);
            mbar_init(smem_addr(&bar_drain[x]), 1);
            mbar_init(smem_addr(&unit_full[x]), 1);
            mbar_init(smem_addr(&unit_free[x]), SOFT + (rank == 0 ? 2 : 0));
            mbar_init(smem_addr(&next_full[x]), 1);
            mbar_init(smem_addr(&next_free[x]), CG);
        }
        mbar_init(smem_addr(&bar_end), 2 * 4 * HS * CG + 2);
        mbar_init(smem_addr(&q_full), 1);
        mbar_init(smem_addr(&q_free), 2);
        for (int x = 0; x < KVS; ++x) {
            mbar_init(smem_addr(&k_full[x]), 1);
            mbar_init(smem_addr(&v_full[x]), 1);
            mbar_init(smem_addr(&k_free[x]), 2);
            mbar_init(smem_addr(&v_free[x]), 2);
        }
        s_failed = 0;
        fence_mbar_init();
    }
    tc_fence_before();
    group_sync<CG>();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    pdl_launch_dependents();
    pdl_wait();

    if (blockIdx.x == 0 && warp == CTRL)
        report_bounds(p);

    auto fail = [&] { *reinterpret_cast<volatile int*>(&s_failed) = 1; };
    auto failed_elsewhere = [&] {
        return __any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&s_failed) != 0) != 0;
    };
    // Every wait: by a whole warp in uniform control flow, bounded; after one
    // that ran out the warp waits for nothing more.
    bool failed = false;
    auto wait1 = [&](unsigned long long* bar, uint32_t parity) {
        if (!failed && __any_sync(0xffffffffu, !mbar_wait_bounded(smem_addr(bar), parity & 1u))) {
            failed = true;
            fail();
        }
    };
    // Key tiles that query tile x of a unit visits (both CTAs' parts of it),
    // -1 when it has no tokens at all.
    auto all_tiles_of = [&](const Unit& u, int x) -> int32_t {
        const int32_t begin = u.tile * tokens + x * CG * tile_tokens;
        if (u.ok <= 0 || begin >= u.n_q)
            return -1;
        int32_t lim = u.n_k;
        if (causal)
            lim = min(lim, min(begin + CG * tile_tokens, u.n_q) + u.n_k - u.n_q);
        return lim <= 0 ? 0 : (lim + BN - 1) / BN;
    };
    // Those that it visits here: all of them, or those of the unit's part.
    auto tiles_of = [&](const Work& u, int x) -> int32_t {
        const int32_t n = all_tiles_of(u, x);
        if constexpr (MODE == kParts)
            return n <= 0 ? n : max(min(n, u.hi) - u.lo, 0);
        return n;
    };
    // Keys before the first of them, and its first key row.
    auto skipped_of = [](const Work& u) -> int32_t {
        if constexpr (MODE == kParts)
            return u.lo * BN;
        return 0;
    };
    auto key0_of = [&](const Work& u) { return u.k0 + skipped_of(u); };
    // Tile number t, counted through all units, lies in ring slot t % KVS.
    auto slot = [](uint32_t t) { return t % KVS; };
    auto phase = [](uint32_t t) { return (t / KVS) & 1u; };
    const int group = p.n_heads / p.n_kv_heads;

    if (warp == LOADW) {
        // --------------------------------------------------------- copy warp
        // Hands out the units (its own cluster's, then those of clusters not
        // yet launched, which it takes over one at a time) and copies their
        // operands.  Each CTA copies its own query tiles, its rows of K and
        // its columns of V; all complete on the even CTA's barriers, where
        // the bytes of both are announced.
        const bool one = lane == 0;
        const int tok_log2 = 8 + (CG - 1) - gp_log2;
        const uint32_t blocks = static_cast<uint32_t>(p.n_heads) >> gp_log2;
        UnitFinder<BN> finder;
        finder.init(p, &s_bounds, tok_log2, MODE != kParts && by_length != 0);
        auto find = [&](uint32_t cta) {
            const uint32_t slot = cta / CG, index = MODE == kParts ? slot / n_parts : slot;
            const uint32_t unit = index / blocks;
            Work u = {finder.find(p, unit, tok_log2)};
            u.head = static_cast<int32_t>((index - unit * blocks) << gp_log2);
            if constexpr (MODE == kParts) {
                const int64_t n = max(0, max(all_tiles_of(u, 0), all_tiles_of(u, 1)));
                const int64_t part = slot - index * n_parts;
                u.lo = static_cast<int32_t>(n * part / n_parts);
                u.hi = static_cast<int32_t>(n * (part + 1) / n_parts);
                u.slot = static_cast<int32_t>(slot);
            }
            return u;
        };
        uint32_t kv = 0, q_uses = 0;
        auto announce = [&](unsigned long long* bar, uint32_t bytes) {
            if (one && rank == 0)
                mbar_arrive_expect_tx(smem_addr(bar), bytes * CG);
            return leader_addr<CG>(smem_addr(bar));
        };
        Work u = find(blockIdx.x);
        for (uint32_t i = 0; !failed; ++i) {
            if (i >= 2)
                wait1(&unit_free[i & 1], (i - 2) >> 1);
            if (one) {
                s_unit[i & 1] = u;
                mbar_arrive(smem_addr(&unit_full[i & 1]));
            }
            if (u.ok < 0)
                break;                                       // no unit is left, and all know
            // Ask for the next unit: the answer of two units ago has been
            // read by both CTAs.
            if (one)
                mbar_arrive_expect_tx(smem_addr(&next_full[i & 1]), 16);
            if (rank == 0) {
                if (i >= 2)
                    wait1(&next_free[i & 1], (i - 2) >> 1);
                if (one)
                    clc_try_cancel<CG>(smem_addr(&s_next[i & 1]), smem_addr(&next_full[i & 1]));
            }
            const int32_t n_kt = max(tiles_of(u, 0), tiles_of(u, 1));
            const int kvh = u.head / group;
            Work next = {};
            if (n_kt > 0) {
                if (q_uses > 0)
                    wait1(&q_free, q_uses - 1);
                ++q_uses;
                const uint32_t bar_q = announce(&q_full, 2 * QT_BYTES);
                if (one && !failed) {
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int c = 0; c < D / 64; ++c)
                            tma_load_3d<CG>(sQ + x * QT_BYTES + c * (kBM * 128), &map_q, c * 64,
                                            u.head, u.q0 + u.tile * tokens +
                                            (x * CG + static_cast<int>(rank)) * tile_tokens, bar_q);
                }
            }
            for (int32_t t = 0; t < max(n_kt, 1) && !failed; ++t) {
                if (t < n_kt) {
                    if (kv >= KVS)
                        wait1(&k_free[slot(kv)], (kv - KVS) / KVS);          // every S done
                    const uint32_t bar_k = announce(&k_full[slot(kv)], KV_BYTES);
                    if (one && !failed) {
#pragma unroll
                        for (int c = 0; c < D / 64; ++c)
                            tma_load_3d<CG>(sK + slot(kv) * KV_BYTES + c * (KR * 128), &map_k,
                                            c * 64, kvh, key0_of(u) + t * BN +
                                            static_cast<int>(rank) * KR, bar_k);
                    }
                    if (kv >= KVS)
                        wait1(&v_free[slot(kv)], (kv - KVS) / KVS);          // every P V done
                    const uint32_t bar_v = announce(&v_full[slot(kv)], KV_BYTES);
                    if (one && !failed)
                        tma_load_3d<CG>(sV + slot(kv) * KV_BYTES, &map_v,
                                        static_cast<int>(rank) * VD, kvh, key0_of(u) + t * BN, bar_v);
                    ++kv;
                }
                // The answer (both CTAs get the same), and which unit that
                // is, while the ring is full and long before it is wanted.
                if (t == min(KVS, max(n_kt, 1)) - 1) {
                    const bool answered = __all_sync(
                        0xffffffffu, mbar_wait_bounded(smem_addr(&next_full[i & 1]), (i >> 1) & 1u));
                    int64_t cta = -1;
                    if (answered)
                        cta = clc_first_cta(smem_addr(&s_next[i & 1]));
                    else
                        fail();
                    fence_proxy_async_smem();                // read before it is written again
                    __syncwarp();
                    if (one)
                        mbar_arrive_leader<CG>(leader_addr<CG>(smem_addr(&next_free[i & 1])));
                    if (cta >= 0)
                        next = find(static_cast<uint32_t>(cta));
                    else
                        next.ok = -1;
                }
                if (failed_elsewhere())
                    failed = true;
            }
            u = next;
        }
        if (rank == 0 && failed_elsewhere()) {
            // Let the copies still in flight land (bounded; after one wait
            // that ran out the others are not waited for).
            failed = false;
            if (q_uses > 0)
                wait1(&q_full, q_uses - 1);
            for (uint32_t t = kv > KVS ? kv - KVS : 0; t < kv; ++t) {
                wait1(&k_full[slot(t)], phase(t));
                wait1(&v_full[slot(t)], phase(t));
            }
        }
    } else if (warp == CTRL || warp == CTRL + 1) {
        // --------------------------------------------------------- MMA warps
        // The even CTA's warps issue every product, a warp for each query
        // tile: a product's issue lasts nearly as long as the product (the
        // tensor core queues one or two), so what one warp spends on waits
        // is filled by the other's products.  They run their loops as whole
        // warps (see umma_f16_warp).
        const int x = warp - CTRL;
        // A 16-element step of Q or K is 32 bytes into the 128-byte atom row,
        // of V (MN-major) 16 key rows.
        const uint64_t dq = smem_desc_sw128(sQ + x * QT_BYTES, 16, 1024);
        const uint64_t dk = smem_desc_sw128(sK, 16, 1024), dv = smem_desc_sw128(sV, 16, 1024);
        const uint32_t tp = tmem + P_COL + static_cast<uint32_t>(x * (BN / 2));
        const uint32_t to = tmem + O_COL + static_cast<uint32_t>(x * D);
        // A wait is on the parity of a phase, so no warp may fall two phases
        // behind a barrier that it waits on.  Within a unit the two tiles'
        // products alternate; past a tile's own last key tile its warp still
        // waits for every K and V and gives it back, and bar_end, which both
        // warps and every softmax warp arrive at, closes the unit's S columns.
        // Of the units before: key tiles, S products of this query tile and
        // of the other, units with work for this tile, units with any.
        uint32_t kv = 0, done = 0, done_other = 0, units = 0, q_uses = 0;
        for (uint32_t i = 0; rank == 0 && !failed; ++i) {
            wait1(&unit_full[i & 1], i >> 1);
            if (failed)
                break;
            const Work u = s_unit[i & 1];
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_addr(&unit_free[i & 1]));
            if (u.ok < 0)
                break;
            const int32_t mine = max(tiles_of(u, x), 0), other = max(tiles_of(u, 1 - x), 0);
            // S of tile t.  The product before it into the same columns has
            // been read by its softmax warps when the wait on bar_ld is over.
            auto next_s = [&](int32_t t) {
                const uint32_t k = kv + static_cast<uint32_t>(t);
                wait1(&k_full[slot(k)], phase(k));
                const int32_t before = x == 0 ? t - 1 : t;   // the other tile's
                if (before >= 0 && before < other)
                    wait1(&bar_ld[1 - x], done_other + static_cast<uint32_t>(before));
                else if (t > 0)
                    wait1(&bar_ld[x], done + static_cast<uint32_t>(t - 1));
                if (failed)
                    return;
                tc_fence_after();
                const uint64_t b = dk + slot(k) * (KV_BYTES >> 4);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    umma_f16_warp<CG>(tmem, dq + ((ks >> 2) * (kBM * 128) + (ks & 3) * 32) / 16,
                                      b + ((ks >> 2) * (KR * 128) + (ks & 3) * 32) / 16, IDESC_S,
                                      ks > 0 ? 1u : 0u);
                umma_commit_warp<CG>(smem_addr(&bar_s[x]));
                umma_commit_warp<CG>(smem_addr(&k_free[slot(k)]));
                if (t + 1 == mine)
                    umma_commit_warp<CG>(smem_addr(&q_free));
            };
            if (i > 0)
                wait1(&bar_end, i - 1);                      // every S of the unit before is read
            if (mine > 0 || other > 0)
                wait1(&q_full, q_uses++);
            if (mine > 0)
                next_s(0);
            else if (other > 0)
                umma_commit_warp<CG>(smem_addr(&q_free));
            for (int32_t t = 0; t < mine && !failed; ++t) {
                if (t + 1 < mine)
                    next_s(t + 1);
                const uint32_t k = kv + static_cast<uint32_t>(t);
                wait1(&v_full[slot(k)], phase(k));
                if (t == 0 && units > 0)
                    wait1(&o_free[x], units - 1);            // O of the unit before has been read
                wait1(&bar_p[x], done + static_cast<uint32_t>(t));
                if (failed)
                    break;
                tc_fence_after();
                const uint64_t b = dv + slot(k) * (KV_BYTES >> 4);
#pragma unroll
                for (int ks = 0; ks < BN / 16; ++ks)
                    umma_f16_ta_warp<CG>(to, tp + ks * 8, b + ks * (2048 / 16), IDESC_PV,
                                         t == 0 && ks == 0 ? 0u : 1u);
                umma_commit_warp<CG>(smem_addr(&bar_pv[x]));
                umma_commit_warp<CG>(smem_addr(&v_free[slot(k)]));
            }
            for (int32_t t = mine; t < other && !failed; ++t) {
                const uint32_t k = kv + static_cast<uint32_t>(t);
                wait1(&k_full[slot(k)], phase(k));
                umma_commit_warp<CG>(smem_addr(&k_free[slot(k)]));
                wait1(&v_full[slot(k)], phase(k));
                umma_commit_warp<CG>(smem_addr(&v_free[slot(k)]));
            }
            if (lane == 0)
                mbar_arrive(smem_addr(&bar_end));
            kv += static_cast<uint32_t>(max(mine, other));
            done += static_cast<uint32_t>(mine);
            done_other += static_cast<uint32_t>(other);
            units += mine > 0 ? 1u : 0u;
        }
    } else {
        // ---------------------------------------------------- softmax warps
        // Warp w: query tile x, TMEM lane group w % 4 (rows 32 (w % 4) ..),
        // and part h of the tile's keys and of O's columns when HS warps
        // share a row.
        const int x = warp / (4 * HS), h = (warp / 4) % HS;
        const int r = (warp & 3) * 32 + lane;                // row of the tile = TMEM lane
        const uint32_t t_row = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t s_col = static_cast<uint32_t>(h * CW);
        const uint32_t p_col = P_COL + static_cast<uint32_t>((x * BN + h * CW) / 2);
        const uint32_t o_col = O_COL + static_cast<uint32_t>(x * D + h * OW);
        const int pair_bar = 5 + x * 4 + (warp & 3);         // the HS warps of 32 rows
        const uint32_t bar_loaded = leader_addr<CG>(smem_addr(&bar_ld[x]));
        const uint32_t bar_weights = leader_addr<CG>(smem_addr(&bar_p[x]));
        const uint32_t bar_over = leader_addr<CG>(smem_addr(&bar_end));
        const uint32_t bar_output = leader_addr<CG>(smem_addr(&o_free[x]));
        const uint32_t stage = sO + static_cast<uint32_t>(warp * kStageBytes);
        // One warp of a tile waits on the barriers in shared memory, the
        // others behind it at a named barrier: sixteen polling warps slow the
        // exponentials down (d = 128, 16384 tokens: 1677 -> 1744 TFLOP/s).
        const bool poller = warp % (4 * HS) == 0;
        auto await = [&](int id, unsigned long long* bar, uint32_t parity, bool wait) {
            if (wait && poller)
                wait1(bar, parity);
            named_barrier(id, 128 * HS);
        };
        uint32_t done = 0;                                   // key tiles of the units before
        for (uint32_t i = 0;; ++i) {
            // The tile's warps stop together (they meet at named barriers): the
            // one that waits says so, in the slot of this unit.
            if (poller) {
                wait1(&unit_full[i & 1], i >> 1);
                const int stop = failed_elsewhere();
                if (lane == 0)
                    s_stop[i & 1][x] = stop;
                __syncwarp();
            }
            named_barrier(1 + x, 128 * HS);
            if (s_stop[i & 1][x])
                break;
            const Work u = s_unit[i & 1];
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_addr(&unit_free[i & 1]));
            if (u.ok < 0)
                break;
            const int32_t my_kt = tiles_of(u, x);
            if (my_kt <= 0 && lane == 0)
                mbar_arrive_leader<CG>(bar_over);
            if (my_kt < 0)
                continue;
            const int32_t off = u.n_k - u.n_q;
            const int32_t first = u.tile * tokens + (x * CG + static_cast<int>(rank)) * tile_tokens;
            const int32_t token = first + (r >> gp_log2);    // of the sequence
            // Keys visible to this row, and to every row of the tile (counted
            // from the first of the part).
            const int32_t skipped = skipped_of(u);
            const int32_t limit = (causal ? min(u.n_k, token + off + 1) : u.n_k) - skipped;
            const int32_t limit_all = (causal ? min(u.n_k, first + off + 1) : u.n_k) - skipped;
            float m = kNegInf, l = 0.0f;                     // l: this warp's part of the sum
            for (int32_t t = 0; t < my_kt; ++t) {
                await(1 + x, &bar_s[x], done + static_cast<uint32_t>(t), true);
                tc_fence_after();
                float sv[NCH][32];
#pragma unroll
                for (int c = 0; c < NCH; ++c)
                    tmem_ld32(t_row + s_col + c * 32, sv[c]);
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {                             // S may be overwritten
                    mbar_arrive_leader<CG>(bar_loaded);
                    if (t + 1 == my_kt)
                        mbar_arrive_leader<CG>(bar_over);
                }
                if ((t + 1) * BN > limit_all) {              // some row has a masked key
                    const int32_t keep = limit - t * BN - h * CW;
#pragma unroll
                    for (int c = 0; c < NCH; ++c)
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (c * 32 + j >= keep)
                                sv[c][j] = kNegInf;
                }
                float mx = kNegInf;
#pragma unroll
                for (int c = 0; c < NCH; ++c)
#pragma unroll
                    for (int j = 0; j < 32; j += 2)
                        mx = max3(mx, sv[c][j], sv[c][j + 1]);
                // The row's maximum over its HS warps (slots by tile parity);
                // and P V of the tile before has read P and written O.
                xmax[t & 1][x][h][r] = mx;
                await(3 + x, &bar_pv[x], done + static_cast<uint32_t>(t - 1), t > 0);
                tc_fence_after();
#pragma unroll
                for (int o = 0; o < HS; ++o)
                    mx = fmaxf(mx, xmax[t & 1][x][o][r]);
                // Lazy rescaling: the reference m (base 2) moves only when the
                // tile's max exceeds it by more than 2^8; O / l and the
                // logsumexp only need m and l to agree.
                const float mx_s = mx * scale_log2;
                float alpha = 1.0f;
                if (mx_s > m + kLazyRescaleLog2) {
                    alpha = ex2_ftz(m - mx_s);
                    m = mx_s;
                }
                const float nref = m == kNegInf ? 0.0f : -m;
                if (t > 0 && !__all_sync(0xffffffffu, alpha == 1.0f)) {
#pragma unroll 1
                    for (int c = 0; c < OW; c += 8)
                        tmem_scale8(t_row + o_col + c, alpha);
                }
                float sum0 = 0.0f, sum1 = 0.0f;
#pragma unroll
                for (int c = 0; c < NCH; ++c) {
                    uint32_t w[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float p0, p1;
                        fma2(p0, p1, sv[c][2 * j], sv[c][2 * j + 1], scale_log2, scale_log2, nref,
                             nref);
                        p0 = ex2_ftz(p0);
                        p1 = ex2_ftz(p1);
                        add2(sum0, sum1, sum0, sum1, p0, p1);
                        w[j] = Elem<T>::pack2(p0, p1);
                    }
                    tmem_st16(t_row + p_col + c * 16, w);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_leader<CG>(bar_weights);     // release: P written, O rescaled
                l = l * alpha + (sum0 + sum1);
            }
            // ---- O / l to global memory, logsumexp
            if (my_kt > 0) {
                await(1 + x, &bar_pv[x], done + static_cast<uint32_t>(my_kt - 1), true);
                tc_fence_after();
            }
            done += static_cast<uint32_t>(my_kt);
            xsum[x][h][r] = l;
            named_barrier(pair_bar, 32 * HS);
            l = 0.0f;
#pragma unroll
            for (int o = 0; o < HS; ++o)
                l += xsum[x][o][r];
            // A masked key's weight is 0, but 0 times an infinite or NaN value
            // of V is NaN.  Rows with a value of O that is not finite, and
            // such a value in the masked part of their key tiles, are done
            // again over their visible keys alone, after the others have been
            // stored; where o is q, nothing may be stored in them before.
            const bool in_place = MODE != kParts && p.o.data == p.q.data;
            float zero0 = 0.0f, zero1 = 0.0f;                // 0 * O: NaN unless O is finite
            auto add_zeros = [&](const float (&v)[32]) {
#pragma unroll
                for (int j = 0; j < 32; j += 2)
                    fma2(zero0, zero1, v[j], v[j + 1], 0.0f, 0.0f, zero0, zero1);
            };
            if (in_place && my_kt > 0) {
#pragma unroll 1
                for (int c = 0; c < OW / 32; ++c) {
                    float ov[32];
                    tmem_ld32(t_row + o_col + c * 32, ov);
                    tmem_wait_ld();
                    add_zeros(ov);
                }
            }
            const bool broken = failed_elsewhere();          // then nothing is stored
            const unsigned seen = __ballot_sync(0xffffffffu, token < u.n_q && limit > 0 && !broken);
            unsigned rows = __ballot_sync(0xffffffffu, token < u.n_q && !broken);
            // The rows that any of the HS warps found not finite.
            auto not_finite = [&] {
                unsigned redo = __ballot_sync(0xffffffffu, !(zero0 + zero1 == 0.0f)) & seen;
                if (lane == 0)
                    xredo[x][h][warp & 3] = redo;
                named_barrier(pair_bar, 32 * HS);
#pragma unroll
                for (int o = 0; o < HS; ++o)
                    redo |= xredo[x][o][warp & 3];
                named_barrier(pair_bar, 32 * HS);            // read before it is written again
                return redo;
            };
            const int kvh = u.head / group;
            // Of those, the ones with such a V in the masked part.
            auto leaked = [&](unsigned redo) {
                if (redo) {
                    const unsigned short* const v = static_cast<const unsigned short*>(p.v.data) +
                                                    static_cast<int64_t>(key0_of(u)) * p.v.row +
                                                    kvh * p.v.head;
                    const int32_t from = __reduce_min_sync(0xffffffffu,
                                                           redo >> lane & 1 ? limit : 0x7fffffff);
                    const int64_t to =
                        min(static_cast<int64_t>(my_kt) * BN, p.total_k - key0_of(u));
                    bool hit = false;
                    for (int64_t e = static_cast<int64_t>(from) * (D / 2) + lane; e < to * (D / 2);
                         e += 32) {
                        float a, b;
                        Elem<T>::unpack2(__ldg(reinterpret_cast<const unsigned*>(
                                             v + (e / (D / 2)) * p.v.row + (e % (D / 2)) * 2)),
                                         a, b);
                        hit = hit || !(fabsf(a) < kInf) || !(fabsf(b) < kInf);
                    }
                    if (!__any_sync(0xffffffffu, hit))
                        redo = 0;
                }
                return redo;
            };
            unsigned redo = 0;
            if constexpr (MODE == kParts) {
                // The sum as it is; a row that has to be done again over what
                // it sees of the part replaces its own.
                auto* const sum = static_cast<PartSum<D>*>(p.workspace) +
                                  (static_cast<int64_t>(u.slot) * 2 + x) * CG + rank;
#pragma unroll 1
                for (int c = 0; c < OW / 32; ++c) {
                    float ov[32];
                    tmem_ld32(t_row + o_col + c * 32, ov);
                    tmem_wait_ld();
                    add_zeros(ov);
                    if (!broken)
#pragma unroll
                        for (int g = 0; g < 8; ++g)
                            sum->o[(h * OW + c * 32) / 4 + g][r] =
                                make_float4(ov[4 * g], ov[4 * g + 1], ov[4 * g + 2], ov[4 * g + 3]);
                }
                if (my_kt > 0) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive_leader<CG>(bar_output);  // O may be overwritten
                }
                if (h == 0 && !broken)
                    sum->ml[r] = make_float2(m, l);          // (-inf, 0): nothing was seen
                redo = not_finite();
                redo = my_kt > 0 ? leaked(redo) : 0;
                if (redo)
                    named_barrier(pair_bar, 32 * HS);        // after the stores above
                while (redo && h == 0) {
                    const int row = (warp & 3) * 32 + __ffs(redo) - 1;
                    redo &= redo - 1;
                    const int32_t tok = first + (row >> gp_log2);
                    const int32_t sees = (causal ? min(u.n_k, tok + off + 1) : u.n_k) - skipped;
                    constexpr int E = D / 32;
                    float ov[E], rm, rl;
                    attend_row<T, D>(
                        p,
                        static_cast<const unsigned short*>(p.q.data) +
                            (u.q0 + static_cast<int64_t>(tok)) * p.q.row +
                            (u.head + (row & (gp - 1))) * p.q.head,
                        static_cast<const unsigned short*>(p.k.data) +
                            static_cast<int64_t>(key0_of(u)) * p.k.row + kvh * p.k.head,
                        static_cast<const unsigned short*>(p.v.data) +
                            static_cast<int64_t>(key0_of(u)) * p.v.row + kvh * p.v.head,
                        min(sees, my_kt * BN), scale_log2, ov, rm, rl);
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        reinterpret_cast<float*>(&sum->o[(lane * E + e) / 4][row])[(lane * E + e) %
                                                                                    4] = ov[e];
                    if (lane == 0)
                        sum->ml[row] = make_float2(rm, rl);
                }
                continue;
            }
            if (in_place) {
                redo = leaked(not_finite());
                rows &= ~redo;
            }
            // A row that sees no key is the softmax of only -inf: NaN.
            const float inv = limit > 0 ? 1.0f / l : __int_as_float(0x7fc00000);
            // 32 columns of 32 rows at a time go through shared memory (64-byte
            // rows in the copy engine's 64-byte swizzle: 16-byte chunks XORed
            // by row pair).  When every row is stored, one tensor-map copy
            // takes them from there and the warp goes on; else each row of 64
            // bytes is stored by four lanes.
            auto staged = [&](int row, int chunk) {
                return stage + static_cast<uint32_t>(row * 64) + ((chunk ^ ((row / 2) % 4)) << 4);
            };
            const bool all_rows = rows == 0xffffffffu;
#pragma unroll 1
            for (int c = 0; c < OW / 32; ++c) {
                float ov[32];
                tmem_ld32(t_row + o_col + c * 32, ov);       // (no key tile: anything, times NaN)
                tmem_wait_ld();
                if (c + 1 == OW / 32 && my_kt > 0) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive_leader<CG>(bar_output);  // O may be overwritten
                }
                add_zeros(ov);
                if (lane == 0)                               // the copy before has read its rows
                    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                __syncwarp();
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const float* f = ov + g * 8;
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                                 :: "r"(staged(lane, g)),
                                    "r"(Elem<T>::pack2(f[0] * inv, f[1] * inv)),
                                    "r"(Elem<T>::pack2(f[2] * inv, f[3] * inv)),
                                    "r"(Elem<T>::pack2(f[4] * inv, f[5] * inv)),
                                    "r"(Elem<T>::pack2(f[6] * inv, f[7] * inv)) : "memory");
                }
                if (all_rows) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        asm volatile(
                            "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group"
                            " [%0, {%1, %2, %3}], [%4];\n\tcp.async.bulk.commit_group;"
                            :: "l"(reinterpret_cast<uint64_t>(&map_o)), "r"(h * OW + c * 32),
                               "r"(u.head), "r"(u.q0 + first + ((warp & 3) * 32 >> gp_log2)),
                               "r"(stage) : "memory");
                } else {
                    __syncwarp();
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const int q = g * 8 + lane / 4, row = (warp & 3) * 32 + q;
                        uint4 w;
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                                     : "r"(staged(q, lane % 4)) : "memory");
                        if (rows >> q & 1)
                            *reinterpret_cast<uint4*>(
                                static_cast<unsigned short*>(p.o.data) +
                                (u.q0 + static_cast<int64_t>(first + (row >> gp_log2))) * p.o.row +
                                (u.head + (row & (gp - 1))) * p.o.head + h * OW + c * 32 +
                                lane % 4 * 8) = w;
                    }
                }
            }
            if (!in_place) {
                redo = leaked(not_finite());
                if (redo) {                                  // after the copies that are under way
                    if (lane == 0)
                        asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
                    named_barrier(pair_bar, 32 * HS);
                }
            }
            if (p.lse && h == 0 && (rows >> lane & 1))
                p.lse[(u.q0 + static_cast<int64_t>(token)) * p.n_heads + u.head + (r & (gp - 1))] =
                    limit > 0 && l != 0.0f ? (m + __log2f(l)) * 0.69314718055994531f : kNegInf;
            while (redo && h == 0) {
                const int row = (warp & 3) * 32 + __ffs(redo) - 1;
                redo &= redo - 1;
                const int32_t tok = first + (row >> gp_log2);
                attend_row_store<T, D>(p, u.q0 + static_cast<int64_t>(tok),
                                       u.head + (row & (gp - 1)), kvh, u.k0,
                                       causal ? min(u.n_k, tok + off + 1) : u.n_k, scale_log2);
            }
        }
        if (lane == 0)                                       // shared memory has been read
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    if ((warp == CTRL || warp == CTRL + 1) && failed_elsewhere()) {
        if (lane == 0)
            atomicOr(&g_error_attention_packed, kErrMbarrierTimeout);
        if (rank == 0) {
            // One more commit: it arrives once every tensor core operation
            // this warp has issued has completed; wait for it (bounded)
            // before tensor memory is freed.
            tc_fence_after();
            umma_commit_warp<CG>(smem_addr(&bar_drain[warp - CTRL]));
            mbar_wait_bounded(smem_addr(&bar_drain[warp - CTRL]), 0u);
        }
        __syncwarp();
    }
    tc_fence_before();
    group_sync<CG>();
    if (warp == CTRL) {
        tc_fence_after();
        tmem_dealloc_group<CG>(tmem, TMEM_COLS);
    }
}

// The rows of a unit from its parts, in their order: blockIdx.x counts units
// and blocks of heads as the parts' kernel does, blockIdx.y blocks of rows; a
// thread takes four columns of one.
constexpr int kJoinThreads = 256;
template <int D> __host__ __device__ constexpr int join_rows() { return kJoinThreads * 4 / D; }

template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads)
attention_packed_join_kernel(const __grid_constant__ PackedProblem p, int gp_log2, int n_parts)
{
    constexpr int CG = Shape<D>::CG, ROWS = join_rows<D>();
    __shared__ Bounds s_bounds;
    __shared__ Unit s_unit;
    const int tid = threadIdx.x;
    const int tile_tokens = kBM >> gp_log2;
    const uint32_t blocks = static_cast<uint32_t>(p.n_heads) >> gp_log2;
    pdl_launch_dependents();
    pdl_wait();
    if (tid < 32) {
        const int tok_log2 = 8 + (CG - 1) - gp_log2;
        UnitFinder<Shape<D>::BN> finder;
        finder.init(p, &s_bounds, tok_log2, false);
        const Unit u = finder.find(p, blockIdx.x / blocks, tok_log2);
        if (tid == 0)
            s_unit = u;
    }
    __syncthreads();
    const Unit u = s_unit;
    const int at = blockIdx.y * ROWS, part_tile = at / kBM;      // query tile x CG + rank
    const int r = at % kBM + tid % ROWS, c4 = tid / ROWS;
    const int32_t token = (u.tile * 2 * CG + part_tile) * tile_tokens + (r >> gp_log2);
    if (u.ok <= 0 || token >= u.n_q)
        return;
    const auto* const sum = static_cast<const PartSum<D>*>(p.workspace) +
                            static_cast<int64_t>(blockIdx.x) * n_parts * 2 * CG + part_tile;
    float m = kNegInf, l = 0.0f;
#pragma unroll 4
    for (int i = 0; i < n_parts; ++i)
        m = fmaxf(m, sum[i * 2 * CG].ml[r].x);
    const float ref = m == kNegInf ? 0.0f : m;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int i = 0; i < n_parts; ++i) {
        const float2 ml = sum[i * 2 * CG].ml[r];
        const float4 v = sum[i * 2 * CG].o[c4][r];
        if (ml.x == kNegInf && ml.y == 0.0f)       // saw nothing (what lies there may be anything)
            continue;
        const float f = ex2_ftz(ml.x - ref);
        l += ml.y * f;
        o.x += v.x * f; o.y += v.y * f; o.z += v.z * f; o.w += v.w * f;
    }
    const float inv = 1.0f / l;                    // nothing seen at all: 0 / 0, NaN
    const int head = static_cast<int>((blockIdx.x % blocks) << gp_log2) + (r & ((1 << gp_log2) - 1));
    const int64_t row = u.q0 + static_cast<int64_t>(token);
    uint2 w;
    w.x = Elem<T>::pack2(o.x * inv, o.y * inv);
    w.y = Elem<T>::pack2(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2*>(static_cast<unsigned short*>(p.o.data) + row * p.o.row +
                              static_cast<int64_t>(head) * p.o.head + c4 * 4) = w;
    if (p.lse && c4 == 0)
        p.lse[row * p.n_heads + head] =
            l == 0.0f ? kNegInf : (m + __log2f(l)) * 0.69314718055994531f;
}

// How a call's work is laid out: heads of a group that share a tile's rows (a
// power of two), units, and the parts that each unit's keys are cut into.
struct PackedShape {
    int gp_log2, parts;
    int64_t units;                                 // of all head blocks; at most
};

inline PackedShape packed_shape(int64_t n_seqs, int64_t total_q, int64_t total_k, int64_t n_heads,
                                int64_t n_kv_heads, int cg, int bn, int sm_count)
{
    // Query rows of a tile are tokens x heads of one group: as many heads as
    // the largest power of two that divides the group.
    const int64_t group = n_heads / n_kv_heads;
    PackedShape s;
    s.gp_log2 = 0;
    while (s.gp_log2 < 5 && group % (2 << s.gp_log2) == 0)
        ++s.gp_log2;
    const int64_t tokens = static_cast<int64_t>(2 * cg * kBM) >> s.gp_log2;
    s.units = (total_q / tokens + n_seqs) * (n_heads >> s.gp_log2);
    // Few units over long sequences: parts of kPartTiles key tiles or more,
    // as many as the device holds at once.
    const int64_t keys = total_k - total_q / 2;    // that the middle query of a prompt sees
    const int64_t tiles = keys / n_seqs / bn, slots = sm_count / cg;
    int64_t parts = s.units > 0 ? slots / s.units : 1;
    parts = parts < tiles / kPartTiles ? parts : tiles / kPartTiles;
    s.parts = parts < 1 ? 1 : static_cast<int>(parts);
    return s;
}

// 3-D tensor map (element, head, row) of a [rows][heads][D] operand: boxes of
// 64 elements (128 bytes, 128-byte swizzle) x box_heads x box_rows, or of 32
// (64 bytes, 64-byte swizzle); rows past the tensor's end read as zero.
inline bool packed_tensor_map(CUtensorMap* map, const Heads& t, int64_t rows, int64_t heads, int d,
                              int box_heads, int box_rows, int dtype, int box_elems = 64)
{
    auto encode = tensor_map_encoder();
    if (!encode)
        return false;
    // A stride that is never taken may be anything; one that repeats an
    // element (0) or passes the map's 40 bits has no map.
    const int64_t hs = heads > 1 ? t.head : d, rs = rows > 1 ? t.row : hs * heads;
    if (hs < d || rs < d || hs >= (int64_t{1} << 38) || rs >= (int64_t{1} << 38))
        return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads),
                                static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(hs) * 2,
                                   static_cast<cuuint64_t>(rs) * 2};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_elems), static_cast<cuuint32_t>(box_heads),
                               static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t estride[3] = {1u, 1u, 1u};
    return encode(map, dtype == SOFTMAX_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                             : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                  3, t.data, dims, strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  box_elems == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D>
cudaError_t launch_join(const PackedProblem& p, const PackedShape& sh, cudaStream_t s)
{
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(sh.units), 2 * Shape<D>::CG * kBM / join_rows<D>(), 1);
    cfg.blockDim = dim3(kJoinThreads, 1, 1);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = static_cast<unsigned>(launch_attrs(attr, 1));
    const cudaError_t err = cudaLaunchKernelEx(&cfg, attention_packed_join_kernel<T, D>, p,
                                               sh.gp_log2, sh.parts);
    note_launch();
    return err;
}

template <typename T, int D, int MODE>
cudaError_t launch_tiles(const PackedProblem& p, const PackedShape& sh, cudaStream_t s)
{
    using S = Shape<D>;
    const int gp_log2 = sh.gp_log2, tile_tokens = kBM >> gp_log2;
    const int64_t units = sh.units * sh.parts;
    if (units * S::CG > 0x7fffffff)
        return cudaErrorNotSupported;
    CUtensorMap mq, mk, mv, mo;
    if (p.total_k == 0 ||
        !packed_tensor_map(&mq, p.q, p.total_q, p.n_heads, D, 1 << gp_log2, tile_tokens, p.dtype) ||
        !packed_tensor_map(&mk, p.k, p.total_k, p.n_kv_heads, D, 1, S::BN / S::CG, p.dtype) ||
        !packed_tensor_map(&mv, p.v, p.total_k, p.n_kv_heads, D, 1, S::BN, p.dtype) ||
        !packed_tensor_map(&mo, p.o, p.total_q, p.n_heads, D, 1 << gp_log2, 32 >> gp_log2, p.dtype,
                           32))
        return cudaErrorNotSupported;                    // nothing launched
    auto* kern = attention_packed_kernel<T, D, MODE>;
    static std::atomic<bool> attr_set[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return cudaErrorInvalidDevice;
    if (!attr_set[dev].load()) {
        const cudaError_t e = cudaFuncSetAttribute(
            kern, cudaFuncAttributeMaxDynamicSharedMemorySize, packed_smem<D>());
        if (e != cudaSuccess)
            return e;
        attr_set[dev].store(true);
    }
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(units * S::CG), 1, 1);
    cfg.blockDim = dim3(kPackedThreads, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(packed_smem<D>());
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = static_cast<unsigned>(launch_attrs(attr, S::CG));
    const float scale_log2 = static_cast<float>(static_cast<double>(p.scale) * 1.4426950408889634);
    // Units that all run at once may come in any order: the sequences' own
    // needs no ranking (90 tokens: 10.4 -> 9.7 us).
    const int by_length = units > sm_count_current() / S::CG;
    const cudaError_t err = cudaLaunchKernelEx(&cfg, kern, mq, mk, mv, mo, p, scale_log2, gp_log2,
                                               sh.parts, by_length);
    note_launch();
    if constexpr (MODE == kParts)
        return err == cudaSuccess ? launch_join<T, D>(p, sh, s) : err;
    return err;
}

template <typename T, int D>
cudaError_t launch_rows(const PackedProblem& p, cudaStream_t s)
{
    const int64_t tiles = p.total_q / kTileTokens + p.n_seqs;
    if (tiles > 0x7fffffff || p.n_heads > 65535)
        return cudaErrorNotSupported;
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(p.n_heads), 1);
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

PackedShape shape_of(int64_t n_seqs, int64_t total_q, int64_t total_k, int64_t n_heads,
                     int64_t n_kv_heads, int64_t d)
{
    return d == 64 ? packed_shape(n_seqs, total_q, total_k, n_heads, n_kv_heads, Shape<64>::CG,
                                  Shape<64>::BN, sm_count_current())
                   : packed_shape(n_seqs, total_q, total_k, n_heads, n_kv_heads, Shape<128>::CG,
                                  Shape<128>::BN, sm_count_current());
}

template <typename T, int D>
cudaError_t launch(const PackedProblem& p, cudaStream_t s)
{
    const PackedShape sh = shape_of(p.n_seqs, p.total_q, p.total_k, p.n_heads, p.n_kv_heads, D);
    const cudaError_t err = sh.parts > 1 ? launch_tiles<T, D, kParts>(p, sh, s)
                            : p.causal   ? launch_tiles<T, D, kCausal>(p, sh, s)
                                         : launch_tiles<T, D, kFull>(p, sh, s);
    return err == cudaErrorNotSupported ? launch_rows<T, D>(p, s) : err;
}

}  // namespace

cudaError_t launch_attention_packed(const PackedProblem& p, cudaStream_t s)
{
    if (p.dtype == SOFTMAX_BF16)
        return p.head_dim == 64 ? launch<BF16Bits, 64>(p, s) : launch<BF16Bits, 128>(p, s);
    return p.head_dim == 64 ? launch<F16Bits, 64>(p, s) : launch<F16Bits, 128>(p, s);
}

size_t attention_packed_workspace(int64_t n_seqs, int64_t total_q, int64_t total_k,
                                  int64_t n_heads, int64_t n_kv_heads, int64_t head_dim)
{
    const PackedShape sh = shape_of(n_seqs, total_q, total_k, n_heads, n_kv_heads, head_dim);
    if (sh.parts == 1)
        return 0;
    const int64_t slots = sh.units * sh.parts * 2;
    return static_cast<size_t>(head_dim == 64 ? slots * Shape<64>::CG * sizeof(PartSum<64>)
                                              : slots * Shape<128>::CG * sizeof(PartSum<128>));
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
