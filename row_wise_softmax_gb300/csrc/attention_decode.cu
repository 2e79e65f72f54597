// Attention of one new token of each sequence over a paged cache:
// o = softmax(scale q K^T) V over the sequence's cached tokens, with the
// running (m, l) softmax of "Triton GPU programming deep dive", section 3.3.
//
//   item     one (sequence, key/value head, block of up to 16 query heads of
//            its group); its tokens are cut into tiles of 64
//            (128 at D = 64).
//   split    all tiles of all items, in order, are cut into as many equal
//            runs as there are CTAs: a CTA's run may begin and end inside an
//            item.  Lengths are on the device, so each CTA finds its run from
//            the lengths itself.  A piece that is a whole item goes straight
//            to the output; a part of one leaves (m, l, O) in fp32 in the
//            workspace, two slots to a CTA (a run has at most one part at
//            either end), and the join kernel merges an item's parts in token
//            order, so results do not depend on timing.
//            Short calls (a few tiles to a CTA) take a cluster of CTAs to an
//            item instead and join through distributed shared memory: one
//            launch and no workspace.
//   warp     16 tokens (32 at D = 64) of each tile, on its own: its K and V
//            rows arrive by cp.async in its own ring of stages (no CTA barrier
//            in the walk), rows past the length as zeros.  Pages are of any
//            size and may end inside a tile, so rows are fetched one by one by
//            their places.  S = Q K^T by mma.sync m16n8k16
//            with the group's heads as the 16 rows; the scores' accumulator
//            layout is the A operand of P V.
//
// Bound by bytes: every cached row is read once from memory, against half a
// multiply-add per byte and query head, which mma.sync's rate covers for the
// 16 heads that share a tile.  Measured (bf16, 32 heads over 8 of 128 unless
// said): 64 ragged sequences up to 8192 tokens 96 us (6.05 TB/s; a plain copy
// runs at 6.7), 4 x 131072 tokens of 64 heads over 8 321 us (6.5 TB/s), 200 x
// 1000 tokens of 16 heads of 64 132 us (6.0 TB/s; half as long rows).  One
// sequence of 700 tokens takes 5.9 us: launch, length, page, row, and the join,
// each waiting for the one before.
#include "common.cuh"
#include "mma_sync.cuh"
#include "serving.h"

#include <atomic>

namespace rwsm {

__device__ unsigned g_error_attention_decode = 0;

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 16;                          // query heads of an item
constexpr int kStages = 3;
constexpr int kCtasPerSm = 2;
constexpr float kLazyRescaleLog2 = 8.0f;           // weights <= 2^8 between rescales

// Tokens of a tile and of a warp's block of it: a block of K and V is 8 KB at
// either head dimension (16-token blocks at D = 64 spent half of the issue
// slots on bookkeeping: 200 x 1000 tokens of 16 heads 150 us).
__host__ __device__ constexpr int warp_tokens(int d) { return d == 128 ? 16 : 32; }
__host__ __device__ constexpr int tile_tokens(int d) { return kWarps * warp_tokens(d); }

// One part of an item in the workspace.
template <int D>
struct Part {
    float m[kRows], l[kRows];
    float o[kRows * D];
};

// What a CTA's run begins and does not end: the item, and the CTA whose run
// ends it (item < 0: nothing).
struct Begun {
    int64_t item;
    int64_t last;
};

// How a call is launched.  cluster > 0: a cluster of that many CTAs to an item
// (CTA r takes tiles r, r + cluster, ...), joined through distributed shared
// memory; one launch, no workspace.  cluster == 0: equal runs of all tiles
// over a grid that fills the device, joined by a second kernel.
struct DecodeShape {
    int32_t group, blocks;                          // heads per kv head, 16-head blocks of them
    int32_t grid, cluster;
    int32_t abreast;                                // run form: items that a CTA walks side by side
};

constexpr int kMaxCluster = 16;
constexpr int kClusterTiles = 16;                   // tiles per CTA up to which clusters are used

inline DecodeShape decode_shape(int64_t n_seqs, int64_t n_heads, int64_t n_kv, int64_t head_dim,
                                int64_t capacity, int sm_count)
{
    DecodeShape s;
    s.group = static_cast<int32_t>(n_heads / n_kv);
    s.blocks = (s.group + kRows - 1) / kRows;
    const int tile = tile_tokens(static_cast<int>(head_dim));
    const int64_t per = capacity > 0 ? (capacity + tile - 1) / tile : 1;
    const int64_t most = static_cast<int64_t>(sm_count) * kCtasPerSm;
    const int64_t items = n_seqs * n_kv * s.blocks;
    s.cluster = 0;
    s.abreast = 1;
    if (items <= most) {
        int c = 1;
        while (c < kMaxCluster && c < per && items * c * 2 <= most)
            c *= 2;
        if (per <= static_cast<int64_t>(c) * kClusterTiles) {
            s.cluster = c;
            s.grid = static_cast<int32_t>(items * c);
            return s;
        }
    }
    // D = 64 and enough items to fill the device: a warp to an item, so that
    // a CTA reads up to four heads' 128-byte rows of a token together (200 x
    // 1000 tokens of 16 heads: 129 us against 133 to 145 one item at a time).
    // 256-byte rows gain nothing from it (61 ragged sequences up to 8192: 104
    // against 101 us), nor do few items (1 x 2000: 12.5 against 9.0 us).
    if (head_dim == 64 && items >= most)
        while (s.abreast < kWarps && n_kv * s.blocks % (2 * s.abreast) == 0)
            s.abreast *= 2;
    const int64_t groups = items / s.abreast;
    const int64_t tile_run = tile / kWarps * (kWarps / s.abreast);
    const int64_t runs = capacity > 0 ? (capacity + tile_run - 1) / tile_run : 1;
    s.grid = static_cast<int32_t>(groups >= most || groups * runs >= most ? most : groups * runs);
    return s;
}

__device__ __forceinline__ int64_t shfl64(int64_t v, int lane)
{
    const int lo = __shfl_sync(0xffffffffu, static_cast<int>(v), lane);
    const int hi = __shfl_sync(0xffffffffu, static_cast<int>(v >> 32), lane);
    return (static_cast<int64_t>(hi) << 32) | static_cast<uint32_t>(lo);
}

// A sequence's length as the kernel uses it; `bad` when it leads out of the
// table (the sequence then has no tokens).
__device__ __forceinline__ int32_t length_of(const DecodeProblem& p, int64_t b, bool& bad)
{
    const int32_t n = __ldg(p.lengths + b);
    bad = n < 0 || n > p.cache.capacity;
    return bad ? 0 : n;
}

// Tiles of an item of n tokens: at least one, so that an empty sequence's
// outputs are written too.
template <int D>
__device__ __forceinline__ int32_t tiles_of(int32_t n)
{
    constexpr int tile = tile_tokens(D);
    return n == 0 ? 1 : (n + tile - 1) / tile;
}

// What a warp carries through an item: the running maxima (base 2), sums and
// output accumulators of rows lane / 4 and lane / 4 + 8, in the accumulator
// layout of m16n8k16 (columns (lane % 4) * 2, + 1 of each 8).
template <int D>
struct WarpSum {
    float m_a, m_b, l_a, l_b;
    float acc[D / 8][4];

    __device__ __forceinline__ void clear()
    {
        m_a = m_b = kNegInf;
        l_a = l_b = 0.0f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
            acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
    }

    // The row sums over the four lanes that share a row; NaN for an item with
    // a bad page or length.
    __device__ __forceinline__ void close(bool bad)
    {
        l_a += __shfl_xor_sync(0xffffffffu, l_a, 1);
        l_a += __shfl_xor_sync(0xffffffffu, l_a, 2);
        l_b += __shfl_xor_sync(0xffffffffu, l_b, 1);
        l_b += __shfl_xor_sync(0xffffffffu, l_b, 2);
        if (__any_sync(0xffffffffu, bad)) {
            l_a = l_b = __int_as_float(0x7fc00000);
            if ((threadIdx.x & 31) == 0)
                atomicOr(&g_error_attention_decode, kErrBadIndex);
        }
    }
};

// Q fragments (A operand) of `rows` heads from h0 on; rows past them are zero.
template <int D>
__device__ __forceinline__ void load_q(const DecodeProblem& p, int64_t seq, int h0, int rows,
                                       uint32_t (&qa)[D / 16][4])
{
    const int lane = threadIdx.x & 31, r_a = lane >> 2, c_q = (lane & 3) * 2;
    const unsigned short* gq = static_cast<const unsigned short*>(p.q.data) + seq * p.q.row +
                               static_cast<int64_t>(h0) * p.q.head;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int r = r_a + (e & 1) * 8, c = kk * 16 + (e >> 1) * 8 + c_q;
            qa[kk][e] = r < rows ? __ldg(reinterpret_cast<const unsigned*>(gq + r * p.q.head + c))
                                 : 0u;
        }
}

// The page that holds token `tok`, -1 past the length.
__device__ __forceinline__ int32_t page_of(const DecodeProblem& p, const int32_t* table,
                                           int32_t tok, int32_t len)
{
    return tok < len ? __ldg(table + divide(tok, p.cache.page)) : -1;
}

// Copy a warp's block of K and V rows of one head into a stage: lane i holds
// the page of token tok0 + i (of 16 tokens, lanes 16..31 hold them again) and
// turns it into its rows' places, in units of 16 bytes.  Tokens past the
// length, and rows of bad pages (true is returned then), arrive as zeros.
template <int D>
__device__ __forceinline__ bool copy_block(const DecodeProblem& p, int kvh, int32_t tok0,
                                           int32_t page, int32_t len, uint32_t dst)
{
    constexpr int TOK = warp_tokens(D);
    constexpr int CH = D / 8;                       // 16-byte chunks of a row
    constexpr uint32_t BLK = TOK * D * 2;
    const int lane = threadIdx.x & 31;
    const unsigned short* gk =
        static_cast<const unsigned short*>(p.cache.k) + kvh * p.cache.k_head;
    const unsigned short* gv =
        static_cast<const unsigned short*>(p.cache.v) + kvh * p.cache.v_head;
    const int32_t tok = tok0 + lane % TOK;
    const bool held = page >= 0 && page < p.cache.n_pages && tok < len;
    int64_t ko = -1, vo = -1;
    if (held) {
        const int64_t row = tok - divide(tok, p.cache.page) * p.cache.page.d;
        ko = (page * p.cache.k_page + row * p.cache.k_row) >> 3;
        vo = (page * p.cache.v_page + row * p.cache.v_row) >> 3;
    }
    auto copy = [&](int i, int64_t k, int64_t v) {
        const int r = (i * 32 + lane) / CH, c = (i * 32 + lane) % CH;
        const int bytes = k < 0 ? 0 : 16;
        k = k < 0 ? 0 : k * 8 + c * 8;
        v = v < 0 ? 0 : v * 8 + c * 8;
        cp_async16_zfill(dst + tile_off<D>(r, c), gk + k, bytes);
        cp_async16_zfill(dst + BLK + tile_off<D>(r, c), gv + v, bytes);
    };
    if (p.cache.near_rows) {                        // places below 2^31, the same for K and V
#pragma unroll
        for (int i = 0; i < TOK * CH / 32; ++i) {
            const int32_t o = __shfl_sync(0xffffffffu, static_cast<int32_t>(ko), (i * 32 + lane) / CH);
            copy(i, o, o);
        }
    } else {
#pragma unroll
        for (int i = 0; i < TOK * CH / 32; ++i) {
            const int r = (i * 32 + lane) / CH;
            copy(i, shfl64(ko, r), shfl64(vo, r));
        }
    }
    return tok < len && !held;
}

// A warp's block of tokens, the first at position j0, of a sequence of len:
// S = Q K^T, the softmax's step, O += P V.  The reference of the softmax moves
// only when a maximum exceeds it by more than 2^8; l and O agree either way.
template <typename T, int D>
__device__ __forceinline__ void attend_block(const uint32_t (&qa)[D / 16][4], uint32_t sK,
                                             int32_t j0, int32_t len, float scale_log2,
                                             WarpSum<D>& w)
{
    constexpr int TOK = warp_tokens(D);
    constexpr int NB = TOK / 8;
    const uint32_t sV = sK + TOK * D * 2;
    const int lane = threadIdx.x & 31, mi = lane >> 3, c_q = (lane & 3) * 2;
    float s[NB][4];
#pragma unroll
    for (int i = 0; i < NB; ++i)
        s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0f;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int n = 0; n < NB; n += 2) {
            uint32_t bk[4];
            ldsm_x4(bk, sK + tile_off<D>(n * 8 + (lane & 7) + (mi >> 1) * 8, kk * 2 + (mi & 1)));
            MmaType<T>::mma(s[n], qa[kk], bk[0], bk[1]);
            MmaType<T>::mma(s[n + 1], qa[kk], bk[2], bk[3]);
        }
    if (j0 + TOK > len) {
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (j0 + n * 8 + c_q + e >= len)
                    s[n][e] = s[n][2 + e] = kNegInf;
    }
    float mx_a = kNegInf, mx_b = kNegInf;
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        mx_a = max3(mx_a, s[n][0], s[n][1]);
        mx_b = max3(mx_b, s[n][2], s[n][3]);
    }
    mx_a *= scale_log2;
    mx_b *= scale_log2;
    // Rows are shared by four lanes, whose maxima are exchanged only when one
    // of them passes the reference.
    if (__any_sync(0xffffffffu,
                   mx_a > w.m_a + kLazyRescaleLog2 || mx_b > w.m_b + kLazyRescaleLog2)) {
        mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, 1));
        mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, 2));
        mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, 1));
        mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, 2));
        const float mn_a = fmaxf(w.m_a, mx_a), mn_b = fmaxf(w.m_b, mx_b);
        const float al_a = mn_a == kNegInf ? 1.0f : ex2_ftz(w.m_a - mn_a);
        const float al_b = mn_b == kNegInf ? 1.0f : ex2_ftz(w.m_b - mn_b);
        w.m_a = mn_a;
        w.m_b = mn_b;
        w.l_a *= al_a;
        w.l_b *= al_b;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            w.acc[i][0] *= al_a; w.acc[i][1] *= al_a;
            w.acc[i][2] *= al_b; w.acc[i][3] *= al_b;
        }
    }
    const float ref_a = w.m_a == kNegInf ? 0.0f : -w.m_a;
    const float ref_b = w.m_b == kNegInf ? 0.0f : -w.m_b;
    uint32_t pa[TOK / 16][4];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        const float p0 = ex2_ftz(fmaf(s[n][0], scale_log2, ref_a));
        const float p1 = ex2_ftz(fmaf(s[n][1], scale_log2, ref_a));
        const float p2 = ex2_ftz(fmaf(s[n][2], scale_log2, ref_b));
        const float p3 = ex2_ftz(fmaf(s[n][3], scale_log2, ref_b));
        w.l_a += p0 + p1;
        w.l_b += p2 + p3;
        pa[n / 2][(n % 2) * 2 + 0] = Elem<T>::pack2(p0, p1);
        pa[n / 2][(n % 2) * 2 + 1] = Elem<T>::pack2(p2, p3);
    }
#pragma unroll
    for (int k = 0; k < TOK / 16; ++k)
#pragma unroll
        for (int dp = 0; dp < D / 16; ++dp) {
            uint32_t bv[4];
            ldsm_x4_trans(bv, sV + tile_off<D>(k * 16 + (lane & 7) + (mi & 1) * 8,
                                               dp * 2 + (mi >> 1)));
            MmaType<T>::mma(w.acc[2 * dp], pa[k], bv[0], bv[1]);
            MmaType<T>::mma(w.acc[2 * dp + 1], pa[k], bv[2], bv[3]);
        }
}

// Columns c .. c + 3 of head h's output from its sum and (m, l); the logsumexp.
template <typename T>
__device__ __forceinline__ void store_head(const DecodeProblem& p, int64_t seq, int h, int c,
                                           const float4& o, float M, float L)
{
    const float inv = 1.0f / L;
    uint2 w;
    w.x = Elem<T>::pack2(o.x * inv, o.y * inv);
    w.y = Elem<T>::pack2(o.z * inv, o.w * inv);
    *reinterpret_cast<uint2*>(static_cast<unsigned short*>(p.o.data) + seq * p.o.row +
                              static_cast<int64_t>(h) * p.o.head + c) = w;
    if (p.lse && c == 0)
        p.lse[seq * p.n_heads + h] = L == 0.0f ? kNegInf : (M + __log2f(L)) * 0.69314718055994531f;
}

// The (m, l) of every warp's rows, and row r's over the warps.
struct RowStats {
    float m[kWarps][kRows], l[kWarps][kRows];

    template <int D>
    __device__ __forceinline__ void put(const WarpSum<D>& w)
    {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        if ((lane & 3) == 0) {
            m[warp][lane >> 2] = w.m_a;
            m[warp][(lane >> 2) + 8] = w.m_b;
            l[warp][lane >> 2] = w.l_a;
            l[warp][(lane >> 2) + 8] = w.l_b;
        }
    }

    __device__ __forceinline__ float max_of(int r) const
    {
        float M = kNegInf;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            M = fmaxf(M, m[w][r]);
        return M;
    }

    __device__ __forceinline__ float sum_of(int r, float M) const
    {
        const float ref = M == kNegInf ? 0.0f : M;
        float L = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            L += l[w][r] * ex2_ftz(m[w][r] - ref);
        return L;
    }

    // What this warp's row r counts for in the merged sum.
    __device__ __forceinline__ float factor(float mine, float M) const
    {
        return M == kNegInf ? 0.0f : ex2_ftz(mine - M);
    }
};

// Which heads an item is: `in` counts (kv head, block of 16 query heads).
struct ItemHeads {
    int kvh, h0, rows;

    __device__ __forceinline__ ItemHeads(const DecodeShape& sh, int in)
    {
        kvh = in / sh.blocks;
        const int hb = in - kvh * sh.blocks;
        h0 = kvh * sh.group + hb * kRows;
        rows = sh.group - hb * kRows < kRows ? sh.group - hb * kRows : kRows;
    }
};

// ------------------------------------------------- a cluster of CTAs per item
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
attention_decode_cluster_kernel(const DecodeProblem p, const DecodeShape sh, float scale_log2)
{
    namespace cg = cooperative_groups;
    constexpr int TOK = warp_tokens(D), kTile = tile_tokens(D);
    constexpr uint32_t BLK = TOK * D * 2;           // bytes of a warp's K (or V) block
    constexpr int PER = kRows * D / 4 / kThreads;   // groups of four columns per thread
    extern __shared__ __align__(128) unsigned char dec_smem[];
    __shared__ RowStats stats;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t ring = smem_addr(dec_smem) + warp * (kStages * 2 * BLK);
    float* const sm_o = reinterpret_cast<float*>(dec_smem);          // [kWarps][kRows][D]
    const int step = sh.cluster;
    const int rank = static_cast<int>(blockIdx.x % static_cast<unsigned>(step));
    const int inner = p.cache.n_kv_heads * sh.blocks;
    const int64_t item = blockIdx.x / static_cast<unsigned>(step);
    const int64_t seq = item / inner;
    const ItemHeads it(sh, static_cast<int>(item - seq * inner));

    pdl_launch_dependents();
    pdl_wait();
    // The first tile's page, the length and Q are read side by side.
    const int32_t* table = p.cache.table + seq * p.cache.table_stride;
    const int32_t tok0 = warp * TOK + lane % TOK;
    const int32_t page0 = page_of(p, table, rank * kTile + tok0, p.cache.capacity);
    bool bad;
    const int32_t len = length_of(p, seq, bad);
    uint32_t qa[D / 16][4];
    load_q<D>(p, seq, it.h0, it.rows, qa);
    const int n_tiles = tiles_of<D>(len);

    WarpSum<D> w;
    w.clear();
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
        const int t = rank + i * step;
        if (t < n_tiles)
            bad |= copy_block<D>(p, it.kvh, t * kTile + warp * TOK,
                                 i == 0 ? page0 : page_of(p, table, t * kTile + tok0, len), len,
                                 ring + i * (2 * BLK));
        cp_async_commit();
    }
    int now = 0;                                    // the stage of tile t
    for (int t = rank; t < n_tiles; t += step) {
        const int next = t + (kStages - 1) * step;
        if (next < n_tiles)
            bad |= copy_block<D>(p, it.kvh, next * kTile + warp * TOK,
                                 page_of(p, table, next * kTile + tok0, len), len,
                                 ring + (now == 0 ? kStages - 1 : now - 1) * (2 * BLK));
        cp_async_commit();
        asm volatile("cp.async.wait_group %0;" :: "n"(kStages - 1) : "memory");
        __syncwarp();
        attend_block<T, D>(qa, ring + now * (2 * BLK), t * kTile + warp * TOK, len,
                           scale_log2, w);
        __syncwarp();                               // the stage may be refilled
        now = now + 1 == kStages ? 0 : now + 1;
    }
    cp_async_wait_all_groups();

    // ---- the four warps' sums into one
    w.close(bad);
    stats.put(w);
    __syncthreads();                                // and every warp's ring is free
    const int r_a = lane >> 2, c_q = (lane & 3) * 2;
    const float f_a = stats.factor(w.m_a, stats.max_of(r_a));
    const float f_b = stats.factor(w.m_b, stats.max_of(r_a + 8));
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
        float* const a = sm_o + (warp * kRows + r_a) * D + i * 8 + c_q;
        *reinterpret_cast<float2*>(a) = make_float2(w.acc[i][0] * f_a, w.acc[i][1] * f_a);
        *reinterpret_cast<float2*>(a + 8 * D) = make_float2(w.acc[i][2] * f_b, w.acc[i][3] * f_b);
    }
    __syncthreads();
    float M[PER], L[PER];
    float4 o[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int i = tid + j * kThreads, r = i / (D / 4), c = (i % (D / 4)) * 4;
        M[j] = stats.max_of(r);
        L[j] = stats.sum_of(r, M[j]);
        o[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int q = 0; q < kWarps; ++q) {
            const float4 x = *reinterpret_cast<const float4*>(sm_o + (q * kRows + r) * D + c);
            o[j].x += x.x; o[j].y += x.y; o[j].z += x.z; o[j].w += x.w;
        }
    }
    if (step == 1) {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int i = tid + j * kThreads, r = i / (D / 4), c = (i % (D / 4)) * 4;
            if (r < it.rows)
                store_head<T>(p, seq, it.h0 + r, c, o[j], M[j], L[j]);
        }
        return;
    }
    // ---- each CTA leaves its sum in the place of warp 0's, and takes every
    // cluster-th group of four columns of all of them, in the order of the CTAs
    __syncthreads();
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int i = tid + j * kThreads, r = i / (D / 4), c = (i % (D / 4)) * 4;
        *reinterpret_cast<float4*>(sm_o + r * D + c) = o[j];
        if (c == 0) {
            stats.m[0][r] = M[j];
            stats.l[0][r] = L[j];
        }
    }
    cg::cluster_group cluster = cg::this_cluster();
    cluster.sync();
    for (int i = rank + tid * step; i < it.rows * (D / 4); i += kThreads * step) {
        const int r = i / (D / 4), c = (i % (D / 4)) * 4;
        float Mx = kNegInf, Lx = 0.0f;
#pragma unroll 8
        for (int q = 0; q < step; ++q)
            Mx = fmaxf(Mx, *cluster.map_shared_rank(&stats.m[0][r], q));
        const float ref = Mx == kNegInf ? 0.0f : Mx;
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
        for (int q = 0; q < step; ++q) {
            const float f = ex2_ftz(*cluster.map_shared_rank(&stats.m[0][r], q) - ref);
            const float4 x =
                *reinterpret_cast<const float4*>(cluster.map_shared_rank(sm_o + r * D + c, q));
            Lx += *cluster.map_shared_rank(&stats.l[0][r], q) * f;
            sum.x += x.x * f; sum.y += x.y * f; sum.z += x.z * f; sum.w += x.w * f;
        }
        store_head<T>(p, seq, it.h0 + r, c, sum, Mx, Lx);
    }
    cluster.sync();                                 // read before a CTA leaves
}

// ------------------------------------------------------- equal runs of tiles
// A CTA walks `HW` items side by side (key/value heads of one sequence: their
// rows of a token lie next to each other in memory), TW = kWarps / HW warps to
// each of them, which take turns of warp_tokens tokens.  A tile is
// TW * warp_tokens tokens of HW items.  Sequences without tokens have no
// tiles; their outputs are written apart.

// A CTA's run [begin, end) of all tiles, and the sequence it begins in.
struct Run {
    int64_t begin, end;                             // tiles
    int64_t total, runs;
    int64_t seq;                                    // sequence of the first tile
    int64_t before;                                 // tiles of the sequences before it
};

template <int TILE>
__device__ __forceinline__ int32_t run_tiles(int32_t n)
{
    return (n + TILE - 1) / TILE;
}

// Every thread gets the same answer.  The sequences' tiles are summed 128 at a
// time; with no more sequences than that, one pass finds total and place.
template <int TILE, int LEAST>
__device__ Run find_run(const DecodeProblem& p, int groups, Run& place, int64_t* scratch)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    auto scan = [&](int64_t b, int64_t& upto) {     // tiles of sequence b, and of the block up to it
        bool bad = false;
        const int64_t n = b < p.n_seqs ? run_tiles<TILE>(length_of(p, b, bad)) : 0;
        upto = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o)
                upto += up;
        }
        __syncthreads();                            // scratch is free
        if (lane == 31)
            scratch[warp] = upto;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            if (w < warp)
                upto += scratch[w];
        return n;
    };
    auto all = [&] {
        int64_t sum = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
            sum += scratch[w];
        return sum;
    };
    Run r = {};
    int64_t upto, n = 0, total = 0;
    for (int64_t b = 0; b < p.n_seqs; b += kThreads) {
        n = scan(b + tid, upto);
        total += all();
    }
    // Runs of LEAST tiles at least (short ones cost more to join than they
    // save), and none that is empty but those of the CTAs past the last: an
    // item's parts lie in consecutive CTAs.
    r.total = total * groups;
    r.runs = (r.total + LEAST - 1) / LEAST;
    r.runs = r.runs < gridDim.x ? r.runs : gridDim.x;
    r.begin = blockIdx.x < r.runs ? r.total * blockIdx.x / r.runs : 0;
    r.end = blockIdx.x < r.runs ? r.total * (blockIdx.x + 1) / r.runs : 0;
    int64_t before = 0;
    for (int64_t b = 0; b < p.n_seqs; b += kThreads) {
        if (p.n_seqs > kThreads)
            n = scan(b + tid, upto);
        if (r.begin < r.end && n > 0 && (before + upto - n) * groups <= r.begin &&
            r.begin < (before + upto) * groups) {
            place.seq = b + tid;
            place.before = (before + upto - n) * groups;
        }
        before += all();
    }
    __syncthreads();
    r.seq = place.seq;
    r.before = place.before;
    return r;
}

// A place in the order of all tiles: tile t of head group g of a sequence.
template <int TILE>
struct Cursor {
    int64_t seq, first;                             // first: the group's first tile among all
    int32_t g, t, n_tiles, len;

    __device__ __forceinline__ void read(const DecodeProblem& p)
    {
        bool bad;
        len = length_of(p, seq, bad);
        n_tiles = run_tiles<TILE>(len);
    }

    __device__ __forceinline__ void begin(const DecodeProblem& p, const Run& run)
    {
        seq = run.seq;
        read(p);
        const int64_t at = run.begin - run.before;
        g = static_cast<int32_t>(at / n_tiles);
        t = static_cast<int32_t>(at - static_cast<int64_t>(g) * n_tiles);
        first = run.before + static_cast<int64_t>(g) * n_tiles;
    }

    // To the next group that has tiles (there must be one).
    __device__ __forceinline__ void next_group(const DecodeProblem& p, int groups)
    {
        first += n_tiles;
        t = 0;
        if (++g == groups) {
            g = 0;
            do {
                ++seq;
                read(p);
            } while (n_tiles == 0);
        }
    }
};

template <typename T, int D, int HW>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
attention_decode_runs_kernel(const DecodeProblem p, const DecodeShape sh, float scale_log2)
{
    constexpr int TOK = warp_tokens(D), TW = kWarps / HW, TILE = TOK * TW;
    constexpr uint32_t BLK = TOK * D * 2;           // bytes of a warp's K (or V) block
    extern __shared__ __align__(128) unsigned char dec_smem[];
    __shared__ RowStats stats;
    __shared__ int64_t sm_scratch[kWarps];
    __shared__ Run sm_place;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int hw = warp % HW, tw = warp / HW;
    const int inner = p.cache.n_kv_heads * sh.blocks, groups = inner / HW;
    const uint32_t ring = smem_addr(dec_smem) + warp * (kStages * 2 * BLK);
    // TW > 1: eight rows of every warp's O, half an item at a time, beside the
    // rings, which go on filling.
    float* const sm_o = reinterpret_cast<float*>(dec_smem + kWarps * kStages * 2 * BLK);
    Part<D>* const parts = static_cast<Part<D>*>(p.workspace);
    Begun* const begun = reinterpret_cast<Begun*>(parts + 2 * HW * static_cast<int64_t>(sh.grid));
    const int64_t mine = static_cast<int64_t>(blockIdx.x) * HW + hw;    // of parts / 2 and begun

    pdl_launch_dependents();
    pdl_wait();
    const Run run = find_run<TILE, HW>(p, groups, sm_place, sm_scratch);
    // Sequences without tokens, dealt to the CTAs: NaN (0 / 0).
    for (int64_t b = blockIdx.x; b < p.n_seqs; b += gridDim.x) {
        bool bad;
        if (length_of(p, b, bad) > 0)
            continue;
        if (bad && tid == 0)
            atomicOr(&g_error_attention_decode, kErrBadIndex);
        const float nan = __int_as_float(0x7fc00000);
        for (int i = tid; i < p.n_heads * (D / 4); i += kThreads)
            store_head<T>(p, b, i / (D / 4), (i % (D / 4)) * 4, make_float4(nan, nan, nan, nan),
                          kNegInf, bad ? nan : 0.0f);
    }
    int64_t begun_item = -1, begun_last = 0;
    if (run.begin < run.end) {
        // Two cursors walk the run: one copies, kStages - 1 tiles ahead and on
        // into the next items, the other computes.
        Cursor<TILE> copy, it;
        it.begin(p, run);
        copy = it;
        int64_t to_copy = run.end - run.begin;
        uint32_t bad_stages = 0;
        const int32_t tok0 = tw * TOK + lane % TOK;
        auto copy_next = [&](int st) {
            if (to_copy > 0) {
                --to_copy;
                const int32_t t = copy.t * TILE;
                const bool bad = copy_block<D>(
                    p, (copy.g * HW + hw) / sh.blocks, t + tw * TOK,
                    page_of(p, p.cache.table + copy.seq * p.cache.table_stride, t + tok0, copy.len),
                    copy.len, ring + static_cast<uint32_t>(st) * (2 * BLK));
                bad_stages = (bad_stages & ~(1u << st)) | (bad ? 1u << st : 0u);
                if (++copy.t == copy.n_tiles && to_copy > 0)
                    copy.next_group(p, groups);
            }
            cp_async_commit();
        };
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i)
            copy_next(i);
        uint32_t qa[D / 16][4];
        {
            const ItemHeads heads(sh, it.g * HW + hw);
            load_q<D>(p, it.seq, heads.h0, heads.rows, qa);
        }
        WarpSum<D> w;
        w.clear();
        bool bad = false;
        int32_t from = it.t;                        // the piece's first tile
        int now = 0;                                // the stage of the tile at hand
        for (int64_t left = run.end - run.begin; left > 0; --left) {
            copy_next(now == 0 ? kStages - 1 : now - 1);
            asm volatile("cp.async.wait_group %0;" :: "n"(kStages - 1) : "memory");
            __syncwarp();
            bad |= (bad_stages >> now & 1u) != 0;
            attend_block<T, D>(qa, ring + static_cast<uint32_t>(now) * (2 * BLK),
                               it.t * TILE + tw * TOK, it.len, scale_log2, w);
            __syncwarp();                           // the stage may be refilled
            now = now + 1 == kStages ? 0 : now + 1;
            if (++it.t < it.n_tiles && left > 1)
                continue;

            // ---- the piece ends
            const ItemHeads heads(sh, it.g * HW + hw);
            const int64_t seq = it.seq;
            const bool whole = from == 0 && it.t == it.n_tiles;
            Part<D>* const part = parts + 2 * mine + (from == 0 ? 1 : 0);
            if (from == 0 && !whole) {
                // The run that holds the item's last tile.
                const int64_t last = it.first + it.n_tiles - 1;
                begun_item = seq * inner + it.g * HW + hw;
                int64_t c = last * run.runs / run.total;
                while (run.total * (c + 1) / run.runs <= last)
                    ++c;
                while (run.total * c / run.runs > last)
                    --c;
                begun_last = c;
            }
            if (left > 1) {                         // the next item's Q meanwhile
                it.next_group(p, groups);
                from = 0;
                const ItemHeads next(sh, it.g * HW + hw);
                load_q<D>(p, it.seq, next.h0, next.rows, qa);
            }
            w.close(bad);
            const int r_a = lane >> 2, c_q = (lane & 3) * 2;
            if constexpr (TW == 1) {
                // The warp's sum is the item's.
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int row = half * 8 + r_a;
                    const float M = half == 0 ? w.m_a : w.m_b, L = half == 0 ? w.l_a : w.l_b;
                    if (row < heads.rows) {
                        if (whole) {
                            const float inv = 1.0f / L;
                            unsigned short* const o = static_cast<unsigned short*>(p.o.data) +
                                seq * p.o.row + static_cast<int64_t>(heads.h0 + row) * p.o.head + c_q;
#pragma unroll
                            for (int i = 0; i < D / 8; ++i)
                                *reinterpret_cast<unsigned*>(o + i * 8) =
                                    Elem<T>::pack2(w.acc[i][half * 2] * inv,
                                                   w.acc[i][half * 2 + 1] * inv);
                            if (p.lse && c_q == 0)
                                p.lse[seq * p.n_heads + heads.h0 + row] =
                                    L == 0.0f ? kNegInf : (M + __log2f(L)) * 0.69314718055994531f;
                        } else {
#pragma unroll
                            for (int i = 0; i < D / 8; ++i)
                                *reinterpret_cast<float2*>(part->o + row * D + i * 8 + c_q) =
                                    make_float2(w.acc[i][half * 2], w.acc[i][half * 2 + 1]);
                            if (c_q == 0) {
                                part->m[row] = M;
                                part->l[row] = L;
                            }
                        }
                    }
                }
            } else {
                // The TW warps' sums into one, in the order of the warps.
                const int most = sh.group < kRows ? sh.group : kRows;    // rows of any item
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (half * 8 >= most)
                        break;
                    __syncthreads();                // sm_o (and stats) have been read
                    if (half == 0)
                        stats.put(w);
                    if (half * 8 + r_a < heads.rows) {
#pragma unroll
                        for (int i = 0; i < D / 8; ++i)
                            *reinterpret_cast<float2*>(sm_o + (warp * 8 + r_a) * D + i * 8 + c_q) =
                                make_float2(w.acc[i][half * 2], w.acc[i][half * 2 + 1]);
                    }
                    __syncthreads();
                    const int rows = heads.rows - half * 8 < 8 ? heads.rows - half * 8 : 8;
                    for (int i = tw * 32 + lane; i < rows * (D / 4); i += TW * 32) {
                        const int r = i / (D / 4), c = (i % (D / 4)) * 4, row = half * 8 + r;
                        float M = kNegInf, L = 0.0f;
#pragma unroll
                        for (int q = 0; q < TW; ++q)
                            M = fmaxf(M, stats.m[q * HW + hw][row]);
                        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                        for (int q = 0; q < TW; ++q) {
                            const int v = q * HW + hw;
                            const float f = stats.factor(stats.m[v][row], M);
                            const float4 x =
                                *reinterpret_cast<const float4*>(sm_o + (v * 8 + r) * D + c);
                            // (M of -inf: no score but -inf or NaN, which l holds)
                            L += stats.l[v][row] * (M == kNegInf ? 1.0f : f);
                            o.x += x.x * f; o.y += x.y * f; o.z += x.z * f; o.w += x.w * f;
                        }
                        if (whole) {
                            store_head<T>(p, seq, heads.h0 + row, c, o, M, L);
                        } else {
                            *reinterpret_cast<float4*>(part->o + row * D + c) = o;
                            if (c == 0) {
                                part->m[row] = M;
                                part->l[row] = L;
                            }
                        }
                    }
                }
            }
            w.clear();
            bad = false;
        }
        cp_async_wait_all_groups();
    }
    if (tw == 0 && lane == 0)
        begun[mine] = Begun{begun_item, begun_last};
}

// Merge the parts of the item that CTA blockIdx.x of the main kernel began
// and did not end, abreast place blockIdx.y: slot 1 of that CTA, then slot 0 of
// each CTA up to the last.
// A thread takes four columns of a row; threads left over take every G-th
// part, and their sums are merged in order.
constexpr int kJoinThreads = 256;

template <int D>
struct JoinSum {
    float m, l;
    float4 o;

    __device__ __forceinline__ void clear()
    {
        m = kNegInf;
        l = 0.0f;
        o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }

    __device__ __forceinline__ void read(const Part<D>* q, int r, int c)
    {
        m = q->m[r];
        l = q->l[r];
        o = *reinterpret_cast<const float4*>(q->o + r * D + c);
    }

    __device__ __forceinline__ void merge(const JoinSum& x)
    {
        const float M = fmaxf(m, x.m), ref = M == kNegInf ? 0.0f : M;
        const float f = ex2_ftz(m - ref), g = ex2_ftz(x.m - ref);
        m = M;
        l = l * f + x.l * g;
        o.x = o.x * f + x.o.x * g;
        o.y = o.y * f + x.o.y * g;
        o.z = o.z * f + x.o.z * g;
        o.w = o.w * f + x.o.w * g;
    }
};

template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads)
attention_decode_join_kernel(const DecodeProblem p, const DecodeShape sh)
{
    __shared__ JoinSum<D> sums[kJoinThreads];
    const int tid = threadIdx.x;
    const Part<D>* const parts = static_cast<const Part<D>*>(p.workspace);
    const Begun* const begun =
        reinterpret_cast<const Begun*>(parts + 2 * sh.abreast * static_cast<int64_t>(sh.grid));
    auto part = [&](int i) {
        return parts + 2 * ((static_cast<int64_t>(blockIdx.x) + i) * sh.abreast + blockIdx.y) +
               (i == 0 ? 1 : 0);
    };
    const int inner = p.cache.n_kv_heads * sh.blocks;
    // Units (row, four columns) of an item with all its rows: items with
    // fewer leave some threads idle.
    const int most = (sh.group < kRows ? sh.group : kRows) * (D / 4);
    const int groups = kJoinThreads / most > 0 ? kJoinThreads / most : 1;
    pdl_launch_dependents();
    pdl_wait();
    const Begun g = begun[static_cast<int64_t>(blockIdx.x) * sh.abreast + blockIdx.y];
    const int n = static_cast<int>(g.last - blockIdx.x) + 1;
    for (int u0 = 0; u0 < most; u0 += kJoinThreads) {
        const int u = u0 + (groups > 1 ? tid % most : tid), mine = groups > 1 ? tid / most : 0;
        const bool on = u < most && mine < groups;
        const int r = u / (D / 4), c = (u % (D / 4)) * 4;
        // This group's first part is read beside the header: an item that was
        // begun and not ended has two parts at least.
        JoinSum<D> s, x[4];
        s.clear();
        if (on && mine < 2 && blockIdx.x + mine < gridDim.x)
            s.read(part(mine), r, c);
        if (g.item < 0)
            return;
        const int64_t seq = g.item / inner;
        const ItemHeads heads(sh, static_cast<int>(g.item - seq * inner));
        if (on && r < heads.rows) {
            int i = mine;
            if (mine < 2)
                i += groups;
            else
                s.clear();
            for (; i < n; i += 4 * groups) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (i + k * groups < n)
                        x[k].read(part(i + k * groups), r, c);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (i + k * groups < n)
                        s.merge(x[k]);
            }
        }
        if (groups > 1) {
            sums[tid] = s;
            __syncthreads();
            if (mine == 0)
                for (int k = 1; k < groups && k < n; ++k)
                    s.merge(sums[k * most + u]);
        }
        if (on && mine == 0 && r < heads.rows)
            store_head<T>(p, seq, heads.h0 + r, c, s.o, s.m, s.l);
    }
}

template <typename T, int D>
cudaError_t launch(const DecodeProblem& p, cudaStream_t s)
{
    const DecodeShape sh = decode_shape(p.n_seqs, p.n_heads, p.cache.n_kv_heads, D, p.cache.capacity,
                                        sm_count_current());
    const int form = sh.cluster > 0 ? 0 : sh.abreast;   // 0, or 1, 2 or 4 abreast
    auto* kern = form == 0 ? attention_decode_cluster_kernel<T, D>
                           : attention_decode_runs_kernel<T, D, 1>;
    if constexpr (D == 64) {
        if (form == 2)
            kern = attention_decode_runs_kernel<T, D, 2>;
        else if (form == 4)
            kern = attention_decode_runs_kernel<T, D, 4>;
    }
    constexpr int kRing = kWarps * kStages * 2 * warp_tokens(D) * D * 2;
    static_assert(kWarps * kRows * D * 4 <= kRing, "the warps' O rows fit in the rings");
    const int smem = kRing + (form == 1 || form == 2 ? kWarps * 8 * D * 4 : 0);
    static std::atomic<bool> attr_set[kWarps + 1][64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return cudaErrorInvalidDevice;
    if (!attr_set[form][dev].load()) {
        cudaError_t e =
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess && sh.cluster > 0)
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess)
            return e;
        attr_set[form][dev].store(true);
    }
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(sh.grid), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = static_cast<unsigned>(launch_attrs(attr, sh.cluster));
    const float scale_log2 = static_cast<float>(static_cast<double>(p.scale) * 1.4426950408889634);
    cudaError_t err = cudaLaunchKernelEx(&cfg, kern, p, sh, scale_log2);
    note_launch();
    if (err != cudaSuccess || sh.cluster > 0)
        return err;
    cfg.gridDim = dim3(static_cast<unsigned>(sh.grid), static_cast<unsigned>(sh.abreast), 1);
    cfg.blockDim = dim3(kJoinThreads, 1, 1);
    cfg.dynamicSmemBytes = 0;
    err = cudaLaunchKernelEx(&cfg, attention_decode_join_kernel<T, D>, p, sh);
    note_launch();
    return err;
}

}  // namespace

size_t attention_decode_workspace(int64_t n_seqs, int64_t n_heads, int64_t n_kv_heads,
                                  int64_t head_dim, int64_t capacity)
{
    const DecodeShape sh = decode_shape(n_seqs, n_heads, n_kv_heads, head_dim, capacity, sm_count_current());
    if (sh.cluster > 0)
        return 0;
    const size_t part = head_dim == 64 ? sizeof(Part<64>) : sizeof(Part<128>);
    return static_cast<size_t>(sh.grid) * sh.abreast * (2 * part + sizeof(Begun));
}

cudaError_t launch_attention_decode(const DecodeProblem& p, cudaStream_t s)
{
    if (p.dtype == SOFTMAX_BF16)
        return p.head_dim == 64 ? launch<BF16Bits, 64>(p, s) : launch<BF16Bits, 128>(p, s);
    return p.head_dim == 64 ? launch<F16Bits, 64>(p, s) : launch<F16Bits, 128>(p, s);
}

unsigned read_error_attention_decode(bool clear)
{
    unsigned v = 0;
    if (cudaMemcpyFromSymbol(&v, g_error_attention_decode, sizeof v) != cudaSuccess)
        return 0;
    if (clear && v) {
        const unsigned zero = 0;
        cudaMemcpyToSymbol(g_error_attention_decode, &zero, sizeof zero);
    }
    return v;
}

}  // namespace rwsm
