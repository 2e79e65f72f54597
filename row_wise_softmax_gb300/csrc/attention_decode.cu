// Attention of one new token of each sequence over a paged cache:
// o = softmax(scale q K^T) V over the sequence's cached tokens, with the
// running (m, l) softmax of "Triton GPU programming deep dive", section 3.3.
//
//   item     one (sequence, key/value head, block of up to 16 query heads of
//            its group); its tokens are cut into tiles of 64.
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
//   warp     16 tokens of each tile, on its own: its K and V rows arrive by
//            cp.async in its own ring of stages (no CTA barrier in the walk),
//            rows past the length as zeros.  S = Q K^T by mma.sync m16n8k16
//            with the group's heads as the 16 rows; the scores' accumulator
//            layout is the A operand of P V.
//
// Bound by bytes: every cached row is read once from memory, against
// 4 multiply-adds per byte and query head.
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
constexpr int kWarpTokens = 16;
constexpr int kTile = kWarps * kWarpTokens;        // tokens of a tile
constexpr int kStages = 3;
constexpr int kCtasPerSm = 2;

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
};

constexpr int kMaxCluster = 16;
constexpr int kClusterTiles = 8;                    // tiles per CTA up to which clusters are used

inline DecodeShape decode_shape(int64_t n_seqs, int64_t n_heads, int64_t n_kv, int64_t capacity,
                                int sm_count)
{
    DecodeShape s;
    s.group = static_cast<int32_t>(n_heads / n_kv);
    s.blocks = (s.group + kRows - 1) / kRows;
    const int64_t per = (capacity + kTile - 1) / kTile > 0 ? (capacity + kTile - 1) / kTile : 1;
    const int64_t most = static_cast<int64_t>(sm_count) * kCtasPerSm;
    const int64_t items = n_seqs * n_kv * s.blocks;
    s.cluster = 0;
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
    s.grid = static_cast<int32_t>(items >= most || items * per >= most ? most : items * per);
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
__device__ __forceinline__ int64_t tiles_of(int32_t n)
{
    return n == 0 ? 1 : (n + kTile - 1) / kTile;
}

// The CTA's run [begin, end) of all tiles, and the item it begins in.  Every
// thread gets the same answer.
struct Run {
    int64_t begin, end;                             // tiles
    int64_t total, runs;
    int64_t seq;                                    // sequence of the first tile
    int64_t before;                                 // tiles of the sequences before it
};

__device__ Run find_run(const DecodeProblem& p, int inner, int64_t* scratch)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int64_t mine = 0;
    for (int64_t b = tid; b < p.n_seqs; b += kThreads) {
        bool bad;
        mine += tiles_of(length_of(p, b, bad));
        if (bad && blockIdx.x == 0)
            atomicOr(&g_error_attention_decode, kErrBadIndex);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0)
        scratch[warp] = mine;
    __syncthreads();
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        total += scratch[w];
    total *= inner;
    Run r;
    // No run is empty but those of the CTAs past the last tile: an item's
    // parts lie in consecutive CTAs.
    r.total = total;
    r.runs = total < gridDim.x ? total : gridDim.x;
    r.begin = blockIdx.x < r.runs ? total * blockIdx.x / r.runs : 0;
    r.end = blockIdx.x < r.runs ? total * (blockIdx.x + 1) / r.runs : 0;
    r.seq = 0;
    r.before = 0;
    // Walk the sequences 32 at a time to the one that holds tile `begin`.
    if (r.begin < r.end) {
        for (int64_t b0 = 0; b0 < p.n_seqs; b0 += 32) {
            bool bad;
            const int64_t n = b0 + lane < p.n_seqs
                                  ? tiles_of(length_of(p, b0 + lane, bad)) * inner : 0;
            int64_t sum = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t up = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o)
                    sum += up;
            }
            const unsigned past = __ballot_sync(0xffffffffu, r.before + sum > r.begin);
            if (past) {
                const int at = __ffs(past) - 1;
                r.before += shfl64(sum - n, at);
                r.seq = b0 + at;
                break;
            }
            r.before += shfl64(sum, 31);
        }
    }
    return r;
}

template <typename T, int D, bool CLUSTER>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
attention_decode_kernel(const DecodeProblem p, const DecodeShape sh, float scale_log2)
{
    constexpr int KS = D / 16;                      // k-steps over the head dimension
    constexpr int DB = D / 8;                       // 8-wide output column blocks
    constexpr int CH = D / 8;                       // 16-byte chunks of a row
    constexpr uint32_t BLK = kWarpTokens * D * 2;   // bytes of a warp's K (or V) block
    extern __shared__ __align__(128) unsigned char dec_smem[];
    __shared__ float sm_m[kWarps][kRows], sm_l[kWarps][kRows];
    __shared__ int64_t sm_scratch[kWarps];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int inner = p.cache.n_kv_heads * sh.blocks;
    const uint32_t ring = smem_addr(dec_smem) + warp * (kStages * 2 * BLK);
    float* const sm_o = reinterpret_cast<float*>(dec_smem);          // [kWarps][kRows][D]
    Part<D>* const parts = static_cast<Part<D>*>(p.workspace);
    Begun* const begun = reinterpret_cast<Begun*>(parts + 2 * static_cast<int64_t>(sh.grid));

    pdl_launch_dependents();
    pdl_wait();
    // The CTA's pieces: runs of tiles of items.  Cluster form: one piece, its
    // tiles every `step`; run form: consecutive tiles, several items in turn.
    const int step = CLUSTER ? sh.cluster : 1;
    const int crank = CLUSTER ? static_cast<int>(blockIdx.x % static_cast<unsigned>(sh.cluster)) : 0;
    Run run = {};
    if constexpr (CLUSTER) {
        run.end = 1;
    } else {
        run = find_run(p, inner, sm_scratch);
    }
    int64_t seq = run.seq, before = run.before;
    int64_t begun_item = -1, begun_last = 0;

    const int r_a = lane >> 2, c_q = (lane & 3) * 2;
    for (int64_t at = run.begin; at < run.end;) {
        // ---- the piece: tiles t0, t0 + step, ... below t1 of item (seq, in)
        bool bad_len;
        int32_t len;
        int in;
        int64_t nt, first = 0, t0, t1;
        int32_t page0 = -1;                         // cluster form: the first tile's page
        if constexpr (CLUSTER) {
            const int64_t item = blockIdx.x / static_cast<unsigned>(sh.cluster);
            seq = item / inner;
            in = static_cast<int>(item - seq * inner);
            const int32_t tok = crank * kTile + warp * kWarpTokens + (lane & 15);
            if (tok < p.cache.capacity)             // in flight beside the length
                page0 = __ldg(p.cache.table + seq * p.cache.table_stride + divide(tok, p.cache.page));
            len = length_of(p, seq, bad_len);
            nt = tiles_of(len);
            t0 = crank;
            t1 = nt;
        } else {
            len = length_of(p, seq, bad_len);
            nt = tiles_of(len);
            while (at >= before + nt * inner) {     // next sequence
                before += nt * inner;
                ++seq;
                len = length_of(p, seq, bad_len);
                nt = tiles_of(len);
            }
            in = static_cast<int>((at - before) / nt);
            first = before + in * nt;               // the item's first tile among all
            t0 = at - first;
            t1 = run.end - first < nt ? run.end - first : nt;
        }
        const int kvh = in / sh.blocks, hb = in - kvh * sh.blocks;
        const int h0 = kvh * sh.group + hb * kRows;
        const int rows = sh.group - hb * kRows < kRows ? sh.group - hb * kRows : kRows;

        // Q fragments (A operand): rows past the group are zero.
        uint32_t qa[KS][4];
        {
            const unsigned short* gq = static_cast<const unsigned short*>(p.q.data) +
                                       seq * p.q.row + static_cast<int64_t>(h0) * p.q.head;
#pragma unroll
            for (int kk = 0; kk < KS; ++kk)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int r = r_a + (e & 1) * 8, c = kk * 16 + (e >> 1) * 8 + c_q;
                    qa[kk][e] = r < rows ? __ldg(reinterpret_cast<const unsigned*>(
                                               gq + r * p.q.head + c)) : 0u;
                }
        }
        const unsigned short* gk =
            static_cast<const unsigned short*>(p.cache.k) + kvh * p.cache.k_head;
        const unsigned short* gv =
            static_cast<const unsigned short*>(p.cache.v) + kvh * p.cache.v_head;
        const int32_t* table = p.cache.table + seq * p.cache.table_stride;

        // Copy this warp's block of tile t into stage `st` of its ring: lanes
        // 0..15 look up their token's K row, lanes 16..31 its V row.
        bool bad = bad_len;
        if (CLUSTER && bad_len && crank == 0 && tid == 0)
            atomicOr(&g_error_attention_decode, kErrBadIndex);
        auto issue = [&](int64_t t, int st) {
            const uint32_t dst = ring + static_cast<uint32_t>(st) * (2 * BLK);
            const int32_t tok = static_cast<int32_t>(t * kTile) + warp * kWarpTokens + (lane & 15);
            int64_t off = -1;
            if (tok < len) {
                const uint32_t slot = divide(tok, p.cache.page);
                const int32_t page = CLUSTER && t == t0 ? page0 : __ldg(table + slot);
                if (page >= 0 && page < p.cache.n_pages) {
                    const int64_t row = tok - slot * p.cache.page.d;
                    off = lane < 16 ? page * p.cache.k_page + row * p.cache.k_row
                                    : page * p.cache.v_page + row * p.cache.v_row;
                } else {
                    bad = true;
                }
            }
#pragma unroll
            for (int i = 0; i < kWarpTokens * CH / 32; ++i) {
                const int r = (i * 32 + lane) / CH, c = (i * 32 + lane) % CH;
                const int64_t ko = shfl64(off, r), vo = shfl64(off, r + 16);
                cp_async16_zfill(dst + tile_off<D>(r, c), gk + (ko < 0 ? 0 : ko + c * 8),
                                 ko < 0 ? 0 : 16);
                cp_async16_zfill(dst + BLK + tile_off<D>(r, c), gv + (vo < 0 ? 0 : vo + c * 8),
                                 vo < 0 ? 0 : 16);
            }
        };

        float m_a = kNegInf, m_b = kNegInf, l_a = 0.0f, l_b = 0.0f;
        float acc[DB][4];
#pragma unroll
        for (int i = 0; i < DB; ++i)
            acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) {
            if (t0 + i * step < t1)
                issue(t0 + i * step, i);
            cp_async_commit();
        }
        int now = 0;                                // the stage of tile t
        for (int64_t t = t0; t < t1; t += step) {
            if (t + (kStages - 1) * step < t1)
                issue(t + (kStages - 1) * step, now == 0 ? kStages - 1 : now - 1);
            cp_async_commit();
            asm volatile("cp.async.wait_group %0;" :: "n"(kStages - 1) : "memory");
            __syncwarp();
            const uint32_t sK = ring + static_cast<uint32_t>(now) * (2 * BLK);
            now = now + 1 == kStages ? 0 : now + 1;
            const uint32_t sV = sK + BLK;
            const int mi = lane >> 3;

            float s[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0f;
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) {
                uint32_t bk[4];
                ldsm_x4(bk, sK + tile_off<D>((lane & 7) + (mi >> 1) * 8, kk * 2 + (mi & 1)));
                MmaType<T>::mma(s[0], qa[kk], bk[0], bk[1]);
                MmaType<T>::mma(s[1], qa[kk], bk[2], bk[3]);
            }
            const int32_t j0 = static_cast<int32_t>(t * kTile) + warp * kWarpTokens;
            float mx_a = kNegInf, mx_b = kNegInf;
#pragma unroll
            for (int nb = 0; nb < 2; ++nb)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const bool past = j0 + nb * 8 + c_q + e >= len;
                    const float xa = past ? kNegInf : s[nb][e] * scale_log2;
                    const float xb = past ? kNegInf : s[nb][2 + e] * scale_log2;
                    s[nb][e] = xa;
                    s[nb][2 + e] = xb;
                    mx_a = fmaxf(mx_a, xa);
                    mx_b = fmaxf(mx_b, xb);
                }
            mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, 1));
            mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, 2));
            mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, 1));
            mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, 2));
            const float mn_a = fmaxf(m_a, mx_a), mn_b = fmaxf(m_b, mx_b);
            const float ref_a = mn_a == kNegInf ? 0.0f : mn_a;
            const float ref_b = mn_b == kNegInf ? 0.0f : mn_b;
            const float al_a = ex2_ftz(m_a - ref_a), al_b = ex2_ftz(m_b - ref_b);
            m_a = mn_a;
            m_b = mn_b;
            l_a *= al_a;
            l_b *= al_b;
#pragma unroll
            for (int i = 0; i < DB; ++i) {
                acc[i][0] *= al_a; acc[i][1] *= al_a;
                acc[i][2] *= al_b; acc[i][3] *= al_b;
            }
            uint32_t pa[4];
#pragma unroll
            for (int nb = 0; nb < 2; ++nb) {
                const float p0 = ex2_ftz(s[nb][0] - ref_a), p1 = ex2_ftz(s[nb][1] - ref_a);
                const float p2 = ex2_ftz(s[nb][2] - ref_b), p3 = ex2_ftz(s[nb][3] - ref_b);
                l_a += p0 + p1;
                l_b += p2 + p3;
                pa[nb * 2 + 0] = Elem<T>::pack2(p0, p1);
                pa[nb * 2 + 1] = Elem<T>::pack2(p2, p3);
            }
#pragma unroll
            for (int dp = 0; dp < D / 16; ++dp) {
                uint32_t bv[4];
                ldsm_x4_trans(bv, sV + tile_off<D>((lane & 7) + (mi & 1) * 8, dp * 2 + (mi >> 1)));
                MmaType<T>::mma(acc[2 * dp], pa, bv[0], bv[1]);
                MmaType<T>::mma(acc[2 * dp + 1], pa, bv[2], bv[3]);
            }
            __syncwarp();                           // the stage may be refilled
        }
        cp_async_wait_all_groups();

        // ---- the four warps' (m, l, O) into one
        l_a += __shfl_xor_sync(0xffffffffu, l_a, 1);
        l_a += __shfl_xor_sync(0xffffffffu, l_a, 2);
        l_b += __shfl_xor_sync(0xffffffffu, l_b, 1);
        l_b += __shfl_xor_sync(0xffffffffu, l_b, 2);
        if (__any_sync(0xffffffffu, bad)) {         // a bad page or length: NaN
            l_a = l_b = __int_as_float(0x7fc00000);
            if (lane == 0)
                atomicOr(&g_error_attention_decode, kErrBadIndex);
        }
        if ((lane & 3) == 0) {
            sm_m[warp][r_a] = m_a;
            sm_m[warp][r_a + 8] = m_b;
            sm_l[warp][r_a] = l_a;
            sm_l[warp][r_a + 8] = l_b;
        }
        __syncthreads();                            // and every warp's ring is free
        float M_a = kNegInf, M_b = kNegInf;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            M_a = fmaxf(M_a, sm_m[w][r_a]);
            M_b = fmaxf(M_b, sm_m[w][r_a + 8]);
        }
        const float f_a = M_a == kNegInf ? 0.0f : ex2_ftz(m_a - M_a);
        const float f_b = M_b == kNegInf ? 0.0f : ex2_ftz(m_b - M_b);
#pragma unroll
        for (int i = 0; i < DB; ++i) {
            float* const a = sm_o + (warp * kRows + r_a) * D + i * 8 + c_q;
            *reinterpret_cast<float2*>(a) = make_float2(acc[i][0] * f_a, acc[i][1] * f_a);
            *reinterpret_cast<float2*>(a + 8 * D) = make_float2(acc[i][2] * f_b, acc[i][3] * f_b);
        }
        __syncthreads();
        // Row r, columns c .. c + 3 of the four warps' sum, with its (m, l).
        auto sum_of = [&](int r, int c, float& M, float& L) {
            M = kNegInf;
            L = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                M = fmaxf(M, sm_m[w][r]);
            const float ref = M == kNegInf ? 0.0f : M;
            float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                L += sm_l[w][r] * ex2_ftz(sm_m[w][r] - ref);
                const float4 x = *reinterpret_cast<const float4*>(sm_o + (w * kRows + r) * D + c);
                o.x += x.x; o.y += x.y; o.z += x.z; o.w += x.w;
            }
            return o;
        };
        auto store = [&](int r, int c, const float4& o, float M, float L) {
            const float inv = 1.0f / L;
            uint2 w2;
            w2.x = Elem<T>::pack2(o.x * inv, o.y * inv);
            w2.y = Elem<T>::pack2(o.z * inv, o.w * inv);
            *reinterpret_cast<uint2*>(static_cast<unsigned short*>(p.o.data) + seq * p.o.row +
                                      static_cast<int64_t>(h0 + r) * p.o.head + c) = w2;
            if (p.lse && c == 0)
                p.lse[seq * p.n_heads + h0 + r] =
                    L == 0.0f ? kNegInf : (M + __log2f(L)) * 0.69314718055994531f;
        };
        if constexpr (CLUSTER) {
            // Each CTA leaves its sum in the place of warp 0's; then CTA r
            // merges every cluster-th group of four columns of all of them, in
            // the order of the CTAs.
            namespace cg = cooperative_groups;
            if (sh.cluster > 1) {
                float M[kRows * D / 4 / kThreads], L[kRows * D / 4 / kThreads];
                float4 o[kRows * D / 4 / kThreads];
#pragma unroll
                for (int j = 0; j < kRows * D / 4 / kThreads; ++j) {
                    const int i = tid + j * kThreads;
                    o[j] = sum_of(i / (D / 4), (i % (D / 4)) * 4, M[j], L[j]);
                }
                __syncthreads();
#pragma unroll
                for (int j = 0; j < kRows * D / 4 / kThreads; ++j) {
                    const int i = tid + j * kThreads, r = i / (D / 4), c = (i % (D / 4)) * 4;
                    *reinterpret_cast<float4*>(sm_o + r * D + c) = o[j];
                    if (c == 0) {
                        sm_m[0][r] = M[j];
                        sm_l[0][r] = L[j];
                    }
                }
                cg::cluster_group cluster = cg::this_cluster();
                cluster.sync();
                for (int i = crank + tid * sh.cluster; i < rows * (D / 4);
                     i += kThreads * sh.cluster) {
                    const int r = i / (D / 4), c = (i % (D / 4)) * 4;
                    float Mx = kNegInf, Lx = 0.0f;
                    for (int q = 0; q < sh.cluster; ++q)
                        Mx = fmaxf(Mx, *cluster.map_shared_rank(&sm_m[0][r], q));
                    const float ref = Mx == kNegInf ? 0.0f : Mx;
                    float4 acc4 = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
                    for (int q = 0; q < sh.cluster; ++q) {
                        const float f = ex2_ftz(*cluster.map_shared_rank(&sm_m[0][r], q) - ref);
                        const float4 x = *reinterpret_cast<const float4*>(
                            cluster.map_shared_rank(sm_o + r * D + c, q));
                        Lx += *cluster.map_shared_rank(&sm_l[0][r], q) * f;
                        acc4.x += x.x * f; acc4.y += x.y * f; acc4.z += x.z * f; acc4.w += x.w * f;
                    }
                    store(r, c, acc4, Mx, Lx);
                }
                cluster.sync();                     // read before a CTA leaves
            } else {
                for (int i = tid; i < rows * (D / 4); i += kThreads) {
                    float M, L;
                    const float4 o = sum_of(i / (D / 4), (i % (D / 4)) * 4, M, L);
                    store(i / (D / 4), (i % (D / 4)) * 4, o, M, L);
                }
            }
            return;
        }
        const bool whole = t0 == 0 && t1 == nt;
        Part<D>* const part = parts + 2 * static_cast<int64_t>(blockIdx.x) + (t0 == 0 ? 1 : 0);
        for (int i = tid; i < rows * (D / 4); i += kThreads) {
            const int r = i / (D / 4), c = (i % (D / 4)) * 4;
            float M, L;
            const float4 o = sum_of(r, c, M, L);
            if (whole) {
                store(r, c, o, M, L);
            } else {
                *reinterpret_cast<float4*>(part->o + r * D + c) = o;
                if (c == 0) {
                    part->m[r] = M;
                    part->l[r] = L;
                }
            }
        }
        if (!whole && t0 == 0) {
            // The run that holds the item's last tile.
            const int64_t last = first + nt - 1;
            begun_item = seq * inner + in;
            int64_t c = last * run.runs / run.total;
            while (run.total * (c + 1) / run.runs <= last)
                ++c;
            while (run.total * c / run.runs > last)
                --c;
            begun_last = c;
        }
        at = first + t1;
        __syncthreads();                            // sm_o is a ring again
    }
    if (tid == 0)
        begun[blockIdx.x] = Begun{begun_item, begun_last};
}

// Merge the parts of the item that CTA blockIdx.x of the main kernel began
// and did not end: slot 1 of that CTA, then slot 0 of each CTA up to the last.
// A warp per query head.
template <typename T, int D>
__global__ void __launch_bounds__(kRows * 32)
attention_decode_join_kernel(const DecodeProblem p, const DecodeShape sh)
{
    constexpr int E = D / 32;                       // elements per lane
    const int lane = threadIdx.x & 31, r = threadIdx.x >> 5;
    const Part<D>* const parts = static_cast<const Part<D>*>(p.workspace);
    const Begun* const begun =
        reinterpret_cast<const Begun*>(parts + 2 * static_cast<int64_t>(sh.grid));
    pdl_launch_dependents();
    pdl_wait();
    const Begun g = begun[blockIdx.x];
    if (g.item < 0)
        return;
    const int inner = p.cache.n_kv_heads * sh.blocks;
    const int64_t seq = g.item / inner;
    const int in = static_cast<int>(g.item - seq * inner);
    const int kvh = in / sh.blocks, hb = in - kvh * sh.blocks;
    const int rows = sh.group - hb * kRows < kRows ? sh.group - hb * kRows : kRows;
    if (r >= rows)
        return;
    const int n = static_cast<int>(g.last - blockIdx.x) + 1;
    auto part = [&](int i) {
        return parts + 2 * (static_cast<int64_t>(blockIdx.x) + i) + (i == 0 ? 1 : 0);
    };
    float M = kNegInf;
    for (int i = lane; i < n; i += 32)
        M = fmaxf(M, part(i)->m[r]);
    M = warp_max(M);
    const float ref = M == kNegInf ? 0.0f : M;
    float L = 0.0f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e)
        o[e] = 0.0f;
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
        const Part<D>* const q = part(i);
        const float f = ex2_ftz(q->m[r] - ref);
        L += q->l[r] * f;
        float x[E];
        if constexpr (E == 4) {
            const float4 w = *reinterpret_cast<const float4*>(q->o + r * D + lane * E);
            x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w;
        } else {
            const float2 w = *reinterpret_cast<const float2*>(q->o + r * D + lane * E);
            x[0] = w.x; x[1] = w.y;
        }
#pragma unroll
        for (int e = 0; e < E; ++e)
            o[e] += x[e] * f;
    }
    const float inv = 1.0f / L;
    const int h = kvh * sh.group + hb * kRows + r;
    unsigned* const dst = reinterpret_cast<unsigned*>(
        static_cast<unsigned short*>(p.o.data) + seq * p.o.row +
        static_cast<int64_t>(h) * p.o.head + lane * E);
#pragma unroll
    for (int e = 0; e < E; e += 2)
        dst[e / 2] = Elem<T>::pack2(o[e] * inv, o[e + 1] * inv);
    if (p.lse && lane == 0)
        p.lse[seq * p.n_heads + h] =
            L == 0.0f ? kNegInf : (M + __log2f(L)) * 0.69314718055994531f;
}

template <typename T, int D>
cudaError_t launch(const DecodeProblem& p, cudaStream_t s)
{
    const DecodeShape sh = decode_shape(p.n_seqs, p.n_heads, p.cache.n_kv_heads, p.cache.capacity,
                                        sm_count_current());
    auto* kern = sh.cluster > 0 ? attention_decode_kernel<T, D, true>
                                : attention_decode_kernel<T, D, false>;
    const int smem = kWarps * kStages * 2 * kWarpTokens * D * 2;
    static_assert(kWarps * kRows * D * 4 <= kWarps * kStages * 2 * kWarpTokens * D * 2,
                  "the warps' O rows fit in the rings");
    static std::atomic<bool> attr_set[2][64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return cudaErrorInvalidDevice;
    if (!attr_set[sh.cluster > 0][dev].load()) {
        cudaError_t e =
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess && sh.cluster > 0)
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess)
            return e;
        attr_set[sh.cluster > 0][dev].store(true);
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
    cfg.blockDim = dim3(kRows * 32, 1, 1);
    cfg.dynamicSmemBytes = 0;
    err = cudaLaunchKernelEx(&cfg, attention_decode_join_kernel<T, D>, p, sh);
    note_launch();
    return err;
}

}  // namespace

size_t attention_decode_workspace(int64_t n_seqs, int64_t n_heads, int64_t n_kv_heads,
                                  int64_t head_dim, int64_t capacity)
{
    const DecodeShape sh = decode_shape(n_seqs, n_heads, n_kv_heads, capacity, sm_count_current());
    if (sh.cluster > 0)
        return 0;
    const size_t part = head_dim == 64 ? sizeof(Part<64>) : sizeof(Part<128>);
    return static_cast<size_t>(sh.grid) * (2 * part + sizeof(Begun));
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
