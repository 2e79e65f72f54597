// Problems and launchers of the serving operators (declared in
// include/softmax.h): cache append with position rotation, packed prompt
// attention, single-token attention over a paged cache.
#pragma once

#include "kernels.h"

namespace rwsm {

// Error word bit of a kernel that met an index leading out of its tensors
// (kErrMbarrierTimeout is bit 0).
enum : unsigned { kErrBadIndex = 2u };

// A [rows][heads][head_dim] tensor, strides in elements.
struct Heads {
    void* data;
    int64_t row, head;
};

// Division of n < 2^31 by an invariant d >= 1 ("Division by invariant
// integers using multiplication", Granlund and Montgomery, PLDI 1994): with
// l = ceil(log2 d) and m = floor(2^(31+l) / d) + 1, n / d = n m / 2^(31+l).
struct Divisor {
    uint32_t d, mul, shift;             // d == 1: shift is unused
};

inline Divisor divisor_of(uint32_t d)
{
    uint32_t l = 0;
    while ((uint64_t{1} << l) < d)
        ++l;
    const uint32_t mul =
        d == 1 ? 0u
               : static_cast<uint32_t>(((static_cast<unsigned __int128>(1) << (31 + l)) / d) + 1);
    return Divisor{d, mul, l == 0 ? 0u : l - 1};
}

#ifdef __CUDACC__
__device__ __forceinline__ uint32_t divide(uint32_t n, const Divisor& v)
{
    return v.d == 1 ? n : __umulhi(n, v.mul) >> v.shift;
}
#endif

struct PagedCache {
    void* k;
    void* v;
    const int32_t* table;
    int64_t k_page, k_row, k_head, v_page, v_row, v_head;
    int64_t n_seqs, table_stride;
    int32_t n_pages, table_width, n_kv_heads, capacity;      // capacity: tokens of a table row
    Divisor page;
    // K and V have the same strides, and every row begins less than 2^31 units
    // of 16 bytes into its cache.
    bool near_rows;
};

struct AppendProblem {
    PagedCache cache;
    Heads k, v, q, q_out;               // q.data null: keys and values only
    const int32_t* positions;
    const int32_t* seq_ids;             // null: token t belongs to sequence t
    const double* inv_freq;
    int64_t n_tokens;
    int32_t n_heads, head_dim, rot_dim, interleaved, dtype;
};
cudaError_t launch_kv_append(const AppendProblem& p, cudaStream_t s);

struct DecodeProblem {
    PagedCache cache;
    Heads q, o;
    float* lse;
    const int32_t* lengths;
    void* workspace;
    int64_t n_seqs;
    int32_t n_heads, head_dim, dtype;
    float scale;
};
cudaError_t launch_attention_decode(const DecodeProblem& p, cudaStream_t s);
size_t attention_decode_workspace(int64_t n_seqs, int64_t n_heads, int64_t n_kv_heads,
                                  int64_t head_dim, int64_t capacity);

struct PackedProblem {
    Heads q, k, v, o;
    float* lse;
    const int32_t* cu_q;
    const int32_t* cu_k;
    int64_t n_seqs, total_q, total_k;
    int32_t n_heads, n_kv_heads, head_dim, causal, dtype;
    float scale;
    void* workspace;
};
cudaError_t launch_attention_packed(const PackedProblem& p, cudaStream_t s);
size_t attention_packed_workspace(int64_t n_seqs, int64_t total_q, int64_t total_k,
                                  int64_t n_heads, int64_t n_kv_heads, int64_t head_dim);

unsigned read_error_kv_append(bool clear);
unsigned read_error_attention_decode(bool clear);
unsigned read_error_attention_packed(bool clear);

// A device of the architecture this library is built for is current.
bool usable_device();

}  // namespace rwsm
