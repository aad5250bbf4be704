// Layout and launchers of the paged entry cache (see csld_paged_cache in csld.h).  Internal.
#pragma once
#include "csld_internal.cuh"

namespace csld {

constexpr int kGroups = kNope / 32;                        // 14 groups of 32 dims
constexpr int kChunk = CSLD_PAGE_CHUNK;                    // 16 tokens
constexpr int kEntry4 = CSLD_ENTRY_FP4_BYTES;              // 368
constexpr int kChunk4Bytes = kChunk * kEntry4;             // 5888
constexpr int kChunk4Exp = kGroups * kChunk * 16;          // 3584: the exponent bytes
constexpr int kChunk4Rope = kChunk4Exp + kChunk * 16;      // 3840: the RoPE rows
static_assert(kChunk4Rope + kChunk * 2 * kRope == kChunk4Bytes, "an FP4 chunk's parts fill it");

// The cache as the kernels get it.
struct PagedView {
    uint8_t* pages;
    const int32_t* table;
    int32_t* seq_len;
    int64_t n_pages;
    int32_t page_size, max_pages, batch;
    __host__ __device__ int64_t capacity() const { return (int64_t)max_pages * page_size; }
};

// Angles of the RoPE pairs in turns per position: base^(-i/32) / (2 pi), formed on the host.
struct RopeTable {
    double turns[kRope / 2];
};

cudaError_t launch_append_paged(const PagedView& c, bool fp4, const uint16_t* kv_new, int64_t seq_stride,
                                int64_t token_stride, int T, const int32_t* n_new, const int32_t* start,
                                double rope_base, int32_t* err, cudaStream_t stream);
cudaError_t launch_read_paged(const PagedView& c, bool fp4, const int32_t* start, int64_t T, uint16_t* out,
                              int num_sms, int32_t* err, cudaStream_t stream);
// W = 0: every token up to the query's own.
size_t paged_attention_ws_bytes(int num_sms);
cudaError_t launch_paged_attention(const PagedView& c, bool fp4, const uint16_t* q, int heads, int Q, int W, int sinks,
                                   float scale, void* out, bool out_bf16, float* lse_out, void* ws, int num_sms,
                                   int32_t* err, cudaStream_t stream);

}  // namespace csld
