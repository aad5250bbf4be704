// Attention over the paged entry cache: sliding window with first tokens that stay visible, or every
// token (layouts: csld_paged_cache in csld.h).
//
// One CTA per (sequence, query, group of 16 heads), one warp per head.  The visible tokens come in tiles
// of 32, decoded to fp32 in shared memory; a warp's lane scores one token of the tile, the warp keeps a
// running maximum and sum, and each lane adds its 16 dims of the output.
#include "paged.cuh"

namespace csld {

namespace {

constexpr int kTile = 32, kPad = kDim + 1;

template <bool kFp4>
__device__ __forceinline__ float entry_value(const PagedView& c, int64_t pg, int in_page, int d) {
    if constexpr (!kFp4) {
        const uint8_t* e = c.pages + (pg * c.page_size + in_page) * kEntry;
        if (d < kNope) return e4m3_to_f32(e[d]);
        return bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(e + kNope)[d - kNope]);
    } else {
        const uint8_t* ch = c.pages + (pg * c.page_size + (in_page & ~(kChunk - 1))) * kEntry4;
        const int tk = in_page & (kChunk - 1);
        if (d >= kNope) return bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(ch + kChunk4Rope + tk * 2 * kRope)[d - kNope]);
        const int g = d >> 5, i = d & 7;
        const uint32_t w = *reinterpret_cast<const uint32_t*>(ch + g * 256 + tk * 16 + 4 * ((d & 31) >> 3));
        const uint32_t ex = ch[kChunk4Exp + g * kChunk + tk];
        const float s = ex == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float(ex << 23);
        const float m = static_cast<float>(__byte_perm(kTwiceE2M1Lo, kTwiceE2M1Hi, (w >> (4 * i)) & 7u) & 0xFFu) * 0.5f * s;
        return (w >> (i < 4 ? 8 * i + 7 : 8 * (i - 4) + 3)) & 1u ? -m : m;
    }
}

template <bool kFp4>
__global__ void __launch_bounds__(512) paged_attention_kernel(const PagedView c, const uint16_t* __restrict__ q, int heads,
                                                              int Q, int W, int sinks, float scale, void* __restrict__ out,
                                                              bool out_bf16, float* __restrict__ lse_out, int32_t* err) {
    extern __shared__ float kv[];   // [kTile][kPad], then q [16][512]
    float* qs = kv + kTile * kPad;
    __shared__ int seen[kTile];
    const int row = blockIdx.x, hg = blockIdx.y, b = row / Q, j = row % Q;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, h = hg * 16 + warp;
    pdl_wait();
    pdl_trigger();
    int64_t n = c.seq_len[b];
    if (n < 0 && tid == 0) dev_error(err, CSLD_DEVERR_SEQ_LEN);
    if (n > c.capacity() && tid == 0) dev_error(err, CSLD_DEVERR_SEQ_LEN);
    n = min64(max64(n, 0), c.capacity());
    const int64_t p = n - Q + j;
    for (int i = tid; i < 16 * kDim; i += 512) {
        const int hh = hg * 16 + i / kDim;
        qs[i] = hh < heads ? bf16_bits_to_f32(q[((int64_t)row * heads + hh) * kDim + i % kDim]) : 0.f;
    }
    const int64_t lo = W > 0 ? max64(0, p - W + 1) : 0, first = min64(sinks, lo);
    const int64_t total = p < 0 ? 0 : first + (p + 1 - lo);
    float m = -INFINITY, l = 0.f, o[16];
    for (int k = 0; k < 16; ++k) o[k] = 0.f;
    for (int64_t i0 = 0; i0 < total; i0 += kTile) {
        __syncthreads();
        for (int e = warp; e < kTile; e += 16) {
            const int64_t i = i0 + e, t = i < first ? i : lo + i - first;
            int64_t pg = -1;
            if (i < total) {
                pg = c.table[(int64_t)b * c.max_pages + t / c.page_size];
                if (pg < 0 || pg >= c.n_pages) {
                    if (lane == 0) dev_error(err, CSLD_DEVERR_PAGE);
                    pg = -1;
                }
            }
            if (lane == 0) seen[e] = pg >= 0;
            for (int d = lane; d < kDim; d += 32)
                kv[e * kPad + d] = pg >= 0 ? entry_value<kFp4>(c, pg, static_cast<int>(t % c.page_size), d) : 0.f;
        }
        __syncthreads();
        float x = 0.f;
        for (int d = 0; d < kDim; ++d) x = fmaf(qs[warp * kDim + d], kv[lane * kPad + d], x);
        x = seen[lane] ? x * scale * 1.4426950408889634f : -INFINITY;
        float tm = x;
        for (int s = 16; s > 0; s >>= 1) {
            const float y = __shfl_xor_sync(0xffffffffu, tm, s);
            tm = tm != tm || y != y ? NAN : fmaxf(tm, y);
        }
        const float mn = m != m || tm != tm ? NAN : fmaxf(m, tm);
        if (mn == -INFINITY) continue;
        const float f = exp2f(m - mn), w = exp2f(x - mn);
        l = l * f + w;
        for (int k = 0; k < 16; ++k) o[k] *= f;
        for (int e = 0; e < kTile; ++e) {
            const float we = __shfl_sync(0xffffffffu, w, e);
            for (int k = 0; k < 16; ++k) o[k] = fmaf(we, kv[e * kPad + lane + 32 * k], o[k]);
        }
        m = mn;
    }
    for (int s = 16; s > 0; s >>= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
    if (h >= heads) return;
    const int64_t at = (int64_t)row * heads + h;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int k = 0; k < 16; ++k) {
        if (out_bf16) reinterpret_cast<uint16_t*>(out)[at * kDim + lane + 32 * k] = static_cast<uint16_t>(f32_to_bf16_bits(o[k] * inv));
        else reinterpret_cast<float*>(out)[at * kDim + lane + 32 * k] = o[k] * inv;
    }
    if (lse_out && lane == 0) lse_out[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace

size_t paged_attention_ws_bytes(int num_sms) { return (size_t)num_sms * 256; }

cudaError_t launch_paged_attention(const PagedView& c, bool fp4, const uint16_t* q, int heads, int Q, int W, int sinks,
                                   float scale, void* out, bool out_bf16, float* lse_out, void* ws, int num_sms,
                                   int32_t* err, cudaStream_t stream) {
    const size_t smem = (kTile * kPad + 16 * kDim) * sizeof(float);
    auto kernel = fp4 ? paged_attention_kernel<true> : paged_attention_kernel<false>;
    cudaError_t e = set_smem_once(kernel, smem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kernel, dim3(c.batch * Q, (heads + 15) / 16), dim3(512), smem, stream, c, q, heads, Q, W, sinks, scale,
                   out, out_bf16, lse_out, err);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace csld
