// Append to and read-back from the paged entry cache (layouts: csld_paged_cache in csld.h).
//
// Source: "DeepSeek-V4: a million-token context that agents can actually use" -- storage paragraph
// (entries in low precision except the RoPE dims in bf16); velog.io paper review, KV-cache-layout
// section (state kept per sequence beside the compressed caches).
#include <cmath>
#include <type_traits>

#include "paged.cuh"

namespace csld {

namespace {

constexpr int kAppendWarps = 8;

// Eight values as E2M1 codes in the cache's word layout: the codes from the hardware's paired converts (nearest, ties
// to the even code, saturating), then the signs moved (nibble i's from bit 4i + 3 to the middle of the bytes).
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("{\n .reg .b8 t;\n cvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n cvt.u32.u8 %0, t;\n}\n" : "=r"(b[i]) : "f"(v[2 * i]), "f"(v[2 * i + 1]));
    const uint32_t w = b[0] | (b[1] << 8) | (b[2] << 16) | (b[3] << 24);
    const uint32_t lo = __byte_perm(w, 0u, 0x1100), hi = __byte_perm(w, 0u, 0x3322);   // byte i: that of nibble i, 4 + i
    return (w & 0x77777777u) | ((lo << 4) & 0x00800080u) | (lo & 0x80008000u) | (hi & 0x00080008u) | ((hi >> 4) & 0x08000800u);
}

// What one sequence appends, the same answer in every thread of the CTA: positions s .. s + n - 1,
// or ok = false where it is refused as a whole.  Reads the page table over the new range.
struct AppendSpan {
    int64_t s;
    int n;
    bool ok;
};
__device__ __forceinline__ AppendSpan append_span(const PagedView& c, int b, int T, const int32_t* n_new,
                                                  const int32_t* start, bool report, int32_t* err) {
    AppendSpan a;
    a.s = start ? start[b] : c.seq_len[b];
    a.n = n_new ? n_new[b] : T;
    uint32_t flag = 0;
    if (a.s < 0 || a.n < 0 || a.n > T) flag = CSLD_DEVERR_SEQ_LEN;
    else if (a.s + a.n > c.capacity()) flag = CSLD_DEVERR_CAPACITY;
    bool bad = false;
    if (!flag && a.n > 0) {
        const int64_t p1 = (a.s + a.n - 1) / c.page_size;
        for (int64_t p = a.s / c.page_size + threadIdx.x; p <= p1; p += blockDim.x) {
            const int32_t pg = c.table[(int64_t)b * c.max_pages + p];
            bad |= pg < 0 || pg >= c.n_pages;
        }
    }
    if (__syncthreads_or(bad)) flag = CSLD_DEVERR_PAGE;
    if (flag && report && threadIdx.x == 0) dev_error(err, flag);
    a.ok = flag == 0;
    return a;
}

// One warp per token: lane l < 28 owns dims 16l..16l+15 of the 448, every lane one RoPE pair.  Moves
// 1024 B in and 576 or 368 B out per token; at one token per sequence (decode) it is a chain of three
// dependent loads (count, length, page; the token beside the length) and bound by their latency.  Every CTA reads
// the page table over the sequence's whole new range, all or nothing being stored: as much as the data
// itself at 800K tokens in pages of 64 (1M fp8 tokens at a time 528 us, eight appends of 128K 437).  The RoPE frequencies come in as
// kernel parameters and angles are reduced to a fraction of a turn in double, so the sine and cosine
// are cheap fp32 ones whatever the position.
// A warp takes kTokens tokens, the CTA's warps in turn; their loads are issued together.
template <bool kFp4, bool kRotate, int kTokens>
__global__ void __launch_bounds__(32 * kAppendWarps) append_paged_kernel(
    const PagedView c, const uint16_t* __restrict__ kv_new, int64_t seq_stride, int64_t token_stride, int T,
    const int32_t* __restrict__ n_new, const int32_t* __restrict__ start, const __grid_constant__ RopeTable rt,
    bool set_len, int32_t* err) {
    const int b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    const int i0 = blockIdx.x * kAppendWarps * kTokens + warp;
    uint4 va[kTokens], vb[kTokens];
    uint32_t vr[kTokens];
    // rows past n_new are not read: where sequences lie closer than T rows they may end the caller's buffer
    const int n_in = n_new ? n_new[b] : T, n_rows = n_in <= T ? n_in : 0;
#pragma unroll
    for (int k = 0; k < kTokens; ++k) {
        const int i = i0 + k * kAppendWarps;
        va[k] = vb[k] = make_uint4(0, 0, 0, 0);
        vr[k] = 0;
        if (i < n_rows) {
            const uint16_t* x = kv_new + b * seq_stride + i * token_stride;
            if (lane < 28) {
                va[k] = __ldg(reinterpret_cast<const uint4*>(x) + 2 * lane);
                vb[k] = __ldg(reinterpret_cast<const uint4*>(x) + 2 * lane + 1);
            }
            vr[k] = __ldg(reinterpret_cast<const uint32_t*>(x + kNope) + lane);
        }
    }
    const AppendSpan a = append_span(c, b, T, n_new, start, blockIdx.x == 0, err);
    // set_len: no other CTA reads seq_len[b] (start is given, or this is the sequence's only CTA, whose
    // threads all read it before the barrier of append_span)
    if (set_len && a.ok && blockIdx.x == 0 && threadIdx.x == 0) c.seq_len[b] = static_cast<int32_t>(a.s + a.n);
    if (!a.ok) return;
#pragma unroll
    for (int k = 0; k < kTokens; ++k) {
        const int i = i0 + k * kAppendWarps;
        if (i >= a.n) return;   // whole warps
        const uint4 v0 = va[k], v1 = vb[k];
        uint32_t r = vr[k];
        const int64_t t = a.s + i;
        const int32_t pg = c.table[(int64_t)b * c.max_pages + t / c.page_size];
        const int in_page = static_cast<int>(t % c.page_size);
        if constexpr (kRotate) {
            const double turn = static_cast<double>(t) * rt.turns[lane];
            float sn, cs;
            sincospif(2.f * static_cast<float>(turn - rint(turn)), &sn, &cs);
            const float x0 = bf16_bits_to_f32(r), x1 = bf16_bits_to_f32(r >> 16);
            r = f32x2_to_bf16x2_bits(x0 * cs - x1 * sn, x0 * sn + x1 * cs);
        }
        const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
        if constexpr (!kFp4) {
            uint8_t* e = c.pages + ((int64_t)pg * c.page_size + in_page) * kEntry;
            if (lane < 28) {
                uint32_t o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t lo = __nv_cvt_float2_to_fp8x2(
                        make_float2(bf16_bits_to_f32(w[2 * k]), bf16_bits_to_f32(w[2 * k] >> 16)), __NV_SATFINITE, __NV_E4M3);
                    const uint32_t hi = __nv_cvt_float2_to_fp8x2(
                        make_float2(bf16_bits_to_f32(w[2 * k + 1]), bf16_bits_to_f32(w[2 * k + 1] >> 16)), __NV_SATFINITE, __NV_E4M3);
                    o[k] = (lo & 0xFFFFu) | (hi << 16);
                }
                reinterpret_cast<uint4*>(e)[lane] = make_uint4(o[0], o[1], o[2], o[3]);
            }
            reinterpret_cast<uint32_t*>(e + kNope)[lane] = r;
        } else {
            uint8_t* ch = c.pages + ((int64_t)pg * c.page_size + (in_page & ~(kChunk - 1))) * kEntry4;
            const int tk = in_page & (kChunk - 1);
            float amax = 0.f;
            bool nan = false;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float x0 = fabsf(bf16_bits_to_f32(w[k])), x1 = fabsf(bf16_bits_to_f32(w[k] >> 16));
                amax = fmaxf(amax, fmaxf(x0, x1));   // fmaxf drops NaNs
                nan |= x0 != x0 || x1 != x1;
            }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            nan |= __shfl_xor_sync(0xffffffffu, static_cast<int>(nan), 1) != 0;
            // 2^e0 <= amax < 2^(e0+1): sigma = 2^(e0-2) where amax <= 1.5 * 2^e0, else 2^(e0-1)
            int e = -126;
            if (amax > 0.f) {
                const uint32_t u = __float_as_uint(amax);
                e = static_cast<int>(u >> 23) - 127 - 2 + ((u & 0x7FFFFFu) > 0x400000u ? 1 : 0);
                e = max(-126, min(125, e));   // bf16 subnormals land on the clamp: their group is below 2^-126 * 6
            }
            const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
            uint32_t word[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float v[8];
#pragma unroll
                for (int d = 0; d < 4; ++d) {
                    v[2 * d] = bf16_bits_to_f32(w[4 * k + d]) * inv;
                    v[2 * d + 1] = bf16_bits_to_f32(w[4 * k + d] >> 16) * inv;
                }
                word[k] = e2m1x8(v);
            }
            const int ebyte = nan ? 255 : e + 127;
            const int emax = __reduce_max_sync(0xffffffffu, lane < 28 && !nan ? ebyte : 1);
            if (lane < 28) {
                *reinterpret_cast<uint2*>(ch + (lane >> 1) * 256 + tk * 16 + 8 * (lane & 1)) = make_uint2(word[0], word[1]);
                if (!(lane & 1)) ch[kChunk4Exp + (lane >> 1) * kChunk + tk] = static_cast<uint8_t>(ebyte);
            } else if (lane < 30) {
                ch[kChunk4Exp + (lane - 14) * kChunk + tk] = lane == 28 ? static_cast<uint8_t>(emax) : 0;
            }
            reinterpret_cast<uint32_t*>(ch + kChunk4Rope + tk * 2 * kRope)[lane] = r;
        }
    }
}

// seq_len += n where several CTAs of a sequence read it while appending: a launch of its own.
__global__ void __launch_bounds__(128) advance_paged_kernel(const PagedView c, int T, const int32_t* __restrict__ n_new) {
    pdl_wait();
    pdl_trigger();
    const AppendSpan a = append_span(c, blockIdx.x, T, n_new, nullptr, false, nullptr);
    if (a.ok && threadIdx.x == 0) c.seq_len[blockIdx.x] = static_cast<int32_t>(a.s + a.n);
}

// One warp per kReadTokens consecutive tokens, all their loads issued before the first store.
constexpr int kReadTokens = 4;
template <bool kFp4>
__global__ void __launch_bounds__(256) read_paged_kernel(const PagedView c, const int32_t* __restrict__ start, int64_t T,
                                                         uint16_t* __restrict__ out, int32_t* err) {
    const int lane = threadIdx.x & 31;
    pdl_wait();
    pdl_trigger();
    const int64_t per_seq = (T + kReadTokens - 1) / kReadTokens, n_items = per_seq * c.batch;
    const int64_t n_warps = (int64_t)gridDim.x * (blockDim.x >> 5);
    for (int64_t it = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); it < n_items; it += n_warps) {
        const int b = static_cast<int>(it / per_seq);
        const int64_t i0 = (it % per_seq) * kReadTokens;
        const int64_t t0 = (int64_t)start[b] + i0, n = c.seq_len[b];
        uint4 v[kReadTokens];
        uint32_t r[kReadTokens], ex[kReadTokens];
#pragma unroll
        for (int k = 0; k < kReadTokens; ++k) {
            const int64_t t = t0 + k;
            v[k] = make_uint4(0, 0, 0, 0);
            r[k] = 0;
            ex[k] = 127;
            if (i0 + k >= T || t < 0 || t >= n || t >= c.capacity()) continue;
            const int32_t pg = c.table[(int64_t)b * c.max_pages + t / c.page_size];
            if (pg < 0 || pg >= c.n_pages) {
                if (lane == 0) dev_error(err, CSLD_DEVERR_PAGE);
                continue;
            }
            const int in_page = static_cast<int>(t % c.page_size);
            if constexpr (!kFp4) {
                const uint8_t* e = c.pages + ((int64_t)pg * c.page_size + in_page) * kEntry;
                if (lane < 28) v[k] = *reinterpret_cast<const uint4*>(e + 16 * lane);
                r[k] = reinterpret_cast<const uint32_t*>(e + kNope)[lane];
            } else {
                const uint8_t* ch = c.pages + ((int64_t)pg * c.page_size + (in_page & ~(kChunk - 1))) * kEntry4;
                const int tk = in_page & (kChunk - 1);
                if (lane < 28) {
                    const uint2 u = *reinterpret_cast<const uint2*>(ch + (lane >> 1) * 256 + tk * 16 + 8 * (lane & 1));
                    v[k].x = u.x;
                    v[k].y = u.y;
                    ex[k] = ch[kChunk4Exp + (lane >> 1) * kChunk + tk];
                }
                r[k] = reinterpret_cast<const uint32_t*>(ch + kChunk4Rope + tk * 2 * kRope)[lane];
            }
        }
#pragma unroll
        for (int k = 0; k < kReadTokens; ++k) {
            if (i0 + k >= T) break;
            uint16_t* o = out + ((int64_t)b * T + i0 + k) * kDim;
            uint32_t w[8];
            if constexpr (!kFp4) {
                const uint32_t u[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t lo, hi;
                    e4m3x4_to_f16x2x2(u[q], lo, hi);
                    const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&lo));
                    const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&hi));
                    w[2 * q] = f32x2_to_bf16x2_bits(f0.x, f0.y);
                    w[2 * q + 1] = f32x2_to_bf16x2_bits(f1.x, f1.y);
                }
            } else {
                // bf16 values of the eight codes at this scale: (e + 126) in the exponent's place plus the code at the mantissa's
                // top bit, but for 0 and 1/2 (half the exponent step below 1; at the smallest scale a subnormal); split into two
                // byte tables, from which a byte permute takes four codes' upper or lower bytes at once
                const uint32_t b = (ex[k] - 1u) << 7, bb = b * 0x10001u;
                uint32_t t01 = (ex[k] == 1 ? 0x0040u : b) << 16, t23 = bb + 0x00C00080u, t45 = bb + 0x01400100u, t67 = bb + 0x01C00180u;
                if (ex[k] == 0) t01 = t23 = t45 = t67 = 0u;   // nothing was stored here
                if (ex[k] == 255) t01 = t23 = t45 = t67 = 0x7FC07FC0u;
                const uint32_t l0 = __byte_perm(t01, t23, 0x6420), l1 = __byte_perm(t45, t67, 0x6420);
                const uint32_t h0 = __byte_perm(t01, t23, 0x7531), h1 = __byte_perm(t45, t67, 0x7531);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const uint32_t word = u ? v[k].y : v[k].x, sel = word & 0x77777777u;
                    const uint32_t lo0 = __byte_perm(l0, l1, sel), lo1 = __byte_perm(l0, l1, sel >> 16);
                    const uint32_t hi0 = __byte_perm(h0, h1, sel) | (word & 0x80808080u);
                    const uint32_t hi1 = __byte_perm(h0, h1, sel >> 16) | ((word << 4) & 0x80808080u);
                    w[4 * u] = __byte_perm(lo0, hi0, 0x5140);
                    w[4 * u + 1] = __byte_perm(lo0, hi0, 0x7362);
                    w[4 * u + 2] = __byte_perm(lo1, hi1, 0x5140);
                    w[4 * u + 3] = __byte_perm(lo1, hi1, 0x7362);
                }
            }
            if (lane < 28) {
                reinterpret_cast<uint4*>(o)[2 * lane] = make_uint4(w[0], w[1], w[2], w[3]);
                reinterpret_cast<uint4*>(o)[2 * lane + 1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
            reinterpret_cast<uint32_t*>(o + kNope)[lane] = r[k];
        }
    }
}

}  // namespace

cudaError_t launch_append_paged(const PagedView& c, bool fp4, const uint16_t* kv_new, int64_t seq_stride,
                                int64_t token_stride, int T, const int32_t* n_new, const int32_t* start,
                                double rope_base, int32_t* err, cudaStream_t stream) {
    RopeTable rt = {};
    if (rope_base > 0.0)
        for (int i = 0; i < kRope / 2; ++i)
            rt.turns[i] = std::pow(rope_base, -i / 32.0) / 6.283185307179586476925286766559;
    // One token a warp, or four in long appends.  fp4, one token against four: 1 x 1,024 tokens 2.4 us against 3.8, 8 x 1,024
    // 5.7 against 6.6; 12 x 1,024 7.3 against 6.7, 64 x 1,024 31.0 against 25.8 (fp8 22.5 against 19.4).
    const bool many = (int64_t)T * c.batch > 8192;
    const int per_cta = kAppendWarps * (many ? 4 : 1);
    const dim3 grid((T + per_cta - 1) / per_cta, c.batch);
    const bool set_len = start != nullptr || grid.x == 1, turn = rope_base > 0.0;
    auto pick = [&](auto tokens) {
        constexpr int k = decltype(tokens)::value;
        return fp4 ? (turn ? append_paged_kernel<true, true, k> : append_paged_kernel<true, false, k>)
                   : (turn ? append_paged_kernel<false, true, k> : append_paged_kernel<false, false, k>);
    };
    auto kernel = many ? pick(std::integral_constant<int, 4>()) : pick(std::integral_constant<int, 1>());
    cudaError_t e = launch_pdl(kernel, grid, dim3(32 * kAppendWarps), 0, stream, c, kv_new, seq_stride, token_stride, T,
                               n_new, start, rt, set_len, err);
    if (e != cudaSuccess) return e;
    if (!set_len) {
        e = launch_pdl(advance_paged_kernel, dim3(c.batch), dim3(128), 0, stream, c, T, n_new);
        if (e != cudaSuccess) return e;
    }
    return cudaGetLastError();
}

cudaError_t launch_read_paged(const PagedView& c, bool fp4, const int32_t* start, int64_t T, uint16_t* out,
                              int num_sms, int32_t* err, cudaStream_t stream) {
    const int64_t items = (T + kReadTokens - 1) / kReadTokens * c.batch;
    const int64_t want = (items + 7) / 8, most = (int64_t)num_sms * 8;
    const dim3 grid(static_cast<unsigned>(want < most ? want : most));
    auto kernel = fp4 ? read_paged_kernel<true> : read_paged_kernel<false>;
    cudaError_t e = launch_pdl(kernel, grid, dim3(256), 0, stream, c, start, T, out, err);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace csld
