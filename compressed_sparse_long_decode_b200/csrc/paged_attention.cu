// Attention over the paged entry cache: a sliding window with first tokens that stay visible, or every
// token (layouts: csld_paged_cache in csld.h), on the 5th-generation tensor cores.
//
// Source: "DeepSeek-V4: a million-token context that agents can actually use" -- CSA and HCA paragraphs
// (a sliding-window branch over the most recent uncompressed tokens), storage paragraph (entries in low
// precision except the RoPE dims in bf16; FP4 where it suffices), layer-pattern paragraph (the
// window-only multi-token-prediction block).
//
// out_h = sum_t p_t k_t / l,  p_t = 2^(scale log2(e) q_h.k_t - m),  l = sum_t p_t over the visible tokens t,
// keys = values = the 512-d entry, 16 heads of one query at a time.
//
// Work.  A row is one (sequence, query, group of 16 heads).  Its token list is made of 16-token chunks, each
// inside one page: the chunks of the first tokens, then those of the window (or all), six chunks to a tile.
// The tiles of all rows, row after row, are dealt out evenly to one CTA per SM, so sequences of any mix of
// lengths load the SMs alike; a CTA walks its share as segments of rows.  A row that lies whole in one share is
// written out directly; of a row cut by shares each CTA leaves its unnormalised O and (m, l), and
// paged_merge_kernel joins them.
//
// A CTA's 24 warps:
//   copy     (warp 22)     pages -> shared memory, bulk copies (fp4: a chunk is 5888 contiguous bytes, staged
//                          as it lies) or tensor-map boxes with the 128-byte swizzle (fp8, into the tile image)
//   convert  (warps 16-21) fp4: codes -> E4M3 bytes in the swizzled tile image.  A 16-byte group of 32 codes is
//                          turned by byte permutes through an 8-byte table of 2^(6-j) times the E2M1 grid, j =
//                          the entry's largest exponent minus the group's, so an entry's image is its values
//                          over one power of two f_e (exact for j <= 14: 0.5 * 2^-8 is E4M3's smallest step).
//                          Both formats: rows of masked or missing tokens are zeroed, whatever was in them.
//   MMA      (warp 23)     S[entry][head] = K Q^T and O^T[dim][head] += V^T P from the one image: E4M3 keys against
//                          the query as two E4M3 terms (exact for bf16), values against the weights as two E4M3
//                          terms with a block scale per 32 entries, RoPE dims in bf16
//   softmax  (warps 0-15)  two streams of 8 warps take the tiles in turn, each with its own running maximum, sum and
//                          O (all in tensor memory), so that one stream's softmax runs under the other's MMAs;
//                          they are joined when a segment ends.  A thread owns one entry and 8 heads.  f_e
//                          multiplies S and P per entry, outside the MMAs.  The maximum is raised lazily: only
//                          where a tile exceeds it by 2^8 is O rescaled.
// Every wait is bounded; a wait that gives up sets CSLD_DEVERR_TIMEOUT and all roles run out without waiting.
#include <stdint.h>

#include "kernels.cuh"
#include "paged.cuh"
#include "sm100.cuh"

namespace csld {

namespace {

constexpr int kThreads = 960;
constexpr int kConvWarp = 16, kConvWarps = 12, kCopyWarp = 28, kMmaWarp = 29;
constexpr int kTile = 96;                        // entries per tile
constexpr int kTileChunks = kTile / kChunk;      // 6
constexpr int kBlkBytes = kTile * 128;           // one 128-byte column block of a tile
constexpr int kRopeBlk = 4;
constexpr int kImgBytes = 5 * kBlkBytes;         // 60 KB
constexpr int kStageBytes = kTileChunks * kChunk4Bytes;
constexpr int kKBlocks = kTile / 32;
// Weights: p = 2^(x + nm); a head's nm is set so that the largest p of a tile is 2^kLift and kept until one exceeds
// 2^kOver.  The PV operand holds p w in E5M2, w = 1 (fp8) or f_e g (fp4; g a power of two set so that the tile's
// largest f_e g is kFeSet, kept until one exceeds kFeMost).  E5M2 bounds the product: 57344 > 2^kOver w.
template <bool kFp4> constexpr float kLift = kFp4 ? 0.f : 5.f;
template <bool kFp4> constexpr float kOver = kFp4 ? 10.f : 15.f;
constexpr float kFeSet = 8.f, kFeMost = 32.f, kUnset = 1e30f;
// tensor-memory columns of stream s: S at kColS + 48 s (16 hi, 16 lo, 16 RoPE), O at kColO + 208 s (four dim blocks
// of 48: the three terms of P; RoPE 16)
constexpr uint32_t kColS = 0, kStepS = 48, kColO = 96, kStepO = 208, kColOR = 192;
constexpr uint32_t kIdQK = idesc_e4m3_m128(32, false, false);
constexpr uint32_t kIdQKr = idesc_bf16_m128(16, false, false);
constexpr uint32_t kIdPV = idesc_e4m3_m128(48, true, true) | (1u << 10);   // B in E5M2
constexpr uint32_t kIdPVr = idesc_bf16_m128(16, true, true);
constexpr int kBarStream = 1, kBarAll = 3;       // named barriers: the streams' (1, 2), both streams' (3)
constexpr int kLutRows = 21;                     // NaN group; j = 0..18; all zero (j >= 19, masked entries)

template <bool kFp4>
struct Smem {
    static constexpr int kBufs = kFp4 ? 2 : 3;   // tile images
    uint8_t img[kBufs][kImgBytes];               // [block][entry][128 B], 128-byte swizzle
    uint8_t qk[4][32 * 128];                     // QK B operand per dim block: rows 0..15 Qhi, 16..31 Qlo (the MMAs also
                                                 // read past the last image into here: rows whose results go unused)
    uint8_t qr[16 * 128];                        // RoPE query
    uint8_t p8[2][kTile * 64];                   // per stream: PV B operand [entry][16 heads x 3 terms], 64-byte swizzle
    uint8_t pbf[2][kTile * 32];                  // per stream: bf16 P [entry][16 heads], 32-byte swizzle
    uint8_t stage[kFp4 ? 2 : 1][kFp4 ? kStageBytes : 16];
    uint2 lut[kLutRows];
    alignas(16) float fe[kBufs][kTile];          // entry factors; -1: masked (before the walk: the scan's sums)
    alignas(16) float c2[kHeads];
    alignas(16) float tmax[2][4][kHeads];        // per stream: tile maxima (then partial sums) per lane quarter
    float femax[2][4], ginv[2];                  // per stream: largest f_e per lane quarter; 1 / g
    float2 ml[2][kHeads];
    int32_t chunk_tok[kBufs][kTileChunks];       // first token of a tile's chunks; -1: none
    uint64_t stfull[kBufs], stempty[2], imgfull[kBufs], imgempty[kBufs], sfull[2], pfull[2], pdone[2], qready, drain;
    int64_t prefix;
    uint32_t tmem_base;
    int32_t fail, b0, n_issued;
};
static_assert(sizeof(Smem<true>) <= 232448 && sizeof(Smem<false>) <= 232448, "227 KB of shared memory");

struct Params {
    PagedView c;
    const uint16_t* q;
    void* out;
    float* lse;
    float* opart;        // [2 CTAs][16][512]
    float2* mlpart;      // [2 CTAs][16]
    int4* meta;          // [CTAs]: (row low, row high, last CTA, -) of the cut row that begins there; last CTA -1: none
    int32_t* err;
    float scale;
    int heads, groups, Q, W, sinks, min_tiles;
    bool out_bf16;
};

__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return ok != 0;
}
// Bounded wait: false once any wait of the CTA has given up (this one after about a second).
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int32_t* fail) {
    for (uint32_t i = 0; i < (1u << 22); ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if (i >= 16) {
            if (*fail) return false;
            __nanosleep(64);
        }
    }
    *fail = 1;
    return false;
}
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
__device__ __forceinline__ float key_to_float(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        :: "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar)) : "memory");
}

// ---- the token list of a sequence -----------------------------------------------------------
// n tokens; chunks [0, cs) hold the first tokens, then come the chunks from wl on, nc in all; tiles per row.
struct SeqInfo {
    int n, cs, wl, nc, tiles;
};
__device__ __forceinline__ SeqInfo seq_info(const Params& P, int b) {
    SeqInfo s;
    const int64_t cap = P.c.capacity();
    s.n = static_cast<int>(max64(0, min64(P.c.seq_len[b], cap)));
    const int last = s.n / kChunk + (s.n % kChunk != 0);
    s.cs = s.wl = 0;
    s.nc = last;
    if (P.W > 0) {
        const int64_t lo = max64(0, (int64_t)s.n - P.Q + 1 - P.W);   // the oldest query's window
        const int cs = static_cast<int>((min64(P.sinks, lo) + kChunk - 1) / kChunk), wl = static_cast<int>(lo / kChunk);
        if (wl > cs) {
            s.cs = cs;
            s.wl = wl;
            s.nc = cs + last - wl;
        }
    }
    s.tiles = max(1, (s.nc + kTileChunks - 1) / kTileChunks);
    return s;
}

// A CTA's walk over its share, segment by segment; every role walks it by itself.
struct Walk {
    int b, rq, t;        // sequence, row within it, first tile of the segment
    int left, len;       // tiles left in the share (this segment included), tiles of this segment
    SeqInfo s;
    __device__ __forceinline__ void begin(const Params& P, int b_, int64_t off, int n_tiles) {
        b = b_;
        s = seq_info(P, b);
        rq = static_cast<int>(off / s.tiles);
        t = static_cast<int>(off % s.tiles);
        left = n_tiles;
        len = min(s.tiles - t, left);
    }
    __device__ __forceinline__ void next(const Params& P) {
        left -= len;
        t = 0;
        if (left <= 0) return;
        if (++rq == P.Q * P.groups) {
            rq = 0;
            s = seq_info(P, ++b);
        }
        len = min(s.tiles, left);
    }
    __device__ __forceinline__ int token_of_chunk(int i) const {   // i: chunk of the row's list
        return i < s.nc ? kChunk * (i < s.cs ? i : s.wl + i - s.cs) : -1;
    }
};
__device__ __forceinline__ bool sees(const Params& P, int t, int p) {
    return t <= p && (P.W == 0 || t < P.sinks || t > p - P.W);
}

// ---- convert: eight E2M1 codes (one word) -> eight E4M3 bytes ---------------------------------
__device__ __forceinline__ void decode8(uint32_t w, uint2 tab, uint32_t& lo, uint32_t& hi) {
    const uint32_t sel = w & 0x77777777u;
    lo = __byte_perm(tab.x, tab.y, sel) | (w & 0x80808080u);
    hi = __byte_perm(tab.x, tab.y, sel >> 16) | ((w << 4) & 0x80808080u);
}

// ---- softmax ----------------------------------------------------------------------------------
// t = x - m for this thread's 8 heads (log2 units; nm = -m), -inf where the entry is masked.
template <bool kFp4>
__device__ __forceinline__ void load_t(float (&t)[8], uint32_t ts, const float* c2, const float (&nm)[8], float fe, bool seen) {
    uint32_t hi[8], lo[8], r[8];
    tmem_ld_32x32b_x8(ts, hi);
    tmem_ld_32x32b_x8(ts + 16u, lo);
    if constexpr (kFp4) tmem_ld_32x32b_x8(ts + 32u, r);
    tmem_ld_wait();
    const float4 ca = *reinterpret_cast<const float4*>(c2), cb = *reinterpret_cast<const float4*>(c2 + 4);
    const float c[8] = {ca.x, ca.y, ca.z, ca.w, cb.x, cb.y, cb.z, cb.w};
#pragma unroll
    for (int h = 0; h < 8; ++h) {
        float v = __uint_as_float(hi[h]) + __uint_as_float(lo[h]);
        if constexpr (kFp4) v = fmaf(v, fe, __uint_as_float(r[h]));
        t[h] = seen ? fmaf(v, c[h], nm[h]) : -INFINITY;
    }
}
__device__ __forceinline__ uint32_t f32x2_to_f16x2(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
// Two f16 -> two E5M2 bytes (round to nearest even).  E5M2 is f16's upper byte, so the way back is a byte permute.
__device__ __forceinline__ uint32_t f16x2_to_e5m2x2(uint32_t v) {
    uint16_t r;
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ uint32_t f16x2_sub(uint32_t a, uint32_t b) {
    const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&v);
}
// t <- p = 2^t, and p into the PV operands of this entry: p w (w = f_e g; fp8: p itself) as f16 and from there as
// three E5M2 terms, each the rounding of what the ones before left (2^-3 of it: 2^-9 in all, and nothing finer
// than E5M2's 2^-16, 2^-23 of the largest weight), 8 heads a store; p in bf16 for the RoPE dims.
template <bool kFp4>
__device__ __forceinline__ void write_p(uint8_t* p8, uint8_t* pb, float (&t)[8], float w, int hg, int e) {
    uint32_t term[3][2], bf[4];
#pragma unroll
    for (int h = 0; h < 8; h += 4) {
        uint32_t v[2], q[3][2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int k = h + 2 * u;
            t[k] = exp2_ftz(t[k]);
            t[k + 1] = exp2_ftz(t[k + 1]);
            bf[k >> 1] = f32x2_to_bf16x2_bits(t[k], t[k + 1]);
            v[u] = kFp4 ? f32x2_to_f16x2(t[k] * w, t[k + 1] * w) : f32x2_to_f16x2(t[k], t[k + 1]);
#pragma unroll
            for (int n = 0; n < 3; ++n) {
                q[n][u] = f16x2_to_e5m2x2(v[u]);
                if (n < 2) v[u] = f16x2_sub(v[u], __byte_perm(q[n][u], 0u, 0x1404));   // exact
            }
        }
#pragma unroll
        for (int n = 0; n < 3; ++n) term[n][h >> 2] = __byte_perm(q[n][0], q[n][1], 0x5410);
    }
    const int sw = (e >> 1) & 3;
#pragma unroll
    for (int n = 0; n < 3; ++n)
        *reinterpret_cast<uint2*>(p8 + 64 * e + 16 * (n ^ sw) + 8 * hg) = make_uint2(term[n][0], term[n][1]);
    *reinterpret_cast<uint4*>(pb + 32 * e + 16 * (hg ^ ((e >> 2) & 1))) = make_uint4(bf[0], bf[1], bf[2], bf[3]);
}
// MN-major operand of rows of 64 or 32 bytes under the swizzle of that width: 8-row groups one after the other.
__device__ __forceinline__ uint64_t desc_rows(const void* p, uint32_t row_bytes) {
    uint64_t d = static_cast<uint64_t>((smem_u32(p) >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>((8 * row_bytes) >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(row_bytes == 64 ? 4u : 6u) << 61;
    return d;
}

// The query of one head as MMA operands, one warp per head, 16 dims per lane: scaled by a power of two so that
// its largest value lies in 2^7..2^8, then (dims 0..447) two E4M3 terms -- bf16's 8 significant bits split
// exactly, down to 2^-10 of the largest -- or (RoPE) bf16.
template <bool kFp4>
__device__ __forceinline__ void prepare_query(Smem<kFp4>& sm, const uint4 (&v)[2], int h, int lane, float scale) {
    const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
    top = __reduce_max_sync(0xffffffffu, top);
    const int sh = top ? max(-100, min(100, 7 - (static_cast<int>(top >> 7) - 127))) : 0;
    const float sq = pow2f(sh);
    if (lane == 0) sm.c2[h] = scale * 1.4426950408889634f / sq;
    if (lane < kNope / 16) {
        uint32_t hw[4], lw[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t hi2[2], lo2[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint32_t x = w[2 * i + u];
                const float x0 = bf16_bits_to_f32(x) * sq, x1 = bf16_bits_to_f32(x >> 16) * sq;
                hi2[u] = __nv_cvt_float2_to_fp8x2(make_float2(x0, x1), __NV_SATFINITE, __NV_E4M3);
                const uint32_t back = e4m3x2_to_f16x2(hi2[u]);
                lo2[u] = __nv_cvt_float2_to_fp8x2(
                    make_float2(x0 - __half2float(__ushort_as_half(static_cast<unsigned short>(back & 0xFFFFu))),
                                x1 - __half2float(__ushort_as_half(static_cast<unsigned short>(back >> 16)))),
                    __NV_SATFINITE, __NV_E4M3);
            }
            hw[i] = (hi2[0] & 0xFFFFu) | (hi2[1] << 16);
            lw[i] = (lo2[0] & 0xFFFFu) | (lo2[1] << 16);
        }
        uint8_t* blk = sm.qk[lane >> 3];
        const int c = 16 * (lane & 7);
        *reinterpret_cast<uint4*>(blk + sw128(h, c)) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
        *reinterpret_cast<uint4*>(blk + sw128(16 + h, c)) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
    } else {
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = f32x2_to_bf16x2_bits(bf16_bits_to_f32(w[i]) * sq, bf16_bits_to_f32(w[i] >> 16) * sq);
        const int c = 32 * (lane - kNope / 16);
        *reinterpret_cast<uint4*>(sm.qr + sw128(h, c)) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(sm.qr + sw128(h, c + 16)) = make_uint4(o[4], o[5], o[6], o[7]);
    }
    fence_proxy_async_smem();
}

__device__ __forceinline__ void store_out(const Params& P, int64_t at, float v) {
    if (P.out_bf16) reinterpret_cast<uint16_t*>(P.out)[at] = static_cast<uint16_t>(f32_to_bf16_bits(v));
    else reinterpret_cast<float*>(P.out)[at] = v;
}

// The MMAs of one tile.  Stream and image are compile-time constants and tensor memory starts at column 0 (all of it
// is allocated), so descriptors are constants over one base: forming them at run time cost the issuing thread about
// 95 cycles an MMA, twice what the tensor pipe takes for these narrow ones (45).
template <bool kFp4, int kSt, int kBuf>
__device__ __forceinline__ void issue_qk(Smem<kFp4>& sm) {
    const uint64_t da = desc_sw128(sm.img[kBuf], 0), dq = desc_sw128(sm.qk[0], 0), dqr = desc_sw128(sm.qr, 0);
    constexpr uint32_t d = kColS + kStepS * kSt;
#pragma unroll
    for (int kb = 0; kb < 4; ++kb)
#pragma unroll
        for (int ks = 0; ks < (kb < 3 ? 4 : 2); ++ks)
            umma_f8f6f4(d, da + (kb * kBlkBytes + 32 * ks) / 16, dq + (kb * 4096 + 32 * ks) / 16, kIdQK, (kb | ks) != 0 ? 1u : 0u);
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)   // fp4: apart, since f_e multiplies only the 4-bit dims
        umma_f16(d + (kFp4 ? 32u : 0u), da + (kRopeBlk * kBlkBytes + 32 * ks) / 16, dqr + (32 * ks) / 16, kIdQKr,
                 kFp4 && ks == 0 ? 0u : 1u);
    umma_commit(&sm.sfull[kSt]);
}
template <bool kFp4, int kSt, int kBuf>
__device__ __forceinline__ void issue_pv(Smem<kFp4>& sm, uint32_t acc0) {   // acc0 = 0: O is overwritten
    const uint64_t da = desc_sw128(sm.img[kBuf], 0), dp = desc_rows(sm.p8[kSt], 64);
    constexpr uint32_t o = kColO + kStepO * kSt;
#pragma unroll
    for (int mb = 0; mb < 4; ++mb)
#pragma unroll
        for (int kb = 0; kb < kKBlocks; ++kb)
            umma_f8f6f4(o + 48u * mb, da + (mb * kBlkBytes + kb * 4096) / 16, dp + (32 * 64 * kb) / 16, kIdPV, kb > 0 ? 1u : acc0);
    const uint64_t dar = desc_sw128(sm.img[kBuf] + kRopeBlk * kBlkBytes, kBlkBytes), dpb = desc_rows(sm.pbf[kSt], 32);
#pragma unroll
    for (int ks = 0; ks < kTile / 16; ++ks)
        umma_f16(o + kColOR, dar + (ks * 2048) / 16, dpb + (16 * 32 * ks) / 16, kIdPVr, ks > 0 ? 1u : acc0);
    umma_commit(&sm.imgempty[kBuf]);
    umma_commit(&sm.pdone[kSt]);
}
// Tile T's stream is T % 2, its image T % 2 (fp4) or T % 3 (fp8): f(stream, image) as compile-time constants.
template <bool kFp4, typename F>
__device__ __forceinline__ void with_tile(int T, F&& f) {
    if constexpr (kFp4) {
        if (T & 1) f.template operator()<1, 1>();
        else f.template operator()<0, 0>();
    } else {
        switch (T % 6) {
            case 0: f.template operator()<0, 0>(); break;
            case 1: f.template operator()<1, 1>(); break;
            case 2: f.template operator()<0, 2>(); break;
            case 3: f.template operator()<1, 0>(); break;
            case 4: f.template operator()<0, 1>(); break;
            default: f.template operator()<1, 2>(); break;
        }
    }
}
template <bool kFp4>
struct IssueQk {
    Smem<kFp4>& sm;
    template <int kSt, int kBuf> __device__ __forceinline__ void operator()() { issue_qk<kFp4, kSt, kBuf>(sm); }
};
template <bool kFp4>
struct IssuePv {
    Smem<kFp4>& sm;
    uint32_t acc0;
    template <int kSt, int kBuf> __device__ __forceinline__ void operator()() { issue_pv<kFp4, kSt, kBuf>(sm, acc0); }
};

}  // namespace

template <bool kFp4>
__global__ void __launch_bounds__(kThreads, 1) paged_attention_kernel(const __grid_constant__ CUtensorMap pages_map,
                                                                      const __grid_constant__ Params P) {
    using S = Smem<kFp4>;
    constexpr int kBufs = S::kBufs;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    S& sm = *reinterpret_cast<S*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    // ---- setup --------------------------------------------------------------------------------
    if (tid == 0) {
        for (int s = 0; s < kBufs; ++s) {
            mbar_init(&sm.stfull[s], 1);
            mbar_init(&sm.imgfull[s], kConvWarps);
            mbar_init(&sm.imgempty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sm.stempty[s], kConvWarps);
            mbar_init(&sm.sfull[s], 1);
            mbar_init(&sm.pfull[s], 8);
            mbar_init(&sm.pdone[s], 1);
        }
        mbar_init(&sm.qready, 16);
        mbar_init(&sm.drain, 1);
        sm.fail = 0;
        sm.n_issued = 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&sm.tmem_base, 512);
        tmem_relinquish();
    }
    if (kFp4 && tid >= 512 && tid < 512 + kLutRows) {   // table rows: 2^(6-j) times the E2M1 grid in E4M3
        const int j = tid - 513;
        const float s = j < 0 ? __uint_as_float(0x7FC00000u) : j == kLutRows - 2 ? 0.f : pow2f(6 - j);
        const float twice[8] = {0.f, 1.f, 2.f, 3.f, 4.f, 6.f, 8.f, 12.f};
        uint32_t w[2] = {0u, 0u};
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k >> 2] |= f32_to_e4m3(0.5f * twice[k] * s) << (8 * (k & 3));
        sm.lut[tid - 512] = make_uint2(w[0], w[1]);
    }
    if (!kFp4 && warp == kCopyWarp && lane == 0) tma_prefetch_map(&pages_map);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait();
    pdl_trigger();

    // ---- this CTA's share of all rows' tiles ------------------------------------------------------
    const int rows_per_seq = P.Q * P.groups;
    int64_t mine = 0;
    for (int b = tid; b < P.c.batch; b += kThreads) {
        const int32_t n = P.c.seq_len[b];
        if ((n < 0 || n > P.c.capacity()) && blockIdx.x == 0) dev_error(P.err, CSLD_DEVERR_SEQ_LEN);
        mine += seq_info(P, b).tiles;
    }
    // tiles of all sequences, then (per batch of 768 sequences) the sequence that the share begins in
    int64_t* red = reinterpret_cast<int64_t*>(sm.fe[0]);
    auto block_scan = [&](int64_t v, int64_t& total) {   // exclusive prefix of v over the threads
        int64_t inc = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        __syncthreads();
        if (lane == 31) red[warp] = inc;
        __syncthreads();
        int64_t before = 0;
        total = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += red[w];
            total += red[w];
        }
        return before + inc - v;
    };
    int64_t all;
    const int64_t pre = block_scan(mine, all);
    const int64_t total = all * rows_per_seq;
    const int64_t n_cta = max64(1, min64((int64_t)gridDim.x, total / P.min_tiles));
    const int64_t u0 = blockIdx.x < n_cta ? total * blockIdx.x / n_cta : 0;
    const int64_t u1 = blockIdx.x < n_cta ? total * (blockIdx.x + 1) / n_cta : 0;
    const int n_tiles = static_cast<int>(u1 - u0);
    if (n_tiles > 0) {
        int64_t base = 0;
        for (int b1 = 0; b1 < P.c.batch; b1 += kThreads) {
            int64_t v, p, tot;
            if (P.c.batch <= kThreads) {
                v = mine;
                p = pre;
                tot = all;
            } else {
                v = b1 + tid < P.c.batch ? seq_info(P, b1 + tid).tiles : 0;
                p = block_scan(v, tot) + base;
            }
            if (v > 0 && p * rows_per_seq <= u0 && u0 < (p + v) * rows_per_seq) {
                sm.b0 = b1 + tid;
                sm.prefix = p * rows_per_seq;
            }
            base += tot;
        }
    }
    __syncthreads();
    const uint32_t tmem = sm.tmem_base;
    volatile int32_t* fail = &sm.fail;
    if (tid == 0) P.meta[blockIdx.x] = make_int4(0, 0, -1, 0);   // its thread overwrites it below where a cut row begins

    if (n_tiles > 0) {
        Walk wk;
        wk.begin(P, sm.b0, u0 - sm.prefix, n_tiles);
        if (warp < 16) {
            // ===== softmax: stream = warp / 8, thread = entry e (TMEM lane), heads 8 hg .. 8 hg + 7 ===============
            const int st = warp >> 3, hg = (warp >> 2) & 1, sub = warp & 3, e = 32 * sub + lane;
            const uint32_t lb = tmem + ((32u * sub) << 16);
            const uint32_t ts = lb + kColS + kStepS * st + 8u * hg, to = lb + kColO + kStepO * st + 8u * hg;
            auto load_query = [&](uint4 (&v)[2]) {
                const int j = wk.rq / P.groups, h = 16 * (wk.rq % P.groups) + warp;
                v[0] = v[1] = make_uint4(0, 0, 0, 0);
                if (h < P.heads) {
                    const uint4* src = reinterpret_cast<const uint4*>(
                        P.q + (((int64_t)wk.b * P.Q + j) * P.heads + h) * kDim + 16 * lane);
                    v[0] = __ldg(src);
                    v[1] = __ldg(src + 1);
                }
            };
            int T = 0;   // running tile of the CTA; stream st takes those with T % 2 == st
            for (; wk.left > 0; wk.next(P)) {
                {
                    uint4 v[2];
                    load_query(v);
                    prepare_query<kFp4>(sm, v, warp, lane, P.scale);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.qready);
                named_barrier(kBarAll, 512);   // c2 of every head
                float nm[8], l[8], g = 0.f;   // nm = kUnset, g = 0: not set yet
#pragma unroll
                for (int h = 0; h < 8; ++h) {
                    nm[h] = kUnset;
                    l[h] = 0.f;
                }
                const int T1 = T + wk.len;
                for (T += (T ^ st) & 1; T < T1; T += 2) {
                    const int buf = kFp4 ? st : T % 3;
                    bool ok = wait(&sm.imgfull[buf], (T / kBufs) & 1, fail);   // (for f_e) done before S is
                    ok = ok && wait(&sm.sfull[st], (T >> 1) & 1, fail);
                    ok = __all_sync(0xffffffffu, ok);
                    tc_fence_after();
                    float t[8], fe = -1.f;
                    bool over = false;
                    const float* c2 = sm.c2 + 8 * hg;
                    // First try against the maximum as it stands (the common case): one meeting of the stream's
                    // warps.  S(T) complete implies PV(T-2) complete, so P and O are free to be written.
                    if (sub < kTile / 32) {
                        fe = ok ? sm.fe[buf][e] : -1.f;
                        load_t<kFp4>(t, ts, c2, nm, fe, fe >= 0.f);
                        float top = t[0];
#pragma unroll
                        for (int h = 1; h < 8; ++h) top = fmaxf(top, t[h]);
                        over = top > kOver<kFp4> || (kFp4 && fe * g > kFeMost);
                        if (!__any_sync(0xffffffffu, over)) write_p<kFp4>(sm.p8[st], sm.pbf[st], t, fe >= 0.f ? fe * g : 0.f, hg, e);
                    }
                    fence_proxy_async_smem();
                    if (named_barrier_or(kBarStream + st, 256, over)) {
                        // some weight is too large, or the first tile: the tile's maxima (of the logits themselves, nm
                        // may be unset), every head that lies more than 2 above its mark set anew, O rescaled
                        const bool seen = fe >= 0.f;
                        if (sub < kTile / 32) {
                            float z[8];
#pragma unroll
                            for (int h = 0; h < 8; ++h) z[h] = 0.f;
                            load_t<kFp4>(t, ts, c2, z, fe, seen);
                            float mine = 0.f;
#pragma unroll
                            for (int h = 0; h < 8; ++h) {
                                const float top = key_to_float(__reduce_max_sync(0xffffffffu, score_key(t[h])));
                                mine = lane == h ? top : mine;
                            }
                            if (lane < 8) sm.tmax[st][sub][8 * hg + lane] = mine;
                            if (kFp4 && hg == 0) {
                                const uint32_t fm = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(fe, 0.f)));
                                if (lane == 0) sm.femax[st][sub] = __uint_as_float(fm);
                            }
                        }
                        named_barrier(kBarStream + st, 256);
                        float f[8], fg = 1.f;
                        bool rescale = false;
                        if constexpr (kFp4) {
                            const float fm = fmaxf(fmaxf(sm.femax[st][0], sm.femax[st][1]), sm.femax[st][2]);
                            if (fm > 0.f && (g == 0.f || fm * g > kFeMost)) {
                                const float gn = kFeSet / fmaxf(fm, 0x1p-110f);
                                if (g != 0.f) {
                                    fg = gn / g;
                                    rescale = true;
                                }
                                g = gn;
                            }
                        }
#pragma unroll
                        for (int h = 0; h < 8; ++h) {
                            float tm = sm.tmax[st][0][8 * hg + h];
#pragma unroll
                            for (int q3 = 1; q3 < kTile / 32; ++q3) tm = fmaxf(tm, sm.tmax[st][q3][8 * hg + h]);
                            const bool first = nm[h] == kUnset;
                            const bool set = first ? tm > -INFINITY : tm + nm[h] > kLift<kFp4> + 2.f;
                            const float to_nm = set ? kLift<kFp4> - tm : nm[h];
                            f[h] = set && !first ? exp2_ftz(to_nm - nm[h]) : 1.f;
                            rescale |= set && !first;
                            l[h] *= f[h];
                            nm[h] = to_nm;
                        }
                        if (rescale) {   // the same answer in every thread of the head group
#pragma unroll 2
                            for (int c = 0; c < 13; ++c) {   // 4 blocks of 3 terms, then RoPE
                                uint32_t o[8];
                                const float fc = c < 12 ? fg : 1.f;
                                tmem_ld_32x32b_x8(to + 16u * c, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int h = 0; h < 8; ++h) o[h] = __float_as_uint(__uint_as_float(o[h]) * (f[h] * fc));
                                tmem_st_32x32b_x8(to + 16u * c, o);
                            }
                            tmem_st_wait();
                        }
                        if (sub < kTile / 32) {
#pragma unroll
                            for (int h = 0; h < 8; ++h) t[h] += nm[h];
                            write_p<kFp4>(sm.p8[st], sm.pbf[st], t, seen ? fe * g : 0.f, hg, e);
                        }
                        fence_proxy_async_smem();
                        named_barrier(kBarStream + st, 256);
                    }
                    if (sub < kTile / 32) {
#pragma unroll
                        for (int h = 0; h < 8; ++h) l[h] += t[h];
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.pfull[st]);
                }
                const int T_last = T - 2;   // the stream's last tile so far (any segment)
                T = T1;
                const bool had = T_last >= T1 - wk.len;   // the stream had a tile of this segment
                if (had) (void)wait(&sm.pdone[st], (T_last >> 1) & 1, fail);
                // ---- the segment's result: sums over the lane quarters, then both streams joined -------------
#pragma unroll
                for (int h = 0; h < 8; ++h) {
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], o);
                    if (lane == h) sm.tmax[st][sub][8 * hg + h] = l[h];
                }
                named_barrier(kBarStream + st, 256);
                if (sub == 0 && lane < 8) {
                    const int hh = 8 * hg + lane;
                    float mm = nm[0];
#pragma unroll
                    for (int h = 1; h < 8; ++h) mm = lane == h ? nm[h] : mm;
                    if (hh == 0) sm.ginv[st] = g != 0.f ? 1.f / g : 1.f;
                    sm.ml[st][hh] = make_float2(-mm, (sm.tmax[st][0][hh] + sm.tmax[st][1][hh]) + (sm.tmax[st][2][hh] + sm.tmax[st][3][hh]));
                }
                tc_fence_before();
                named_barrier(kBarAll, 512);
                tc_fence_after();
                // l == 0: the stream saw nothing (its O may be stale); a NaN sum is no zero
                float a0[8], a1[8], M[8], L[8];
                bool use0 = false, use1 = false;
#pragma unroll
                for (int h = 0; h < 8; ++h) {
                    const float2 s0 = sm.ml[0][8 * hg + h], s1 = sm.ml[1][8 * hg + h];
                    const bool z0 = s0.y == 0.f, z1 = s1.y == 0.f;
                    M[h] = z0 ? (z1 ? -INFINITY : s1.x) : (z1 ? s0.x : fmaxf(s0.x, s1.x));
                    a0[h] = z0 ? 0.f : exp2_ftz(s0.x - M[h]);
                    a1[h] = z1 ? 0.f : exp2_ftz(s1.x - M[h]);
                    L[h] = a0[h] * s0.y + a1[h] * s1.y;
                    use0 |= !z0;
                    use1 |= !z1;
                }
                const bool whole = wk.t == 0 && wk.len == wk.s.tiles;
                const int j = wk.rq / P.groups, h0 = 16 * (wk.rq % P.groups) + 8 * hg;
                const int64_t at = ((int64_t)wk.b * P.Q + j) * P.heads + h0;
                const int64_t slot = 2 * (int64_t)blockIdx.x + (wk.t == 0 ? 1 : 0);
                if (!*fail) {
                    // stream 0's warps write dims 0..255, stream 1's the rest
                    float inv[8];
#pragma unroll
                    for (int h = 0; h < 8; ++h) inv[h] = whole ? (L[h] == 0.f ? 0.f : 1.f / L[h]) : 1.f;
                    const uint32_t o0 = lb + kColO + 8u * hg;
                    const float gi[2] = {sm.ginv[0], sm.ginv[1]};
#pragma unroll 1
                    for (int c = 2 * st; c < 2 + 3 * st; ++c) {
                        const bool rope = c == 4;
                        float v[8];
#pragma unroll
                        for (int h = 0; h < 8; ++h) v[h] = 0.f;
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            if (!(k ? use1 : use0)) continue;   // uniform in the warp
#pragma unroll 1
                            for (int n = 0; n < (rope ? 1 : 3); ++n) {
                                uint32_t o[8];
                                tmem_ld_32x32b_x8(o0 + kStepO * k + 48u * c + 16u * n, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int h = 0; h < 8; ++h) {
                                    const float a = (k ? a1[h] : a0[h]) * (rope ? 1.f : gi[k]);
                                    if (a != 0.f) v[h] = fmaf(a, __uint_as_float(o[h]), v[h]);
                                }
                            }
                        }
                        const int d = rope ? kNope + e : 128 * c + e;
                        if (rope ? e < kRope : d < kNope) {
#pragma unroll
                            for (int h = 0; h < 8; ++h) {
                                if (whole) {
                                    if (h0 + h < P.heads) store_out(P, (at + h) * kDim + d, v[h] * inv[h]);
                                } else {
                                    P.opart[(slot * kHeads + 8 * hg + h) * kDim + d] = v[h];
                                }
                            }
                        }
                    }
                    if (st == 0 && sub == 0 && lane < 8) {
                        float mm = M[0], ll = L[0];
#pragma unroll
                        for (int h = 1; h < 8; ++h) {
                            mm = lane == h ? M[h] : mm;
                            ll = lane == h ? L[h] : ll;
                        }
                        if (!whole) P.mlpart[slot * kHeads + 8 * hg + lane] = make_float2(mm, ll);
                        else if (P.lse && h0 + lane < P.heads)
                            P.lse[at + lane] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * 0.69314718055994531f;
                    }
                    if (tid == 0 && wk.t == 0 && wk.len < wk.s.tiles) {   // a cut row begins here: its last CTA
                        const int64_t row = (int64_t)wk.b * rows_per_seq + wk.rq;
                        const int64_t end = u1 - wk.left + wk.s.tiles;    // unit behind the row
                        int64_t c = (end - 1) * n_cta / total;
                        while (total * (c + 1) / n_cta <= end - 1) ++c;
                        while (total * c / n_cta > end - 1) --c;
                        P.meta[blockIdx.x] = make_int4(static_cast<int>(row), static_cast<int>(row >> 32), static_cast<int>(c), 0);
                    }
                }
                tc_fence_before();
                named_barrier(kBarAll, 512);   // O, c2 and the query operands are free for the next row
                tc_fence_after();
            }
        } else if (warp < kConvWarp + kConvWarps) {
            // ===== convert ==================================================================================
            const int ct = tid - 32 * kConvWarp, e = ct % kTile, part = ct / kTile;   // part: groups part, part + 4, ..
            int T = 0;
            for (; wk.left > 0; wk.next(P)) {
                const int p = wk.s.n - P.Q + wk.rq / P.groups;   // the query's position
                for (int t = 0; t < wk.len; ++t, ++T) {
                    const int buf = T % kBufs;
                    bool ok = wait(&sm.stfull[buf], (T / kBufs) & 1, fail);
                    if (kFp4 && T >= kBufs) ok = ok && wait(&sm.imgempty[buf], (T / kBufs - 1) & 1, fail);
                    ok = __all_sync(0xffffffffu, ok);
                    uint8_t* img = sm.img[buf];
                    const int ck = e / kChunk, tk = e % kChunk;
                    auto seen = [&](int en) {
                        const int c0 = sm.chunk_tok[buf][en / kChunk];
                        return c0 >= 0 && sees(P, c0 + en % kChunk, p);
                    };
                    const bool vis = ok && seen(e);
                    if constexpr (kFp4) {
                        const uint8_t* ch = sm.stage[buf] + ck * kChunk4Bytes;
                        const int ex0 = ch[kChunk4Exp + kGroups * kChunk + tk];
                        if (part == 0) sm.fe[buf][e] = vis ? ldexpf(1.f, ex0 - 133) : -1.f;
                        const int base = vis ? ex0 : 4096;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int g = part + 4 * i;
                            if (g >= kGroups) break;   // whole warps
                            const uint4 w = *reinterpret_cast<const uint4*>(ch + g * 256 + tk * 16);
                            const int ex = ch[kChunk4Exp + g * kChunk + tk];   // 255 (NaN) is above every base
                            const uint2 tab = sm.lut[1 + max(-1, min(base - ex, kLutRows - 2))];
                            uint4 a, b;
                            decode8(w.x, tab, a.x, a.y);
                            decode8(w.y, tab, a.z, a.w);
                            decode8(w.z, tab, b.x, b.y);
                            decode8(w.w, tab, b.z, b.w);
                            uint8_t* dst = img + i * kBlkBytes;
                            *reinterpret_cast<uint4*>(dst + sw128(e, 32 * part)) = a;
                            *reinterpret_cast<uint4*>(dst + sw128(e, 32 * part + 16)) = b;
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) {   // RoPE rows, eight threads per entry (no bank conflicts)
                            const int en = (ct >> 3) + 48 * i, c = ct & 7;
                            uint4 w = *reinterpret_cast<const uint4*>(sm.stage[buf] + (en / kChunk) * kChunk4Bytes + kChunk4Rope +
                                                                      (en % kChunk) * 2 * kRope + 16 * c);
                            if (!(ok && seen(en))) w = make_uint4(0, 0, 0, 0);
                            *reinterpret_cast<uint4*>(img + kRopeBlk * kBlkBytes + sw128(en, 16 * c)) = w;
                        }
                    } else {
                        if (part == 0) sm.fe[buf][e] = vis ? 1.f : -1.f;
                        if (!vis && ok) {
                            for (int c = part; c < 40; c += 4)
                                *reinterpret_cast<uint4*>(img + (c >> 3) * kBlkBytes + sw128(e, 16 * (c & 7))) = make_uint4(0, 0, 0, 0);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&sm.imgfull[buf]);
                        if (kFp4) mbar_arrive(&sm.stempty[buf]);
                    }
                }
            }
        } else if (warp == kCopyWarp) {
            // ===== copy ====================================================================================
            int T = 0;
            // lane i < 6: chunk i of the tile; its first token and page, loaded one tile ahead
            auto look = [&](const Walk& w, int t, int& tok, int32_t& pg) {
                tok = lane < kTileChunks && t < w.s.tiles ? w.token_of_chunk((w.t + t) * kTileChunks + lane) : -1;
                pg = tok >= 0 ? __ldg(P.c.table + (int64_t)w.b * P.c.max_pages + tok / P.c.page_size) : -1;
            };
            for (; wk.left > 0; wk.next(P)) {
                int tok, tok1 = -1;
                int32_t pg, pg1 = -1;
                look(wk, 0, tok, pg);
                for (int t = 0; t < wk.len; ++t, ++T) {
                    if (t + 1 < wk.len) look(wk, t + 1, tok1, pg1);
                    const int buf = T % kBufs;
                    bool ok = !*fail;
                    if (T >= kBufs)
                        ok = ok && wait(kFp4 ? &sm.stempty[buf & 1] : &sm.imgempty[buf], (T / kBufs - 1) & 1, fail);
                    if (!__all_sync(0xffffffffu, ok)) break;
                    if (tok >= 0 && (pg < 0 || pg >= P.c.n_pages)) {
                        dev_error(P.err, CSLD_DEVERR_PAGE);
                        tok = -1;
                    }
                    if (lane < kTileChunks) sm.chunk_tok[buf][lane] = tok;
                    const int n = __popc(__ballot_sync(0xffffffffu, tok >= 0));
                    if (lane == 0) mbar_arrive_expect_tx(&sm.stfull[buf], n * kChunk * (kFp4 ? kEntry4 : 5 * 128));
                    __syncwarp();
                    const int64_t row = (int64_t)pg * P.c.page_size + (tok >= 0 ? tok % P.c.page_size : 0);
                    if constexpr (kFp4) {
                        if (tok >= 0)
                            bulk_g2s(sm.stage[buf] + lane * kChunk4Bytes, P.c.pages + row * kEntry4, kChunk4Bytes, &sm.stfull[buf]);
                    } else {
                        const int ck = lane / 5, blk = lane % 5;   // one box of 16 rows by 128 bytes per lane
                        const int tk = __shfl_sync(0xffffffffu, tok, ck < kTileChunks ? ck : 0);
                        const int y = __shfl_sync(0xffffffffu, static_cast<int>(row), ck < kTileChunks ? ck : 0);
                        if (ck < kTileChunks && tk >= 0)
                            tma_load_2d(sm.img[buf] + blk * kBlkBytes + ck * kChunk * 128, &pages_map, blk < 4 ? 128 * blk : kNope, y,
                                        &sm.stfull[buf]);
                    }
                    tok = tok1;
                    pg = pg1;
                    if (lane == 0) sm.n_issued = T + 1;
                }
            }
        } else if (lane == 0) {
            // ===== MMA issue ==================================================================================
            if (tmem != 0) *fail = 1;   // the MMAs' column constants
            Walk wp = wk;                              // the walks of QK and of PV
            int nq = 0, np = 0, qt = 0, pt = 0, seg = 0;   // running tiles, tiles within the segments
            uint32_t idle = 0;
            while (np < n_tiles) {
                if (*fail) break;
                if (np < nq && mbar_test(&sm.pfull[np & 1], (np >> 1) & 1)) {
                    tc_fence_after();
                    with_tile<kFp4>(np, IssuePv<kFp4>{sm, pt >= 2 ? 1u : 0u});   // a stream's first tile of a segment overwrites O
                    ++np;
                    if (++pt == wp.len) {
                        pt = 0;
                        wp.next(P);
                    }
                    idle = 0;
                    continue;
                }
                if (nq < n_tiles && nq < np + 2 && mbar_test(&sm.imgfull[nq % kBufs], (nq / kBufs) & 1) &&
                    (qt > 0 || mbar_test(&sm.qready, seg & 1))) {
                    tc_fence_after();
                    with_tile<kFp4>(nq, IssueQk<kFp4>{sm});
                    ++nq;
                    if (++qt == wk.len) {
                        qt = 0;
                        ++seg;
                        wk.next(P);
                    }
                    idle = 0;
                    continue;
                }
                if (++idle > (1u << 22)) {   // nothing became ready for about a second
                    *fail = 1;
                    break;
                }
                if (idle > 64) __nanosleep(20);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (sm.fail) {   // let the copies and MMAs in flight finish (bounded), then report
        if (tid == 0) {
            dev_error(P.err, CSLD_DEVERR_TIMEOUT);
            const int n = sm.n_issued;
            for (int T = max(0, n - kBufs); T < n; ++T) (void)mbar_wait(&sm.stfull[T % kBufs], (T / kBufs) & 1);
        }
        if (warp == kMmaWarp && lane == 0) {
            umma_commit(&sm.drain);
            (void)mbar_wait(&sm.drain, 0);
        }
        __syncthreads();
    }
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Joins the CTAs' parts of the cut rows: block (y, h) takes the y-th cut row, head h.  512 threads: thread t owns
// dims 4 (t % 128) .. + 3 of every fourth part from t / 128 on.
constexpr int kMergeThreads = 512, kMergeU = 8;
__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(const __grid_constant__ Params P, int n_cta) {
    __shared__ float4 red[3][kDim / 4];
    __shared__ float2 mls[1024];
    __shared__ int cnt[kMergeThreads / 32], found;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, h = blockIdx.x;
    pdl_wait();
    pdl_trigger();
    int first = -1;   // the CTA where the y-th cut row begins
    int before = 0;
    for (int c0 = 0; c0 < n_cta && first < 0; c0 += kMergeThreads) {   // one round on every B200
        const int c = c0 + tid;
        const bool cut = c < n_cta && __ldcg(&P.meta[c]).z >= 0;
        const uint32_t bal = __ballot_sync(0xffffffffu, cut);
        if (lane == 0) cnt[warp] = __popc(bal);
        if (tid == 0) found = -1;
        __syncthreads();
        int at = before + __popc(bal & ((1u << lane) - 1));
        for (int w = 0; w < warp; ++w) at += cnt[w];
        if (cut && at == (int)blockIdx.y) found = c;
        for (int w = 0; w < kMergeThreads / 32; ++w) before += cnt[w];
        __syncthreads();
        first = found;
        __syncthreads();
    }
    if (first < 0) return;
    const int4 mt = __ldcg(&P.meta[first]);
    const int n = mt.z - first + 1;
    auto slot = [&](int i) { return 2 * (int64_t)(first + i) + (i == 0 ? 1 : 0); };
    const int d4 = tid % (kDim / 4), g = tid / (kDim / 4);
    const float4* ob = reinterpret_cast<const float4*>(P.opart) + (int64_t)h * (kDim / 4) + d4;
    float4 v[kMergeU];
#pragma unroll
    for (int u = 0; u < kMergeU; ++u) {
        const int i = g + 4 * u;
        v[u] = i < n ? __ldcg(ob + slot(i) * (kHeads * kDim / 4)) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int i = tid; i < n; i += kMergeThreads) mls[i] = __ldcg(&P.mlpart[slot(i) * kHeads + h]);
    __syncthreads();
    float M = -INFINITY, L = 0.f;
    for (int i = lane; i < n; i += 32)
        if (mls[i].y != 0.f) M = fmaxf(M, mls[i].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    for (int i = lane; i < n; i += 32)
        if (mls[i].y != 0.f) L += exp2_ftz(mls[i].x - M) * mls[i].y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](int i, const float4& x) {
        const float f = mls[i].y == 0.f ? 0.f : exp2_ftz(mls[i].x - M);
        if (f != 0.f) {
            acc.x = fmaf(f, x.x, acc.x);
            acc.y = fmaf(f, x.y, acc.y);
            acc.z = fmaf(f, x.z, acc.z);
            acc.w = fmaf(f, x.w, acc.w);
        }
    };
#pragma unroll
    for (int u = 0; u < kMergeU; ++u)
        if (g + 4 * u < n) add(g + 4 * u, v[u]);
#pragma unroll 4
    for (int i = g + 4 * kMergeU; i < n; i += 4) add(i, __ldcg(ob + slot(i) * (kHeads * kDim / 4)));
    if (g > 0) red[g - 1][d4] = acc;
    __syncthreads();
    const int64_t row = (static_cast<int64_t>(mt.y) << 32) | static_cast<uint32_t>(mt.x);
    const int rq = static_cast<int>(row % (P.Q * P.groups)), hh = 16 * (rq % P.groups) + h;
    if (g != 0 || hh >= P.heads) return;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        acc.x += red[k][d4].x;
        acc.y += red[k][d4].y;
        acc.z += red[k][d4].z;
        acc.w += red[k][d4].w;
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const int64_t at = (row / (P.Q * P.groups) * P.Q + rq / P.groups) * P.heads + hh;
    if (P.out_bf16)
        reinterpret_cast<uint2*>(P.out)[at * (kDim / 4) + d4] =
            make_uint2(f32x2_to_bf16x2_bits(acc.x * inv, acc.y * inv), f32x2_to_bf16x2_bits(acc.z * inv, acc.w * inv));
    else
        reinterpret_cast<float4*>(P.out)[at * (kDim / 4) + d4] = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    if (P.lse && tid == 0) P.lse[at] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
}

namespace {
constexpr size_t kPartBytes = 2 * kHeads * (kDim * sizeof(float) + sizeof(float2)) + sizeof(int4);   // per CTA
}

size_t paged_attention_ws_bytes(int num_sms) { return num_sms * kPartBytes; }

cudaError_t launch_paged_attention(const PagedView& c, bool fp4, const uint16_t* q, int heads, int Q, int W, int sinks,
                                   float scale, void* out, bool out_bf16, float* lse_out, void* ws, int num_sms,
                                   int32_t* err, cudaStream_t stream) {
    Params P;
    P.c = c;
    P.q = q;
    P.out = out;
    P.lse = lse_out;
    P.opart = static_cast<float*>(ws);
    P.mlpart = reinterpret_cast<float2*>(P.opart + (size_t)num_sms * 2 * kHeads * kDim);
    P.meta = reinterpret_cast<int4*>(P.mlpart + (size_t)num_sms * 2 * kHeads);
    P.err = err;
    P.scale = scale;
    P.heads = heads;
    P.groups = (heads + kHeads - 1) / kHeads;
    P.Q = Q;
    P.W = W;
    P.sinks = sinks;
    P.min_tiles = 1;
    P.out_bf16 = out_bf16;
    CUtensorMap map = {};   // fp8: the pages as rows of 576 bytes
    if (!fp4 && !make_tensor_map_2d_u8(&map, c.pages, kEntry, (uint64_t)c.n_pages * c.page_size, 128, kChunk))
        return cudaErrorInvalidValue;
    const size_t smem = fp4 ? sizeof(Smem<true>) : sizeof(Smem<false>);
    auto kernel = fp4 ? paged_attention_kernel<true> : paged_attention_kernel<false>;
    cudaError_t e = set_smem_once(kernel, smem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kernel, dim3(num_sms), dim3(kThreads), smem, stream, map, P);
    if (e != cudaSuccess) return e;
    const int64_t rows = (int64_t)c.batch * Q * P.groups, most = rows < num_sms - 1 ? rows : num_sms - 1;
    e = launch_pdl(paged_merge_kernel, dim3(kHeads, static_cast<unsigned>(most)), dim3(kMergeThreads), 0, stream, P, num_sms);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace csld
