// Attention over the paged entry cache: a sliding window with first tokens that stay visible, or every
// token (layouts: csld_paged_cache in csld.h).
//
// Source: "DeepSeek-V4: a million-token context that agents can actually use" -- CSA and HCA paragraphs
// (a sliding-window branch over the most recent uncompressed tokens), storage paragraph (entries in low
// precision except the RoPE dims in bf16; FP4 where it suffices), layer-pattern paragraph (the
// window-only multi-token-prediction block).
//
// out_h = sum_t p_t k_t / l,  p_t = 2^(scale log2(e) q_h.k_t + nm),  l = sum_t p_t over the visible tokens t,
// keys = values = the 512-d entry, 16 heads of one query at a time.
//
// Work.  A row is one (sequence, query, group of 16 heads).  Its token list is made of 16-token chunks, each
// inside one page: the chunks of the first tokens, then those of the window (or all), four chunks to a tile.
// The tiles of all rows, row after row, are dealt out evenly to one CTA per SM, so sequences of any mix of
// lengths load the SMs alike; a CTA walks its share as segments of rows.  A row that lies whole in one share is
// written out directly; of a row cut by shares each CTA leaves its unnormalised O and (m, l), and
// paged_merge_kernel joins them.
//
// Which tensor instructions.  With 16 heads one side of every product is 16 rows.  A tcgen05.mma reads its
// 128-row operand, here the entries, from shared memory at 128 B a cycle: 45 cycles for 128 x 32 x 32 (measured;
// 16 at full rate), and a version of this kernel built on it moved 326 KB through shared memory for 96 fp4
// entries and took 3000 cycles (1M fp4 tokens 222 us).  The warp-level E4M3 mma.sync runs at 3800 MAC a cycle
// and SM (measured) with its operands in registers: the query stays there for a whole row, 4-bit keys go from a
// code word to a B fragment without touching shared memory, and only the values take that way.
//
// A CTA's roles (16 warps; registers moved from the copy warps to the score warps):
//   copy   (warp 12)    pages -> a ring of tiles in shared memory: fp4 chunks as they lie (5888 contiguous bytes, bulk
//                       copies), fp8 entries as five 128-byte column blocks with the 128-byte swizzle (tensor map)
//   score  (warps 0-3)  warp w takes the tile's chunk w.  S = Q K^T by m16n8k32 E4M3 MMAs, the bf16 query as two E4M3
//                       terms (exact: 4 + 4 significant bits and a sign), the RoPE dims by bf16 MMAs.  fp4: lane
//                       (n, c) = (lane / 4, lane % 4) decodes word c of entry n's group: its 8 codes are that
//                       lane's whole share of the group's 32-dim MMA step, in whatever order, since the query's
//                       dims are laid out the same.  E2M1 -> E4M3 is a byte permute through 8 table bytes, 2^(6-j)
//                       times the grid, j = the entry's largest exponent minus the group's: all normal numbers, so
//                       j only subtracts 8 j from each (j > 11 or a NaN group: from a table in shared memory); an
//                       entry's decoded bytes are its values over one power of two f_e, applied to S and to P.
//                       The decoded bytes also go to the value image.  Then the softmax: p relative to a mark nm that
//                       is only raised when some p exceeds 2^10..15, one meeting of the four warps a tile, and P as
//                       A fragments in shared memory: p f_e as three E5M2 terms, p as bf16 for the RoPE dims.
//   value  (warps 4-11) warp w owns 64 of the 512 dims and keeps its O in registers: O += P V by m16n8k32 E5M2 x E4M3
//                       MMAs, V fragments by transposing 8-bit matrix loads of the image (fp8: of the copied tile
//                       itself); warp 11 the RoPE dims, bf16
// Rows of masked or missing tokens are zeroed before they are used, whatever was in them.  Every wait is
// bounded; a wait that gives up sets CSLD_DEVERR_TIMEOUT and all roles run out without waiting.
#include <stdint.h>

#include "kernels.cuh"
#include "paged.cuh"
#include "sm100.cuh"

namespace csld {

namespace {

constexpr int kThreads = 512;
constexpr int kScoreWarps = 4, kValueWarp = 4, kValueWarps = 8, kCopyWarp = 12;
// registers a thread: the launch gives 512 x 128 = 65,536; 128 x 216 + 256 x 120 + 128 x 40 = 63,488
constexpr int kRegsScore = 216, kRegsValue = 120, kRegsCopy = 40;
constexpr int kTile = 64, kTileChunks = kTile / kChunk;   // entries per tile; a chunk per score warp
static_assert(kTileChunks == kScoreWarps, "score warp w takes chunk w");
constexpr int kBlkBytes = kTile * 128;           // one 128-byte column block of a tile
constexpr int kImgBytes = 5 * kBlkBytes;         // dims 0..127, 128..255, 256..383, 384..447, RoPE
constexpr int kSteps = kGroups;                  // 32-dim steps of the 448 dims
// Marks: a head's nm is set so that the largest p of a tile is 2^kLift and kept until one exceeds 2^kOver.  The
// operand holds p w in f16, w = 1 (fp8) or f_e g (fp4; g a power of two set so that the tile's largest f_e g is
// kFeSet, kept until one exceeds kFeMost).  f16 bounds the product: 2^kOver w <= 2^15.
template <bool kFp4> constexpr float kLift = kFp4 ? 0.f : 5.f;
template <bool kFp4> constexpr float kOver = kFp4 ? 10.f : 15.f;
constexpr float kFeSet = 8.f, kFeMost = 32.f, kUnset = 1e30f;
constexpr int kBarScore = 1;                     // named barrier of the score warps

template <bool kFp4>
struct Smem {
    static constexpr int kStages = 5;
    static constexpr int kStageBytes = kFp4 ? kTileChunks * kChunk4Bytes : kImgBytes;
    uint8_t img[kFp4 ? 2 : 1][kFp4 ? kImgBytes : 1024];   // fp4: value images [block][entry][128 B], 128-byte swizzle
    uint8_t stage[kStages][kStageBytes];         // fp8: the same layout, as copied
    uint4 p16[2][kTileChunks][32];               // P in f16: [chunk][lane] A fragments
    uint4 pbf[2][kTileChunks][32];               // bf16 P: [chunk][lane]
    float fn[2][kHeads], fr[2][kHeads];          // factors of O before a tile's MMAs (448 dims; RoPE dims)
    float tmax[kScoreWarps][kHeads], femax[kScoreWarps];
    float lsum[2][kScoreWarps][kHeads], mseg[2][kHeads], ginv[2];   // a segment's sums, marks and 1 / g
    int32_t chunk_tok[kStages][kTileChunks];     // first token of a tile's chunks; -1: none
    int32_t resc[2];                             // 0: O stays, 1: O *= f, 2: O = 0 (first tile of a segment)
    uint64_t full[kStages], empty[kStages], pfull[2], pempty[2], segfull[2], segempty[2];
    int64_t red[kThreads / 32], prefix;
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
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        :: "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two 16 x 16 byte matrices, transposed: lane i gives the address of row i (16 B).  r0, r2: bytes of rows 4 (lane % 4)
// .. + 3 of the first and second matrix at column lane / 4; r1, r3: at column 8 + lane / 4.
__device__ __forceinline__ void ldmatrix_b8_trans_x2(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldmatrix_b16_trans_x4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
template <int kRegs>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs)); }
template <int kRegs>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs)); }

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

// ---- numbers --------------------------------------------------------------------------------
// Eight E2M1 codes (one word) -> eight bytes of the table tab with the codes' signs.
__device__ __forceinline__ void decode8(uint32_t w, uint2 tab, uint32_t& lo, uint32_t& hi) {
    const uint32_t sel = w & 0x77777777u;
    lo = __byte_perm(tab.x, tab.y, sel) | (w & 0x80808080u);
    hi = __byte_perm(tab.x, tab.y, sel >> 16) | ((w << 4) & 0x80808080u);
}
// 2^13 times the E2M1 grid (0, 4096, 8192, 12288, 16384, 24576, 32768, 49152) in E5M2, and what a factor of 1/2 takes off.
constexpr uint32_t kTabX = 0x72706C00u, kTabY = 0x7A787674u, kTabDx = 0x04040400u, kTabDy = 0x04040404u;
constexpr int kMaxJ = 26;                        // the table's smallest entry stays a normal number

// Two bytes of v, E5M2 or E4M3, as two f16 (exact).  E5M2 is f16's upper byte.
template <bool kE5M2, int kHalf>
__device__ __forceinline__ uint32_t bytes_to_f16x2(uint32_t v) {
    if constexpr (kE5M2) return __byte_perm(v, 0u, kHalf ? 0x3424 : 0x1404);
    else return e4m3x2_to_f16x2(kHalf ? v >> 16 : v & 0xFFFFu);
}
__device__ __forceinline__ uint32_t f32x2_to_f16x2(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// ---- the query ---------------------------------------------------------------------------------
// A fragments of 16 heads' queries: lane (g, c) holds heads g and g + 8, of every 32-dim step the dims 8c..8c+7
// (f16: two 16-dim MMA steps, the dims in the order that the lane's eight key bytes come in), of every 16-dim
// RoPE step the dims 4c..4c+3 (bf16), scaled per head by a power of two so that its largest value lies in
// 2^7..2^8: exact in f16 down to 2^-21 of it.
struct Query {
    uint32_t f[kSteps][2][4], rope[4][4];
    float c2[2];         // logit factor (log2 units) of the two heads
    __device__ __forceinline__ void load(const Params& P, int b, int rq, int g, int c) {
        const int j = rq / P.groups, h0 = 16 * (rq % P.groups) + g;
        const uint16_t* q0 = P.q + (((int64_t)b * P.Q + j) * P.heads + h0) * kDim;
        uint32_t top[2] = {0, 0};
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint4 v = h0 + 8 * r < P.heads ? __ldg(reinterpret_cast<const uint4*>(q0 + 8 * r * kDim + 32 * s + 8 * c))
                                                     : make_uint4(0, 0, 0, 0);
                f[s][0][r] = v.x;
                f[s][0][2 + r] = v.y;
                f[s][1][r] = v.z;
                f[s][1][2 + r] = v.w;
            }
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint2 v = h0 + 8 * r < P.heads
                                    ? __ldg(reinterpret_cast<const uint2*>(q0 + 8 * r * kDim + kNope + 16 * s + 4 * c)) : make_uint2(0, 0);
                rope[s][r] = v.x;
                rope[s][2 + r] = v.y;
            }
        auto peak = [&](int i, uint32_t x) { top[i & 1] = max(top[i & 1], max(x & 0x7FFFu, (x >> 16) & 0x7FFFu)); };
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                peak(i, f[s][0][i]);
                peak(i, f[s][1][i]);
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) peak(i, rope[s][i]);
        }
        float sq[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            top[r] = max(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
            top[r] = max(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
            const int sh = top[r] ? max(-100, min(100, 134 - static_cast<int>(top[r] >> 7))) : 0;
            sq[r] = pow2f(sh);
            c2[r] = P.scale * 1.4426950408889634f / sq[r];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    f[s][u][i] = f32x2_to_f16x2(bf16_bits_to_f32(f[s][u][i]) * sq[i & 1], bf16_bits_to_f32(f[s][u][i] >> 16) * sq[i & 1]);
#pragma unroll
            for (int s = 0; s < 4; ++s)
                rope[s][i] = f32x2_to_bf16x2_bits(bf16_bits_to_f32(rope[s][i]) * sq[i & 1], bf16_bits_to_f32(rope[s][i] >> 16) * sq[i & 1]);
        }
    }
};

__device__ __forceinline__ void store_out2(const Params& P, int64_t at, float a, float b) {
    if (P.out_bf16) *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(P.out) + at) = f32x2_to_bf16x2_bits(a, b);
    else *reinterpret_cast<float2*>(reinterpret_cast<float*>(P.out) + at) = make_float2(a, b);
}

// ---- score warps ---------------------------------------------------------------------------------
template <bool kFp4>
__device__ __forceinline__ void score_role(Smem<kFp4>& sm, const Params& P, Walk wk, int w, int lane, int64_t u1, int64_t n_cta,
                                           int64_t total) {
    constexpr int kStages = Smem<kFp4>::kStages;
    volatile int32_t* fail = &sm.fail;
    const int g = lane >> 2, c = lane & 3;
    // place of this lane's eight bytes of step s, entry n = 8 nt + g of chunk w: block s / 4, row 16 w + n
    uint32_t at[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) at[q] = (16 * w + g) * 128 + ((((c >> 1) ^ g) ^ (2 * q)) << 4) + 8 * (c & 1);
    Query qy;
    int T = 0, seg = 0;
    for (; wk.left > 0; wk.next(P), ++seg) {
        qy.load(P, wk.b, wk.rq, g, c);
        const int p = wk.s.n - P.Q + wk.rq / P.groups;   // the query's position
        float nm[2] = {kUnset, kUnset}, l[2] = {0.f, 0.f}, gs = 0.f;   // gs = 0: g not set yet
        for (int t = 0; t < wk.len; ++t, ++T) {
            const int st = T % kStages, buf = T & 1;
            bool ok = wait(&sm.full[st], (T / kStages) & 1, fail);
            if (T >= 2) ok = ok && wait(&sm.pempty[buf], ((T >> 1) - 1) & 1, fail);
            ok = __all_sync(0xffffffffu, ok);
            const int tok0 = ok ? sm.chunk_tok[st][w] : -1;
            auto sees_entry = [&](int en) { return tok0 >= 0 && sees(P, tok0 + en, p); };
            float acc[2][2][4], racc[2][4];   // [entries 8 nt ..][half of a step: independent chains], RoPE part
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[nt][0][i] = acc[nt][1][i] = racc[nt][i] = 0.f;
            uint8_t* img = kFp4 ? sm.img[kFp4 ? buf : 0] : sm.stage[st];
            float fe[2][2];   // of the entries 8 nt + 2 c + i: the columns of this lane's scores
            if constexpr (kFp4) {
                const uint8_t* ch = sm.stage[st] + w * kChunk4Bytes;
                // RoPE rows into the image, eight lanes a row
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int en = 4 * i + (lane >> 3), k = lane & 7;
                    uint4 v = *reinterpret_cast<const uint4*>(ch + kChunk4Rope + en * 2 * kRope + 16 * k);
                    if (!sees_entry(en)) v = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4*>(img + 4 * kBlkBytes + sw128(16 * w + en, 16 * k)) = v;
                }
                int base[2];
                uint32_t tx[2], ty[2], dx[2], dy[2];
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    const bool vis = sees_entry(8 * nt + g);   // masked: every byte decodes to a signed zero
                    base[nt] = ch[kChunk4Exp + kGroups * kChunk + 8 * nt + g];
                    tx[nt] = vis ? kTabX : 0u;
                    ty[nt] = vis ? kTabY : 0u;
                    dx[nt] = vis ? kTabDx : 0u;
                    dy[nt] = vis ? kTabDy : 0u;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t eb = ch[kChunk4Exp + kGroups * kChunk + 8 * nt + 2 * c + i];
                        fe[nt][i] = __uint_as_float(eb << 23) * 0x1p-13f;
                    }
                }
                // j above kMaxJ (a group of 2^-26 of the entry's largest: zero) or below 0 (a NaN group) in some entry.
                // Lane (g, c) looks at the groups c, c + 4, ..
                uint32_t most = 0;
#pragma unroll
                for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        if (dx[nt] && 4 * s + c < kSteps)
                            most = max(most, static_cast<uint32_t>(base[nt] - ch[kChunk4Exp + (4 * s + c) * kChunk + 8 * nt + g]));
                const bool far = __any_sync(0xffffffffu, most > kMaxJ);
                // words and exponents come in blocks of four steps, a block ahead of their use (a load may not pass a
                // store to the image, as far as the compiler knows)
                uint32_t wd[2][4][2];
                int ex[2][4][2];
                auto fetch = [&](int blk) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int nt = 0; nt < 2; ++nt) {
                            const int s = 4 * blk + i;
                            if (s >= kSteps) continue;
                            wd[blk & 1][i][nt] = *reinterpret_cast<const uint32_t*>(ch + s * 256 + (8 * nt + g) * 16 + 4 * c);
                            ex[blk & 1][i][nt] = ch[kChunk4Exp + s * kChunk + 8 * nt + g];
                        }
                };
                fetch(0);
#pragma unroll
                for (int blk = 0; blk < 4; ++blk) {
                    if (blk < 3) fetch(blk + 1);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int nt = 0; nt < 2; ++nt) {
                            const int s = 4 * blk + i;
                            if (s >= kSteps) continue;
                            const int j = base[nt] - ex[blk & 1][i][nt];
                            uint2 tab = make_uint2(tx[nt] - j * dx[nt], ty[nt] - j * dy[nt]);
                            if (far && dx[nt] && (j < 0 || j > kMaxJ)) tab.x = tab.y = j < 0 ? 0x7F7F7F7Fu : 0u;
                            uint32_t b0, b1;
                            decode8(wd[blk & 1][i][nt], tab, b0, b1);
                            *reinterpret_cast<uint2*>(img + blk * kBlkBytes + nt * 1024 + at[i]) = make_uint2(b0, b1);
                            mma_f16(acc[nt][0], qy.f[s][0], bytes_to_f16x2<true, 0>(b0), bytes_to_f16x2<true, 1>(b0));
                            mma_f16(acc[nt][1], qy.f[s][1], bytes_to_f16x2<true, 0>(b1), bytes_to_f16x2<true, 1>(b1));
                        }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.empty[st]);
            } else {
                fe[0][0] = fe[0][1] = fe[1][0] = fe[1][1] = 1.f;
                // masked rows are zeroed for the value warps
                if (!__all_sync(0xffffffffu, sees_entry(lane & 15))) {
                    for (int en = 0; en < 16; ++en)
                        if (!sees_entry(en))
                            for (int k = lane; k < 40; k += 32)
                                *reinterpret_cast<uint4*>(img + (k >> 3) * kBlkBytes + sw128(16 * w + en, 16 * (k & 7))) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();   // the ring's next copy writes there too
                    __syncwarp();
                }
#pragma unroll
                for (int s = 0; s < kSteps; ++s)
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) {
                        const uint2 b = *reinterpret_cast<const uint2*>(img + (s >> 2) * kBlkBytes + nt * 1024 + at[s & 3]);
                        mma_f16(acc[nt][0], qy.f[s][0], bytes_to_f16x2<false, 0>(b.x), bytes_to_f16x2<false, 1>(b.x));
                        mma_f16(acc[nt][1], qy.f[s][1], bytes_to_f16x2<false, 0>(b.y), bytes_to_f16x2<false, 1>(b.y));
                    }
            }
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    const uint2 b = *reinterpret_cast<const uint2*>(img + 4 * kBlkBytes + nt * 1024 + at[s]);
                    mma_bf16(racc[nt], qy.rope[s][0], qy.rope[s][1], qy.rope[s][2], qy.rope[s][3], b.x, b.y);
                }
            // logits x[nt][2 r + i]: entry 8 nt + 2 c + i, head g + 8 r (log2 units), -inf where masked
            float x[2][4];
            bool see[2][2];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    see[nt][i] = sees_entry(8 * nt + 2 * c + i);
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int k = 2 * r + i;
                        const float v = kFp4 ? fmaf(acc[nt][0][k] + acc[nt][1][k], fe[nt][i], racc[nt][k])
                                             : (acc[nt][0][k] + acc[nt][1][k]) + racc[nt][k];
                        x[nt][k] = see[nt][i] ? v * qy.c2[r] : -INFINITY;
                    }
                    if (!see[nt][i]) fe[nt][i] = 0.f;
                }
            float top[2], fmost = fmaxf(fmaxf(fe[0][0], fe[0][1]), fmaxf(fe[1][0], fe[1][1]));
#pragma unroll
            for (int r = 0; r < 2; ++r) top[r] = fmaxf(fmaxf(x[0][2 * r], x[0][2 * r + 1]), fmaxf(x[1][2 * r], x[1][2 * r + 1]));
            const bool over = top[0] + nm[0] > kOver<kFp4> || top[1] + nm[1] > kOver<kFp4> || (kFp4 && fmost * gs > kFeMost);
            int resc = t == 0 ? 2 : 0;
            if (named_barrier_or(kBarScore, 32 * kScoreWarps, over)) {
                // some weight is too large, or the first tile: the tile's maxima; a head that lies more than 2 above its
                // mark gets a new one, and the value warps the factors of what they hold
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
                    top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
                    if (c == 0) sm.tmax[w][g + 8 * r] = top[r];
                }
                if constexpr (kFp4) {
                    const uint32_t fm = __reduce_max_sync(0xffffffffu, __float_as_uint(fmost));
                    if (lane == 0) sm.femax[w] = __uint_as_float(fm);
                }
                named_barrier(kBarScore, 32 * kScoreWarps);
                float fg = 1.f;
                if constexpr (kFp4) {
                    const float fm = fmaxf(fmaxf(sm.femax[0], sm.femax[1]), fmaxf(sm.femax[2], sm.femax[3]));
                    if (fm > 0.f && (gs == 0.f || fm * gs > kFeMost)) {
                        const float gn = kFeSet / fmaxf(fm, 0x1p-110f);
                        if (gs != 0.f) fg = gn / gs;
                        gs = gn;
                    }
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float tm = sm.tmax[0][g + 8 * r];
#pragma unroll
                    for (int k = 1; k < kScoreWarps; ++k) tm = fmaxf(tm, sm.tmax[k][g + 8 * r]);
                    const bool first = nm[r] == kUnset;
                    const bool set = first ? tm > -INFINITY : tm + nm[r] > kLift<kFp4> + 2.f;
                    const float to = set ? kLift<kFp4> - tm : nm[r];
                    const float f = set && !first ? exp2_ftz(to - nm[r]) : 1.f;
                    l[r] *= f;
                    nm[r] = to;
                    if (w == 0 && c == 0) {
                        sm.fn[buf][g + 8 * r] = f * fg;
                        sm.fr[buf][g + 8 * r] = f;
                    }
                }
                if (t > 0) resc = 1;
            }
            // P: p = 2^(x + nm), as A fragments: of the chunk's 16 entries a lane holds 8 nt + 2 c + i, the MMA's k slots
            // 2c + i (nt = 0) and 2c + 8 + i
            uint32_t pb[2][2], ph[2][2];   // [r][nt]
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    const float p0 = exp2_ftz(x[nt][2 * r] + nm[r]), p1 = exp2_ftz(x[nt][2 * r + 1] + nm[r]);
                    l[r] += p0 + p1;
                    pb[r][nt] = f32x2_to_bf16x2_bits(p0, p1);
                    ph[r][nt] = kFp4 ? f32x2_to_f16x2(p0 * (fe[nt][0] * gs), p1 * (fe[nt][1] * gs)) : f32x2_to_f16x2(p0, p1);
                }
            sm.p16[buf][w][lane] = make_uint4(ph[0][0], ph[1][0], ph[0][1], ph[1][1]);
            sm.pbf[buf][w][lane] = make_uint4(pb[0][0], pb[1][0], pb[0][1], pb[1][1]);
            if (w == 0 && lane == 0) sm.resc[buf] = resc;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.pfull[buf]);
        }
        // ---- the segment's sums --------------------------------------------------------------------
        const int sb = seg & 1;
        if (seg >= 2) (void)wait(&sm.segempty[sb], ((seg >> 1) - 1) & 1, fail);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            if (c == 0) {
                sm.lsum[sb][w][g + 8 * r] = l[r];
                if (w == 0) sm.mseg[sb][g + 8 * r] = -nm[r];
            }
        }
        if (w == 0 && lane == 0) {
            sm.ginv[sb] = gs != 0.f ? 1.f / gs : 1.f;
            if (wk.t == 0 && wk.len < wk.s.tiles) {   // a cut row begins here: which CTA holds its end
                const int64_t row = (int64_t)wk.b * P.Q * P.groups + wk.rq;
                const int64_t end = u1 - wk.left + wk.s.tiles;    // unit behind the row
                int64_t e = (end - 1) * n_cta / total;
                while (total * (e + 1) / n_cta <= end - 1) ++e;
                while (total * e / n_cta > end - 1) --e;
                P.meta[blockIdx.x] = make_int4(static_cast<int>(row), static_cast<int>(row >> 32), static_cast<int>(e), 0);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.segfull[sb]);
    }
}

// ---- value warps ---------------------------------------------------------------------------------
template <bool kFp4>
__device__ __forceinline__ void value_role(Smem<kFp4>& sm, const Params& P, Walk wk, int w, int lane) {
    constexpr int kStages = Smem<kFp4>::kStages;
    volatile int32_t* fail = &sm.fail;
    const int g = lane >> 2, c = lane & 3;
    const bool rope = w == kValueWarps - 1;
    // this lane's row address of the matrix loads within a 32-entry block (448 dims) or a 16-entry chunk (RoPE), and
    // the 16-byte column it starts from
    int row, col;
    if (!rope) {
        const int k = lane & 15, i = k & 3;   // row k of a transposing load (slots 4c + i) -> entry of the chunk lane / 16
        row = 16 * (lane >> 4) + (i < 2 ? 2 * (k >> 2) + i : 8 + 2 * (k >> 2) + i - 2);
        col = 4 * (w & 1);
    } else {
        row = (lane & 7) + 8 * ((lane >> 3) & 1);
        col = lane >> 4;
    }
    const uint32_t off = (rope ? 4 : w >> 1) * kBlkBytes + (row >> 3) * 1024 + (row & 7) * 128;
    float o[8][4];
    int T = 0, seg = 0;
    for (; wk.left > 0; wk.next(P), ++seg) {
        for (int t = 0; t < wk.len; ++t, ++T) {
            const int buf = T & 1, st = T % kStages;
            bool ok = wait(&sm.pfull[buf], (T >> 1) & 1, fail);
            if (!kFp4) ok = ok && wait(&sm.full[st], (T / kStages) & 1, fail);   // complete: makes the copy visible here
            ok = __all_sync(0xffffffffu, ok);
            const int resc = sm.resc[buf];
            if (resc == 2) {
#pragma unroll
                for (int q = 0; q < 8; ++q)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[q][i] = 0.f;
            } else if (resc == 1) {
                const float* f = rope ? sm.fr[buf] : sm.fn[buf];
                const float f0 = f[g], f1 = f[g + 8];
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    o[q][0] *= f0;
                    o[q][1] *= f0;
                    o[q][2] *= f1;
                    o[q][3] *= f1;
                }
            }
            if (ok) {
                const uint32_t base = smem_u32(kFp4 ? sm.img[kFp4 ? buf : 0] : sm.stage[st]) + off;
                if (!rope) {
#pragma unroll
                    for (int kb = 0; kb < kTile / 32; ++kb) {
                        const uint4 p0 = sm.p16[buf][2 * kb][lane], p1 = sm.p16[buf][2 * kb + 1][lane];
                        const uint32_t a0[4] = {p0.x, p0.y, p0.z, p0.w}, a1[4] = {p1.x, p1.y, p1.z, p1.w};
                        uint32_t v[4][4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) ldmatrix_b8_trans_x2(v[q], base + kb * 4096 + (((col + q) ^ (row & 7)) << 4));
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            mma_f16(o[2 * q], a0, bytes_to_f16x2<kFp4, 0>(v[q][0]), bytes_to_f16x2<kFp4, 1>(v[q][0]));
                            mma_f16(o[2 * q + 1], a0, bytes_to_f16x2<kFp4, 0>(v[q][1]), bytes_to_f16x2<kFp4, 1>(v[q][1]));
                        }
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            mma_f16(o[2 * q], a1, bytes_to_f16x2<kFp4, 0>(v[q][2]), bytes_to_f16x2<kFp4, 1>(v[q][2]));
                            mma_f16(o[2 * q + 1], a1, bytes_to_f16x2<kFp4, 0>(v[q][3]), bytes_to_f16x2<kFp4, 1>(v[q][3]));
                        }
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < kTileChunks; ++k) {
                        const uint4 a = sm.pbf[buf][k][lane];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t v[4];
                            ldmatrix_b16_trans_x4(v, base + k * 2048 + (((col + 2 * q) ^ (row & 7)) << 4));
                            mma_bf16(o[2 * q], a.x, a.y, a.z, a.w, v[0], v[1]);
                            mma_bf16(o[2 * q + 1], a.x, a.y, a.z, a.w, v[2], v[3]);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sm.pempty[buf]);
                if (!kFp4) mbar_arrive(&sm.empty[st]);
            }
        }
        // ---- the segment's result ------------------------------------------------------------------
        const int sb = seg & 1;
        const bool ok = __all_sync(0xffffffffu, wait(&sm.segfull[sb], (seg >> 1) & 1, fail));
        float L[2], M[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int h = g + 8 * r;
            L[r] = (sm.lsum[sb][0][h] + sm.lsum[sb][1][h]) + (sm.lsum[sb][2][h] + sm.lsum[sb][3][h]);
            M[r] = sm.mseg[sb][h];
        }
        const float gi = rope ? 1.f : sm.ginv[sb];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.segempty[sb]);
        if (!ok) continue;
        const bool whole = wk.t == 0 && wk.len == wk.s.tiles;
        const int j = wk.rq / P.groups, h0 = 16 * (wk.rq % P.groups) + g;
        const int64_t head = ((int64_t)wk.b * P.Q + j) * P.heads + h0;
        const int64_t slot = 2 * (int64_t)blockIdx.x + (wk.t == 0 ? 1 : 0);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float f = whole ? (L[r] == 0.f ? 0.f : gi / L[r]) : gi;
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const int d = 64 * w + 8 * q + 2 * c;
                const float v0 = o[q][2 * r] * f, v1 = o[q][2 * r + 1] * f;
                if (!whole) *reinterpret_cast<float2*>(P.opart + (slot * kHeads + g + 8 * r) * kDim + d) = make_float2(v0, v1);
                else if (h0 + 8 * r < P.heads) store_out2(P, (head + 8 * r) * kDim + d, v0, v1);
            }
            if (w == 0 && c == 0) {
                if (!whole) P.mlpart[slot * kHeads + g + 8 * r] = make_float2(M[r], L[r]);
                else if (P.lse && h0 + 8 * r < P.heads)
                    P.lse[head + 8 * r] = L[r] == 0.f ? -INFINITY : (M[r] + log2f(L[r])) * 0.69314718055994531f;
            }
        }
    }
}

// ---- copy warp -------------------------------------------------------------------------------------
template <bool kFp4>
__device__ __forceinline__ void copy_role(Smem<kFp4>& sm, const Params& P, Walk wk, int lane, const CUtensorMap* pages_map) {
    constexpr int kStages = Smem<kFp4>::kStages;
    volatile int32_t* fail = &sm.fail;
    int T = 0;
    // lane i < 4: chunk i of the tile; its first token and page, loaded one tile ahead
    auto look = [&](const Walk& w, int t, int& tok, int32_t& pg) {
        tok = lane < kTileChunks ? w.token_of_chunk((w.t + t) * kTileChunks + lane) : -1;
        pg = tok >= 0 ? __ldg(P.c.table + (int64_t)w.b * P.c.max_pages + tok / P.c.page_size) : -1;
    };
    for (; wk.left > 0; wk.next(P)) {
        int tok, tok1 = -1;
        int32_t pg, pg1 = -1;
        look(wk, 0, tok, pg);
        for (int t = 0; t < wk.len; ++t, ++T) {
            if (t + 1 < wk.len) look(wk, t + 1, tok1, pg1);
            const int st = T % kStages;
            bool ok = !*fail;
            if (T >= kStages) ok = ok && wait(&sm.empty[st], (T / kStages - 1) & 1, fail);
            if (!__all_sync(0xffffffffu, ok)) return;
            if (tok >= 0 && (pg < 0 || pg >= P.c.n_pages)) {
                dev_error(P.err, CSLD_DEVERR_PAGE);
                tok = -1;
            }
            if (lane < kTileChunks) sm.chunk_tok[st][lane] = tok;
            const int n = __popc(__ballot_sync(0xffffffffu, tok >= 0));
            __syncwarp();
            if (lane == 0) {
                sm.n_issued = T + 1;
                mbar_arrive_expect_tx(&sm.full[st], n * kChunk * (kFp4 ? kEntry4 : 5 * 128));
            }
            __syncwarp();
            const int64_t row = (int64_t)pg * P.c.page_size + (tok >= 0 ? tok % P.c.page_size : 0);
            if constexpr (kFp4) {
                if (tok >= 0) bulk_g2s(sm.stage[st] + lane * kChunk4Bytes, P.c.pages + row * kEntry4, kChunk4Bytes, &sm.full[st]);
            } else {
                const int ck = lane / 5, blk = lane % 5;   // one box of 16 rows by 128 bytes a lane
                const int tk = __shfl_sync(0xffffffffu, tok, ck < kTileChunks ? ck : 0);
                const int y = __shfl_sync(0xffffffffu, static_cast<int>(row), ck < kTileChunks ? ck : 0);
                if (ck < kTileChunks && tk >= 0)
                    tma_load_2d(sm.stage[st] + blk * kBlkBytes + ck * kChunk * 128, pages_map, blk < 4 ? 128 * blk : kNope, y, &sm.full[st]);
            }
            tok = tok1;
            pg = pg1;
        }
    }
}

}  // namespace

template <bool kFp4>
__global__ void __launch_bounds__(kThreads, 1) paged_attention_kernel(const __grid_constant__ CUtensorMap pages_map,
                                                                      const __grid_constant__ Params P) {
    using S = Smem<kFp4>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    S& sm = *reinterpret_cast<S*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    // ---- setup --------------------------------------------------------------------------------
    if (tid == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], kFp4 ? kScoreWarps : kValueWarps);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sm.pfull[s], kScoreWarps);
            mbar_init(&sm.pempty[s], kValueWarps);
            mbar_init(&sm.segfull[s], kScoreWarps);
            mbar_init(&sm.segempty[s], kValueWarps);
        }
        sm.fail = 0;
        sm.n_issued = 0;
        fence_barrier_init();
    }
    if (!kFp4 && warp == kCopyWarp && lane == 0) tma_prefetch_map(&pages_map);
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
    auto block_scan = [&](int64_t v, int64_t& total) {   // exclusive prefix of v over the threads
        int64_t inc = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        __syncthreads();
        if (lane == 31) sm.red[warp] = inc;
        __syncthreads();
        int64_t before = 0;
        total = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += sm.red[w];
            total += sm.red[w];
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
    if (n_tiles > 0) {   // the sequence that the share begins in
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
    if (tid == 0) P.meta[blockIdx.x] = make_int4(0, 0, -1, 0);   // overwritten by this thread where a cut row begins
    __syncthreads();
    if (n_tiles > 0) {
        Walk wk;
        wk.begin(P, sm.b0, u0 - sm.prefix, n_tiles);
        if (warp < kScoreWarps) {
            regs_inc<kRegsScore>();
            score_role<kFp4>(sm, P, wk, warp, lane, u1, n_cta, total);
        } else if (warp < kValueWarp + kValueWarps) {
            regs_dec<kRegsValue>();
            value_role<kFp4>(sm, P, wk, warp - kValueWarp, lane);
        } else {
            regs_dec<kRegsCopy>();
            if (warp == kCopyWarp) copy_role<kFp4>(sm, P, wk, lane, &pages_map);
        }
    }
    __syncthreads();
    if (sm.fail && tid == 0) {   // let the copies in flight finish (bounded), then report
        dev_error(P.err, CSLD_DEVERR_TIMEOUT);
        const int n = sm.n_issued;
        for (int T = max(0, n - S::kStages); T < n; ++T) (void)mbar_wait(&sm.full[T % S::kStages], (T / S::kStages) & 1);
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
