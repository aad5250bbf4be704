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
// Where windows or capacities are short a CTA takes whole rows instead, without looking at the lengths (launch_paged_attention).
//
// Which tensor instructions.  With 16 heads one side of every product is 16 rows.  A tcgen05.mma reads its
// 128-row operand, here the entries, from shared memory at 128 B a cycle: 45 cycles for 128 x 32 x 32 (measured;
// 16 at full rate), and a version of this kernel built on it moved 326 KB through shared memory for 96 fp4
// entries (2,550 cycles at best) and took 3,000 (1M fp4 tokens 222 us).  Warp-level E4M3 mma.sync is slower still
// (62 cycles an m16n8k32 and scheduler: 538 us).  The warp-level f16 one runs at 1,013 MAC a cycle and SM (measured;
// 16.2 cycles an entry), takes the bf16 query exactly, P in one term, and 4-bit keys in registers: a code word
// becomes a B fragment without touching shared memory, and only the values take that way.
//
// A CTA's roles (20 warps; registers are moved from the copy warps to the others):
//   copy   (warp 16)    pages -> a ring of 64-entry tiles in shared memory: fp4 chunks as they lie (5,888 contiguous
//                       bytes, bulk copies), fp8 entries as five 128-byte column blocks with the 128-byte swizzle (tensor maps)
//   score  (warps 0-7)  two groups of four take the tiles in turn, so that one's softmax runs under the other's
//                       products; warp w of a group takes the tile's chunk w.  S = Q K^T, the RoPE dims by bf16 MMAs.
//                       fp4: lane (n, c) = (lane / 4, lane % 4) decodes word c of entry n's group: its 8 codes are the
//                       lane's whole share of the group's two 16-dim MMA steps, in whatever order, since the query's
//                       dims are laid out the same.  E2M1 -> E5M2 is a byte permute through 8 table bytes, 2^(13-j)
//                       times the grid, j = the entry's largest exponent minus the group's: all normal numbers, so j
//                       only subtracts 4 j from each (a group 2^-26 or less of the entry's largest is zero); E5M2 is
//                       f16's upper byte, so another permute makes the f16 pair.  An entry's decoded bytes are its values
//                       over one power of two f_e, applied to S and to P.  They also go to the value image.  fp8: the
//                       hardware's E4M3 -> f16 converts.  Then the softmax: p relative to a mark nm that is raised only
//                       when some p exceeds it by 2^10, the marks handed from tile to tile, one meeting of the
//                       four warps a tile, and P as A fragments in shared memory: in f16 (2^-11) p, fp4 p f_e 2^dm with a
//                       second mark dm that follows a head's largest p f_e, so that an entry far larger than those
//                       that carry the weight costs them nothing; for the RoPE dims p in bf16.
//   value  (warps 8-15) warp w owns 64 of the 512 dims and keeps its O in registers: O += P V, V fragments by
//                       transposing 8-bit matrix loads of the image (fp8: of the copied tile itself); the last warp the
//                       RoPE dims, bf16
// Where a query has more than 16 heads and there is work for all SMs a row is two groups of 16 (R = 2): keys are decoded
// and values loaded once for both.
//
// What bounds it (R = 1, a 64-entry tile, 512K tokens; per SM, by ncu's counters): fp4 6,100
// instructions, 1,520 a scheduler, 1,780 shared-memory wavefronts, 1,024 cycles of f16 MMAs, 975 of HBM; taken: 2,990 cycles, start-up
// included (1M tokens, merge launch included: 2,670 at the same clock).  No resource is full (issue 0.51, shared memory
// 0.61, MMAs 0.34): the time goes into latencies and hand-overs between the roles, once per 64 entries, as the stalls at barriers
// say.  1M tokens: 179 us, 2.16 TB/s, 0.33 of the copy rate.  fp8: 2,540 cycles (issue 0.45, shared memory 0.58, MMAs 0.40);
// 8 x 64K tokens 85 to 86 us, 3.5 TB/s, 0.54.  Registers spill a little (bytes stored and loaded, fp8 104 and 156, R = 2 252 and
// 292; fp4 56 and 80, R = 2 216 and 248).
// A third score group (with four value warps of 128 dims) gave 181 us where two gave 176, more or larger stages nothing.
// Rows of masked or missing tokens are zeroed before they are used, whatever was in them.  The waits for copies are
// bounded; one that gives up sets CSLD_DEVERR_TIMEOUT and all roles run out without waiting for copies.
#include <stdint.h>

#include "kernels.cuh"
#include "paged.cuh"
#include "sm100.cuh"

namespace csld {

namespace {

constexpr int kThreads = 640;
constexpr int kGroupWarps = 4, kScoreWarps = 8, kValueWarp = 8, kValueWarps = 8, kCopyWarp = 16;
// registers a thread: the launch gives 640 x 96 = 61,440; R = 1 takes 256 x 112 + 256 x 104 + 128 x 40 = 60,416 of
// them, R = 2 256 x 112 + 256 x 112 + 128 x 32 = 61,440
constexpr int kRegsScore = 112;
template <int R> constexpr int kRegsValue = R == 1 ? 104 : 112;
template <int R> constexpr int kRegsCopy = R == 1 ? 40 : 32;
constexpr int kTile = 64, kTileChunks = kTile / kChunk;   // entries per tile; a chunk per warp of a score group
static_assert(kTileChunks == kGroupWarps, "a group's warp w takes chunk w");
constexpr int kBlkBytes = kTile * 128;           // one 128-byte column block of a tile
// fp8, as copied: column blocks of dims 0..127, 128..255, 256..383, 384..447 (and half of the RoPE part), RoPE
constexpr int kTile8Bytes = 5 * kBlkBytes;
// fp4, as decoded: the same, but for rows of 64 bytes in the block of dims 384..447
constexpr int kImgBytes = 4 * kBlkBytes + kBlkBytes / 2;
template <bool kFp4> constexpr int kRopeAt = kFp4 ? 3 * kBlkBytes + kBlkBytes / 2 : 4 * kBlkBytes;
constexpr int kSteps = kGroups;                  // 32-dim steps of the 448 dims
constexpr int kQSteps = 2 * kSteps + 4;          // 16-dim MMA steps of the query, the RoPE ones last
// Marks: a head's nm is set so that the largest p of a tile is 2^kLift and kept until one exceeds 2^kOver.  The f16
// operand holds w = p (fp8), or w = p f_e 2^dm (fp4), dm a whole number per head: set so that the tile's largest w lies in
// 2^(kLiftW - 1) .. 2^kLiftW, moved against nm when that moves (w stays as it was, but for a fraction er of a bit that is
// carried along, at most 1/2), and set anew when some w exceeds 2^kOverW.  So a w of 2^-18 of the head's largest keeps
// f16's 11 bits, and no w is off by more than 2^-29 of the largest.
template <bool kFp4> constexpr float kLift = kFp4 ? 0.f : 5.f;
template <bool kFp4> constexpr float kOver = kFp4 ? 10.f : 15.f;
constexpr float kLiftW = 6.f, kOverW = 15.f, kUnset = 3e38f;   // kUnset: above any negative logit's size
constexpr int kExpBias = 127 + 13;               // f_e = 2^(exponent byte - 140): the table holds 2^13 times the grid
// hardware barriers: the score groups' own (1, 2), both groups' (3); from a group to the value warps: P of a tile is there
// (4, 5), back: its slot is free (6, 7), a value image is free (8, 9, 10); from group to group: the marks are there (11,
// 12); from the score to the value warps: a segment's sums (13), back: taken (14).  No warp can meet an earlier or a
// later use of a barrier than its own: P slots and marks keep to one group each (a group's tiles have one parity); the
// images turn among three, so that their groups alternate, but the marks of the tile between order the turns.
constexpr int kBarGroup = 1, kBarScore = 3, kBarP = 4, kBarPFree = 6, kBarImg = 8, kBarMark = 11, kBarSeg = 13, kBarSegFree = 14;
constexpr int kGroupThreads = 32 * kGroupWarps, kScoreThreads = 32 * kScoreWarps, kValueThreads = 32 * kValueWarps;
constexpr int kHandover = kGroupThreads + kValueThreads;

template <bool kFp4, int R>
struct Smem {
    static constexpr int kStages = !kFp4 && R == 1 ? 5 : 4;
    static constexpr int kStageBytes = kFp4 ? kTileChunks * kChunk4Bytes : kTile8Bytes;
    static constexpr int kImgs = kFp4 ? (R == 1 ? 3 : 2) : 1;   // what fits beside the stages
    uint8_t stage[kStages][kStageBytes];         // tiles as copied (fp8: multiples of 1024 bytes, for the tensor map's swizzle)
    uint8_t img[kImgs][kFp4 ? kImgBytes : 16];   // fp4: value images
    uint4 qf[R][kQSteps][32];                    // the query's A fragments
    uint4 p16[2][R][kTileChunks][32];            // P in f16: [chunk][lane] A fragments
    uint4 pbf[2][R][kTileChunks][32];            // bf16 P
    float fn[2][R][kHeads], fr[2][R][kHeads];    // factors of O before a tile's MMAs (448 dims; RoPE dims)
    float nm[R][kHeads], dm[R][kHeads], er[R][kHeads];   // the marks
    float tmax[2][kGroupWarps][R][kHeads], wmax[2][kGroupWarps][kFp4 ? R : 1][kHeads];
    float lsum[kScoreWarps][R][kHeads], mseg[R][kHeads], dseg[R][kHeads];   // a segment's sums and marks
    int32_t chunk_tok[kStages][kTileChunks];     // first token of a tile's chunks; -1: none
    int32_t resc[2];                             // 0: O stays, 1: O *= f, 2: O = 0 (first tile of a segment)
    uint64_t full[kStages], empty[kStages];
    int64_t red[kThreads / 32], prefix;
    int32_t fail, b0, n_issued;
};
static_assert(sizeof(Smem<true, 1>) <= 232448 && sizeof(Smem<false, 1>) <= 232448, "227 KB of shared memory");
static_assert(sizeof(Smem<true, 2>) <= 232448 && sizeof(Smem<false, 2>) <= 232448, "227 KB of shared memory");

struct Params {
    PagedView c;
    const uint16_t* q;
    void* out;
    float* lse;
    float* opart;        // [2 CTAs][a row's heads][512]
    float2* mlpart;      // [2 CTAs][a row's heads]
    int4* meta;          // [CTAs]: (row low, row high, last CTA, -) of the cut row that begins there; last CTA -1: none
    int32_t* err;
    float scale;
    int heads, rows_per_seq, row_groups, Q, W, sinks;   // row_groups: rows per query
    bool out_bf16, whole;   // whole: shares are whole rows
};

// fp8: the pages as rows of 576 bytes, by boxes of 128 bytes by 16, 32 and 64 rows.
struct PageMaps {
    CUtensorMap rows[3];
};

// Bounded wait for a copy or a ring slot: false once any such wait of the CTA has given up (this one after about a
// second).  Only these poll.  The roles hand work to one another through hardware barriers (below), where a waiting
// warp takes no issue slots: with mbarriers there too, polls were 35 % of all instructions.
template <bool kSleep>
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int32_t* fail) {
    for (uint32_t i = 0; i < (1u << 22); ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if (kSleep || i >= 16) {
            if (*fail) return false;
            __nanosleep(kSleep ? 100 : 64);
        }
    }
    *fail = 1;
    return false;
}
// Producer and consumer sides of a hardware barrier of n threads in all.  Every arrival of one use is met by exactly one
// sync, in the failure path too (a role that gives up on a copy goes on through its barriers).
__device__ __forceinline__ void bar_arrive(int id, int n) {
    __syncwarp();
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_sync(int id, int n) {
    __syncwarp();
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        :: "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar)) : "memory");
}
// Shared memory by 32-bit address.
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ int lds8(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
    return static_cast<int>(v);
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ void sts64(uint32_t a, uint32_t x, uint32_t y) {
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}
template <bool kZero>   // kZero: d is overwritten
__device__ __forceinline__ void mma_bf16_frag(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
    if constexpr (kZero)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3]) : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(0.f));
    else
        mma_bf16(d, a.x, a.y, a.z, a.w, b0, b1);
}
template <bool kZero>
__device__ __forceinline__ void mma_f16_frag(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
    if constexpr (kZero)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3]) : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
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
    int left, len;       // tiles (whole rows: rows) left in the share, this segment included; tiles of this segment
    SeqInfo s;
    __device__ __forceinline__ void begin(const Params& P, int b_, int64_t off, int n) {
        b = b_;
        s = seq_info(P, b);
        left = n;
        if (P.whole) {
            rq = static_cast<int>(off);
            t = 0;
            len = s.tiles;
            return;
        }
        rq = static_cast<int>(off / s.tiles);
        t = static_cast<int>(off % s.tiles);
        len = min(s.tiles - t, left);
    }
    __device__ __forceinline__ void next(const Params& P) {
        left -= P.whole ? 1 : len;
        t = 0;
        if (left <= 0) return;
        if (++rq == P.rows_per_seq) {
            rq = 0;
            s = seq_info(P, ++b);
        }
        len = P.whole ? s.tiles : min(s.tiles, left);
    }
    __device__ __forceinline__ int token_of_chunk(int i) const {   // i: chunk of the row's list
        return i < s.nc ? kChunk * (i < s.cs ? i : s.wl + i - s.cs) : -1;
    }
};
// ---- rows in shared memory ---------------------------------------------------------------------
// A score warp's 16 entries are two MMA column tiles of 8; entry_of: where column col of tile nt lies in the chunk.
// A row's 16-byte chunks lie at their index XOR a function of the row.  fp8: the 128-byte swizzle of the tensor map
// (row % 8); fp4: free to choose.  Both are such that the 64-bit accesses of the score warps (four rows at a time,
// a 32-byte step of each) and the transposing loads of the value warps (eight rows at a time: two columns of either
// tile, twice) meet every bank once.
template <bool kFp4>
__device__ __forceinline__ int entry_of(int nt, int col) {
    return kFp4 ? 8 * nt + col : 8 * (col >> 2) + 2 * (col & 3) + nt;
}
template <bool kFp4>
__device__ __forceinline__ int swz_wide(int r) { return kFp4 ? ((r & 3) << 1) | ((r >> 3) & 1) : r & 7; }      // 128-byte rows
__device__ __forceinline__ int swz_half(int r) { return (r & 2) | ((r >> 3) & 1); }                             // fp4: 64-byte rows
template <bool kFp4>
__device__ __forceinline__ int swz_rope(int r) { return kFp4 ? ((r & 3) << 1) | ((r >> 2) & 1) : r & 7; }

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

__device__ __forceinline__ void store_out2(const Params& P, int64_t at, float a, float b) {
    if (P.out_bf16) *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(P.out) + at) = f32x2_to_bf16x2_bits(a, b);
    else *reinterpret_cast<float2*>(reinterpret_cast<float*>(P.out) + at) = make_float2(a, b);
}

// ---- the query ---------------------------------------------------------------------------------
// A row's A fragments, by the eight score warps: each head scaled by a power of two so that its largest value lies in
// 2^7..2^8 (exact in f16 down to 2^-21 of it).  MMA step k < 28 holds of every 32 dims half (k % 2), lane (g, c) the
// dims 8c + 4 (k % 2) .. + 3 of heads g and g + 8: the order in which a lane's eight key bytes come; steps 28..31 the
// RoPE dims 16 (k - 28) + 4c .. + 3 in bf16.  Warp w builds the steps 4w .. 4w + 3.
template <int R>
struct QueryPart {
    static constexpr int kN = kQSteps / kScoreWarps;
    uint2 v[R][kN][2];   // [step][head g, g + 8]: four dims
    __device__ __forceinline__ static int dim_of(int k, int c) {
        return k < 2 * kSteps ? 32 * (k >> 1) + 8 * c + 4 * (k & 1) : kNope + 16 * (k - 2 * kSteps) + 4 * c;
    }
    __device__ __forceinline__ void load(const Params& P, int b, int rq, int warp, int g, int c) {
        const int j = rq / P.row_groups, hr = 16 * R * (rq % P.row_groups);   // the row's first head
        const uint16_t* q = P.q + (((int64_t)b * P.Q + j) * P.heads + hr) * kDim;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < kN; ++i)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int h = 16 * r + g + 8 * u;
                    v[r][i][u] = hr + h < P.heads ? __ldcg(reinterpret_cast<const uint2*>(q + h * kDim + dim_of(warp * kN + i, c)))
                                                  : make_uint2(0, 0);
                }
    }
    // largest magnitude (bf16 bits) of head g + 8 u of group r in this warp's steps
    __device__ __forceinline__ uint32_t top(int r, int u) const {
        uint32_t t = 0;
#pragma unroll
        for (int i = 0; i < kN; ++i)
            t = max(t, max(max(v[r][i][u].x & 0x7FFFu, (v[r][i][u].x >> 16) & 0x7FFFu),
                           max(v[r][i][u].y & 0x7FFFu, (v[r][i][u].y >> 16) & 0x7FFFu)));
        t = max(t, __shfl_xor_sync(0xffffffffu, t, 1));
        return max(t, __shfl_xor_sync(0xffffffffu, t, 2));
    }
    template <bool kFp4>
    __device__ __forceinline__ void store(Smem<kFp4, R>& sm, int r, const float (&sq)[2], int warp, int lane) const {
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const int k = warp * kN + i;
            uint32_t a[4];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const uint32_t w = n ? v[r][i][u].y : v[r][i][u].x;
                    const float x0 = bf16_bits_to_f32(w) * sq[u], x1 = bf16_bits_to_f32(w >> 16) * sq[u];
                    a[u + 2 * n] = k < 2 * kSteps ? f32x2_to_f16x2(x0, x1) : f32x2_to_bf16x2_bits(x0, x1);
                }
            sm.qf[r][k][lane] = make_uint4(a[0], a[1], a[2], a[3]);
        }
    }
};

// ---- score warps ---------------------------------------------------------------------------------
// S of this warp's 16 entries, fp4: decodes them (into the value image too).  kFar: some group lies more than 2^26 below
// its entry's largest, or is NaN.
template <int R, bool kFar>
__device__ __forceinline__ void score_fp4(Smem<true, R>& sm, const uint8_t* ch, uint8_t* img, int w, uint32_t vis, int g, int c, int lane,
                                          float (&acc)[R][2][2][4]) {
    // this lane's eight bytes of step s, entry r: row r, chunk 2 (s % 4) + c / 2
    uint32_t wide[2], half[2], x[4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
        const uint32_t r = 16 * w + 8 * nt + g, b = (((c >> 1) ^ nt) << 4) + 8 * (c & 1);
        wide[nt] = r * 128 + b;
        half[nt] = 3 * kBlkBytes + r * 64 + b;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = (i ^ (g & 3)) << 5;
    const uint32_t xh = ((g >> 1) & 1) << 5;
    int base[2];
    uint32_t tx[2], ty[2], dx[2], dy[2];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
        const bool see = (vis >> (8 * nt + g)) & 1;   // masked: every byte decodes to a signed zero
        base[nt] = ch[kChunk4Exp + kGroups * kChunk + 8 * nt + g];
        tx[nt] = see ? kTabX : 0u;
        ty[nt] = see ? kTabY : 0u;
        dx[nt] = see ? kTabDx : 0u;
        dy[nt] = see ? kTabDy : 0u;
    }
    // words, exponents and fragments come kPer steps at a time (as registers allow), the words a round ahead of their use
    constexpr int kPer = R == 1 ? 2 : 1;
    const uint32_t cw = smem_u32(ch) + g * 16 + 4 * c, ce = smem_u32(ch) + kChunk4Exp + g, qa = smem_u32(&sm.qf[0][0][lane]), im = smem_u32(img);
    uint32_t to[2][4], th[2];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
        for (int i = 0; i < 4; ++i) to[nt][i] = im + wide[nt] + x[i];
        th[nt] = im + half[nt] + xh;
    }
    uint32_t wd[2][kPer][2];
    int ex[2][kPer][2];
    auto fetch = [&](int rd) {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
                const int s = kPer * rd + i;
                wd[rd & 1][i][nt] = lds32(cw + s * 256 + 128 * nt);
                ex[rd & 1][i][nt] = lds8(ce + s * kChunk + 8 * nt);
            }
    };
    fetch(0);
#pragma unroll
    for (int rd = 0; rd < kSteps / kPer; ++rd) {
        uint4 a[R][2 * kPer];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int k = 0; k < 2 * kPer; ++k) a[r][k] = lds128(qa + (r * kQSteps + 2 * kPer * rd + k) * 512);
        if (rd + 1 < kSteps / kPer) fetch(rd + 1);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
                const int s = kPer * rd + i, j = base[nt] - ex[rd & 1][i][nt];
                uint2 tab = make_uint2(tx[nt] - j * dx[nt], ty[nt] - j * dy[nt]);
                if (kFar && dx[nt] && (j < 0 || j > kMaxJ)) tab.x = tab.y = j < 0 ? 0x7F7F7F7Fu : 0u;
                uint32_t b0, b1;
                decode8(wd[rd & 1][i][nt], tab, b0, b1);
                sts64(s < 12 ? to[nt][s & 3] + (s >> 2) * kBlkBytes : th[nt] ^ ((s & 1) << 5), b0, b1);
                const uint32_t f0 = bytes_to_f16x2<true, 0>(b0), f1 = bytes_to_f16x2<true, 1>(b0);
                const uint32_t f2 = bytes_to_f16x2<true, 0>(b1), f3 = bytes_to_f16x2<true, 1>(b1);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    if (s == 0) {
                        mma_f16_frag<true>(acc[r][nt][0], a[r][2 * i], f0, f1);
                        mma_f16_frag<true>(acc[r][nt][1], a[r][2 * i + 1], f2, f3);
                    } else {
                        mma_f16_frag<false>(acc[r][nt][0], a[r][2 * i], f0, f1);
                        mma_f16_frag<false>(acc[r][nt][1], a[r][2 * i + 1], f2, f3);
                    }
                }
            }
    }
}
template <int R>
__device__ __forceinline__ void score_fp8(Smem<false, R>& sm, const uint8_t* img, const uint32_t (&row)[2], const uint32_t (&x)[4], int lane,
                                          float (&acc)[R][2][2][4]) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        uint4 a[R][2];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int k = 0; k < 2; ++k) a[r][k] = sm.qf[r][2 * s + k][lane];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
            const uint2 b = *reinterpret_cast<const uint2*>(img + (s >> 2) * kBlkBytes + row[nt] + x[s & 3]);
            const uint32_t f0 = bytes_to_f16x2<false, 0>(b.x), f1 = bytes_to_f16x2<false, 1>(b.x);
            const uint32_t f2 = bytes_to_f16x2<false, 0>(b.y), f3 = bytes_to_f16x2<false, 1>(b.y);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (s == 0) {
                    mma_f16_frag<true>(acc[r][nt][0], a[r][0], f0, f1);
                    mma_f16_frag<true>(acc[r][nt][1], a[r][1], f2, f3);
                } else {
                    mma_f16_frag<false>(acc[r][nt][0], a[r][0], f0, f1);
                    mma_f16_frag<false>(acc[r][nt][1], a[r][1], f2, f3);
                }
            }
        }
    }
}

template <bool kFp4, int R>
__device__ __forceinline__ void score_role(Smem<kFp4, R>& sm, const Params& P, Walk wk, int warp, int lane, int64_t u1, int64_t n_cta,
                                           int64_t total) {
    constexpr int kS = Smem<kFp4, R>::kStages, kI = Smem<kFp4, R>::kImgs;
    volatile int32_t* fail = &sm.fail;
    const int gr = warp >> 2, w = warp & 3, g = lane >> 2, c = lane & 3;   // group gr takes the tiles T % 2 == gr
    // this lane's eight bytes of step s of a 128-byte block (RoPE; fp8: all), column g of tile nt: row[nt] + x[s % 4]
    uint32_t row[2], x32[4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
        const int e = entry_of<kFp4>(nt, g);
        row[nt] = (16 * w + e) * 128 + (((c >> 1) ^ (swz_rope<kFp4>(e) & 1)) << 4) + 8 * (c & 1);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) x32[i] = (i ^ (g & 3)) << 5;   // both tiles: the swizzle's upper bits are g % 4
    auto mine = [&](int nt, int i) { return entry_of<kFp4>(nt, 2 * c + i); };   // the columns of this lane's scores
    int T = 0, seg = 0;
    for (; wk.left > 0; wk.next(P), ++seg) {
        QueryPart<R> qp;
        qp.load(P, wk.b, wk.rq, warp, g, c);
        uint32_t top_bits[R][2];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int u = 0; u < 2; ++u) top_bits[r][u] = qp.top(r, u);
        named_barrier(kBarScore, kScoreThreads);   // the last row's fragments, marks and maxima are done with
        if (c == 0)
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int u = 0; u < 2; ++u) sm.tmax[gr][w][r][g + 8 * u] = __uint_as_float(top_bits[r][u]);
        if (warp == 0) {
            if (lane < kHeads)
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    sm.nm[r][lane] = kUnset;
                    sm.dm[r][lane] = sm.er[r][lane] = 0.f;
                }
        }
        named_barrier(kBarScore, kScoreThreads);
        float c2[R][2];   // logit factors (log2 units) of heads g, g + 8
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float sq[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                uint32_t t = 0;
#pragma unroll
                for (int i = 0; i < kScoreWarps; ++i) t = max(t, __float_as_uint(sm.tmax[i >> 2][i & 3][r][g + 8 * u]));
                const int sh = t ? min(126, 134 - static_cast<int>(t >> 7)) : 0;   // -121 .. 126: 2^sh and 2^-sh are normal numbers
                sq[u] = pow2f(sh);
                c2[r][u] = P.scale * (1.4426950408889634f * pow2f(-sh));   // the scale may be tiny where the query is large
            }
            qp.store(sm, r, sq, warp, lane);
        }
        named_barrier(kBarScore, kScoreThreads);
        const int p = wk.s.n - P.Q + wk.rq / P.row_groups;   // the query's position; it sees t <= p, t > lo or t < sinks
        const int lo = P.W > 0 ? max(p, 0) - P.W : -1;
        float nm[R][2], l[R][2];   // heads g, g + 8; l is relative to nm
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                nm[r][k] = kUnset;
                l[r][k] = 0.f;
            }
        const int T0 = T, T1 = T + wk.len;
        for (T += (T ^ gr) & 1; T < T1; T += 2) {
            const int st = T % kS, buf = T & 1, im = T % kI;
            const bool ok = __all_sync(0xffffffffu, wait<false>(&sm.full[st], (T / kS) & 1, fail));
            if (kFp4 && T >= kI) bar_sync(kBarImg + im, kHandover);
            const int tok0 = ok ? sm.chunk_tok[st][w] : -1, tk = tok0 + (lane & 15);
            const uint32_t vis = __ballot_sync(0xffffffffu, tok0 >= 0 && tk <= p && (tk > lo || tk < P.sinks)) & 0xFFFFu;
            float acc[R][2][2][4], racc[R][2][4];   // [entries 8 nt ..][half of a step: independent chains]; RoPE part
            uint8_t* img = kFp4 ? sm.img[im] : sm.stage[st];
            uint32_t eb = 0;   // fp4: the exponent bytes of the entries mine(nt, i), entry 2 nt + i in byte 2 nt + i
            auto byte_of = [&](int nt, int i) { return (eb >> (8 * (2 * nt + i))) & 0xFFu; };
            auto seen = [&](int nt, int i) { return (vis >> mine(nt, i)) & 1; };
            if constexpr (kFp4) {
                const uint8_t* ch = sm.stage[st] + w * kChunk4Bytes;
                // RoPE rows into the image, eight lanes a row
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int en = 4 * i + (lane >> 3), k = lane & 7;
                    uint4 v = *reinterpret_cast<const uint4*>(ch + kChunk4Rope + en * 2 * kRope + 16 * k);
                    if (!((vis >> en) & 1)) v = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4*>(img + kRopeAt<kFp4> + (16 * w + en) * 128 + ((k ^ swz_rope<kFp4>(en)) << 4)) = v;
                }
                // groups whose scale lies far below the entry's largest (zero there), or NaN groups (byte 255).  Lane (g, c) looks
                // at the groups c, c + 4, .. of entries g and 8 + g
                uint32_t most = 0;
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    const int base = ch[kChunk4Exp + kGroups * kChunk + 8 * nt + g];
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        if (4 * s + c < kSteps && (vis >> (8 * nt + g)) & 1)
                            most = max(most, static_cast<uint32_t>(base - ch[kChunk4Exp + (4 * s + c) * kChunk + 8 * nt + g]));
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        eb |= static_cast<uint32_t>(ch[kChunk4Exp + kGroups * kChunk + mine(nt, i)]) << (8 * (2 * nt + i));
                }
                if (__any_sync(0xffffffffu, most > static_cast<uint32_t>(kMaxJ))) score_fp4<R, true>(sm, ch, img, w, vis, g, c, lane, acc);
                else score_fp4<R, false>(sm, ch, img, w, vis, g, c, lane, acc);
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.empty[st]);
            } else {
                if (vis != 0xFFFFu) {   // masked rows are zeroed for the value warps, eight lanes a row (unrolled, the full tiles lose 2 %)
#pragma unroll 1
                    for (int en = lane >> 3; en < 16; en += 4)
                        if (!((vis >> en) & 1))
#pragma unroll
                            for (int k = 0; k < 5; ++k)
                                *reinterpret_cast<uint4*>(img + k * kBlkBytes + sw128(16 * w + en, 16 * (lane & 7))) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();   // the ring's next copy writes there too
                    __syncwarp();
                }
                score_fp8<R>(sm, img, row, x32, lane, acc);
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                uint4 a[R];
#pragma unroll
                for (int r = 0; r < R; ++r) a[r] = sm.qf[r][2 * kSteps + s][lane];
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    const uint2 b = *reinterpret_cast<const uint2*>(img + kRopeAt<kFp4> + row[nt] + x32[s]);
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        if (s == 0) mma_bf16_frag<true>(racc[r][nt], a[r], b.x, b.y);
                        else mma_bf16_frag<false>(racc[r][nt], a[r], b.x, b.y);
                    }
                }
            }
            // logits x[r][nt][2 k + i]: entry mine(nt, i), head g + 8 k (log2 units), -inf where masked
            float (&x)[R][2][4] = racc;
            float top[R][2];
            // fp4: f_e and its log2 (of masked entries -inf)
            auto fe = [&](int nt, int i) { return __uint_as_float(byte_of(nt, i) << 23) * 0x1p-13f; };
            float lfe[2][2], lmost = -INFINITY;
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    lfe[nt][i] = !kFp4 ? 0.f : seen(nt, i) ? __uint_as_float(0x4B000000u | byte_of(nt, i)) - (0x1p23f + kExpBias) : -INFINITY;
                    lmost = fmaxf(lmost, lfe[nt][i]);
                }
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    top[r][k] = -INFINITY;
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int n = 2 * k + i;
                            const float sum = acc[r][nt][0][n] + acc[r][nt][1][n];
                            const float v = kFp4 ? fmaf(sum, fe(nt, i), racc[r][nt][n]) : sum + racc[r][nt][n];
                            x[r][nt][n] = seen(nt, i) ? v * c2[r][k] : -INFINITY;
                            top[r][k] = fmaxf(top[r][k], x[r][nt][n]);
                        }
                }
            // the marks, as the tile before left them; the slot of P (and of the factors) is free once its last tile is used
            if (T > T0) bar_sync(kBarMark + ((T - 1) & 1), kScoreThreads);
            if (T >= 2) bar_sync(kBarPFree + buf, kHandover);
            float mk[R][2], dm[R][2];
            bool over = false;
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    mk[r][k] = sm.nm[r][g + 8 * k];
                    dm[r][k] = kFp4 ? sm.dm[r][g + 8 * k] : 0.f;
                    over |= top[r][k] + mk[r][k] > kOver<kFp4>;
                    if (kFp4) over |= (top[r][k] + mk[r][k]) + (lmost + dm[r][k]) > kOverW;   // at least any w of the lane's
                }
            int resc = T == T0 ? 2 : 0;
            if (named_barrier_or(kBarGroup + gr, kGroupThreads, over)) {
                // some weight may be too large, or the first tile: the tile's maxima (fp4: of p f_e as well, relative to the warp's
                // largest p, so that no logit is rounded by adding to it); a head that lies more than 2 above its mark gets a new
                // one, and the value warps the factors of what they hold
                float er[R][2];
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        er[r][k] = kFp4 ? sm.er[r][g + 8 * k] : 0.f;
                        top[r][k] = fmaxf(top[r][k], __shfl_xor_sync(0xffffffffu, top[r][k], 1));
                        top[r][k] = fmaxf(top[r][k], __shfl_xor_sync(0xffffffffu, top[r][k], 2));
                        if (c == 0) sm.tmax[gr][w][r][g + 8 * k] = top[r][k];
                        if constexpr (kFp4) {
                            float wt = -INFINITY;
#pragma unroll
                            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                                for (int i = 0; i < 2; ++i)
                                    if (top[r][k] > -INFINITY) wt = fmaxf(wt, (x[r][nt][2 * k + i] - top[r][k]) + lfe[nt][i]);
                            wt = fmaxf(wt, __shfl_xor_sync(0xffffffffu, wt, 1));
                            wt = fmaxf(wt, __shfl_xor_sync(0xffffffffu, wt, 2));
                            if (c == 0) sm.wmax[gr][w][r][g + 8 * k] = wt;
                        }
                    }
                named_barrier(kBarGroup + gr, kGroupThreads);
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float tm = sm.tmax[gr][0][r][g + 8 * k];
#pragma unroll
                        for (int i = 1; i < kGroupWarps; ++i) tm = fmaxf(tm, sm.tmax[gr][i][r][g + 8 * k]);
                        const bool first = mk[r][k] == kUnset;
                        const bool set = first ? tm > -INFINITY : tm + mk[r][k] > kLift<kFp4> + 2.f;
                        const float to = set ? kLift<kFp4> - tm : mk[r][k];
                        const float down = set && !first ? to - mk[r][k] : 0.f, f = exp2_ftz(down);
                        float fw = f;
                        if constexpr (kFp4) {
                            const float turn = rintf(down + er[r][k]);
                            float wt = -INFINITY, d = dm[r][k] - turn;
                            er[r][k] = (down + er[r][k]) - turn;
#pragma unroll
                            for (int i = 0; i < kGroupWarps; ++i)
                                wt = fmaxf(wt, sm.wmax[gr][i][r][g + 8 * k] + (sm.tmax[gr][i][r][g + 8 * k] + to));
                            if (first ? set : wt + d > kLiftW + 2.f) {
                                d = floorf(kLiftW - wt);
                                er[r][k] = 0.f;
                            }
                            fw = first ? 1.f : exp2_ftz(down + (d - dm[r][k]));
                            dm[r][k] = d;
                        }
                        mk[r][k] = to;
                        if (w == 0 && c == 0) {
                            sm.fn[buf][r][g + 8 * k] = fw;
                            sm.fr[buf][r][g + 8 * k] = f;
                            sm.nm[r][g + 8 * k] = to;
                            if (kFp4) {
                                sm.dm[r][g + 8 * k] = dm[r][k];
                                sm.er[r][g + 8 * k] = er[r][k];
                            }
                        }
                    }
                if (T > T0) resc = 1;
            }
            bar_arrive(kBarMark + buf, kScoreThreads);
            // P: p = 2^(x + nm), as A fragments: the lane's columns 2c + i are the MMA's k slots 2c + i (nt = 0) and 2c + 8 + i
#pragma unroll
            for (int r = 0; r < R; ++r) {
                uint32_t pb[2][2], ph[2][2];   // [head][nt]
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if (mk[r][k] != nm[r][k]) {   // the mark moved, in this tile or in the other group's
                        l[r][k] *= exp2_ftz(mk[r][k] - nm[r][k]);
                        nm[r][k] = mk[r][k];
                    }
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) {
                        const float y0 = x[r][nt][2 * k] + nm[r][k], y1 = x[r][nt][2 * k + 1] + nm[r][k];
                        const float p0 = exp2_ftz(y0), p1 = exp2_ftz(y1);
                        l[r][k] += p0 + p1;
                        pb[k][nt] = f32x2_to_bf16x2_bits(p0, p1);
                        // fp4: a second exponential (whole numbers added to y), since p may vanish where p f_e does not
                        ph[k][nt] = kFp4 ? f32x2_to_f16x2(exp2_ftz(y0 + (lfe[nt][0] + dm[r][k])), exp2_ftz(y1 + (lfe[nt][1] + dm[r][k])))
                                         : f32x2_to_f16x2(p0, p1);
                    }
                }
                sm.p16[buf][r][w][lane] = make_uint4(ph[0][0], ph[1][0], ph[0][1], ph[1][1]);
                sm.pbf[buf][r][w][lane] = make_uint4(pb[0][0], pb[1][0], pb[0][1], pb[1][1]);
            }
            if (w == 0 && lane == 0) sm.resc[buf] = resc;
            bar_arrive(kBarP + buf, kHandover);
        }
        T = T1;
        // ---- the segment's sums, relative to the last marks --------------------------------------------
        // The group of the last tile has the marks in registers: its warps have not met since warp 0 of it may have stored them.
        const bool last_own = ((T1 - 1) & 1) == gr;
        if (!last_own) bar_sync(kBarMark + ((T1 - 1) & 1), kScoreThreads);
        if (seg >= 1) bar_sync(kBarSegFree, kScoreThreads + kValueThreads);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float mk = last_own ? nm[r][k] : sm.nm[r][g + 8 * k];
                float v = mk != nm[r][k] ? l[r][k] * exp2_ftz(mk - nm[r][k]) : l[r][k];
                v += __shfl_xor_sync(0xffffffffu, v, 1);
                v += __shfl_xor_sync(0xffffffffu, v, 2);
                if (c == 0) {
                    sm.lsum[warp][r][g + 8 * k] = v;
                    if (warp == 0) {   // dm: stored by this thread itself, or the other group's, which it waited for
                        sm.mseg[r][g + 8 * k] = -mk;
                        sm.dseg[r][g + 8 * k] = sm.dm[r][g + 8 * k];
                    }
                }
            }
        if (warp == 0 && lane == 0) {
            if (wk.t == 0 && wk.len < wk.s.tiles) {   // a cut row begins here: which CTA holds its end
                const int64_t row = (int64_t)wk.b * P.rows_per_seq + wk.rq;
                const int64_t end = u1 - wk.left + wk.s.tiles;    // unit behind the row
                int64_t e = (end - 1) * n_cta / total;
                while (total * (e + 1) / n_cta <= end - 1) ++e;
                while (total * e / n_cta > end - 1) --e;
                P.meta[blockIdx.x] = make_int4(static_cast<int>(row), static_cast<int>(row >> 32), static_cast<int>(e), 0);
            }
        }
        bar_arrive(kBarSeg, kScoreThreads + kValueThreads);
    }
}

// ---- value warps ---------------------------------------------------------------------------------
template <bool kFp4, int R>
__device__ __forceinline__ void value_role(Smem<kFp4, R>& sm, const Params& P, Walk wk, int w, int lane) {
    constexpr int kS = Smem<kFp4, R>::kStages, kI = Smem<kFp4, R>::kImgs;
    volatile int32_t* fail = &sm.fail;
    const int g = lane >> 2, c = lane & 3;
    const bool rope = w == kValueWarps - 1;
    // this lane's row of the matrix loads, within a 32-entry block (448 dims) or a 16-entry chunk (RoPE); the 16-byte
    // column that it starts from and its swizzle; bytes from one block or chunk of entries to the next
    uint32_t off, col, swz, step;
    if (!rope) {
        const int k = lane & 15, i = k & 3;   // row k of a transposing load: column 2 (k / 4) + i % 2 of tile i / 2
        const int e = entry_of<kFp4>(i >> 1, 2 * (k >> 2) + (i & 1)), r = 16 * (lane >> 4) + e;
        const bool half = kFp4 && w == 6;
        off = (w >> 1) * kBlkBytes + r * (half ? 64 : 128);
        col = half ? 0 : 4 * (w & 1);
        swz = half ? swz_half(e) : swz_wide<kFp4>(e);
        step = half ? 2048 : 4096;
    } else {
        const int e = entry_of<kFp4>((lane >> 3) & 1, lane & 7);
        off = kRopeAt<kFp4> + e * 128;
        col = lane >> 4;
        swz = swz_rope<kFp4>(e);
        step = 2048;
    }
    uint32_t at[4];   // by q
#pragma unroll
    for (int q = 0; q < 4; ++q) at[q] = off + (((col + (rope ? 2 : 1) * q) ^ swz) << 4);
    float o[R][8][4];
    int T = 0;
    for (; wk.left > 0; wk.next(P)) {
        for (int t = 0; t < wk.len; ++t, ++T) {
            const int buf = T & 1, st = T % kS;
            bar_sync(kBarP + buf, kHandover);
            if (!kFp4) (void)wait<false>(&sm.full[st], (T / kS) & 1, fail);   // complete by now: makes the copy visible here
            const bool ok = __all_sync(0xffffffffu, !*fail);
            const int resc = sm.resc[buf];
            if (resc == 2) {
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int q = 0; q < 8; ++q)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[r][q][i] = 0.f;
            } else if (resc == 1) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float* f = rope ? sm.fr[buf][r] : sm.fn[buf][r];
                    const float f0 = f[g], f1 = f[g + 8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        o[r][q][0] *= f0;
                        o[r][q][1] *= f0;
                        o[r][q][2] *= f1;
                        o[r][q][3] *= f1;
                    }
                }
            }
            if (ok) {
                const uint32_t tile = smem_u32(kFp4 ? sm.img[T % kI] : sm.stage[st]);
                if (!rope) {
#pragma unroll
                    for (int kb = 0; kb < kTile / 32; ++kb) {
                        uint4 a[R][2];
#pragma unroll
                        for (int r = 0; r < R; ++r)
#pragma unroll
                            for (int u = 0; u < 2; ++u) a[r][u] = sm.p16[buf][r][2 * kb + u][lane];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t v[4];   // dims 16 q + lane / 4 (+ 8: odd), chunk 2 kb (+ 1: v[2], v[3])
                            ldmatrix_b8_trans_x2(v, tile + at[q] + kb * step);
#pragma unroll
                            for (int u = 0; u < 2; ++u)
#pragma unroll
                                for (int n = 0; n < 2; ++n) {
                                    const uint32_t b0 = bytes_to_f16x2<kFp4, 0>(v[2 * u + n]), b1 = bytes_to_f16x2<kFp4, 1>(v[2 * u + n]);
#pragma unroll
                                    for (int r = 0; r < R; ++r) mma_f16_frag<false>(o[r][2 * q + n], a[r][u], b0, b1);
                                }
                        }
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < kTileChunks; ++k) {
                        uint4 a[R];
#pragma unroll
                        for (int r = 0; r < R; ++r) a[r] = sm.pbf[buf][r][k][lane];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t v[4];
                            ldmatrix_b16_trans_x4(v, tile + at[q] + k * step);
#pragma unroll
                            for (int r = 0; r < R; ++r) {
                                mma_bf16_frag<false>(o[r][2 * q], a[r], v[0], v[1]);
                                mma_bf16_frag<false>(o[r][2 * q + 1], a[r], v[2], v[3]);
                            }
                        }
                    }
                }
            }
            bar_arrive(kBarPFree + buf, kHandover);
            if (kFp4) bar_arrive(kBarImg + T % kI, kHandover);
            else if (lane == 0) mbar_arrive(&sm.empty[st]);
        }
        // ---- the segment's result ------------------------------------------------------------------
        bar_sync(kBarSeg, kScoreThreads + kValueThreads);
        const bool whole = wk.t == 0 && wk.len == wk.s.tiles;
        const int j = wk.rq / P.row_groups, h0 = 16 * R * (wk.rq % P.row_groups) + g;
        const int64_t head = ((int64_t)wk.b * P.Q + j) * P.heads + h0;
        const int64_t slot = 2 * (int64_t)blockIdx.x + (wk.t == 0 ? 1 : 0);
        if (__all_sync(0xffffffffu, !*fail)) {
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int h = 16 * r + 8 * k;   // from this lane's first head
                    float L = 0.f;
#pragma unroll
                    for (int i = 0; i < kScoreWarps; ++i) L += sm.lsum[i][r][g + 8 * k];
                    // 2^-dm in two factors: it may lie below fp32's normal range, and the product not
                    const int dm = kFp4 && !rope ? static_cast<int>(sm.dseg[r][g + 8 * k]) : 0, half = dm >> 1;
                    const float M = sm.mseg[r][g + 8 * k], f0 = pow2f(-half), f1 = pow2f(half - dm);
                    const float f = whole ? (L == 0.f ? 0.f : f1 / L) : f1;
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const int d = 64 * w + 8 * q + 2 * c;
                        const float v0 = o[r][q][2 * k] * f0 * f, v1 = o[r][q][2 * k + 1] * f0 * f;
                        if (!whole) *reinterpret_cast<float2*>(P.opart + (slot * R * kHeads + g + h) * kDim + d) = make_float2(v0, v1);
                        else if (h0 + h < P.heads) store_out2(P, (head + h) * kDim + d, v0, v1);
                    }
                    if (w == 0 && c == 0) {
                        if (!whole) P.mlpart[slot * R * kHeads + g + h] = make_float2(M, L);
                        else if (P.lse && h0 + h < P.heads)
                            P.lse[head + h] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
                    }
                }
        }
        bar_arrive(kBarSegFree, kScoreThreads + kValueThreads);
    }
}

// ---- copy warp -------------------------------------------------------------------------------------
template <bool kFp4, int R>
__device__ __forceinline__ void copy_role(Smem<kFp4, R>& sm, const Params& P, Walk wk, int lane, const PageMaps& maps) {
    constexpr int kS = Smem<kFp4, R>::kStages;
    volatile int32_t* fail = &sm.fail;
    int T = 0;
    for (; wk.left > 0; wk.next(P)) {
        if (lane == 0) {
            const int32_t n = P.c.seq_len[wk.b];
            if (n < 0 || n > P.c.capacity()) dev_error(P.err, CSLD_DEVERR_SEQ_LEN);
        }
        // pages come for kAhead tiles at a time (lane 4 t + i: chunk i of the t-th), the next ones while these are copied
        constexpr int kAhead = 32 / kTileChunks;
        auto look = [&](int t, int& tok, int32_t& pg) {
            tok = wk.token_of_chunk((wk.t + t) * kTileChunks + lane);
            pg = tok >= 0 ? __ldg(P.c.table + (int64_t)wk.b * P.c.max_pages + tok / P.c.page_size) : -1;
        };
        int tok_v, tok_n;
        int32_t pg_v, pg_n;
        look(0, tok_n, pg_n);
        for (int t0 = 0; t0 < wk.len; t0 += kAhead) {
            tok_v = tok_n;
            pg_v = pg_n;
            if (t0 + kAhead < wk.len) look(t0 + kAhead, tok_n, pg_n);
            if (tok_v >= 0 && (pg_v < 0 || pg_v >= P.c.n_pages)) {
                if (lane < kTileChunks * (wk.len - t0)) dev_error(P.err, CSLD_DEVERR_PAGE);
                tok_v = -1;
            }
            const int row_v = tok_v >= 0 ? pg_v * P.c.page_size + tok_v % P.c.page_size : 0;   // at most 2^31 - 1 rows
            const int n_t = min(kAhead, wk.len - t0);
            for (int t = 0; t < n_t; ++t, ++T) {
                const int st = T % kS;
                bool ok = !*fail;
                if (T >= kS) ok = ok && wait<true>(&sm.empty[st], (T / kS - 1) & 1, fail);
                if (!__all_sync(0xffffffffu, ok)) return;
                // fp4: lane i < 4 copies chunk i; fp8: lane 5 i + k column block k of chunk i (a box of 16 rows by 128 bytes)
                const int ck = kFp4 ? lane : lane / 5, blk = lane % 5, from = kTileChunks * t + min(ck, kTileChunks - 1);
                const int tok = __shfl_sync(0xffffffffu, tok_v, from), row = __shfl_sync(0xffffffffu, row_v, from);
                const bool mine = ck < kTileChunks && tok >= 0;
                // fp8: chunks whose rows follow one another go in one request, made by the first of them, all four or in pairs (a
                // request costs this warp about 110 cycles; 20 boxes a tile held 8 x 64K tokens at 88 us, five give 85)
                int span = 1;
                if constexpr (!kFp4) {
                    const int i = min(ck, kTileChunks - 1), at = kTileChunks * t;
                    const int tok_p = __shfl_sync(0xffffffffu, tok_v, at + (i ^ 1)), row_p = __shfl_sync(0xffffffffu, row_v, at + (i ^ 1));
                    const int row_q = __shfl_sync(0xffffffffu, row_v, at + (i ^ 2));
                    const bool pair = tok >= 0 && tok_p >= 0 && row_p - row == (i & 1 ? -kChunk : kChunk);
                    const bool quad = __all_sync(0xffffffffu, pair && row_q - row == (i & 2 ? -2 * kChunk : 2 * kChunk));
                    span = quad ? 4 : pair ? 2 : 1;
                }
                if (ck < kTileChunks && (kFp4 || blk == 0)) sm.chunk_tok[st][ck] = tok;
                const int n = __popc(__ballot_sync(0xffffffffu, mine));
                __syncwarp();   // orders the lanes' chunk_tok before lane 0's arrive, which is all there is for a tile without chunks
                if (lane == 0) {
                    sm.n_issued = T + 1;
                    mbar_arrive_expect_tx(&sm.full[st], n * (kFp4 ? kChunk4Bytes : kChunk * 128));
                }
                __syncwarp();
                if (mine) {
                    if constexpr (kFp4)
                        bulk_g2s(sm.stage[st] + ck * kChunk4Bytes, P.c.pages + (int64_t)row * kEntry4, kChunk4Bytes, &sm.full[st]);
                    else if ((ck & (span - 1)) == 0)
                        tma_load_2d(sm.stage[st] + blk * kBlkBytes + ck * kChunk * 128, &maps.rows[span >> 1], blk < 4 ? 128 * blk : kNope, row,
                                    &sm.full[st]);
                }
            }
        }
    }
}

}  // namespace

template <bool kFp4, int R>
__global__ void __launch_bounds__(kThreads, 1) paged_attention_kernel(const __grid_constant__ PageMaps maps,
                                                                      const __grid_constant__ Params P) {
    using S = Smem<kFp4, R>;
    constexpr int kS = Smem<kFp4, R>::kStages;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    S& sm = *reinterpret_cast<S*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    // ---- setup --------------------------------------------------------------------------------
    if (tid == 0) {
        for (int s = 0; s < kS; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], kFp4 ? kGroupWarps : kValueWarps);
        }
        sm.fail = 0;
        sm.n_issued = 0;
        fence_barrier_init();
    }
    if (!kFp4 && warp == kCopyWarp && lane < 3) tma_prefetch_map(&maps.rows[lane]);
    pdl_wait();
    pdl_trigger();

    // ---- this CTA's share -------------------------------------------------------------------------
    const int rows_per_seq = P.rows_per_seq;
    int64_t total = 0, n_cta = gridDim.x, u1 = 0, first = 0;   // of split rows: all tiles, CTAs with a share, its end; its begin
    int b0, n_units;
    if (P.whole) {
        const int64_t rows = (int64_t)P.c.batch * rows_per_seq, r0 = rows * blockIdx.x / n_cta;
        n_units = static_cast<int>(rows * (blockIdx.x + 1) / n_cta - r0);
        b0 = static_cast<int>(r0 / rows_per_seq);
        first = r0 % rows_per_seq;
        __syncthreads();
    } else {
        int64_t mine = 0;
        for (int b = tid; b < P.c.batch; b += kThreads) mine += seq_info(P, b).tiles;
        auto block_scan = [&](int64_t v, int64_t& sum) {   // exclusive prefix of v over the threads
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
            sum = 0;
            for (int w = 0; w < kThreads / 32; ++w) {
                if (w < warp) before += sm.red[w];
                sum += sm.red[w];
            }
            return before + inc - v;
        };
        int64_t all;
        const int64_t pre = block_scan(mine, all);
        total = all * rows_per_seq;
        n_cta = min64(n_cta, total);
        const int64_t u0 = blockIdx.x < n_cta ? total * blockIdx.x / n_cta : 0;
        u1 = blockIdx.x < n_cta ? total * (blockIdx.x + 1) / n_cta : 0;
        n_units = static_cast<int>(u1 - u0);
        if (n_units > 0) {   // the sequence that the share begins in
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
        b0 = sm.b0;
        first = u0 - sm.prefix;
    }
    if (n_units > 0) {
        Walk wk;
        wk.begin(P, b0, first, n_units);
        if (warp < kScoreWarps) {
            regs_inc<kRegsScore>();
            score_role<kFp4, R>(sm, P, wk, warp, lane, u1, n_cta, total);
        } else if (warp < kValueWarp + kValueWarps) {
            regs_inc<kRegsValue<R>>();
            value_role<kFp4, R>(sm, P, wk, warp - kValueWarp, lane);
        } else {
            regs_dec<kRegsCopy<R>>();
            if (warp == kCopyWarp) copy_role<kFp4, R>(sm, P, wk, lane, maps);
        }
    }
    __syncthreads();
    if (sm.fail && tid == 0) {   // let the copies in flight finish (bounded), then report
        dev_error(P.err, CSLD_DEVERR_TIMEOUT);
        const int n = sm.n_issued;
        for (int T = max(0, n - kS); T < n; ++T) (void)mbar_wait(&sm.full[T % kS], (T / kS) & 1);
    }
}

// Joins the CTAs' parts of the cut rows: block (y, h) takes the y-th cut row, head h.  512 threads: thread t owns
// dims 4 (t % 128) .. + 3 of every fourth part from t / 128 on.
constexpr int kMergeThreads = 512, kMergeU = 8;
__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(const __grid_constant__ Params P, int n_cta) {
    __shared__ float4 red[3][kDim / 4];
    __shared__ float2 mls[1024];
    __shared__ int cnt[kMergeThreads / 32], found;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, h = blockIdx.x, n_heads = gridDim.x;   // heads of a row
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
    const int64_t step = (int64_t)n_heads * (kDim / 4);
    float4 v[kMergeU];
#pragma unroll
    for (int u = 0; u < kMergeU; ++u) {
        const int i = g + 4 * u;
        v[u] = i < n ? __ldcg(ob + slot(i) * step) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int i = tid; i < n; i += kMergeThreads) mls[i] = __ldcg(&P.mlpart[slot(i) * n_heads + h]);
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
    for (int i = g + 4 * kMergeU; i < n; i += 4) add(i, __ldcg(ob + slot(i) * step));
    if (g > 0) red[g - 1][d4] = acc;
    __syncthreads();
    const int64_t row = (static_cast<int64_t>(mt.y) << 32) | static_cast<uint32_t>(mt.x);
    const int rq = static_cast<int>(row % P.rows_per_seq), hh = n_heads * (rq % P.row_groups) + h;
    if (g != 0 || hh >= P.heads) return;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        acc.x += red[k][d4].x;
        acc.y += red[k][d4].y;
        acc.z += red[k][d4].z;
        acc.w += red[k][d4].w;
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const int64_t at = (row / P.rows_per_seq * P.Q + rq / P.row_groups) * P.heads + hh;
    if (P.out_bf16)
        reinterpret_cast<uint2*>(P.out)[at * (kDim / 4) + d4] =
            make_uint2(f32x2_to_bf16x2_bits(acc.x * inv, acc.y * inv), f32x2_to_bf16x2_bits(acc.z * inv, acc.w * inv));
    else
        reinterpret_cast<float4*>(P.out)[at * (kDim / 4) + d4] = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    if (P.lse && tid == 0) P.lse[at] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
}

namespace {
constexpr int kMaxR = 2;
constexpr int kMergeTiles = 4;   // what cutting rows costs at the least, in tiles of a CTA's time: the scan of lengths and the merge launch
constexpr size_t kPartBytes = 2 * kMaxR * kHeads * (kDim * sizeof(float) + sizeof(float2)) + sizeof(int4);   // per CTA

template <bool kFp4, int R>
cudaError_t launch_rows(const PageMaps& maps, const Params& P, int n_cta, cudaStream_t stream) {
    cudaError_t e = set_smem_once(paged_attention_kernel<kFp4, R>, sizeof(Smem<kFp4, R>));
    if (e != cudaSuccess) return e;
    return launch_pdl(paged_attention_kernel<kFp4, R>, dim3(n_cta), dim3(kThreads), sizeof(Smem<kFp4, R>), stream, maps, P);
}
}  // namespace

size_t paged_attention_ws_bytes(int num_sms) { return num_sms * kPartBytes; }

cudaError_t launch_paged_attention(const PagedView& c, bool fp4, const uint16_t* q, int heads, int Q, int W, int sinks,
                                   float scale, void* out, bool out_bf16, float* lse_out, void* ws, int num_sms,
                                   int32_t* err, cudaStream_t stream) {
    // The longest row has t tiles, as far as the host knows (the window, or the capacity).
    int64_t chunks = (c.capacity() + kChunk - 1) / kChunk;
    if (W > 0) chunks = min64(chunks, (min64(sinks, c.capacity()) + kChunk - 1) / kChunk + (min64(W, c.capacity()) + Q - 1 + 2 * kChunk - 2) / kChunk);
    const int64_t t = (chunks + kTileChunks - 1) / kTileChunks;
    // Two 16-head groups a row save decoding where the groups are even in number and there is work for all SMs: 4 x 64K tokens with
    // 64 heads, 55 tiles a CTA: fp4 175 -> 163 us, fp8 150 -> 127; 16 windows of 6,144 with 64 heads, 21 tiles: fp4 85.2 -> 82.7, fp8
    // 74.7 -> 69.0; of 4,096, 14 tiles: 66.0 -> 66.7, 58.3 -> 56.8; with 32 heads, 7 tiles: 39.9 -> 44.8, 35.6 -> 38.7.  Of three groups
    // the second row is half empty: 20 windows of 8,192 with 48 heads, 34 tiles: fp4 99 -> 115, fp8 90 -> 102.  Short sequences in a
    // table for long ones take R = 2 too, and lose these few percent.
    const int groups = (heads + kHeads - 1) / kHeads;
    const int R = groups % 2 == 0 && (int64_t)c.batch * Q * (groups / 2) * t >= 14 * num_sms ? 2 : 1;
    Params P;
    P.c = c;
    P.q = q;
    P.out = out;
    P.lse = lse_out;
    P.opart = static_cast<float*>(ws);
    P.mlpart = reinterpret_cast<float2*>(P.opart + (size_t)num_sms * 2 * kMaxR * kHeads * kDim);
    P.meta = reinterpret_cast<int4*>(P.mlpart + (size_t)num_sms * 2 * kMaxR * kHeads);
    P.err = err;
    P.scale = scale;
    P.heads = heads;
    P.row_groups = (heads + R * kHeads - 1) / (R * kHeads);
    P.rows_per_seq = Q * P.row_groups;
    P.Q = Q;
    P.W = W;
    P.sinks = sinks;
    P.out_bf16 = out_bf16;
    PageMaps maps = {};
    for (int i = 0; !fp4 && i < 3; ++i)
        if (!make_tensor_map_2d_u8(&maps.rows[i], c.pages, kEntry, (uint64_t)c.n_pages * c.page_size, 128, kChunk << i))
            return cudaErrorInvalidValue;
    // Whole rows a CTA, or rows cut into even shares.  Cutting costs the scan and the merge launch, 9 to 10 us (148 windows of 768
    // tokens, one row a CTA: fp8 25.2 -> 34.0 us, fp4 26.4 -> 36.0; of 4,096: fp8 95 -> 105; 64 of 128: 11.0 -> 28.4), and pays
    // where rows do not divide well, or are of unlike lengths, which the host does not know: whole rows are bounded by how far
    // the longest may exceed the shares.  A window is mostly full, and whole rows stay up to 64 tiles a CTA, where cutting costs
    // a tenth.  A capacity says little of the lengths: up to 8 tiles, as much again as cutting costs (148 sequences
    // of up to 128K tokens, log-uniform: whole 2,784 us, cut 722; 37 x 4 queries 2,715 and 911; 140 of up to 4,096: 91.5 and 61.9).
    const int64_t rows = (int64_t)c.batch * P.rows_per_seq, n_cta = min64(num_sms, rows), per = (rows + n_cta - 1) / n_cta;
    P.whole = per * t <= rows * t / num_sms + kMergeTiles && per * (t - 1) <= (W > 0 ? 64 : 2 * kMergeTiles);
    cudaError_t e = fp4 ? (R == 2 ? launch_rows<true, 2>(maps, P, P.whole ? n_cta : num_sms, stream)
                                  : launch_rows<true, 1>(maps, P, P.whole ? n_cta : num_sms, stream))
                        : (R == 2 ? launch_rows<false, 2>(maps, P, P.whole ? n_cta : num_sms, stream)
                                  : launch_rows<false, 1>(maps, P, P.whole ? n_cta : num_sms, stream));
    if (e != cudaSuccess) return e;
    if (P.whole) return cudaGetLastError();
    const int64_t most = rows < num_sms - 1 ? rows : num_sms - 1;
    e = launch_pdl(paged_merge_kernel, dim3(R * kHeads, static_cast<unsigned>(most)), dim3(kMergeThreads), 0, stream, P, num_sms);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace csld
