// paged_attend.cu -- attention over pages for few query rows a sequence (single tokens, drafts
// of a few tokens):
//     o_r = sum_t softmax_t(scale * <q_r, K_t>) V_t,   rows r = (token, head of the group).
//
// With a handful of rows the call is a stream over the K and V rows (512 bytes a token and KV
// head in bf16, 258 in 8 bits), bound by HBM; the aim is to read each of them once, to keep enough
// copies under way, and to spend few instructions a token:
//  - all rows of a tile (up to 8 or 16: tokens x heads of the KV head's group) share one pass
//    over K and V;
//  - the (head, sequence) streams of a batch form one axis of 64- or 128-token blocks that is cut
//    into equal ranges, two CTAs an SM, so ragged lengths leave no SM idle (see Plan). A block has
//    128 tokens in 8 bits: what a block costs besides its bytes (the loading warp's walk, the
//    waits) bounds 64-token blocks there (131072 tokens of 8 heads: 66.8 us with 64, 58.9 with 128);
//  - one warp walks the range and brings the pages by TMA into rings of K and of V tiles, across
//    the ends of sequences; four warps take 16 of every 64 tokens each, held together by mbarriers
//    only (no barrier of the CTA in the loop);
//  - both products run on mma.sync (m16n8k16, bf16, fp32 accumulators): S^T = K Q^T and O^T +=
//    V^T P^T, so a lane's softmax state and its accumulators belong to the same two rows of each
//    8-row group. K and V are read once, so tcgen05 tiles of 128 rows would be 1/16 full;
//  - bf16 rows come as fragments by ldmatrix. 8-bit rows are widened to fp16 in registers (one
//    instruction a pair; fp16 holds every code): which element of the head dimension, and which
//    token, stands at which position of a fragment is free as long as both factors agree, so a
//    lane reads 16 consecutive codes and uses them for four MMAs. Q becomes fp16 too, each row
//    times a power of two;
//  - the 8-bit rows' scales are powers of two: K's multiply the scores, V's go into the exponents
//    of the weights, which a whole number a row (ex) brings to where they fit fp16;
//  - P enters the second product in parts: two of bf16 (16 bits; 8-bit pages: one of fp16, 11
//    bits, 8 at 2^-24 of the largest), three (24 bits and more) for fp32 output;
//  - a row's maximum is only brought up to date (three shuffles, O rescaled) when a score exceeds
//    it by more than 2^8; sums stay per lane until the end of a range, where the warps merge.
//
// Measured (8 KV heads, groups of 4, whole calls): 16 sequences of 65536 bf16 tokens 602 us, 7.1
// TB/s, HBM's bound; 16 of 32768 8-bit tokens 204 us, 5.3 TB/s; one of 131072 58 us, 4.6 TB/s, with
// the chain of launch, lengths, page ids, first tiles and join in it, and one of 4096 bf16 tokens 17.5
// us, the host's part of a call (12.2 in a captured graph: that chain). To fp32: 4 tokens over 65536
// 77.7 us in 8 bits and 67.8 in bf16, 16 of 32768 8-bit tokens 242 us. (Three CTAs an SM with
// 64-token blocks: 61 us for the one of 131072.) Why tiles of 8 and of 16 rows: 2 tokens over 65536
// (8 rows) take 53.2 us in tiles of 8 and 55.0 in tiles of 16 in bf16, 39.6 and 57.0 in 8 bits. Why
// not the chunk kernel's tiles up to 16 rows: 4 tokens over 65536 take 59.2 us here and 66.2 there in
// bf16, 61.4 and 85.2 in 8 bits; 8 sequences of 32768 170 and 204, 170 and 263.
#include <cuda_fp16.h>

#include "paged_async.cuh"

namespace pkv {

namespace {

constexpr int kFW = 4;                        // warps, 16 of every 64 tokens each
// Sequences that every CTA plans for itself. The plan kernel costs 5 us more at 1 sequence (52.0 and
// 57.0 us a call over 65536 tokens) and still 14 us at 256 of 2000 tokens (306 and 319); the sums
// of 256 sequences are what shared memory is kept for.
constexpr int kInline = 256;
constexpr int kSegs = 8;                      // segment records between the loads and the others
constexpr float kGrow = 8.0f;                 // growth of a maximum (base 2) that rescales O
// 8-bit pages: the largest fp16 weight of a row is put between 2^(kLift - 1) and 2^kLift when O is
// rescaled for it, and may grow to 2^kTop before that happens again (fp16 ends just below 2^16). fp16's
// steps end at 2^-24, so one part of a weight is off by 2^-12 of it or by 2^-32 of the largest,
// whichever is more: 8 bits down to 2^-24, and all weights that can be lost are less than 2^-12 of the
// largest together (180 GB of rows are 2^20 tokens a warp at most). What one part leaves is taken
// kPartStep times for the next, so three have 24 bits and more down to 2^-30, and are off by 2^-54 of
// the largest below. (Were the largest 1 and the parts as they are, weights would be cut at 2^-25 of
// it, in three parts as in one, while their sum has them in full: a tail of 131072 tokens at 2^-26
// would be missing. 2^13, with rescaling at a growth of 2^2, takes 62.4 us for 4 tokens over 65536,
// 2^7 60.8, as without any. With the maxima of those weights in fp32 beside mx, in place of whole
// numbers, 4 tokens to fp32 took 81.6 us, now 77.7, and above 2^24 their steps broke the 2^15.)
constexpr float kLift = 8.0f, kTop = 15.0f;
constexpr float kNoExp = -512.0f;             // the exponent of an O that has nothing in it
constexpr float kPartStep = 2048.0f;

template <bool kE4m3> struct FewShape {
    static constexpr int kRowB = kE4m3 ? D : 2 * D;          // bytes of a row
    static constexpr int kBlk = few_block(kE4m3);            // tokens of a block
    static constexpr int kSub = kBlk / (16 * kFW);           // a warp takes 16 tokens of each 64
    static constexpr int kTile = kBlk * kRowB;               // a K or V tile: 16 KB
    static constexpr int kNK = 3, kNV = 2;
    static constexpr int kScales = (kNK + kNV) * kTile;      // its scale bytes (8-bit)
    static constexpr int kScratch = kScales + (kE4m3 ? (kNK + kNV) * kBlk : 0);
    static constexpr int kPart = D + 4;                      // a row's partial in the scratch
    static constexpr int kSmem = kScratch + kFW * 8 * kPart * 4 + 1024;   // + alignment
};
static_assert(FewShape<true>::kNK < kSegs, "a record outlives the entries behind it");
static_assert(FewShape<true>::kNK < 4, "one barrier is left that nothing arrives at");

enum : int { kFirst = 1, kLast = 2, kEnd = 4 };
struct Meta {
    int32_t block, flags;
    uint32_t runs;         // 16-token runs that hold something a row may see
};
struct Seg {
    int64_t pos0;
    int32_t row0, first, nrow, head, end, kv, whole, part;
};
struct Control {
    uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4], met;
    Meta meta[4];
    Seg seg[kSegs];
    int64_t pre[kInline + 1];
    int64_t warp_sum[8];
    int32_t bad[2][D];     // first token whose V is not finite in this element, by segment
    int32_t abort;
};

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t r[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t r[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
// d = a * b + c (m16n8k16, fp32 accumulators; bf16 factors, or fp16 ones)
template <bool kF16>
__device__ __forceinline__ void mma16(float d[4], const uint32_t a[4], uint32_t b0, uint32_t b1,
                                      float c0, float c1, float c2, float c3) {
    if (kF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
            "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1),
              "f"(c2), "f"(c3));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
            "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1),
              "f"(c2), "f"(c3));
}
template <bool kF16>
__device__ __forceinline__ void mma16(float d[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
    mma16<kF16>(d, a, b0, b1, d[0], d[1], d[2], d[3]);
}
// o[j][i] += f * (the parts of 16 tokens' weights) for every group j of 8 rows. The tensor cores
// truncate their sums, which over a long range would shrink o by half a step a product; three
// parts are wanted for more than that leaves, so their sum begins anew every time and is added with
// rounding. (16 sequences of 4 tokens, 16 rows, over 16384 8-bit tokens: 241 us with the parts' sums
// apart, which are some 40 more one after the other; single tokens over 32768 242 with either.)
template <bool kF16, int NT, int kParts>
__device__ __forceinline__ void accumulate(float (&o)[NT][8][4], int i, const uint32_t f[4],
                                           const uint32_t (&p)[NT][kParts][2]) {
    if constexpr (kParts < 3) {
#pragma unroll
        for (int k = 0; k < kParts; ++k)
#pragma unroll
            for (int j = 0; j < NT; ++j) mma16<kF16>(o[j][i], f, p[j][k][0], p[j][k][1]);
    } else {
        // (bf16 parts into one sum; fp16 parts, each kPartStep times as large as it counts, apart)
        constexpr int kSums = kF16 ? kParts : 1;
        float z[kSums][NT][4];
#pragma unroll
        for (int k = kParts - 1; k >= 0; --k)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float(&y)[4] = z[kF16 ? k : 0][j];
                if (kF16 || k == kParts - 1)
                    mma16<kF16>(y, f, p[j][k][0], p[j][k][1], 0.0f, 0.0f, 0.0f, 0.0f);
                else
                    mma16<kF16>(y, f, p[j][k][0], p[j][k][1]);
            }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float y = z[kSums - 1][j][e];
#pragma unroll
                for (int k = kSums - 2; k >= 0; --k) y = fmaf(y, 1.0f / kPartStep, z[k][j][e]);
                o[j][i][e] += y;
            }
    }
}
__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t bf2(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ float2 bf2_f(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

__device__ __forceinline__ uint32_t h2(float lo, float hi) {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ float2 h2_f(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
// two e4m3 codes as fp16 values (exact: fp16 has the exponents and the bits)
__device__ __forceinline__ uint32_t widen2(uint16_t codes) {
    uint32_t y;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(y) : "h"(codes));
    return y;
}
__device__ __forceinline__ uint32_t widen_lo(uint32_t w) {
    return widen2(static_cast<uint16_t>(w));
}
__device__ __forceinline__ uint32_t widen_hi(uint32_t w) {
    return widen2(static_cast<uint16_t>(w >> 16));
}

// The last of n + 1 sums with pre[i] <= x.
__device__ __forceinline__ int find_pre(const int64_t* pre, int n, int64_t x) {
    int lo = 0, len = n;
    while (len > 1) {
        const int half = len >> 1;
        if (pre[lo + half] <= x) {
            lo += half;
            len -= half;
        } else {
            len = half;
        }
    }
    return lo;
}

// Where a CTA's range lies. Up to kInline sequences (a tile each, the host sees to that) are
// planned here, by every CTA for itself.
struct Range {
    int64_t x, hi, per_head, n;   // n: CTAs with work
    int32_t nt;
    bool inline_plan;
};

__device__ __forceinline__ Tile tile_record(const AttendArgs& a, int s, int64_t pre) {
    const SeqView v = seq_view(a.seqs, a.pool.shift, s);
    Tile t;
    t.pre = pre;
    t.pos0 = v.pos0;
    t.seq = s;
    t.row0 = v.row0;
    t.first = 0;
    t.nrow = static_cast<int32_t>(
        min64(a.shape.tile_rows, static_cast<int64_t>(v.rows) * a.shape.group));
    t.end = tile_end(v, a.shape, 0);
    t.kv = v.kv;
    t.pad[0] = t.pad[1] = 0;
    return t;
}

__device__ __forceinline__ Range make_range(const AttendArgs& a, Control& c, bool inline_plan) {
    Range r;
    r.inline_plan = inline_plan;
    if (inline_plan) {
        r.nt = a.seqs.batch;
        // a thread sums up consecutive sequences, then the threads' sums are scanned
        constexpr int kT = (kFW + 1) * 32;
        const int per = (r.nt + kT - 1) / kT, s0 = threadIdx.x * per;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        int64_t sum = 0;
        for (int i = 0; i < per && s0 + i < r.nt; ++i) {
            const SeqView v = seq_view(a.seqs, a.pool.shift, s0 + i);
            c.pre[s0 + i] = sum;
            sum += v.rows > 0 ? tile_blocks(v, a.shape, 0) : 0;
        }
        int64_t scan = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, scan, o);
            if (lane >= o) scan += y;
        }
        if (lane == 31) c.warp_sum[warp] = scan;
        __syncthreads();
        int64_t before = scan - sum, all = 0;
        for (int w = 0; w <= kFW; ++w) {
            if (w < warp) before += c.warp_sum[w];
            all += c.warp_sum[w];
        }
        for (int i = 0; i < per && s0 + i < r.nt; ++i) c.pre[s0 + i] += before;
        if (threadIdx.x == 0) c.pre[r.nt] = all;
        r.per_head = all;
        __syncthreads();
    } else {
        r.nt = *a.plan.ntiles;
        r.per_head = a.plan.tile[r.nt].pre;
    }
    const int64_t total = r.per_head * a.heads;
    r.n = cuts(total, gridDim.x);
    const bool work = blockIdx.x < r.n;
    r.x = work ? cut(total, r.n, blockIdx.x) : 0;
    r.hi = work ? cut(total, r.n, blockIdx.x + 1) : 0;
    return r;
}

// ---------------------------------------------------------------------------------- loads
template <bool kE4m3>
__device__ void few_loads(const AttendArgs& a, const CUtensorMap* mk, const CUtensorMap* mv,
                          Control& c, uint8_t* smem, const Range& range) {
    using S = FewShape<kE4m3>;
    const int lane = threadIdx.x & 31, shift = a.pool.shift;
    constexpr int kBlk = S::kBlk, kLog = kBlk == 128 ? 7 : 6;
    static_assert(kBlk == 1 << kLog, "64 or 128 tokens");
    const int rs = min(shift, kLog), run = 1 << rs, ns = kLog - rs, nrun = 1 << ns;
    const int per_win = 32 >> ns;
    volatile int32_t* ab = &c.abort;
    int64_t x = range.x, h = 0;
    uint32_t n = 0, seg = 0;
    int tile = 0;
    if (x < range.hi) {
        h = x / range.per_head;
        const int64_t rest = x - h * range.per_head;
        tile = range.inline_plan ? find_pre(c.pre, range.nt, rest)
                                 : find_tile(a.plan.tile, range.nt, rest);
    }
    if (x >= range.hi && lane == 0) a.cut[blockIdx.x].parts = 0;
    while (x < range.hi) {
        const Tile t = range.inline_plan ? tile_record(a, tile, c.pre[tile]) : a.plan.tile[tile];
        const int64_t nb = (range.inline_plan ? c.pre[tile + 1] : a.plan.tile[tile + 1].pre) - t.pre;
        const int64_t start = h * range.per_head + t.pre;
        const int b0 = static_cast<int>(x - start);
        const int b1 = static_cast<int>(min64(nb, range.hi - start));
        if (seg == 0 && lane == 0)
            a.cut[blockIdx.x] =
                cut_record(t, range.per_head * a.heads, range.n, start, start + nb, b0, h);
        const int32_t* table = a.seqs.table + static_cast<int64_t>(t.seq) * a.seqs.stride;
        // page ids come 32 at a time, a lane a run, one window ahead
        auto fetch = [&](int w) -> int {
            const int tok = w * kBlk + lane * run;
            return w + (lane >> ns) < b1 && tok < t.end ? table[tok >> shift] : -1;
        };
        int win = b0, id = fetch(b0), id_next = fetch(b0 + per_win);
        uint32_t valid = 0;
        int page = 0;
        // the next block with a page that is there, from b on
        auto live = [&](int b) -> int {
            for (; b < b1; ++b) {
                if (b >= win + per_win) {
                    win += per_win;
                    id = id_next;
                    id_next = fetch(win + per_win);
                }
                const uint32_t ok = __ballot_sync(
                    0xffffffffu, static_cast<uint32_t>(id) < static_cast<uint32_t>(a.pool.num_pages));
                const int at = (b - win) << ns;
                valid = (ok >> at) & ((1u << nrun) - 1);
                page = __shfl_sync(0xffffffffu, id, (at + lane) & 31);
                if (valid) return b;
            }
            valid = 0;
            return -1;
        };
        bool first = true;
        int b = live(b0);
        while (first || b >= 0) {
            const uint32_t cur_valid = valid;
            const int cur_page = page, cur = b;
            if (b >= 0) b = live(b + 1);
            const int ks = n % S::kNK, vs = n % S::kNV;
            const bool mine = lane < nrun && (cur_valid >> lane & 1);
            const int tok = cur * kBlk + lane * run;
            const int row = (static_cast<int>(h) << shift) + (tok & ((1 << shift) - 1));
            if (!warp_wait(&c.k_empty[ks], ((n / S::kNK) & 1) ^ 1, ab)) return;
            const uint32_t bytes = __popc(cur_valid) * run * (kE4m3 ? D + 1 : 2 * D);
            if (lane == 0) {
                if (first) {
                    Seg g;
                    g.pos0 = t.pos0;
                    g.row0 = t.row0;
                    g.first = t.first;
                    g.nrow = t.nrow;
                    g.head = static_cast<int>(h);
                    g.end = t.end;
                    g.kv = t.kv;
                    g.whole = b0 == 0 && b1 == nb;
                    g.part = 2 * static_cast<int>(blockIdx.x) + (b0 == 0);
                    c.seg[seg % kSegs] = g;
                }
                Meta m;
                m.block = cur;
                m.flags = (first ? kFirst : 0) | (b < 0 ? kLast : 0);
                m.runs = 0;
                for (int i = 0; i < kBlk / 16; ++i)
                    if ((cur_valid >> (16 * i >> rs) & 1) && cur * kBlk + 16 * i < t.end)
                        m.runs |= 1u << i;
                c.meta[ks] = m;
                mbar_arrive_expect_tx(smem_addr(&c.k_full[ks]), bytes);
            }
            __syncwarp();
            auto bring = [&](int slot, int of, uint64_t* bar) {
                uint8_t* dst = smem + slot * S::kTile + lane * run * 128;
                const CUtensorMap* m = of ? mv : mk;
                tma_load3(smem_addr(dst), m, 0, row, cur_page, smem_addr(bar));
                if (kE4m3)
                    bulk_g2s(smem_addr(smem + S::kScales + slot * kBlk + lane * run),
                             (of ? a.pool.vs : a.pool.ks) + cur_page * a.pool.scale_stride + row,
                             run, smem_addr(bar));
                else
                    tma_load3(smem_addr(dst + S::kTile / 2), m, 64, row, cur_page, smem_addr(bar));
            };
            if (mine) bring(ks, 0, &c.k_full[ks]);
            if (!warp_wait(&c.v_empty[vs], ((n / S::kNV) & 1) ^ 1, ab)) return;
            if (lane == 0) mbar_arrive_expect_tx(smem_addr(&c.v_full[vs]), bytes);
            __syncwarp();
            if (mine) bring(S::kNK + vs, 1, &c.v_full[vs]);
            first = false;
            ++n;
        }
        ++seg;
        x = start + b1;
        if (b1 == nb) {
            // (sequences without rows have no blocks)
            do {
                if (++tile == range.nt) {
                    tile = 0;
                    ++h;
                }
            } while (range.inline_plan && x < range.hi && c.pre[tile + 1] == c.pre[tile]);
        }
    }
    const int ks = n % S::kNK;
    if (!warp_wait(&c.k_empty[ks], ((n / S::kNK) & 1) ^ 1, ab)) return;
    if (lane == 0) {
        c.meta[ks].flags = kEnd;
        arrive(&c.k_full[ks]);
    }
}

// NT groups of 8 rows; kParts bf16 parts of P.
template <bool kE4m3, int NT, int kParts, typename Out>
__device__ void few_consume(const AttendArgs& a, Control& c, uint8_t* smem) {
    using S = FewShape<kE4m3>;
    constexpr int R = 8 * NT, kPart = S::kPart, kSub = S::kSub;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3, mi = lane >> 3, j8 = lane & 7;
    // the token of a lane's first row of S (the second is 8 on), and the 16-byte piece of a V row
    // that it reads: orders in which 8 lanes' reads of swizzled 8-bit rows meet no bank twice
    const int pg = kE4m3 ? (g >> 1) | (g & 1) << 2 : g;
    const int G = a.shape.group;
    const float qs = a.scale * kLog2e;
    volatile int32_t* ab = &c.abort;
    float* scr = reinterpret_cast<float*>(smem + S::kScratch);

    uint32_t n = 0, seg = 0, nm = 0;      // entries, segments, meetings
    Seg sg = {};
    uint32_t qb[NT][8][2];
    int lim[NT][2], shared = 0;
    int down[NT][2];     // exponents that undo what the rows of Q were multiplied by (8-bit)
    float mx[NT][2], den[NT][2], o[NT][8][4];
    float ex[NT][2];     // O is relative to mx + ex (8-bit; whole numbers)
    // the last token a row may attend
    auto limit = [&](int r) -> int {
        if (r >= sg.nrow) return -1;
        const int64_t l = a.shape.causal ? sg.pos0 + (sg.first + r) / G : sg.kv - 1;
        return static_cast<int>(max64(-1, min64(l, sg.kv - 1)));
    };
    auto meet = [&]() -> bool {           // of the four warps
        __syncwarp();
        if (lane == 0) arrive(&c.met);
        return warp_wait(&c.met, nm++ & 1, ab);
    };
#pragma unroll 1
    while (true) {
        const int ks = n % S::kNK, vs = n % S::kNV;
        if (!warp_wait(&c.k_full[ks], (n / S::kNK) & 1, ab)) return;
        const Meta m = c.meta[ks];
        if (m.flags & kEnd) return;
        if (m.flags & kFirst) {
            sg = c.seg[seg % kSegs];
            shared = limit(0);
            // B fragments of Q^T: row 8 j + g of the tile; with 8-bit pages, position k of MMA m
            // is element 64 (m / 4) + 16 t + 4 (m % 4) + ... of the row, as the K codes are read
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int r = 8 * j + g;
                const bool ok = r < sg.nrow;
                const int rr = sg.first + (ok ? r : 0);
                const uint32_t* qr = reinterpret_cast<const uint32_t*>(
                    a.q + (sg.row0 + rr / G) * a.q_ld +
                    (static_cast<int64_t>(sg.head) * G + rr % G) * D);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int i0 = kE4m3 ? 32 * (i >> 2) + 8 * t + 2 * (i & 3) : 8 * i + t;
                    const int i1 = kE4m3 ? i0 + 1 : i0 + 4;
                    qb[j][i][0] = ok ? qr[i0] : 0u;
                    qb[j][i][1] = ok ? qr[i1] : 0u;
                }
                float up = 1.0f;
                if (kE4m3) {
                    // the fp16 of the row times a power of two that brings its largest magnitude
                    // to [2^14, 2^15): exact but for what is 2^31 times smaller than that
                    uint32_t top = 0;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const uint32_t x = qb[j][i >> 1][i & 1];
                        top = max(top, max(x & 0x7fffu, x >> 16 & 0x7fffu));
                    }
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    // (in two steps: the power itself may be out of range)
                    const int e =
                        top >= 0x7f80u || top < 0x80u ? 0 : 127 + 14 - static_cast<int>(top >> 7);
                    const float f0 = pow2f(e / 2), f1 = pow2f(e - e / 2);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 x = bf2_f(qb[j][i >> 1][i & 1]);
                        qb[j][i >> 1][i & 1] = h2(x.x * f0 * f1, x.y * f0 * f1);
                    }
                    up = __int_as_float(e);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    // (that row's exponent is with the lanes whose g it is)
                    const int k = __float_as_int(__shfl_sync(0xffffffffu, up, 4 * (2 * t + e)));
                    down[j][e] = kE4m3 ? -k : 0;
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    lim[j][e] = limit(8 * j + 2 * t + e);
                    mx[j][e] = -INFINITY;
                    ex[j][e] = kNoExp;
                    den[j][e] = 0.0f;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    o[j][i][0] = o[j][i][1] = o[j][i][2] = o[j][i][3] = 0.0f;
            }
        }
        // the warp's 16 tokens of each 64: rows 64 u + 16 warp ... of the tiles
        bool live[kSub];
        int tok[kSub];                                   // this lane's: tok, tok + 8
        bool any = false;
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
            live[u] = m.runs >> (kFW * u + warp) & 1;
            any = any || live[u];
            tok[u] = m.block * S::kBlk + 64 * u + 16 * warp + pg;
        }

        // S^T: 16 tokens x R rows
        float sc[kSub][NT][4];
        float ka[kSub], kb[kSub];
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
            ka[u] = kb[u] = 1.0f;
#pragma unroll
            for (int j = 0; j < NT; ++j) sc[u][j][0] = sc[u][j][1] = sc[u][j][2] = sc[u][j][3] = 0.0f;
            if (!live[u]) continue;
            const int r0 = 64 * u + 16 * warp;
            const uint8_t* kt = smem + ks * S::kTile;
            if (kE4m3) {
                const uint8_t* sp = smem + S::kScales + ks * S::kBlk + r0 + pg;
                ka[u] = scale_value(sp[0]);
                kb[u] = scale_value(sp[8]);
                const uint32_t base = smem_addr(kt + (r0 + pg) * 128);
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const uint32_t at = base + (((4 * hh + t) ^ pg) << 4);
                    const uint4 lo = lds128(at), up = lds128(at + 8 * 128);
                    const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w};
                    const uint32_t wu[4] = {up.x, up.y, up.z, up.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t f[4] = {widen_lo(wl[i]), widen_lo(wu[i]), widen_hi(wl[i]),
                                               widen_hi(wu[i])};
#pragma unroll
                        for (int j = 0; j < NT; ++j)
                            mma16<kE4m3>(sc[u][j], f, qb[j][4 * hh + i][0], qb[j][4 * hh + i][1]);
                    }
                }
            } else {
                const int row = r0 + j8 + 8 * (mi & 1), kc = mi >> 1;
                const uint32_t base = smem_addr(kt + row * 128);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint32_t f[4];
                    const int ch = 2 * i + kc;
                    ldsm_x4(base + (ch >> 3) * (S::kTile / 2) + (((ch & 7) ^ (row & 7)) << 4), f);
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        mma16<kE4m3>(sc[u][j], f, qb[j][i][0], qb[j][i][1]);
                }
            }
        }
        __syncwarp();
        if (lane == 0) arrive(&c.k_empty[ks]);

        // softmax: weights with the maxima as they are, unless a score is far above
        float w[kSub][NT][4];
        using Block = float[kSub][NT][4];
        // the largest of a row in the block
        auto highest = [&](const Block& x, int j, int e) -> float {
            float bm = -INFINITY;
#pragma unroll
            for (int u = 0; u < kSub; ++u) bm = fmaxf(bm, fmaxf(x[u][j][e], x[u][j][2 + e]));
#pragma unroll
            for (int k = 4; k < 32; k <<= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, k));
            return bm;
        };
        // whether the warp has anything above its row's bound
        auto above = [&](const Block& x, auto bound) -> bool {
            bool some = false;
#pragma unroll
            for (int u = 0; u < kSub; ++u)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        some = some || fmaxf(x[u][j][e], x[u][j][2 + e]) > bound(j, e);
            return __any_sync(0xffffffffu, some);
        };
        auto rescale = [&](const float (&co)[NT][2]) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    o[j][i][0] *= co[j][0]; o[j][i][1] *= co[j][1];
                    o[j][i][2] *= co[j][0]; o[j][i][3] *= co[j][1];
                }
        };
        if (any) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    // (the power that undoes Q's may be out of range: two steps)
                    const float d0 = kE4m3 ? pow2f(down[j][e] / 2) : 1.0f;
                    const float d1 = kE4m3 ? pow2f(down[j][e] - down[j][e] / 2) : 1.0f;
#pragma unroll
                    for (int u = 0; u < kSub; ++u) {
                        const float s0 = kE4m3 ? sc[u][j][e] * d0 * d1 : sc[u][j][e];
                        const float s1 = kE4m3 ? sc[u][j][2 + e] * d0 * d1 : sc[u][j][2 + e];
                        sc[u][j][e] = live[u] && tok[u] <= lim[j][e] ? s0 * (qs * ka[u]) : -INFINITY;
                        sc[u][j][2 + e] =
                            live[u] && tok[u] + 8 <= lim[j][e] ? s1 * (qs * kb[u]) : -INFINITY;
                    }
                }
            float co[NT][2];
            if (above(sc, [&](int j, int e) { return mx[j][e] + kGrow; })) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float m1 = fmaxf(mx[j][e], highest(sc, j, e));
                        const float down = mx[j][e] - (m1 == -INFINITY ? 0.0f : m1);
                        co[j][e] = exp2f(down);
                        den[j][e] *= co[j][e];
                        mx[j][e] = m1;
                        if (kE4m3) {   // O keeps its place, but for less than a step up
                            const float k = ceilf(-down);
                            const bool far = !(k < 600.0f);
                            co[j][e] = far ? 0.0f : exp2f(down + k);
                            ex[j][e] = far ? kNoExp : ex[j][e] - k;
                        }
                    }
                rescale(co);
            }
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float ms = mx[j][e] == -INFINITY ? 0.0f : mx[j][e];
#pragma unroll
                    for (int u = 0; u < kSub; ++u)
#pragma unroll
                        for (int i = e; i < 4; i += 2) {
                            sc[u][j][i] -= ms;
                            w[u][j][i] = exp2f(sc[u][j][i]);
                        }
                }
#pragma unroll
            for (int u = 0; u < kSub; ++u)
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    den[j][0] += w[u][j][0] + w[u][j][2];
                    den[j][1] += w[u][j][1] + w[u][j][3];
                }
        }
        if (!warp_wait(&c.v_full[vs], (n / S::kNV) & 1, ab)) return;
        if (any) {
            uint8_t* vt = smem + (S::kNK + vs) * S::kTile;
            const uint8_t* vsc = smem + S::kScales + (S::kNK + vs) * S::kBlk;   // (8-bit)
            // What no row or not every row may see must not reach them: 0 * NaN is NaN. So rows
            // behind the end of the sequence are cleared, and what is not finite in the rows of
            // the chunk itself (8-bit: a NaN row) is taken out and put back at the end into the
            // rows that see it.
            const int last = m.block * S::kBlk + S::kBlk - 1;
            const bool repair = last > shared && (sg.end - 1 > shared || last >= sg.end);
            if (repair) {
                int32_t* bad_at = c.bad[seg & 1];
                constexpr int kPieces = S::kRowB / 16;
#pragma unroll 1
                for (int i = lane; i < kSub * 16 * kPieces; i += 32) {
                    const int r = i / kPieces, ch = i % kPieces;
                    const int row = 64 * (r >> 4) + 16 * warp + (r & 15);
                    const int tk = m.block * S::kBlk + row;
                    if (tk <= shared || !(m.runs >> (row >> 4) & 1)) continue;
                    uint4* e = reinterpret_cast<uint4*>(vt + (ch >> 3) * (S::kTile / 2) + row * 128 +
                                                        (((ch & 7) ^ (row & 7)) << 4));
                    if (tk >= sg.end) {
                        *e = make_uint4(0, 0, 0, 0);
                        continue;
                    }
                    if (kE4m3) {
                        if (vsc[row] != kNanRow) continue;
                        for (int k = 0; k < 16; ++k) atomicMin(&bad_at[16 * ch + k], tk);
                        *e = make_uint4(0, 0, 0, 0);
                        continue;
                    }
                    const uint4 y = *e;
                    uint32_t x[4] = {y.x, y.y, y.z, y.w};
                    bool odd = false;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if ((x[k] & 0x7f80u) == 0x7f80u) {
                            atomicMin(&bad_at[8 * ch + 2 * k], tk);
                            x[k] &= 0xffff0000u;
                            odd = true;
                        }
                        if ((x[k] & 0x7f800000u) == 0x7f800000u) {
                            atomicMin(&bad_at[8 * ch + 2 * k + 1], tk);
                            x[k] &= 0xffffu;
                            odd = true;
                        }
                    }
                    if (odd) *e = make_uint4(x[0], x[1], x[2], x[3]);
                }
                fence_async_smem();
                __syncwarp();
            }
            if (kE4m3) {
                // the weights of O: with V's scales and the row's ex in the exponent, which are whole
                // numbers, so that a weight has the bits that it has in den however large mx is
                float ea[kSub][2];
#pragma unroll
                for (int u = 0; u < kSub; ++u)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint8_t byte = vsc[64 * u + 16 * warp + pg + 8 * k];
                        ea[u][k] = static_cast<float>(byte - 127);
                        // (a cleared NaN row weighs nothing)
                        if (repair && tok[u] + 8 * k > shared && byte == kNanRow) ea[u][k] = -INFINITY;
                    }
                // (one part is far coarser than what in-place exponents lose when ex grows)
                constexpr bool kAnew = kParts > 1;
                Block& x = kAnew ? w : sc;
                auto place = [&] {
#pragma unroll
                    for (int u = 0; u < kSub; ++u)
#pragma unroll
                        for (int j = 0; j < NT; ++j)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                x[u][j][i] = sc[u][j][i] + (ea[u][i >> 1] - ex[j][i & 1]);
                };
                place();
                if (above(x, [](int, int) { return kTop; })) {
                    float co[NT][2];
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float k = fmaxf(ceilf(highest(x, j, e)) - kLift, 0.0f);
                            co[j][e] = exp2f(-k);
                            ex[j][e] += k;
#pragma unroll
                            for (int u = 0; u < kSub && !kAnew; ++u) {
                                x[u][j][e] -= k;
                                x[u][j][2 + e] -= k;
                            }
                        }
                    rescale(co);
                    if (kAnew) place();
                }
#pragma unroll
                for (int u = 0; u < kSub; ++u)
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) w[u][j][i] = exp2f(x[u][j][i]);
            }
#pragma unroll
            for (int u = 0; u < kSub; ++u) {
                if (!live[u]) continue;
                const int r0 = 64 * u + 16 * warp;
                // the weights as B fragments (k = tokens, n = rows), in parts
                uint32_t pb[NT][kParts][2];
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int k = 0; k < kParts; ++k) {
                        float(&x)[4] = w[u][j];
                        const uint32_t h01 = kE4m3 ? h2(x[0], x[1]) : bf2(x[0], x[1]);
                        const uint32_t h23 = kE4m3 ? h2(x[2], x[3]) : bf2(x[2], x[3]);
                        pb[j][k][0] = movm_t(h01);
                        pb[j][k][1] = movm_t(h23);
                        const float2 f01 = kE4m3 ? h2_f(h01) : bf2_f(h01);
                        const float2 f23 = kE4m3 ? h2_f(h23) : bf2_f(h23);
                        x[0] -= f01.x; x[1] -= f01.y; x[2] -= f23.x; x[3] -= f23.y;
                        if (kE4m3) {   // (a part of what is left would run into fp16's last steps)
                            x[0] *= kPartStep; x[1] *= kPartStep;
                            x[2] *= kPartStep; x[3] *= kPartStep;
                        }
                    }
                // O^T += V^T P^T. MMA i covers elements 16 i + g and 16 i + g + 8 of a row (bf16),
                // or 16 pg + 2 i and 16 pg + 2 i + 1 (8-bit)
                if (kE4m3) {
                    uint32_t wv[4][4];   // S rows 2t, 2t+1, 2t+8, 2t+9: tokens t, t+4, t+8, t+12
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int row = r0 + t + 4 * k;
                        const uint4 q4 =
                            lds128(smem_addr(vt + row * 128) + ((pg ^ (row & 7)) << 4));
                        wv[k][0] = q4.x; wv[k][1] = q4.y; wv[k][2] = q4.z; wv[k][3] = q4.w;
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        // two elements of two neighbouring tokens: a pair a register
                        uint32_t f[4];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t a0 = wv[2 * k][i >> 1], a1 = wv[2 * k + 1][i >> 1];
                            const uint32_t y = i & 1 ? prmt_i<0x7362>(a0, a1) : prmt_i<0x5140>(a0, a1);
                            f[2 * k] = widen_lo(y);
                            f[2 * k + 1] = widen_hi(y);
                        }
                        accumulate<kE4m3>(o, i, f, pb);
                    }
                } else {
                    const int row = r0 + j8 + 8 * (mi >> 1), vc = mi & 1;
                    const uint32_t base = smem_addr(vt + row * 128);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        uint32_t f[4];
                        const int ch = 2 * i + vc;
                        ldsm_x4_t(base + (ch >> 3) * (S::kTile / 2) + (((ch & 7) ^ (row & 7)) << 4),
                                  f);
                        accumulate<kE4m3>(o, i, f, pb);
                    }
                }
            }
        }
        __syncwarp();
        if (lane == 0) arrive(&c.v_empty[vs]);
        ++n;
        if (!(m.flags & kLast)) continue;

        // the warps' partials of 8 rows at a time, merged
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int k = 4; k < 32; k <<= 1)
                    den[j][e] += __shfl_xor_sync(0xffffffffu, den[j][e], k);
                float* p = scr + (warp * 8 + 2 * t + e) * kPart;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    p[kE4m3 ? 16 * pg + 2 * i : 16 * i + g] = o[j][i][e];
                    p[kE4m3 ? 16 * pg + 2 * i + 1 : 16 * i + g + 8] = o[j][i][2 + e];
                }
                if (g == 0) {
                    p[D] = mx[j][e];
                    p[D + 1] = den[j][e];
                    p[D + 2] = ex[j][e];
                }
            }
            if (!meet()) return;
            float* part = a.work + static_cast<int64_t>(sg.part) * part_floats(R);
            for (int r8 = warp; r8 < 8 && 8 * j + r8 < sg.nrow; r8 += kFW) {
                const int r = 8 * j + r8;
                float M = -INFINITY;
#pragma unroll
                for (int x = 0; x < kFW; ++x) M = fmaxf(M, scr[(x * 8 + r8) * kPart + D]);
                const float ms = M == -INFINITY ? 0.0f : M;
                float dn = 0.0f, y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int x = 0; x < kFW; ++x) {
                    const float* src = scr + (x * 8 + r8) * kPart;
                    float f = exp2f(src[D] - ms);
                    dn += src[D + 1] * f;
                    if (kE4m3) {   // (whole numbers apart, and in two steps: each may be out of range)
                        const float d = fmaxf(src[D] - ms, -1000.0f);
                        const int k = max(-252, min(252, static_cast<int>(floorf(d) + src[D + 2])));
                        f = exp2f(d - floorf(d)) * pow2f(k / 2) * pow2f(k - k / 2);
                    }
                    const float4 z = *reinterpret_cast<const float4*>(src + 4 * lane);
                    y[0] += z.x * f; y[1] += z.y * f; y[2] += z.z * f; y[3] += z.w * f;
                }
                const int lr = limit(r);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (c.bad[seg & 1][4 * lane + i] <= lr) y[i] = __uint_as_float(0x7fc00000u);
                if (sg.whole) {
                    const float inv = dn == 0.0f ? 0.0f : 1.0f / dn;
                    const int rr = sg.first + r;
                    const int64_t at = (sg.row0 + rr / G) * (static_cast<int64_t>(a.heads) * G) +
                                       static_cast<int64_t>(sg.head) * G + rr % G;
                    Out* dst = static_cast<Out*>(a.out) + at * D + 4 * lane;
                    if constexpr (sizeof(Out) == 2)
                        *reinterpret_cast<uint2*>(dst) =
                            make_uint2(bf2(y[0] * inv, y[1] * inv), bf2(y[2] * inv, y[3] * inv));
                    else
                        *reinterpret_cast<float4*>(dst) =
                            make_float4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
                    if (a.lse && lane == 0)
                        a.lse[at] = dn == 0.0f ? -INFINITY : M * kLn2 + logf(dn);
                } else {
                    *reinterpret_cast<float4*>(part + r * D + 4 * lane) =
                        make_float4(y[0], y[1], y[2], y[3]);
                    if (lane == 0) {
                        part[R * D + r] = M;
                        part[R * D + R + r] = dn;
                    }
                }
            }
            if (j == NT - 1) c.bad[(seg + 1) & 1][tid] = INT32_MAX;
            if (!meet()) return;   // the scratch is free again
        }
        ++seg;
    }
}

template <bool kE4m3, int NT, int kParts, typename Out>
__global__ void __launch_bounds__((kFW + 1) * 32, 2)
attend_few_kernel(const AttendArgs a, const __grid_constant__ CUtensorMap mk,
                  const __grid_constant__ CUtensorMap mv, int inline_plan) {
    using S = FewShape<kE4m3>;
    extern __shared__ uint8_t raw_smem[];
    __shared__ __align__(16) Control c;
    uint8_t* smem = raw_smem + ((1024 - (smem_addr(raw_smem) & 1023)) & 1023);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        c.abort = 0;
        for (int i = 0; i < 4; ++i) {
            mbar_init(smem_addr(&c.k_full[i]), 1);
            mbar_init(smem_addr(&c.k_empty[i]), kFW);
            mbar_init(smem_addr(&c.v_full[i]), 1);
            mbar_init(smem_addr(&c.v_empty[i]), kFW);
        }
        mbar_init(smem_addr(&c.met), kFW);
        mbar_fence_init();
        tma_prefetch_map(&mk);
        tma_prefetch_map(&mv);
    }
    if (threadIdx.x < D) c.bad[0][threadIdx.x] = c.bad[1][threadIdx.x] = INT32_MAX;
    pdl_wait();
    pdl_launch_dependents();
    const Range range = make_range(a, c, inline_plan != 0);
    __syncthreads();
    if (warp == kFW)
        few_loads<kE4m3>(a, &mk, &mv, c, smem, range);
    else if (a.inject_wait && warp == 0)   // test hook: a wait for an arrival that never comes
        wait_for(&c.k_full[S::kNK], 0, &c.abort, 1000000ull);
    else
        few_consume<kE4m3, NT, kParts, Out>(a, c, smem);
    __syncthreads();
    if (c.abort && warp == kFW) {
        // copies that were under way when a wait ran out write into this CTA's memory: give them
        // the time that any of them takes before the CTA ends
        const uint64_t t0 = now_ns();
        while (now_ns() - t0 < 10000000ull) {}
    }
}

template <bool kE4m3, int NT, int kParts, typename Out>
cudaError_t launch_few(const AttendArgs& a, const CUtensorMap maps[2], int ctas, bool inline_plan,
                       cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    constexpr int smem = FewShape<kE4m3>::kSmem;
    auto kernel = attend_few_kernel<kE4m3, NT, kParts, Out>;
    const cudaError_t e = raise_smem_limit(kernel, smem, done);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3(ctas), dim3((kFW + 1) * 32), smem, st, a, maps[0], maps[1],
                      inline_plan ? 1 : 0);
}

template <bool kE4m3, int NT>
cudaError_t launch_few_out(const AttendArgs& a, const CUtensorMap maps[2], bool f32_out, int ctas,
                           bool inline_plan, cudaStream_t st) {
    return f32_out ? launch_few<kE4m3, NT, 3, float>(a, maps, ctas, inline_plan, st)
                   : launch_few<kE4m3, NT, kE4m3 ? 1 : 2, __nv_bfloat16>(a, maps, ctas, inline_plan,
                                                                         st);
}

}  // namespace

int few_ctas(int sms) { return 2 * sms; }

bool few_plans_inline(int batch) { return batch <= kInline; }

cudaError_t launch_attend_few(const AttendArgs& a, int format, bool f32_out, int ctas,
                              cudaStream_t st) {
    const bool e4 = format == PARISKV_PAGES_E4M3, in = few_plans_inline(a.seqs.batch);
    const uint64_t el = e4 ? 1 : 2;
    CUtensorMap maps[2];
    for (int t = 0; t < 2; ++t)
        if (!encode_rows(&maps[t], t ? a.pool.v : a.pool.k, e4, true,
                         static_cast<uint64_t>(a.heads) << a.pool.shift, a.pool.num_pages, el * D,
                         a.pool.page_bytes, e4 ? D : 64, min(1 << a.pool.shift, few_block(e4)), 1))
            return cudaErrorInvalidValue;
    const bool one = a.shape.tile_rows == 8;
    if (e4)
        return one ? launch_few_out<true, 1>(a, maps, f32_out, ctas, in, st)
                   : launch_few_out<true, 2>(a, maps, f32_out, ctas, in, st);
    return one ? launch_few_out<false, 1>(a, maps, f32_out, ctas, in, st)
               : launch_few_out<false, 2>(a, maps, f32_out, ctas, in, st);
}

cudaError_t take_few_waits_out(bool* out, cudaStream_t st) { return take_waits_out(out, st); }

}  // namespace pkv
