// paged_chunk.cu -- attention of a chunk of new tokens over pages, on the tcgen05 tensor cores:
//     S = scale Q K^T (masked),  P = exp(S - m),  O += P V,  out = O / sum P.
//
// With many query rows a K/V head the call is bound by the two products (4 * 128 flops a pair of
// row and token) and, right behind them, by the exponentials: 128 x 128 scores take 1024 cycles
// of products and 1024 of the SM's 16 exponentials a cycle. So the kernel's aim is to keep the
// tensor cores and the exponential units busy at the same time:
//  - a tile is 2 x 128 query rows (tokens x heads of one KV head's group) against blocks of 128
//    tokens, so a K or V block that has come to shared memory serves 256 rows;
//  - S of both halves (2 x 128 columns) and O of both halves (2 x 128 columns) fill the 512 columns
//    of tensor memory; P overwrites S as bf16 and is the second product's operand from there, so
//    neither S nor P ever touches shared memory;
//  - two warpgroups do the softmax, one a half, a thread a row (no shuffles); a block is taken in
//    two turns of 64 tokens, and the scores of the next turn are there before this one's are done;
//  - O is rescaled only when a row's maximum has grown by more than 2^8 since the last time (P is
//    then at most 2^8, which costs bf16 nothing), so tensor memory is not read back each block;
//  - to bf16, P is rounded to bf16: off by half a step each, which the sum averages, so that outputs
//    are off by 2.1e-3 (relative, all elements) where the output's own rounding makes 1.7e-3. A second
//    part would take half as many products again, and they are what bounds the kernel; fp32 output
//    (below) is there for whoever wants more;
//  - K, V and Q tiles come by TMA through a ring of 32 KB stages, one copy a page and 64 columns;
//    with 8-bit pages they come as bytes, and seven or eight warps widen them into the ring, scale
//    and all (a power of two: the bf16 values are exact);
//  - blocks in which some token must not reach some row (the causal edge, the end of the cache,
//    pages that are not there) are marked: their scores are masked, and their V rows are made
//    finite first, because 0 * NaN is NaN; what was not finite is put back into the rows that see
//    it at the end;
//  - blocks without a single page that is there are passed over, and count nothing when the work
//    is cut into equal ranges (the plan leaves a bit a block).
//
// fp32 output takes P in three bf16 parts (24 bits, three products); a tile is then 128 rows, and the
// other half's columns of tensor memory take the third parts and a sum of O: the tensor cores
// truncate, which shrinks O by half a step a product, so every 2 blocks O is added to the sum with
// rounding and begins anew. (512 tokens over 16384, 8 bits: 357 us and off by 9.5e-7 of the output,
// a sum in fp32 steps by 2.2e-6; every 8 blocks 322 us and 2.6e-6, every block 405 us and 7.1e-7;
// without the sum over 65536 tokens 8.6e-5.)
//
// Measured (8 KV heads, groups of 4, whole calls, flops counted once a pair): 2048 tokens over
// 32768 in bf16 1106 us, 963 TFLOP/s; 1024 over 65536 in 8 bits 1260 us, 866 TFLOP/s; a prompt of
// 8192 630 us, 873 TFLOP/s; a mixed batch with pages given back, 8 bits to fp32, 179 us. In bf16
// the board's power limit lowers the clock to 1.65 GHz or so at that rate, and within a block the
// softmax waits for the products' latency; in 8 bits the widening takes half of all instructions;
// short tiles lose their ends (Q's load, the last products, the output's store).
//
// Roles, by warp: 0-3 and 4-7 softmax and output of the halves, 8 loads, 9 to 12 the halves'
// scores and products, 13 and up repair (bf16) or widening (8-bit); with one half there are four
// softmax and two product warps. They meet in mbarriers; every wait gives up after kWaitLimitNs,
// which ends the whole CTA in order and reaches the caller as a status.
#include "paged_async.cuh"

namespace pkv {

namespace {

constexpr int kBlk = 128;                      // tokens of a block
constexpr int kTurn = 64;                      // tokens whose scores are worked on at a time
constexpr int kHalfB = kBlk * 128;             // 64 columns x 128 rows of bf16: one swizzled tile
constexpr int kStageB = 2 * kHalfB;            // a K, V or Q tile: 32 KB
constexpr int kRawB = kBlk * D;                // a tile of codes: 16 KB
constexpr int kRing = 8;                       // block entries between the loads and the others
constexpr float kRescale = 8.0f;               // growth of a maximum (base 2) that rescales O
constexpr int kFold = 2;                       // blocks after which O goes into its sum (fp32 output)

template <bool kE4m3, int kParts> struct Shape {
    static constexpr int kHalves = kParts == 1 ? 2 : 1;
    static constexpr int kStages = kE4m3 ? 3 : 4;
    static constexpr int kRaw = kE4m3 ? 3 : 0;
    static constexpr int kAuxWarps = kE4m3 ? (kParts == 1 ? 7 : 8) : 3;
    static constexpr int kSoft = 4 * kHalves;                 // softmax warps
    static constexpr int kAux0 = kSoft + 1 + 2 * kHalves;     // first of the others
    static constexpr int kThreads = (kAux0 + kAuxWarps) * 32;
    // tensor memory columns
    static constexpr int kS = 0;                              // + 128 half + 64 turn
    // weights of a turn: over its scores (the third part: 128 + 32 turn)
    static constexpr int kO = kParts == 1 ? 256 : 192;        // + 128 half
    static constexpr int kSum = kO + 128;                     // (three parts) O's sum so far
    static __device__ __forceinline__ constexpr int weights(int turn, int part) {
        return part < 2 ? 64 * turn + 32 * part : 128 + 32 * turn;   // + 128 half
    }
    // shared memory
    static constexpr int kQ = 0;
    static constexpr int kKV = kHalves * kStageB;
    static constexpr int kRawAt = kKV + kStages * kStageB;
    static constexpr int kScaleAt = kRawAt + kRaw * kRawB;
    static constexpr int kSmem = kScaleAt + kRaw * kBlk + 1024;   // + alignment
};

// kFirst/kLast: of a segment; kEmpty: a segment without a block; kFix: scores are masked; kTwo:
// both halves have rows; kEnd: no more entries
enum : int { kFirst = 1, kLast = 2, kEmpty = 4, kFix = 8, kTwo = 16, kEnd = 32 };

// a block on its way from the load warp to the others
struct Entry {
    int32_t block, flags;
    uint32_t mask[4];      // tokens that are there
};
// a range of one tile's blocks
struct Seg {
    int64_t pos0;          // position of the sequence's first new token
    int32_t row0, first, nrow, head;
    int32_t shared;        // last token that every row of the tile may attend
    int32_t kv;            // tokens of the sequence
    int32_t whole, part;   // output, or the slot of the unfinished part
};

struct Shared {
    uint64_t info_full[kRing], info_empty[kRing], bad_full[kRing];
    uint64_t q_full, q_empty, s_full[2][2], p_full[2][2], pv_done[2][2], o_full[2], drain[4];
    uint64_t kv_full[4], kv_empty[4], fixed[4], raw_full[4], raw_empty[4];
    Entry entry[kRing];
    Seg seg[kRing];
    int32_t bad[kRing][D];   // per segment: first token whose V is not finite in this element
    int32_t any_bad[kRing];
    uint32_t tmem;
    int32_t abort;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
__device__ __forceinline__ uint32_t bf2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t mul_bf2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// the last token that row r of a tile may attend (-1: none)
__device__ __forceinline__ int row_limit(const Seg& g, int causal, int group, int r) {
    if (r >= g.nrow) return -1;
    const int64_t lim = causal ? g.pos0 + (g.first + r) / group : g.kv - 1;
    return static_cast<int>(max64(-1, min64(lim, g.kv - 1)));
}

// The CTAs that have work. A part of a tile costs about what a block does (its 128 KB are written
// and read again), so tiles of 8 blocks and more are cut no finer than by two: 64 tokens over 2000
// take 34.6 us a call cut by single blocks and 32.3 by two, 32 tokens of one head over 20000 51.2
// and 39.6. Shorter tiles are cut by single blocks (two would often be of two tiles, one after the
// other): a prompt of 300 takes 29.4 us so, and 36.8 by two.
__device__ __forceinline__ int64_t chunk_cuts(int64_t per_head, int nt, int64_t total) {
    return cuts(per_head >= 8 * static_cast<int64_t>(nt) ? ceil_div(total, 2) : total, gridDim.x);
}

// ---------------------------------------------------------------------------------- loads
// The whole warp walks the CTA's blocks; a lane handles one page of a block.
template <bool kE4m3, int kParts>
__device__ void load_role(const AttendArgs& a, const CUtensorMap* mq, const CUtensorMap* mk,
                          const CUtensorMap* mv, Shared& sh, uint8_t* smem, int64_t x, int64_t hi,
                          int64_t per_head, int nt) {
    using S = Shape<kE4m3, kParts>;
    const int lane = threadIdx.x & 31;
    const int G = a.shape.group, shift = a.pool.shift, causal = a.shape.causal;
    const int rt = a.shape.tile_rows / S::kHalves;             // rows of a half
    const int rs = min(shift, 7), run = 1 << rs, nrun = kBlk >> rs;  // tokens a copy, copies a block
    const int ns = 7 - rs;                                     // log2(nrun)
    int64_t h = x / per_head;
    int tile = find_tile(a.plan.tile, nt, x - h * per_head);
    Tile v = a.plan.tile[tile];
    uint32_t n = 0, seg = 0, ld = 0, nq = 0;   // entries, segments, tiles loaded, Q tiles loaded
    int word_seq = -1, word0 = 0;              // the bits that are held: of which sequence, from where
    uint32_t words = 0;
    volatile int32_t* ab = &sh.abort;

    while (x < hi) {
        // the next tile's record is under way while this one is worked on
        const int64_t after = a.plan.tile[tile + 1].pre;
        const int next = tile + 1 == nt ? 0 : tile + 1;
        const Tile ahead = a.plan.tile[next];
        const int64_t start = h * per_head + v.pre, nb = after - v.pre;
        const int b0 = static_cast<int>(x - start), b1 = static_cast<int>(min64(nb, hi - start));
        Seg g;
        g.first = v.first;
        g.pos0 = v.pos0;
        g.row0 = v.row0;
        g.nrow = v.nrow;
        g.head = static_cast<int>(h);
        g.kv = v.kv;
        g.whole = b0 == 0 && b1 == nb;
        g.part = 2 * static_cast<int>(blockIdx.x) + (b0 == 0);
        g.shared = row_limit(g, causal, G, 0);
        if (seg == 0 && lane == 0) {
            const int64_t total = per_head * a.heads;
            a.cut[blockIdx.x] = cut_record(v, total, chunk_cuts(per_head, nt, total), start,
                                           after + h * per_head, b0, h);
        }
        const int end = v.end;
        const int32_t* table = a.seqs.table + static_cast<int64_t>(v.seq) * a.seqs.stride;

        // The tile's blocks [b0, b1), counting those with a page that is there. The sequence's bits
        // are held 32 words at a time, a lane a word, and stay for its next tile.
        const int blocks = static_cast<int>(ceil_div(end, kBlk)), nwords = (blocks + 31) >> 5;
        const int kv_words = static_cast<int>(ceil_div(v.kv, 32 * kBlk));
        const uint32_t* bits = a.plan.live + static_cast<int64_t>(v.seq) * a.plan.words;
        auto hold = [&](int w) {
            word0 = w;
            word_seq = v.seq;
            words = w + lane < kv_words ? bits[w + lane] : 0u;
        };
        if (word_seq != v.seq || word0 != 0) hold(0);
        int at_word = -1, left = b1 - b0;
        uint32_t rest = 0;                              // bits of that word not yet taken
        auto take = [&]() -> int {
            if (left-- <= 0) return -1;
            while (rest == 0) {
                if (++at_word >= nwords) return -1;
                if (at_word >= word0 + 32) hold(at_word);
                rest = __shfl_sync(0xffffffffu, words, at_word - word0);
                if (at_word == nwords - 1 && (blocks & 31)) rest &= (1u << (blocks & 31)) - 1;
            }
            const int b = 32 * at_word + __ffs(rest) - 1;
            rest &= rest - 1;
            return b;
        };
        if (b0 > 0) {                                   // pass the first b0
            int skip = b0, sum, total;
            while (true) {
                sum = __popc(words);
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, sum, o);
                    if (lane >= o) sum += y;
                }
                total = __shfl_sync(0xffffffffu, sum, 31);
                if (skip < total || word0 + 32 >= kv_words) break;
                skip -= total;
                hold(word0 + 32);
            }
            const int k = __popc(__ballot_sync(0xffffffffu, sum <= skip)) & 31;
            rest = __shfl_sync(0xffffffffu, words, k);
            skip -= __shfl_sync(0xffffffffu, sum, k) - __popc(rest);
            at_word = word0 + k;
            const bool it = (rest >> lane & 1) && __popc(rest & ((1u << lane) - 1)) == skip;
            const uint32_t from = __ballot_sync(0xffffffffu, it);   // one bit
            rest &= ~(from - 1);
            if (at_word == nwords - 1 && (blocks & 31)) rest &= (1u << (blocks & 31)) - 1;
        }
        // page ids come a window of blocks at a time, a lane a run, one window ahead
        const int per_win = min(8, 32 >> ns);
        auto fetch = [&](int* block) -> int {
            *block = -1;
            for (int i = 0; i < per_win; ++i) {
                const int b = take();
                if (lane >> ns == i) *block = b;
            }
            const int64_t tok = static_cast<int64_t>(*block) * kBlk + (lane & (nrun - 1)) * run;
            return *block >= 0 && tok < v.kv ? table[tok >> shift] : -1;
        };
        int block = -1, block_next = -1, at = 0;
        int id = fetch(&block), id_next = fetch(&block_next);
        uint32_t valid = 0;                             // pages of the block that are there
        int page = 0;                                   // this lane's
        auto advance = [&]() -> int {
            if (at == per_win) {
                at = 0;
                block = block_next;
                id = id_next;
                id_next = fetch(&block_next);
            }
            const uint32_t ok = __ballot_sync(
                0xffffffffu, static_cast<uint32_t>(id) < static_cast<uint32_t>(a.pool.num_pages));
            const int l0 = at++ << ns;
            valid = (ok >> l0) & ((1u << nrun) - 1);
            page = __shfl_sync(0xffffffffu, id, (l0 + lane) & 31);
            return __shfl_sync(0xffffffffu, block, l0);
        };
        int b = advance();
        bool first = true;
        while (first || b >= 0) {
            const uint32_t cur_valid = valid;
            const int cur_page = page, cur = b;
            if (b >= 0) b = advance();
            // the entry
            const int slot = n % kRing;
            if (!warp_nap(&sh.info_empty[slot], ((n / kRing) & 1) ^ 1, ab)) return;
            Entry e;
            e.block = cur;
            e.flags = (first ? kFirst : 0) | (b < 0 ? kLast : 0) | (cur < 0 ? kEmpty : 0) |
                      (S::kHalves == 2 && g.nrow > rt ? kTwo : 0);
            bool full = cur >= 0;
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                const uint32_t l = cur_valid >> (32 * f >> rs) & 1,
                               u = cur_valid >> ((32 * f + 16) >> rs) & 1;
                const int more = end - (cur * kBlk + 32 * f);
                e.mask[f] = cur < 0 || more <= 0
                                ? 0u
                                : ((l ? 0xffffu : 0u) | (u ? 0xffff0000u : 0u)) &
                                      (more >= 32 ? ~0u : (1u << more) - 1);
                full = full && e.mask[f] == ~0u;
            }
            const int last_tok = cur * kBlk + min(end - cur * kBlk, kBlk) - 1;
            if (!full || (causal && last_tok > g.shared)) e.flags |= kFix;
            if (first)
                for (int i = lane; i < D; i += 32) sh.bad[seg % kRing][i] = INT32_MAX;
            __syncwarp();
            if (lane == 0) {
                if (first) {
                    sh.seg[seg % kRing] = g;
                    sh.any_bad[seg % kRing] = 0;
                }
                sh.entry[slot] = e;
                arrive(&sh.info_full[slot]);
            }
            ++n;
            if (cur < 0) break;
            if (first) {
                if (!warp_nap(&sh.q_empty, (nq & 1) ^ 1, ab)) return;
                if (lane == 0) {
                    const int halves = e.flags & kTwo ? 2 : 1;
                    mbar_arrive_expect_tx(smem_addr(&sh.q_full), halves * 2 * rt * 128);
                    for (int i = 0; i < halves; ++i)
                        for (int c = 0; c < 2; ++c)
                            tma_load3(smem_addr(smem + S::kQ + i * kStageB + c * kHalfB), mq, 64 * c,
                                      g.head * G, g.row0 + (g.first + i * rt) / G,
                                      smem_addr(&sh.q_full));
                }
                ++nq;
            }
            first = false;
            // K, then V
            const bool mine = lane < nrun && (cur_valid >> lane & 1);
            const int row = (g.head << shift) + ((cur * kBlk + lane * run) & ((1 << shift) - 1));
            for (int t = 0; t < 2; ++t) {
                constexpr int kSlots = kE4m3 ? S::kRaw : S::kStages;
                const int st = ld % kSlots;
                // bf16 rows that are looked over before they are used land for those who do that
                const bool look = !kE4m3 && t == 1 && (e.flags & kFix);
                uint64_t* full_bar = kE4m3 || look ? &sh.raw_full[st] : &sh.kv_full[st];
                if (!warp_nap(kE4m3 ? &sh.raw_empty[st] : &sh.kv_empty[st],
                              ((ld / kSlots) & 1) ^ 1, ab))
                    return;
                if (lane == 0) {
                    mbar_arrive_expect_tx(smem_addr(full_bar),
                                          __popc(cur_valid) * run * (kE4m3 ? D + 1 : 2 * D));
                    if (look) arrive(&sh.kv_full[st]);
                }
                __syncwarp();
                if (mine) {
                    const CUtensorMap* m = t ? mv : mk;
                    if (kE4m3) {
                        tma_load3(smem_addr(smem + S::kRawAt + st * kRawB + lane * run * D), m, 0,
                                  row, cur_page, smem_addr(full_bar));
                        bulk_g2s(smem_addr(smem + S::kScaleAt + st * kBlk + lane * run),
                                 (t ? a.pool.vs : a.pool.ks) + cur_page * a.pool.scale_stride + row,
                                 run, smem_addr(full_bar));
                    } else {
                        uint8_t* dst = smem + S::kKV + st * kStageB + lane * run * 128;
                        tma_load3(smem_addr(dst), m, 0, row, cur_page, smem_addr(full_bar));
                        tma_load3(smem_addr(dst + kHalfB), m, 64, row, cur_page, smem_addr(full_bar));
                    }
                }
                ++ld;
            }
        }
        ++seg;
        x = start + b1;
        h += next == 0 ? 1 : 0;   // (a range that ends inside the tile is the last)
        tile = next;
        v = ahead;
    }
    // the end: an entry without a segment
    const int slot = n % kRing;
    if (!warp_nap(&sh.info_empty[slot], ((n / kRing) & 1) ^ 1, ab)) return;
    if (lane == 0) {
        sh.entry[slot].flags = kEnd;
        sh.entry[slot].block = -1;
        arrive(&sh.info_full[slot]);
    }
}

// ------------------------------------------------------------------------------- products
// Two warps a half, one for the scores and one for the weights' product: what each waits for and
// looks up (some 100 cycles a wait) hides behind the other three's products. A whole warp keeps
// the books (the compiler then sees uniform values); one elected thread issues. A block is taken
// in two turns of 64 tokens, each with its own columns of S and P, and the scores of a turn are
// issued as soon as the weights of the turn two before it have been used: the softmax never waits
// for the products' latency. (Scores of 64 tokens cost 1.5 times their share of 128 tokens' - Q is
// read from shared memory for half as many columns - which is less than the waits were.)

// The flags of the next block with work and kSome, 0 at the end, -1 after a wait ran out.
constexpr int kSome = 64;
__device__ __forceinline__ int next_block(Shared& sh, uint32_t& n, bool leader) {
    while (true) {
        const int slot = n % kRing;
        if (!warp_wait(&sh.info_full[slot], (n / kRing) & 1, &sh.abort)) return -1;
        const int f = uniform(static_cast<uint32_t>(sh.entry[slot].flags));
        const int b = uniform(static_cast<uint32_t>(sh.entry[slot].block));
        if (leader) arrive(&sh.info_empty[slot]);
        ++n;
        if (b >= 0) return f | kSome;
        if (f & kEnd) return 0;
    }
}

template <bool kE4m3, int kParts>
__device__ void score_role(Shared& sh, uint8_t* smem, uint32_t tmem, int half, bool inject) {
    using S = Shape<kE4m3, kParts>;
    constexpr uint32_t kQK = mma_desc(kTurn, false);
    volatile int32_t* ab = &sh.abort;
    const bool leader = elect_one();
    const uint64_t q_desc = smem_desc(uniform(smem_addr(smem + S::kQ + half * kStageB)), 16);
    const uint64_t k_desc = smem_desc(uniform(smem_addr(smem + S::kKV)), 16);
    const uint32_t s_at = uniform(tmem + S::kS + 128 * half);
    if (inject) {   // test hook: a wait for an arrival that never comes
        wait_for(&sh.raw_empty[3], 0, ab, 1000000ull);
        return;
    }
    uint32_t n = 0, nq = 0, nb = 0, used = 0;   // entries, Q tiles, blocks of the half, K/V tiles
#pragma unroll 1
    while (true) {
        const int flags = next_block(sh, n, leader);
        if (flags <= 0) return;
        const int st = used % S::kStages;
        if ((flags & kFirst) && !warp_wait(&sh.q_full, nq++ & 1, ab)) return;
        if (!warp_wait(&sh.kv_full[st], (used / S::kStages) & 1, ab)) return;
        const bool mine = half == 0 || (flags & kTwo);
        const uint64_t k0 = k_desc + st * (kStageB >> 4);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            if (mine) {
                // they go where the weights of the same turn of the last block were read
                if (nb > 0 && !warp_wait(&sh.pv_done[half][w], (nb - 1) & 1, ab)) return;
                tc_fence_after();
#pragma unroll
                for (int j = 0; j < D / 16; ++j) {
                    const uint32_t at = ((j >> 2) * kHalfB + (j & 3) * 32) >> 4;
                    mma_ss(leader, s_at + kTurn * w, q_desc + at, k0 + (w * kTurn * 128 >> 4) + at, kQK,
                           j > 0);
                }
                mma_commit(leader, smem_addr(&sh.s_full[half][w]));
            }
        }
        mma_commit(leader, smem_addr(&sh.kv_empty[st]));
        if (flags & kLast) mma_commit(leader, smem_addr(&sh.q_empty));
        __syncwarp();
        nb += mine ? 1 : 0;
        used += 2;
    }
}

template <bool kE4m3, int kParts>
__device__ void weight_role(Shared& sh, uint8_t* smem, uint32_t tmem, int half) {
    using S = Shape<kE4m3, kParts>;
    constexpr uint32_t kPV = mma_desc(D, true);
    volatile int32_t* ab = &sh.abort;
    const bool leader = elect_one();
    const uint64_t v_desc = smem_desc(uniform(smem_addr(smem + S::kKV)), kHalfB);
    const uint32_t o_at = uniform(tmem + S::kO + 128 * half), p_at = uniform(tmem + 128 * half);
    uint32_t n = 0, nb = 0, used = 1, fix = 0, run = 0;   // run: blocks of the tile
#pragma unroll 1
    while (true) {
        const int flags = next_block(sh, n, leader);
        if (flags <= 0) return;
        const int st = used % S::kStages;
        if (!warp_wait(&sh.kv_full[st], (used / S::kStages) & 1, ab)) return;
        if (!kE4m3 && (flags & kFix)) {
            if (!warp_wait(&sh.fixed[st], fix >> st & 1, ab)) return;
            fix ^= 1u << st;
        }
        const bool mine = half == 0 || (flags & kTwo);
        const uint64_t v0 = v_desc + st * (kStageB >> 4);
        run = flags & kFirst ? 0 : run + 1;
        const bool anew = kParts == 1 ? flags & kFirst : run % kFold == 0;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            if (mine) {
                if (!warp_wait(&sh.p_full[half][w], nb & 1, ab)) return;
                tc_fence_after();
#pragma unroll
                for (int p = 0; p < kParts; ++p)
#pragma unroll
                    for (int j = 0; j < kTurn / 16; ++j)
                        mma_ts(leader, o_at, p_at + S::weights(w, p) + 8 * j,
                               v0 + ((w * kTurn * 128 + j * 16 * 128) >> 4), kPV,
                               !anew || w > 0 || p > 0 || j > 0);
                mma_commit(leader, smem_addr(&sh.pv_done[half][w]));
                if ((flags & kLast) && w == 1) mma_commit(leader, smem_addr(&sh.o_full[half]));
            }
        }
        mma_commit(leader, smem_addr(&sh.kv_empty[st]));
        __syncwarp();
        nb += mine ? 1 : 0;
        used += 2;
    }
}

// ----------------------------------------------------------------- softmax and the output
// 128 columns of a thread's row: to = O, or O and what is in the sum (out of line: the softmax's
// loop is what the instruction cache is for)
__device__ __noinline__ void fold(uint32_t to, uint32_t at, uint32_t sum, bool kept) {
#pragma unroll 1
    for (int i = 0; i < 128; i += 16) {
        uint32_t o[16], x[16];
        tmem_ld16(at + i, o);
        tmem_ld16(sum + i, x);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 16; ++k)
            o[k] = __float_as_uint(__uint_as_float(o[k]) + (kept ? __uint_as_float(x[k]) : 0.0f));
        tmem_st16(to + i, o);
    }
    tmem_wait_st();
}

// A warpgroup a half, a thread a row.
template <bool kE4m3, int kParts, typename Out>
__device__ void softmax_role(const AttendArgs& a, Shared& sh, uint32_t tmem, int half) {
    using S = Shape<kE4m3, kParts>;
    const int quad = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
    const int G = a.shape.group, R = a.shape.tile_rows, rt = R / S::kHalves;
    const int rl = 32 * quad + lane;                            // row of the half
    const int r = rl < rt ? half * rt + rl : INT32_MAX;         // row of the tile
    const uint32_t at0 = tmem + (quad << 21) + 128 * half;
    volatile int32_t* ab = &sh.abort;
    // scores times a positive factor c, after a sign (negative scales) or zero (scale 0)
    const float c = a.scale == 0.0f ? 1.0f : fabsf(a.scale) * kLog2e;
    const float sign = a.scale > 0.0f ? 1.0f : a.scale < 0.0f ? -1.0f : 0.0f;

    uint32_t n = 0, seg = 0, nt = 0, no = 0;   // entries, segments; turns, outputs of this half
    float m = -INFINITY, l = 0.0f;      // the row's maximum (times c) as last used, and its sum
    int lim = -1;
    uint32_t run = 0;                   // blocks of the tile (fp32 output)
    while (true) {
        const int slot = n % kRing;
        if (!warp_wait(&sh.info_full[slot], (n / kRing) & 1, ab)) return;
        const int flags = sh.entry[slot].flags, block = sh.entry[slot].block;
        if (flags & kEnd) return;
        const Seg& g = sh.seg[seg % kRing];
        if (flags & kFirst) {
            lim = row_limit(g, a.shape.causal, G, r);
            m = -INFINITY;
            l = 0.0f;
            run = 0;
        }
        const bool mine = half == 0 || (flags & kTwo);
        if (mine && !(flags & kEmpty)) {
#pragma unroll 1
            for (int w = 0; w < 2; ++w, ++nt) {
                const int turn = nt & 1;
                if (kParts > 1 && w == 0 && run > 0 && run % kFold == 0) {
                    // (after the products into O of all turns so far)
                    if (!warp_wait(&sh.pv_done[half][turn ^ 1], (nt - 1) >> 1 & 1, ab)) return;
                    tc_fence_after();
                    fold(at0 + S::kSum, at0 + S::kO, at0 + S::kSum, run > kFold);
                }
                if (!warp_wait(&sh.s_full[half][turn], nt >> 1 & 1, ab)) return;
                tc_fence_after();
                uint32_t s[kTurn];
                tmem_ld32(at0 + S::kS + kTurn * turn, s);
                tmem_ld32(at0 + S::kS + kTurn * turn + 32, s + 32);
                tmem_wait_ld();
                if (__builtin_expect(sign != 1.0f, 0)) {
#pragma unroll
                    for (int i = 0; i < kTurn; ++i)
                        s[i] = __float_as_uint(__uint_as_float(s[i]) * sign);
                }
                if (__builtin_expect(flags & kFix, 0)) {
                    const int left = lim - block * kBlk - kTurn * w + 1;   // up to the row's limit
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                        const int k = left - 32 * f;
                        const uint32_t seen = k <= 0 ? 0u
                                                     : sh.entry[slot].mask[2 * w + f] &
                                                           (k >= 32 ? ~0u : (1u << k) - 1);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!(seen >> i & 1)) s[32 * f + i] = 0xff800000u;
                    }
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < kTurn; i += 8)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mx[k] = max3(mx[k], __uint_as_float(s[i + 2 * k]),
                                     __uint_as_float(s[i + 2 * k + 1]));
                const float top = max3(mx[0], mx[1], fmaxf(mx[2], mx[3])) * c;
                if ((flags & kFirst) && w == 0) {
                    m = top;
                } else if (__builtin_expect(__any_sync(0xffffffffu, top > m + kRescale), 0)) {
                    const float m1 = top > m + kRescale ? top : m;
                    const float f = m1 == -INFINITY ? 1.0f : ex2(m - m1);
                    m = m1;
                    l *= f;
                    // the last product into O has to be there before it is rescaled (the one
                    // before it is: its weights' columns hold these scores)
                    if (!warp_wait(&sh.pv_done[half][turn ^ 1], (nt - 1) >> 1 & 1, ab)) return;
                    tc_fence_after();
                    const int cols = kParts > 1 && run >= kFold ? 256 : 128;   // the sum too
#pragma unroll 1
                    for (int i = 0; i < cols; i += 16) {
                        uint32_t o[16];
                        tmem_ld16(at0 + S::kO + i, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                        tmem_st16(at0 + S::kO + i, o);
                    }
                }
                const float ms = m == -INFINITY ? 0.0f : m;
                const uint64_t c2 = pack2(c, c), m2 = pack2(-ms, -ms);
                uint64_t sum[2] = {0, 0};
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    float p[32];
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float2 y = unpack2(
                            fma2(pack2u(s[32 * q + i], s[32 * q + i + 1]), c2, m2));
                        p[i] = ex2(y.x);
                        p[i + 1] = ex2(y.y);
                        sum[(i >> 1) & 1] = add2(sum[(i >> 1) & 1], pack2(p[i], p[i + 1]));
                    }
#pragma unroll
                    for (int k = 0; k < kParts; ++k) {
                        uint32_t x[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            x[i] = bf2(p[2 * i], p[2 * i + 1]);
                            if (k + 1 < kParts) {
                                p[2 * i] -= lo_f(x[i]);
                                p[2 * i + 1] -= hi_f(x[i]);
                            }
                        }
                        tmem_st16(at0 + S::weights(turn, k) + 16 * q, x);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive(&sh.p_full[half][turn]);
                const float2 y = unpack2(add2(sum[0], sum[1]));
                l += y.x + y.y;
            }
            ++run;
        }
        if (flags & kLast) {
            if (mine) {
                const bool empty = flags & kEmpty;
                if (!empty) {
                    if (!warp_wait(&sh.o_full[half], no++ & 1, ab)) return;
                    tc_fence_after();
                    if (kParts > 1 && run > kFold)
                        fold(at0 + S::kO, at0 + S::kO, at0 + S::kSum, true);
                }
                if (!warp_wait(&sh.bad_full[seg % kRing], (seg / kRing) & 1, ab)) return;
                const bool bad = sh.any_bad[seg % kRing] != 0;
                const bool live = r < g.nrow;
                const float inv = !g.whole ? 1.0f : l == 0.0f ? 0.0f : 1.0f / l;
                const int rr = g.first + (live ? r : 0);
                const int64_t at = (g.row0 + rr / G) * (static_cast<int64_t>(a.heads) * G) +
                                   g.head * G + rr % G;
                float* part = a.work + g.part * part_floats(R);
                const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
                // 32 columns at a time; a thread's 64 or 128 bytes of a row in whole sectors
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    const int col = 32 * q;
                    uint32_t o[32];
                    if (!empty) {
                        tmem_ld32(at0 + S::kO + col, o);
                        tmem_wait_ld();
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float y = empty ? 0.0f : __uint_as_float(o[i]) * inv;
                        o[i] = __float_as_uint(y);
                    }
                    if (__builtin_expect(bad, 0)) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (sh.bad[seg % kRing][col + i] <= lim) o[i] = 0x7fc00000u;
                    }
                    if (live && g.whole && sizeof(Out) == 2) {
                        uint32_t u[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            u[i] = bf2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1]));
                        store_words<16>(static_cast<__nv_bfloat16*>(a.out) + at * D + col, u, wide);
                    } else if (live) {
                        store_words<32>(g.whole ? static_cast<float*>(a.out) + at * D + col
                                                : part + static_cast<size_t>(r) * D + col,
                                        o, wide && g.whole);
                    }
                    __syncwarp();
                }
                if (live && g.whole && a.lse)
                    a.lse[at] = l == 0.0f ? -INFINITY : m * kLn2 + logf(l);
                if (live && !g.whole) {
                    part[static_cast<size_t>(R) * D + r] = m;
                    part[static_cast<size_t>(R) * D + R + r] = l;
                }
                tc_fence_before();
            }
            ++seg;
        }
        __syncwarp();
        if (lane == 0) arrive(&sh.info_empty[slot]);
        ++n;
    }
}

// ---------------------------------------------------------------- repair, and widening
template <bool kE4m3, int kParts>
__device__ void aux_role(const AttendArgs& a, Shared& sh, uint8_t* smem) {
    using S = Shape<kE4m3, kParts>;
    const int tid = threadIdx.x - S::kAux0 * 32, lane = tid & 31;
    volatile int32_t* ab = &sh.abort;
    uint32_t n = 0, seg = 0, use = 0;   // use: tiles of the ring seen
    uint32_t looked = 0;                // a bit a stage: parity of the looks at it (bf16)
    // (8-bit: this thread's places in a tile of codes and in a tile of bf16)
    const int j = lane & 3, odd = lane >> 2 & 1;
    const int in0 = 16 * (j + 4 * odd), in1 = 16 * (j + 4 - 4 * odd);
    const int at_row = ((2 * j) ^ (lane >> 2)) << 4;
    const int out0 = odd * kHalfB + at_row, out1 = (1 - odd) * kHalfB + at_row;
    int turn = tid >> 5;
    while (true) {
        const int slot = n % kRing;
        if (!warp_nap(&sh.info_full[slot], (n / kRing) & 1, ab)) return;
        const int flags = sh.entry[slot].flags, block = sh.entry[slot].block;
        if (flags & kEnd) return;
        const int sg = seg % kRing;
        const int shared = sh.seg[sg].shared;
        auto mark = [&](int d, int tok) {
            atomicMin(&sh.bad[sg][d], tok);
            sh.any_bad[sg] = 1;
        };
        if (!(flags & kEmpty)) {
            if constexpr (kE4m3) {
                for (int t = 0; t < 2; ++t) {
                    const int raw = use % S::kRaw, st = use % S::kStages;
                    if (!warp_nap(&sh.raw_full[raw], (use / S::kRaw) & 1, ab)) return;
                    if (!warp_nap(&sh.kv_empty[st], ((use / S::kStages) & 1) ^ 1, ab)) return;
                    // A warp takes 8 rows at a time, 4 lanes a row, a lane its pieces of 16 codes j
                    // and j + 4 (odd rows the other way round): in every access 8 lanes meet no
                    // bank twice. Which warp takes a piece more moves on from tile to tile.
                    const uint8_t* src = smem + S::kRawAt + raw * kRawB;
                    const uint8_t* sc = smem + S::kScaleAt + raw * kBlk;
                    uint8_t* dst = smem + S::kKV + st * kStageB;
#pragma unroll 1
                    for (int g = turn; g < kBlk / 8; g += S::kAuxWarps) {
                        const int row = 8 * g + (lane >> 2), byte = sc[row];
                        // code * 2^(byte - 127): the bf16 patterns are 2^-120 too small; the
                        // factor 2^(byte - 7) takes two steps where it is above 2^127
                        uint32_t f = static_cast<uint32_t>(min(byte + 120, 254)) << 7;
                        if (byte == kNanRow) f = 0x7fc0u;
                        f |= f << 16;
                        bool zero = false;
                        if (__builtin_expect(flags & kFix, 0)) {
                            const int tok = block * kBlk + row;
                            zero = !(sh.entry[slot].mask[row >> 5] >> (row & 31) & 1);
                            if (t == 1 && !zero && byte == kNanRow && tok > shared) {
#pragma unroll 1
                                for (int k = 0; k < D; k += 4) mark(k + j, tok);
                                zero = true;
                            }
                        }
#pragma unroll
                        for (int p = 0; p < 2; ++p) {
                            const uint4 w4 =
                                *reinterpret_cast<const uint4*>(src + row * D + (p ? in1 : in0));
                            const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
                            uint32_t y[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                const uint32_t x = k & 1 ? prmt_i<0x3424>(w[k >> 1], 0)
                                                         : prmt_i<0x1404>(w[k >> 1], 0);
                                y[k] = mul_bf2((x & 0x80008000u) | ((x >> 4) & 0x07f007f0u), f);
                            }
                            if (__builtin_expect(zero || (byte > 134 && byte != kNanRow), 0)) {
                                const uint32_t f2 = static_cast<uint32_t>(byte - 134 + 127) << 7;
#pragma unroll
                                for (int k = 0; k < 8; ++k)
                                    y[k] = zero ? 0u : mul_bf2(y[k], f2 | f2 << 16);
                            }
                            uint8_t* to = dst + row * 128;
                            const int c = p ? out1 : out0;
                            *reinterpret_cast<uint4*>(to + c) = make_uint4(y[0], y[1], y[2], y[3]);
                            *reinterpret_cast<uint4*>(to + (c ^ 16)) =
                                make_uint4(y[4], y[5], y[6], y[7]);
                        }
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        arrive(&sh.kv_full[st]);
                        arrive(&sh.raw_empty[raw]);
                    }
                    ++use;
                    turn += (S::kAuxWarps - kBlk / 8 % S::kAuxWarps) % S::kAuxWarps;
                    turn -= turn >= S::kAuxWarps ? S::kAuxWarps : 0;
                }
            } else {
                const int st = (use + 1) % S::kStages;
                if (flags & kFix) {
                    // (a barrier of their own, waited for at each of its phases: a wait for a phase
                    // of kv_full, of which some are passed over, could be answered for the one
                    // two before it)
                    if (!warp_nap(&sh.raw_full[st], looked >> st & 1, ab)) return;
                    looked ^= 1u << st;
                    // rows from the first one that needs a look: all past `shared`, and all of a
                    // block that is not whole; a warp takes 4 rows of 64 columns at a time, 4
                    // such pieces in flight
                    bool full = true;
                    for (int f = 0; f < 4; ++f) full = full && sh.entry[slot].mask[f] == ~0u;
                    const int row0 = full ? max(0, shared + 1 - block * kBlk) & ~3 : 0;
                    uint8_t* tile = smem + S::kKV + st * kStageB;
                    const int warp = tid >> 5, npc = 2 * (kBlk - row0) / 4;
                    for (int pc = warp; pc < npc; pc += 4 * S::kAuxWarps) {
                        uint4 v[4];
                        uint4* at[4];
                        int tok[4], d[4];
                        bool there[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const int p = pc + u * S::kAuxWarps;
                            const int half = p & 1, row = row0 + 4 * (p >> 1) + (lane >> 3);
                            const bool in = p < npc;
                            at[u] = reinterpret_cast<uint4*>(tile + half * kHalfB +
                                                             (in ? row : 0) * 128 + (lane & 7) * 16);
                            tok[u] = in ? block * kBlk + row : -1;
                            d[u] = half * 64 + ((lane & 7) ^ (row & 7)) * 8;
                            there[u] = !in || (sh.entry[slot].mask[row >> 5] >> (row & 31) & 1);
                            v[u] = *at[u];
                        }
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            if (!there[u]) {
                                *at[u] = make_uint4(0, 0, 0, 0);
                                continue;
                            }
                            // an exponent of all ones carries into the (cleared) sign bit
                            uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w}, odd = 0;
#pragma unroll
                            for (int k = 0; k < 4; ++k) odd |= (w[k] & 0x7f807f80u) + 0x00800080u;
                            if (!(odd & 0x80008000u) || tok[u] <= shared) continue;
                            for (int k = 0; k < 4; ++k) {
                                if ((w[k] & 0x7f80u) == 0x7f80u) {
                                    mark(d[u] + 2 * k, tok[u]);
                                    w[k] &= 0xffff0000u;
                                }
                                if ((w[k] & 0x7f800000u) == 0x7f800000u) {
                                    mark(d[u] + 2 * k + 1, tok[u]);
                                    w[k] &= 0xffffu;
                                }
                            }
                            *at[u] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) arrive(&sh.fixed[st]);
                }
                use += 2;
            }
        }
        __syncwarp();
        if (lane == 0) {
            if (flags & kLast) arrive(&sh.bad_full[sg]);
            arrive(&sh.info_empty[slot]);
        }
        if (flags & kLast) ++seg;
        ++n;
    }
}

template <bool kE4m3, int kParts, typename Out>
__global__ void __launch_bounds__(Shape<kE4m3, kParts>::kThreads, 1)
attend_chunk_kernel(const AttendArgs a, const __grid_constant__ CUtensorMap mq,
                    const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
    using S = Shape<kE4m3, kParts>;
    extern __shared__ uint8_t raw_smem[];
    __shared__ __align__(16) Shared sh;
    uint8_t* smem = raw_smem + ((1024 - (smem_addr(raw_smem) & 1023)) & 1023);
    const int warp = uniform(threadIdx.x >> 5);   // (known to be the same in a warp)
    if (threadIdx.x == 0) {
        sh.abort = 0;
        auto init = [&](uint64_t* b, uint32_t count) { mbar_init(smem_addr(b), count); };
        for (int i = 0; i < kRing; ++i) {
            init(&sh.info_full[i], 1);
            init(&sh.info_empty[i], S::kSoft + 2 * S::kHalves + S::kAuxWarps);
            init(&sh.bad_full[i], S::kAuxWarps);
        }
        init(&sh.q_full, 1);
        init(&sh.q_empty, S::kHalves);
        for (int i = 0; i < 2; ++i) {
            for (int k = 0; k < 2; ++k) {
                init(&sh.s_full[i][k], 1);
                init(&sh.pv_done[i][k], 1);
                init(&sh.p_full[i][k], 4);
            }
            init(&sh.o_full[i], 1);
            init(&sh.drain[2 * i], 1);
            init(&sh.drain[2 * i + 1], 1);
        }
        for (int i = 0; i < 4; ++i) {
            init(&sh.kv_full[i], kE4m3 ? S::kAuxWarps : 1);
            init(&sh.kv_empty[i], S::kHalves);
            init(&sh.fixed[i], S::kAuxWarps);
            init(&sh.raw_full[i], 1);
            init(&sh.raw_empty[i], S::kAuxWarps);
        }
        mbar_fence_init();
        tma_prefetch_map(&mq);
        tma_prefetch_map(&mk);
        tma_prefetch_map(&mv);
    }
    if (warp == S::kSoft + 1) {
        tmem_alloc(smem_addr(&sh.tmem), 512);
        tmem_relinquish();
    }
    // (everything up to here needs nothing of the plan)
    pdl_wait();
    pdl_launch_dependents();
    const int nt = *a.plan.ntiles;
    const int64_t per_head = a.plan.tile[nt].pre, total = per_head * a.heads;
    const int64_t ncut = chunk_cuts(per_head, nt, total);
    const bool work = blockIdx.x < ncut;
    const int64_t x = work ? cut(total, ncut, blockIdx.x) : 0;
    const int64_t hi = work ? cut(total, ncut, blockIdx.x + 1) : 0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&sh.tmem);

    if (!work) {
        // nothing to do but to give the tensor memory back
        if (threadIdx.x == 0) a.cut[blockIdx.x].parts = 0;
    } else if (warp < S::kSoft) {
        softmax_role<kE4m3, kParts, Out>(a, sh, tmem, warp >> 2);
    } else if (warp == S::kSoft) {
        load_role<kE4m3, kParts>(a, &mq, &mk, &mv, sh, smem, x, hi, per_head, nt);
    } else if (warp < S::kAux0) {
        const int i = warp - S::kSoft - 1, half = i >> 1;
        if (i & 1)
            weight_role<kE4m3, kParts>(sh, smem, tmem, half);
        else
            score_role<kE4m3, kParts>(sh, smem, tmem, half, a.inject_wait);
        // nothing may be under way in tensor memory when it is given back
        __syncwarp();
        mma_commit(elect_one(), smem_addr(&sh.drain[i]));
        int32_t no = 0;
        warp_wait(&sh.drain[i], 0, &no);
    } else {
        aux_role<kE4m3, kParts>(a, sh, smem);
    }
    tc_fence_before();
    __syncthreads();
    if (sh.abort && warp == S::kSoft && (threadIdx.x & 31) == 0) {
        // copies that were under way when a wait ran out write into this CTA's memory: give them
        // the time that any of them takes before the CTA ends
        const uint64_t t0 = now_ns();
        while (now_ns() - t0 < 10000000ull) {}
    }
    __syncthreads();
    if (warp == S::kSoft + 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <bool kE4m3, int kParts, typename Out>
cudaError_t launch_chunk(const AttendArgs& a, const CUtensorMap maps[3], int ctas, cudaStream_t st) {
    using S = Shape<kE4m3, kParts>;
    static std::atomic<uint64_t> done{0};
    auto kernel = attend_chunk_kernel<kE4m3, kParts, Out>;
    const cudaError_t e = raise_smem_limit(kernel, S::kSmem, done);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3(ctas), dim3(S::kThreads), S::kSmem, st, a, maps[0], maps[1],
                      maps[2]);
}

}  // namespace

int chunk_tile_rows(int group, bool f32_out) { return (f32_out ? 1 : 2) * (128 / group) * group; }

cudaError_t launch_attend_chunk(const AttendArgs& a, int format, bool f32_out, int ctas,
                                cudaStream_t st) {
    const bool e4 = format == PARISKV_PAGES_E4M3;
    const int G = a.shape.group;
    const uint64_t rows = static_cast<uint64_t>(a.heads) << a.pool.shift;
    const uint32_t run = min(1 << a.pool.shift, kBlk);
    const uint64_t el = e4 ? 1 : 2;
    CUtensorMap maps[3];
    if (!encode_rows(&maps[0], a.q, false, true, static_cast<uint64_t>(a.heads) * G,
                     a.seqs.total_q, 2 * D, a.q_ld * 2, 64, G, 128 / G))
        return cudaErrorInvalidValue;
    for (int t = 0; t < 2; ++t)
        if (!encode_rows(&maps[1 + t], t ? a.pool.v : a.pool.k, e4, !e4, rows, a.pool.num_pages,
                         el * D, a.pool.page_bytes, e4 ? D : 64, run, 1))
            return cudaErrorInvalidValue;
    if (e4)
        return f32_out ? launch_chunk<true, 3, float>(a, maps, ctas, st)
                       : launch_chunk<true, 1, __nv_bfloat16>(a, maps, ctas, st);
    return f32_out ? launch_chunk<false, 3, float>(a, maps, ctas, st)
                   : launch_chunk<false, 1, __nv_bfloat16>(a, maps, ctas, st);
}

cudaError_t take_chunk_waits_out(bool* out, cudaStream_t st) { return take_waits_out(out, st); }

}  // namespace pkv
