// paged.cuh -- what the paged-cache kernels share: the device view of the pages and of a chunk
// of new tokens, the scale arithmetic of the 8-bit rows, and the plan that spreads an
// attention's work evenly over the CTAs.
#pragma once

#include "common.cuh"
#include "internal.hpp"
#include "pariskv_paged.h"

namespace pkv {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ---- 8-bit rows: element = code * 2^(byte - 127), byte 255 marks a row that is NaN ----
constexpr int kMinExp = -120, kMaxExp = 119;
constexpr uint8_t kNanRow = 255;

// Scale byte of a row by its largest magnitude (finite): the least e with amax <= 448 * 2^e.
// 448 = 1.75 * 2^8: with amax = m * 2^x, 1 <= m < 2, that is x - 8 for m <= 1.75, else x - 7;
// the addition carries into the exponent exactly when the mantissa is above 1.75. Subnormal
// amax fall under the clamp.
__device__ __forceinline__ int scale_byte(float amax) {
    const int e = static_cast<int>((__float_as_uint(amax) + 0x1fffffu) >> 23) - 127 - 8;
    return min(max(e, kMinExp), kMaxExp) + 127;
}
// 2^e for e in [-126, 127]
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }
// the value of a scale byte (bytes a write leaves lie in [7, 246]; 0 only marks unread rows)
__device__ __forceinline__ float scale_value(uint32_t byte) {
    return byte == kNanRow ? __uint_as_float(0x7fc00000u) : __uint_as_float(byte << 23);
}

// kN words to memory, 32 bytes a store where the address is a multiple of 32 (else 16)
template <int kN>
__device__ __forceinline__ void store_words(void* dst, const uint32_t* w, bool wide) {
#pragma unroll
    for (int i = 0; i < kN; i += 8) {
        uint32_t* d = static_cast<uint32_t*>(dst) + i;
        const uint32_t* x = w + i;
        if (wide) {
            asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                         :: "l"(d), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]),
                            "r"(x[5]), "r"(x[6]), "r"(x[7]) : "memory");
        } else {
            reinterpret_cast<uint4*>(d)[0] = make_uint4(x[0], x[1], x[2], x[3]);
            reinterpret_cast<uint4*>(d)[1] = make_uint4(x[4], x[5], x[6], x[7]);
        }
    }
}

// ---- device views ----
struct PagePool {
    uint8_t* k;
    uint8_t* v;
    uint8_t* ks;
    uint8_t* vs;
    int64_t page_bytes;    // between pages of k and v
    int64_t scale_stride;
    int32_t num_pages;
    int32_t shift;         // log2(page_size)
};
struct Seqs {
    const int32_t* table;
    const int32_t* kv_len;
    const int32_t* q_start;
    int32_t total_q, width, stride, max_q, batch;
};

// One sequence's part of a chunk. rows: new tokens that are worked on, from row0 of the
// per-token arrays on; token j is at position pos0 + j; kv: tokens the table can hold.
struct SeqView {
    int32_t row0, rows;
    int64_t pos0;
    int32_t kv;
};
__device__ __forceinline__ SeqView seq_view(const Seqs& c, int shift, int s) {
    const int32_t a = c.q_start[s], b = c.q_start[s + 1], n = c.kv_len[s];
    SeqView v;
    v.row0 = a;
    const int64_t len = static_cast<int64_t>(b) - a;
    // rows outside the per-token arrays are never touched, whatever q_start holds
    v.rows = a < 0 ? 0
                   : static_cast<int32_t>(max64(
                         0, min64(min64(len, c.max_q), static_cast<int64_t>(c.total_q) - a)));
    v.pos0 = n - max64(0, len);
    v.kv = static_cast<int32_t>(min64(max(n, 0), static_cast<int64_t>(c.width) << shift));
    return v;
}

// ---- the plan of an attention ----
// A tile is up to `tile_rows` query rows of one sequence (row = token * group + head of the
// group); its cost is the number of KV blocks its rows can see (at least 1, so that rows which
// see nothing are still written). The tiles of all sequences, once per KV head, form one axis
// of `heads * blocks` blocks which is cut into equal ranges, one per CTA, whatever the lengths
// of the sequences are. A tile that a cut goes through is computed in parts (unnormalised
// accumulators, maxima and sums in the workspace) which a second kernel joins in order.
struct __align__(16) Tile {
    int64_t pre;       // blocks of the tiles before this one (entry ntiles: of all)
    int64_t pos0;      // position of the sequence's first new token
    int32_t seq;
    int32_t row0;      // its row in the per-token arrays
    int32_t first;     // first row of the tile within the sequence (row = token * group + head)
    int32_t nrow;      // rows of the tile
    int32_t end;       // tokens [0, end) are all that its rows may see
    int32_t kv;        // tokens of the sequence
    int32_t pad[2];
};
struct Plan {
    Tile* tile;        // [max_tiles + 1]
    int32_t* ntiles;   // [1]
    int32_t max_tiles;
    // a bit a block and sequence, [batch][words]: some page of it is there. With it (not NULL) a
    // tile's cost is the number of those blocks, and its range of blocks counts them alone.
    uint32_t* live;
    int32_t words;
};
struct PlanShape {
    int32_t group, tile_rows, block;   // block: tokens of a KV block
    int32_t causal;
};

// the tokens [0, end) that rows [row, row + tile_rows) of a sequence can see at most
__device__ __forceinline__ int32_t tile_end(const SeqView& v, const PlanShape& p, int32_t row) {
    if (!p.causal) return v.kv;
    const int64_t last = min64(static_cast<int64_t>(v.rows) * p.group,
                               static_cast<int64_t>(row) + p.tile_rows) - 1;
    return static_cast<int32_t>(max64(0, min64(v.kv, v.pos0 + last / p.group + 1)));
}
__device__ __forceinline__ int32_t tile_blocks(const SeqView& v, const PlanShape& p, int32_t row) {
    return max(1, static_cast<int32_t>(ceil_div(tile_end(v, p, row), p.block)));
}

// Of `ctas` CTAs, cuts(total, ctas) have work (one block each at least); CTA c of n works on blocks
// [cut(c), cut(c + 1)) of `total`; cut_of is the CTA of a block.
__device__ __forceinline__ int64_t cuts(int64_t total, int64_t ctas) { return min64(total, ctas); }
__device__ __forceinline__ int64_t cut(int64_t total, int64_t n, int64_t c) {
    return total * c / n;
}
__device__ __forceinline__ int64_t cut_of(int64_t total, int64_t n, int64_t x) {
    return ((x + 1) * n - 1) / total;
}

// The last tile of n with pre <= x, by a whole warp: 32 probes a round.
__device__ __forceinline__ int find_tile(const Tile* t, int n, int64_t x) {
    const int lane = threadIdx.x & 31;
    int lo = 0, len = n;
    while (len > 1) {
        const int step = (len + 31) / 32;
        const bool le = lane * step < len && t[lo + lane * step].pre <= x;
        const int end = lo + len;
        lo += (__popc(__ballot_sync(0xffffffffu, le)) - 1) * step;
        len = min(step, end - lo);
    }
    return lo;
}

// The parts of cut tiles: slot 2 * cta holds the CTA's first tile when it begins before the
// CTA's range, slot 2 * cta + 1 its last tile when it begins inside and ends past the range.
// A slot is tile_rows rows of 128 accumulators, then the rows' maxima (base-2 units) and sums; each
// begins on 16 bytes (tile_rows may be odd).
__host__ __device__ __forceinline__ size_t part_floats(int tile_rows) {
    return static_cast<size_t>(round_up(static_cast<int64_t>(tile_rows) * (D + 2), 4));
}

// What the join needs of the cut before CTA c, left by that CTA: the tile it goes through, if it is
// that tile's first cut (parts > 0), and the CTAs whose parts make it up.
struct Cut {
    int32_t parts, c0;         // number of parts, and the CTA of the first
    int32_t row0, first, nrow, head;
};

struct AttendArgs {
    PagePool pool;
    Seqs seqs;
    Plan plan;
    PlanShape shape;
    const __nv_bfloat16* q;
    int64_t q_ld;
    int32_t heads;          // KV heads
    float scale;
    void* out;
    float* lse;             // or NULL
    float* work;            // parts
    Cut* cut;               // [ctas]
    int32_t inject_wait;    // test hook: a wait runs out
};

// The record of CTA c, of the tile that its range begins in (block b0 of the tile's blocks [start,
// end) on the whole axis).
__device__ __forceinline__ Cut cut_record(const Tile& t, int64_t total, int64_t n, int64_t start,
                                          int64_t end, int b0, int64_t head) {
    Cut r;
    r.c0 = static_cast<int32_t>(cut_of(total, n, start));
    const bool mine = b0 > 0 && r.c0 == static_cast<int32_t>(blockIdx.x) - 1;
    r.parts = mine ? static_cast<int32_t>(cut_of(total, n, end - 1)) - r.c0 + 1 : 0;
    r.row0 = t.row0;
    r.first = t.first;
    r.nrow = t.nrow;
    r.head = static_cast<int32_t>(head);
    return r;
}

// paged.cu
cudaError_t launch_plan(const AttendArgs& a, cudaStream_t st);
cudaError_t launch_join(const AttendArgs& a, int ctas, bool f32_out, cudaStream_t st);
// paged_attend.cu: up to kFewRows rows a sequence (mma.sync, K/V streamed once), in tiles of 8 or
// 16. It plans for itself where few_plans_inline says so (no launch_plan then).
constexpr int kFewRows = 16;
constexpr int few_block(bool e4m3) { return e4m3 ? 128 : 64; }   // tokens of a block
int few_ctas(int sms);
bool few_plans_inline(int batch);
cudaError_t launch_attend_few(const AttendArgs& a, int format, bool f32_out, int ctas,
                              cudaStream_t st);
cudaError_t take_few_waits_out(bool* out, cudaStream_t st);     // since the last time
// paged_chunk.cu: many rows a sequence (tcgen05); one CTA an SM
constexpr int kChunkBlock = 128;
int chunk_tile_rows(int group, bool f32_out);
cudaError_t launch_attend_chunk(const AttendArgs& a, int format, bool f32_out, int ctas,
                                cudaStream_t st);
cudaError_t take_chunk_waits_out(bool* out, cudaStream_t st);   // since the last time

}  // namespace pkv
