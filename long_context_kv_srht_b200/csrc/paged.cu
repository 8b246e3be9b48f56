// paged.cu -- the paged K/V cache (pariskv_paged.h): argument checks, the kernels that write a
// chunk into its pages and read pages back, and the plan and join kernels around the attention.
#include <cuda_fp8.h>

#include "paged.cuh"
#include "pariskv_debug.h"

namespace pkv {

namespace {

__device__ __forceinline__ void unpack8(uint4 a, float v[8]) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint4 pack8(const float v[8]) {
    return make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]),
                      bf16_pair(v[6], v[7]));
}

// ------------------------------------------------------------------------------------ write
// A warp takes one new token, a head at a time: 16 lanes its K row and 16 its V row, 8 elements a
// lane. The first rows are under way while the warp finds out where they go (a chain of dependent
// loads: starts, lengths, the page's id). Bound by HBM: it reads each row once and writes 256 or 129
// bytes of it; neighbouring tokens are in neighbouring warps of a CTA, so the 128-byte pieces of a
// head's rows meet in L2. 131072 tokens of 8 heads from bf16 to 8 bits: 142 us, 5.7 TB/s, two thirds
// of it reads (158 us when a lane's rows were K's of one head and then another's: twice the
// instructions; 170 us with 32 lanes a row, whose maximum is one instruction, but whose stores are
// half as wide). 16 tokens: 8 us, which is the host's part of a call; 3.3 us each in a captured graph,
// the launch and the chain of four dependent loads.
constexpr int kWriteWarps = 8;

// four values to e4m3, nearest even, saturating
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}

// 8 elements of a row, as they are in memory. top(): the fp32 bits of the largest magnitude in
// the 16 lanes of a row (a NaN's are above infinity's); codes(e): the codes of x / 2^e.
template <typename In> struct Raw8;
template <> struct Raw8<float> {
    float4 a, b;
    static constexpr int kRows = 4;      // heads in flight
    __device__ __forceinline__ void load(const float* p) {
        a = __ldcs(reinterpret_cast<const float4*>(p));
        b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ uint4 bf16() const {
        return make_uint4(bf16_pair(a.x, a.y), bf16_pair(a.z, a.w), bf16_pair(b.x, b.y),
                          bf16_pair(b.z, b.w));
    }
    __device__ __forceinline__ uint32_t top() const {
        const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        uint32_t t = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) t = max(t, __float_as_uint(v[k]) & 0x7fffffffu);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) t = max(t, __shfl_xor_sync(0xffffffffu, t, o));
        return t;
    }
    __device__ __forceinline__ uint2 codes(int e) const {
        const float f = pow2f(-e);
        return make_uint2(codes4(a.x * f, a.y * f, a.z * f, a.w * f),
                          codes4(b.x * f, b.y * f, b.z * f, b.w * f));
    }
};
template <> struct Raw8<__nv_bfloat16> {
    uint4 a;
    static constexpr int kRows = 8;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        a = __ldcs(reinterpret_cast<const uint4*>(p));
    }
    __device__ __forceinline__ uint4 bf16() const { return a; }
    __device__ __forceinline__ uint32_t top() const {   // two magnitudes a word
        constexpr uint32_t m = 0x7fff7fffu;
        uint32_t t = __vmaxu2(__vmaxu2(a.x & m, a.y & m), __vmaxu2(a.z & m, a.w & m));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) t = __vmaxu2(t, __shfl_xor_sync(0xffffffffu, t, o));
        return max(t & 0xffff0000u, t << 16);
    }
    __device__ __forceinline__ uint2 codes(int e) const {
        // the product with a power of two is exact in bf16 (or far below the least code)
        const uint32_t bits = static_cast<uint32_t>(127 - e) << 7, f = bits | bits << 16;
        uint32_t y[4] = {a.x, a.y, a.z, a.w};
        uint2 c;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y[k]) : "r"(y[k]), "r"(f));
        auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
        auto hi = [](uint32_t w) { return __uint_as_float(w & 0xffff0000u); };
        c.x = codes4(lo(y[0]), hi(y[0]), lo(y[1]), hi(y[1]));
        c.y = codes4(lo(y[2]), hi(y[2]), lo(y[3]), hi(y[3]));
        return c;
    }
};

template <typename In, bool kE4m3>
__global__ void __launch_bounds__(kWriteWarps * 32)
paged_write_kernel(const PagePool pool, const Seqs c, int heads, const In* __restrict__ kn,
                   const In* __restrict__ vn, int64_t k_ld, int64_t v_ld) {
    constexpr int kRows = Raw8<In>::kRows;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t tok = static_cast<int64_t>(blockIdx.x) * kWriteWarps + warp;
    if (tok >= c.total_q) return;
    const int half = lane >> 4, l8 = (lane & 15) * 8;
    const In* const src = (half ? vn + tok * v_ld : kn + tok * k_ld) + l8;
    Raw8<In> x[kRows];
    auto load = [&](int h0) {
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            if (h0 + i < heads) x[i].load(src + (h0 + i) * D);
    };
    load(0);
    // the sequence of the token: the last start <= tok
    int lo = 0;
    for (int len = c.batch + 1; len > 1;) {
        const int step = (len + 31) / 32, i = lo + lane * step;
        const bool le = lane * step < len && i <= c.batch && c.q_start[i] <= tok;
        const int cnt = __popc(__ballot_sync(0xffffffffu, le));
        if (cnt == 0) return;   // before the first sequence
        lo += (cnt - 1) * step;
        len = step;
    }
    if (lo >= c.batch) return;  // behind the last sequence
    const SeqView v = seq_view(c, pool.shift, lo);
    const int64_t j = tok - v.row0, pos = v.pos0 + j;
    if (j < 0 || j >= v.rows || pos < 0 || pos >= v.kv) return;
    const int32_t page = c.table[static_cast<int64_t>(lo) * c.stride + (pos >> pool.shift)];
    if (page < 0 || page >= pool.num_pages) return;
    const int slot = static_cast<int>(pos) & ((1 << pool.shift) - 1);

    constexpr int kEl = kE4m3 ? 1 : 2;
    uint8_t* to = (half ? pool.v : pool.k) + page * pool.page_bytes + (slot * D + l8) * kEl;
    uint8_t* scale = (half ? pool.vs : pool.ks) + (page * pool.scale_stride + slot);
    for (int h0 = 0; h0 < heads; h0 += kRows) {
        if (h0 > 0) load(h0);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            if (h0 + i >= heads) break;
            if (!kE4m3) {
                *reinterpret_cast<uint4*>(to) = x[i].bf16();
            } else {
                const uint32_t top = x[i].top();
                const bool finite = top < 0x7f800000u;
                const int byte = finite ? scale_byte(__uint_as_float(top)) : kNanRow;
                *reinterpret_cast<uint2*>(to) =
                    finite ? x[i].codes(byte - 127) : make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
                if ((lane & 15) == 0) *scale = static_cast<uint8_t>(byte);
                scale += int64_t{1} << pool.shift;
            }
            to += static_cast<int64_t>(D * kEl) << pool.shift;
        }
    }
}

// ------------------------------------------------------------------------------------- read
// A warp takes 16 consecutive positions (aligned, so they lie in one page) of one KV head of K
// or of V: 8 loads of two rows in flight, then 8 stores. Both sides are contiguous runs of 16
// rows. Bound by HBM: 131072 tokens of 8 heads from 8 bits to bf16 132 us, 6.1 TB/s; a window of
// bf16 pages to fp32 31 us, 5.35 TB/s, with 32 bytes a store (37 us with two stores of 16, which
// is what slabs that begin off 32 bytes get).
constexpr int kReadWarps = 8;
constexpr int kReadRun = 16;

template <typename Out, bool kE4m3>
__global__ void __launch_bounds__(kReadWarps * 32)
paged_read_kernel(const PagePool pool, const Seqs c, int heads, int64_t first, int64_t n,
                  Out* __restrict__ K, Out* __restrict__ V, int64_t ld, int64_t runs,
                  int64_t total) {
    const int lane = threadIdx.x & 31;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * kReadWarps + (threadIdx.x >> 5);
    if (w >= total) return;
    const int64_t run = w % runs, x = w / runs;
    const int h = static_cast<int>(x % heads);
    const int64_t y = x / heads;
    const int s = static_cast<int>(y % c.batch);
    const bool is_v = K == nullptr || y >= c.batch;
    const int64_t p0 = ((first >> 4) + run) << 4;        // first position of the run
    const int64_t end = min64(min64(first + n, c.kv_len[s]),
                              static_cast<int64_t>(c.width) << pool.shift);
    if (p0 >= end) return;
    const int32_t page = c.table[static_cast<int64_t>(s) * c.stride + (p0 >> pool.shift)];
    if (page < 0 || page >= pool.num_pages) return;
    const int slot = static_cast<int>(p0) & ((1 << pool.shift) - 1);
    const int64_t row = (static_cast<int64_t>(h) << pool.shift) + slot + (lane >> 4);
    const int l8 = (lane & 15) * 8;
    const uint8_t* src = (is_v ? pool.v : pool.k) + page * pool.page_bytes +
                         (row * D + l8) * (kE4m3 ? 1 : 2);
    const uint8_t* sc = kE4m3 ? (is_v ? pool.vs : pool.ks) + page * pool.scale_stride + row
                              : nullptr;
    uint4 raw[kReadRun / 2];
    uint32_t byte[kReadRun / 2];
#pragma unroll
    for (int i = 0; i < kReadRun / 2; ++i) {
        const int64_t pos = p0 + 2 * i + (lane >> 4);
        const bool ok = pos >= first && pos < end;
        if (kE4m3) {
            const uint2 t = ok ? __ldcs(reinterpret_cast<const uint2*>(src + 2 * i * D))
                               : make_uint2(0, 0);
            raw[i] = make_uint4(t.x, t.y, 0, 0);
            byte[i] = ok ? sc[2 * i] : 0;
        } else {
            raw[i] = ok ? __ldcs(reinterpret_cast<const uint4*>(src + 4 * i * D))
                        : make_uint4(0, 0, 0, 0);
        }
    }
    Out* dst = (is_v ? V : K) + ((static_cast<int64_t>(s) * heads + h) * ld) * D + l8;
    const bool wide = (reinterpret_cast<uintptr_t>(dst) & 31) == 0;
#pragma unroll
    for (int i = 0; i < kReadRun / 2; ++i) {
        const int64_t pos = p0 + 2 * i + (lane >> 4);
        if (pos < first || pos >= end) continue;
        Out* o = dst + (pos - first) * D;
        float v[8];
        if (kE4m3) {
            const float f = scale_value(byte[i]);
            const uint32_t w2[2] = {raw[i].x, raw[i].y};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(
                    static_cast<__nv_fp8x2_storage_t>(w2[k >> 1] >> (16 * (k & 1))), __NV_E4M3);
                const float2 t = __half22float2(__half2(hr));
                v[2 * k] = t.x * f;
                v[2 * k + 1] = t.y * f;
            }
        } else {
            unpack8(raw[i], v);
        }
        if constexpr (sizeof(Out) == 2) {
            *reinterpret_cast<uint4*>(o) = kE4m3 ? pack8(v) : raw[i];
        } else {
            uint32_t u[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) u[k] = __float_as_uint(v[k]);
            store_words<8>(o, u, wide);
        }
    }
}

// ------------------------------------------------------------------------------------- plan
constexpr int kPlanT = 1024;

// inclusive scan over the CTA; *total is the sum
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t* s_warp, int64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();           // the last scan's readers are done with s_warp
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    int64_t before = 0, all = 0;
    for (int w = 0; w < kPlanT / 32; ++w) {
        const int64_t y = s_warp[w];
        before += w < warp ? y : 0;
        all += y;
    }
    *total = all;
    return x + before;
}

// Marks the blocks of a sequence (with new tokens) of which some page is there: a warp 32 blocks, a
// lane a block. With few sequences several warps share one.
__device__ __forceinline__ void mark_live(const Seqs& c, const PagePool& pool, const PlanShape& p,
                                          const Plan& plan) {
    constexpr int kWarps = kPlanT / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, shift = pool.shift;
    const int per = c.batch < kWarps ? kWarps / c.batch : 1, step = kWarps / per;
    for (int s = warp / per; s < c.batch && warp < per * step; s += step) {
        const SeqView v = seq_view(c, shift, s);
        if (v.rows == 0) continue;
        const int32_t* table = c.table + static_cast<int64_t>(s) * c.stride;
        const int n = static_cast<int>(ceil_div(v.kv, 32 * static_cast<int64_t>(p.block)));
#pragma unroll 2
        for (int w = warp % per; w < n; w += per) {
            const int64_t tok = (static_cast<int64_t>(w) * 32 + lane) * p.block;
            bool any = false;
#pragma unroll
            for (int i = 0; i < kChunkBlock / 16; ++i) {   // pages have 16 tokens at least
                const int64_t t = tok + (static_cast<int64_t>(i) << shift);
                if ((i << shift) < p.block && t < v.kv)
                    any |= static_cast<uint32_t>(table[t >> shift]) <
                           static_cast<uint32_t>(pool.num_pages);
            }
            const uint32_t word = __ballot_sync(0xffffffffu, any);
            if (lane == 0) plan.live[static_cast<int64_t>(s) * plan.words + w] = word;
        }
    }
}

// One CTA: counts each sequence's tiles, writes the tiles in order, and sums their blocks. Bound by
// latency (a scan, and a chain of loads a sequence): 5 us of a call.
__global__ void __launch_bounds__(kPlanT)
plan_kernel(const Seqs c, const PagePool pool, const PlanShape p, const Plan plan) {
    const int shift = pool.shift;
    __shared__ int64_t s_warp[kPlanT / 32];
    __shared__ int32_t s_first[kPlanT], s_count[kPlanT];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_launch_dependents();
    if (plan.live) {
        mark_live(c, pool, p, plan);
        __syncthreads();
    }
    int64_t tiles = 0;
    for (int s0 = 0; s0 < c.batch; s0 += kPlanT) {
        const int s = s0 + threadIdx.x;
        int64_t nt = 0, all;
        if (s < c.batch)
            nt = ceil_div(static_cast<int64_t>(seq_view(c, shift, s).rows) * p.group,
                          p.tile_rows);
        const int64_t at = tiles + block_scan(nt, s_warp, &all) - nt;
        // malformed starts (overlapping sequences) can ask for more tiles than there is room
        s_first[threadIdx.x] = static_cast<int32_t>(min64(at, plan.max_tiles));
        s_count[threadIdx.x] = static_cast<int32_t>(min64(nt, max64(0, plan.max_tiles - at)));
        __syncthreads();
        for (int i = warp; i < min(kPlanT, c.batch - s0); i += kPlanT / 32) {
            const int n = s_count[i];
            if (n == 0) continue;
            const SeqView v = seq_view(c, shift, s0 + i);
            for (int t = lane; t < n; t += 32) {
                Tile x;
                x.first = t * p.tile_rows;
                x.end = tile_end(v, p, x.first);
                int64_t blocks = ceil_div(x.end, p.block);
                if (plan.live) {
                    const uint32_t* live = plan.live + static_cast<int64_t>(s0 + i) * plan.words;
                    const int n = static_cast<int>(blocks), left = n & 31;
                    blocks = left ? __popc(live[n >> 5] & ((1u << left) - 1)) : 0;
#pragma unroll 4
                    for (int w = 0; w < n >> 5; ++w) blocks += __popc(live[w]);
                }
                x.pre = max64(1, blocks);   // (its own, until they are summed)
                x.pos0 = v.pos0;
                x.seq = s0 + i;
                x.row0 = v.row0;
                x.nrow = static_cast<int32_t>(
                    min64(p.tile_rows, static_cast<int64_t>(v.rows) * p.group - x.first));
                x.kv = v.kv;
                x.pad[0] = x.pad[1] = 0;
                plan.tile[s_first[i] + t] = x;
            }
        }
        tiles = min64(tiles + all, plan.max_tiles);
        __syncthreads();
    }
    const int nt = static_cast<int>(tiles);
    int64_t sum = 0;
    for (int t0 = 0; t0 < nt; t0 += kPlanT) {
        const int t = t0 + threadIdx.x;
        int64_t all;
        const int64_t own = t < nt ? plan.tile[t].pre : 0;
        const int64_t x = block_scan(own, s_warp, &all);
        if (t < nt) plan.tile[t].pre = sum + x - own;
        sum += all;
    }
    if (threadIdx.x == 0) {
        plan.tile[nt].pre = sum;
        *plan.ntiles = nt;
    }
}

// ------------------------------------------------------------------------------------- join
// The tile that the cut before CTA blockIdx.x + 1 goes through, if that cut is the tile's first: its
// parts are rescaled to the common maximum and summed. A warp a row, 4 elements a lane. Where a
// tile has many parts and fewer rows than there are warps (few rows, a long token axis), the
// CTA's warps share a row's parts and add their sums up in order. Measured, whole calls: one row a
// group of 4 over 65536 tokens 52.0 us with shared rows, 58.3 without (37 parts a head); 64 tokens
// over 65536 (256 rows a head, 19 parts) 129 us with shared rows, 118 without. Bound by the latency
// of its two dependent loads (record, parts), some 4 us of a call, and by the parts' bytes from L2
// (64 tokens over 2000, 16 parts of 256 rows a head: 42.1 us a call with 4 warps a CTA, 34.7 with 8,
// 34.8 with 16, which cost few rows 1 us).
constexpr int kJoinWarps = 8;
constexpr int kJoinShared = 8;    // parts from which on the warps share a row

template <typename Out>
__global__ void __launch_bounds__(kJoinWarps * 32)
join_kernel(const AttendArgs a) {
    __shared__ float s_sum[kJoinWarps][D + 2];
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Cut t = a.cut[blockIdx.x + 1];
    if (t.parts == 0) return;
    const int parts = t.parts;
    const int64_t h = t.head;
    const int R = a.shape.tile_rows, G = a.shape.group;
    const bool shared = parts >= kJoinShared && t.nrow < static_cast<int>(gridDim.y) * kJoinWarps;
    const size_t step = 2 * part_floats(R);
    // part i: slot 2 (c0 + i), the first one 2 c0 + 1
    const float* base = a.work + 2 * static_cast<size_t>(t.c0) * part_floats(R);
    auto part = [&](int i) { return base + i * step + (i == 0 ? part_floats(R) : 0); };
    const int i0 = shared ? warp : 0, istep = shared ? kJoinWarps : 1;
    const int r0 = shared ? blockIdx.y : blockIdx.y * kJoinWarps + warp;
    for (int r = r0; r < t.nrow; r += gridDim.y * (shared ? 1 : kJoinWarps)) {
        float M = -INFINITY;
        for (int i = lane; i < parts; i += 32) M = fmaxf(M, part(i)[R * D + r]);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
        const float m = M == -INFINITY ? 0.0f : M;
        float den = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
        for (int i = i0; i < parts; i += istep) {
            const float* w = part(i);
            const float f = exp2f(w[R * D + r] - m);
            den += w[R * D + R + r] * f;
            const float4 x = *reinterpret_cast<const float4*>(w + r * D + 4 * lane);
            o[0] += x.x * f; o[1] += x.y * f; o[2] += x.z * f; o[3] += x.w * f;
        }
        if (shared) {
            *reinterpret_cast<float2*>(&s_sum[warp][4 * lane]) = make_float2(o[0], o[1]);
            *reinterpret_cast<float2*>(&s_sum[warp][4 * lane + 2]) = make_float2(o[2], o[3]);
            if (lane == 0) s_sum[warp][D] = den;
            __syncthreads();
            if (warp == 0) {
                for (int w = 1; w < kJoinWarps; ++w) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) o[k] += s_sum[w][4 * lane + k];
                    den += s_sum[w][D];
                }
            }
            __syncthreads();
            if (warp != 0) continue;
        }
        // a row without tokens has den == 0 (a NaN must come through)
        const float inv = den == 0.0f ? 0.0f : 1.0f / den;
        const int rr = t.first + r;
        const int64_t at = (t.row0 + rr / G) * (static_cast<int64_t>(a.heads) * G) + h * G + rr % G;
        Out* dst = static_cast<Out*>(a.out) + at * D + 4 * lane;
        if constexpr (sizeof(Out) == 2)
            *reinterpret_cast<uint2*>(dst) = make_uint2(bf16_pair(o[0] * inv, o[1] * inv),
                                                        bf16_pair(o[2] * inv, o[3] * inv));
        else
            *reinterpret_cast<float4*>(dst) =
                make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
        if (a.lse && lane == 0) a.lse[at] = den == 0.0f ? -INFINITY : M * kLn2 + logf(den);
    }
}

}  // namespace

cudaError_t launch_plan(const AttendArgs& a, cudaStream_t st) {
    return launch_pdl(plan_kernel, dim3(1), dim3(kPlanT), 0, st, a.seqs, a.pool, a.shape, a.plan);
}

cudaError_t launch_join(const AttendArgs& a, int ctas, bool f32_out, cudaStream_t st) {
    if (ctas < 2) return cudaSuccess;
    const dim3 grid(ctas - 1, min(16, a.shape.tile_rows));
    return launch_pdl(f32_out ? join_kernel<float> : join_kernel<__nv_bfloat16>, grid,
                      dim3(kJoinWarps * 32), 0, st, a);
}

namespace {

// Device memory of the current device.
pariskv_status check_here(const void* p, size_t align, const char* name, int dev) {
    if (!p) return fail(PARISKV_EINVAL, "%s is NULL", name);
    if (reinterpret_cast<uintptr_t>(p) % align)
        return fail(PARISKV_EINVAL, "%s is not %zu-byte aligned", name, align);
    cudaPointerAttributes at;
    if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
        cudaGetLastError();
        return fail(PARISKV_EINVAL, "%s is not a CUDA-visible pointer", name);
    }
    if (at.type != cudaMemoryTypeDevice)
        return fail(PARISKV_EINVAL, "%s is not device memory", name);
    if (at.device != dev)
        return fail(PARISKV_EINVAL, "%s lies on device %d but device %d is current", name,
                    at.device, dev);
    return PARISKV_OK;
}

// The checks that need no device come first, so that they hold without one.
pariskv_status check_shapes(const pariskv_config* cfg, const pariskv_pages* p,
                            const pariskv_chunk* c) {
    pariskv_status s = validate_config(cfg);
    if (s != PARISKV_OK) return s;
    if (!p) return fail(PARISKV_EINVAL, "pages is NULL");
    if (!c) return fail(PARISKV_EINVAL, "chunk is NULL");
    if (p->format != PARISKV_PAGES_BF16 && p->format != PARISKV_PAGES_E4M3)
        return fail(PARISKV_EINVAL, "page format %d unknown", p->format);
    if (p->page_size < 16 || p->page_size > 256 || (p->page_size & (p->page_size - 1)))
        return fail(PARISKV_EINVAL, "page_size %d is not 16, 32, 64, 128 or 256", p->page_size);
    if (p->num_pages < 1 || p->num_pages > INT32_MAX)
        return fail(PARISKV_EINVAL, "num_pages %lld not in [1, 2^31 - 1]",
                    static_cast<long long>(p->num_pages));
    const int64_t el = p->format == PARISKV_PAGES_BF16 ? 2 : 1;
    const int64_t rows = static_cast<int64_t>(cfg->num_kv_heads) * p->page_size;
    if (p->page_stride < rows * D || p->page_stride * el % 16 ||
        p->page_stride > (int64_t(1) << 38))
        return fail(PARISKV_EINVAL, "page_stride %lld: need >= num_kv_heads * page_size * 128 "
                    "elements, a multiple of 16 bytes and at most 2^38",
                    static_cast<long long>(p->page_stride));
    if (p->format == PARISKV_PAGES_E4M3 &&
        (p->scale_stride < rows || p->scale_stride % 16 || p->scale_stride > (int64_t(1) << 31)))
        return fail(PARISKV_EINVAL, "scale_stride %lld: need >= num_kv_heads * page_size, a "
                    "multiple of 16 and at most 2^31", static_cast<long long>(p->scale_stride));
    if (c->table_width < 1 || c->table_stride < c->table_width)
        return fail(PARISKV_EINVAL, "need 1 <= table_width <= table_stride");
    if (c->total_q < 0 || c->total_q > INT32_MAX || c->max_q < 0)
        return fail(PARISKV_EINVAL, "need 0 <= total_q < 2^31 and max_q >= 0");
    return PARISKV_OK;
}

pariskv_status check_buffers(const pariskv_pages* p, const pariskv_chunk* c, bool starts, int dev) {
    pariskv_status s;
    if ((s = check_here(p->k, 16, "pages.k", dev)) != PARISKV_OK) return s;
    if ((s = check_here(p->v, 16, "pages.v", dev)) != PARISKV_OK) return s;
    if (p->format == PARISKV_PAGES_E4M3) {
        if ((s = check_here(p->k_scale, 16, "pages.k_scale", dev)) != PARISKV_OK) return s;
        if ((s = check_here(p->v_scale, 16, "pages.v_scale", dev)) != PARISKV_OK) return s;
    }
    if ((s = check_here(c->page_table, 4, "page_table", dev)) != PARISKV_OK) return s;
    if ((s = check_here(c->kv_len, 4, "kv_len", dev)) != PARISKV_OK) return s;
    if (starts && (s = check_here(c->q_start, 4, "q_start", dev)) != PARISKV_OK) return s;
    return PARISKV_OK;
}

pariskv_status check_launch(int* dev) {
    if (cudaGetDevice(dev) != cudaSuccess) return cuda_fail(cudaGetLastError(), "no device");
    if (launch_fault_injected())
        return fail(PARISKV_ECUDA, "injected launch failure (PARISKV_FAULT=launch)");
    return PARISKV_OK;
}

PagePool pool_of(const pariskv_pages* p) {
    PagePool v;
    v.k = static_cast<uint8_t*>(p->k);
    v.v = static_cast<uint8_t*>(p->v);
    v.ks = p->k_scale;
    v.vs = p->v_scale;
    v.page_bytes = p->page_stride * (p->format == PARISKV_PAGES_BF16 ? 2 : 1);
    v.scale_stride = p->scale_stride;
    v.num_pages = static_cast<int32_t>(p->num_pages);
    v.shift = 0;
    while ((1 << v.shift) < p->page_size) ++v.shift;
    return v;
}

std::atomic<int> g_inject_wait{0};   // pariskv_debug_inject_paged_timeout

Seqs seqs_of(const pariskv_config* cfg, const pariskv_chunk* c) {
    return Seqs{c->page_table, c->kv_len, c->q_start, static_cast<int32_t>(c->total_q),
                c->table_width, c->table_stride, c->max_q, cfg->batch};
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

pariskv_status pariskv_paged_write(const pariskv_config* cfg, const pariskv_pages* pages,
                                   const pariskv_chunk* chunk, const void* k_new,
                                   const void* v_new, int64_t k_ld, int64_t v_ld, void* stream) {
    pariskv_status s = check_shapes(cfg, pages, chunk);
    if (s != PARISKV_OK) return s;
    const bool f32 = cfg->dtype == PARISKV_F32;
    const int64_t row = static_cast<int64_t>(cfg->num_kv_heads) * D, word = f32 ? 4 : 8;
    if (k_ld < row || v_ld < row || k_ld % word || v_ld % word)
        return fail(PARISKV_EINVAL, "k_ld and v_ld must be >= num_kv_heads * 128 and whole "
                    "16-byte words");
    int dev = 0;
    if ((s = check_launch(&dev)) != PARISKV_OK) return s;
    if ((s = check_buffers(pages, chunk, true, dev)) != PARISKV_OK) return s;
    set_last_launches(0);
    if (chunk->total_q == 0) return PARISKV_OK;
    if ((s = check_here(k_new, 16, "k_new", dev)) != PARISKV_OK) return s;
    if ((s = check_here(v_new, 16, "v_new", dev)) != PARISKV_OK) return s;
    const PagePool p = pool_of(pages);
    const Seqs c = seqs_of(cfg, chunk);
    const unsigned grid = static_cast<unsigned>(ceil_div(chunk->total_q, kWriteWarps));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int h = cfg->num_kv_heads, t = kWriteWarps * 32;
    const bool e4 = pages->format == PARISKV_PAGES_E4M3;
    const float* kf = static_cast<const float*>(k_new);
    const float* vf = static_cast<const float*>(v_new);
    const __nv_bfloat16* kb = static_cast<const __nv_bfloat16*>(k_new);
    const __nv_bfloat16* vb = static_cast<const __nv_bfloat16*>(v_new);
    if (f32) {
        auto kernel = e4 ? paged_write_kernel<float, true> : paged_write_kernel<float, false>;
        kernel<<<grid, t, 0, st>>>(p, c, h, kf, vf, k_ld, v_ld);
    } else {
        auto kernel = e4 ? paged_write_kernel<__nv_bfloat16, true>
                         : paged_write_kernel<__nv_bfloat16, false>;
        kernel<<<grid, t, 0, st>>>(p, c, h, kb, vb, k_ld, v_ld);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "page write launch");
    set_last_launches(1);
    return PARISKV_OK;
}

pariskv_status pariskv_paged_read(const pariskv_config* cfg, const pariskv_pages* pages,
                                  const pariskv_chunk* chunk, int64_t first, int64_t n, void* K,
                                  void* V, int64_t ld_tok, void* stream) {
    pariskv_status s = check_shapes(cfg, pages, chunk);
    if (s != PARISKV_OK) return s;
    if (first < 0 || n < 0 || first > INT32_MAX || n > INT32_MAX || ld_tok < n)
        return fail(PARISKV_EINVAL, "need 0 <= first, 0 <= n <= ld_tok (below 2^31)");
    if (!K && !V) return fail(PARISKV_EINVAL, "K and V are both NULL");
    int dev = 0;
    if ((s = check_launch(&dev)) != PARISKV_OK) return s;
    if ((s = check_buffers(pages, chunk, false, dev)) != PARISKV_OK) return s;
    if (K && (s = check_device_pointer(K, 16, "K")) != PARISKV_OK) return s;
    if (V && (s = check_device_pointer(V, 16, "V")) != PARISKV_OK) return s;
    set_last_launches(0);
    if (n == 0) return PARISKV_OK;
    const PagePool p = pool_of(pages);
    const Seqs c = seqs_of(cfg, chunk);
    const int64_t runs = ((first + n - 1) >> 4) - (first >> 4) + 1;
    const int64_t total = runs * cfg->num_kv_heads * cfg->batch * (K && V ? 2 : 1);
    const int64_t blocks = ceil_div(total, kReadWarps);
    if (blocks > INT32_MAX) return fail(PARISKV_EINVAL, "too many rows for one call");
    const unsigned grid = static_cast<unsigned>(blocks);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int h = cfg->num_kv_heads, t = kReadWarps * 32;
    const bool e4 = pages->format == PARISKV_PAGES_E4M3, f32 = cfg->dtype == PARISKV_F32;
    float *Kf = static_cast<float*>(K), *Vf = static_cast<float*>(V);
    __nv_bfloat16 *Kb = static_cast<__nv_bfloat16*>(K), *Vb = static_cast<__nv_bfloat16*>(V);
    if (f32) {
        auto kernel = e4 ? paged_read_kernel<float, true> : paged_read_kernel<float, false>;
        kernel<<<grid, t, 0, st>>>(p, c, h, first, n, Kf, Vf, ld_tok, runs, total);
    } else {
        auto kernel = e4 ? paged_read_kernel<__nv_bfloat16, true>
                         : paged_read_kernel<__nv_bfloat16, false>;
        kernel<<<grid, t, 0, st>>>(p, c, h, first, n, Kb, Vb, ld_tok, runs, total);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "page read launch");
    set_last_launches(1);
    return PARISKV_OK;
}

pariskv_status pariskv_paged_attend(const pariskv_config* cfg, const pariskv_pages* pages,
                                    const pariskv_chunk* chunk, const void* q, int64_t q_ld,
                                    float scale, int32_t causal, void* out, int32_t out_dtype,
                                    float* lse, void* stream) {
    pariskv_status s = check_shapes(cfg, pages, chunk);
    if (s != PARISKV_OK) return s;
    if (cfg->dtype != PARISKV_BF16) return fail(PARISKV_EINVAL, "paged attention takes bf16 q");
    if (cfg->group > 128) return fail(PARISKV_EINVAL, "group %d > 128", cfg->group);
    if (out_dtype != PARISKV_F32 && out_dtype != PARISKV_BF16)
        return fail(PARISKV_EINVAL, "out_dtype %d unknown", out_dtype);
    if (!(scale == scale)) return fail(PARISKV_EINVAL, "scale is NaN");
    const int64_t hq = static_cast<int64_t>(cfg->num_kv_heads) * cfg->group;
    if (q_ld < hq * D || q_ld % 8 || q_ld > (int64_t(1) << 38))
        return fail(PARISKV_EINVAL, "q_ld must be >= query heads * 128, a multiple of 8 and at "
                    "most 2^38");
    if (chunk->total_q * cfg->group > INT32_MAX)
        return fail(PARISKV_EINVAL, "total_q * group must be below 2^31");
    int dev = 0, sms = 0;
    if ((s = check_launch(&dev)) != PARISKV_OK) return s;
    if ((s = check_buffers(pages, chunk, true, dev)) != PARISKV_OK) return s;
    set_last_launches(0);
    if (chunk->total_q == 0 || chunk->max_q == 0) return PARISKV_OK;
    if ((s = check_here(q, 16, "q", dev)) != PARISKV_OK) return s;
    if ((s = check_here(out, 16, "out", dev)) != PARISKV_OK) return s;
    if (lse && (s = check_here(lse, 4, "lse", dev)) != PARISKV_OK) return s;
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);

    AttendArgs a{};
    a.pool = pool_of(pages);
    a.seqs = seqs_of(cfg, chunk);
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.q_ld = q_ld;
    a.heads = cfg->num_kv_heads;
    a.scale = scale;
    a.out = out;
    a.lse = lse;
    a.shape.group = cfg->group;
    a.shape.causal = causal != 0;
    const bool f32 = out_dtype == PARISKV_F32;
    // up to one tile of the streaming kernel a sequence: it reads each K/V row once
    const int64_t most = static_cast<int64_t>(chunk->max_q) * cfg->group;
    const bool few = most <= kFewRows;
    a.shape.tile_rows = few ? (most <= 8 ? 8 : kFewRows) : chunk_tile_rows(cfg->group, f32);
    a.shape.block = few ? few_block(pages->format == PARISKV_PAGES_E4M3) : kChunkBlock;
    const int ctas = few ? few_ctas(sms) : sms;
    const bool plan_first = !few || !few_plans_inline(cfg->batch);
    a.inject_wait = g_inject_wait.exchange(0);
    // tiles: every sequence may end in a part of one
    const int64_t tiles = min64(cfg->batch * ceil_div(most, a.shape.tile_rows),
                                chunk->total_q * cfg->group / a.shape.tile_rows + cfg->batch);
    if (tiles > (1 << 28)) return fail(PARISKV_EINVAL, "too many query rows for one call");
    const size_t plan = round_up((tiles + 1) * sizeof(Tile), 256);
    const size_t parts = round_up(2 * ctas * part_floats(a.shape.tile_rows) * 4, 256);
    const size_t cuts = round_up(ctas * sizeof(Cut), 256);
    const int64_t held = min64(INT32_MAX, static_cast<int64_t>(chunk->table_width) << a.pool.shift);
    a.plan.words = few ? 0 : static_cast<int32_t>(ceil_div(held, 32 * kChunkBlock));
    const size_t live = static_cast<size_t>(cfg->batch) * a.plan.words * sizeof(uint32_t);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    void* ws = nullptr;
    if ((s = take_workspace(&ws, parts + cuts + plan + 256 + live, st)) != PARISKV_OK) return s;
    uint8_t* w = static_cast<uint8_t*>(ws);
    a.work = reinterpret_cast<float*>(w);
    a.cut = reinterpret_cast<Cut*>(w + parts);
    a.plan.tile = reinterpret_cast<Tile*>(w + parts + cuts);
    a.plan.ntiles = reinterpret_cast<int32_t*>(w + parts + cuts + plan);
    a.plan.max_tiles = static_cast<int32_t>(tiles);
    a.plan.live = few ? nullptr : reinterpret_cast<uint32_t*>(w + parts + cuts + plan + 256);
    cudaError_t e = plan_first ? launch_plan(a, st) : cudaSuccess;
    if (e == cudaSuccess)
        e = few ? launch_attend_few(a, pages->format, f32, ctas, st)
                : launch_attend_chunk(a, pages->format, f32, ctas, st);
    if (e == cudaSuccess) e = launch_join(a, ctas, f32, st);
    cudaFreeAsync(ws, st);
    if (e != cudaSuccess) return cuda_fail(e, "paged attention launch");
    set_last_launches(plan_first ? 3 : 2);
    return PARISKV_OK;
}

pariskv_status pariskv_paged_sync(void* stream) {
    bool few = false, chunk = false;
    cudaError_t e = take_chunk_waits_out(&chunk, static_cast<cudaStream_t>(stream));
    if (e == cudaSuccess) e = take_few_waits_out(&few, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "paged attention");
    if (few || chunk)
        return fail(PARISKV_ETIMEOUT, "a bounded device-side wait of the paged attention expired");
    return PARISKV_OK;
}

pariskv_status pariskv_debug_inject_paged_timeout(void) {
    g_inject_wait = 1;
    return PARISKV_OK;
}

}  // extern "C"
