// paged_attend.cu -- attention over pages for few query rows a sequence (single tokens, drafts
// of a few tokens):
//     o_r = sum_t softmax_t(scale * <q_r, K_t>) V_t,   rows r = (token, head of the group).
//
// With a handful of rows the call is a stream over the K and V rows (512 bytes a token and KV
// head in bf16, 258 in 8 bits), bound by HBM; the aim is to read each of them once and to spend
// few instructions a token:
//  - all rows of a tile (up to 16: tokens x heads of the KV head's group) share one pass over
//    K and V;
//  - the (head, sequence) streams of a batch form one axis of 64-token blocks that is cut into
//    equal ranges, two CTAs an SM, so ragged lengths leave no SM idle (see Plan);
//  - blocks are staged by a cp.async ring (16-byte copies; page ids ride in the same ring ahead
//    of the rows that need them), rows that are not there are zero-filled and masked;
//  - both products run on mma.sync (m16n8k16, bf16, fp32 accumulators), each warp taking 16
//    tokens of a block: S^T = K Q^T and O^T += V^T P^T, so a lane's softmax state and its
//    accumulators belong to the same two rows of each 8-row group;
//  - bf16 rows come as fragments by ldmatrix. 8-bit rows are widened in registers: which element
//    of the head dimension stands at which position of a fragment is free as long as both
//    factors agree, so a lane reads 16 consecutive codes and uses them for four MMAs;
//  - the 8-bit rows' scales are powers of two and multiply the scores (K) and the weights (V);
//  - P enters the second product as two bf16 parts (16 bits), or three (24) for fp32 output;
//  - base-2 online softmax over 16-token blocks per warp; the four warps merge at the end of a
//    range.
#include "paged.cuh"

namespace pkv {

namespace {

constexpr int kFW = 4;                        // warps, 16 tokens of a block each
static_assert(kFewBlock == 16 * kFW, "a warp takes 16 tokens of a block");
constexpr int kIdRing = 16;                   // blocks whose page ids are held
constexpr int kRuns = kFewBlock / 16;         // page ids a block: 16 tokens lie in one page

template <bool kE4m3> struct FewShape {
    static constexpr int kRowB = kE4m3 ? D : 2 * D;          // bytes of a row
    static constexpr int kStages = kE4m3 ? 6 : 3;            // 96 KB either way: 2 CTAs an SM
    static constexpr int kTensor = kFewBlock * kRowB;
    static constexpr int kStage = 2 * kTensor + (kE4m3 ? 2 * kFewBlock : 0);
    static constexpr int kSmem = kStages * kStage;
};
static_assert(2 * FewShape<true>::kStages - 1 <= kIdRing, "ids of loaded and computed blocks");

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
__device__ __forceinline__ void mma_bf16(float d[4], const uint32_t a[4], uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// Two e4m3 codes, in bytes 1 and 3 of r (the other bytes are ignored), as bf16 values: sign and
// the seven bits below it, moved four places down, are a bf16 number 2^-120 times the code's
// value (the exponent biases differ by 120; subnormal codes become subnormal bf16 numbers), and
// the product with 2^120 is exact.
__device__ __forceinline__ uint32_t widen2(uint32_t r) {
    const uint32_t w = (r & 0x80008000u) | ((r >> 4) & 0x07f007f0u);
    __nv_bfloat162 v, f;
    *reinterpret_cast<uint32_t*>(&v) = w;
    *reinterpret_cast<uint32_t*>(&f) = 0x7b807b80u;   // 2^120, 2^120
    v = __hmul2(v, f);
    return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 :: "r"(dst), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" :: "r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// NT groups of 8 rows; kParts bf16 parts of P.
template <bool kE4m3, int NT, int kParts, typename Out>
__global__ void __launch_bounds__(kFW * 32, 2)
attend_few_kernel(const AttendArgs a) {
    using S = FewShape<kE4m3>;
    constexpr int R = 8 * NT;
    constexpr int kPart = D + 4;     // a row's partial in the merge scratch
    static_assert(kFW * R * kPart * 4 <= S::kSmem, "the merge scratch fits in the stages");
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int32_t s_page[kIdRing][kRuns];
    __shared__ int32_t s_bad[D];     // first token whose V is not finite in this element

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, t = lane & 3;
    pdl_wait();
    pdl_launch_dependents();
    const int nt = *a.plan.ntiles;
    const int64_t per_head = a.plan.tile[nt].pre, total = per_head * a.heads;
    const int64_t ncut = cuts(total, gridDim.x);
    if (blockIdx.x >= ncut) return;
    const int64_t hi = cut(total, ncut, blockIdx.x + 1);
    int64_t x = cut(total, ncut, blockIdx.x);
    int64_t h = x / per_head;
    int tile = find_tile(a.plan.tile, nt, x - h * per_head);
    const int G = a.shape.group, shift = a.pool.shift;
    const float qs = a.scale * kLog2e;

    while (x < hi) {
        const Tile v = a.plan.tile[tile];
        const int64_t start = h * per_head + v.pre;
        const int64_t nb = a.plan.tile[tile + 1].pre - v.pre;
        const int b0 = static_cast<int>(x - start);
        const int b1 = static_cast<int>(min64(nb, hi - start));
        const int s = v.seq, first = v.first, end = v.end, nrow = v.nrow;
        const int32_t* table = a.seqs.table + static_cast<int64_t>(s) * a.seqs.stride;
        // the last token a row may attend
        auto limit = [&](int r) -> int {
            if (r >= nrow) return -1;
            const int64_t lim = a.shape.causal ? v.pos0 + (first + r) / G : v.kv - 1;
            return static_cast<int>(max64(-1, min64(lim, v.kv - 1)));
        };
        // tokens past this one (and before `end`) are seen by some rows of the tile and not by
        // others
        const int shared = limit(0);

        s_bad[tid] = INT32_MAX;
        // page ids of block b, run i: -1 where the run holds nothing that is attended
        auto id_source = [&](int b, int i, const int32_t** src) -> bool {
            const int tok = b * kFewBlock + 16 * i;
            *src = table + (tok >> shift);
            return b < b1 && tok < end;
        };
        if (tid < (S::kStages - 1) * kRuns) {
            const int b = b0 + tid / kRuns, i = tid % kRuns;
            const int32_t* src;
            s_page[b % kIdRing][i] = id_source(b, i, &src) ? *src : -1;
        }
        __syncthreads();

        auto load_ids = [&](int b) {
            if (tid < kRuns) {
                const int32_t* src;
                int32_t* dst = &s_page[b % kIdRing][tid];
                if (id_source(b, tid, &src))
                    cp4(smem_addr(dst), src);
                else
                    *dst = -1;
            }
        };
        auto load_block = [&](int b, int stage) {
            uint8_t* st = smem + stage * S::kStage;
            constexpr int kChunks = S::kRowB / 16;
            constexpr int kLoads = 2 * kFewBlock * kChunks / (kFW * 32);
            constexpr int kRowsPass = kFW * 32 / kChunks;
            const int c = tid % kChunks;
#pragma unroll
            for (int j = 0; j < kLoads; ++j) {
                const int id = tid / kChunks + kRowsPass * j;
                const int is_v = id / kFewBlock, row = id % kFewBlock;
                const int tok = b * kFewBlock + row;
                const int32_t page = s_page[b % kIdRing][row >> 4];
                const bool ok = tok < end && static_cast<uint32_t>(page) <
                                                 static_cast<uint32_t>(a.pool.num_pages);
                const int64_t slot = (h << shift) + (tok & ((1 << shift) - 1));
                const uint8_t* src = (is_v ? a.pool.v : a.pool.k) +
                                     (ok ? page * a.pool.page_bytes + slot * S::kRowB : 0) + c * 16;
                // 16-byte pieces of a row change places so that the fragment reads below hit
                // different banks
                const int sw = !kE4m3 ? (row & 7) : is_v ? ((row >> 1) & 3) << 1 : (row & 1) << 2;
                cp16(smem_addr(st + is_v * S::kTensor + row * S::kRowB + ((c ^ sw) << 4)), src, ok);
            }
            if (kE4m3 && tid < 2 * kRuns) {
                const int is_v = tid / kRuns, i = tid % kRuns;
                const int tok = b * kFewBlock + 16 * i;
                const int32_t page = s_page[b % kIdRing][i];
                const bool ok = tok < end && static_cast<uint32_t>(page) <
                                                 static_cast<uint32_t>(a.pool.num_pages);
                const int64_t slot = (h << shift) + (tok & ((1 << shift) - 1));
                const uint8_t* src = (is_v ? a.pool.vs : a.pool.ks) +
                                     (ok ? page * a.pool.scale_stride + slot : 0);
                cp16(smem_addr(st + 2 * S::kTensor + is_v * kFewBlock + 16 * i), src, ok);
            }
        };
#pragma unroll
        for (int i = 0; i < S::kStages - 1; ++i) {
            if (b0 + i < b1) load_block(b0 + i, i);
            load_ids(b0 + i + S::kStages - 1);
            cp_commit();
        }

        // B fragments of Q^T: row 8 j + g of the tile; with 8-bit pages, position k of MMA m is
        // element 64 (m / 4) + 16 t + 4 (m % 4) + ... of the row, as the K codes are read below
        uint32_t qb[NT][8][2];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int r = 8 * j + g;
            const bool ok = r < nrow;
            const int rr = first + (ok ? r : 0);
            const uint32_t* qr = reinterpret_cast<const uint32_t*>(
                a.q + (v.row0 + rr / G) * a.q_ld + (h * G + rr % G) * D);
#pragma unroll
            for (int m = 0; m < 8; ++m) {
                const int i0 = kE4m3 ? 32 * (m >> 2) + 8 * t + 2 * (m & 3) : 8 * m + t;
                const int i1 = kE4m3 ? i0 + 1 : i0 + 4;
                qb[j][m][0] = ok ? qr[i0] : 0u;
                qb[j][m][1] = ok ? qr[i1] : 0u;
            }
        }
        int lim[NT][2];
        float mx[NT][2], den[NT][2], o[NT][8][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                lim[j][e] = limit(8 * j + 2 * t + e);
                mx[j][e] = -INFINITY;
                den[j][e] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) o[j][i][0] = o[j][i][1] = o[j][i][2] = o[j][i][3] = 0.0f;
        }

        const int mi = lane >> 3, j8 = lane & 7;
        for (int b = b0; b < b1; ++b) {
            asm volatile("cp.async.wait_group %0;" :: "n"(S::kStages - 2) : "memory");
            __syncthreads();
            const int it = b - b0, ahead = it + S::kStages - 1;
            if (b0 + ahead < b1) load_block(b0 + ahead, ahead % S::kStages);
            load_ids(b0 + ahead + S::kStages - 1);
            cp_commit();
            uint8_t* st = smem + (it % S::kStages) * S::kStage;
            const int32_t page = s_page[b % kIdRing][warp];
            if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.pool.num_pages)) continue;
            const int tok = b * kFewBlock + 16 * warp + g;    // this lane's tokens: tok, tok + 8

            float ka = 1.0f, kb = 1.0f, va = 1.0f, vb = 1.0f;
            if (kE4m3) {
                const uint8_t* sc = st + 2 * S::kTensor + 16 * warp + g;
                ka = scale_value(sc[0]);
                kb = scale_value(sc[8]);
                va = scale_value(sc[kFewBlock]);
                vb = scale_value(sc[kFewBlock + 8]);
            }
            // V of a token that some rows may not see must not reach them: 0 * NaN is NaN, so
            // what is not finite is taken out here and put back into the rows that see it
            const int tok15 = b * kFewBlock + 16 * warp + 15;
            if (end - 1 > shared && tok15 > shared) {
                if (kE4m3) {
                    int bad = INT32_MAX;
                    if (tok + 8 > shared && vb != vb) { bad = tok + 8; vb = 0.0f; }
                    if (tok > shared && va != va) { bad = tok; va = 0.0f; }
                    bad = __reduce_min_sync(0xffffffffu, bad);
                    if (bad < end)
                        for (int i = 0; i < 4; ++i) atomicMin(&s_bad[4 * lane + i], bad);
                } else {
                    for (int i = lane; i < 16 * D; i += 32) {
                        const int row = 16 * warp + i / D, d = i % D, tk = b * kFewBlock + row;
                        uint16_t* e = reinterpret_cast<uint16_t*>(
                            st + S::kTensor + row * S::kRowB +
                            (((d >> 3) ^ (row & 7)) << 4) + (d & 7) * 2);
                        if (tk > shared && (*e & 0x7f80u) == 0x7f80u) {
                            atomicMin(&s_bad[d], tk);
                            *e = 0;
                        }
                    }
                }
                __syncwarp();
            }

            // S^T: 16 tokens x R rows
            float sc[NT][4];
#pragma unroll
            for (int j = 0; j < NT; ++j) sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.0f;
            if (kE4m3) {
                const uint32_t base = smem_addr(st + (16 * warp + g) * S::kRowB);
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const uint32_t at = base + (((4 * hh + t) ^ ((g & 1) << 2)) << 4);
                    const uint4 lo = lds128(at), up = lds128(at + 8 * S::kRowB);
                    const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w};
                    const uint32_t wu[4] = {up.x, up.y, up.z, up.w};
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        const uint32_t f[4] = {widen2(prmt_i<0x1404>(wl[m], 0)),
                                               widen2(prmt_i<0x1404>(wu[m], 0)),
                                               widen2(prmt_i<0x3424>(wl[m], 0)),
                                               widen2(prmt_i<0x3424>(wu[m], 0))};
#pragma unroll
                        for (int j = 0; j < NT; ++j)
                            mma_bf16(sc[j], f, qb[j][4 * hh + m][0], qb[j][4 * hh + m][1]);
                    }
                }
            } else {
                const int krow = 16 * warp + j8 + 8 * (mi & 1), kc = mi >> 1;
                const uint32_t base = smem_addr(st + krow * S::kRowB);
#pragma unroll
                for (int m = 0; m < 8; ++m) {
                    uint32_t f[4];
                    ldsm_x4(base + (((2 * m + kc) ^ (krow & 7)) << 4), f);
#pragma unroll
                    for (int j = 0; j < NT; ++j) mma_bf16(sc[j], f, qb[j][m][0], qb[j][m][1]);
                }
            }

            // softmax; the weights as B fragments (k = tokens, n = rows)
            uint32_t pb[NT][kParts][2];
            const float fa = qs * ka, fb = qs * kb;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float w[4];
                float co[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float s0 = tok <= lim[j][e] ? sc[j][e] * fa : -INFINITY;
                    const float s1 = tok + 8 <= lim[j][e] ? sc[j][2 + e] * fb : -INFINITY;
                    float bm = fmaxf(s0, s1);
#pragma unroll
                    for (int k = 4; k < 32; k <<= 1)
                        bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, k));
                    const float m1 = fmaxf(mx[j][e], bm);
                    const float ms = m1 == -INFINITY ? 0.0f : m1;
                    co[e] = exp2f(mx[j][e] - ms);
                    const float p0 = exp2f(s0 - ms), p1 = exp2f(s1 - ms);
                    float sum = p0 + p1;
#pragma unroll
                    for (int k = 4; k < 32; k <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
                    den[j][e] = den[j][e] * co[e] + sum;
                    mx[j][e] = m1;
                    // (a masked token's scale may be anything)
                    w[e] = tok <= lim[j][e] ? p0 * va : 0.0f;
                    w[2 + e] = tok + 8 <= lim[j][e] ? p1 * vb : 0.0f;
                }
                if (!__all_sync(0xffffffffu, co[0] == 1.0f && co[1] == 1.0f)) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        o[j][i][0] *= co[0]; o[j][i][1] *= co[1];
                        o[j][i][2] *= co[0]; o[j][i][3] *= co[1];
                    }
                }
#pragma unroll
                for (int k = 0; k < kParts; ++k) {
                    const uint32_t h01 = bf2(w[0], w[1]), h23 = bf2(w[2], w[3]);
                    pb[j][k][0] = movm_t(h01);
                    pb[j][k][1] = movm_t(h23);
                    const float2 f01 = bf2_f(h01), f23 = bf2_f(h23);
                    w[0] -= f01.x; w[1] -= f01.y; w[2] -= f23.x; w[3] -= f23.y;
                }
            }

            // O^T += V^T P^T. MMA i covers elements 16 i + g and 16 i + g + 8 of a row (bf16),
            // or 16 g + 2 i and 16 g + 2 i + 1 (8-bit)
            if (kE4m3) {
                uint32_t wv[4][4];   // rows 2t, 2t+1, 2t+8, 2t+9: 16 codes from element 16 g on
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int row = 16 * warp + 2 * t + (k & 1) + 8 * (k >> 1);
                    const uint4 q4 = lds128(smem_addr(st + S::kTensor + row * S::kRowB) +
                                            ((g ^ (((row >> 1) & 3) << 1)) << 4));
                    wv[k][0] = q4.x; wv[k][1] = q4.y; wv[k][2] = q4.z; wv[k][3] = q4.w;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int w = i >> 1;
                    // the same element of two neighbouring tokens, side by side
                    uint32_t f[4];
                    if (i & 1) {
                        f[0] = widen2(prmt_i<0x6020>(wv[0][w], wv[1][w]));
                        f[1] = widen2(prmt_i<0x7030>(wv[0][w], wv[1][w]));
                        f[2] = widen2(prmt_i<0x6020>(wv[2][w], wv[3][w]));
                        f[3] = widen2(prmt_i<0x7030>(wv[2][w], wv[3][w]));
                    } else {
                        f[0] = widen2(prmt_i<0x4000>(wv[0][w], wv[1][w]));
                        f[1] = widen2(prmt_i<0x5010>(wv[0][w], wv[1][w]));
                        f[2] = widen2(prmt_i<0x4000>(wv[2][w], wv[3][w]));
                        f[3] = widen2(prmt_i<0x5010>(wv[2][w], wv[3][w]));
                    }
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int k = 0; k < kParts; ++k)
                            mma_bf16(o[j][i], f, pb[j][k][0], pb[j][k][1]);
                }
            } else {
                const int vrow = 16 * warp + j8 + 8 * (mi >> 1), vc = mi & 1;
                const uint32_t base = smem_addr(st + S::kTensor + vrow * S::kRowB);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    uint32_t f[4];
                    ldsm_x4_t(base + (((2 * i + vc) ^ (vrow & 7)) << 4), f);
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int k = 0; k < kParts; ++k)
                            mma_bf16(o[j][i], f, pb[j][k][0], pb[j][k][1]);
                }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();   // the stages become the merge scratch

        float* scr = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float* w = scr + (warp * R + 8 * j + 2 * t + e) * kPart;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    w[kE4m3 ? 16 * g + 2 * i : 16 * i + g] = o[j][i][e];
                    w[kE4m3 ? 16 * g + 2 * i + 1 : 16 * i + g + 8] = o[j][i][2 + e];
                }
                if (g == 0) {
                    w[D] = mx[j][e];
                    w[D + 1] = den[j][e];
                }
            }
        __syncthreads();
        const bool whole = b0 == 0 && b1 == nb;
        float* part = a.work + (2 * static_cast<int64_t>(blockIdx.x) + (b0 == 0)) * part_floats(R);
        for (int r = warp; r < nrow; r += kFW) {
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kFW; ++w) M = fmaxf(M, scr[(w * R + r) * kPart + D]);
            const float ms = M == -INFINITY ? 0.0f : M;
            float dn = 0.0f, y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int w = 0; w < kFW; ++w) {
                const float* src = scr + (w * R + r) * kPart;
                const float f = exp2f(src[D] - ms);
                dn += src[D + 1] * f;
                const float4 z = *reinterpret_cast<const float4*>(src + 4 * lane);
                y[0] += z.x * f; y[1] += z.y * f; y[2] += z.z * f; y[3] += z.w * f;
            }
            const int lr = limit(r);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (s_bad[4 * lane + i] <= lr) y[i] = __uint_as_float(0x7fc00000u);
            if (whole) {
                const float inv = dn == 0.0f ? 0.0f : 1.0f / dn;
                const int rr = first + r;
                const int64_t at = (v.row0 + rr / G) * (static_cast<int64_t>(a.heads) * G) +
                                   h * G + rr % G;
                Out* dst = static_cast<Out*>(a.out) + at * D + 4 * lane;
                if constexpr (sizeof(Out) == 2)
                    *reinterpret_cast<uint2*>(dst) =
                        make_uint2(bf2(y[0] * inv, y[1] * inv), bf2(y[2] * inv, y[3] * inv));
                else
                    *reinterpret_cast<float4*>(dst) =
                        make_float4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
                if (a.lse && lane == 0) a.lse[at] = dn == 0.0f ? -INFINITY : M * kLn2 + logf(dn);
            } else {
                *reinterpret_cast<float4*>(part + r * D + 4 * lane) =
                    make_float4(y[0], y[1], y[2], y[3]);
                if (lane == 0) {
                    part[R * D + r] = M;
                    part[R * D + R + r] = dn;
                }
            }
        }
        __syncthreads();   // the scratch becomes the stages again
        x = start + b1;
        if (b1 == nb && ++tile == nt) {
            tile = 0;
            ++h;
        }
    }
}

template <bool kE4m3, int kParts, typename Out>
cudaError_t launch_few(const AttendArgs& a, int ctas, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    constexpr int smem = FewShape<kE4m3>::kSmem;
    auto kernel = attend_few_kernel<kE4m3, 2, kParts, Out>;
    const cudaError_t e = raise_smem_limit(kernel, smem, done);
    if (e != cudaSuccess) return e;
    kernel<<<ctas, kFW * 32, smem, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

int few_ctas(int sms) { return 2 * sms; }

cudaError_t launch_attend_few(const AttendArgs& a, int format, bool f32_out, int ctas,
                              cudaStream_t st) {
    if (format == PARISKV_PAGES_E4M3)
        return f32_out ? launch_few<true, 3, float>(a, ctas, st)
                       : launch_few<true, 2, __nv_bfloat16>(a, ctas, st);
    return f32_out ? launch_few<false, 3, float>(a, ctas, st)
                   : launch_few<false, 2, __nv_bfloat16>(a, ctas, st);
}

}  // namespace pkv
