// Attention of a batch's new rows over each sequence's own cache and, where the
// sequences continue one prompt, over that prompt's cache.
//
// Row r of sequence b sees the prompt's slots [0, P), its sequence's slots
// [0, s_b) and the call's rows that its mask names:
//     out = sum_j p_j v_j / sum_j p_j,   p_j = 2^(c q.k_j - m),   c = scale log2 e,
// with m the largest exponent seen.  The prompt is read once for the whole
// batch: the query vectors of all sequences and of a KV head's group of query
// heads form one list (vector i of KV head g: row i / G, head g G + i % G), and
// every tile of prompt keys meets all of them.  Each part of a row's keys (a
// range of the prompt, a range of the sequence's own slots) leaves a partial
// state (m, sum p, sum p v) in 32 bits; one warp a (row, head) joins them.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "attend.cuh"

namespace spec {

constexpr int kRowThreads = 128;
// Query vectors a KV head up to which the row kernel takes the prompt: 16, and 64 where (blocks of 16)
// x KV heads x slots are few.  Measured per call (us, row kernel / tile kernel; 8 KV heads, 8 bits, sequences of
// one row behind 32 slots of their own): 16 vectors over 32768 slots 31 / 51; 32 over 32768 44 / 53 (bf16
// 50 / 48); 32 over 4096 19 / 24; 64 over 4096 27 / 28; 64 over 512 17 / 25; 128 over 512 24 / 30.
constexpr int kRowVectors = 16, kRowVectorsShort = 64, kRowKeysShort = 65536;
// least keys of a range: one sequence of 256 slots takes 12.8 us a call at 256, 10.8 at 128, 14.5 at 512; 16 of
// 10 rows over 671 slots 33 at 256, 35 at 128, 37 at 512
constexpr int kMinKeys = 256;

SPEC_DEV void mma16816_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// ---------------------------------------------------------------------------
// The row kernel: 16 query vectors a CTA, the M side of mma.sync m16n8k16, its
// four warps in turn on 16-key tiles that go from global memory to fragments,
// the next tile's loads ahead of this one's arithmetic in 8-bit caches.  Inside
// a k-step the order of the head dimensions, and inside a tile the order of the
// keys, is free (both factors use the same), so they are chosen such that every
// load is a piece of a K or V row and that the scores' accumulator fragment is
// P's operand fragment:
//   lane (g, c) = (lane / 4, lane % 4);
//   scores, key half h: column g is tile key 4 (g / 2) + 2 h + g % 2, so lane
//     (g, c) ends with keys 4c .. 4c+3 of rows g and g + 8;
//   k-step of dims: bf16 piece p of a K row (8 dims at 32 p + 8 c) serves two
//     k-steps, an e4m3 piece (16 dims at 64 p + 16 c) four;
//   values: n-tile nt of column g is dim (hd / 8) g + nt, so lane (g, c) reads
//     hd / 8 consecutive dims of V rows 4c .. 4c+3.
//
// bf16 caches: P is split into bf16 hi + lo, so its rounding does not show.
// Windows (WIN): the list of keys leaves out what lies between the sinks and the
// first row's window, and only tiles that not every row sees whole take masks.  64
// sequences of one row over windows of 4096, 8 KV heads of 128: 144 us a call, 6.5 TB/s,
// 96 % of a copy's rate.
//
// 8-bit caches: products in f16, which holds every e4m3 value (one conversion
// for two values; to bf16 it takes four).  The queries are scaled by a power of
// two a row to a magnitude of 2^13 .. 2^14 (bf16 queries stay exact down to
// 2^-31 of the row's largest); a key's 2^e multiplies its scores; a value's
// 2^e goes into the exponent of its probability, relative to a maximum of its
// own (R, over s + e): P' = 2^(15 + s + e - R) is at most 2^15 and in f16 off by
// 2^-11 of itself (the cache's own values are off by 2^-4 of what was written),
// below 2^-29 of the row's largest by 2^-40 of it; the sum of p takes p in 32 bits.
// f32 queries are split into hi + lo (QF32).
//
// Bound by latency: 64 sequences of 512 slots on average (hd 128, 8 KV heads, 8 bits, 4
// vectors) take 28 us, 2.4 TB/s, of which half a CTA's life is its start (lengths, pages,
// queries, first tiles) and end (the warps' states joined); a warp has five tiles of 2500
// cycles, 600 instructions a tile with the starts shared out, and the issue slots are 34 %
// used.  One long cache does better: 8 vectors over 32768 slots of 32 KV heads take 72 us a
// call in 8 bits (3.7 TB/s) and 89 in bf16 (6.0 TB/s, 89 % of the measured copy rate).
//
// 8-bit caches: a lane's pieces of the next two tiles are copied ahead into shared memory, in slots of
// the lane's own: no other lane reads them, so a lane waits for its own copies only (8 vectors over
// 32768 keys and 32 KV heads: 82 us; one tile ahead in registers: 95).  bf16 tiles go straight to
// registers: the tile as it is loaded is its fragments (94 us; through shared memory: 127).
SPEC_DEV int few_v_key(int cq, int r) { return 2 * cq + (r & 1) + 8 * (r >> 1); }

template <int HD, bool FEW>
struct TileSlot {
    static constexpr int kStages = 2;                  // tiles ahead
    static constexpr int kK = HD / 32;                 // 16-byte pieces of K a lane
    static constexpr int kVBytes = HD / 8;             // bytes of each of its four V rows
    static constexpr int kWords = FEW ? 4 : 2;         // words of exponents a lane
    static constexpr int kVAt = 32 * 16 * kK, kWordsAt = kVAt + 32 * kVBytes * 4;
    static constexpr int kBytes = kWordsAt + 32 * 4 * kWords;
    static constexpr int kRing = 4 * kStages * kBytes;
};

template <int BYTES>
SPEC_DEV void copy_ahead(uint32_t dst, const void* src) {
    if (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" :: "r"(dst), "l"(src), "n"(BYTES) : "memory");
}
SPEC_DEV void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
SPEC_DEV void copies_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

// first row of the 16-key tile at kt (0 past the range's end): tiles start at multiples of 16 and pages
// hold a multiple of 16 slots, so no tile crosses a page
template <bool WIN>
SPEC_DEV long long tile_row(const AttendArgs& a, const CacheView& cv, const KeyMap& km, int seq, int g, int kt, int k_end) {
    return kt < k_end ? kv_row_in_layer(cv.pages, a.Hkv, seq, g, key_slot<WIN>(km, kt)) : 0;
}

// this lane's pieces of the tile at kt, whose first row is `row`, into its slots
template <int HD, bool FEW>
SPEC_DEV void copy_tile(const AttendArgs& a, const CacheView& cv, long long row, int kt, int k_end, uint32_t slot) {
    using S = TileSlot<HD, FEW>;
    const int lane = threadIdx.x & 31, gq = lane >> 2, cq = lane & 3, last = k_end - 1 - kt;
    if (row < 0) { dev_error(a.err, SPEC_DEVERR_CAPACITY); row = 0; }
    const char* K = static_cast<const char*>(cv.k) + row * HD;
    const char* V = static_cast<const char*>(cv.v) + row * HD;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int key = min(FEW ? gq + 8 * h : 4 * (gq >> 1) + 2 * h + (gq & 1), last);
#pragma unroll
        for (int p = 0; p < S::kK / 2; ++p)
            copy_ahead<16>(slot + 512 * (h * (S::kK / 2) + p) + 16 * lane, K + key * HD + 16 * (4 * p + cq));
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int key = min(FEW ? few_v_key(cq, r) : 4 * cq + r, last);
        copy_ahead<S::kVBytes>(slot + S::kVAt + S::kVBytes * (32 * r + lane), V + key * HD + S::kVBytes * gq);
    }
    // the pages hold a multiple of 16 slots: four exponents are one aligned word
#pragma unroll
    for (int w = 0; w < S::kWords; ++w) {
        const uint8_t* e = (w >= S::kWords / 2 ? cv.ve : cv.ke) + row;
        copy_ahead<4>(slot + S::kWordsAt + 4 * (32 * w + lane), e + 4 * (FEW ? 2 * (w & 1) + (gq >> 2) : cq));
    }
}

// QB (16 or 8) query vectors: rows to shared memory in 32 bits, then fragments in lane order
// (dims as the K pieces of the cache's kind order them), as the A operand of 16 rows or the B
// operand of 8 columns.  sS: the factor of a row's raw scores.
template <int HD, int QB>
struct QueryPieces { float x[(QB * HD / 8 + kRowThreads - 1) / kRowThreads][8]; };

// this thread's pieces of the query rows from memory
template <int HD, bool QF32, int QB>
SPEC_DEV void fetch_queries(const AttendArgs& a, int g, int G, int list_row0, int q0, int nq, QueryPieces<HD, QB>& qp) {
    constexpr int N = sizeof(qp.x) / sizeof(qp.x[0]);
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int i = threadIdx.x + n * kRowThreads, r = i / (HD / 8), ch = i % (HD / 8), qg = q0 + r;
        float (&x)[8] = qp.x[n];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 0.f;
        if (r >= nq) continue;
        const long long off = (list_row0 + qg / G) * a.q_stride + (g * G + qg % G) * HD + ch * 8;
        if (QF32) {
            const float* p = static_cast<const float*>(a.q) + off;
            const float4 u = *reinterpret_cast<const float4*>(p), w = *reinterpret_cast<const float4*>(p + 4);
            x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w; x[4] = w.x; x[5] = w.y; x[6] = w.z; x[7] = w.w;
        } else {
            const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(a.q) + off;
            if (a.q_vec) {
                const uint4 w = *reinterpret_cast<const uint4*>(p);
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[2 * e] = __uint_as_float(u[e] << 16);
                    x[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = __bfloat162float(p[e]);
            }
        }
    }
}

template <int HD, bool QF32, int QB>
SPEC_DEV void load_queries(const AttendArgs& a, bool q8, const QueryPieces<HD, QB>& qp, uint4* sQ, float* sS, float* rows) {
    constexpr int KS = HD / 16, LD = HD + 4, N = sizeof(qp.x) / sizeof(qp.x[0]);
    const int t = threadIdx.x;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int i = t + n * kRowThreads, r = i / (HD / 8), ch = i % (HD / 8);
        if (i >= QB * (HD / 8)) break;                      // whole warps
        const float (&x)[8] = qp.x[n];
        // the row's largest magnitude, over the HD / 8 lanes that hold it
        float m = finite_amax(x);
#pragma unroll
        for (int o = HD / 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        // 2^13 .. 2^14 after scaling (the factor at most 2^100)
        const int e = q8 ? min(127 + 13 - (int)(__float_as_uint(m) >> 23), 100) : 0;
        const float f = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
        for (int k = 0; k < 8; k += 4)
            *reinterpret_cast<float4*>(rows + r * LD + ch * 8 + k) = make_float4(x[k] * f, x[k + 1] * f, x[k + 2] * f, x[k + 3] * f);
        if (ch == 0) sS[r] = a.c * __uint_as_float((uint32_t)(127 - e) << 23);
    }
    __syncthreads();
    for (int i = t; i < KS * 32; i += kRowThreads) {
        const int ks = i / 32, ln = i % 32, fg = ln >> 2, fc = ln & 3;
        const int d0 = q8 ? 64 * (ks >> 2) + 16 * fc + 4 * (ks & 3) : 32 * (ks >> 1) + 8 * fc + 4 * (ks & 1);
        const float4 u = *reinterpret_cast<const float4*>(rows + fg * LD + d0);
        if (QB == 8) {
            uint2* s8 = reinterpret_cast<uint2*>(sQ);
            s8[i] = q8 ? make_uint2(pack_f16(u.x, u.y), pack_f16(u.z, u.w)) : make_uint2(pack_bf16(u.x, u.y), pack_bf16(u.z, u.w));
            if (QF32)
                s8[KS * 32 + i] = q8 ? make_uint2(pack_f16(u.x - f16_round(u.x), u.y - f16_round(u.y)),
                                                  pack_f16(u.z - f16_round(u.z), u.w - f16_round(u.w)))
                                     : make_uint2(pack_bf16_lo(u.x, u.y), pack_bf16_lo(u.z, u.w));
            continue;
        }
        const float4 w = *reinterpret_cast<const float4*>(rows + (fg + 8) * LD + d0);
        if (q8) {
            sQ[i] = make_uint4(pack_f16(u.x, u.y), pack_f16(w.x, w.y), pack_f16(u.z, u.w), pack_f16(w.z, w.w));
            if (QF32)
                sQ[KS * 32 + i] = make_uint4(pack_f16(u.x - f16_round(u.x), u.y - f16_round(u.y)),
                                             pack_f16(w.x - f16_round(w.x), w.y - f16_round(w.y)),
                                             pack_f16(u.z - f16_round(u.z), u.w - f16_round(u.w)),
                                             pack_f16(w.z - f16_round(w.z), w.w - f16_round(w.w)));
        } else {
            sQ[i] = make_uint4(pack_bf16(u.x, u.y), pack_bf16(w.x, w.y), pack_bf16(u.z, u.w), pack_bf16(w.z, w.w));
            if (QF32)
                sQ[KS * 32 + i] = make_uint4(pack_bf16_lo(u.x, u.y), pack_bf16_lo(w.x, w.y), pack_bf16_lo(u.z, u.w), pack_bf16_lo(w.z, w.w));
        }
    }
}

// two values of which one is NaN or an infinity (f16: as bits of an exponent of ones)
template <bool Q8>
SPEC_DEV bool not_finite2(uint32_t w) {
    constexpr uint32_t E = Q8 ? 0x7C00u : 0x7F80u;
    return (w & E) == E || (w & (E << 16)) == (E << 16);
}

// P' of 8-bit caches: up to the top of f16's range, so that its smallest numbers lie far below any weight that counts
constexpr float kF16Top = 32768.f;

// running state of a lane's two rows: m and l of the sums of p (l over the lane's keys; joined
// over the quad at the end), R the reference of O (8-bit caches; else R = m)
template <int HD>
struct RowState { float o[HD / 8][4], m[2], l[2], R[2]; };

template <int HD>
SPEC_DEV void scale_rows(RowState<HD>& s, float f0, float f1) {
    // most tiles raise no maximum
    if (__all_sync(0xffffffffu, f0 == 1.f && f1 == 1.f)) return;
#pragma unroll
    for (int nt = 0; nt < HD / 8; ++nt) {
        s.o[nt][0] *= f0;
        s.o[nt][1] *= f0;
        s.o[nt][2] *= f1;
        s.o[nt][3] *= f1;
    }
}

// x: the tile's scores of this lane's two rows; y: what the exponents of P are (x, or x + e).
// Leaves P in y and returns O's factors.
template <bool Q8>
SPEC_DEV void softmax_tile(float (&x)[2][4], float (&y)[2][4], float (&m)[2], float (&l)[2], float (&R)[2], float (&f)[2]) {
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
        float mt = fmaxf(fmaxf(x[rr][0], x[rr][1]), fmaxf(x[rr][2], x[rr][3]));
        mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 1));
        mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 2));
        const float mn = fmaxf(m[rr], mt), mu = mn == -INFINITY ? 0.f : mn;   // nothing seen yet: p = 0
        const float alpha = ex2(m[rr] - mu);
        float ps = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[rr][e] = ex2(x[rr][e] - mu);
            ps += x[rr][e];
        }
        l[rr] = l[rr] * alpha + ps;
        m[rr] = mn;
        if (Q8) {
            float rt = fmaxf(fmaxf(y[rr][0], y[rr][1]), fmaxf(y[rr][2], y[rr][3]));
            rt = fmaxf(rt, __shfl_xor_sync(0xffffffffu, rt, 1));
            rt = fmaxf(rt, __shfl_xor_sync(0xffffffffu, rt, 2));
            const float rn = fmaxf(R[rr], rt), ru = rn == -INFINITY ? 0.f : rn;
            f[rr] = R[rr] == rn ? 1.f : ex2(R[rr] - ru);
            R[rr] = rn;
#pragma unroll
            for (int e = 0; e < 4; ++e) y[rr][e] = ex2(y[rr][e] - ru) * kF16Top;
        } else {
            f[rr] = alpha;
#pragma unroll
            for (int e = 0; e < 4; ++e) y[rr][e] = x[rr][e];
        }
    }
}

// Keys [k_begin, k_end) of one (sequence, KV head) against the CTA's queries.
// Keys below n_ctx are seen by every row; key n_ctx + x by the rows whose mask has bit x.
template <int HD, bool Q8, bool QF32, bool WIN>
SPEC_DEV void attend_range(const AttendArgs& a, const CacheView& cv, const KeyMap& km, int seq, int g, int k_begin, int k_end,
                           int n_ctx, const QueryPieces<HD, 16>& qp, const RowSight* sSight, uint4* sQ, float* sS,
                           float* rows, char* ring, RowState<HD>& st) {
    constexpr int KS = HD / 16, VD = HD / 8;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gq = lane >> 2, cq = lane & 3;
    using S = TileSlot<HD, false>;
    const uint32_t slot0 = smem_u32(ring) + warp * S::kStages * S::kBytes;
    const char* slots = ring + warp * S::kStages * S::kBytes;
    int kt = k_begin + 16 * warp;
    // the first tiles' copies go out before the queries are taken; rows are looked up a tile before their use
    long long row = tile_row<WIN>(a, cv, km, seq, g, kt, k_end), row_nx = tile_row<WIN>(a, cv, km, seq, g, kt + 64, k_end);
    if (Q8) {
        const long long row_2 = tile_row<WIN>(a, cv, km, seq, g, kt + 64 * S::kStages, k_end);
        if (kt < k_end) copy_tile<HD, false>(a, cv, row, kt, k_end, slot0);
        copies_commit();
        if (kt + 64 < k_end) copy_tile<HD, false>(a, cv, row_nx, kt + 64, k_end, slot0 + S::kBytes);
        copies_commit();
        row_nx = row_2;
    }
    load_queries<HD, QF32, 16>(a, Q8, qp, sQ, sS, rows);
    __syncthreads();
    const float c0 = sS[gq], c1 = sS[gq + 8];
    const RowSight see0 = sSight[gq], see1 = sSight[gq + 8];
    for (int stage = 0; kt < k_end; kt += 64, stage = stage + 1 < S::kStages ? stage + 1 : 0) {
        const char* slot = slots + stage * S::kBytes;
        auto k_piece = [&](int h, int p) { return *reinterpret_cast<const uint4*>(slot + 512 * (h * (S::kK / 2) + p) + 16 * lane); };
        if (Q8) copies_wait<S::kStages - 1>();
        uint32_t kb[2][KS][2], vb[4][KS];
        uint32_t ke = 0, ve = 0;
        if (Q8) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int p = 0; p < HD / 64; ++p) {
                    const uint4 u = k_piece(h, p);
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        kb[h][4 * p + s][0] = e4m3x2_f16(w[s]);
                        kb[h][4 * p + s][1] = e4m3x2_f16(w[s] >> 16);
                    }
                }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if (S::kVBytes == 16) {
                    const uint4 w = *reinterpret_cast<const uint4*>(slot + S::kVAt + 16 * (32 * r + lane));
                    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int i = 0; i < HD / 32; ++i) { vb[r][2 * i] = e4m3x2_f16(u[i]); vb[r][2 * i + 1] = e4m3x2_f16(u[i] >> 16); }
                } else {
                    const uint2 w = *reinterpret_cast<const uint2*>(slot + S::kVAt + 8 * (32 * r + lane));
                    vb[r][0] = e4m3x2_f16(w.x); vb[r][1] = e4m3x2_f16(w.x >> 16);
                    vb[r][2] = e4m3x2_f16(w.y); vb[r][3] = e4m3x2_f16(w.y >> 16);
                }
            }
            ke = *reinterpret_cast<const uint32_t*>(slot + S::kWordsAt + 4 * lane);
            ve = *reinterpret_cast<const uint32_t*>(slot + S::kWordsAt + 4 * (32 + lane));
            // the slot is read: the tile after the next one into it
            __syncwarp();
            if (kt + 64 * S::kStages < k_end)
                copy_tile<HD, false>(a, cv, row_nx, kt + 64 * S::kStages, k_end, slot0 + stage * S::kBytes);
            copies_commit();
        } else {
            if (row < 0) { dev_error(a.err, SPEC_DEVERR_CAPACITY); row = 0; }
            const __nv_bfloat16* K = static_cast<const __nv_bfloat16*>(cv.k) + row * HD;
            const __nv_bfloat16* V = static_cast<const __nv_bfloat16*>(cv.v) + row * HD;
            const int last = k_end - 1 - kt;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int key = min(4 * (gq >> 1) + 2 * h + (gq & 1), last);
#pragma unroll
                for (int p = 0; p < HD / 32; ++p) {
                    const uint4 w = __ldg(reinterpret_cast<const uint4*>(K + key * HD) + 4 * p + cq);
                    kb[h][2 * p][0] = w.x; kb[h][2 * p][1] = w.y;
                    kb[h][2 * p + 1][0] = w.z; kb[h][2 * p + 1][1] = w.w;
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int key = min(4 * cq + r, last);
#pragma unroll
                for (int p = 0; p < HD / 64; ++p) {
                    const uint4 w = __ldg(reinterpret_cast<const uint4*>(V + key * HD) + (HD / 64) * gq + p);
                    vb[r][4 * p] = w.x; vb[r][4 * p + 1] = w.y; vb[r][4 * p + 2] = w.z; vb[r][4 * p + 3] = w.w;
                }
            }
            row = row_nx;
        }
        row_nx = tile_row<WIN>(a, cv, km, seq, g, kt + 64 * (Q8 ? S::kStages + 1 : 2), k_end);
        if (kt + 16 > k_end) {
            // values of keys past the range: their probability is zero, and zero times what the slot holds must be zero
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (kt + 4 * cq + r >= k_end)
#pragma unroll
                    for (int i = 0; i < KS; ++i) vb[r][i] = 0u;
        }
        // a new row's NaN or infinity must not reach the rows that do not see it (0 * NaN): it leaves the
        // product, and the rows that see it become NaN
        uint32_t bad = 0;
        const int at_slot = key_slot<WIN>(km, kt);
        const bool edge = at_slot + 16 > n_ctx || (WIN && at_slot < km.low_max);   // not every row sees every key
        if (edge) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                bool b = false;
#pragma unroll
                for (int i = 0; i < KS; ++i) b |= not_finite2<Q8>(vb[r][i]);
                if (!WIN && kt + 4 * cq + r < n_ctx) b = false;
                if (b)
#pragma unroll
                    for (int i = 0; i < KS; ++i) vb[r][i] = 0u;
                // any of the eight lanes that hold the key's values
                if (__ballot_sync(0xffffffffu, b) & (0x11111111u << cq)) bad |= 1u << r;
            }
        }
        // two sums a key half: chains of KS / 2 products
        float sc[2][4], sd[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[h][e] = sd[h][e] = 0.f;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const uint4 qh = sQ[s * 32 + lane];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float (&acc)[4] = s & 1 ? sd[h] : sc[h];
                if (Q8) mma16816_f16(acc, qh.x, qh.y, qh.z, qh.w, kb[h][s][0], kb[h][s][1]);
                else mma16816(acc, qh.x, qh.y, qh.z, qh.w, kb[h][s][0], kb[h][s][1]);
            }
            if (QF32) {
                const uint4 ql = sQ[KS * 32 + s * 32 + lane];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float (&acc)[4] = s & 1 ? sd[h] : sc[h];
                    if (Q8) mma16816_f16(acc, ql.x, ql.y, ql.z, ql.w, kb[h][s][0], kb[h][s][1]);
                    else mma16816(acc, ql.x, ql.y, ql.z, ql.w, kb[h][s][0], kb[h][s][1]);
                }
            }
        }
        // lane: rows g (sc[h][0..1]) and g + 8 (sc[h][2..3]) at keys 4c + 2h + {0, 1}
        float x[2][4], y[2][4], f[2];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float kf = Q8 ? kv8_scale((ke >> (8 * k)) & 0xFF) : 1.f;
            x[0][k] = (sc[k >> 1][k & 1] + sd[k >> 1][k & 1]) * (Q8 ? c0 * kf : c0);
            x[1][k] = (sc[k >> 1][2 + (k & 1)] + sd[k >> 1][2 + (k & 1)]) * (Q8 ? c1 * kf : c1);
        }
        if (edge || kt + 16 > k_end) {                        // ... or a tile that reaches the end
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int slot_k = at_slot + 4 * cq + k;
                const bool in = kt + 4 * cq + k < k_end;
                if (!(in && row_sees<WIN>(km, see0, slot_k, n_ctx))) x[0][k] = -INFINITY;
                if (!(in && row_sees<WIN>(km, see1, slot_k, n_ctx))) x[1][k] = -INFINITY;
                if ((bad >> k) & 1u) {
                    if (x[0][k] != -INFINITY) x[0][k] = __int_as_float(0x7fc00000);
                    if (x[1][k] != -INFINITY) x[1][k] = __int_as_float(0x7fc00000);
                }
            }
        }
        if (Q8) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float e = (float)((int)((ve >> (8 * k)) & 0xFF) - 127);
                y[0][k] = x[0][k] + e;
                y[1][k] = x[1][k] + e;
            }
        }
        softmax_tile<Q8>(x, y, st.m, st.l, st.R, f);
        scale_rows<HD>(st, f[0], f[1]);
        uint32_t pa[4], pl[4];
        if (Q8) {
            pa[0] = pack_f16(y[0][0], y[0][1]); pa[1] = pack_f16(y[1][0], y[1][1]);
            pa[2] = pack_f16(y[0][2], y[0][3]); pa[3] = pack_f16(y[1][2], y[1][3]);
        } else {
            pa[0] = pack_bf16(y[0][0], y[0][1]); pa[1] = pack_bf16(y[1][0], y[1][1]);
            pa[2] = pack_bf16(y[0][2], y[0][3]); pa[3] = pack_bf16(y[1][2], y[1][3]);
            pl[0] = pack_bf16_lo(y[0][0], y[0][1]); pl[1] = pack_bf16_lo(y[1][0], y[1][1]);
            pl[2] = pack_bf16_lo(y[0][2], y[0][3]); pl[3] = pack_bf16_lo(y[1][2], y[1][3]);
        }
#pragma unroll
        for (int nt = 0; nt < VD; ++nt) {
            const int i = nt >> 1;
            const uint32_t b0 = (nt & 1) ? pair_hi(vb[0][i], vb[1][i]) : pair_lo(vb[0][i], vb[1][i]);
            const uint32_t b1 = (nt & 1) ? pair_hi(vb[2][i], vb[3][i]) : pair_lo(vb[2][i], vb[3][i]);
            if (Q8) {
                mma16816_f16(st.o[nt], pa[0], pa[1], pa[2], pa[3], b0, b1);
            } else {
                mma16816(st.o[nt], pa[0], pa[1], pa[2], pa[3], b0, b1);
                mma16816(st.o[nt], pl[0], pl[1], pl[2], pl[3], b0, b1);
            }
        }
    }
    if (!Q8) { st.R[0] = st.m[0]; st.R[1] = st.m[1]; }
}

// The same for at most 8 query vectors: the keys are the M side (16 keys by 8 queries), so a
// tile takes half the products and half the accumulators.
//   scores: lane (g, c) holds keys g and g + 8 of queries 2c and 2c + 1; K pieces as above, of
//     rows g and g + 8;
//   values: O is kept transposed, dims by queries: m-tile mt holds dims (hd / 8) g + 2 mt (row g)
//     and + 1 (row g + 8), so lane (g, c) reads hd / 8 consecutive dims of V rows 2c, 2c + 1,
//     2c + 8, 2c + 9; P goes from the scores' layout to the operand's by a transposing move.
template <int HD>
struct FewState { float o[HD / 16][4], m[2], l[2], R[2]; };

SPEC_DEV uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
template <int HD, bool Q8, bool QF32, bool WIN>
SPEC_DEV void attend_range_few(const AttendArgs& a, const CacheView& cv, const KeyMap& km, int seq, int g, int k_begin, int k_end,
                               int n_ctx, const QueryPieces<HD, 8>& qp, const RowSight* sSight, uint4* sQ4, float* sS,
                               float* rows, char* ring, FewState<HD>& st) {
    constexpr int KS = HD / 16, MT = HD / 16;
    const uint2* sQ = reinterpret_cast<const uint2*>(sQ4);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, gq = lane >> 2, cq = lane & 3;
    using S = TileSlot<HD, true>;
    const uint32_t slot0 = smem_u32(ring) + warp * S::kStages * S::kBytes;
    const char* slots = ring + warp * S::kStages * S::kBytes;
    int kt = k_begin + 16 * warp;
    // the first tiles' copies go out before the queries are taken; rows are looked up a tile before their use
    long long row = tile_row<WIN>(a, cv, km, seq, g, kt, k_end), row_nx = tile_row<WIN>(a, cv, km, seq, g, kt + 64, k_end);
    if (Q8) {
        const long long row_2 = tile_row<WIN>(a, cv, km, seq, g, kt + 64 * S::kStages, k_end);
        if (kt < k_end) copy_tile<HD, true>(a, cv, row, kt, k_end, slot0);
        copies_commit();
        if (kt + 64 < k_end) copy_tile<HD, true>(a, cv, row_nx, kt + 64, k_end, slot0 + S::kBytes);
        copies_commit();
        row_nx = row_2;
    }
    load_queries<HD, QF32, 8>(a, Q8, qp, sQ4, sS, rows);
    __syncthreads();
    const float cf[2] = {sS[2 * cq], sS[2 * cq + 1]};
    for (int stage = 0; kt < k_end; kt += 64, stage = stage + 1 < S::kStages ? stage + 1 : 0) {
        const char* slot = slots + stage * S::kBytes;
        auto k_piece = [&](int h, int p) { return *reinterpret_cast<const uint4*>(slot + 512 * (h * (S::kK / 2) + p) + 16 * lane); };
        if (Q8) copies_wait<S::kStages - 1>();
        uint32_t ka[KS][4], vb[4][MT];
        float kf[2] = {1.f, 1.f}, vf[2] = {0.f, 0.f};
        if (Q8) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int p = 0; p < HD / 64; ++p) {
                    const uint4 u = k_piece(h, p);
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        ka[4 * p + s][h] = e4m3x2_f16(w[s]);
                        ka[4 * p + s][2 + h] = e4m3x2_f16(w[s] >> 16);
                    }
                }
                // the words of keys g and g + 8
                const uint32_t ew = *reinterpret_cast<const uint32_t*>(slot + S::kWordsAt + 4 * (32 * h + lane));
                const uint32_t vw = *reinterpret_cast<const uint32_t*>(slot + S::kWordsAt + 4 * (32 * (2 + h) + lane));
                kf[h] = kv8_scale((ew >> (8 * (gq & 3))) & 0xFF);
                vf[h] = (float)((int)((vw >> (8 * (gq & 3))) & 0xFF) - 127);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if (S::kVBytes == 16) {
                    const uint4 w = *reinterpret_cast<const uint4*>(slot + S::kVAt + 16 * (32 * r + lane));
                    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int i = 0; i < HD / 32; ++i) { vb[r][2 * i] = e4m3x2_f16(u[i]); vb[r][2 * i + 1] = e4m3x2_f16(u[i] >> 16); }
                } else {
                    const uint2 w = *reinterpret_cast<const uint2*>(slot + S::kVAt + 8 * (32 * r + lane));
                    vb[r][0] = e4m3x2_f16(w.x); vb[r][1] = e4m3x2_f16(w.x >> 16);
                    vb[r][2] = e4m3x2_f16(w.y); vb[r][3] = e4m3x2_f16(w.y >> 16);
                }
            }
            // the slot is read: the tile after the next one into it
            __syncwarp();
            if (kt + 64 * S::kStages < k_end)
                copy_tile<HD, true>(a, cv, row_nx, kt + 64 * S::kStages, k_end, slot0 + stage * S::kBytes);
            copies_commit();
        } else {
            if (row < 0) { dev_error(a.err, SPEC_DEVERR_CAPACITY); row = 0; }
            const __nv_bfloat16* K = static_cast<const __nv_bfloat16*>(cv.k) + row * HD;
            const __nv_bfloat16* V = static_cast<const __nv_bfloat16*>(cv.v) + row * HD;
            const int last = k_end - 1 - kt;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int key = min(gq + 8 * h, last);
#pragma unroll
                for (int p = 0; p < HD / 32; ++p) {
                    const uint4 w = __ldg(reinterpret_cast<const uint4*>(K + key * HD) + 4 * p + cq);
                    ka[2 * p][h] = w.x; ka[2 * p][2 + h] = w.y;
                    ka[2 * p + 1][h] = w.z; ka[2 * p + 1][2 + h] = w.w;
                }
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int key = min(few_v_key(cq, r), last);
#pragma unroll
                for (int p = 0; p < HD / 64; ++p) {
                    const uint4 w = __ldg(reinterpret_cast<const uint4*>(V + key * HD) + (HD / 64) * gq + p);
                    vb[r][4 * p] = w.x; vb[r][4 * p + 1] = w.y; vb[r][4 * p + 2] = w.z; vb[r][4 * p + 3] = w.w;
                }
            }
            row = row_nx;
        }
        row_nx = tile_row<WIN>(a, cv, km, seq, g, kt + 64 * (Q8 ? S::kStages + 1 : 2), k_end);
        if (kt + 16 > k_end) {
            // values of keys past the range: their probability is zero, and zero times what the slot holds must be zero
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (kt + few_v_key(cq, r) >= k_end)
#pragma unroll
                    for (int i = 0; i < MT; ++i) vb[r][i] = 0u;
        }
        // a new row's NaN or infinity must not reach the rows that do not see it (0 * NaN): it leaves the
        // product, and the rows that see it become NaN
        uint32_t bad = 0;                                     // bit k: tile key k
        const int at_slot = key_slot<WIN>(km, kt);
        const bool edge = at_slot + 16 > n_ctx || (WIN && at_slot < km.low_max);   // not every row sees every key
        if (edge) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                bool b = false;
#pragma unroll
                for (int i = 0; i < MT; ++i) b |= not_finite2<Q8>(vb[r][i]);
                if (!WIN && kt + few_v_key(cq, r) < n_ctx) b = false;
                if (b)
#pragma unroll
                    for (int i = 0; i < MT; ++i) vb[r][i] = 0u;
                const uint32_t any = __ballot_sync(0xffffffffu, b);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (any & (0x11111111u << c)) bad |= 1u << few_v_key(c, r);
            }
        }
        float sc[2][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[0][e] = sc[1][e] = 0.f;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const uint2 qh = sQ[s * 32 + lane];
            if (Q8) mma16816_f16(sc[s & 1], ka[s][0], ka[s][1], ka[s][2], ka[s][3], qh.x, qh.y);
            else mma16816(sc[s & 1], ka[s][0], ka[s][1], ka[s][2], ka[s][3], qh.x, qh.y);
            if (QF32) {
                const uint2 ql = sQ[KS * 32 + s * 32 + lane];
                if (Q8) mma16816_f16(sc[s & 1], ka[s][0], ka[s][1], ka[s][2], ka[s][3], ql.x, ql.y);
                else mma16816(sc[s & 1], ka[s][0], ka[s][1], ka[s][2], ka[s][3], ql.x, ql.y);
            }
        }
        // x[j][h]: query 2c + j, key g + 8 h; y: what the exponent of P is
        float x[2][2], y[2][2], f[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) x[j][h] = (sc[0][2 * h + j] + sc[1][2 * h + j]) * (Q8 ? cf[j] * kf[h] : cf[j]);
        if (edge || kt + 16 > k_end) {                        // ... or a tile that reaches the end
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const RowSight see = sSight[2 * cq + j];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (!(kt + gq + 8 * h < k_end && row_sees<WIN>(km, see, at_slot + gq + 8 * h, n_ctx))) x[j][h] = -INFINITY;
                    else if ((bad >> (gq + 8 * h)) & 1u) x[j][h] = __int_as_float(0x7fc00000);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float mt = fmaxf(x[j][0], x[j][1]);
            y[j][0] = x[j][0] + vf[0];
            y[j][1] = x[j][1] + vf[1];
            float rt = fmaxf(y[j][0], y[j][1]);
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) {
                mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
                if (Q8) rt = fmaxf(rt, __shfl_xor_sync(0xffffffffu, rt, o));
            }
            const float mn = fmaxf(st.m[j], mt), mu = mn == -INFINITY ? 0.f : mn;   // nothing seen yet: p = 0
            const float alpha = st.m[j] == mn ? 1.f : ex2(st.m[j] - mu);
            const float p0 = ex2(x[j][0] - mu), p1 = ex2(x[j][1] - mu);
            st.l[j] = st.l[j] * alpha + (p0 + p1);            // this lane's keys; joined at the end
            st.m[j] = mn;
            if (Q8) {
                const float rn = fmaxf(st.R[j], rt), ru = rn == -INFINITY ? 0.f : rn;
                f[j] = st.R[j] == rn ? 1.f : ex2(st.R[j] - ru);
                st.R[j] = rn;
                y[j][0] = ex2(y[j][0] - ru) * kF16Top;
                y[j][1] = ex2(y[j][1] - ru) * kF16Top;
            } else {
                f[j] = alpha;
                y[j][0] = p0;
                y[j][1] = p1;
            }
        }
        if (!__all_sync(0xffffffffu, f[0] == 1.f && f[1] == 1.f)) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                st.o[mt][0] *= f[0];
                st.o[mt][1] *= f[1];
                st.o[mt][2] *= f[0];
                st.o[mt][3] *= f[1];
            }
        }
        uint32_t b[2], bl[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            b[h] = transpose8(Q8 ? pack_f16(y[0][h], y[1][h]) : pack_bf16(y[0][h], y[1][h]));
            if (!Q8) bl[h] = transpose8(pack_bf16_lo(y[0][h], y[1][h]));
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const uint32_t a0 = pair_lo(vb[0][mt], vb[1][mt]), a1 = pair_hi(vb[0][mt], vb[1][mt]);
            const uint32_t a2 = pair_lo(vb[2][mt], vb[3][mt]), a3 = pair_hi(vb[2][mt], vb[3][mt]);
            if (Q8) {
                mma16816_f16(st.o[mt], a0, a1, a2, a3, b[0], b[1]);
            } else {
                mma16816(st.o[mt], a0, a1, a2, a3, b[0], b[1]);
                mma16816(st.o[mt], a0, a1, a2, a3, bl[0], bl[1]);
            }
        }
    }
    if (!Q8) { st.R[0] = st.m[0]; st.R[1] = st.m[1]; }
}

constexpr int row_ctas_per_sm(int hd, int qb) { return hd == 128 ? 3 : (qb == 8 ? 5 : 4); }

template <int HD, bool QF32, int QB, bool WIN>
__global__ void __launch_bounds__(kRowThreads, row_ctas_per_sm(HD, QB))
attend_rows_kernel(const __grid_constant__ AttendArgs a) {
    // Behind the tile kernel too: what the launches before that one wrote (the new rows) is visible to a grid
    // that waits, not to one that was only let start.  Working beside the tile kernel took 3 to 9 us less a call.
    pdl_wait();
    pdl_trigger();
    constexpr int KS = HD / 16, VD = HD / 8;
    constexpr int LS = HD + 4;                                              // a state row: O, m, l, R
    extern __shared__ float smf[];
    uint4* sQ = reinterpret_cast<uint4*>(smf);                              // [QF32 ? 2 : 1][KS][32] (8 queries: uint2)
    float* sRows = smf + (QF32 ? 2 : 1) * KS * 32 * (QB / 4);               // [QB][LS] the queries before
    RowSight* sSight = reinterpret_cast<RowSight*>(sRows + QB * LS);        // [QB]
    float* sS = reinterpret_cast<float*>(sSight + QB);                      // [QB]
    float* sState = sS + QB;                                                // [4 warps][QB][LS]
    char* ring = reinterpret_cast<char*>(sState);                           // the tiles, before the states
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, gq = lane >> 2, cq = lane & 3;
    const int G = a.H / a.Hkv;
    // the prompt's blocks first (the longer ones), then the sequences' own
    int id = blockIdx.x;
    // (with a window the sequences see different parts of it, so each has blocks of its own there too)
    const int n_pre = a.pre_splits * a.pre_qb * a.Hkv * (WIN ? a.span.batch : 1);
    const bool is_pre = id < n_pre;
    int b = 0, list_row0 = 0, rows = a.span.T;
    if (!is_pre) id -= n_pre;
    const int g = id % a.Hkv;
    id /= a.Hkv;
    const int qb = id % (is_pre ? a.pre_qb : a.own_qb);
    id /= is_pre ? a.pre_qb : a.own_qb;
    int split, n_splits, n_ctx, n_keys, range;
    int base = 0, prompt = 0;                                               // WIN: index of the first row, length of the prompt
    if (is_pre) {
        split = id;
        n_splits = a.pre_splits;
        n_keys = n_ctx = min(a.pre.len[a.pre_seq], a.pre.cap);
        if (WIN) {
            split = id % a.pre_splits;
            b = id / a.pre_splits;
            list_row0 = a.span.row0[b];
            rows = a.span.row0[b + 1] - list_row0;
            base = n_keys + a.own.len[b] + a.span.extra;
        }
        range = split;
    } else {
        split = id % a.own_splits;
        b = id / a.own_splits;
        n_splits = a.own_splits;
        list_row0 = a.span.row0[b];
        rows = a.span.row0[b + 1] - list_row0;
        n_ctx = a.own.len[b] + a.span.extra;
        n_keys = min(n_ctx + rows, a.own.cap);
        if (n_ctx + rows > a.own.cap && rows > 0 && t == 0) dev_error(a.err, SPEC_DEVERR_CAPACITY);
        range = a.own_range0 + split;
        if (WIN) {
            if (a.pre.len) prompt = min(a.pre.len[a.pre_seq], a.pre.cap);
            base = prompt + n_ctx;
        }
    }
    const int q0 = qb * QB, nq = min(QB, rows * G - q0);
    if (nq <= 0) return;
    QueryPieces<HD, QB> qp;                                                 // on their way while the lengths are read
    fetch_queries<HD, QF32, QB>(a, g, G, list_row0, q0, nq, qp);
    KeyMap km{0, 0, 0, 0};
    if (WIN) {
        // slots that the sequence's first row sees: the later ones see none before them but the sinks
        const int lo = max(0, base - prompt - a.window + 1) & ~15;
        km.sinks = min(max(a.sinks - prompt, 0), n_ctx);
        km.sink_keys = (km.sinks + 15) & ~15;
        km.lo = lo;
        if (km.sink_keys >= lo) km.sink_keys = km.lo = 0;                   // one run of keys
        n_keys = km.lo < n_keys ? km.sink_keys + n_keys - km.lo : min(km.sink_keys, n_keys);
    }
    int chunk = max(kMinKeys, (n_keys + n_splits - 1) / n_splits);
    chunk = (chunk + 63) / 64 * 64;
    const int k_begin = min(n_keys, split * chunk), k_end = min(n_keys, k_begin + chunk);
    const CacheView& cv = is_pre ? a.pre : a.own;
    const int seq = is_pre ? a.pre_seq : b;
    const size_t TH = (size_t)a.span.T * a.H;
    auto vec_of = [&](int r) { return range * TH + (size_t)(list_row0 + (q0 + r) / G) * a.H + g * G + (q0 + r) % G; };
    if (k_begin >= k_end) {                                                 // nothing in this range
        if (WIN && a.direct) {
            for (int i = t; i < nq * HD; i += kRowThreads)
                put_out(a.out, (list_row0 + (q0 + i / HD) / G) * a.out.stride + (g * G + (q0 + i / HD) % G) * HD + i % HD, __int_as_float(0x7fc00000));
            return;
        }
        if (t < nq) *reinterpret_cast<float2*>(a.part_ml + 2 * vec_of(t)) = make_float2(-INFINITY, 0.f);
        return;
    }
    if (t < QB) {
        RowSight rs{0ull, 0};
        const int j = (q0 + t) / G;
        if ((WIN || !is_pre) && t < nq) rs.mask = row_mask(a.span, b, j);
        if (WIN) {
            const int d = t < nq ? __popcll(rs.mask) - 1 : 0;
            rs.low = base - prompt + d - a.window + 1;
            rs.mask = is_pre ? 0ull : window_mask(a.span, b, rs.mask, d, a.window, a.sinks - base);
        }
        sSight[t] = rs;
    }
    // depths are at most the row's index, so no row's bound lies past the last row's
    if (WIN) km.low_max = base - prompt + (q0 + nq - 1) / G - a.window + 1;
    if constexpr (QB == 8) {
        FewState<HD> rs;
#pragma unroll
        for (int j = 0; j < 2; ++j) { rs.m[j] = rs.R[j] = -INFINITY; rs.l[j] = 0.f; }
#pragma unroll
        for (int mt = 0; mt < HD / 16; ++mt) rs.o[mt][0] = rs.o[mt][1] = rs.o[mt][2] = rs.o[mt][3] = 0.f;
        if (cv.q8) attend_range_few<HD, true, QF32, WIN>(a, cv, km, seq, g, k_begin, k_end, n_ctx, qp, sSight, sQ, sS, sRows, ring, rs);
        else attend_range_few<HD, false, QF32, WIN>(a, cv, km, seq, g, k_begin, k_end, n_ctx, qp, sSight, sQ, sS, sRows, ring, rs);
        __syncthreads();                     // the states lie where the tiles were
        // warp states -> shared: queries 2c and 2c + 1, dims VD * g ..
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) rs.l[j] += __shfl_xor_sync(0xffffffffu, rs.l[j], o);
            float* st = sState + ((size_t)warp * QB + 2 * cq + j) * LS;
            if (gq == 0) { st[HD] = rs.m[j]; st[HD + 1] = rs.l[j]; st[HD + 2] = rs.R[j]; }
#pragma unroll
            for (int mt = 0; mt < HD / 16; ++mt)
                *reinterpret_cast<float2*>(st + VD * gq + 2 * mt) = make_float2(rs.o[mt][j], rs.o[mt][2 + j]);
        }
    } else {
        RowState<HD> rs;
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) { rs.m[rr] = rs.R[rr] = -INFINITY; rs.l[rr] = 0.f; }
#pragma unroll
        for (int nt = 0; nt < VD; ++nt) rs.o[nt][0] = rs.o[nt][1] = rs.o[nt][2] = rs.o[nt][3] = 0.f;
        if (cv.q8) attend_range<HD, true, QF32, WIN>(a, cv, km, seq, g, k_begin, k_end, n_ctx, qp, sSight, sQ, sS, sRows, ring, rs);
        else attend_range<HD, false, QF32, WIN>(a, cv, km, seq, g, k_begin, k_end, n_ctx, qp, sSight, sQ, sS, sRows, ring, rs);
        __syncthreads();
        // warp states -> shared: rows g and g + 8, dims VD * 2c + nt and VD * (2c + 1) + nt
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
            rs.l[rr] += __shfl_xor_sync(0xffffffffu, rs.l[rr], 1);
            rs.l[rr] += __shfl_xor_sync(0xffffffffu, rs.l[rr], 2);
            float* st = sState + ((size_t)warp * QB + gq + 8 * rr) * LS;
            if (cq == 0) { st[HD] = rs.m[rr]; st[HD + 1] = rs.l[rr]; st[HD + 2] = rs.R[rr]; }
#pragma unroll
            for (int nt = 0; nt < VD; nt += 4) {
                *reinterpret_cast<float4*>(st + VD * (2 * cq) + nt) =
                    make_float4(rs.o[nt][2 * rr], rs.o[nt + 1][2 * rr], rs.o[nt + 2][2 * rr], rs.o[nt + 3][2 * rr]);
                *reinterpret_cast<float4*>(st + VD * (2 * cq + 1) + nt) =
                    make_float4(rs.o[nt][2 * rr + 1], rs.o[nt + 1][2 * rr + 1], rs.o[nt + 2][2 * rr + 1], rs.o[nt + 3][2 * rr + 1]);
            }
        }
    }
    __syncthreads();
    // the warps' states in warp order: sums relative to the largest m, O first to the largest R, then to m
    for (int i = t; i < nq * (HD / 4); i += kRowThreads) {
        const int r = i / (HD / 4), d = 4 * (i % (HD / 4));
        float M = -INFINITY, RR = -INFINITY;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float* st = sState + ((size_t)w * QB + r) * LS + HD;
            M = fmaxf(M, st[0]);
            RR = fmaxf(RR, st[2]);
        }
        float L = 0.f;
        float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float* st = sState + ((size_t)w * QB + r) * LS;
            if (st[HD] == -INFINITY && !(st[HD + 1] != 0.f)) continue;        // this warp saw nothing
            L += st[HD + 1] * ex2(st[HD] - M);
            const float wt = ex2(st[HD + 2] - RR);
            const float4 o = *reinterpret_cast<const float4*>(st + d);
            O.x = fmaf(o.x, wt, O.x);
            O.y = fmaf(o.y, wt, O.y);
            O.z = fmaf(o.z, wt, O.z);
            O.w = fmaf(o.w, wt, O.w);
        }
        const float f = (M == -INFINITY ? 1.f : ex2(RR - M)) * (cv.q8 ? 1.f / kF16Top : 1.f);
        if (WIN && a.direct) {
            const float inv = f / L;
            const long long at = (list_row0 + (q0 + r) / G) * a.out.stride + (g * G + (q0 + r) % G) * HD + d;
            put_out(a.out, at, O.x * inv);
            put_out(a.out, at + 1, O.y * inv);
            put_out(a.out, at + 2, O.z * inv);
            put_out(a.out, at + 3, O.w * inv);
            continue;
        }
        const size_t vec = vec_of(r);
        *reinterpret_cast<float4*>(a.part_o + vec * HD + d) = make_float4(O.x * f, O.y * f, O.z * f, O.w * f);
        if (d == 0) *reinterpret_cast<float2*>(a.part_ml + 2 * vec) = make_float2(M, L);
    }
}

// The ranges' states of a (row, head) joined: the prompt's, then the sequence's own, by
// one warp (eight ranges in flight), or by four that take every fourth range each and
// whose sums are added in warp order.  Many rows of few ranges are bound by reading the
// states, few rows of many by the latency of it: more than 12 ranges take four warps
// (2048 rows of 21 ranges: 12.5 us by one warp, 8.9 by four; 16384 rows of 5: 39 us by
// four warps).  With the sums fetched beside the maxima 16384 rows of 5 ranges take 12.5 us,
// 2.9 TB/s at half the issue slots, and 2048 rows of 21 ranges 8.4 us, 2.6 TB/s.
struct JoinArgs {
    const float* part_o; const float* part_ml;
    int own_range0, own_ranges, pre_ranges;     // pre_ranges: the row kernel's prompt ranges
    int tile_ctas;                              // > 0: the tile kernel's prompt ranges, counted on the device
    const int* pre_len; int pre_cap;
    int TH, H, G, Hkv;
    __nv_bfloat16* out;
    long long stride;
    size_t lo;                        // 0: one bf16 row; else hi rows and lo rows at this offset
};

template <int HD, int NW>
__global__ void __launch_bounds__(128)
attend_join_kernel(const __grid_constant__ JoinArgs a) {
    pdl_wait();
    pdl_trigger();
    constexpr int E = HD / 32, U = 8;
    __shared__ float sO[3][HD], sL[3];
    const int w = NW == 4 ? threadIdx.x >> 5 : 0, lane = threadIdx.x & 31;
    const int v = NW == 4 ? blockIdx.x : blockIdx.x * 4 + (threadIdx.x >> 5);
    if (NW == 1 && v >= a.TH) return;
    int pre = a.pre_ranges;
    if (a.tile_ctas) {
        const int KB = (min(*a.pre_len, a.pre_cap) + 127) / 128;
        const long long W = (long long)a.Hkv * KB;
        pre = tile_range_count((v % a.H) / a.G, KB, W, tile_ctas_at_work(a.tile_ctas, W));
    }
    const int n = pre + a.own_ranges;
    auto slot = [&](int s) { return (size_t)(s < pre ? s : a.own_range0 + s - pre) * a.TH + v; };
    // U ranges' sums are on their way while the maxima are looked at (those of an empty range, whatever
    // they hold, are dropped)
    float2 ml[U];
    float x[U][E];
    auto fetch = [&](int s0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = s0 + NW * u;
            ml[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int e = 0; e < E; ++e) x[u][e] = 0.f;
            if (s < n) {
                const size_t at = slot(s);
                ml[u] = *reinterpret_cast<const float2*>(a.part_ml + 2 * at);
                const float* src = a.part_o + at * HD + lane * E;
                if (E == 4) {
                    const float4 f = *reinterpret_cast<const float4*>(src);
                    x[u][0] = f.x; x[u][1] = f.y; x[u][E - 2] = f.z; x[u][E - 1] = f.w;
                } else {
                    const float2 f = *reinterpret_cast<const float2*>(src);
                    x[u][0] = f.x; x[u][1] = f.y;
                }
            }
        }
    };
    fetch(w);
    float M = -INFINITY;
    for (int s = lane; s < n; s += 32) M = fmaxf(M, a.part_ml[2 * slot(s)]);
    M = warp_max(M);
    float L = 0.f, O[E];
#pragma unroll
    for (int e = 0; e < E; ++e) O[e] = 0.f;
    if (M != -INFINITY) {
        for (int s0 = w; s0 < n;) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool none = ml[u].x == -INFINITY;
                const float ws = ex2(ml[u].x - M);
                L = fmaf(ml[u].y, ws, L);
#pragma unroll
                for (int e = 0; e < E; ++e) O[e] = fmaf(ws, none ? 0.f : x[u][e], O[e]);
            }
            s0 += NW * U;
            if (s0 < n) fetch(s0);
        }
    }
    if (NW == 4) {
        if (w > 0) {
            if (lane == 0) sL[w - 1] = L;
#pragma unroll
            for (int e = 0; e < E; ++e) sO[w - 1][lane * E + e] = O[e];
        }
        __syncthreads();
        if (w > 0) return;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            L += sL[k];
#pragma unroll
            for (int e = 0; e < E; ++e) O[e] += sO[k][lane * E + e];
        }
    }
    const float inv = 1.0f / L;
    const long long o = (v / a.H) * a.stride + (v % a.H) * HD + lane * E;
    if (a.lo) {
#pragma unroll
        for (int e = 0; e < E; ++e) store_act(a.out, (size_t)(o + e), a.lo, O[e] * inv);
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) a.out[o + e] = __float2bfloat16_rn(O[e] * inv);
    }
}

// ---------------------------------------------------------------------------
// host side

CacheView cache_view(const spec_kv* kv, int layer) {
    const size_t off = (size_t)layer * kv->n_pages * kv->m->cfg.n_kv_heads * kv->page;
    CacheView v{};
    v.k = (const char*)kv->k + off * kv->m->cfg.head_dim * kv->elem;
    v.v = (const char*)kv->v + off * kv->m->cfg.head_dim * kv->elem;
    v.ke = kv->q8 ? kv->ke + off : nullptr;
    v.ve = kv->q8 ? kv->ve + off : nullptr;
    v.pages = kv->pages();
    v.len = kv->len;
    v.cap = kv->max_ctx;
    v.q8 = kv->q8;
    return v;
}

int make_span(AttendSpan* s, int batch, const int* n_rows, int extra, const int* tree_parent, const int* dev_parent) {
    s->batch = batch;
    s->extra = extra;
    s->tree = dev_parent ? 2 : (tree_parent ? 1 : 0);
    s->dev_parent = dev_parent;
    s->max_rows = 0;
    int r = 0;
    for (int b = 0; b < batch; ++b) {
        s->row0[b] = (short)r;
        r += n_rows[b];
        s->max_rows = std::max(s->max_rows, n_rows[b]);
    }
    s->row0[batch] = (short)r;
    s->T = r;
    if (tree_parent && !dev_parent) {
        for (int j = 0; j < s->max_rows; ++j)
            s->mask[j] = (1ull << j) | (j > 0 ? s->mask[tree_parent[j]] : 0ull);
    }
    return SPEC_OK;
}

template <int HD, bool FEW>
static size_t ring_bytes(bool q8) {
    return q8 ? TileSlot<HD, FEW>::kRing : 0;
}
// shared memory of the row kernel; q8: one of its caches is in 8 bits
static size_t rows_smem(int hd, bool qf32, int qb, bool q8) {
    const size_t ring = hd == 128 ? (qb == 8 ? ring_bytes<128, true>(q8) : ring_bytes<128, false>(q8))
                                  : (qb == 8 ? ring_bytes<64, true>(q8) : ring_bytes<64, false>(q8));
    const size_t row = (size_t)(hd + 4) * sizeof(float);
    return (qf32 ? 2 : 1) * (hd / 16) * 32 * qb + qb * (row + sizeof(RowSight) + 4) + std::max(ring, 4 * qb * row);
}

// Query vectors whose partial states fit.  The row kernel's two parts keep to (ranges) x
// (T * H) <= 16 x 512 + T H each.  The tile kernel's CTAs are one an SM, so its ranges
// are (SMs / pairs of query tiles) / Hkv + 2, with T * H <= 256 Hkv (pairs): 256 SMs + 2 T H.
size_t attend_floats_needed(const spec_model* m) {
    const size_t th = (size_t)m->cfg.max_rows * m->cfg.n_heads;
    return (2 * 16 * 512 + 256 * (size_t)m->num_sms + 4 * th) * (m->cfg.head_dim + 2);
}

int launch_attend(spec_kv* kv, int layer, const AttendSpan& span, const void* q, int q_f32, long long q_stride,
                  float scale, const AttendOut& out, cudaStream_t st) {
    spec_model* m = kv->m;
    const spec_model_config& c = m->cfg;
    const int hd = c.head_dim, H = c.n_heads, Hkv = c.n_kv_heads, G = H / Hkv;
    const spec_kv* pre = kv->prefix;
    AttendArgs a{};
    a.q = q;
    a.q_f32 = q_f32;
    a.q_vec = (reinterpret_cast<uintptr_t>(q) & 15) == 0 && q_stride % 8 == 0;
    a.layer = layer;
    a.q_stride = q_stride;
    a.c = scale * 1.4426950408889634f;
    a.own = cache_view(kv, layer);
    if (pre) a.pre = cache_view(pre, layer);
    a.pre_seq = kv->prefix_seq;
    a.H = H;
    a.Hkv = Hkv;
    a.span = span;
    a.err = m->err;
    const int TH = span.T * H;
    const size_t fit = m->attend_part_floats / (hd + 2) / TH;      // ranges the workspace holds
    const long long pre_work = pre ? (long long)((span.T * G + 15) / 16) * Hkv * pre->max_ctx : 0;
    const bool rows_do = span.T * G <= kRowVectors || (span.T * G <= kRowVectorsShort && pre_work <= kRowKeysShort);
    const bool win = kv->window_of(layer) > 0;
    const bool tile = pre && !win && !rows_do && attend_tile_ok(pre);
    // blocks of 8 query vectors where one holds all of a part's, else of 16
    const bool blocks = win && span.max_rows * G > kWindowVectors && attend_window_ok(kv);
    const int QB = blocks ? attend_window_block(span.max_rows * G) : span.max_rows * G <= 8 && (!pre || win || tile || span.T * G <= 8) ? 8 : 16;
    a.own_qb = (span.max_rows * G + QB - 1) / QB;
    a.pre_qb = pre && !tile ? ((win ? span.max_rows : span.T) * G + QB - 1) / QB : 0;
    // the most keys of a part
    long long own_ctx = kv->max_ctx, pre_ctx = pre ? pre->max_ctx : 0;
    if (win) {
        a.window = kv->window_of(layer);
        a.sinks = kv->sinks[layer];
        const long long seen = (long long)a.window + a.sinks + 30;       // whole tiles of both
        own_ctx = std::min(own_ctx, seen + span.max_rows);
        pre_ctx = std::min(pre_ctx, seen);
    }
    const long long own_blocks = (long long)span.batch * Hkv * a.own_qb;
    const long long pre_blocks = (long long)Hkv * a.pre_qb * (win ? span.batch : 1);
    const long long keys = own_blocks * own_ctx + pre_blocks * pre_ctx;
    // ranges: as many CTAs as run at a time, by each part's share of the keys; more only add starts and
    // partial states (8 vectors, 32 KV heads, 32768 slots: one wave 72 us in 8 bits and 89 in bf16, two 86
    // and 117)
    const long long wave = (long long)(blocks ? attend_window_ctas(hd) : row_ctas_per_sm(hd, QB)) * m->num_sms;
    const long long per = std::max<long long>(kMinKeys, keys / wave + 1), round = per > kMinKeys ? per / 2 : per - 1;
    auto splits = [&](long long n_blocks, long long ctx) {
        if (n_blocks == 0) return 0;
        long long n = (ctx + round) / per;
        // whole caches that would be among the longest CTAs are halved: sequences differ in length
        if (!blocks && n == 1 && 2 * ctx > per && ctx > 2 * kMinKeys) n = 2;
        // (windows: all that the workspace holds; it is shared by the two parts)
        const long long most = win ? (long long)fit / (pre ? 2 : 1) : (16 * 512) / (16 * n_blocks) + 1;
        return (int)std::max<long long>(1, std::min<long long>({n, 64, most}));
    };
    a.own_splits = splits(own_blocks, own_ctx);
    a.pre_splits = splits(pre_blocks, pre_ctx);
    int tile_ranges = 0;
    if (tile) {
        a.tile_ctas = attend_tile_ctas(m, span, q_f32, pre->max_ctx);
        while (a.tile_ctas > 1 && (size_t)(a.own_splits + attend_tile_ranges(m, a.tile_ctas)) > fit) --a.tile_ctas;
        tile_ranges = attend_tile_ranges(m, a.tile_ctas);
    }
    a.own_range0 = a.pre_splits + tile_ranges;
    const int ranges = a.own_splits + a.own_range0;
    if ((size_t)ranges > fit) return set_error(SPEC_ERR_CAPACITY, "attention workspace too small");
    a.part_o = m->attend_part;
    a.part_ml = m->attend_part + (size_t)ranges * TH * hd;
    const dim3 grid((unsigned)(a.pre_splits * pre_blocks + a.own_splits * own_blocks));
    const size_t smem = rows_smem(hd, q_f32, QB, a.own.q8 || (a.pre_qb > 0 && a.pre.q8));
    void (*const kernels[16])(AttendArgs) = {
        attend_rows_kernel<64, false, 8, false>, attend_rows_kernel<64, false, 16, false>,
        attend_rows_kernel<64, true, 8, false>, attend_rows_kernel<64, true, 16, false>,
        attend_rows_kernel<128, false, 8, false>, attend_rows_kernel<128, false, 16, false>,
        attend_rows_kernel<128, true, 8, false>, attend_rows_kernel<128, true, 16, false>,
        attend_rows_kernel<64, false, 8, true>, attend_rows_kernel<64, false, 16, true>,
        attend_rows_kernel<64, true, 8, true>, attend_rows_kernel<64, true, 16, true>,
        attend_rows_kernel<128, false, 8, true>, attend_rows_kernel<128, false, 16, true>,
        attend_rows_kernel<128, true, 8, true>, attend_rows_kernel<128, true, 16, true>};
    const int which = (win ? 8 : 0) + (hd == 128 ? 4 : 0) + (q_f32 ? 2 : 0) + (QB == 16 ? 1 : 0);
    void (*f)(AttendArgs) = kernels[which];
    static std::atomic<unsigned long long> set[16] = {};       // devices where a kernel may take more than 48 KB
    const unsigned long long bit = 1ull << (m->device & 63);
    if (smem > 48 * 1024 && !(set[which].load() & bit)) {
        SPEC_TRY(check_cuda(cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)rows_smem(hd, true, QB, true)),
                            "attention rows attribute"));
        set[which].fetch_or(bit);
    }
    a.out = out;
    a.direct = win && !pre && a.own_splits == 1;
    const int slot = prof_start(m, st);
    if (tile) SPEC_TRY(launch_attend_tile(pre, a, st));
    cudaError_t e = cudaSuccess;
    if (blocks) SPEC_TRY(launch_attend_window(kv, a, st));
    else e = launch_k(m->pdl, f, grid, dim3(kRowThreads), smem, st, a);
    SPEC_TRY(check_cuda(e, "attention rows launch"));
    ++m->launches;
    if (a.direct) {
        prof_stop(m, slot, st, PROF_ATTN, 0.0);
        return SPEC_OK;
    }
    JoinArgs j{};
    j.part_o = a.part_o;
    j.part_ml = a.part_ml;
    j.own_range0 = a.own_range0;
    j.own_ranges = a.own_splits;
    j.pre_ranges = a.pre_splits;
    j.tile_ctas = a.tile_ctas;
    if (pre) j.pre_len = pre->len + kv->prefix_seq;
    if (pre) j.pre_cap = pre->max_ctx;
    j.TH = TH;
    j.H = H;
    j.G = G;
    j.Hkv = Hkv;
    j.out = out.p;
    j.stride = out.stride;
    j.lo = out.lo;
    void (*jf)(JoinArgs) = ranges > 12 ? (hd == 128 ? attend_join_kernel<128, 4> : attend_join_kernel<64, 4>)
                                       : (hd == 128 ? attend_join_kernel<128, 1> : attend_join_kernel<64, 1>);
    e = launch_k(m->pdl, jf, dim3(ranges > 12 ? TH : (TH + 3) / 4), dim3(128), 0, st, j);
    ++m->launches;
    prof_stop(m, slot, st, PROF_ATTN, 0.0);
    return check_cuda(e, "attention join launch");
}

}  // namespace spec

using namespace spec;

extern "C" int spec_kv_set_prefix(spec_kv* kv, spec_kv* prefix, int32_t seq) {
    if (!kv) return set_error(SPEC_ERR_ARG, "spec_kv_set_prefix: null cache");
    if (prefix) {
        if (prefix == kv) return set_error(SPEC_ERR_ARG, "spec_kv_set_prefix: a cache cannot be its own prefix");
        if (prefix->m != kv->m) return set_error(SPEC_ERR_ARG, "spec_kv_set_prefix: cache of another model");
        if (seq < 0 || seq >= prefix->batch) return set_error(SPEC_ERR_ARG, "spec_kv_set_prefix: seq out of range");
        if (prefix->prefix || prefix->prefix_lost)
            return set_error(SPEC_ERR_UNSUPPORTED, "spec_kv_set_prefix: the prefix has a prefix of its own");
        if (!kv->users.empty()) return set_error(SPEC_ERR_UNSUPPORTED, "spec_kv_set_prefix: the cache is a prefix itself");
        if (!kv->m->bf16) return set_error(SPEC_ERR_UNSUPPORTED, "spec_kv_set_prefix: bf16 models only");
    }
    kv_detach_prefix(kv);
    if (prefix) {
        try {
            prefix->users.push_back(kv);
        } catch (...) {
            return set_error(SPEC_ERR_CAPACITY, "spec_kv_set_prefix: out of host memory");
        }
        kv->prefix = prefix;
        kv->prefix_seq = seq;
    }
    return SPEC_OK;
}

extern "C" int spec_kv_set_window(spec_kv* kv, int32_t layer0, int32_t n_layers, int32_t window, int32_t sinks) {
    if (!kv) return set_error(SPEC_ERR_ARG, "spec_kv_set_window: null cache");
    const int N = kv->m->cfg.n_layers;
    if (layer0 < 0 || n_layers < 1 || layer0 >= N || n_layers > N - layer0)
        return set_error(SPEC_ERR_ARG, "spec_kv_set_window: layers out of range");
    if (window < 0 || sinks < 0) return set_error(SPEC_ERR_ARG, "spec_kv_set_window: window and sinks must not be negative");
    if (!kv->m->bf16) return set_error(SPEC_ERR_UNSUPPORTED, "spec_kv_set_window: bf16 models only");
    if (kv->window.empty()) {
        if (window == 0) return SPEC_OK;
        try {
            std::vector<int> w(N, 0), s(N, 0);
            kv->window.swap(w);
            kv->sinks.swap(s);
        } catch (...) {
            return set_error(SPEC_ERR_CAPACITY, "spec_kv_set_window: out of host memory");
        }
    }
    for (int l = layer0; l < layer0 + n_layers; ++l) {
        kv->window[l] = window;
        kv->sinks[l] = window ? sinks : 0;
    }
    if (*std::max_element(kv->window.begin(), kv->window.end()) == 0) {
        kv->window.clear();
        kv->sinks.clear();
    }
    return SPEC_OK;
}

extern "C" int spec_attend(spec_kv* kv, int32_t layer, int32_t batch, const int32_t* n_rows, const void* q,
                           int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                           const int32_t* tree_parent, void* out, int64_t out_stride, void* stream) {
    if (!kv || !n_rows) return set_error(SPEC_ERR_ARG, "spec_attend: null pointer");
    if ((k == nullptr) != (v == nullptr)) return set_error(SPEC_ERR_ARG, "spec_attend: k and v go together");
    spec_model* m = kv->m;
    const spec_model_config& c = m->cfg;
    if (!m->bf16) return set_error(SPEC_ERR_UNSUPPORTED, "spec_attend: bf16 models only");
    int dev = -1;
    SPEC_TRY(check_cuda(cudaGetDevice(&dev), "spec_attend: cudaGetDevice"));
    if (dev != m->device) return set_error(SPEC_ERR_ARG, "spec_attend: the model is on another device than the current one");
    SPEC_TRY(kv_check_prefix(kv, "spec_attend"));
    if (layer < 0 || layer >= c.n_layers) return set_error(SPEC_ERR_ARG, "spec_attend: layer out of range");
    if (batch < 1 || batch > kv->batch) return set_error(SPEC_ERR_ARG, "spec_attend: bad batch");
    int T = 0, n_max = 0;
    for (int b = 0; b < batch; ++b) {
        if (n_rows[b] < 0 || n_rows[b] > kMaxSeqRows) return set_error(SPEC_ERR_ARG, "spec_attend: n_rows[b] must be in [0, 64]");
        T += n_rows[b];
        n_max = std::max(n_max, (int)n_rows[b]);
    }
    if (T > c.max_rows) return set_error(SPEC_ERR_CAPACITY, "spec_attend: sum of n_rows > max_rows");
    const int64_t qd = (int64_t)c.n_heads * c.head_dim, kd = (int64_t)c.n_kv_heads * c.head_dim;
    if (q_stride < qd || out_stride < qd || (k && (k_stride < kd || v_stride < kd)))
        return set_error(SPEC_ERR_ARG, "spec_attend: a row stride is shorter than its row");
    if (tree_parent) {
        if (n_max > 0 && tree_parent[0] != -1) return set_error(SPEC_ERR_ARG, "tree_parent[0] must be -1");
        for (int i = 1; i < n_max; ++i)
            if (tree_parent[i] < 0 || tree_parent[i] >= i) return set_error(SPEC_ERR_ARG, "tree_parent[i] must be in [0, i)");
        for (int b = 0; b < batch; ++b)
            if (n_rows[b] != n_max) return set_error(SPEC_ERR_ARG, "tree mode: every sequence has the tree's node count");
    }
    if (T == 0) return SPEC_OK;
    if (!q || !out) return set_error(SPEC_ERR_ARG, "spec_attend: null pointer");
    cudaStream_t st = (cudaStream_t)stream;
    AttendSpan span{};
    SPEC_TRY(make_span(&span, batch, n_rows, 0, tree_parent, nullptr));
    if (k) {
        SPEC_TRY(kv_ensure_pages(kv, batch, n_rows, true, st));
        SPEC_TRY(launch_append(kv, layer, span, k, k_stride, v, v_stride, st));
    }
    const AttendOut o{(__nv_bfloat16*)out, out_stride, 0};
    return launch_attend(kv, layer, span, q, 0, q_stride, 1.0f / sqrtf((float)c.head_dim), o, st);
}
