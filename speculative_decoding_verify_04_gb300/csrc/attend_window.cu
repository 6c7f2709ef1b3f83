// Attention over a window for many query vectors: trees of drafted tokens, chains of
// many heads a KV head.
//
// A CTA takes the query vectors of one sequence and KV head in a block of 32 or 64 and a
// run of the keys that its first row's window and the sinks hold, in tiles of 64: the
// softmax's running maximum and sum in registers, S = Q K^T and O += P V by mma.sync
// m16n8k16, four warps that share every tile.  Each warp holds 16 query vectors; in a
// block of 32 two warps share them and take half of a tile's keys each, and join at the
// end.  A fifth warp copies the tiles ahead by tensor boxes (128-byte swizzle, a tile of K
// and one of V a stage).  The window's bounds cost masks only in the tiles where not every
// row sees every key; there a value that is not finite is taken out of the product (zero
// times it is not zero) and reaches the rows that see it as NaN.
//
// mma.sync and not tcgen05: a block of the latter has 128 rows, and a list of 32 query
// vectors is bound by reading its keys once (32 flops a byte) long before that.
// 32 sequences of 8 rows over windows of 8192 keys, 8 KV heads of 128 (32 vectors a block) take
// 153 us a call, 5.9 TB/s, 87 % of a copy's rate: 256 CTAs on 304 places, each with a whole window,
// so that nothing is joined (cut into ranges 172).  16 trees of 29 nodes over 2048 keys, 4 KV heads of
// 64 (116 vectors, two blocks of 64 that read the keys twice): 34 us with their append.
//
// bf16 caches only: 8-bit tiles turned into bf16 ones in shared memory made a call slower than
// the row kernel's products in f16 (32 sequences, 2048 keys, 8 KV heads of 128: 24 vectors 95 us
// against 76, 32 97 / 78, 64 122 / 118, 116 223 / 229).  In bf16 the row kernel is the faster one up to
// 16 vectors (16: 55 against 61 us; 24: 85 / 63; 32: 88 / 65; 64: 137 / 91; 116: 253 / 160).
#include <algorithm>
#include <atomic>
#include <climits>

#include "attend.cuh"

namespace spec {

constexpr int kWinKeys = 64;                           // keys of a tile
constexpr int kWinWarps = 4;
constexpr int kWinThreads = 32 * (kWinWarps + 1);

struct WinBars {
    uint64_t full[4], empty[4];
    uint16_t flags[2][kWinWarps];                      // by warp: keys of its 16 whose values are not finite
    int abort;
};

template <int HD, bool QF32, int RB>
struct WinShape {
    static constexpr int QR = 16 * RB;
    static constexpr int kTile = kWinKeys * HD * 2;    // a K or V tile in bf16
    static constexpr int kStage = 2 * kTile;
    static constexpr int kQ = RB * 16 * HD * 2;        // the block's query vectors
    static constexpr int kQBytes = (QF32 ? 2 : 1) * kQ;
    static constexpr int kStages = HD == 64 ? (kQBytes > 8192 ? 3 : 4) : (kQBytes > 16384 ? 2 : 3);
    static constexpr int kRing = kStages * kStage;
    static constexpr int kJoin = RB == 2 ? 32 * (HD + 2) * 4 : 0;
    static_assert(kRing >= kJoin, "the second half's states");
    static constexpr int kSmem = kRing + kQBytes + QR * 12 + (int)sizeof(WinBars);
    static constexpr int kCtas = HD == 64 ? 3 : 2;     // an SM
    static_assert(kSmem <= 233472 / kCtas - 1024, "CTAs an SM");
};

// row r, 16-byte piece c of a tile of [64 dims][rows] halves with 128-byte rows
SPEC_DEV uint32_t swz(int half_bytes, int r, int c) { return (c >> 3) * half_bytes + r * 128 + (((c & 7) ^ (r & 7)) << 4); }

template <int HD, bool QF32, int RB>
__global__ void __launch_bounds__(kWinThreads, WinShape<HD, QF32, RB>::kCtas)
attend_window_kernel(const __grid_constant__ AttendArgs a, const __grid_constant__ CUtensorMap own_k,
                     const __grid_constant__ CUtensorMap own_v, const __grid_constant__ CUtensorMap pre_k,
                     const __grid_constant__ CUtensorMap pre_v) {
    pdl_wait();
    pdl_trigger();
    using S = WinShape<HD, QF32, RB>;
    constexpr int KG = kWinWarps / RB, KW = kWinKeys / KG;     // key groups, keys a warp takes of a tile
    constexpr int QR = RB * 16, NT = KW / 8, KS = HD / 16, CH = HD / 8;
    constexpr int kKHalf = kWinKeys * 128, kQHalf = QR * 128;
    extern __shared__ __align__(1024) char ring[];     // the tiles' swizzle counts on 1024 bytes
    char* sQ = ring + S::kRing;
    WinBars& B = *reinterpret_cast<WinBars*>(sQ + S::kQBytes);
    unsigned long long* sMask = reinterpret_cast<unsigned long long*>(&B + 1);   // [QR] the rows' sight
    int* sLow = reinterpret_cast<int*>(sMask + QR);
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int G = a.H / a.Hkv;
    // the prompt's blocks first, then the sequences' own
    int id = blockIdx.x;
    const int n_pre = a.pre_splits * a.pre_qb * a.Hkv * a.span.batch;
    const bool is_pre = id < n_pre;
    if (!is_pre) id -= n_pre;
    const int g = id % a.Hkv;
    id /= a.Hkv;
    const int qb = id % a.own_qb;
    id /= a.own_qb;
    const int n_splits = is_pre ? a.pre_splits : a.own_splits, split = id % n_splits, b = id / n_splits;
    const int row0 = a.span.row0[b], rows = a.span.row0[b + 1] - row0;
    const int q0 = qb * QR, nq = min(QR, rows * G - q0);
    if (nq <= 0) return;
    const CacheView& cv = is_pre ? a.pre : a.own;
    const int seq = is_pre ? a.pre_seq : b;
    const int prompt_len = a.pre.len ? min(a.pre.len[a.pre_seq], a.pre.cap) : 0;
    const int ctx = a.own.len[b] + a.span.extra;
    const int base = prompt_len + ctx;                 // index of the first row
    const int shift = is_pre ? 0 : prompt_len;         // index of the part's slot 0
    const int n_ctx = is_pre ? prompt_len : ctx;
    int n_keys = is_pre ? prompt_len : min(ctx + rows, a.own.cap);
    if (!is_pre && ctx + rows > a.own.cap && t == 0) dev_error(a.err, SPEC_DEVERR_CAPACITY);
    KeyMap km{0, 0, 0, 0};
    {
        const int lo = max(0, base - shift - a.window + 1) & ~(kWinKeys - 1);
        km.sinks = min(max(a.sinks - shift, 0), n_ctx);
        km.sink_keys = (km.sinks + kWinKeys - 1) & ~(kWinKeys - 1);
        km.lo = lo;
        if (km.sink_keys >= lo) km.sink_keys = km.lo = 0;
        n_keys = km.lo < n_keys ? km.sink_keys + n_keys - km.lo : min(km.sink_keys, n_keys);
        km.low_max = base - shift + (q0 + nq - 1) / G - a.window + 1;
    }
    const int tiles = (n_keys + kWinKeys - 1) / kWinKeys, per = (tiles + n_splits - 1) / n_splits;
    const int t0 = min(tiles, split * per), t1 = min(tiles, t0 + per), n_tiles = t1 - t0;
    const size_t TH = (size_t)a.span.T * a.H;
    const int range = (is_pre ? 0 : a.own_range0) + split;
    auto row_of = [&](int r) { return row0 + (q0 + r) / G; };
    auto head_of = [&](int r) { return g * G + (q0 + r) % G; };
    if (n_tiles <= 0) {                                // nothing in this range
        for (int r = t; r < nq; r += kWinThreads) {
            if (a.direct) {
                for (int d = 0; d < HD; ++d) put_out(a.out, row_of(r) * a.out.stride + head_of(r) * HD + d, __int_as_float(0x7fc00000));
            } else {
                *reinterpret_cast<float2*>(a.part_ml + 2 * (range * TH + (size_t)row_of(r) * a.H + head_of(r))) = make_float2(-INFINITY, 0.f);
            }
        }
        return;
    }
    if (t == 0) {
        for (int i = 0; i < 4; ++i) { mbar_init(&B.full[i], 1); mbar_init(&B.empty[i], kWinWarps); }
        B.abort = 0;
        fence_mbar_init();
    }
    // the rows' sight, and the query vectors in bf16 (f32: and what is left of them)
    if (t < QR) {
        RowSight rs{0ull, INT_MAX};
        if (t < nq) {
            const unsigned long long mk = row_mask(a.span, b, (q0 + t) / G);
            const int d = __popcll(mk) - 1;
            rs.low = base - shift + d - a.window + 1;
            rs.mask = is_pre ? 0ull : window_mask(a.span, b, mk, d, a.window, a.sinks - base);
        }
        sMask[t] = rs.mask;
        sLow[t] = rs.low;
    }
    for (int i = t; i < QR * CH; i += kWinThreads) {
        const int r = i / CH, c = i % CH;
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 0.f;
        if (r < nq) {
            const long long off = row_of(r) * a.q_stride + head_of(r) * HD + c * 8;
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
        char* dst = sQ + swz(kQHalf, r, c);
        *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
        if (QF32)
            *reinterpret_cast<uint4*>(dst + S::kQ) = make_uint4(pack_bf16_lo(x[0], x[1]), pack_bf16_lo(x[2], x[3]),
                                                                pack_bf16_lo(x[4], x[5]), pack_bf16_lo(x[6], x[7]));
    }
    __syncthreads();
    volatile int* ab = &B.abort;
    constexpr int n_stages = S::kStages;

    if (warp == kWinWarps) {
        // -------- copies
        if (lane == 0) {
            const uint64_t keep = l2_policy_evict_first();
            const CUtensorMap* mk = is_pre ? &pre_k : &own_k;
            const CUtensorMap* mv = is_pre ? &pre_v : &own_v;
            int issued = 0;
            for (int i = 0; i < n_tiles; ++i) {
                const int s = i % n_stages, use = i / n_stages;
                if (use > 0 && !mbar_wait(&B.empty[s], (use - 1) & 1, ab, a.err)) break;
                // 64 slots from a multiple of 64 on: no page is crossed
                long long row = kv_row_in_layer(cv.pages, a.Hkv, seq, g, key_slot<true>(km, (t0 + i) * kWinKeys));
                if (row < 0) { dev_error(a.err, SPEC_DEVERR_CAPACITY); row = 0; }
                mbar_arrive_expect_tx(&B.full[s], S::kStage);
                char* dst = ring + s * S::kStage;
#pragma unroll
                for (int h = 0; h < HD / 64; ++h) {
                    tma_load_3d(dst + h * kKHalf, mk, 64 * h, (int)row, a.layer, &B.full[s], keep);
                    tma_load_3d(dst + S::kTile + h * kKHalf, mv, 64 * h, (int)row, a.layer, &B.full[s], keep);
                }
                ++issued;
            }
            // no copy may be in flight when the CTA ends: after an abort, the last use of each slot lands first
            if (*ab)
                for (int i = max(0, issued - n_stages); i < issued; ++i) mbar_wait(&B.full[i % n_stages], (i / n_stages) & 1, nullptr, a.err);
        }
        return;
    }

    const int rb = warp % RB, kg = warp / RB, gq = lane >> 2, cq = lane & 3;
    const uint32_t q_base = smem_u32(sQ);
    // the A operand of k-step ks: rows 16 rb .., dims 16 ks ..
    auto q_frag = [&](uint32_t at, int ks, uint32_t (&f)[4]) {
        const int r = 16 * rb + (lane & 15), c = 2 * ks + (lane >> 4);
        ldmatrix_x4(at + swz(kQHalf, r, c), f[0], f[1], f[2], f[3]);
    };
    uint32_t qf[KS][4];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) q_frag(q_base, ks, qf[ks]);
    const RowSight see[2] = {{sMask[16 * rb + gq], sLow[16 * rb + gq]}, {sMask[16 * rb + gq + 8], sLow[16 * rb + gq + 8]}};
    float o[HD / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int n = 0; n < HD / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    bool ok = true;
    for (int i = 0; i < n_tiles && ok; ++i) {
        const int s = i % n_stages;
        ok = __all_sync(0xffffffffu, mbar_wait(&B.full[s], (i / n_stages) & 1, ab, a.err));
        char* tile = ring + s * S::kStage;
        const int kt = (t0 + i) * kWinKeys, slot = key_slot<true>(km, kt), valid = n_keys - kt;
        const bool edge = slot + kWinKeys > n_ctx || slot < km.low_max || valid < kWinKeys;
        unsigned long long bad = 0ull;                 // bit k: key k's values are not finite
        if (edge) {
            // a warp looks at 16 rows of V, two lanes a row
            if (ok) {
                const int key = 16 * warp + (lane >> 1);
                char* v = tile + S::kTile;
                bool inf = key >= valid;
                for (int c = lane & 1; c < CH && !inf; c += 2) {
                    const uint4 w = *reinterpret_cast<const uint4*>(v + swz(kKHalf, key, c));
                    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) inf |= (u[e] & 0x7F80u) == 0x7F80u || (u[e] & 0x7F800000u) == 0x7F800000u;
                }
                const uint32_t any = __ballot_sync(0xffffffffu, inf), two = (any | any >> 1) & 0x55555555u;
                if ((two >> (lane & ~1)) & 1u)
                    for (int c = lane & 1; c < CH; c += 2) *reinterpret_cast<uint4*>(v + swz(kKHalf, key, c)) = make_uint4(0, 0, 0, 0);
                fence_async_smem();                    // the next copy comes over what was written here
                if (lane == 0) {
                    uint32_t f = 0;
#pragma unroll
                    for (int k = 0; k < 16; ++k) f |= ((two >> (2 * k)) & 1u) << k;
                    B.flags[i & 1][warp] = (uint16_t)f;
                }
            }
            named_bar(1, 32 * kWinWarps);
#pragma unroll
            for (int w = 0; w < kWinWarps; ++w) bad |= (unsigned long long)B.flags[i & 1][w] << (16 * w);
        }
        if (!ok) break;
        // S = Q K^T for this warp's keys
        const uint32_t kb = smem_u32(tile), vb = kb + S::kTile;
        float x[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) x[n][0] = x[n][1] = x[n][2] = x[n][3] = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            uint32_t ql[4];
            if (QF32) q_frag(q_base + S::kQ, ks, ql);
#pragma unroll
            for (int n = 0; n < NT; n += 2) {
                uint32_t f[4];
                const int key = kg * KW + 8 * n + (lane & 7) + ((lane >> 4) << 3), c = 2 * ks + ((lane >> 3) & 1);
                ldmatrix_x4(kb + swz(kKHalf, key, c), f[0], f[1], f[2], f[3]);
                mma16816(x[n], qf[ks][0], qf[ks][1], qf[ks][2], qf[ks][3], f[0], f[1]);
                mma16816(x[n + 1], qf[ks][0], qf[ks][1], qf[ks][2], qf[ks][3], f[2], f[3]);
                if (QF32) {
                    mma16816(x[n], ql[0], ql[1], ql[2], ql[3], f[0], f[1]);
                    mma16816(x[n + 1], ql[0], ql[1], ql[2], ql[3], f[2], f[3]);
                }
            }
        }
        if (edge) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int k = kg * KW + 8 * n + 2 * cq + (e & 1);
                    if (k >= valid || !row_sees<true>(km, see[e >> 1], slot + k, n_ctx)) x[n][e] = -INFINITY;
                    else if ((bad >> k) & 1ull) x[n][e] = __int_as_float(0x7fc00000);
                }
        }
        float f[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float mt = fmaxf(x[0][2 * h], x[0][2 * h + 1]);
#pragma unroll
            for (int n = 1; n < NT; ++n) mt = fmaxf(mt, fmaxf(x[n][2 * h], x[n][2 * h + 1]));
            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 1));
            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 2));
            const float mn = fmaxf(m[h], mt * a.c), mu = mn == -INFINITY ? 0.f : mn;
            f[h] = m[h] == mn ? 1.f : ex2(m[h] - mu);
            m[h] = mn;
            float sum = 0.f;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                x[n][2 * h] = ex2(fmaf(x[n][2 * h], a.c, -mu));
                x[n][2 * h + 1] = ex2(fmaf(x[n][2 * h + 1], a.c, -mu));
                sum += x[n][2 * h] + x[n][2 * h + 1];
            }
            l[h] = l[h] * f[h] + sum;
        }
        if (!__all_sync(0xffffffffu, f[0] == 1.f && f[1] == 1.f)) {
#pragma unroll
            for (int n = 0; n < HD / 8; ++n) {
                o[n][0] *= f[0];
                o[n][1] *= f[0];
                o[n][2] *= f[1];
                o[n][3] *= f[1];
            }
        }
        // O += P V, P rounded to bf16 (f32 queries: and what is left of it)
#pragma unroll
        for (int k = 0; k < KW / 16; ++k) {
            const float (&p0)[4] = x[2 * k];
            const float (&p1)[4] = x[2 * k + 1];
            const uint32_t pa[4] = {pack_bf16(p0[0], p0[1]), pack_bf16(p0[2], p0[3]), pack_bf16(p1[0], p1[1]), pack_bf16(p1[2], p1[3])};
            uint32_t pl[4];
            if (QF32) {
                pl[0] = pack_bf16_lo(p0[0], p0[1]); pl[1] = pack_bf16_lo(p0[2], p0[3]);
                pl[2] = pack_bf16_lo(p1[0], p1[1]); pl[3] = pack_bf16_lo(p1[2], p1[3]);
            }
#pragma unroll
            for (int n = 0; n < HD / 8; n += 2) {
                uint32_t v[4];
                const int key = kg * KW + 16 * k + (lane & 15), c = n + (lane >> 4);
                ldmatrix_x4_trans(vb + swz(kKHalf, key, c), v[0], v[1], v[2], v[3]);
                mma16816(o[n], pa[0], pa[1], pa[2], pa[3], v[0], v[1]);
                mma16816(o[n + 1], pa[0], pa[1], pa[2], pa[3], v[2], v[3]);
                if (QF32) {
                    mma16816(o[n], pl[0], pl[1], pl[2], pl[3], v[0], v[1]);
                    mma16816(o[n + 1], pl[0], pl[1], pl[2], pl[3], v[2], v[3]);
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.empty[s]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }
    if (KG == 2) {
        // the second half's states through shared memory (every tile has been read)
        float* st = reinterpret_cast<float*>(ring);    // [2 x 16 rows][HD + 2]
        named_bar(1, 32 * kWinWarps);
        if (kg == 1) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float* r = st + (16 * rb + gq + 8 * h) * (HD + 2);
#pragma unroll
                for (int n = 0; n < HD / 8; ++n) *reinterpret_cast<float2*>(r + 8 * n + 2 * cq) = make_float2(o[n][2 * h], o[n][2 * h + 1]);
                if (cq == 0) *reinterpret_cast<float2*>(r + HD) = make_float2(m[h], l[h]);
            }
        }
        named_bar(1, 32 * kWinWarps);
        if (kg == 1) return;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float* r = st + (16 * rb + gq + 8 * h) * (HD + 2);
            const float2 ml = *reinterpret_cast<const float2*>(r + HD);
            const float M = fmaxf(m[h], ml.x), mu = M == -INFINITY ? 0.f : M, w0 = ex2(m[h] - mu), w1 = ex2(ml.x - mu);
            l[h] = l[h] * w0 + ml.y * w1;
            m[h] = M;
#pragma unroll
            for (int n = 0; n < HD / 8; ++n) {
                const float2 x = *reinterpret_cast<const float2*>(r + 8 * n + 2 * cq);
                o[n][2 * h] = o[n][2 * h] * w0 + x.x * w1;
                o[n][2 * h + 1] = o[n][2 * h + 1] * w0 + x.y * w1;
            }
        }
    }
    if (!ok) return;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = 16 * rb + gq + 8 * h;
        if (r >= nq) continue;
        if (a.direct) {
            const float inv = 1.0f / l[h];
            const long long at = row_of(r) * a.out.stride + head_of(r) * HD + 2 * cq;
#pragma unroll
            for (int n = 0; n < HD / 8; ++n) {
                put_out(a.out, at + 8 * n, o[n][2 * h] * inv);
                put_out(a.out, at + 8 * n + 1, o[n][2 * h + 1] * inv);
            }
        } else {
            const size_t vec = range * TH + (size_t)row_of(r) * a.H + head_of(r);
#pragma unroll
            for (int n = 0; n < HD / 8; ++n)
                *reinterpret_cast<float2*>(a.part_o + vec * HD + 8 * n + 2 * cq) = make_float2(o[n][2 * h], o[n][2 * h + 1]);
            if (cq == 0) *reinterpret_cast<float2*>(a.part_ml + 2 * vec) = make_float2(m[h], l[h]);
        }
    }
}

// ---------------------------------------------------------------------------
bool attend_window_ok(const spec_kv* kv) { return !kv->q8 && kv->tmaps && (!kv->prefix || (!kv->prefix->q8 && kv->prefix->tmaps)); }
int attend_window_block(int vectors) { return vectors <= 32 ? 32 : 64; }
int attend_window_ctas(int hd) { return hd == 64 ? 3 : 2; }

template <int HD, bool QF32, int RB>
static int launch_window(const spec_kv* kv, const AttendArgs& a, cudaStream_t st) {
    using S = WinShape<HD, QF32, RB>;
    static std::atomic<unsigned long long> set{0};            // devices whose kernel has its shared memory
    const unsigned long long bit = 1ull << (kv->m->device & 63);
    cudaError_t e;
    if (!(set.load() & bit)) {
        e = cudaFuncSetAttribute(attend_window_kernel<HD, QF32, RB>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
        if (e != cudaSuccess) return check_cuda(e, "window attention kernel attribute");
        set.fetch_or(bit);
    }
    const spec_kv* pre = kv->prefix ? kv->prefix : kv;
    const long long blocks = (long long)a.span.batch * a.Hkv * a.own_qb;
    const dim3 grid((unsigned)(blocks * (a.own_splits + a.pre_splits)));
    e = launch_k(kv->m->pdl, attend_window_kernel<HD, QF32, RB>, grid, dim3(kWinThreads), S::kSmem, st, a, kv->tm_k64, kv->tm_v64,
                 pre->tm_k64, pre->tm_v64);
    return check_cuda(e, "window attention launch");
}

int launch_attend_window(const spec_kv* kv, const AttendArgs& a, cudaStream_t st) {
    int (*const launch[8])(const spec_kv*, const AttendArgs&, cudaStream_t) = {
        launch_window<64, false, 2>, launch_window<64, false, 4>, launch_window<64, true, 2>, launch_window<64, true, 4>,
        launch_window<128, false, 2>, launch_window<128, false, 4>, launch_window<128, true, 2>, launch_window<128, true, 4>};
    const int rb = attend_window_block(a.span.max_rows * (a.H / a.Hkv)) / 16;
    return launch[(kv->m->cfg.head_dim == 128 ? 4 : 0) + (a.q_f32 ? 2 : 0) + (rb == 4 ? 1 : 0)](kv, a, st);
}

}  // namespace spec
