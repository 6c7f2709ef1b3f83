// The shared prompt against many query vectors: tiles of 128 query vectors by
// 128 keys on the tensor cores (tcgen05), accumulators in tensor memory.
//
// The (KV head, key tile) list of a pair of query tiles is cut evenly over the
// pair's CTAs, so all end together whatever the sizes; a CTA takes its part head
// by head, with two streams.  With two tiles of query vectors the streams are the
// tiles, and every K and V tile serves both; with one tile the streams take the
// key tiles in turn and their states are joined at the end.  Per stream and key tile:
//     S = Q K^T          tcgen05.mma, both operands in shared memory, S in TMEM
//     P = 2^(c S - m)    one thread a query vector: S row from TMEM, running max
//                        and sum in registers, P as bf16 over S in TMEM
//     O += P V           tcgen05.mma with P as the TMEM operand; V as it lies in
//                        the cache ([key][dim]: the MN-major form)
// While one stream's threads do the softmax the tensor cores work for the other.
// The running maximum used in the exponent moves only when the true one has
// grown by more than 8 (a factor of 256: sums and O stay far inside f32), so O
// is rescaled rarely.  Partial states (m, sum p, sum p v) leave in 32 bits.
//
// Roles: warps 0-3 and 4-7 the streams' softmax, warp 8 the copies (TMA tensor
// boxes with the 128-byte swizzle), warp 9 the MMAs; 8-bit caches add four warps
// (12-15) that turn raw e4m3 tiles into swizzled f16 tiles, y 2^e, where every
// exponent of the turn's keys lies in [-15, 7] or its row is zeros (two instructions for two values), else
// into bf16 tiles (six); both are exact.  f16 queries are scaled by a power of two a row.
//
// P is rounded to the product's type, by 2^-8 of itself in bf16 and by 2^-11 in f16 (there,
// below 2^-21 of the row's largest, by 2^-32 of it); the sum of p takes p in 32 bits.  With bf16
// queries, whose results leave in bf16, that is all.  f32 queries (the forward calls, whose
// attention splits Q and P wherever it runs: P in one bf16 alone is past their bound in 32 layers)
// take two operands, hi + lo, each with products of its own: Q in either type, P in bf16, the lo
// part in the half of S's columns that P leaves; f16 keeps one P.  Q's lo part lies where the
// second tile of query vectors would, so a CTA has one tile and a K or V tile serves half as many:
// 64 x 8 rows of 32 heads over 8, 32768 tokens, take about 510 us instead of 182 (8 bits 606 instead of 280).
//
// 128 query vectors a stream is what one MMA takes and what one thread a vector serves;
// two streams are what the 512 columns of tensor memory hold (S and O of 128 each).  Keys
// come in tiles of 128: at 64 the hand-overs between MMAs and softmax would double.
// Bound by that hand-over: 64 x 8 rows of 32 heads over 8 KV heads, hd 128, 32768 tokens
// in bf16 take 182 us, 1.51 PFLOP/s (79 % of the measured peak, tensor pipe 67 %): 3060
// cycles a key tile against 2048 of products.  Short lists are bound by their starts:
// 6.7 key tiles a CTA (64 vectors x 4 heads, 16384 tokens in 8 bits) take 32 us.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "attend.cuh"

namespace spec {

constexpr int kBlkQ = 128;
constexpr int kBlkK = 128;
constexpr float kLazy = 8.0f;            // log2 of the growth of the maximum that is let pass
constexpr float kF16Log2 = 7.0f;         // P in f16 is 2^7 times what it is in bf16: 2^15 at most with kLazy

template <int HD, bool Q8>
struct TileShape {
    static constexpr int kTileBytes = kBlkK * HD * 2;          // one K or V tile in bf16
    static constexpr int kQBytes = kBlkQ * HD * 2;
    static constexpr int kRawBytes = kBlkK * HD;
    static constexpr int kStages = HD == 128 ? (Q8 ? 4 : 5) : 8;
    static constexpr int kRaw = Q8 ? (HD == 128 ? 2 : 4) : 0;
    static constexpr int kThreads = Q8 ? 512 : 384;
    static constexpr int kTiles = 2 * kQBytes + kStages * kTileBytes + kRaw * kRawBytes;
    static constexpr int kExpBytes = kRaw * kBlkK;
    // partial states leave through the ring (and the raw tiles behind it): 256 padded rows, or 128 behind the exchange
    static_assert(kStages * kTileBytes + kRaw * kRawBytes >= 256 * (HD * 4 + 16), "states");
    static constexpr int kSmem = kTiles + kExpBytes + 512 + (Q8 ? 1024 : 0) + 1024;   // barriers, row factors; the tiles start on 1024 bytes
};

struct TileBars {                        // (a form with fewer stages leaves the last of full .. raw_empty unused)
    uint64_t full[8], empty[8];          // K/V ring
    uint64_t raw_full[4], raw_empty[4];  // raw e4m3 ring
    uint64_t mode;                       // 8-bit caches: the operands' type is known
    uint64_t q_full, s_full[2], p_full[2], done;
    uint32_t tmem;
    int abort;
    int half;                            // 8-bit caches: 3 where this turn's products are in f16 (bit 0: no exponent
                                         // speaks against it, bit 1: not all rows are zeros)
};
static_assert(sizeof(TileBars) <= 512, "barriers");

// D[tmem] (+)= A[tmem] * B[smem]
SPEC_DEV void tc_mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                 :: "r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}
// a bounded wait of the whole warp
SPEC_DEV bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* ab, int* err) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, ab, err));
}
// [key][64 dims] tiles, 128-byte swizzle, read as the MN-major operand: 64-dim
// pieces lie `lead` bytes apart, groups of 8 keys 1024 bytes
SPEC_DEV uint64_t smem_desc_mn(uint32_t saddr, uint32_t lead) {
    uint64_t d = static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(lead >> 4) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}
SPEC_DEV void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                   "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                   "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(taddr));
}
SPEC_DEV void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
SPEC_DEV void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
SPEC_DEV void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
                 :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
                    "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}
SPEC_DEV void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
                 "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
                 "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
                 :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
                    "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
                    "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
                    "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
                 : "memory");
}
// the larger of three, the last two as bits
SPEC_DEV float max3(float x, uint32_t y, uint32_t z) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(__uint_as_float(y)), "f"(__uint_as_float(z)));
    return r;
}
SPEC_DEV void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// What a CTA does in one turn: a KV head, its query tiles and a run of its keys.
struct TileJob {
    int g, nq, q0;                       // vectors [q0, q0 + nq) of the head's list, nq <= 256
    int two;                             // two tiles of query vectors (else the streams share one)
    int k_begin, n_keys, n_kb;           // keys [k_begin, k_begin + n_keys) in n_kb tiles
    int n_jobs;                          // (stream, key tile) pairs: job n is stream n & 1
};
SPEC_DEV int job_kb(const TileJob& J, int n) { return J.two ? n >> 1 : n; }

// query vectors of a CTA
constexpr int tile_vectors(bool q_f32) { return q_f32 ? kBlkQ : 2 * kBlkQ; }

template <int HD, bool Q8, bool QF32>
__global__ void __launch_bounds__(TileShape<HD, Q8>::kThreads, 1)
attend_tile_kernel(const __grid_constant__ AttendArgs a, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v) {
    using S = TileShape<HD, Q8>;
    constexpr int NST = S::kStages, NRAW = S::kRaw > 0 ? S::kRaw : 1;
    constexpr uint32_t kHalf = kBlkK * 128;                  // bytes of 64 dims of a tile
    extern __shared__ char smraw[];
    char* tiles = smraw + ((1024u - (smem_u32(smraw) & 1023u)) & 1023u);
    char* sQ = tiles;
    char* ring = sQ + 2 * S::kQBytes;
    char* raw = ring + NST * S::kTileBytes;
    uint8_t* rexp = reinterpret_cast<uint8_t*>(raw + S::kRaw * S::kRawBytes);
    TileBars& B = *reinterpret_cast<TileBars*>(tiles + S::kTiles + S::kExpBytes);
    float* row_factor = reinterpret_cast<float*>(tiles + S::kTiles + S::kExpBytes + 512);   // [256], 8-bit caches
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;

    const int G = a.H / a.Hkv, NQ = a.span.T * G;
    const int q0 = (int)(blockIdx.x / a.tile_ctas) * tile_vectors(QF32);
    const bool two = !QF32 && NQ - q0 > kBlkQ;    // two tiles of query vectors: both streams free each K and V tile
    // every barrier of this kernel form, with its arrivals: what is taken down between turns is what was set up
    auto each_bar = [&](auto f) {
        for (int i = 0; i < NST; ++i) { f(&B.full[i], Q8 ? 4 : 1); f(&B.empty[i], two ? 2 : 1); }
        for (int i = 0; i < NRAW; ++i) { f(&B.raw_full[i], 1); f(&B.raw_empty[i], 4); }
        f(&B.mode, 4);
        f(&B.q_full, 8);
        for (int i = 0; i < 2; ++i) { f(&B.s_full[i], 1); f(&B.p_full[i], 5); }
        f(&B.done, 1);
    };
    auto init_bars = [&]() {
        each_bar([](uint64_t* b, int arrivals) { mbar_init(b, arrivals); });
        B.half = 1;
        fence_mbar_init();
    };
    if (warp == 9) tmem_alloc(&B.tmem, 512);
    if (t == 0) {
        init_bars();
        B.abort = 0;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = B.tmem;
    pdl_wait();
    pdl_trigger();

    // the pair's (KV head, key tile) list, cut evenly over its CTAs: this one's part, head by head
    const int P = min(a.pre.len[a.pre_seq], a.pre.cap), KB = (P + kBlkK - 1) / kBlkK;
    const long long W = (long long)a.Hkv * KB;
    const int cta = blockIdx.x % a.tile_ctas, ctas = tile_ctas_at_work(a.tile_ctas, W);
    long long at = cta < ctas ? cta * W / ctas : 0;
    const long long stop = cta < ctas ? (cta + 1) * W / ctas : 0;
    volatile int* ab = &B.abort;

    // a turn's job; between turns every warp meets twice and the barriers start afresh
    auto take = [&](TileJob& J) {
        J.g = (int)(at / KB);
        J.q0 = q0;
        J.nq = min(tile_vectors(QF32), NQ - q0);
        J.two = two;
        J.k_begin = (int)(at - (long long)J.g * KB) * kBlkK;
        J.n_kb = (int)min(stop - at, (long long)(J.g + 1) * KB - at);
        J.n_keys = min(P - J.k_begin, J.n_kb * kBlkK);
        J.n_jobs = J.two ? 2 * J.n_kb : J.n_kb;
        at += J.n_kb;
    };
    auto turn_over = [&]() {
        __syncthreads();
        if (*ab || at >= stop) return true;
        if (t == 0) {
            each_bar([](uint64_t* b, int) {
                asm volatile("mbarrier.inval.shared::cta.b64 [%0];" :: "r"(smem_u32(b)) : "memory");
            });
            init_bars();
        }
        __syncthreads();
        return false;
    };

    // the launch's registers, split by role: 512 x 128 = 256 x 200 + 128 x 48 + 128 x 64 and
    // 384 x 168 = 256 x 216 + 128 x 72
    if (warp < 8) {
        if (Q8) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        else asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        for (TileJob J; at < stop;) {
        take(J);
        const int range = cta - tile_first_cta(J.g, KB, W, ctas);
        // -------- queries into shared memory, then the softmax of stream `warp / 4`
        // a thread takes one 16-byte piece of every RPP-th row; eight loads go out before the first store
        constexpr int CPR = HD / 8, RPP = 256 / CPR, NB = HD == 128 && !QF32 ? 8 : 4;
        const int ch = t % CPR;
        bool ok = true, half = false;
        // f16: the row's largest magnitude to 2^13 .. 2^14 (CPR lanes hold a row); the power of two, its inverse kept
        auto half_factor = [&](const float (&x)[8], int r) {
            float m = finite_amax(x);
#pragma unroll
            for (int o = CPR / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const int e = min(127 + 13 - (int)(__float_as_uint(m) >> 23), 100);
            if (ch == 0) row_factor[r] = __uint_as_float((uint32_t)(127 - e) << 23);
            return __uint_as_float((uint32_t)(127 + e) << 23);
        };
        auto q_piece = [&](int r) {                           // where the thread's piece of row r goes
            const int rr = r & (kBlkQ - 1);
            return reinterpret_cast<uint4*>(sQ + (r / kBlkQ) * S::kQBytes + (ch >> 3) * kHalf + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4));
        };
        for (int r0 = t / CPR; r0 < (J.two ? 2 * kBlkQ : kBlkQ); r0 += NB * RPP) {
            if constexpr (QF32) {
                float x[NB][8];
#pragma unroll
                for (int k = 0; k < NB; ++k) {
                    const int r = r0 + k * RPP, qi = J.q0 + r;
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[k][e] = 0.f;
                    if (r >= J.nq) continue;
                    const float* p = static_cast<const float*>(a.q) + (qi / G) * a.q_stride + (J.g * G + qi % G) * HD + ch * 8;
                    const float4 u = __ldg(reinterpret_cast<const float4*>(p)), w = __ldg(reinterpret_cast<const float4*>(p + 4));
                    x[k][0] = u.x; x[k][1] = u.y; x[k][2] = u.z; x[k][3] = u.w;
                    x[k][4] = w.x; x[k][5] = w.y; x[k][6] = w.z; x[k][7] = w.w;
                }
                if (Q8 && r0 == t / CPR) {                    // (the first loads are on their way)
                    ok = warp_wait(&B.mode, 0, ab, a.err);
                    half = B.half == 3;
                }
#pragma unroll
                for (int k = 0; k < NB; ++k) {
                    const int r = r0 + k * RPP;
                    uint32_t hi[4], lo[4];
                    if (half) {
                        const float f = half_factor(x[k], r);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float y = x[k][2 * i] * f, z = x[k][2 * i + 1] * f;
                            hi[i] = pack_f16(y, z);
                            lo[i] = pack_f16(y - f16_round(y), z - f16_round(z));
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            hi[i] = pack_bf16(x[k][2 * i], x[k][2 * i + 1]);
                            lo[i] = pack_bf16_lo(x[k][2 * i], x[k][2 * i + 1]);
                        }
                    }
                    *q_piece(r) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *q_piece(r + kBlkQ) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            } else {
                uint4 w[NB];
#pragma unroll
                for (int k = 0; k < NB; ++k) {
                    const int r = r0 + k * RPP, qi = J.q0 + r;
                    w[k] = make_uint4(0, 0, 0, 0);
                    if (r >= J.nq) continue;
                    const long long off = (qi / G) * a.q_stride + (J.g * G + qi % G) * HD + ch * 8;
                    if (a.q_vec) {
                        w[k] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + off));
                    } else {
                        const unsigned short* p = static_cast<const unsigned short*>(a.q) + off;
                        w[k] = make_uint4(p[0] | (uint32_t)p[1] << 16, p[2] | (uint32_t)p[3] << 16,
                                          p[4] | (uint32_t)p[5] << 16, p[6] | (uint32_t)p[7] << 16);
                    }
                }
                if (Q8 && r0 == t / CPR) {                    // (the first loads are on their way)
                    ok = warp_wait(&B.mode, 0, ab, a.err);
                    half = B.half == 3;
                }
                if (half) {
#pragma unroll
                    for (int k = 0; k < NB; ++k) {
                        const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
                        float x[8];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            x[2 * i] = __uint_as_float(u[i] << 16);
                            x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
                        }
                        const float f = half_factor(x, r0 + k * RPP);
                        w[k] = make_uint4(pack_f16(x[0] * f, x[1] * f), pack_f16(x[2] * f, x[3] * f), pack_f16(x[4] * f, x[5] * f),
                                          pack_f16(x[6] * f, x[7] * f));
                    }
                }
#pragma unroll
                for (int k = 0; k < NB; ++k) *q_piece(r0 + k * RPP) = w[k];
            }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.q_full);

        const int st = warp >> 2, row = t & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;                   // TMEM lane 32 * (warp % 4)
        const uint32_t tS = tmem + st * 128 + lanes, tO = tmem + 256 + st * HD + lanes;
        float m = -INFINITY, l = 0.f;                                        // m: the maximum that the exponents use
        int q = 0;                                                           // job of this stream
        int kslot = J.two ? 0 : 2 * st, vslot = 0;                           // ring slots of its next K and last V tile
        while (kslot >= NST) kslot -= NST;
        float c = a.c;
        for (int n = st; n < J.n_jobs && ok; n += 2, ++q) {
            const int kb = job_kb(J, n), valid = min(kBlkK, J.n_keys - kb * kBlkK);
            ok = warp_wait(&B.s_full[st], q & 1, ab, a.err);
            if (!ok) break;
            tc_fence_after();
            if ((warp & 3) == 0 && lane == 0) {
                // S is there, and with it every product before it: this K tile is free, and the V
                // tile of the stream's product before
                mbar_arrive(&B.empty[kslot]);
                if (q > 0) mbar_arrive(&B.empty[vslot]);
            }
            vslot = kslot + 1 == NST ? 0 : kslot + 1;
            kslot += J.two ? 2 : 4;
            while (kslot >= NST) kslot -= NST;
            if (half && q == 0) c *= row_factor[(J.two ? st * kBlkQ : 0) + row];
            // the whole row at once: 128 scores in registers
            uint32_t r[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, r[c]);
            tmem_wait_ld();
            if (valid != kBlkK) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (32 * c + i >= valid) r[c][i] = 0xFF800000u;       // -inf
            }
            float mx4[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) mx4[c] = __uint_as_float(r[c][0]);
#pragma unroll
            for (int i = 1; i < 32; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) mx4[c] = fmaxf(mx4[c], __uint_as_float(r[c][i]));

            float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
            mx *= c;
            if (__any_sync(0xffffffffu, mx > m + kLazy || m == -INFINITY)) {
                const float mn = fmaxf(m, mx);
                const float f = ex2(m - (mn == -INFINITY ? 0.f : mn));
                l *= f;
                m = mn;
                if (q > 0) {
#pragma unroll
                    for (int c = 0; c < HD / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32(tO + 32 * c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                        tmem_st32(tO + 32 * c, o);
                    }
                }
            }
            const float mu = (m == -INFINITY ? 0.f : m) - (half ? kF16Log2 : 0.f);
            const float2 cc = make_float2(c, c), mm = make_float2(-mu, -mu);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            auto exponentials = [&](auto f16) {
                constexpr bool kSplit = QF32 && !decltype(f16)::value;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t p[16], pl[kSplit ? 16 : 1];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float2 x = fma2(make_float2(__uint_as_float(r[c][2 * i]), __uint_as_float(r[c][2 * i + 1])), cc, mm);
                        x.x = ex2(x.x);
                        x.y = ex2(x.y);
                        sum[i & 1] = add2(sum[i & 1], x);
                        p[i] = f16.value ? pack_f16(x.x, x.y) : bf16x2(x.x, x.y);
                        if constexpr (kSplit) pl[i] = bf16x2(x.x - __uint_as_float(p[i] << 16), x.y - __uint_as_float(p[i] & 0xFFFF0000u));
                    }
                    tmem_st16(tS + 16 * c, p);                // P's columns lie over S columns
                    if constexpr (kSplit) tmem_st16(tS + 64 + 16 * c, pl);
                }
            };
            if (half) exponentials(std::true_type{});
            else exponentials(std::false_type{});
            sum[0] = add2(sum[0], sum[1]);
            l += sum[0].x + sum[0].y;
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&B.p_full[st]);
        }
        // -------- the state: this stream's own rows, or (one tile) joined with the other stream's
        const int n1 = J.n_jobs / 2;                          // jobs of stream 1
        if (ok) ok = warp_wait(&B.done, 0, ab, a.err);
        tc_fence_after();
        if (half) m -= kF16Log2;                              // what the state's sums are relative to
        float* xo = reinterpret_cast<float*>(ring);           // every product has ended: the ring is free
        float* xml = reinterpret_cast<float*>(sQ + S::kQBytes);
        if (!J.two) {
            if (st == 1) {
                xml[row] = m;
                xml[kBlkQ + row] = l;
                if (ok && n1 > 0) {
#pragma unroll
                    for (int c = 0; c < HD / 32; ++c) {
                        uint32_t r[32];
                        tmem_ld32(tO + 32 * c, r);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) xo[(32 * c + i) * kBlkQ + row] = __uint_as_float(r[i]);
                    }
                }
            }
            named_bar(1, 256);
        }
        const int qi = st * kBlkQ + row;                     // two tiles: this stream's row; one: stream 0's
        if (ok && (J.two || st == 0)) {
            float w0 = 1.f, w1 = 0.f;
            if (!J.two) {
                const float m1 = xml[row], l1 = xml[kBlkQ + row], M = fmaxf(m, m1), Mu = M == -INFINITY ? 0.f : M;
                w0 = ex2(m - Mu);
                w1 = ex2(m1 - Mu);
                l = l * w0 + l1 * w1;
                m = M;
            }
            const bool out = qi < J.nq;
            const int v = J.q0 + qi;
            const size_t vec = (size_t)range * a.span.T * a.H + (size_t)(v / G) * a.H + J.g * G + v % G;
            if (out) *reinterpret_cast<float2*>(a.part_ml + 2 * vec) = make_float2(m, l);
            if (q > 0) {
                // the row goes out as one bulk copy from shared memory (rows 16 bytes apart in banks):
                // stored from registers, every instruction of a warp would meet 32 lines
                constexpr int kRow = HD * 4 + 16;
                char* so = ring + (J.two ? 0 : HD * kBlkQ * 4) + qi * kRow;
#pragma unroll
                for (int c = 0; c < HD / 32; ++c) {
                    uint32_t r[32];
                    tmem_ld32(tO + 32 * c, r);
                    tmem_wait_ld();
                    if (!J.two) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float x1 = n1 > 0 ? xo[(32 * c + i) * kBlkQ + row] * w1 : 0.f;
                            r[i] = __float_as_uint(fmaf(__uint_as_float(r[i]), w0, x1));
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<uint4*>(so + 128 * c + 16 * i) = make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
                }
                fence_async_smem();
                if (out) {
                    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;"
                                 :: "l"(reinterpret_cast<uint64_t>(a.part_o + vec * HD)), "r"(smem_u32(so)), "r"(HD * 4) : "memory");
                    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
                }
            }
        }
        fence_async_smem();                                   // the next copies come over what was written here
        tc_fence_before();
        if (turn_over()) break;
        }
    } else if (warp < 12) {
        if (Q8) asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        for (TileJob J; at < stop;) {
        take(J);
        if (warp == 8) {
        // -------- copies: entries K0, V0, K1, V1, ... of the ring
        constexpr int kBox = 64;                              // slots a tensor box (no page holds fewer)
        constexpr int kBoxes = kBlkK / kBox * (HD / 64);      // boxes of a tile, one a lane
        const uint64_t keep = l2_policy_evict_last();         // the prompt is read by every query tile
        int issued = 0;
        for (int e = 0; e < 2 * J.n_kb; ++e) {
            const int kt = J.k_begin + (e >> 1) * kBlkK;
            if (Q8) {
                const int s = e % NRAW, use = e / NRAW;
                if (use > 0 && !__all_sync(0xffffffffu, mbar_wait(&B.raw_empty[s], (use - 1) & 1, ab, a.err))) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&B.raw_full[s], S::kRawBytes + kBlkK);
                    const uint8_t* base = static_cast<const uint8_t*>(e & 1 ? a.pre.v : a.pre.k);
                    const uint8_t* ex = e & 1 ? a.pre.ve : a.pre.ke;
                    for (int p = 0; p < kBlkK / 64; ++p) {
                        // 64 slots never cross a page; slots past the keys are read from the first piece again
                        const int slot = kt + 64 * p < J.k_begin + J.n_keys ? kt + 64 * p : kt;
                        long long row = kv_row_in_layer(a.pre.pages, a.Hkv, a.pre_seq, J.g, slot);
                        if (row < 0) { dev_error(a.err, SPEC_DEVERR_CAPACITY); row = 0; }
                        bulk_load(raw + s * S::kRawBytes + p * 64 * HD, base + row * HD, 64 * HD, &B.raw_full[s], keep);
                        bulk_load(rexp + s * kBlkK + p * 64, ex + row, 64, &B.raw_full[s], keep);
                    }
                }
            } else {
                const int s = e % NST, use = e / NST;
                if (use > 0 && !__all_sync(0xffffffffu, mbar_wait(&B.empty[s], (use - 1) & 1, ab, a.err))) break;
                if (lane == 0) mbar_arrive_expect_tx(&B.full[s], S::kTileBytes);
                __syncwarp();
                if (lane < kBoxes) {
                    const int p = lane / (HD / 64), h = lane % (HD / 64);
                    const int slot = kt + kBox * p < J.k_begin + J.n_keys ? kt + kBox * p : kt;
                    long long row = kv_row_in_layer(a.pre.pages, a.Hkv, a.pre_seq, J.g, slot);
                    if (row < 0) { dev_error(a.err, SPEC_DEVERR_CAPACITY); row = 0; }
                    tma_load_3d(ring + s * S::kTileBytes + h * kHalf + p * kBox * 128, e & 1 ? &tm_v : &tm_k, 64 * h, (int)row,
                                a.layer, &B.full[s], keep);
                }
                __syncwarp();
            }
            ++issued;
        }
        // no copy may be in flight when the CTA ends: after an abort, the last use of each slot lands first
        if (*ab) {
            const int ns = Q8 ? NRAW : NST;
            for (int e = max(0, issued - ns); e < issued; ++e)
                mbar_wait(Q8 ? &B.raw_full[e % ns] : &B.full[e % ns], (e / ns) & 1, nullptr, a.err);
        }
        } else if (warp == 9) {
        // -------- MMAs, by one thread: the streams' jobs alternate, so that one stream's softmax runs
        // while the other's products do (two threads let both fall into step: 4190 cycles a pair of
        // jobs instead of 3300).  An MMA takes the tensor cores 64 cycles (hd 128) and hardly more
        // than one waits in the thread's queue, so every look at a barrier and every commit lets the
        // cores run dry (measured, 16 MMAs: 1024 cycles, with one commit and one, two or three waits
        // 1124, 1221 or 1303).  So a stream's P V and its next S go out together behind one wait: the
        // gate's arrival on p_full stands for the V tile and the next K tile.  And with one commit: it
        // covers every MMA before it, and the softmax threads that see S complete free the K tile
        // and the V tile before it.
        if (lane == 0) {
            const uint64_t qd = smem_desc_sw128(smem_u32(sQ)), kd = smem_desc_sw128(smem_u32(ring));
            const uint64_t vd = smem_desc_mn(smem_u32(ring), kHalf);
            bool ok = mbar_wait(&B.q_full, 0, ab, a.err);
            tc_fence_after();
            // A and B in bf16, or in f16 (both format fields zero)
            const uint32_t types = Q8 && B.half == 3 ? ~((1u << 7) | (1u << 10)) : ~0u;
            const bool split_p = QF32 && types == ~0u;
            const uint32_t kIdS = idesc_bf16_f32(kBlkQ, kBlkK) & types;
            const uint32_t kIdO = (idesc_bf16_f32(kBlkQ, HD) | (1u << 16)) & types;     // B is MN-major
            int ks_ = 0, vs_ = 1;                             // ring slots of the next K and V tiles
            auto scores = [&](int i) {
                const uint64_t q0 = qd + (J.two && i ? S::kQBytes >> 4 : 0), k0 = kd + ks_ * (S::kTileBytes >> 4);
#pragma unroll
                for (int ks = 0; ks < HD / 16; ++ks) {
                    const uint32_t o = ((ks >> 2) * kHalf + (ks & 3) * 32) >> 4;
                    tc_mma_f16(tmem + i * 128, q0 + o, k0 + o, kIdS, ks > 0);
                }
                if constexpr (QF32) {
                    const uint64_t ql = q0 + (S::kQBytes >> 4);
#pragma unroll
                    for (int ks = 0; ks < HD / 16; ++ks) {
                        const uint32_t o = ((ks >> 2) * kHalf + (ks & 3) * 32) >> 4;
                        tc_mma_f16(tmem + i * 128, ql + o, k0 + o, kIdS, 1);
                    }
                }
                tc_commit(&B.s_full[i]);
                if (!J.two || i == 1) ks_ = ks_ + 2 >= NST ? ks_ + 2 - NST : ks_ + 2;
            };
            for (int n = 0; n < 2 && n < J.n_jobs; ++n) {
                ok = ok && mbar_wait(&B.full[ks_], 0, ab, a.err);
                if (ok) scores(n);
            }
            for (int n = 0; n < J.n_jobs && ok; ++n) {
                const int i = n & 1;
                const uint64_t v0 = vd + vs_ * (S::kTileBytes >> 4);
                const uint32_t d = tmem + 256 + i * HD, p = tmem + i * 128;
                const int steps = min(kBlkK, J.n_keys - job_kb(J, n) * kBlkK + 15) / 16;
                ok = mbar_wait(&B.p_full[i], (n >> 1) & 1, ab, a.err);
                if (!ok) break;
                tc_fence_after();
                if (steps == kBlkK / 16) {
#pragma unroll
                    for (int ks = 0; ks < kBlkK / 16; ++ks)
                        tc_mma_f16_ts(d, p + 8 * ks, v0 + ks * (2048 >> 4), kIdO, n > 1 || ks > 0);
                } else {
                    for (int ks = 0; ks < steps; ++ks)
                        tc_mma_f16_ts(d, p + 8 * ks, v0 + ks * (2048 >> 4), kIdO, n > 1 || ks > 0);
                }
                if (split_p)
                    for (int ks = 0; ks < steps; ++ks) tc_mma_f16_ts(d, p + 64 + 8 * ks, v0 + ks * (2048 >> 4), kIdO, 1);
                if (!J.two || i == 1) vs_ = vs_ + 2 >= NST ? vs_ + 2 - NST : vs_ + 2;
                if (n + 2 < J.n_jobs) scores(i);
            }
            tc_commit(&B.done);                               // every MMA; after an abort too, before the memory goes
            if (!ok) mbar_wait(&B.done, 0, nullptr, a.err);
        }
        __syncwarp();
        } else if (warp == 10) {
        // -------- the gate: a job's V tile and the K tile of the stream's next job have come
        bool first = true;                                    // the first K tiles, so that every slot's phases are waited for in turn
        for (int n = 0; n < 2 && n < J.n_jobs && first; ++n) first = warp_wait(&B.full[2 * job_kb(J, n) % NST], 0, ab, a.err);
        for (int n = 0; n < J.n_jobs && first; ++n) {
            const int kb = job_kb(J, n), ev = 2 * kb + 1, ek = 2 * job_kb(J, n + 2), valid = J.n_keys - kb * kBlkK;
            // (two tiles: stream 1 finds what stream 0 waited for)
            bool ok = warp_wait(&B.full[ev % NST], (ev / NST) & 1, ab, a.err);
            if (ok && n + 2 < J.n_jobs) ok = warp_wait(&B.full[ek % NST], (ek / NST) & 1, ab, a.err);
            if (!ok) break;
            if (!Q8 && valid < kBlkK && (!J.two || !(n & 1))) {
                // the last 16 keys' slots past the range: P is zero there, and V must be finite
                char* vt = ring + (ev % NST) * S::kTileBytes;
                for (int h = 0; h < HD / 64; ++h)
                    for (int x = valid * 8 + lane; x < (valid + 15) / 16 * 128; x += 32)
                        *reinterpret_cast<uint4*>(vt + h * kHalf + x * 16) = make_uint4(0, 0, 0, 0);
                fence_async_smem();
                __syncwarp();
            }
            // p_full takes one gate arrival a phase: this job's S comes after the stream's last P V, so the
            // last phase is over (every phase of s_full is waited for in turn, the first ones too: a
            // parity alone does not tell a phase from the one before the last)
            if (!warp_wait(&B.s_full[n & 1], (n >> 1) & 1, ab, a.err)) break;
            if (lane == 0) mbar_arrive(&B.p_full[n & 1]);
            __syncwarp();
        }
        }
        if (turn_over()) break;
        }
    } else if (Q8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        for (TileJob J; at < stop;) {
        take(J);
        // -------- raw e4m3 tiles to swizzled bf16 tiles
        const int ct = t - 384;
        // f16 holds the turn's rows where every exponent lies in [-15, 7] (values 2^-24 .. 57344)
        {
            bool fits = true, seen = false;
            for (int i = ct; i < (J.n_keys + 15) / 16 * 2 && fits; i += 128) {
                const int slot = J.k_begin + i / 2 * 16;
                const long long row = kv_row_in_layer(a.pre.pages, a.Hkv, a.pre_seq, J.g, slot);
                if (row < 0) continue;                        // (the copies report it)
                const uint4 w = __ldg(reinterpret_cast<const uint4*>((i & 1 ? a.pre.ve : a.pre.ke) + row));
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
                uint32_t least = 0;                           // rows of the least exponent
#pragma unroll
                for (int b = 0; b < 16; ++b) {
                    const int e = (int)((u[b >> 2] >> (8 * (b & 3))) & 0xFF) - 127;
                    if (slot + b >= J.k_begin + J.n_keys) continue;
                    if (e == -124) least |= 1u << b;
                    else seen = true;
                    if (e != -124 && (e < -15 || e > 7)) fits = false;
                }
                // they fit where they are zeros; what they hold else lies below f16's range
                const uint4* y = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(i & 1 ? a.pre.v : a.pre.k) + row * HD);
#pragma unroll 1
                for (; least && fits; least &= least - 1) {
                    const uint4* at_b = y + (__ffs(least) - 1) * (HD / 16);
#pragma unroll 1
                    for (int p = 0; p < HD / 16; ++p) {
                        const uint4 x = __ldg(at_b + p);
                        if ((x.x | x.y | x.z | x.w) & 0x7F7F7F7Fu) fits = false;
                    }
                }
            }
            if (!fits) atomicAnd(&B.half, 2);
            if (seen) atomicOr(&B.half, 2);
            __syncwarp();
            if (lane == 0) mbar_arrive(&B.mode);
        }
        const bool mode_ok = warp_wait(&B.mode, 0, ab, a.err);
        const bool half = B.half == 3;
        for (int e = 0; e < 2 * J.n_kb; ++e) {
            const int rs = e % NRAW, s = e % NST, use = e / NST;
            bool ok = mode_ok && mbar_wait(&B.raw_full[rs], (e / NRAW) & 1, ab, a.err);
            if (ok && use > 0) ok = mbar_wait(&B.empty[s], (use - 1) & 1, ab, a.err);
            if (!__all_sync(0xffffffffu, ok)) break;
            const int valid = J.n_keys - (e >> 1) * kBlkK;
            const char* src = raw + rs * S::kRawBytes;
            char* dst = ring + s * S::kTileBytes;
            constexpr int CPK = HD / 16;                      // 16-byte pieces of a raw row
            auto convert = [&](auto f16) {
#pragma unroll
                for (int j0 = 0; j0 < CPK; j0 += 4) {
                    // four pieces' loads before the first conversion
                    uint4 w[4];
                    int eb[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int id = ct + 128 * (j0 + j);
                        w[j] = *reinterpret_cast<const uint4*>(src + id * 16);
                        eb[j] = rexp[rs * kBlkK + id / CPK];
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int id = ct + 128 * (j0 + j), key = id / CPK, ch = id % CPK;
                        const uint32_t ws[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
                        uint32_t o[8];
                        if (f16.value) {
                            // 2^e as f16 (2^-15 is a denormal; rows of the least exponent are zeros: 0)
                            const uint32_t h = eb[j] >= 127 - 14 ? (uint32_t)(eb[j] - 127 + 15) << 10 : (eb[j] == 127 - 15 ? 0x0200u : 0u);
                            const uint32_t hh = h | (h << 16);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                o[2 * i] = f16x2_mul(e4m3x2_f16(ws[i]), hh);
                                o[2 * i + 1] = f16x2_mul(e4m3x2_f16(ws[i] >> 16), hh);
                            }
                        } else {
                            const float sc = kv8_scale(eb[j]);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float2 x = e4m3x2_f32(ws[i]), y = e4m3x2_f32(ws[i] >> 16);
                                o[2 * i] = bf16x2(x.x * sc, x.y * sc);
                                o[2 * i + 1] = bf16x2(y.x * sc, y.y * sc);
                            }
                        }
                        if (key >= valid)
#pragma unroll
                            for (int i = 0; i < 8; ++i) o[i] = 0u;    // a NaN there stays out
                        char* d = dst + (ch >> 2) * kHalf + key * 128;
                        const int c0 = (2 * (ch & 3)) ^ (key & 7), c1 = (2 * (ch & 3) + 1) ^ (key & 7);
                        // the upper 64 dims' pieces in the other order: both halves' banks are then distinct
                        const bool flip = (ch >> 2) & 1;
                        const uint4 lo = make_uint4(o[0], o[1], o[2], o[3]), hi = make_uint4(o[4], o[5], o[6], o[7]);
                        *reinterpret_cast<uint4*>(d + ((flip ? c1 : c0) << 4)) = flip ? hi : lo;
                        *reinterpret_cast<uint4*>(d + ((flip ? c0 : c1) << 4)) = flip ? lo : hi;
                    }
                }
            };
            if (half) convert(std::true_type{});
            else convert(std::false_type{});
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&B.full[s]);
                mbar_arrive(&B.raw_empty[rs]);
            }
        }
        if (turn_over()) break;
        }
    }
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_relinquish();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------------------
bool attend_tile_ok(const spec_kv* pre) { return pre->q8 || pre->tmaps; }

// CTAs a pair of query tiles, one CTA an SM: the choice whose longest CTA ends
// soonest, counted in key tiles.  A turn costs about 12000 cycles beyond its keys
// (queries in, pipeline start, state out), a key tile 1500 a tile of query vectors (f32: 3000);
// cuts that fall on heads (a multiple of Hkv CTAs) need one turn, others two.
// (64 samples x 8 rows over 32768 tokens: 19 CTAs a pair 182 us, the next
// multiple, 16, 206; 8 chains over 4096 tokens with 32 heads: 152 CTAs 22 us, 128 15 us.)
int attend_tile_ctas(const spec_model* m, const AttendSpan& span, bool q_f32, int prompt_cap) {
    const spec_model_config& c = m->cfg;
    const int H = c.n_kv_heads, NQ = span.T * (c.n_heads / H), QV = tile_vectors(q_f32), pairs = (NQ + QV - 1) / QV;
    const long long W = (long long)H * std::max(1, (prompt_cap + kBlkK - 1) / kBlkK);
    const int turn = NQ > kBlkQ || q_f32 ? 4 : 8;
    int best = 1;
    long long least = -1;
    for (int n = 1; n <= m->num_sms && (n == 1 || 2 * n <= W); ++n) {
        const long long waves = ((long long)pairs * n + m->num_sms - 1) / m->num_sms;
        const int turns = n % H == 0 ? 1 : (H % n == 0 ? H / n : H / n + 2);
        const long long cost = waves * ((W + n - 1) / n + turn * turns);
        if (least < 0 || cost < least) { least = cost; best = n; }
    }
    return best;
}
int attend_tile_ranges(const spec_model* m, int ctas) { return ctas / m->cfg.n_kv_heads + 2; }

template <int HD, bool Q8, bool QF32>
static int launch_tile(const spec_kv* pre, const AttendArgs& a, cudaStream_t st) {
    using S = TileShape<HD, Q8>;
    static std::atomic<unsigned long long> set{0};            // devices whose kernel has its shared memory
    const unsigned long long bit = 1ull << (pre->m->device & 63);
    cudaError_t e;
    if (!(set.load() & bit)) {
        e = cudaFuncSetAttribute(attend_tile_kernel<HD, Q8, QF32>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
        if (e != cudaSuccess) return check_cuda(e, "attention tile kernel attribute");
        set.fetch_or(bit);
    }
    const int NQ = a.span.T * (a.H / a.Hkv), QV = tile_vectors(QF32);
    const dim3 grid((unsigned)((NQ + QV - 1) / QV * a.tile_ctas));
    e = launch_k(pre->m->pdl, attend_tile_kernel<HD, Q8, QF32>, grid, dim3(S::kThreads), S::kSmem, st, a, pre->tm_k64, pre->tm_v64);
    ++pre->m->launches;
    return check_cuda(e, "attention tile launch");
}

int launch_attend_tile(const spec_kv* pre, const AttendArgs& a, cudaStream_t st) {
    int (*const launch[8])(const spec_kv*, const AttendArgs&, cudaStream_t) = {
        launch_tile<64, false, false>, launch_tile<64, false, true>, launch_tile<64, true, false>, launch_tile<64, true, true>,
        launch_tile<128, false, false>, launch_tile<128, false, true>, launch_tile<128, true, false>, launch_tile<128, true, true>};
    return launch[(pre->m->cfg.head_dim == 128 ? 4 : 0) + (pre->q8 ? 2 : 0) + (a.q_f32 ? 1 : 0)](pre, a, st);
}

}  // namespace spec
