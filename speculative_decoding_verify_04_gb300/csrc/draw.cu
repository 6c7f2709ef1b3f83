// One token a row of logits from a given random number, after temperature, top-k,
// top-p and min-p.
//
// With m = max x and w_i = 2^(c (x_i - m)), c = log2 e / T, the kept tokens are
//     the k largest logits (ties to the lower id),
//     of those the shortest run, by decreasing logit, whose w reach p of theirs,
//     of those the w >= min_p,
// and the token is the first by id at which the sum of the kept w passes u times
// their sum.  Which token's interval u meets, and which token ends the nucleus, are
// matters of the last bits: sums of 32-bit floats over a large vocabulary would give
// another token once in a few dozen rows.  So a weight is held as a 64-bit integer in
// units of 2^-q of about the best token's (q = 50, less where the row's mass takes more bits: 45
// for 131072 equal tokens), exact to 2^-35 of itself and a unit, and sums of integers are
// exact in any order.
//
// A weight, relative to 2^N (N the least integer not below the best token's log2 w): t = 2048 c x
// as a sum of two floats, the nearest integer 2048 n + j split off, 2^(j / 2048) from a table in
// shared memory (made by each CTA, products of two small ones), and 2^r of the rest
// (|r| <= 1 / 4096) as 1 + two terms; the product and the shift by N - n are integer
// arithmetic.  About 20 instructions a logit.  (A table of 32 steps in the warp's lanes and six terms,
// the first in two floats, takes 30: 512 rows of 131072 to their nuclei in 622 us against 547 then.)
//
// A row is taken by a cluster of 1 to 4 CTAs, each warp on a contiguous run of spans
// of 1024 tokens.  One pass finds the maximum and leaves the maximum of every lane's 32
// tokens of a span in shared memory, and where the row's whole mass is asked for (no
// top-k, and a nucleus or nothing else) the mass of every span, relative to the span's own
// maximum: N changes a mass by a shift.  A bound below which no token can be kept follows
// from what is asked: the best lanes' maxima (k tokens are not below the least of k of
// them), min_p, or the row's mass S (tokens below (1 - p) S / V of it add up to less than
// what the nucleus leaves out).  The tokens above the bound, by id, go into a list in the
// first CTA's shared memory (a span whose maxima lie below it is not read again), where
// the k-th logit and the nucleus' last one are found, by counting what ranks before each token
// (up to 256) or by bisection over the order of the floats.  A row with more such tokens
// than the list holds is looked through where it lies (in L2 by then): a histogram of
// 2048 steps of the logit, of counts or of masses in 32 bits, names the few steps in which
// the border lies, a second look adds up exactly what lies above them, and the tokens in
// them are listed and searched.  (What defeats that, a row of equal logits, is bisected as
// a whole.)
//
// Bound by instructions and latency, not by the row's bytes: 512 rows of 131072 f32 logits
// to their nuclei (p 0.95) 400 us, 0.7 TB/s; 100 rows of 50257 with mixed settings 79 us;
// one row of 32000 18 us a call.  One block of 512 threads an SM: its rows take less of a wave
// each and its list holds twice the tokens (two blocks of 256: 502 and 100 us; a launch of its own for
// the rows without a list, which gives the others three blocks of 256 an SM, 754).  Not faster either:
// 80 registers a thread (spills), logits through registers instead of the ring of copies.
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <climits>
#include <cmath>
#include <cooperative_groups.h>

#include "logits.cuh"

namespace cg = cooperative_groups;

namespace spec {

constexpr int kDrThreads = 512;
// CTAs an SM up to which rows are cut into more of them: a single row's time counts where rows are few.  (100 mixed
// rows of 50257 take 82 us with one CTA a row, 79 with two, 95 with four; a row of 32000 19.6 with one, 18.1 with
// two or four; 512 rows of 131072 397 with one, 520 with four.)
constexpr int kDrCtasWanted = 1;
constexpr int kDrWarps = kDrThreads / 32;
constexpr int kDrMaxCtas = 4;
static_assert(kDrMaxCtas * kDrWarps <= 64, "two warps' numbers a lane");
constexpr int kDrSegs = 4;                             // segments of a span
constexpr int kDrSpan = kDrSegs * kLpSeg;
constexpr int kDrEach = 8;                             // listed tokens a thread
constexpr int kDrList = kDrEach * kDrThreads;
constexpr int kDrSpanUnit = 51;                        // 1024 weights in units of 2^-51 fit 64 bits, and so does a listed token's
constexpr int kDrListUnit = 50;
constexpr int kDrStage = 384;                          // tokens a warp holds before they go to the list (one CTA's sixteen: 256 on average)
constexpr int kDrBins = 2048;                          // steps of a histogram; it lies where the stages do
static_assert(kDrBins * 4 <= kDrWarps * kDrStage * 8 && kDrList <= kDrWarps * kDrStage, "histogram, masses by place");
constexpr int kDrRing = 4;                             // segments a warp has room for
constexpr int kDrCtasSm = 1;
constexpr int kDrMaxVocab = 1 << 20;
constexpr int kDrCtaVocab = 1 << 18;                   // a CTA's share at most: its lanes' maxima take 32 KB

struct DrawArgs {
    const void* x; long long stride;
    int V, per, q;                                     // per: spans a warp; q: the whole row's weights fit 64 bits as integers
                                                       // in units of 2^-q, whatever they are
    const float* u;
    float T, p, mp; int k;
    const float* Ts; const float* ps; const float* mps; const int* ks;   // settings by row; null: the ones above
    int* tok; float* lp;
    float* probs; long long p_stride; int p_vec;
    unsigned long long coarse[32], fine[64];           // 2^(62 + j / 32), 2^(63 + j / 2048)
};

typedef unsigned long long u64;

// a float's place in the order of the floats (both zeros alike)
SPEC_DEV uint32_t dr_ord(float v) {
    const uint32_t u = __float_as_uint(v + 0.f);
    return u >> 31 ? ~u : u | 0x80000000u;
}
SPEC_DEV float dr_value(uint32_t o) { return __uint_as_float(o >> 31 ? o & 0x7FFFFFFFu : ~o); }

// f * S for a float f in [0, 1], rounded down or up to an integer
SPEC_DEV u64 dr_part(float f, u64 S, bool up) {
    const uint32_t b = __float_as_uint(f);
    const int ex = (int)(b >> 23);
    const u64 mant = (b & 0x7FFFFFu) | (ex ? 0x800000u : 0u);
    const int sh = 150 - (ex ? ex : 1);                // f = mant * 2^-sh, sh >= 23
    const u64 lo = mant * S, hi = __umul64hi(mant, S);
    u64 r, rest;
    if (sh < 64) {
        r = (hi << (64 - sh)) | (lo >> sh);
        rest = lo << (64 - sh);
    } else {
        const int s = sh - 64;
        r = s < 64 ? hi >> s : 0;
        rest = lo | (s == 0 ? 0 : (s < 64 ? hi << (64 - s) : hi));
    }
    return r + (up && rest ? 1 : 0);
}

SPEC_DEV u64 dr_warp_sum(u64 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// exclusive sum over the lanes before this one
SPEC_DEV u64 dr_warp_before(u64 v, u64& total) {
    const int lane = threadIdx.x & 31;
    u64 s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 t = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += t;
    }
    total = __shfl_sync(0xffffffffu, s, 31);
    return s - v;
}

struct DrSmem {
    u64 red[2][kDrWarps];
    u64 part[2][kDrMaxCtas * kDrWarps];                // every warp's number, in every CTA
    float offer[kDrMaxCtas * kDrWarps];                // every warp's bound for top-k, and how many lanes' maxima reach it
    int reach[kDrMaxCtas * kDrWarps];
    float wmax[kDrWarps], cmax[kDrMaxCtas];
    int wbad[kDrWarps], cbad[kDrMaxCtas];
    u64 S;                                             // the first CTA's results for the others
    float cv;
    int ci, holds;
    int bin_lo, bin_hi, bin_at, stop;
};

// A weight's arithmetic.
constexpr int kDrSteps = 2048;                         // of the table, an octave
constexpr int kDrMagic = 0x4B400000;                   // 1.5 * 2^23: adding it leaves a float's nearest integer in the low bits
struct DrExp {
    float b, ch, cl;                                   // b: 0, or the maximum where c x has too many digits
    float most;                                        // -2048 t of a logit whose weight is below a unit
    int N, q;
    int shift;                                         // a weight's shift is this less its integer's upper bits
    uint32_t table;                                    // 2^(62 + j / 2048), in shared memory
    // weights relative to 2^N for logits up to `top`
    SPEC_DEV void refer_to(float top) { refer_to_n((int)ceilf((top - b) * ch * (1.f / kDrSteps))); }
    SPEC_DEV void refer_to_n(int n) {
        N = n;
        most = (float)(-kDrSteps * (N - q - 1));       // there the shift is 63, and leaves nothing
        shift = 62 - q + N + (kDrMagic >> 11);
    }
};
// c x as the arithmetic takes it: beyond, logits are taken relative to the maximum (exactly: those near it lie within
// a factor of two of it)
constexpr float kDrDigits = 2097152.f;

// ln 2 / 2048 and half its square, by 2^36
constexpr double kDrL = 0.69314718055994530942 / kDrSteps;
constexpr float kDrL1 = (float)(kDrL * 68719476736.0), kDrL2 = (float)(kDrL * kDrL / 2 * 68719476736.0);

SPEC_DEV float2 both(float x) { return make_float2(x, x); }

// weights of two logits: w = v * 2^-s in units of 2^-q, s in [0, 63], v in [2^62, 2^63)
SPEC_DEV void dr_weight2(const DrExp& E, float x0, float x1, u64 (&v)[2], int (&s)[2]) {
    const float2 neg = both(-1.f);
    const float2 d = add2(make_float2(x0, x1), both(-E.b));
    // p + e = 2048 t; p leaves its nearest integer.  (Where p is cut short, e, NaN for a masked logit, is
    // anything: what comes of it is shifted out.)
    float2 np = mul2(d, both(-E.ch));
    float2 e = fma2(d, both(E.ch), np);
    e = fma2(d, both(E.cl), e);
    np = make_float2(fminf(np.x, E.most), fminf(np.y, E.most));
    const float2 magic = both(__int_as_float(kDrMagic));
    const float2 k = fma2(np, neg, magic), nk = fma2(k, neg, magic), r = fma2(np, neg, nk);
    // 2^((r + e) / 2048) - 1 in units of 2^-36: off by 2^-36 of a weight, its f32 sums; the table's value to 26 bits
    // is enough for the product
    const float2 t = add2(r, e), f = mul2(fma2(both(kDrL2), t, both(kDrL1)), t);
    const float kf[2] = {k.x, k.y}, ff[2] = {f.x, f.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int ki = __float_as_int(kf[i]);
        u64 T;
        asm("ld.shared.u64 %0, [%1];" : "=l"(T) : "r"(E.table + (ki & (kDrSteps - 1)) * 8));
        v[i] = T + (u64)((long long)((int)(T >> 32) >> 4) * __float2int_rn(ff[i]));
        s[i] = E.shift - (ki >> 11);
    }
}
SPEC_DEV void dr_weights(const DrExp& E, const float (&x)[8], u64 (&w)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        u64 v[2];
        int s[2];
        dr_weight2(E, x[i], x[i + 1], v, s);
        w[i] = v[0] >> s[0];
        w[i + 1] = v[1] >> s[1];
    }
}
// a mass in units of 2^-by, to the nearest
SPEC_DEV u64 dr_rescale(u64 w, int by) { return by <= 0 ? w << -by : (by > 63 ? 0 : ((w >> (by - 1)) + 1) >> 1); }

// a kept logit: above the cut's value, or equal to it with an id not above the cut's
struct DrCut { float v; int id; };
SPEC_DEV bool dr_kept(const DrCut& c, float x, int id) { return x > c.v || (x == c.v && id <= c.id); }

template <typename T>
__global__ void __launch_bounds__(kDrThreads, kDrCtasSm)
draw_kernel(const __grid_constant__ DrawArgs a) {
    pdl_wait();
    pdl_trigger();
    constexpr int VE = 16 / sizeof(T), NP = 8 / VE;
    __shared__ DrSmem sm;
    extern __shared__ __align__(16) u64 dyn[];
    u64* list = dyn;                                   // [kDrList] (value's order, id) by id; the first CTA's
    u64* staged = dyn + kDrList;                       // [kDrWarps][kDrStage] what each warp has for it
    uint32_t* hist = reinterpret_cast<uint32_t*>(staged);       // [kDrBins] at other times
    u64* table = staged + kDrWarps * kDrStage;         // [kDrSteps]
    char* ring = reinterpret_cast<char*>(table + kDrSteps);     // [kDrWarps][kDrRing][NP][32] pieces
    u64* span_sum = reinterpret_cast<u64*>(ring + kDrWarps * kDrRing * NP * 512);       // [kDrWarps][per] masses, relative to 2^N
    int* span_n = reinterpret_cast<int*>(span_sum + kDrWarps * a.per);         // [kDrWarps][per] ... to 2^span_n at first
    float* lane_max = reinterpret_cast<float*>(span_n + kDrWarps * a.per);     // [kDrWarps][per][32]
    cg::cluster_group cl = cg::this_cluster();
    const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank(), NW = C * kDrWarps;
    const long long row_i = blockIdx.x / C;
    const int t = threadIdx.x, lane = t & 31, w = t >> 5, gw = rank * kDrWarps + w;
    const T* row = static_cast<const T*>(a.x) + row_i * a.stride;
    const int V = a.V, mis = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    const int n_span = (V + mis + kDrSpan - 1) / kDrSpan;
    const int s0 = min(n_span, gw * a.per), s1 = min(n_span, s0 + a.per);
    auto cluster_sync = [&]() {
        if (C > 1) cl.sync();
        else __syncthreads();
    };
    auto everywhere = [&](auto* p, auto value) {       // by one warp: the same variable of every CTA
        if (lane < C) *cl.map_shared_rank(p, lane) = value;
    };
    if (C > 1) cluster_arrive();                       // this CTA has started: its shared memory may be written

    const float temp = a.Ts ? a.Ts[row_i] : a.T, top_p = a.ps ? a.ps[row_i] : a.p, min_p = a.mps ? a.mps[row_i] : a.mp;
    const int top_k = a.ks ? a.ks[row_i] : a.k;
    const float u = a.u[row_i];
    const bool settings = (temp == 0.f || (temp >= 1e-30f && temp <= 1e30f)) && top_p >= 0.f && min_p >= 0.f && min_p <= 1.f &&
                          top_k >= 0 && u >= 0.f && u < 1.f;
    // temperature 0: the best token
    const int K = temp == 0.f ? 1 : (top_k >= V ? 0 : top_k);
    const float T_ = temp == 0.f ? 1.f : temp;
    const bool nucleus = top_p < 1.f;
    const bool whole = K == 0 && (nucleus || min_p == 0.f);        // the row's mass is asked for
    DrExp E;
    {   // 2048 log2 e / T in two floats
        constexpr double c = 1.4426950408889634074 * kDrSteps;
        constexpr float c_hi = (float)c, c_lo = (float)(c - (double)c_hi);
        E.ch = c_hi / T_;
        E.cl = (fmaf(-E.ch, T_, c_hi) + c_lo) / T_;
    }
    E.b = 0.f;
    E.q = kDrSpanUnit;
    E.table = smem_u32(table);
    for (int i = t; i < kDrSteps; i += kDrThreads) table[i] = __umul64hi(a.coarse[i >> 6], a.fine[i & 63]) << 1;
    __syncthreads();

    // this warp's part of an array by span (a span's owner is warp s / per of the cluster)
    u64* my_sum = span_sum + w * a.per;
    int* my_n = span_n + w * a.per;
    float* my_max = lane_max + w * a.per * 32;

    // the piece at row index i0, which the row does not fill: masked where it does not
    auto edge_piece = [&](int i0) {
        uint32_t u4[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (sizeof(T) == 4) {
                u4[j] = i0 + j >= 0 && i0 + j < V ? __float_as_uint(to_f32<T>(row[i0 + j])) : 0xFF800000u;
            } else {
                u4[j] = 0;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int d = i0 + 2 * j + h;
                    u4[j] |= (d >= 0 && d < V ? __float_as_uint(to_f32<T>(row[d])) >> 16 : 0xFF80u) << (16 * h);
                }
            }
        }
        return make_uint4(u4[0], u4[1], u4[2], u4[3]);
    };
    // a segment's pieces of this lane, as they lie in memory
    auto load_raw = [&](int seg, uint4 (&p)[NP]) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int i0 = seg * kLpSeg + (i * 32 + lane) * VE - mis;
            p[i] = i0 >= 0 && i0 + VE <= V ? __ldg(reinterpret_cast<const uint4*>(row + i0)) : edge_piece(i0);
        }
    };
    auto unpack = [&](const uint4 (&p)[NP], float (&x)[8]) {
#pragma unroll
        for (int i = 0; i < NP; ++i) lp_unpack<T>(p[i], &x[i * VE]);
    };
    // every span of this warp from s on that `wanted` names
    auto next_span = [&](int s, auto wanted) {
        while (s < s1 && !wanted(s)) ++s;
        return s;
    };
    // The segments of the spans that `wanted` names, in order (of each span all four, or one), f(logits, segment); then
    // done(span).  Three segments are copied ahead into the warp's ring, a lane's pieces into slots of its own, so
    // that a lane waits for its own copies only.
    const uint32_t slots = smem_u32(ring) + (w * kDrRing * NP * 32 + lane) * 16;
    auto stream = [&](auto wanted, bool one_of_four, auto f, auto done) {
        float x[8];
        int ls = next_span(s0, wanted), lg = one_of_four ? ls & 3 : 0, to = 0;      // the next segment to copy
        auto copy_next = [&]() {
            if (ls < s1) {
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    const int i0 = (ls * kDrSegs + lg) * kLpSeg + (i * 32 + lane) * VE - mis;
                    const uint32_t dst = slots + (to * NP + i) * 512;
                    if (i0 >= 0 && i0 + VE <= V) {
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(row + i0) : "memory");
                    } else {
                        const uint4 v = edge_piece(i0);
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" :: "r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
                    }
                }
                if (one_of_four || ++lg == kDrSegs) {
                    ls = next_span(ls + 1, wanted);
                    lg = one_of_four ? ls & 3 : 0;
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            to = (to + 1) % kDrRing;
        };
        int s = ls, at = 0;
#pragma unroll
        for (int i = 0; i < kDrRing - 1; ++i) copy_next();
        while (s < s1) {
#pragma unroll 1
            for (int g = one_of_four ? s & 3 : 0; g < kDrSegs; ++g) {
                asm volatile("cp.async.wait_group %0;" :: "n"(kDrRing - 2) : "memory");
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    uint4 v;
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(slots + (at * NP + i) * 512) : "memory");
                    lp_unpack<T>(v, &x[i * VE]);
                }
                at = (at + 1) % kDrRing;
                copy_next();
                f(x, s * kDrSegs + g);
                if (one_of_four) break;
            }
            done(s);
            s = next_span(s + 1, wanted);
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    };
    auto every = [&](int) { return true; };
    // spans that hold a logit not below `least`
    auto reaching = [&](float least) {
        return [&, least](int s) { return __any_sync(0xffffffffu, my_max[(s - s0) * 32 + lane] >= least); };
    };

    // -------- the maximum, every lane's maxima, the spans' masses, and whether the row has a distribution
    float mx = -INFINITY, lm = -INFINITY;
    bool bad = false;
    if (whole && settings) {
        u64 sum = 0;
        int N = INT_MIN;
        stream(every, false, [&](const float (&x)[8], int) {
            float gm = x[0];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                bad |= !(x[i] <= FLT_MAX);             // NaN or +inf
                gm = fmaxf(gm, x[i]);
            }
            lm = fmaxf(lm, gm);
            const float top = warp_redux_max(gm);
            // (logits this large: none of the row's mass, or its maximum is one of them and the pass does not count)
            if (!(fabsf(top * E.ch) < kDrDigits)) return;
            const int n = (int)ceilf(top * E.ch * (1.f / kDrSteps));
            if (n > N) {
                if (N != INT_MIN) sum = dr_rescale(sum, n - N);
                N = n;
                E.refer_to_n(N);
            }
            u64 wt[8];
            dr_weights(E, x, wt);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += wt[i];
        }, [&](int s) {
            my_max[(s - s0) * 32 + lane] = lm;
            mx = fmaxf(mx, lm);
            sum = dr_warp_sum(sum);
            if (lane == 0) {
                my_sum[s - s0] = sum;
                my_n[s - s0] = N;
            }
            lm = -INFINITY;
            sum = 0;
            N = INT_MIN;
        });
    } else {
        stream(every, false, [&](const float (&x)[8], int) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                bad |= !(x[i] <= FLT_MAX);
                lm = fmaxf(lm, x[i]);
            }
        }, [&](int s) {
            my_max[(s - s0) * 32 + lane] = lm;
            mx = fmaxf(mx, lm);
            lm = -INFINITY;
        });
    }
    mx = warp_redux_max(mx);
    bad = __any_sync(0xffffffffu, bad);
    __syncwarp();
    // This warp's share of the bound for top-k: of the warps with a full run of whole spans (none: no bound) each
    // offers the value of (about) its r-th largest lane maximum.  The least of these has r tokens a warp that are not
    // below it; below, a larger one is taken that has k all the same.
    float low = INFINITY;
    const int full = (V + mis) / kDrSpan / a.per, r_low = K > 1 && full > 0 ? (K + full - 1) / full : 0;
    if (r_low > 0 && gw < full) {
        low = -INFINITY;
        if (r_low == 1) {
            low = mx;
        } else if (r_low <= 32 * a.per) {
            uint32_t lo = 0, hi = dr_ord(mx);          // at least r not below lo; hi: fewer (or not looked at)
            while (hi - lo > 1) {
                const uint32_t mid = lo + (hi - lo) / 2;
                const float v = dr_value(mid);
                int n = 0;
                for (int i = 0; i < a.per; ++i) n += my_max[i * 32 + lane] >= v;
                n = __reduce_add_sync(0xffffffffu, n);
                if (n >= r_low) {
                    lo = mid;
                    if (n <= r_low + r_low / 16) break;
                } else {
                    hi = mid;
                }
            }
            low = dr_value(lo);
            if (!(low >= -FLT_MAX)) low = -INFINITY;
        }
    }
    if (lane == 0) { sm.wmax[w] = mx; sm.wbad[w] = bad; }
    __syncthreads();
    if (C > 1) cluster_wait();
    everywhere(&sm.offer[gw], low);
    if (w == 0) {
        const float m = warp_redux_max(lane < kDrWarps ? sm.wmax[lane] : -INFINITY);
        const bool b = __any_sync(0xffffffffu, lane < kDrWarps && sm.wbad[lane]);
        everywhere(&sm.cmax[rank], m);
        everywhere(&sm.cbad[rank], (int)b);
    }
    cluster_sync();
    const float m = warp_redux_max(lane < C ? sm.cmax[lane] : -INFINITY);
    bad = __any_sync(0xffffffffu, lane < C && sm.cbad[lane]);
    float* probs = a.probs ? a.probs + row_i * a.p_stride : nullptr;
    if (bad || m == -INFINITY || !settings) {          // no distribution, or settings out of range
        const float nan = __int_as_float(0x7fc00000);
        if (rank == 0 && t == 0) {
            a.tok[row_i] = -1;
            if (a.lp) a.lp[row_i] = nan;
        }
        if (probs)
            for (int i = rank * kDrThreads + t; i < V; i += C * kDrThreads) probs[i] = nan;
        return;
    }
    const bool far = !(fabsf(m * E.ch) < kDrDigits);
    if (far) E.b = m;
    u64 one, w_min;                                    // the best token's weight, the least that min_p leaves
    auto set_unit = [&](int q) {
        E.q = q;
        E.refer_to(m);
        u64 v[2];
        int s[2];
        dr_weight2(E, m, m, v, s);
        one = v[0] >> s[0];
        w_min = dr_part(min_p, one, true);
    };

    // Every warp's number in every CTA (two buffers in turn: whoever writes one has passed the barrier of the other,
    // which comes after everybody's reading of this one): their sum, and the sum of the warps before this one.
    int turn = 0;
    auto exchange = [&](u64 mine, u64& before) {
        everywhere(&sm.part[turn][gw], mine);
        cluster_sync();
        const u64 x = 2 * lane < NW ? sm.part[turn][2 * lane] : 0, y = 2 * lane < NW ? sm.part[turn][2 * lane + 1] : 0;
        turn ^= 1;
        u64 all;
        const u64 at = dr_warp_before(x + y, all) + (gw & 1 ? x : 0);
        before = __shfl_sync(0xffffffffu, at, gw >> 1);
        return all;
    };
    auto sum_all = [&](u64 v) {                        // of what the warps hold (in every lane)
        u64 before;
        return exchange(v, before);
    };
    // sums over the CTA
    int par = 0;
    auto sum_cta = [&](u64 v) {
        v = dr_warp_sum(v);
        if (lane == 0) sm.red[par][w] = v;
        __syncthreads();
        u64 s = 0;
#pragma unroll
        for (int i = 0; i < kDrWarps; ++i) s += sm.red[par][i];
        par ^= 1;
        return s;
    };
    // what the threads before this one hold, and all
    auto before_cta = [&](u64 v, u64& all) {
        u64 in_warp, at = dr_warp_before(v, in_warp);
        if (lane == 0) sm.red[par][w] = in_warp;
        __syncthreads();
        all = 0;
#pragma unroll
        for (int i = 0; i < kDrWarps; ++i) {
            if (i == w) at += all;
            all += sm.red[par][i];
        }
        par ^= 1;
        return at;
    };
    // Weights of the segments that reach `least` by f(logits, segment, weights): every span's sum in my_sum, the warp's
    // returned.
    auto span_masses = [&](float least, auto f) {
        u64 sum = 0, mine = 0;
        for (int i = lane; i < s1 - s0; i += 32) my_sum[i] = 0;
        __syncwarp();
        stream(reaching(least), false, [&](const float (&x)[8], int seg) {
            u64 wt[8];
            f(x, seg, wt);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += wt[i];
        }, [&](int s) {
            sum = dr_warp_sum(sum);
            if (lane == 0) my_sum[s - s0] = sum;
            mine += sum;
            sum = 0;
        });
        __syncwarp();
        return mine;
    };
    auto kept_weights = [&](const DrCut& cut, float least, u64 w_least) {
        return [&, cut, least, w_least](const float (&x)[8], int seg, u64 (&wt)[8]) {
            dr_weights(E, x, wt);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (!(x[i] >= least) || wt[i] < w_least || !dr_kept(cut, x[i], lp_index<T>(mis, seg, i))) wt[i] = 0;
        };
    };
    // With every span's sum in my_sum, `mine` a warp's: the token by id, weighed by f, at which the sum passes the
    // target; found(id, logit, total) is called by one thread of the cluster.
    auto locate = [&](u64 mine, auto f, auto target_of, auto found) {
        u64 before;
        const u64 total = exchange(mine, before), target = target_of(total);
        if (before <= target && target < before + mine) {
            u64 left = target - before;
            int s = s0;
            while (s + 1 < s1 && left >= my_sum[s - s0]) left -= my_sum[s++ - s0];
            // (the first pass' masses are rounded on their way to a common unit: the span's own, once more)
            u64 exact = 0;
            uint4 p[NP];
            float x[8];
            u64 wt[8];
#pragma unroll 1
            for (int g = 0; g < kDrSegs; ++g) {
                load_raw(s * kDrSegs + g, p);
                unpack(p, x);
                f(x, s * kDrSegs + g, wt);
#pragma unroll
                for (int i = 0; i < 8; ++i) exact += wt[i];
            }
            exact = dr_warp_sum(exact);
            const bool ones = exact == 0;
            left = ones ? 0 : min(left, exact - 1);
            bool done = false;
#pragma unroll 1
            for (int g = 0; g < kDrSegs && !done; ++g) {
                load_raw(s * kDrSegs + g, p);
                unpack(p, x);
                f(x, s * kDrSegs + g, wt);
                if (ones)
#pragma unroll
                    for (int i = 0; i < 8; ++i) wt[i] = x[i] >= -FLT_MAX ? 1 : 0;
#pragma unroll
                for (int k = 0; k < NP; ++k) {
                    u64 sum = 0, all;
#pragma unroll
                    for (int i = 0; i < VE; ++i) sum += wt[k * VE + i];
                    const u64 pre = dr_warp_before(sum, all);
                    if (!done && left < all) {
                        if (pre <= left && left < pre + sum) {
                            u64 at = pre;
                            bool hit = false;
#pragma unroll
                            for (int i = 0; i < VE; ++i) {
                                at += wt[k * VE + i];
                                if (!hit && left < at) {
                                    hit = true;
                                    found(lp_index<T>(mis, s * kDrSegs + g, k * VE + i), x[k * VE + i], total);
                                }
                            }
                        }
                        done = true;
                    }
                    left -= done ? 0 : all;
                }
            }
        }
        return total;
    };
    auto finish = [&](int id, float x, u64 S) {
        a.tok[row_i] = id;
        if (a.lp) {
            // log S without cancellation where one token holds nearly all of it
            const float ls = S < 2 * one ? log1pf((float)(S - one) / (float)one) : logf((float)S / (float)one);
            a.lp[row_i] = (x - m) / T_ - ls;
        }
    };
    // The kept tokens in [from, to), by id, into the first CTA's list if it holds them (their number, or more than
    // the list's length); weighed: and the mass of the kept tokens from `to` on, the spans' in my_sum.
    u64 over_mass = 0;                                 // this warp's
    auto make_list = [&](float from, float to, const DrCut& old, bool cut_some, bool weighed) {
        u64* mine = staged + w * kDrStage;
        int n = 0, told = 0;
        u64 sum = 0;
        over_mass = 0;
        if (t == 0) sm.stop = 0;
        if (weighed)
            for (int i = lane; i < s1 - s0; i += 32) my_sum[i] = 0;
        __syncthreads();
        const auto reach = reaching(from);
        stream([&](int s) { return (weighed || !__any_sync(0xffffffffu, *(volatile int*)&sm.stop > kDrList)) && reach(s); }, false, [&](const float (&x)[8], int seg) {
            uint32_t in = 0, above = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) in |= x[i] >= from ? 1u << i : 0u;
            if (to < INFINITY) {
#pragma unroll
                for (int i = 0; i < 8; ++i) above |= x[i] >= to ? 1u << i : 0u;
                in &= ~above;
            }
            if (cut_some)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (!dr_kept(old, x[i], lp_index<T>(mis, seg, i))) in &= ~(1u << i);
            if (weighed && __any_sync(0xffffffffu, above != 0)) {
                u64 wt[8];
                dr_weights(E, x, wt);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if ((above >> i) & 1u && (!cut_some || dr_kept(old, x[i], lp_index<T>(mis, seg, i)))) sum += wt[i];
            }
            if (!__any_sync(0xffffffffu, in != 0)) return;
            // places by piece, lane, element: two pieces' counts in one scan
            const uint32_t c = NP == 1 ? __popc(in) : __popc(in & 0xFu) | (uint32_t)__popc(in >> 4) << 16;
            uint32_t upto = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
            const uint32_t all = __shfl_sync(0xffffffffu, upto, 31);
            int at = n + (int)((upto - c) & 0xFFFFu), at2 = n + (int)(all & 0xFFFFu) + (int)((upto - c) >> 16);
            for (; in; in &= in - 1u) {                // (most lanes have none)
                const int i = __ffs(in) - 1, k = i < VE ? at++ : at2++;
                float v = x[0];
#pragma unroll
                for (int j = 1; j < 8; ++j) v = i == j ? x[j] : v;
                if (k < kDrStage) mine[k] = (u64)dr_ord(v) << 32 | (uint32_t)lp_index<T>(mis, seg, i);
            }
            __syncwarp();
            n += (int)(all & 0xFFFFu) + (int)(all >> 16);
        }, [&](int s) {
            if (!weighed) {
                // what the CTA's warps have found: once the list will not hold it, they stop
                if (lane == 0) atomicAdd(&sm.stop, n - told);
                told = n;
                return;
            }
            sum = dr_warp_sum(sum);
            if (lane == 0) my_sum[s - s0] = sum;
            over_mass += sum;
            sum = 0;
        });
        __syncwarp();
        // a warp with more than its stage holds takes another look (order unlike chance's), if the list takes them
        u64 before;
        const u64 total = exchange((u64)n, before);
        if (total <= kDrList && n > 0) {
            u64* first = cl.map_shared_rank(list, 0) + before;
            if (n <= kDrStage) {
                for (int i = lane; i < n; i += 32) first[i] = mine[i];
            } else {
                int at = 0;
                for (int s = s0; s < s1; ++s) {
                    if (!reach(s)) continue;
                    for (int i0 = s * kDrSpan - mis; i0 < (s + 1) * kDrSpan - mis; i0 += 32) {
                        const int id = i0 + lane;
                        const float x = id >= 0 && id < V ? to_f32<T>(row[id]) : -INFINITY;
                        const bool in = x >= from && x < to && dr_kept(old, x, id);
                        const uint32_t b = __ballot_sync(0xffffffffu, in);
                        if (in) first[at + __popc(b & ((1u << lane) - 1u))] = (u64)dr_ord(x) << 32 | (uint32_t)id;
                        at += __popc(b);
                    }
                }
            }
        }
        cluster_sync();
        return total;
    };

    // -------- a bound below which nothing is kept
    const float slack = 1e-3f;
    const DrCut nothing{-INFINITY, -1};                // (every finite logit is kept)
    float low_bound = -FLT_MAX;
    u64 S = 0, p_target = 0, mine_all = 0;             // the row's mass, this warp's part of it
    auto below = [&](float z) {                        // safely below m + T z
        const float v = m + T_ * (z - slack);
        return fmaxf(v - fabsf(v) * 1e-6f, -FLT_MAX);
    };
    if (whole) {
        // the row's mass in units of 2^-43 (2^20 tokens at most), and with it the unit for the rest
        constexpr int kRowUnit = 43;
        set_unit(kRowUnit);
        if (far) {
            mine_all = span_masses(-FLT_MAX, kept_weights(nothing, -FLT_MAX, 0));
        } else {
            for (int i = 0; i < s1 - s0; ++i) mine_all += my_n[i] == INT_MIN ? 0 : dr_rescale(my_sum[i], E.N - my_n[i] + kDrSpanUnit - kRowUnit);
        }
        S = sum_all(mine_all);
        const int q = min(kDrListUnit, kRowUnit + __clzll(S) - 2);      // S < 2^62 of them
        set_unit(q);
        for (int i = lane; i < s1 - s0; i += 32)
            my_sum[i] = far ? dr_rescale(my_sum[i], kRowUnit - q) : (my_n[i] == INT_MIN ? 0 : dr_rescale(my_sum[i], E.N - my_n[i] + kDrSpanUnit - q));
        __syncwarp();
        mine_all = 0;
        for (int i = 0; i < s1 - s0; ++i) mine_all += my_sum[i];
        S = dr_rescale(S, kRowUnit - q);
    } else {
        set_unit(kDrListUnit);
    }
    bool listed = true;
    if (K == 1) {
        low_bound = m;
    } else if (K > 0) {
        if (full > 0) {
            // Of the warps' offers the largest that K lanes' maxima reach: every warp counts its own for each of the
            // offers (two a lane), and the counts add up in every CTA.
            const float a0 = lane < NW ? sm.offer[lane] : INFINITY, a1 = lane + 32 < NW ? sm.offer[lane + 32] : INFINITY;
            int n0 = 0, n1 = 0;
            for (int s = s0; s < s1; ++s)
                for (int i = 0; i < 32; ++i) {
                    const float v = my_max[(s - s0) * 32 + i];
                    n0 += v >= a0;
                    n1 += v >= a1;
                }
            if (t < kDrMaxCtas * kDrWarps) sm.reach[t] = 0;
            cluster_sync();
            for (int i = 0; i < C; ++i) {
                int* r = cl.map_shared_rank(sm.reach, i);
                if (n0) atomicAdd(r + lane, n0);
                if (n1) atomicAdd(r + lane + 32, n1);
            }
            cluster_sync();
            float best = -FLT_MAX;
            if (lane < NW && a0 < INFINITY && sm.reach[lane] >= K) best = fmaxf(best, a0);
            if (lane + 32 < NW && a1 < INFINITY && sm.reach[lane + 32] >= K) best = fmaxf(best, a1);
            low_bound = warp_redux_max(best);
        }
    } else if (nucleus) {
        p_target = max(dr_part(top_p, S, true), 1ull);
        low_bound = below(logf(fmaxf((1.f - top_p) * ((float)S / (float)one) / (float)V, 1e-30f)));
    } else {
        listed = min_p > 0.f;
    }
    // (min_p leaves out of top-k's and the nucleus' tokens, whose number and mass count them)
    if (min_p > 0.f && K == 0) low_bound = fmaxf(low_bound, below(logf(min_p)));
    u64 n_list = 0;
    if (listed) {
        n_list = make_list(low_bound, INFINITY, nothing, false, false);
        listed = n_list <= kDrList;
    }

    DrCut cut = nothing;
    u64 S_kept = 0;
    // -------- the first CTA's threads with `each` neighbours of the list
    uint32_t o[kDrEach];
    int id[kDrEach];
    u64 wt[kDrEach];
    auto take_list = [&](int n) {
        const int each = (n + kDrThreads - 1) / kDrThreads;
        float x[kDrEach];
#pragma unroll
        for (int e = 0; e < kDrEach; ++e) {
            const int i = t * each + e;
            const bool in = e < each && i < n;
            const u64 key = in ? list[i] : 0;
            o[e] = (uint32_t)(key >> 32);
            id[e] = (int)(uint32_t)key;
            x[e] = in ? dr_value(o[e]) : -INFINITY;
        }
        dr_weights(E, x, wt);
#pragma unroll
        for (int e = 0; e < kDrEach; ++e)
            if (o[e] == 0) wt[e] = 0;
    };
    // Keeps the tokens of the list that come first, by decreasing logit (equal ones by id), until they number `first`
    // and, of these, until they weigh need(weight of all of these) (no more than what stays where they do not).
    // A token's place: 2048 steps of the logit from `top` down to `from`, counted, and inside its step by comparing.
    auto cut_list = [&](int n, float from, float top, u64 first, bool weighed, auto need) {
        u64* sorted = list;
        u64* by_place = staged;
        const float step = (float)(kDrBins - 1) / fmaxf(top - from, 1e-30f);
        auto bin_of = [&](uint32_t ord) { return max(0, min(kDrBins - 1, (int)((top - dr_value(ord)) * step))); };
        for (int i = t; i < kDrBins; i += kDrThreads) hist[i] = 0;
        __syncthreads();                               // (and the list has been taken)
        int in_bin[kDrEach];
#pragma unroll
        for (int e = 0; e < kDrEach; ++e)
            if (o[e]) in_bin[e] = (int)atomicAdd(&hist[bin_of(o[e])], 1u);
        __syncthreads();
        constexpr int kEachBin = kDrBins / kDrThreads;
        uint32_t h[kEachBin];
        u64 sum = 0, all;
        bool crowd = false;
#pragma unroll
        for (int e = 0; e < kEachBin; ++e) {
            h[e] = hist[t * kEachBin + e];
            sum += h[e];
            crowd |= h[e] > 64;
        }
        crowd = __syncthreads_or(crowd);
        u64 at = before_cta(sum, all);
        if (crowd) {
            // many equal or nearly equal logits: by bisection over the order of the floats
            const uint32_t o_from = max(dr_ord(-INFINITY) + 1, dr_ord(from)), o_to = dr_ord(m) + 1;
            auto cut_at = [&](uint32_t v, u64 k) {     // the first k by id of the tokens equal to v stay, and those above
                u64 mine = 0, every;
#pragma unroll
                for (int e = 0; e < kDrEach; ++e) mine += o[e] == v ? 1 : 0;
                u64 place = before_cta(mine, every);
#pragma unroll
                for (int e = 0; e < kDrEach; ++e) {
                    if (o[e] == v && place++ >= k) o[e] = 0;
                    if (o[e] < v) o[e] = 0;
                    if (o[e] == 0) wt[e] = 0;
                }
            };
            auto reach = [&](uint32_t v, bool weigh) {
                u64 s = 0;
#pragma unroll
                for (int e = 0; e < kDrEach; ++e) s += o[e] >= v && o[e] ? (weigh ? wt[e] : 1) : 0;
                return sum_cta(s);
            };
            auto bisect = [&](u64 goal, bool weigh) {
                uint32_t lo = o_from, hi = o_to;
                while (hi - lo > 1) {
                    const uint32_t mid = lo + (hi - lo) / 2;
                    if (reach(mid, weigh) >= goal) lo = mid;
                    else hi = mid;
                }
                return lo;
            };
            if (first < (u64)n) {
                const uint32_t v = bisect(first, false);
                cut_at(v, first - reach(v + 1, false));
            }
            if (weighed) {
                const u64 mass = reach(1, true), goal = need(mass);
                if (mass >= goal) {
                    const uint32_t v = bisect(goal, true);
                    const u64 rest = goal - reach(v + 1, true);
                    u64 w1 = 0;                        // tokens of one value have one weight
#pragma unroll
                    for (int e = 0; e < kDrEach; ++e)
                        if (o[e] == v) w1 = wt[e];
                    const u64 holders = sum_cta(w1 ? 1 : 0);
                    w1 = sum_cta(w1) / holders;
                    cut_at(v, (rest + w1 - 1) / w1);
                }
            }
            return;
        }
#pragma unroll
        for (int e = 0; e < kEachBin; ++e) {
            hist[t * kEachBin + e] = (uint32_t)at;     // the tokens of the steps before
            at += h[e];
        }
        __syncthreads();
        const int each = (n + kDrThreads - 1) / kDrThreads;
#pragma unroll
        for (int e = 0; e < kDrEach; ++e)
            if (o[e]) sorted[hist[bin_of(o[e])] + in_bin[e]] = (u64)o[e] << 32 | (uint32_t)~(t * each + e);
        __syncthreads();
        int place[kDrEach];
#pragma unroll
        for (int e = 0; e < kDrEach; ++e) {
            if (!o[e]) continue;
            const int b = bin_of(o[e]), b0 = hist[b], b1 = b + 1 < kDrBins ? (int)hist[b + 1] : n;
            const u64 key = (u64)o[e] << 32 | (uint32_t)~(t * each + e);
            place[e] = b0;
            for (int j = b0; j < b1; ++j) place[e] += sorted[j] > key;
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < kDrEach; ++e) {
            if (!o[e]) continue;
            if ((u64)place[e] >= first) { o[e] = 0; wt[e] = 0; }
            if (weighed) by_place[place[e]] = wt[e];
        }
        if (!weighed) return;
        __syncthreads();
        u64 mine[kDrEach], mass = 0;
#pragma unroll
        for (int e = 0; e < kDrEach; ++e) {
            const int i = t * kDrEach + e;
            mine[e] = i < n ? by_place[i] : 0;
            mass += mine[e];
        }
        at = before_cta(mass, all);
#pragma unroll
        for (int e = 0; e < kDrEach; ++e) {
            by_place[t * kDrEach + e] = at;            // the mass before the place
            at += mine[e];
        }
        __syncthreads();
        const u64 goal = need(all);
#pragma unroll
        for (int e = 0; e < kDrEach; ++e)
            if (o[e] && by_place[place[e]] >= goal) { o[e] = 0; wt[e] = 0; }
    };
    // the least kept token of the list as (value's order, ~id)
    auto least_key = [&]() {
        u64 least = ~0ull;
#pragma unroll
        for (int e = 0; e < kDrEach; ++e)
            if (o[e]) least = min(least, (u64)o[e] << 32 | (uint32_t)~id[e]);
#pragma unroll
        for (int b = 16; b > 0; b >>= 1) least = min(least, __shfl_xor_sync(0xffffffffu, least, b));
        if (lane == 0) sm.red[par][w] = least;
        __syncthreads();
        for (int i = 0; i < kDrWarps; ++i) least = min(least, sm.red[par][i]);
        par ^= 1;
        return least;
    };
    if (listed) {
        if (rank == 0) {
            const int n = (int)n_list;
            take_list(n);
            if ((K > 0 && n > K) || nucleus)
                cut_list(n, low_bound, m, K > 0 ? (u64)K : ~0ull, nucleus, [&](u64 all) {
                    return K > 0 ? max(dr_part(top_p, all, true), 1ull) : p_target;
                });
            u64 mine = 0, sum;
#pragma unroll
            for (int e = 0; e < kDrEach; ++e) {
                if (wt[e] < w_min) wt[e] = 0;
                mine += wt[e];
            }
            u64 at = before_cta(mine, sum);
            const u64 target = dr_part(u, sum, false);
            if (at <= target && target < at + mine) {
                bool hit = false;
#pragma unroll
                for (int e = 0; e < kDrEach; ++e) {
                    at += wt[e];
                    if (!hit && target < at) {
                        hit = true;
                        finish(id[e], dr_value(o[e]), sum);
                    }
                }
            }
            if (probs) {
                const u64 least = least_key();
                if (w == 0) {
                    everywhere(&sm.S, sum);
                    everywhere(&sm.cv, dr_value((uint32_t)(least >> 32)));
                    everywhere(&sm.ci, (int)~(uint32_t)least);
                }
            }
        }
        if (!probs) return;
        cluster_sync();
        S_kept = sm.S;
        cut = DrCut{sm.cv, sm.ci};
    } else {
        // -------- the row where it lies
        if (!whole) set_unit(a.q);
        bool masses = whole;                           // my_sum holds the spans' masses of what is kept
        u64 mine = mine_all;
        // The cut at which the kept tokens, by decreasing logit, reach `need`, counted or weighed (`all` in all).
        auto select = [&](u64 need, bool weighed, u64 all) {
            const DrCut old = cut;
            const bool cut_some = old.v > -INFINITY;
            constexpr int kEachBin = kDrBins / kDrThreads;
            constexpr float kWholeUnits = 1073741824.f;                        // the whole mass in a histogram's units
            const float per_one = weighed ? kWholeUnits / ((float)all / (float)one) : 1.f, c2 = E.ch * (1.f / kDrSteps);
            const long long goal = weighed ? (long long)((float)need / (float)all * kWholeUnits) : (long long)need;
            // A histogram of the kept tokens in [from, to) by the logit, from the top down, and from it the steps that may
            // hold the border: [from, to) shrinks to them.  A look at every fourth segment (masses only) is filled up
            // to the whole mass from the top, so that what it errs by is its error of the mass below the border.
            auto narrow = [&](float& from, float& to, bool quarter) {
                const float top = fminf(to, m), step = (float)(kDrBins - 1) / fmaxf(top - from, 1e-30f);
                const bool by_order = from == -FLT_MAX;        // (without a bound the steps are steps of the floats' order)
                const uint32_t o_max = dr_ord(m), o_inf = dr_ord(-INFINITY);
                for (int i = t; i < kDrBins; i += kDrThreads) hist[i] = 0;
                __syncthreads();
                u64 outside = 0, under = 0;            // what lies above, and below
                auto look = [&](const float (&x)[8], int seg) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const bool in = x[i] >= -FLT_MAX && (!cut_some || dr_kept(old, x[i], lp_index<T>(mis, seg, i)));
                        const uint32_t c = !in ? 0u : weighed ? __float2uint_rn(ex2((x[i] - m) * c2) * per_one) : 1u;
                        const bool inside = x[i] >= from && x[i] < to;
                        if (inside && c) atomicAdd(&hist[by_order ? (o_max - dr_ord(x[i])) >> 21 : min(kDrBins - 1, (int)((top - x[i]) * step))], c);
                        if (to < INFINITY) outside += x[i] >= to ? c : 0u;
                        if (quarter) under += x[i] < from ? c : 0u;
                    }
                };
                if (quarter) stream(every, true, look, [](int) {});
                else stream(reaching(from), false, look, [](int) {});
                under = sum_all(dr_warp_sum(under));
                const u64 over = sum_all(dr_warp_sum(outside));                // (and the histograms are there)
                u64 h[kEachBin], sum = 0, inside;
#pragma unroll
                for (int e = 0; e < kEachBin; ++e) h[e] = 0;
#pragma unroll
                for (int i = 0; i < kDrMaxCtas; ++i) {
                    const uint4* r = reinterpret_cast<const uint4*>(cl.map_shared_rank(hist, min(i, C - 1))) + t * (kEachBin / 4);
#pragma unroll
                    for (int e = 0; e < kEachBin / 4; ++e) {
                        const uint4 v = i < C ? r[e] : make_uint4(0, 0, 0, 0);
                        h[4 * e] += v.x;
                        h[4 * e + 1] += v.y;
                        h[4 * e + 2] += v.z;
                        h[4 * e + 3] += v.w;
                    }
                }
#pragma unroll
                for (int e = 0; e < kEachBin; ++e) sum += h[e];
                if (t == 0) { sm.bin_lo = kDrBins; sm.bin_hi = sm.bin_at = 0; }
                long long at = (long long)before_cta(sum, inside), err = weighed ? 8192 : 0;    // (masses are rounded and a little off)
                at += (long long)over;
                const int scale = quarter ? 4 : 1;
                if (quarter) {
                    at += ((long long)kWholeUnits - 4 * (long long)(over + inside + under)) / 4;   // in quarters of the units
                    // the mass below the border is off by a few parts of a hundred: as many tokens on either side as the
                    // list may hold, but 1 / 48 of that mass at least and 1 / 8 at most
                    long long sum_to = at;
                    int b_at = 0;
#pragma unroll
                    for (int e = 0; e < kEachBin; ++e) {
                        sum_to += (long long)h[e];
                        if (4 * sum_to < goal) b_at = t * kEachBin + e + 1;
                    }
                    atomicMax(&sm.bin_at, b_at);
                    __syncthreads();
                    const float w_at = ex2((top - (float)sm.bin_at / step - m) * c2) * per_one;
                    const long long rest = (long long)kWholeUnits - goal;
                    err += min(max(rest / 48, (long long)(800.f * w_at)), rest / 8);
                }
#pragma unroll
                for (int e = 0; e < kEachBin; ++e) {
                    at += (long long)h[e];
                    if (scale * at + err >= goal) atomicMin(&sm.bin_lo, t * kEachBin + e);      // first that may hold the border
                    if (scale * at < goal + err) atomicMax(&sm.bin_hi, t * kEachBin + e + 1);   // past it: the last that may
                }
                cluster_sync();                        // (the histograms are read; their memory may be written)
                const int b_lo = min(sm.bin_lo, kDrBins - 1), b_hi = min(sm.bin_hi, kDrBins - 1);
                __syncthreads();                       // (before they are set again)
                if (by_order) {
                    const uint32_t up = (uint32_t)b_lo << 21, down = ((uint32_t)b_hi + 1) << 21;
                    if (b_lo > 0) to = dr_value(o_max - up + 1);
                    from = b_hi + 1 < 2048 && down < o_max - o_inf ? dr_value(o_max - down) : -FLT_MAX;
                } else {
                    // a step more on either side: what the steps' rounding may move
                    if (b_lo > 1) to = top - (float)(b_lo - 1) / step;
                    from = fmaxf(from, top - (float)(b_hi + 2) / step);
                }
            };
            // The border among the tokens of [from, to), if the list holds them and it lies there.
            auto settle = [&](float from, float to) {
                const u64 n = make_list(from, to, old, cut_some, weighed);
                if (n > kDrList) return false;
                u64 over = 0;
                if (weighed) {
                    over = over_mass;
                } else {
                    stream(reaching(to), false, [&](const float (&x)[8], int seg) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) over += x[i] >= to && dr_kept(old, x[i], lp_index<T>(mis, seg, i)) ? 1 : 0;
                    }, [](int) {});
                    over = dr_warp_sum(over);
                }
                over = sum_all(over);
                masses = weighed;
                if (rank == 0) {
                    take_list((int)n);
                    u64 in = 0;
#pragma unroll
                    for (int e = 0; e < kDrEach; ++e) in += o[e] ? (weighed ? wt[e] : 1) : 0;
                    in = sum_cta(in);
                    const bool holds = over < need && need <= over + in;
                    if (holds) {
                        cut_list((int)n, from, fminf(to, m), weighed ? ~0ull : need - over, weighed, [&](u64) { return need - over; });
                        const u64 least = least_key();
                        if (weighed) {
                            // the listed tokens that stay, to the masses of their spans
#pragma unroll
                            for (int e = 0; e < kDrEach; ++e)
                                if (o[e]) {
                                    const int s = (id[e] + mis) / kDrSpan, owner = s / a.per;
                                    atomicAdd(cl.map_shared_rank(&span_sum[(owner % kDrWarps) * a.per + s - owner * a.per], owner / kDrWarps), wt[e]);
                                }
                        }
                        if (w == 0) {
                            everywhere(&sm.cv, dr_value((uint32_t)(least >> 32)));
                            everywhere(&sm.ci, (int)~(uint32_t)least);
                        }
                    }
                    if (w == 0) everywhere(&sm.holds, (int)holds);
                }
                cluster_sync();
                if (!sm.holds) return false;
                cut = DrCut{sm.cv, sm.ci};
                if (weighed) {
                    mine = 0;
                    for (int i = 0; i < s1 - s0; ++i) mine += my_sum[i];
                }
                return true;
            };
            float from = low_bound, to = INFINITY;
            if (weighed && !cut_some && from > -FLT_MAX) {
                narrow(from, to, true);
                if (settle(from, to)) return;
                from = low_bound;
                to = INFINITY;
            }
            for (int round = 0; round < 3; ++round) {
                narrow(from, to, false);
                if (settle(from, to)) return;
            }
            // the whole row by bisection: more equal logits than the list holds, or a border below the bound
            masses = false;
            uint32_t lo = max(dr_ord(-INFINITY) + 1, dr_ord(low_bound)), hi = dr_ord(m) + 1;
            auto of = [&](uint32_t v) {
                if (weighed) return sum_all(span_masses(dr_value(v), kept_weights(old, dr_value(v), 0)));
                u64 n = 0;
                const float least = dr_value(v);
                stream(reaching(least), false, [&](const float (&x)[8], int seg) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) n += x[i] >= least && dr_kept(old, x[i], lp_index<T>(mis, seg, i)) ? 1 : 0;
                }, [](int) {});
                return sum_all(dr_warp_sum(n));
            };
            if (of(lo) < need) return;
            while (hi - lo > 1) {
                const uint32_t mid = lo + (hi - lo) / 2;
                if (of(mid) >= need) lo = mid;
                else hi = mid;
            }
            const float v = dr_value(lo);
            u64 rest = need - (v < m ? of(lo + 1) : 0);
            if (weighed) {
                u64 vv[2];
                int sh[2];
                dr_weight2(E, v, v, vv, sh);
                const u64 w1 = vv[0] >> sh[0];
                rest = (rest + w1 - 1) / w1;
            }
            // the id of the last of the equal tokens that stay
            auto tie = [&](const float (&x)[8], int seg, u64 (&wt8)[8]) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int d = lp_index<T>(mis, seg, i);
                    wt8[i] = x[i] == v && d >= 0 && d < V && dr_kept(old, v, d) ? 1 : 0;
                }
            };
            const u64 ties = span_masses(v, tie);
            locate(ties, tie, [&](u64) { return rest - 1; }, [&](int d, float, u64) {
                for (int i = 0; i < C; ++i) *cl.map_shared_rank(&sm.ci, i) = d;
            });
            cluster_sync();
            cut = DrCut{v, sm.ci};
        };
        if (K > 0) {
            // (at least K tokens are finite, or every finite one stays)
            u64 n = 0;
            stream(reaching(-FLT_MAX), false, [&](const float (&x)[8], int) {
#pragma unroll
                for (int i = 0; i < 8; ++i) n += x[i] >= -FLT_MAX ? 1 : 0;
            }, [](int) {});
            if (sum_all(dr_warp_sum(n)) > (u64)K) select((u64)K, false, 0);
            if (nucleus) {
                S = sum_all(span_masses(fmaxf(cut.v, -FLT_MAX), kept_weights(cut, -FLT_MAX, 0)));
                p_target = max(dr_part(top_p, S, true), 1ull);
                low_bound = fmaxf(low_bound, cut.v);
            }
        }
        if (nucleus) select(p_target, true, S);
        const auto f = kept_weights(cut, -FLT_MAX, w_min);
        if (!masses || w_min > 1) mine = span_masses(fmaxf(cut.v, -FLT_MAX), f);
        S_kept = locate(mine, f, [&](u64 total) { return dr_part(u, total, false); }, finish);
    }
    if (!probs) {
        cluster_sync();                                // (a CTA's shared memory stays while others read it)
        return;
    }

    // -------- the distribution
    const float inv = 1.f / (float)S_kept;
    const float least = fmaxf(cut.v, -FLT_MAX);
    const u64 w_some = max(w_min, 1ull);
#pragma unroll 1
    for (int s = s0; s < s1; ++s) {
        const bool any = __any_sync(0xffffffffu, my_max[(s - s0) * 32 + lane] >= least);
#pragma unroll 1
        for (int g = 0; g < kDrSegs; ++g) {
            uint4 p[NP];
            float x[8], y[8];
            if (any) {
                load_raw(s * kDrSegs + g, p);
                unpack(p, x);
            }
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                y[i] = y[i + 1] = 0.f;
                if (!any) continue;
                u64 v[2];
                int sh[2];
                dr_weight2(E, x[i], x[i + 1], v, sh);
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    if (x[i + j] >= least && dr_kept(cut, x[i + j], lp_index<T>(mis, s * kDrSegs + g, i + j)) && v[j] >> sh[j] >= w_some)
                        y[i + j] = (float)v[j] * __uint_as_float((uint32_t)(127 - sh[j]) << 23) * inv;
            }
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const int d = lp_index<T>(mis, s * kDrSegs + g, k * VE);
                if (a.p_vec && d >= 0 && d + VE <= V) {
#pragma unroll
                    for (int i = 0; i < VE; i += 4)
                        *reinterpret_cast<float4*>(probs + d + i) = make_float4(y[k * VE + i], y[k * VE + i + 1], y[k * VE + i + 2], y[k * VE + i + 3]);
                } else {
#pragma unroll
                    for (int i = 0; i < VE; ++i)
                        if (d + i >= 0 && d + i < V) probs[d + i] = y[k * VE + i];
                }
            }
        }
    }
    cluster_sync();
}

static size_t dr_smem(int per, size_t elem) {
    return (size_t)(kDrList + kDrWarps * kDrStage + kDrSteps) * 8 + (size_t)kDrWarps * kDrRing * (elem / 2) * 512 +
           (size_t)kDrWarps * per * (8 + 4 + 32 * 4);
}

}  // namespace spec

using namespace spec;

extern "C" int spec_sample_logits(const void* logits, int32_t dtype, int64_t lg_stride, int32_t rows, int32_t vocab,
                                  const float* u, const spec_sample_config* cfg, int32_t* tokens, float* logprob,
                                  float* probs, int64_t p_stride, void* stream) {
    if (!cfg) return set_error(SPEC_ERR_ARG, "spec_sample_logits: null pointer");
    if (dtype != SPEC_DTYPE_F32 && dtype != SPEC_DTYPE_BF16) return set_error(SPEC_ERR_ARG, "spec_sample_logits: unknown dtype");
    if (rows < 0 || vocab < 1 || lg_stride < vocab || (probs && p_stride < vocab)) return set_error(SPEC_ERR_ARG, "spec_sample_logits: bad sizes");
    if (vocab > kDrMaxVocab) return set_error(SPEC_ERR_UNSUPPORTED, "spec_sample_logits: vocab must be at most 1048576");
    if (rows > INT_MAX / kDrMaxCtas) return set_error(SPEC_ERR_UNSUPPORTED, "spec_sample_logits: too many rows");
    const spec_sample_config& c = *cfg;
    if (!c.temperatures && !(c.temperature == 0.f || (c.temperature >= 1e-30f && c.temperature <= 1e30f)))
        return set_error(SPEC_ERR_ARG, "spec_sample_logits: temperature must be 0 or in [1e-30, 1e30]");
    if (!c.top_ks && c.top_k < 0) return set_error(SPEC_ERR_ARG, "spec_sample_logits: top_k must not be negative");
    if (!c.top_ps && !(c.top_p >= 0.f)) return set_error(SPEC_ERR_ARG, "spec_sample_logits: top_p must not be negative");
    if (!c.min_ps && !(c.min_p >= 0.f && c.min_p <= 1.f)) return set_error(SPEC_ERR_ARG, "spec_sample_logits: min_p must be in [0, 1]");
    if (rows == 0) return SPEC_OK;
    if (!logits || !u || !tokens) return set_error(SPEC_ERR_ARG, "spec_sample_logits: null pointer");
    const size_t elem = dtype == SPEC_DTYPE_BF16 ? 2 : 4;
    if (reinterpret_cast<uintptr_t>(logits) % elem) return set_error(SPEC_ERR_ARG, "spec_sample_logits: logits not aligned to their type");
    int dev = 0, sms = 0;
    SPEC_TRY(check_cuda(cudaGetDevice(&dev), "cudaGetDevice"));
    SPEC_TRY(check_cuda(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev), "attr"));
    DrawArgs a{};
    a.x = logits;
    a.stride = lg_stride;
    a.V = vocab;
    a.u = u;
    a.T = c.temperature;
    a.p = c.top_p;
    a.mp = c.min_p;
    a.k = c.top_k;
    a.Ts = c.temperatures;
    a.ps = c.top_ps;
    a.mps = c.min_ps;
    a.ks = c.top_ks;
    a.tok = tokens;
    a.lp = logprob;
    a.probs = probs;
    a.p_stride = p_stride;
    // a row's pieces start 16 bytes apart in either array where both rows do
    a.p_vec = probs && reinterpret_cast<uintptr_t>(probs) % 16 == 0 && p_stride % 4 == 0 && reinterpret_cast<uintptr_t>(logits) % 16 == 0 &&
              lg_stride % (16 / (int64_t)elem) == 0;
    a.q = 61;
    while ((1ll << (62 - a.q)) < vocab) --a.q;
    static const struct Table {
        unsigned long long coarse[32], fine[64];
        Table() {
            for (int j = 0; j < 32; ++j) coarse[j] = (unsigned long long)std::ldexp(std::exp2((long double)j / 32), 62);
            for (int j = 0; j < 64; ++j) fine[j] = (unsigned long long)std::ldexp(std::exp2((long double)j / kDrSteps), 63);
        }
    } table;
    std::copy(table.coarse, table.coarse + 32, a.coarse);
    std::copy(table.fine, table.fine + 64, a.fine);
    const int n_span = (vocab + 7 + kDrSpan - 1) / kDrSpan;
    int C = 1;
    while (C < kDrMaxCtas && ((long long)vocab > (long long)C * kDrCtaVocab || ((long long)rows * C < kDrCtasWanted * sms && n_span > C * kDrWarps))) C *= 2;
    a.per = (n_span + C * kDrWarps - 1) / (C * kDrWarps);
    const size_t smem = dr_smem(a.per, elem);
    const bool half = dtype == SPEC_DTYPE_BF16;
    void (*f)(DrawArgs) = half ? draw_kernel<__nv_bfloat16> : draw_kernel<float>;
    static std::atomic<unsigned long long> set[2] = {};        // devices where a kernel may take more than 48 KB
    const unsigned long long bit = 1ull << (dev & 63);
    if (smem > 48 * 1024 && !(set[half].load() & bit)) {
        // (the most that any call takes)
        constexpr int most_per = (kDrCtaVocab / kDrSpan + 1 + kDrWarps) / kDrWarps;
        SPEC_TRY(check_cuda(cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)dr_smem(most_per, elem)), "spec_sample_logits attribute"));
        set[half].fetch_or(bit);
    }
    cudaLaunchConfig_t cfg_l = {};
    cfg_l.gridDim = dim3((unsigned)(rows * C));
    cfg_l.blockDim = dim3(kDrThreads);
    cfg_l.dynamicSmemBytes = smem;
    cfg_l.stream = (cudaStream_t)stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = C;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg_l.attrs = at;
    cfg_l.numAttrs = C > 1 ? 2 : 1;
    return check_cuda(cudaLaunchKernelEx(&cfg_l, f, a), "spec_sample_logits launch");
}
