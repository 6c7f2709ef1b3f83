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
// the first in two floats: 30, and 622 us a call for 512 rows of 131072 to their nuclei.)
//
// A row is taken by a cluster of 1 to 8 CTAs, each warp on a contiguous run of spans
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
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>
#include <cooperative_groups.h>

#include "logits.cuh"

namespace cg = cooperative_groups;

namespace spec {

constexpr int kDrThreads = 256;
constexpr int kDrCtasWanted = 3;                       // CTAs an SM up to which rows are cut into more of them
constexpr int kDrWarps = kDrThreads / 32;
constexpr int kDrMaxCtas = 8;
constexpr int kDrSegs = 4;                             // segments of a span
constexpr int kDrSpan = kDrSegs * kLpSeg;
constexpr int kDrEach = 8;                             // listed tokens a thread
constexpr int kDrList = kDrEach * kDrThreads;
constexpr int kDrSpanUnit = 51;                        // 1024 weights in units of 2^-51 fit 64 bits, and so does a listed token's
constexpr int kDrListUnit = 50;
constexpr int kDrBins = 2048;                          // steps of a histogram; it lies where the list does
static_assert(kDrBins * 4 <= kDrList * 8, "histogram");
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
    u64 redc[2][kDrMaxCtas];
    u64 part[kDrMaxCtas * kDrWarps];                   // every warp's sum, in every CTA; a barrier lies between its uses
    u64 mass[kDrMaxCtas * kDrWarps];                   // every warp's share of the row's mass
    float wmax[kDrWarps], wlow[kDrWarps];
    float cmax[kDrMaxCtas], clow[kDrMaxCtas];
    int cbad[kDrMaxCtas], wbad[kDrWarps];
    u64 S;                                             // the first CTA's results for the others
    uint32_t cv; int ci, holds;
    int bin_lo, bin_hi;
};

// A weight's arithmetic.
constexpr int kDrSteps = 2048;                         // of the table, an octave
struct DrExp {
    float b, ch, cl;                                   // b: 0, or the maximum where c x has too many digits
    float most;                                        // -2048 t of a logit without a weight
    int N, q;
    const u64* table;                                  // 2^(62 + j / 2048), in shared memory
    // weights relative to 2^N for logits up to `top`
    SPEC_DEV void refer_to(float top) { refer_to_n((int)ceilf((top - b) * ch * (1.f / kDrSteps))); }
    SPEC_DEV void refer_to_n(int n) {
        N = n;
        most = (float)(-kDrSteps * (N - q - 4));       // well below 2^-q
    }
};
// c x as the arithmetic takes it: beyond, logits are taken relative to the maximum (exactly: those near it lie within
// a factor of two of it)
constexpr float kDrDigits = 2097152.f;

// ln 2 / 2048 and half its square, by 2^36
constexpr double kDrL = 0.69314718055994530942 / kDrSteps;
constexpr float kDrL1 = (float)(kDrL * 68719476736.0), kDrL2 = (float)(kDrL * kDrL / 2 * 68719476736.0);

SPEC_DEV float2 both(float x) { return make_float2(x, x); }

// weights of two logits: w = v * 2^-n with v in units of 2^-62
SPEC_DEV void dr_weight2(const DrExp& E, float x0, float x1, u64 (&v)[2], int (&n)[2]) {
    const float2 neg = both(-1.f);
    const float2 d = add2(make_float2(x0, x1), both(-E.b));
    // p + e = 2048 t; p leaves its nearest integer.  (Where p is cut short, e, NaN for a masked logit, is
    // anything: what comes of it is shifted out.)
    float2 np = mul2(d, both(-E.ch));
    float2 e = fma2(d, both(E.ch), np);
    e = fma2(d, both(E.cl), e);
    np = make_float2(fminf(np.x, E.most), fminf(np.y, E.most));
    const float2 magic = both(12582912.f);
    const float2 k = fma2(np, neg, magic), nk = fma2(k, neg, magic), r = fma2(np, neg, nk);
    // 2^((r + e) / 2048) - 1 in units of 2^-36: off by 2^-36 of a weight, its f32 sums; the table's value to 26 bits
    // is enough for the product
    const float2 s = add2(r, e), f = mul2(fma2(both(kDrL2), s, both(kDrL1)), s);
    const float kf[2] = {k.x, k.y}, ff[2] = {f.x, f.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int ki = __float_as_int(kf[i]) - 0x4B400000;
        const u64 T = E.table[ki & (kDrSteps - 1)];
        v[i] = T + (u64)((long long)((int)(T >> 32) >> 4) * __float2int_rn(ff[i]));
        n[i] = E.N - (ki >> 11);
    }
}
// v * 2^-n in units of 2^-q, cut off (shifts of 64 and more give zero)
SPEC_DEV u64 dr_units(const DrExp& E, u64 v, int n) {
    u64 r;
    asm("shr.u64 %0, %1, %2;" : "=l"(r) : "l"(v), "r"(62 - E.q + n));
    return r;
}
SPEC_DEV void dr_weights(const DrExp& E, const float (&x)[8], u64 (&w)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        u64 v[2];
        int n[2];
        dr_weight2(E, x[i], x[i + 1], v, n);
        w[i] = dr_units(E, v[0], n[0]);
        w[i + 1] = dr_units(E, v[1], n[1]);
    }
}
// a mass in units of 2^-by, to the nearest
SPEC_DEV u64 dr_rescale(u64 w, int by) { return by <= 0 ? w << -by : (by > 63 ? 0 : ((w >> (by - 1)) + 1) >> 1); }

// a kept logit: above the cut's value, or equal to it with an id not above the cut's
struct DrCut { uint32_t v; int id; };
SPEC_DEV bool dr_kept(const DrCut& c, uint32_t o, int id) { return o > c.v || (o == c.v && id <= c.id); }

template <typename T>
__global__ void __launch_bounds__(kDrThreads, 2)
draw_kernel(const __grid_constant__ DrawArgs a) {
    pdl_wait();
    pdl_trigger();
    constexpr int VE = 16 / sizeof(T), NP = 8 / VE;
    __shared__ DrSmem sm;
    extern __shared__ __align__(16) u64 dyn[];
    u64* list = dyn;                                   // [kDrList] (value's order, id) by id; the first CTA's
    uint32_t* hist = reinterpret_cast<uint32_t*>(dyn); // [kDrBins] while there is no list
    u64* span_sum = dyn + kDrList;                     // [kDrWarps][per] masses, relative to 2^N
    int* span_n = reinterpret_cast<int*>(span_sum + kDrWarps * a.per);         // [kDrWarps][per] ... to 2^span_n at first
    float* lane_max = reinterpret_cast<float*>(span_n + kDrWarps * a.per);     // [kDrWarps][per][32]
    u64* table = reinterpret_cast<u64*>(lane_max + kDrWarps * a.per * 32);     // [kDrSteps]
    cg::cluster_group cl = cg::this_cluster();
    const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
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
    E.table = table;
    for (int i = t; i < kDrSteps; i += kDrThreads) table[i] = __umul64hi(a.coarse[i >> 6], a.fine[i & 63]) << 1;
    __syncthreads();

    // a span's logits, 32 a lane
    auto load_span = [&](int s, float (&x)[kDrSegs][8]) {
        if (s * kDrSpan >= mis && (s + 1) * kDrSpan - mis <= V) {
            uint4 p[kDrSegs][NP];
            const T* at = row + (s * kDrSpan - mis + lane * VE);
#pragma unroll
            for (int g = 0; g < kDrSegs; ++g)
#pragma unroll
                for (int i = 0; i < NP; ++i) p[g][i] = __ldg(reinterpret_cast<const uint4*>(at + g * kLpSeg + i * 32 * VE));
#pragma unroll
            for (int g = 0; g < kDrSegs; ++g)
#pragma unroll
                for (int i = 0; i < NP; ++i) lp_unpack<T>(p[g][i], &x[g][i * VE]);
        } else {
#pragma unroll
            for (int g = 0; g < kDrSegs; ++g) lp_load(row, V, mis, s * kDrSegs + g, x[g]);
        }
    };
    // a span's logits, 8 a lane at a time: f(logits, segment), the next ones on their way
    auto walk_span = [&](int s, auto f) {
        float x[8];
        if (s * kDrSpan >= mis && (s + 1) * kDrSpan - mis <= V) {
            uint4 nx[NP];
            const T* at = row + (s * kDrSpan - mis + lane * VE);
#pragma unroll
            for (int i = 0; i < NP; ++i) nx[i] = __ldg(reinterpret_cast<const uint4*>(at + i * 32 * VE));
#pragma unroll 1
            for (int g = 0; g < kDrSegs; ++g) {
#pragma unroll
                for (int i = 0; i < NP; ++i) lp_unpack<T>(nx[i], &x[i * VE]);
                at += kLpSeg;
                if (g + 1 < kDrSegs)
#pragma unroll
                    for (int i = 0; i < NP; ++i) nx[i] = __ldg(reinterpret_cast<const uint4*>(at + i * 32 * VE));
                f(x, s * kDrSegs + g);
            }
        } else {
#pragma unroll 1
            for (int g = 0; g < kDrSegs; ++g) {
                lp_load(row, V, mis, s * kDrSegs + g, x);
                f(x, s * kDrSegs + g);
            }
        }
    };
    // this warp's part of an array by span (a span's owner is warp s / per of the cluster)
    u64* my_sum = span_sum + w * a.per;
    int* my_n = span_n + w * a.per;
    float* my_max = lane_max + w * a.per * 32;

    // -------- the maximum, every lane's maxima, the spans' masses, and whether the row has a distribution
    float mx = -INFINITY;
    bool bad = false;
    if (whole && settings) {
        for (int s = s0; s < s1; ++s) {
            float lm = -INFINITY;
            u64 sum = 0;
            int N = INT_MIN;
            walk_span(s, [&](const float (&x)[8], int) {
                float gm = x[0];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    bad |= !(x[i] <= FLT_MAX);         // NaN or +inf
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
            });
            my_max[(s - s0) * 32 + lane] = lm;
            mx = fmaxf(mx, lm);
            sum = dr_warp_sum(sum);
            if (lane == 0) {
                my_sum[s - s0] = sum;
                my_n[s - s0] = N;
            }
        }
    } else {
        for (int s = s0; s < s1; ++s) {
            float x[kDrSegs][8], g4[kDrSegs];
            load_span(s, x);
#pragma unroll
            for (int g = 0; g < kDrSegs; ++g) {
                g4[g] = x[g][0];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    bad |= !(x[g][i] <= FLT_MAX);
                    g4[g] = fmaxf(g4[g], x[g][i]);
                }
            }
            const float g = fmaxf(fmaxf(g4[0], g4[1]), fmaxf(g4[2], g4[3]));
            my_max[(s - s0) * 32 + lane] = g;
            mx = fmaxf(mx, g);
        }
    }
    mx = warp_redux_max(mx);
    bad = __any_sync(0xffffffffu, bad);
    __syncwarp();
    // This warp's share of the bound for top-k: of the warps with a full run of whole spans (none: no bound) each gives the value of
    // (about) its r-th largest lane maximum; the least of these has r tokens a warp that are not below it.
    float low = INFINITY;
    const int full = (V + mis) / kDrSpan / a.per, r_low = full > 0 ? (K + full - 1) / full : 0;
    if (K > 0 && gw < full) {
        low = mx;
        if (r_low > 32 * a.per) {
            low = -INFINITY;
        } else if (r_low > 1) {
            uint32_t lo = 0, hi = dr_ord(mx);          // at least r not below lo; hi: fewer (or not looked at)
            while (hi - lo > 1) {
                const uint32_t mid = lo + (hi - lo) / 2;
                const float v = dr_value(mid);
                int n = 0;
                for (int i = 0; i < a.per; ++i) n += my_max[i * 32 + lane] >= v;
                n = __reduce_add_sync(0xffffffffu, n);
                if (n >= r_low) {
                    lo = mid;
                    if (n <= r_low + r_low / 8) break;
                } else {
                    hi = mid;
                }
            }
            low = dr_value(lo);
            if (!(low >= -FLT_MAX)) low = -INFINITY;
        }
    }
    if (lane == 0) { sm.wmax[w] = mx; sm.wlow[w] = low; sm.wbad[w] = bad; }
    __syncthreads();
    if (C > 1) cluster_wait();
    if (w == 0) {
        float m = lane < kDrWarps ? sm.wmax[lane] : -INFINITY, l = lane < kDrWarps ? sm.wlow[lane] : INFINITY;
        const bool b = __any_sync(0xffffffffu, lane < kDrWarps && sm.wbad[lane]);
        m = warp_redux_max(m);
        l = -warp_redux_max(-l);
        everywhere(&sm.cmax[rank], m);
        everywhere(&sm.clow[rank], l);
        everywhere(&sm.cbad[rank], (int)b);
    }
    cluster_sync();
    float m = -INFINITY, k_low = INFINITY;
    bad = false;
    for (int i = 0; i < C; ++i) {
        m = fmaxf(m, sm.cmax[i]);
        k_low = fminf(k_low, sm.clow[i]);
        bad |= sm.cbad[i] != 0;
    }
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
        int n[2];
        dr_weight2(E, m, m, v, n);
        one = dr_units(E, v[0], n[0]);
        w_min = dr_part(min_p, one, true);
    };
    const uint32_t o_max = dr_ord(m), o_inf = dr_ord(-INFINITY);

    // sums over the CTA, or over the cluster (the first CTA takes more of the former: each kind has its own turns)
    int par = 0, cpar = 0;
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
    auto sum_all = [&](u64 v) {
        u64 s = sum_cta(v);
        if (C > 1) {
            if (w == 0) everywhere(&sm.redc[cpar][rank], s);
            cl.sync();
            s = 0;
            for (int i = 0; i < C; ++i) s += sm.redc[cpar][i];
            cpar ^= 1;
        }
        return s;
    };
    // every segment of this warp's spans that hold a logit not below `least`: f(logits, segment), then done(span) (also
    // for the others)
    auto each_segment = [&](float least, auto f, auto done) {
        for (int s = s0; s < s1; ++s) {
            if (__any_sync(0xffffffffu, my_max[(s - s0) * 32 + lane] >= least)) walk_span(s, f);
            done(s);
        }
    };
    // the same for whole spans: f(logits, span)
    auto each_span = [&](float least, auto f) {
        for (int s = s0; s < s1; ++s) {
            if (!__any_sync(0xffffffffu, my_max[(s - s0) * 32 + lane] >= least)) continue;
            float x[kDrSegs][8];
            load_span(s, x);
            f(x, s);
        }
    };
    // weights of a segment by f(logits, segment, weights): every span's sum in my_sum, the warp's returned
    auto span_masses = [&](float least, auto f) {
        u64 sum = 0, mine = 0;
        each_segment(least, [&](const float (&x)[8], int seg) {
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
    auto kept_weights = [&](const DrCut& cut, uint32_t least, u64 w_least) {
        const float at_least = dr_value(least), cut_v = dr_value(cut.v);
        const int cut_id = cut.id;
        return [&, at_least, cut_v, cut_id, w_least](const float (&x)[8], int seg, u64 (&wt)[8]) {
            dr_weights(E, x, wt);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (!(x[i] >= at_least) || wt[i] < w_least || !(x[i] > cut_v || (x[i] == cut_v && lp_index<T>(mis, seg, i) <= cut_id))) wt[i] = 0;
        };
    };
    // the sum of the weights of the kept logits not below `least`
    auto row_mass = [&](uint32_t least, const DrCut& cut) {
        const u64 mine = span_masses(dr_value(least), kept_weights(cut, least, 0));
        return sum_all(lane == 0 ? mine : 0);
    };
    auto row_count = [&](uint32_t least, const DrCut&) {
        u64 n = 0;
        each_span(dr_value(least), [&](const float (&x)[kDrSegs][8], int) {
#pragma unroll
            for (int g = 0; g < kDrSegs; ++g)
#pragma unroll
                for (int i = 0; i < 8; ++i) n += dr_ord(x[g][i]) >= least ? 1 : 0;
        });
        return sum_all(n);
    };
    // With every span's sum in my_sum, `mine` a warp's: the token by id, weighed by f, at which the sum passes the
    // target; found(id, logit, total) is called by one thread of the cluster.
    auto locate = [&](u64 mine, auto f, auto target_of, auto found) {
        everywhere(&sm.part[gw], mine);
        cluster_sync();
        u64 total = 0, before = 0;
        for (int i = 0; i < C * kDrWarps; ++i) {
            if (i == gw) before = total;
            total += sm.part[i];
        }
        const u64 target = target_of(total);
        if (before <= target && target < before + mine) {
            u64 left = target - before;
            int s = s0;
            while (s + 1 < s1 && left >= my_sum[s - s0]) left -= my_sum[s++ - s0];
            // (the first pass' masses are rounded on their way to a common unit: a few of 2^-45)
            bool done = false, ones = false;
            {
                u64 exact = 0;
#pragma unroll 1
                for (int g = 0; g < kDrSegs; ++g) {
                    float x[8];
                    u64 wt[8];
                    lp_load(row, V, mis, s * kDrSegs + g, x);
                    f(x, s * kDrSegs + g, wt);
#pragma unroll
                    for (int i = 0; i < 8; ++i) exact += wt[i];
                }
                exact = dr_warp_sum(exact);
                ones = exact == 0;
                left = ones ? 0 : min(left, exact - 1);
            }
#pragma unroll 1
            for (int g = 0; g < kDrSegs && !done; ++g) {
                float x[8];
                u64 wt[8];
                lp_load(row, V, mis, s * kDrSegs + g, x);
                f(x, s * kDrSegs + g, wt);
                if (ones)
#pragma unroll
                    for (int i = 0; i < 8; ++i) wt[i] = x[i] >= -FLT_MAX ? 1 : 0;
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    u64 sum = 0, all;
#pragma unroll
                    for (int i = 0; i < VE; ++i) sum += wt[p * VE + i];
                    const u64 pre = dr_warp_before(sum, all);
                    if (!done && left < all) {
                        if (pre <= left && left < pre + sum) {
                            u64 at = pre;
                            bool hit = false;
#pragma unroll
                            for (int i = 0; i < VE; ++i) {
                                at += wt[p * VE + i];
                                if (!hit && left < at) {
                                    hit = true;
                                    found(lp_index<T>(mis, s * kDrSegs + g, p * VE + i), x[p * VE + i], total);
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
    // Tokens for which in(logit, segment, element) holds, by id, into the first CTA's list; their number, and
    // whether the list holds them.
    auto make_list = [&](float least, int& n_list, auto in) {
        int n = 0;
        each_span(least, [&](const float (&x)[kDrSegs][8], int s) {
#pragma unroll
            for (int g = 0; g < kDrSegs; ++g)
#pragma unroll
                for (int i = 0; i < 8; ++i) n += in(x[g][i], s * kDrSegs + g, i) ? 1 : 0;
        });
        n = __reduce_add_sync(0xffffffffu, n);
        everywhere(&sm.part[gw], (u64)n);
        cluster_sync();
        int before = 0;
        n_list = 0;
        for (int i = 0; i < C * kDrWarps; ++i) {
            if (i == gw) before = n_list;
            n_list += (int)sm.part[i];
        }
        if (n_list <= kDrList && n > 0) {
            u64* first = cl.map_shared_rank(list, 0);
            each_span(least, [&](const float (&x)[kDrSegs][8], int s) {
#pragma unroll
                for (int g = 0; g < kDrSegs; ++g)
#pragma unroll
                    for (int p = 0; p < NP; ++p) {
                        uint32_t mine = 0;
#pragma unroll
                        for (int i = 0; i < VE; ++i) mine |= in(x[g][p * VE + i], s * kDrSegs + g, p * VE + i) ? 1u << i : 0u;
                        if (!__any_sync(0xffffffffu, mine != 0)) continue;
                        const int c = __popc(mine);
                        int upto = c;
#pragma unroll
                        for (int o = 1; o < 32; o <<= 1) {
                            const int v = __shfl_up_sync(0xffffffffu, upto, o);
                            if (lane >= o) upto += v;
                        }
                        int at = before + upto - c;
#pragma unroll
                        for (int i = 0; i < VE; ++i)
                            if ((mine >> i) & 1u)
                                first[at++] = (u64)dr_ord(x[g][p * VE + i]) << 32 | (uint32_t)lp_index<T>(mis, s * kDrSegs + g, p * VE + i);
                        before += __shfl_sync(0xffffffffu, upto, 31);
                    }
            });
        }
        cluster_sync();
        return n_list <= kDrList;
    };

    // -------- a bound below which nothing is kept
    const float slack = 1e-3f;
    float low_bound = -FLT_MAX;
    u64 S = 0, p_target = 0, mine_all = 0;             // the row's mass, this warp's part of it
    auto below = [&](float z) {                        // safely below m + T z
        const float v = m + T_ * (z - slack);
        return fmaxf(v - fabsf(v) * 1e-6f, -FLT_MAX);
    };
    if (whole) {
        // the warps' masses in units of 2^-46 (33 spans at most), their sum S 2^46 in 128 bits: what unit the row's have
        constexpr int kWarpUnit = 46;
        const DrCut all{o_inf, -1};
        set_unit(kWarpUnit);
        if (far) {
            mine_all = span_masses(-FLT_MAX, kept_weights(all, o_inf + 1, 0));
        } else {
            for (int i = 0; i < s1 - s0; ++i) mine_all += my_n[i] == INT_MIN ? 0 : dr_rescale(my_sum[i], E.N - my_n[i] + kDrSpanUnit - kWarpUnit);
        }
        everywhere(&sm.mass[gw], mine_all);
        cluster_sync();
        unsigned __int128 sum = 0;
        for (int i = 0; i < C * kDrWarps; ++i) sum += sm.mass[i];
        const int bits = (u64)(sum >> 64) ? 128 - __clzll((u64)(sum >> 64)) : 64 - __clzll((u64)sum);   // S < 2^(bits - 46)
        const int q = min(kDrListUnit, 62 + kWarpUnit - bits);
        set_unit(q);
        S = q >= kWarpUnit ? (u64)sum << (q - kWarpUnit) : (u64)(sum >> (kWarpUnit - q));
        if (far) {
            for (int i = lane; i < s1 - s0; i += 32) my_sum[i] = dr_rescale(my_sum[i], kWarpUnit - q);
        } else {
            for (int i = lane; i < s1 - s0; i += 32) my_sum[i] = my_n[i] == INT_MIN ? 0 : dr_rescale(my_sum[i], E.N - my_n[i] + kDrSpanUnit - q);
        }
        __syncwarp();
        mine_all = 0;
        for (int i = 0; i < s1 - s0; ++i) mine_all += my_sum[i];
    } else {
        set_unit(kDrListUnit);
    }
    bool listed = true;
    if (K == 1) {
        low_bound = m;
    } else if (K > 0) {
        low_bound = full > 0 ? fmaxf(k_low, -FLT_MAX) : -FLT_MAX;
    } else if (nucleus) {
        p_target = max(dr_part(top_p, S, true), 1ull);
        low_bound = below(logf(fmaxf((1.f - top_p) * ((float)S / (float)one) / (float)V, 1e-30f)));
    } else {
        listed = min_p > 0.f;
    }
    // (min_p leaves out of top-k's and the nucleus' tokens, whose number and mass count them)
    if (min_p > 0.f && K == 0) low_bound = fmaxf(low_bound, below(logf(min_p)));
    int n_list = 0;
    if (listed) listed = make_list(low_bound, n_list, [&](float x, int, int) { return x >= low_bound; });

    DrCut cut{o_inf, -1};
    u64 S_kept = 0;
    // -------- the first CTA's threads with `each` neighbours of the list
    uint32_t o[kDrEach];
    int id[kDrEach];
    u64 wt[kDrEach];
    float x[kDrEach];
    auto take_list = [&](int n) {
        const int each = (n + kDrThreads - 1) / kDrThreads;
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
    // the first `n` by id of the tokens equal to v, and those above it, stay
    auto cut_at = [&](uint32_t v, u64 n) {
        u64 mine = 0;
#pragma unroll
        for (int e = 0; e < kDrEach; ++e) mine += o[e] == v ? 1 : 0;
        u64 all, at = dr_warp_before(mine, all);
        if (lane == 0) sm.red[par][w] = all;
        __syncthreads();
        for (int i = 0; i < w; ++i) at += sm.red[par][i];
        par ^= 1;
#pragma unroll
        for (int e = 0; e < kDrEach; ++e) {
            if (o[e] == v && at++ >= n) o[e] = 0;
            if (o[e] < v) o[e] = 0;
            if (o[e] == 0) wt[e] = 0;
        }
    };
    auto count = [&](int) -> u64 { return 1; };
    auto mass = [&](int e) -> u64 { return wt[e]; };
    auto above = [&](uint32_t v, auto of) {
        u64 s = 0;
#pragma unroll
        for (int e = 0; e < kDrEach; ++e) s += o[e] > v ? of(e) : 0;
        return sum_cta(s);
    };
    // the tokens of the list that come first, by decreasing logit, until they weigh (or count) `need`, which all of
    // them do
    auto cut_to = [&](u64 need, uint32_t from, bool weighed, auto of) {
        uint32_t lo = max(o_inf + 1, from), hi = o_max + 1;   // largest lo whose tokens not below it reach `need`
        while (hi - lo > 1) {
            const uint32_t mid = lo + (hi - lo) / 2;
            u64 s = 0;
#pragma unroll
            for (int e = 0; e < kDrEach; ++e) s += o[e] >= mid ? of(e) : 0;
            if (sum_cta(s) >= need) lo = mid;
            else hi = mid;
        }
        u64 rest = need - above(lo, of);
        if (weighed) {
            // tokens of one value have one weight
            u64 w1 = 0;
#pragma unroll
            for (int e = 0; e < kDrEach; ++e)
                if (o[e] == lo) w1 = wt[e];
            const u64 holders = sum_cta(w1 ? 1 : 0);
            w1 = sum_cta(w1) / holders;
            rest = (rest + w1 - 1) / w1;
        }
        cut_at(lo, rest);
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
            take_list(n_list);
            const uint32_t from = dr_ord(low_bound);
            if (n_list <= kDrThreads) {
                // one token a thread: its place is the number of tokens that rank before it
                const uint32_t mine = o[0];
                int place = 0;
                for (int i = 0; i < n_list; ++i) {
                    const uint32_t other = (uint32_t)(list[i] >> 32);
                    place += other > mine || (other == mine && i < t) ? 1 : 0;
                }
                if (K > 0 && place >= K) o[0] = 0;
                if (o[0] == 0) wt[0] = 0;
                if (nucleus) {
                    // masses by place, and what comes before each
                    u64* by_place = list + kDrThreads;
                    if (t < n_list) by_place[place] = wt[0];
                    __syncthreads();
                    u64 all, at = dr_warp_before(t < n_list ? by_place[t] : 0, all);
                    if (lane == 0) sm.red[par][w] = all;
                    __syncthreads();
                    all = 0;
                    for (int i = 0; i < kDrWarps; ++i) {
                        if (i == w) at += all;
                        all += sm.red[par][i];
                    }
                    par ^= 1;
                    by_place[kDrThreads + t] = at;
                    __syncthreads();
                    const u64 target = K > 0 ? max(dr_part(top_p, all, true), 1ull) : p_target;
                    if (t < n_list && by_place[kDrThreads + place] >= target) o[0] = 0;
                    if (o[0] == 0) wt[0] = 0;
                }
            } else {
                if (K > 0 && n_list > K) cut_to((u64)K, from, false, count);
                if (nucleus) {
                    const u64 all = above(0, mass), target = K > 0 ? max(dr_part(top_p, all, true), 1ull) : p_target;
                    if (all >= target) cut_to(target, from, true, mass);
                }
            }
            u64 mine = 0;
#pragma unroll
            for (int e = 0; e < kDrEach; ++e) {
                if (wt[e] < w_min) wt[e] = 0;
                mine += wt[e];
            }
            u64 all, at = dr_warp_before(mine, all);
            if (lane == 0) sm.red[par][w] = all;
            __syncthreads();
            u64 sum = 0;
            for (int i = 0; i < kDrWarps; ++i) {
                if (i == w) at += sum;
                sum += sm.red[par][i];
            }
            par ^= 1;
            const u64 target = dr_part(u, sum, false);
            if (at <= target && target < at + mine) {
                bool hit = false;
#pragma unroll
                for (int e = 0; e < kDrEach; ++e) {
                    at += wt[e];
                    if (!hit && target < at) {
                        hit = true;
                        finish(id[e], x[e], sum);
                    }
                }
            }
            if (probs) {
                const u64 least = least_key();
                if (w == 0) {
                    everywhere(&sm.S, sum);
                    everywhere(&sm.cv, (uint32_t)(least >> 32));
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
            auto kept = [&](float v, int seg, int i) { return dr_kept(old, dr_ord(v), lp_index<T>(mis, seg, i)); };
            float from = low_bound, to = INFINITY;     // the border lies in [from, to)
            bool found = false;
            int n = 0;
            for (int round = 0; round < 4 && !found; ++round) {
                // 1. a histogram of [from, to) by the logit, from the top down, in units of 2^-30 of the whole mass, and
                // what lies above.  (Without a bound the steps are steps of the floats' order.)
                const float top = fminf(to, m), step = (float)(kDrBins - 1) / fmaxf(top - from, 1e-30f);
                const bool by_order = from == -FLT_MAX;
                const float per_one = weighed ? 1073741824.f / ((float)all / (float)one) : 1.f, c2 = E.ch * (1.f / kDrSteps);
                for (int i = t; i < kDrBins; i += kDrThreads) hist[i] = 0;
                __syncthreads();
                u64 over = 0;
                each_span(from, [&](const float (&v)[kDrSegs][8], int s) {
#pragma unroll
                    for (int g = 0; g < kDrSegs; ++g)
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            if (!(v[g][i] >= from) || !kept(v[g][i], s * kDrSegs + g, i)) continue;
                            const uint32_t c = weighed ? __float2uint_rn(ex2((v[g][i] - m) * c2) * per_one) : 1u;
                            if (v[g][i] >= to) over += c;
                            else atomicAdd(&hist[by_order ? (o_max - dr_ord(v[g][i])) >> 21 : min(kDrBins - 1, (int)((top - v[g][i]) * step))], c);
                        }
                });
                over = sum_all(over);                  // (and the histograms are there)
                // 2. the whole row's histogram, 8 steps a thread, and the steps that may hold the border
                constexpr int kEachBin = kDrBins / kDrThreads;
                u64 h[kEachBin], sum = 0;
#pragma unroll
                for (int e = 0; e < kEachBin; ++e) {
                    h[e] = 0;
                    for (int i = 0; i < C; ++i) h[e] += *cl.map_shared_rank(&hist[t * kEachBin + e], i);
                    sum += h[e];
                }
                u64 wall, at = dr_warp_before(sum, wall);
                if (lane == 0) sm.red[par][w] = wall;
                if (t == 0) { sm.bin_lo = kDrBins; sm.bin_hi = 0; }
                __syncthreads();
                u64 whole_sum = over;
                at += over;
                for (int i = 0; i < kDrWarps; ++i) {
                    if (i < w) at += sm.red[par][i];
                    whole_sum += sm.red[par][i];
                }
                par ^= 1;
                // (masses are rounded and a little off; a border outside these steps is noticed below)
                const u64 goal = weighed ? (u64)((float)need / (float)all * 1073741824.f) : need, err = weighed ? 8192 : 0;
#pragma unroll
                for (int e = 0; e < kEachBin; ++e) {
                    at += h[e];
                    if (at + err >= goal) atomicMin(&sm.bin_lo, t * kEachBin + e);      // first that may hold the border
                    if (at < goal + err) atomicMax(&sm.bin_hi, t * kEachBin + e + 1);   // past it: the last that may
                }
                cluster_sync();                        // (the histograms are read; the list may be written)
                if (whole_sum + err < goal) break;     // the border lies below the bound (min_p's), as far as this sum goes
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
                // 3. the tokens of these steps, if the list holds them; else the steps are taken apart
                found = make_list(from, n, [&](float v, int seg, int i) { return v >= from && v < to && kept(v, seg, i); });
            }
            if (found) {
                // 4. what lies above them, exactly, and the border among the listed
                u64 over = 0;
                if (weighed) {
                    mine = span_masses(to, [&](const float (&v)[8], int seg, u64 (&wt8)[8]) {
                        bool any = false;
#pragma unroll
                        for (int i = 0; i < 8; ++i) any |= v[i] >= to;
                        if (__any_sync(0xffffffffu, any)) dr_weights(E, v, wt8);
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (!(v[i] >= to) || !kept(v[i], seg, i)) wt8[i] = 0;
                    });
                    over = sum_all(lane == 0 ? mine : 0);
                } else {
                    each_span(to, [&](const float (&v)[kDrSegs][8], int s) {
#pragma unroll
                        for (int g = 0; g < kDrSegs; ++g)
#pragma unroll
                            for (int i = 0; i < 8; ++i) over += v[g][i] >= to && kept(v[g][i], s * kDrSegs + g, i) ? 1 : 0;
                    });
                    over = sum_all(over);
                }
                masses = weighed;
                if (rank == 0) {
                    take_list(n);
                    const u64 in = weighed ? above(0, mass) : above(0, count);
                    const bool holds = over < need && need <= over + in;
                    if (holds) {
                        if (weighed) cut_to(need - over, o_inf + 1, true, mass);
                        else cut_to(need - over, o_inf + 1, false, count);
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
                            everywhere(&sm.cv, (uint32_t)(least >> 32));
                            everywhere(&sm.ci, (int)~(uint32_t)least);
                        }
                    }
                    if (w == 0) everywhere(&sm.holds, (int)holds);
                }
                cluster_sync();
                if (sm.holds) {
                    cut = DrCut{sm.cv, sm.ci};
                    if (weighed) {
                        mine = 0;
                        for (int i = 0; i < s1 - s0; ++i) mine += my_sum[i];
                    }
                    return;
                }
            }
            // the whole row by bisection (more equal logits than the list holds), where the border lies above the bound
            masses = false;
            uint32_t lo = max(o_inf + 1, dr_ord(low_bound)), hi = o_max + 1;
            auto of = [&](uint32_t v) { return weighed ? row_mass(v, old) : row_count(v, old); };
            if (of(lo) < need) return;
            while (hi - lo > 1) {
                const uint32_t mid = lo + (hi - lo) / 2;
                if (of(mid) >= need) lo = mid;
                else hi = mid;
            }
            u64 rest = need - (lo < o_max ? of(lo + 1) : 0);
            if (weighed) {
                float v[8];
                u64 wt8[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = dr_value(lo);
                dr_weights(E, v, wt8);
                rest = (rest + wt8[0] - 1) / wt8[0];
            }
            // the id of the last of the equal tokens that stay
            auto tie = [&](const float (&v)[8], int seg, u64 (&wt8)[8]) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int d = lp_index<T>(mis, seg, i);
                    wt8[i] = dr_ord(v[i]) == lo && d >= 0 && d < V && dr_kept(old, lo, d) ? 1 : 0;
                }
            };
            const u64 ties = span_masses(dr_value(lo), tie);
            locate(ties, tie, [&](u64) { return rest - 1; }, [&](int d, float, u64) {
                for (int i = 0; i < C; ++i) *cl.map_shared_rank(&sm.ci, i) = d;
            });
            cluster_sync();
            cut = DrCut{lo, sm.ci};
        };
        if (K > 0) {
            // (at least K tokens are finite, or every finite one stays)
            if (row_count(o_inf + 1, cut) > (u64)K) select((u64)K, false, 0);
            if (nucleus) {
                S = row_mass(o_inf + 1, cut);
                p_target = max(dr_part(top_p, S, true), 1ull);
            }
        }
        if (nucleus) select(p_target, true, S);
        const auto f = kept_weights(cut, o_inf + 1, w_min);
        if (!masses || w_min > 1) mine = span_masses(dr_value(max(cut.v, o_inf + 1)), f);
        S_kept = locate(mine, f, [&](u64 total) { return dr_part(u, total, false); }, finish);
    }
    if (!probs) {
        cluster_sync();                                // (a CTA's shared memory stays while others read it)
        return;
    }

    // -------- the distribution
    const float inv = (float)(1ull << E.q) / (float)S_kept;
    const float least = dr_value(max(cut.v, o_inf + 1));
#pragma unroll 1
    for (int s = s0; s < s1; ++s) {
        const bool any = __any_sync(0xffffffffu, my_max[(s - s0) * 32 + lane] >= least);
#pragma unroll 1
        for (int g = 0; g < kDrSegs; ++g) {
            float v[8], y[8];
            if (any) lp_load(row, V, mis, s * kDrSegs + g, v);
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                y[i] = y[i + 1] = 0.f;
                if (!any) continue;
                u64 vv[2];
                int n[2];
                dr_weight2(E, v[i], v[i + 1], vv, n);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float l = v[i + j];
                    const bool in = dr_kept(cut, dr_ord(l), lp_index<T>(mis, s * kDrSegs + g, i + j)) &&
                                    dr_units(E, vv[j], n[j]) >= max(w_min, 1ull);
                    if (in) y[i + j] = (float)vv[j] * __uint_as_float((uint32_t)(127 - 62 - n[j]) << 23) * inv;
                }
            }
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const int d = lp_index<T>(mis, s * kDrSegs + g, p * VE);
                if (a.p_vec && d >= 0 && d + VE <= V) {
#pragma unroll
                    for (int i = 0; i < VE; i += 4)
                        *reinterpret_cast<float4*>(probs + d + i) = make_float4(y[p * VE + i], y[p * VE + i + 1], y[p * VE + i + 2], y[p * VE + i + 3]);
                } else {
#pragma unroll
                    for (int i = 0; i < VE; ++i)
                        if (d + i >= 0 && d + i < V) probs[d + i] = y[p * VE + i];
                }
            }
        }
    }
    cluster_sync();
}

static size_t dr_smem(int per) { return (size_t)kDrList * 8 + (size_t)kDrSteps * 8 + (size_t)kDrWarps * per * (8 + 4 + 32 * 4); }

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
    const size_t smem = dr_smem(a.per);
    void (*f)(DrawArgs) = dtype == SPEC_DTYPE_BF16 ? draw_kernel<__nv_bfloat16> : draw_kernel<float>;
    if (smem > 48 * 1024) {
        // the most that any call takes: another thread's call may come between this one's two steps
        constexpr int most_per = (kDrCtaVocab / kDrSpan + 1 + kDrWarps) / kDrWarps;
        SPEC_TRY(check_cuda(cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)dr_smem(most_per)), "spec_sample_logits attribute"));
    }
    cudaLaunchConfig_t cfg_l = {};
    cfg_l.gridDim = dim3((unsigned)(rows * C));
    cfg_l.blockDim = dim3(kDrThreads);
    cfg_l.dynamicSmemBytes = smem;
    cfg_l.stream = (cudaStream_t)stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = C;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg_l.attrs = at;
    cfg_l.numAttrs = 2;
    return check_cuda(cudaLaunchKernelEx(&cfg_l, f, a), "spec_sample_logits launch");
}
