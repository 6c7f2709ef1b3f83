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
// units of 2^-q of the best token's (q = 62 - log2 V, 45 for 131072 tokens), exact to
// 2^-38 of itself and half a unit, and sums of integers are exact in any order.
//
// A weight: d = x - m with its rounding error, t = 32 c d as a sum of two floats, the
// nearest integer 32 n + j split off, 2^(j / 32) from a table that lies in the warp's
// lanes, and 2^r of the rest (|r| <= 1 / 64) as 1 + a polynomial whose first term is
// taken in two floats; the product and the shift by n are integer arithmetic.
//
// A row is taken by a cluster of 1 to 8 CTAs, each warp on a contiguous run of spans
// of 1024 tokens.  One pass finds the maximum and leaves the maximum of every lane's 32
// tokens of a span in shared memory.  A bound below which no token can be kept follows
// from what is asked: the best lanes' maxima (k tokens are not below the least of k of
// them), min_p, or the row's mass (tokens below (1 - p) S / V of it add up to less than
// what the nucleus leaves out).  The tokens above the bound, by id, go into a list in the
// first CTA's shared memory (a span whose maxima lie below it is not read again), where
// the k-th logit and the nucleus' last one are found by bisection over the order of the
// floats.  A row with more such tokens than the list holds is bisected where it lies (in
// L2 by then).
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cmath>
#include <cooperative_groups.h>

#include "logits.cuh"

namespace cg = cooperative_groups;

namespace spec {

constexpr int kDrThreads = 256;
constexpr int kDrWarps = kDrThreads / 32;
constexpr int kDrMaxCtas = 8;
constexpr int kDrSegs = 4;                             // segments of a span
constexpr int kDrSpan = kDrSegs * kLpSeg;
constexpr int kDrEach = 8;                             // listed tokens a thread
constexpr int kDrList = kDrEach * kDrThreads;
constexpr int kDrMaxVocab = 1 << 20;
constexpr int kDrCtaVocab = 1 << 18;                   // a CTA's share at most: its lanes' maxima take 32 KB

struct DrawArgs {
    const void* x; long long stride;
    int V, per, q;                                     // per: spans a warp; q: a weight of 1 is 2^q
    const float* u;
    float T, p, mp; int k;
    const float* Ts; const float* ps; const float* mps; const int* ks;   // settings by row; null: the ones above
    int* tok; float* lp;
    float* probs; long long p_stride; int p_vec;
    unsigned long long pow[32];                        // 2^(62 + j / 32)
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
    u64 part[kDrMaxCtas * kDrWarps];                   // every warp's sum, in every CTA
    float wmax[kDrWarps], wlow[kDrWarps];
    float cmax[kDrMaxCtas], clow[kDrMaxCtas];
    int cbad[kDrMaxCtas], wbad[kDrWarps];
    float T, p, mp, u, ch, cl;
    int k, ok;
    u64 S;                                             // the list's result for the other CTAs
    uint32_t cv; int ci;
};

// A weight's arithmetic, the same in every lane but for the lane's entry of the table.
struct DrExp {
    float m, xmin, ch, cl;
    int q;
    uint32_t t_lo, t_hi;                               // 2^(62 + lane / 32)
};

// ln 2 / 32 in two floats, its powers over the factorials, all by 2^37
constexpr double kDrL = 0.69314718055994530942 / 32, kDrUnit = 137438953472.0;
constexpr float kDrL1h = (float)(kDrL * kDrUnit), kDrL1l = (float)(kDrL * kDrUnit - (double)kDrL1h);
constexpr float kDrL2 = (float)(kDrL * kDrL / 2 * kDrUnit), kDrL3 = (float)(kDrL * kDrL * kDrL / 6 * kDrUnit),
                kDrL4 = (float)(kDrL * kDrL * kDrL * kDrL / 24 * kDrUnit),
                kDrL5 = (float)(kDrL * kDrL * kDrL * kDrL * kDrL / 120 * kDrUnit);

SPEC_DEV float2 both(float x) { return make_float2(x, x); }

// weights of two logits: w = v * 2^-n with v in units of 2^-62
SPEC_DEV void dr_weight2(const DrExp& E, float x0, float x1, u64 (&v)[2], int (&n)[2]) {
    const float2 neg = both(-1.f), x = make_float2(fmaxf(x0, E.xmin), fmaxf(x1, E.xmin)), nm = both(-E.m);
    // d + dl = x - m exactly
    const float2 d = add2(x, nm), b = fma2(x, neg, d), a = fma2(b, neg, d);
    const float2 dl = add2(fma2(a, neg, x), fma2(b, neg, nm));
    // -p - e = -t
    const float2 np = mul2(d, both(-E.ch));
    float2 e = fma2(d, both(E.ch), np);
    e = fma2(d, both(E.cl), e);
    e = fma2(dl, both(E.ch), e);
    const float2 magic = both(12582912.f);
    const float2 k = fma2(np, neg, magic), nk = fma2(k, neg, magic), r = fma2(np, neg, nk);
    // 2^((r + e) / 32) - 1 in units of 2^-37
    const float2 s = add2(r, e);
    float2 g = fma2(both(kDrL5), s, both(kDrL4));
    g = fma2(g, s, both(kDrL3));
    g = fma2(g, s, both(kDrL2));
    g = mul2(g, s);
    const float2 na = mul2(r, both(-kDrL1h));
    float2 ae = fma2(r, both(kDrL1h), na);
    ae = fma2(r, both(kDrL1l), ae);
    ae = fma2(e, both(kDrL1h), ae);
    ae = fma2(g, s, ae);
    const float kf[2] = {k.x, k.y}, nf[2] = {na.x, na.y}, af[2] = {ae.x, ae.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int ki = __float_as_int(kf[i]) - 0x4B400000;
        const uint32_t lo = __shfl_sync(0xffffffffu, E.t_lo, ki & 31), hi = __shfl_sync(0xffffffffu, E.t_hi, ki & 31);
        const int delta = __float2int_rn(af[i]) - __float2int_rn(nf[i]);
        v[i] = (((u64)hi << 32) | lo) + (u64)(((long long)(int)hi * delta + 16) >> 5);
        n[i] = -(ki >> 5);
    }
}
// to units of 2^-q, to the nearest: cut off, the many small weights of a large vocabulary would be missed in the
// sum by half a unit each; logits below xmin, which lies 2^-q under the maximum, have no weight
SPEC_DEV int dr_shift(const DrExp& E, float x, int n) { return x >= E.xmin ? 62 - E.q + n : 64; }
SPEC_DEV u64 dr_round(u64 v, int shift) { return ((v >> (shift - 1)) + 1) >> 1; }
SPEC_DEV void dr_weights(const DrExp& E, const float (&x)[8], u64 (&w)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        u64 v[2];
        int n[2];
        dr_weight2(E, x[i], x[i + 1], v, n);
        w[i] = dr_round(v[0], dr_shift(E, x[i], n[0]));
        w[i + 1] = dr_round(v[1], dr_shift(E, x[i + 1], n[1]));
    }
}

// a kept logit: above the cut's value, or equal to it with an id not above the cut's
struct DrCut { uint32_t v; int id; };
SPEC_DEV bool dr_kept(const DrCut& c, uint32_t o, int id) { return o > c.v || (o == c.v && id <= c.id); }

template <typename T>
__global__ void __launch_bounds__(kDrThreads, 3)
draw_kernel(const __grid_constant__ DrawArgs a) {
    pdl_wait();
    pdl_trigger();
    constexpr int VE = 16 / sizeof(T), NP = 8 / VE;
    __shared__ DrSmem sm;
    extern __shared__ __align__(16) u64 dyn[];
    u64* list = dyn;                                   // [kDrList] (value's order, id) by id; the first CTA's
    u64* span_sum = dyn + kDrList;                     // [kDrWarps][per]
    float* lane_max = reinterpret_cast<float*>(span_sum + kDrWarps * a.per);   // [kDrWarps][per][32]
    cg::cluster_group cl = cg::this_cluster();
    const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const long long row_i = blockIdx.x / C;
    const int t = threadIdx.x, lane = t & 31, w = t >> 5, gw = rank * kDrWarps + w;
    const T* row = static_cast<const T*>(a.x) + row_i * a.stride;
    const int V = a.V, mis = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    const int n_span = (V + mis + kDrSpan - 1) / kDrSpan;
    const int s0 = min(n_span, gw * a.per), s1 = min(n_span, s0 + a.per);
    span_sum += w * a.per;
    lane_max += w * a.per * 32;
    auto cluster_sync = [&]() {
        if (C > 1) cl.sync();
        else __syncthreads();
    };
    auto everywhere = [&](auto* p, auto value) {       // by one warp: the same variable of every CTA
        if (lane < C) *cl.map_shared_rank(p, lane) = value;
    };
    cluster_sync();                                    // every CTA has started: its shared memory may be written

    if (t == 0) {
        const float temp = a.Ts ? a.Ts[row_i] : a.T, p = a.ps ? a.ps[row_i] : a.p, mp = a.mps ? a.mps[row_i] : a.mp;
        const int k = a.ks ? a.ks[row_i] : a.k;
        const float u = a.u[row_i];
        sm.ok = (temp == 0.f || (temp >= 1e-30f && temp <= 1e30f)) && p >= 0.f && mp >= 0.f && mp <= 1.f && k >= 0 && u >= 0.f && u < 1.f;
        // temperature 0: the best token
        sm.k = temp == 0.f ? 1 : (k >= V ? 0 : k);
        sm.T = temp == 0.f ? 1.f : temp;
        sm.p = p;
        sm.mp = mp;
        sm.u = u;
        const double c = 46.166241308446828384 / (double)sm.T;     // 32 log2 e / T
        sm.ch = (float)c;
        sm.cl = (float)(c - (double)sm.ch);
    }

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

    // -------- the maximum, every lane's maxima, and whether the row has a distribution
    float mx = -INFINITY;
    bool bad = false;
    for (int s = s0; s < s1; ++s) {
        float x[kDrSegs][8], g4[kDrSegs];
        load_span(s, x);
#pragma unroll
        for (int g = 0; g < kDrSegs; ++g) {
            g4[g] = x[g][0];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                bad |= !(x[g][i] <= FLT_MAX);          // NaN or +inf
                g4[g] = fmaxf(g4[g], x[g][i]);
            }
        }
        const float g = fmaxf(fmaxf(g4[0], g4[1]), fmaxf(g4[2], g4[3]));
        lane_max[(s - s0) * 32 + lane] = g;
        mx = fmaxf(mx, g);
    }
    mx = warp_redux_max(mx);
    bad = __any_sync(0xffffffffu, bad);
    __syncthreads();                                   // the settings are there
    const int K = sm.k;
    // This warp's share of the bound for top-k: of the warps with a full run of spans each gives the value of
    // (about) its r-th largest lane maximum; the least of these has r tokens a warp that are not below it.
    float low = INFINITY;
    const int full = n_span / a.per, r_low = K > 0 ? (K + full - 1) / full : 0;
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
                for (int i = 0; i < a.per; ++i) n += lane_max[i * 32 + lane] >= v;
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
    if (bad || m == -INFINITY || !sm.ok) {             // no distribution, or settings out of range
        const float nan = __int_as_float(0x7fc00000);
        if (rank == 0 && t == 0) {
            a.tok[row_i] = -1;
            if (a.lp) a.lp[row_i] = nan;
        }
        if (probs)
            for (int i = rank * kDrThreads + t; i < V; i += C * kDrThreads) probs[i] = nan;
        return;
    }
    DrExp E;
    E.m = m;
    E.ch = sm.ch;
    E.cl = sm.cl;
    E.xmin = m - (float)(32 * a.q) / E.ch;             // 62 - q + n is 63 at most
    E.q = a.q;
    E.t_lo = (uint32_t)a.pow[lane];
    E.t_hi = (uint32_t)(a.pow[lane] >> 32);
    const u64 one = 1ull << a.q, w_min = dr_part(sm.mp, one, true);
    const uint32_t o_max = dr_ord(m), o_inf = dr_ord(-INFINITY);

    int par = 0;
    // sums over the CTA, or over the cluster
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
        const int p = par;
        u64 s = sum_cta(v);
        if (C > 1) {
            if (w == 0) everywhere(&sm.redc[p][rank], s);
            cl.sync();
            s = 0;
            for (int i = 0; i < C; ++i) s += sm.redc[p][i];
        }
        return s;
    };
    // every span of this warp that holds a logit not below `least`: f(logits, span)
    auto each_span = [&](float least, auto f) {
        for (int s = s0; s < s1; ++s) {
            if (!__any_sync(0xffffffffu, lane_max[(s - s0) * 32 + lane] >= least)) continue;
            float x[kDrSegs][8];
            load_span(s, x);
            f(x, s);
        }
    };
    // the sum of the weights of the kept logits not below `least`
    auto row_mass = [&](uint32_t least, const DrCut& cut) {
        u64 sum = 0;
        each_span(dr_value(least), [&](const float (&x)[kDrSegs][8], int s) {
#pragma unroll 1
            for (int g = 0; g < kDrSegs; ++g) {
                u64 wt[8];
                dr_weights(E, x[g], wt);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t o = dr_ord(x[g][i]);
                    if (o >= least && dr_kept(cut, o, lp_index<T>(mis, s * kDrSegs + g, i))) sum += wt[i];
                }
            }
        });
        return sum_all(sum);
    };
    auto row_count = [&](uint32_t least) {
        u64 n = 0;
        each_span(dr_value(least), [&](const float (&x)[kDrSegs][8], int) {
#pragma unroll
            for (int g = 0; g < kDrSegs; ++g)
#pragma unroll
                for (int i = 0; i < 8; ++i) n += dr_ord(x[g][i]) >= least ? 1 : 0;
        });
        return sum_all(n);
    };
    // Tokens by id, weighed by f(logits of a segment, segment, weights): the one at which the sum passes `target`.
    // found(id, logit) is called by one thread of the cluster; returns the sum of all.
    auto row_locate = [&](float least, auto f, auto target_of, auto found) {
        u64 mine = 0;
        for (int s = s0; s < s1; ++s) {
            u64 sum = 0;
            if (__any_sync(0xffffffffu, lane_max[(s - s0) * 32 + lane] >= least)) {
                float x[kDrSegs][8];
                load_span(s, x);
#pragma unroll 1
                for (int g = 0; g < kDrSegs; ++g) {
                    u64 wt[8];
                    f(x[g], s * kDrSegs + g, wt);
#pragma unroll
                    for (int i = 0; i < 8; ++i) sum += wt[i];
                }
            }
            sum = dr_warp_sum(sum);
            if (lane == 0) span_sum[s - s0] = sum;
            mine += sum;
        }
        __syncwarp();
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
            while (left >= span_sum[s - s0]) left -= span_sum[s++ - s0];
            float x[kDrSegs][8];
            load_span(s, x);
#pragma unroll 1
            for (int g = 0; g < kDrSegs; ++g) {
                u64 wt[8];
                f(x[g], s * kDrSegs + g, wt);
                bool done = false;
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
                                    found(lp_index<T>(mis, s * kDrSegs + g, p * VE + i), x[g][p * VE + i]);
                                }
                            }
                        }
                        done = true;
                    }
                    left -= done ? 0 : all;
                }
                if (done) break;
            }
        }
        return total;
    };
    auto finish = [&](int id, float x, u64 S) {
        a.tok[row_i] = id;
        if (a.lp) {
            // log S without cancellation where one token holds nearly all of it
            const float ls = S < 2 * one ? log1pf((float)(S - one) / (float)one) : logf((float)S / (float)one);
            a.lp[row_i] = (x - m) / sm.T - ls;
        }
    };

    // -------- a bound below which nothing is kept
    const float T_ = sm.T, slack = 1e-3f;
    float low_bound = -FLT_MAX;
    u64 p_target = 0;
    const bool nucleus = sm.p < 1.f;
    bool listed = true;
    auto below = [&](float z) {                        // safely below m + T z
        const float v = m + T_ * (z - slack);
        return fmaxf(v - fabsf(v) * 1e-6f, -FLT_MAX);
    };
    if (K == 1) {
        low_bound = m;
    } else if (K > 0) {
        low_bound = fmaxf(k_low, -FLT_MAX);
    } else if (nucleus) {
        const u64 S = row_mass(o_inf + 1, DrCut{o_inf, -1});
        p_target = max(dr_part(sm.p, S, true), 1ull);
        low_bound = below(logf(fmaxf((1.f - sm.p) * ((float)S / (float)one) / (float)V, 1e-30f)));
    } else {
        listed = sm.mp > 0.f;
    }
    // (min_p leaves out of top-k's and the nucleus' tokens, whose number and mass count them)
    if (sm.mp > 0.f && K == 0) low_bound = fmaxf(low_bound, below(logf(sm.mp)));

    // -------- the list
    int n_list = 0;
    if (listed) {
        int n = 0;
        each_span(low_bound, [&](const float (&x)[kDrSegs][8], int) {
#pragma unroll
            for (int g = 0; g < kDrSegs; ++g)
#pragma unroll
                for (int i = 0; i < 8; ++i) n += x[g][i] >= low_bound ? 1 : 0;
        });
        n = __reduce_add_sync(0xffffffffu, n);
        everywhere(&sm.part[gw], (u64)n);
        cluster_sync();
        int before = 0;
        for (int i = 0; i < C * kDrWarps; ++i) {
            if (i == gw) before = n_list;
            n_list += (int)sm.part[i];
        }
        listed = n_list <= kDrList;
        if (listed) {
            u64* first = cl.map_shared_rank(list, 0);
            each_span(low_bound, [&](const float (&x)[kDrSegs][8], int s) {
#pragma unroll
                for (int g = 0; g < kDrSegs; ++g)
#pragma unroll
                    for (int p = 0; p < NP; ++p) {
                        int c = 0;
#pragma unroll
                        for (int i = 0; i < VE; ++i) c += x[g][p * VE + i] >= low_bound ? 1 : 0;
                        if (!__any_sync(0xffffffffu, c > 0)) continue;
                        int upto = c;
#pragma unroll
                        for (int o = 1; o < 32; o <<= 1) {
                            const int v = __shfl_up_sync(0xffffffffu, upto, o);
                            if (lane >= o) upto += v;
                        }
                        int at = before + upto - c;
#pragma unroll
                        for (int i = 0; i < VE; ++i)
                            if (x[g][p * VE + i] >= low_bound)
                                first[at++] = (u64)dr_ord(x[g][p * VE + i]) << 32 | (uint32_t)lp_index<T>(mis, s * kDrSegs + g, p * VE + i);
                        before += __shfl_sync(0xffffffffu, upto, 31);
                    }
            });
        }
        cluster_sync();
    }

    DrCut cut{o_inf, -1};
    u64 S_kept = 0;
    if (listed) {
        if (rank == 0) {
            // every thread holds `each` neighbours of the list
            const int each = (n_list + kDrThreads - 1) / kDrThreads;
            uint32_t o[kDrEach];
            int id[kDrEach];
            u64 wt[kDrEach];
            float x[kDrEach];
#pragma unroll
            for (int e = 0; e < kDrEach; ++e) {
                const int i = t * each + e;
                const bool in = e < each && i < n_list;
                const u64 key = in ? list[i] : 0;
                o[e] = (uint32_t)(key >> 32);
                id[e] = (int)(uint32_t)key;
                x[e] = in ? dr_value(o[e]) : -INFINITY;
            }
            dr_weights(E, x, wt);
#pragma unroll
            for (int e = 0; e < kDrEach; ++e)
                if (o[e] == 0) wt[e] = 0;
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
            // largest v whose tokens not below it weigh (or count) at least `need`
            auto bisect = [&](u64 need, auto of) {
                uint32_t lo = o_inf + 1, hi = o_max + 1;
                const uint32_t from = dr_ord(low_bound);
                lo = max(lo, from);
                while (hi - lo > 1) {
                    const uint32_t mid = lo + (hi - lo) / 2;
                    u64 s = 0;
#pragma unroll
                    for (int e = 0; e < kDrEach; ++e) s += o[e] >= mid ? of(e) : 0;
                    if (sum_cta(s) >= need) lo = mid;
                    else hi = mid;
                }
                return lo;
            };
            auto above = [&](uint32_t v, auto of) {
                u64 s = 0;
#pragma unroll
                for (int e = 0; e < kDrEach; ++e) s += o[e] > v ? of(e) : 0;
                return sum_cta(s);
            };
            auto count = [&](int) -> u64 { return 1; };
            auto mass = [&](int e) -> u64 { return wt[e]; };
            if (K > 0 && n_list > K) {
                const uint32_t v = bisect((u64)K, count);
                cut_at(v, (u64)K - above(v, count));
            }
            if (nucleus) {
                const u64 all = above(0, mass), target = K > 0 ? max(dr_part(sm.p, all, true), 1ull) : p_target;
                if (all >= target) {
                    const uint32_t v = bisect(target, mass);
                    const u64 rest = target - above(v, mass);
                    // tokens of one value have one weight
                    u64 one_w = 0;
#pragma unroll
                    for (int e = 0; e < kDrEach; ++e)
                        if (o[e] == v) one_w = wt[e];
                    const u64 holders = sum_cta(one_w ? 1 : 0), sum_w = sum_cta(one_w);
                    const u64 w1 = sum_w / holders;
                    cut_at(v, (rest + w1 - 1) / w1);
                }
            }
            u64 mine = 0, least = ~0ull;
#pragma unroll
            for (int e = 0; e < kDrEach; ++e) {
                if (o[e]) least = min(least, (u64)o[e] << 32 | (uint32_t)~id[e]);
                if (wt[e] < w_min) wt[e] = 0;
                mine += wt[e];
            }
            u64 all, at = dr_warp_before(mine, all);
            if (lane == 0) sm.red[par][w] = all;
            __syncthreads();
            u64 S = 0;
            for (int i = 0; i < kDrWarps; ++i) {
                if (i == w) at += S;
                S += sm.red[par][i];
            }
            par ^= 1;
            const u64 target = dr_part(sm.u, S, false);
            if (at <= target && target < at + mine) {
                bool hit = false;
#pragma unroll
                for (int e = 0; e < kDrEach; ++e) {
                    at += wt[e];
                    if (!hit && target < at) {
                        hit = true;
                        finish(id[e], x[e], S);
                    }
                }
            }
            if (probs) {
#pragma unroll
                for (int o2 = 16; o2 > 0; o2 >>= 1) least = min(least, __shfl_xor_sync(0xffffffffu, least, o2));
                if (lane == 0) sm.red[par][w] = least;
                __syncthreads();
                for (int i = 0; i < kDrWarps; ++i) least = min(least, sm.red[par][i]);
                if (w == 0) {
                    everywhere(&sm.S, S);
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
        // the id of the n-th (from 0) of the tokens that equal v
        auto tie_cut = [&](uint32_t v, u64 n, const DrCut& old) {
            row_locate(dr_value(v), [&](const float (&x)[8], int seg, u64 (&wt)[8]) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int id = lp_index<T>(mis, seg, i);
                    wt[i] = dr_ord(x[i]) == v && id >= 0 && id < V && dr_kept(old, v, id) ? 1 : 0;
                }
            }, [&](u64) { return n; }, [&](int id, float) {
                for (int i = 0; i < C; ++i) *cl.map_shared_rank(&sm.ci, i) = id;
            });
            cluster_sync();
            return DrCut{v, sm.ci};
        };
        auto bisect = [&](u64 need, auto of) {
            uint32_t lo = max(o_inf + 1, dr_ord(low_bound)), hi = o_max + 1;
            while (hi - lo > 1) {
                const uint32_t mid = lo + (hi - lo) / 2;
                if (of(mid) >= need) lo = mid;
                else hi = mid;
            }
            return lo;
        };
        if (K > 0) {
            // (at least K tokens are finite, or every finite one stays)
            if (row_count(o_inf + 1) > (u64)K) {
                const uint32_t v = bisect((u64)K, row_count);
                const u64 over = v < o_max ? row_count(v + 1) : 0;
                cut = tie_cut(v, (u64)K - over - 1, cut);
            }
        }
        if (nucleus) {
            if (K > 0) p_target = max(dr_part(sm.p, row_mass(o_inf + 1, cut), true), 1ull);
            auto mass = [&](uint32_t v) { return row_mass(v, cut); };
            const uint32_t v = bisect(p_target, mass);
            if (mass(v) >= p_target) {
                const u64 rest = p_target - (v < o_max ? mass(v + 1) : 0);
                float x[8];
                u64 wt[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = dr_value(v);
                dr_weights(E, x, wt);
                cut = tie_cut(v, (rest + wt[0] - 1) / wt[0] - 1, cut);
            }
        }
        S_kept = row_locate(dr_value(max(cut.v, o_inf + 1)), [&](const float (&x)[8], int seg, u64 (&wt)[8]) {
            dr_weights(E, x, wt);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (wt[i] < w_min || !dr_kept(cut, dr_ord(x[i]), lp_index<T>(mis, seg, i))) wt[i] = 0;
        }, [&](u64 total) { return dr_part(sm.u, total, false); }, [&](int id, float x) {
            u64 total = 0;
            for (int i = 0; i < C * kDrWarps; ++i) total += sm.part[i];
            finish(id, x, total);
        });
    }
    if (!probs) {
        cluster_sync();                                // (a CTA's shared memory stays while others read it)
        return;
    }

    // -------- the distribution
    const float inv = (float)one / (float)S_kept;
    const float least = dr_value(max(cut.v, o_inf + 1));
    for (int s = s0; s < s1; ++s) {
        const bool any = __any_sync(0xffffffffu, lane_max[(s - s0) * 32 + lane] >= least);
        float x[kDrSegs][8];
        if (any) load_span(s, x);
#pragma unroll 1
        for (int g = 0; g < kDrSegs; ++g) {
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                y[i] = y[i + 1] = 0.f;
                if (!any) continue;
                u64 v[2];
                int n[2];
                dr_weight2(E, x[g][i], x[g][i + 1], v, n);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float l = x[g][i + j];
                    const bool in = l >= E.xmin && dr_kept(cut, dr_ord(l), lp_index<T>(mis, s * kDrSegs + g, i + j)) &&
                                    dr_round(v[j], dr_shift(E, l, n[j])) >= w_min;
                    if (in) y[i + j] = (float)v[j] * __uint_as_float((uint32_t)(127 - 62 - n[j]) << 23) * inv;
                }
            }
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const int id = lp_index<T>(mis, s * kDrSegs + g, p * VE);
                if (a.p_vec && id >= 0 && id + VE <= V) {
#pragma unroll
                    for (int i = 0; i < VE; i += 4)
                        *reinterpret_cast<float4*>(probs + id + i) = make_float4(y[p * VE + i], y[p * VE + i + 1], y[p * VE + i + 2], y[p * VE + i + 3]);
                } else {
#pragma unroll
                    for (int i = 0; i < VE; ++i)
                        if (id + i >= 0 && id + i < V) probs[id + i] = y[p * VE + i];
                }
            }
        }
    }
    cluster_sync();
}

static size_t dr_smem(int per) { return (size_t)kDrList * 8 + (size_t)kDrWarps * per * (8 + 32 * 4); }

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
        unsigned long long t[32];
        Table() { for (int j = 0; j < 32; ++j) t[j] = (unsigned long long)std::ldexp(std::exp2((long double)j / 32), 62); }
    } table;
    std::copy(table.t, table.t + 32, a.pow);
    const int n_span = (vocab + 7 + kDrSpan - 1) / kDrSpan;
    int C = 1;
    while (C < kDrMaxCtas && ((long long)vocab > (long long)C * kDrCtaVocab || ((long long)rows * C < 3 * sms && n_span > C * kDrWarps))) C *= 2;
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
