// Log probabilities of given tokens, entropy and best alternatives of logits rows.
//
// With m = max x, d = c (x - m), c = log2 e / T, S = sum 2^d, U = sum 2^d d:
//     log p(t) = (x_t - m) / T - ln 2 log2 S
//     H        = ln 2 (log2 S - U / S)
// in one pass over the row: a thread keeps a running maximum and the two sums
// relative to it, rescaled when the maximum grows, and the threads' states join
// by the same rule.  The difference is taken before the product, so rows masked by
// the type's lowest value do not overflow.  Bound by reading the logits once (512 f32
// rows of 131072: 42 us, 6.3 TB/s, 94 % of the measured copy rate; with 20
// alternatives 54); half-precision rows by the instructions, about twenty a logit: 60 %
// of the issue slots (333 rows of 100003: 21 us, 3.2 TB/s; with one alternative 27).
//
// The n best tokens come from the same pass: every 256 consecutive logits (one
// step of a warp) leave their maximum in shared memory.  The n best by (value
// down, id up) lie in the n segments that are best by (maximum down, position
// up): a segment outside them has n segments before it, whose maxima are n
// tokens that rank before each of its own.  Those n segments are read again,
// their logits not below the least of the n maxima are listed, and a listed
// token's place is the number of listed tokens that rank before it.
//
// A row is taken by a cluster of 1 to 4 CTAs, each on a contiguous run of
// segments; the others leave their states and maxima in the first one's shared
// memory and end.
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cooperative_groups.h>

#include "attend.cuh"

namespace cg = cooperative_groups;

namespace spec {

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpSeg = 256;
constexpr int kLpMaxTop = 32;
constexpr int kLpMaxVocab = 1 << 20;
constexpr int kLpMaxCtas = 4;

struct LogprobArgs {
    const void* x;
    long long stride;
    int V;
    float T, c;                  // temperature, log2(e) / T
    const int* tok; float* lp; float* ent;
    int n_top; int* top_id; float* top_lp;
};

// running state of a set of logits: m = max x, s = sum 2^d, u = sum 2^d d with d = c (x - m)
struct LpState { float m, s, u; };

// the state relative to a larger (or equal) maximum
SPEC_DEV void lp_raise(LpState& a, float m, float c) {
    if (a.m == m) return;
    const float d = (a.m - m) * c, f = ex2(d);
    // nothing seen yet (m = -inf): the sums are zero (or NaN)
    a.u = a.m == -INFINITY ? a.u : (f > 0.f ? (a.u + a.s * d) * f : 0.f);
    a.s = a.m == -INFINITY ? a.s : a.s * f;
    a.m = m;
}
SPEC_DEV void lp_merge(LpState& a, LpState b, float c) {
    const float m = fmaxf(a.m, b.m);
    lp_raise(a, m, c);
    lp_raise(b, m, c);
    a.s += b.s;
    a.u += b.u;
}

// (value, id) as a number that is larger for what ranks before: by value down (both zeros alike), id up
SPEC_DEV unsigned long long lp_key(float v, int id) {
    const uint32_t u = __float_as_uint(v + 0.f);
    return (unsigned long long)(u >> 31 ? ~u : u | 0x80000000u) << 32 | (uint32_t)~id;
}
SPEC_DEV int lp_key_id(unsigned long long k) { return (int)~(uint32_t)k; }
SPEC_DEV float lp_key_value(unsigned long long k) {
    const uint32_t u = (uint32_t)(k >> 32);
    return __uint_as_float(u >> 31 ? u & 0x7FFFFFFFu : ~u);
}
// appends `key` of the lanes with `in` to a list, in lane order behind one addition a warp
SPEC_DEV void lp_list(unsigned long long* list, int* count, unsigned long long key, bool in) {
    const uint32_t m = __ballot_sync(0xffffffffu, in);
    if (m == 0) return;
    const int lane = threadIdx.x & 31;
    int at = 0;
    if (lane == 0) at = atomicAdd(count, __popc(m));
    at = __shfl_sync(0xffffffffu, at, 0) + __popc(m & ((1u << lane) - 1u));
    if (in) list[at] = key;
}
// Of a segment's elements that equal the least listed value (bits eq of in) only the n of the lowest
// ids stay: a row of equal logits would else list whole segments (512 rows of 131072 with one token
// left by a mask and 20 alternatives: 330 us).
template <typename T>
SPEC_DEV uint32_t lp_first_equal(uint32_t in, uint32_t eq, int n) {
    constexpr int VE = 16 / sizeof(T);                      // ids rise over a piece's VE elements, lanes, pieces
    const int lane = threadIdx.x & 31;
    int seen = 0;
#pragma unroll
    for (int p = 0; p < 8 / VE; ++p) {
        const uint32_t mine = (eq >> (p * VE)) & ((1u << VE) - 1u);
        int upto = __popc(mine);                            // of the lanes up to this one
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += v;
        }
        int at = seen + upto - __popc(mine);
#pragma unroll
        for (int e = 0; e < VE; ++e)
            if ((mine >> e) & 1u)
                if (at++ >= n) in &= ~(1u << (p * VE + e));
        seen += __shfl_sync(0xffffffffu, upto, 31);
    }
    return in;
}
// How many of nc listed keys are larger than `key`, counted until there are n.
SPEC_DEV int lp_place(const unsigned long long* list, int nc, int n, unsigned long long key) {
    int before = 0, j = 0;
    for (; j + 8 <= nc && before < n; j += 8) {
#pragma unroll
        for (int q = 0; q < 8; ++q) before += list[j + q] > key ? 1 : 0;
    }
    if (before < n)
        for (; j < nc; ++j) before += list[j] > key ? 1 : 0;
    return before;
}

SPEC_DEV float warp_redux_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// a 16-byte piece as floats
template <typename T>
SPEC_DEV void lp_unpack(const uint4& w, float* x) {
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (sizeof(T) == 4) {
            x[i] = __uint_as_float(a[i]);
        } else {
            x[2 * i] = __uint_as_float(a[i] << 16);
            x[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
        }
    }
}

// One segment of a row: 8 logits a lane.  Element i of the row sits at position
// i + mis, mis the elements between a 16-byte boundary and the row's start, so
// whole pieces are aligned; pieces that the row does not fill are read one by one.
template <typename T>
SPEC_DEV void lp_load(const T* row, int V, int mis, int seg, float (&x)[8]) {
    constexpr int VE = 16 / sizeof(T), NP = 8 / VE;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int i0 = seg * kLpSeg + (p * 32 + lane) * VE - mis;
        if (i0 >= 0 && i0 + VE <= V) {
            lp_unpack<T>(__ldg(reinterpret_cast<const uint4*>(row + i0)), &x[p * VE]);
        } else {
#pragma unroll
            for (int i = 0; i < VE; ++i)
                x[p * VE + i] = i0 + i >= 0 && i0 + i < V ? to_f32<T>(row[i0 + i]) : -INFINITY;
        }
    }
}
// row index of the lane's element e of a segment
template <typename T>
SPEC_DEV int lp_index(int mis, int seg, int e) {
    constexpr int VE = 16 / sizeof(T);
    return seg * kLpSeg + ((e / VE) * 32 + (threadIdx.x & 31)) * VE + e % VE - mis;
}

SPEC_DEV void lp_add(LpState& a, const float (&x)[8], float c, float xm) {
    const float m = fmaxf(a.m, xm);
    if (m == -INFINITY) {
        // masked logits only; a NaN among them still has to show
#pragma unroll
        for (int i = 0; i < 8; ++i) a.s += x[i] != x[i] ? x[i] : 0.f;
        return;
    }
    lp_raise(a, m, c);
    const float2 cc = make_float2(c, c), nn = make_float2(-m, -m);
    float2 s = make_float2(0.f, 0.f), u = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float2 d = mul2(add2(make_float2(x[2 * i], x[2 * i + 1]), nn), cc);
        const float2 e = make_float2(ex2(d.x), ex2(d.y));
        d.x = fmaxf(d.x, -FLT_MAX);                   // a masked logit: 0 * -max, not 0 * -inf
        d.y = fmaxf(d.y, -FLT_MAX);
        s = add2(s, e);
        u = fma2(e, d, u);
    }
    a.s += s.x + s.y;
    a.u += u.x + u.y;
}

struct LpSmem {
    LpState w[kLpWarps];
    LpState cta[kLpMaxCtas];          // the first CTA's: every CTA's state
    int sel[kLpMaxTop];
    float low, least;
    int n_near, n_cand;
};

// a cluster barrier in two halves
SPEC_DEV void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
SPEC_DEV void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

template <typename T, int TOP>
__global__ void __launch_bounds__(kLpThreads, sizeof(T) == 4 ? 4 : 5)
logprobs_kernel(const __grid_constant__ LogprobArgs a) {
    pdl_wait();
    pdl_trigger();
    __shared__ LpSmem sm;
    extern __shared__ __align__(16) float dyn[];
    cg::cluster_group cl = cg::this_cluster();
    const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    if (C > 1) cluster_arrive();                            // started: its shared memory may be written
    const long long r = blockIdx.x / C;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const T* row = static_cast<const T*>(a.x) + r * a.stride;
    const int mis = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    const int n_seg = (a.V + mis + kLpSeg - 1) / kLpSeg, per = (n_seg + C - 1) / C;
    const int g0 = min(n_seg, rank * per), g1 = min(n_seg, g0 + per);
    float* seg_max = dyn;                                   // [n_seg]; each CTA's own part, the first one's all of it
    LpState st{-INFINITY, 0.f, 0.f};
    constexpr int U = 4;                                    // segments in flight a warp
    constexpr int VE = 16 / sizeof(T), NP = 8 / VE;
    auto take = [&](const float (&x)[8], int g) {
        float xm = x[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) xm = fmaxf(xm, x[i]);
        lp_add(st, x, a.c, xm);
        if (TOP) {
            const float top = warp_redux_max(xm);
            if (lane == 0) seg_max[g] = top;
        }
    };
    for (int g = g0 + w; g < g1; g += U * kLpWarps) {
        const int last = g + (U - 1) * kLpWarps;
        if (last < g1 && g * kLpSeg >= mis && (last + 1) * kLpSeg - mis <= a.V) {
            // every piece whole: all loads before the first value is looked at
            uint4 p[U][NP];
            const T* at = row + (g * kLpSeg - mis + lane * VE);
#pragma unroll
            for (int k = 0; k < U; ++k)
#pragma unroll
                for (int q = 0; q < NP; ++q)
                    p[k][q] = __ldg(reinterpret_cast<const uint4*>(at + k * kLpWarps * kLpSeg + q * 32 * VE));
#pragma unroll
            for (int k = 0; k < U; ++k) {
                float x[8];
#pragma unroll
                for (int q = 0; q < NP; ++q) lp_unpack<T>(p[k][q], &x[q * VE]);
                take(x, g + k * kLpWarps);
            }
        } else {
            for (int k = 0; k < U && g + k * kLpWarps < g1; ++k) {
                float x[8];
                lp_load(row, a.V, mis, g + k * kLpWarps, x);
                take(x, g + k * kLpWarps);
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        LpState t;
        t.m = __shfl_xor_sync(0xffffffffu, st.m, o);
        t.s = __shfl_xor_sync(0xffffffffu, st.s, o);
        t.u = __shfl_xor_sync(0xffffffffu, st.u, o);
        lp_merge(st, t, a.c);
    }
    if (lane == 0) sm.w[w] = st;
    if (threadIdx.x == 0) sm.n_near = sm.n_cand = 0;
    __syncthreads();
    if (w == 0) {
        st = lane < kLpWarps ? sm.w[lane] : LpState{-INFINITY, 0.f, 0.f};
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            LpState t;
            t.m = __shfl_xor_sync(0xffffffffu, st.m, o);
            t.s = __shfl_xor_sync(0xffffffffu, st.s, o);
            t.u = __shfl_xor_sync(0xffffffffu, st.u, o);
            lp_merge(st, t, a.c);
        }
        if (lane == 0 && rank == 0) sm.cta[0] = st;
    }
    if (C > 1) {
        cluster_wait();
        if (rank > 0) {
            if (threadIdx.x == 0) *cl.map_shared_rank(&sm.cta[rank], 0) = st;
            if (TOP) {
                float* first = cl.map_shared_rank(seg_max, 0);
                for (int i = g0 + threadIdx.x; i < g1; i += kLpThreads) first[i] = seg_max[i];
            }
        }
        cluster_arrive();
        if (rank > 0) return;                                // (a barrier waits for threads that have not ended)
        cluster_wait();
    } else {
        __syncthreads();
    }
    st = sm.cta[0];
    for (int k = 1; k < C; ++k) lp_merge(st, sm.cta[k], a.c);
    // a row with NaN, +inf or nothing but -inf has no distribution
    const bool good = st.m > -INFINITY && st.m < INFINITY && st.s < INFINITY;
    const float l2 = log2f(st.s), lse = l2 * 0.6931471805599453f, nan = __int_as_float(0x7fc00000);
    if (threadIdx.x == 0) {
        if (a.lp) {
            const int t = a.tok[r];
            const bool in = t >= 0 && t < a.V;
            a.lp[r] = good && in ? (to_f32<T>(row[in ? t : 0]) - st.m) / a.T - lse : nan;
        }
        if (a.ent) a.ent[r] = good ? (l2 - st.u / st.s) * 0.6931471805599453f : nan;
    }
    if (!TOP) return;
    const int n = a.n_top;
    int* out_id = a.top_id + r * n;
    float* out_lp = a.top_lp + r * n;
    if (!good) {
        if (threadIdx.x < n) { out_id[threadIdx.x] = -1; out_lp[threadIdx.x] = nan; }
        return;
    }
    // The n best segments.  Of the best segments of 32 interleaved parts the n-th is a lower bound
    // of the n-th best of all; the segments not below it are listed (few more than n), and a listed
    // one's place is the number of listed ones before it.
    const int n_sel = min(n, n_seg);
    unsigned long long* near = reinterpret_cast<unsigned long long*>(dyn + (n_seg + 1) / 2 * 2);   // [n_seg] listed maxima, segments
    if (w == 0) {
        float bv = -INFINITY;
#pragma unroll 4
        for (int i = lane; i < n_seg; i += 32) bv = fmaxf(bv, seg_max[i]);
        int before = 0;
        for (int k = 0; k < 32; ++k) {
            const float v = __shfl_sync(0xffffffffu, bv, k);
            before += v > bv || (v == bv && k < lane);
        }
        // (a part without segments counts as -inf)
        if (before == n_sel - 1) sm.low = bv;
    }
    __syncthreads();
    const float low = sm.low;
    for (int i0 = 0; i0 < n_seg; i0 += kLpThreads) {
        const int i = i0 + threadIdx.x;
        const float v = i < n_seg ? seg_max[i] : 0.f;
        lp_list(near, &sm.n_near, lp_key(v, i), i < n_seg && v >= low);
    }
    __syncthreads();
    const int n_near = sm.n_near;
    for (int i = threadIdx.x; i < n_near; i += kLpThreads) {
        const unsigned long long key = near[i];
        const int before = lp_place(near, n_near, n_sel, key);
        if (before < n_sel) sm.sel[before] = lp_key_id(key);
        // rows of fewer segments than n: every token is listed
        if (before == n_sel - 1) sm.least = n_sel < n ? -INFINITY : lp_key_value(key);
    }
    __syncthreads();
    const float least = sm.least;
    unsigned long long* cand = near + n_seg;                // [n_sel * 256] listed tokens
    for (int k0 = w; k0 < n_sel; k0 += 4 * kLpWarps) {
        float x[4][8];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (k0 + q * kLpWarps < n_sel) lp_load(row, a.V, mis, sm.sel[k0 + q * kLpWarps], x[q]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (k0 + q * kLpWarps >= n_sel) break;
            const int g = sm.sel[k0 + q * kLpWarps];
            uint32_t in = 0, eq = 0;                        // bit e: listed, equal to the least
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int id = lp_index<T>(mis, g, e);
                if (id >= 0 && id < a.V && x[q][e] >= least) in |= 1u << e;
                if (x[q][e] == least) eq |= in & (1u << e);
            }
            if (__reduce_add_sync(0xffffffffu, __popc(eq)) > n) in = lp_first_equal<T>(in, eq, n);
            if (in) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if ((in >> e) & 1u) cand[atomicAdd(&sm.n_cand, 1)] = lp_key(x[q][e], lp_index<T>(mis, g, e));
            }
        }
    }
    __syncthreads();
    const int nc = sm.n_cand;
    for (int i = threadIdx.x; i < nc; i += kLpThreads) {
        const unsigned long long key = cand[i];
        const int before = lp_place(cand, nc, n, key);
        if (before < n) {
            out_id[before] = lp_key_id(key);
            out_lp[before] = (lp_key_value(key) - st.m) / a.T - lse;
        }
    }
}

// segments' maxima and keys, and the listed tokens
constexpr size_t lp_smem(int n_seg, int n_top) {
    return n_top ? (size_t)(n_seg + 1) / 2 * 8 + ((size_t)n_seg + (size_t)(n_top < n_seg ? n_top : n_seg) * kLpSeg) * 8 : 0;
}

}  // namespace spec

using namespace spec;

extern "C" int spec_logprobs(const void* logits, int32_t dtype, int64_t lg_stride, int32_t rows, int32_t vocab,
                             float temperature, const int32_t* tokens, float* logprob, float* entropy, int32_t n_top,
                             int32_t* top_ids, float* top_logprobs, void* stream) {
    if (!logits) return set_error(SPEC_ERR_ARG, "spec_logprobs: null pointer");
    if (dtype != SPEC_DTYPE_F32 && dtype != SPEC_DTYPE_BF16) return set_error(SPEC_ERR_ARG, "spec_logprobs: unknown dtype");
    if (rows < 0 || vocab < 1 || lg_stride < vocab) return set_error(SPEC_ERR_ARG, "spec_logprobs: bad sizes");
    if (vocab > kLpMaxVocab) return set_error(SPEC_ERR_UNSUPPORTED, "spec_logprobs: vocab must be at most 1048576");
    if (!(temperature > 0.f) || !(temperature <= FLT_MAX) || !(1.4426950408889634f / temperature <= FLT_MAX))
        return set_error(SPEC_ERR_ARG, "spec_logprobs: temperature must be positive and finite");
    if ((tokens == nullptr) != (logprob == nullptr)) return set_error(SPEC_ERR_ARG, "spec_logprobs: tokens and logprob go together");
    if (n_top < 0 || n_top > kLpMaxTop || n_top > vocab) return set_error(SPEC_ERR_ARG, "spec_logprobs: n_top must be in [0, min(32, vocab)]");
    if ((n_top > 0) != (top_ids != nullptr) || (n_top > 0) != (top_logprobs != nullptr))
        return set_error(SPEC_ERR_ARG, "spec_logprobs: top_ids and top_logprobs go with n_top > 0");
    const size_t elem = dtype == SPEC_DTYPE_BF16 ? 2 : 4;
    if (reinterpret_cast<uintptr_t>(logits) % elem) return set_error(SPEC_ERR_ARG, "spec_logprobs: logits not aligned to their type");
    if (!logprob && !entropy && n_top == 0) return set_error(SPEC_ERR_ARG, "spec_logprobs: no output asked for");
    if (rows == 0) return SPEC_OK;
    int dev = 0, sms = 0;
    SPEC_TRY(check_cuda(cudaGetDevice(&dev), "cudaGetDevice"));
    SPEC_TRY(check_cuda(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev), "attr"));
    LogprobArgs a{logits, lg_stride, vocab, temperature, 1.4426950408889634f / temperature, tokens, logprob, entropy, n_top, top_ids, top_logprobs};
    // CTAs a row: until there are three an SM (four or five are resident), 16 segments a CTA or more
    // (512 rows of 131072: 42 us by one CTA a row, 57 by two; 333 rows of 100003, half
    // precision: 39 us by one, 26 by two, 29 by four)
    const int n_seg = (vocab + 7 + kLpSeg - 1) / kLpSeg;
    int C = 1;
    while (C < kLpMaxCtas && (long long)rows * C < 3 * sms && n_seg / (2 * C) >= 16) C *= 2;
    void (*f)(LogprobArgs) = dtype == SPEC_DTYPE_BF16 ? (n_top ? logprobs_kernel<__nv_bfloat16, 1> : logprobs_kernel<__nv_bfloat16, 0>)
                                                      : (n_top ? logprobs_kernel<float, 1> : logprobs_kernel<float, 0>);
    const size_t smem = lp_smem(n_seg, n_top);
    if (smem > 48 * 1024) {
        // the most that any call takes: another thread's call may come between this one's two steps
        constexpr int most = (int)lp_smem((kLpMaxVocab + 7 + kLpSeg - 1) / kLpSeg, kLpMaxTop);
        SPEC_TRY(check_cuda(cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, most), "spec_logprobs attribute"));
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * C));
    cfg.blockDim = dim3(kLpThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = C;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return check_cuda(cudaLaunchKernelEx(&cfg, f, a), "spec_logprobs launch");
}
