// Log probabilities of given tokens, entropy and best alternatives of logits rows.
//
// With m = max x, d = c (x - m), c = log2 e / T, S = sum 2^d, U = sum 2^d d:
//     log p(t) = (x_t - m) / T - ln 2 log2 S
//     H        = ln 2 (log2 S - U / S)
// in one pass over the row: a thread keeps a running maximum and the two sums
// relative to it, rescaled when the maximum grows, and the threads' states join
// by the same rule.  Bound by reading the logits once.
//
// The n best tokens come from the same pass: every 256 consecutive logits (one
// step of a warp) leave their maximum in shared memory.  The n best by (value
// down, id up) lie in the n segments that are best by (maximum down, position
// up): a segment outside them has n segments before it, whose maxima are n
// tokens that rank before each of its own.  Those n segments are read again,
// their logits not below the least of the n maxima are listed, and a listed
// token's place is the number of listed tokens that rank before it.
//
// A row is taken by a cluster of 1 to 8 CTAs, each on a contiguous run of
// segments; the first CTA gathers the others' states and maxima from their
// shared memory.
#include <algorithm>
#include <cfloat>
#include <climits>
#include <cooperative_groups.h>

#include "attend.cuh"

namespace cg = cooperative_groups;

namespace spec {

constexpr int kLpThreads = 512;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpSeg = 256;
constexpr int kLpMaxTop = 32;
constexpr int kLpMaxVocab = 1 << 20;

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

SPEC_DEV float lp_ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// the state relative to a larger (or equal) maximum
SPEC_DEV void lp_raise(LpState& a, float m, float c) {
    if (a.m == m) return;
    const float d = (a.m - m) * c, f = lp_ex2(d);
    // nothing seen yet (m = -inf): the sums are zero
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

SPEC_DEV float warp_redux_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
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
            const uint4 w = __ldg(reinterpret_cast<const uint4*>(row + i0));
            const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (sizeof(T) == 4) {
                    x[p * VE + i] = __uint_as_float(a[i]);
                } else {
                    x[p * VE + (2 * i) % VE] = __uint_as_float(a[i] << 16);
                    x[p * VE + (2 * i + 1) % VE] = __uint_as_float(a[i] & 0xFFFF0000u);
                }
            }
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
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float d = (x[i] - m) * c, e = lp_ex2(d);
        a.s += e;
        a.u = fmaf(e, fmaxf(d, -FLT_MAX), a.u);       // a masked logit: 0 * -max, not 0 * -inf
    }
}

struct LpSmem {
    LpState w[kLpWarps];
    LpState cta;
    int sel[kLpMaxTop];
    float least;
    int n_cand;
};

template <typename T, int TOP>
__global__ void __launch_bounds__(kLpThreads)
logprobs_kernel(const __grid_constant__ LogprobArgs a) {
    pdl_wait();
    pdl_trigger();
    __shared__ LpSmem sm;
    extern __shared__ float dyn[];
    cg::cluster_group cl = cg::this_cluster();
    const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const long long r = blockIdx.x / C;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const T* row = static_cast<const T*>(a.x) + r * a.stride;
    const int mis = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    const int n_seg = (a.V + mis + kLpSeg - 1) / kLpSeg, per = (n_seg + C - 1) / C;
    const int g0 = min(n_seg, rank * per), g1 = min(n_seg, g0 + per);
    float* seg_max = dyn;                                   // [per] this CTA's; the first CTA: [n_seg] in the end
    LpState st{-INFINITY, 0.f, 0.f};
    for (int g = g0 + w; g < g1; g += 2 * kLpWarps) {
        float x[2][8];
        const bool two = g + kLpWarps < g1;
        lp_load(row, a.V, mis, g, x[0]);
        if (two) lp_load(row, a.V, mis, g + kLpWarps, x[1]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (k == 1 && !two) break;
            float xm = x[k][0];
#pragma unroll
            for (int i = 1; i < 8; ++i) xm = fmaxf(xm, x[k][i]);
            lp_add(st, x[k], a.c, xm);
            if (TOP) {
                const float sm_ = warp_redux_max(xm);
                if (lane == 0) seg_max[g + k * kLpWarps - g0] = sm_;
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
    if (threadIdx.x == 0) sm.n_cand = 0;
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
        if (lane == 0) sm.cta = st;
    }
    cl.sync();
    if (rank == 0) {
        st = sm.cta;
        for (int k = 1; k < C; ++k) lp_merge(st, *cl.map_shared_rank(&sm.cta, k), a.c);
        if (TOP)
            for (int k = 1; k < C; ++k) {
                const float* far = cl.map_shared_rank(seg_max, k);
                const int n = min(n_seg, (k + 1) * per) - min(n_seg, k * per);
                for (int i = threadIdx.x; i < n; i += kLpThreads) seg_max[k * per + i] = far[i];
            }
    }
    cl.sync();                                              // the others' shared memory has been read
    if (rank != 0) return;
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
    // the n best segments, by one warp: each lane keeps the best of its own (every 32nd)
    const int n_sel = min(n, n_seg);
    if (w == 0) {
        float bv = -INFINITY;
        int bi = INT_MAX;
        auto best = [&]() {
            bv = -INFINITY;
            bi = INT_MAX;
            for (int i = lane; i < n_seg; i += 32) {
                const float v = seg_max[i];
                // taken segments are marked by NaN
                if (v > bv || (v == bv && bi == INT_MAX)) { bv = v; bi = i; }
            }
        };
        best();
        float last = 0.f;
        for (int k = 0; k < n_sel; ++k) {
            // -inf segments count too (a mask may leave fewer tokens than n): a lane without any has bi = INT_MAX
            const float v = warp_redux_max(bv);
            const unsigned win = __reduce_min_sync(0xffffffffu, (unsigned)(bv == v ? bi : INT_MAX));
            if (lane == 0) sm.sel[k] = (int)win;
            last = v;
            if (bi == (int)win) {
                seg_max[win] = nan;
                best();
            }
        }
        // rows of fewer segments than n: every token is listed
        if (lane == 0) sm.least = n_sel < n ? -INFINITY : last;
    }
    __syncthreads();
    const float least = sm.least;
    float* cv = dyn + n_seg;                                // [n_sel * 256] values
    int* ci = reinterpret_cast<int*>(cv + n_sel * kLpSeg);  // and ids of the listed tokens
    for (int k = w; k < n_sel; k += kLpWarps) {
        const int g = sm.sel[k];
        float x[8];
        lp_load(row, a.V, mis, g, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int id = lp_index<T>(mis, g, e);
            if (id >= 0 && id < a.V && x[e] >= least) {
                const int at = atomicAdd(&sm.n_cand, 1);
                cv[at] = x[e];
                ci[at] = id;
            }
        }
    }
    __syncthreads();
    const int nc = sm.n_cand;
    for (int i = threadIdx.x; i < nc; i += kLpThreads) {
        const float v = cv[i];
        const int id = ci[i];
        int before = 0;
        for (int j = 0; j < nc; ++j) before += cv[j] > v || (cv[j] == v && ci[j] < id);
        if (before < n) {
            out_id[before] = id;
            out_lp[before] = (v - st.m) / a.T - lse;
        }
    }
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
    // CTAs a row: as many as keep every SM busy, each with 16 segments (one a warp) or more
    const int n_seg = (vocab + 7 + kLpSeg - 1) / kLpSeg;
    int C = 1;
    while (C < 8 && (long long)rows * C * 2 <= 2 * sms && n_seg / (2 * C) >= kLpWarps / 2) C *= 2;
    void (*f)(LogprobArgs) = dtype == SPEC_DTYPE_BF16 ? (n_top ? logprobs_kernel<__nv_bfloat16, 1> : logprobs_kernel<__nv_bfloat16, 0>)
                                                      : (n_top ? logprobs_kernel<float, 1> : logprobs_kernel<float, 0>);
    const size_t smem = n_top ? (size_t)(n_seg + C + (size_t)std::min(n_top, n_seg) * kLpSeg * 2) * 4 : 0;
    if (smem > 48 * 1024)
        SPEC_TRY(check_cuda(cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem), "spec_logprobs attribute"));
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
