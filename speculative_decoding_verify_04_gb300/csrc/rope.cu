// Rotary positions of query and key rows, for positions of one or several axes.
//
// A row's first 2 n dims are n pairs (x_i, x_{i+n}); pair i is turned by the angle
//     a_i = position[axis of i] theta^(-i / n):
//     y_i = x_i cos a_i - x_{i+n} sin a_i,   y_{i+n} = x_{i+n} cos a_i + x_i sin a_i,
// the row's other dims pass.  An angle of a far position is many turns, of which 32
// bits would keep few digits: a pair's frequency is held in turns as a 64-bit fraction
// F = 2^64 theta^(-i / n) / 2 pi, the product position x F is taken modulo 2^64 (whole
// turns fall off by themselves), its nearest quarter turn is split off, and what is left,
// at most an eighth of a turn either way, is exact enough as a float (2^-28 of a radian).
//
// A CTA takes `group` rows: their angles once, in shared memory, for all heads, while the
// rows' own loads are on their way; then 16 bytes of each half of a head a thread at a time.
// Bound by memory (three operations a value): 16384 bf16 rows of 32 + 8 heads of 128 with three axes
// take 58 us a call, 5.8 TB/s of reads and writes, 85 % of a copy's rate; without the loads ahead
// of the angles 67.6.  One row: 9.1 us, a call's own time.
#include <algorithm>
#include <cmath>

#include "attend.cuh"

namespace spec {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxPairs = 128;           // head_dim <= 256
constexpr int kRopeMaxAxes = 4;
constexpr int kRopeMaxGroup = 4;
constexpr int kRopeAhead = 4;                // pieces of each half that a thread has on their way

struct RopeArgs {
    const void* src[2];                      // queries, keys
    void* dst[2];
    long long src_stride[2], dst_stride[2];  // elements
    int heads[2];                            // 0: no such rows
    int hd, n, rows, group;
    int rest;                                // the dims past the pairs are copied
    const int* pos; long long pos_stride;    // positions [axis][row]; null: from the cache
    const int* len; const int* pre_len; int pre_cap;
    uint64_t freq[kRopeMaxPairs];
    uint8_t axis[kRopeMaxPairs];
};

// position id of row r of the span: what its sequence holds, and the row's depth in its chain or tree
SPEC_DEV int row_position(const RopeArgs& a, const AttendSpan& s, int r) {
    int lo = 0, hi = s.batch - 1;            // last sequence with row0 <= r
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s.row0[mid] <= r) lo = mid;
        else hi = mid - 1;
    }
    const int j = r - s.row0[lo];
    return (a.pre_len ? min(*a.pre_len, a.pre_cap) : 0) + a.len[lo] + (s.tree ? __popcll(s.mask[j]) - 1 : j);
}

// cosine and sine of `turns` / 2^64 turns
SPEC_DEV float2 cos_sin(uint64_t turns) {
    const uint32_t q = (uint32_t)((turns + (1ull << 61)) >> 62);       // nearest quarter
    const float f = (float)(int64_t)(turns - ((uint64_t)q << 62)) * 1.0842021724855044e-19f;   // 2^-63: half turns
    float s, c;
    sincospif(f, &s, &c);
    const float x = q & 1 ? -s : c, y = q & 1 ? c : s;
    return q & 2 ? make_float2(-x, -y) : make_float2(x, y);
}

// VE elements of a head as they lie in memory (VE * sizeof(T) = 16 bytes, or one element)
template <typename T, int VE>
struct RopePiece {
    uint4 raw;
    SPEC_DEV void load(const T* p) {
        if constexpr (VE == 1) raw.x = sizeof(T) == 4 ? *reinterpret_cast<const uint32_t*>(p) : (uint32_t)*reinterpret_cast<const uint16_t*>(p) << 16;
        else raw = *reinterpret_cast<const uint4*>(p);      // (a plain load: results may lie over their inputs)
    }
    SPEC_DEV void get(float (&x)[VE]) const {
        if constexpr (VE == 1) {
            x[0] = __uint_as_float(raw.x);
        } else {
            const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (sizeof(T) == 4) {
                    x[i] = __uint_as_float(u[i]);
                } else {
                    x[2 * i] = __uint_as_float(u[i] << 16);
                    x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
                }
            }
        }
    }
    SPEC_DEV static void store(T* p, const float (&x)[VE]) {
        if constexpr (VE == 1) {
            if constexpr (sizeof(T) == 4) *p = x[0];
            else *p = __float2bfloat16_rn(x[0]);
        } else if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
        } else {
            *reinterpret_cast<uint4*>(p) = make_uint4(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]), bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
        }
    }
};

template <typename T, int VE>
__global__ void __launch_bounds__(kRopeThreads)
rope_kernel(const __grid_constant__ RopeArgs a, const __grid_constant__ AttendSpan span) {
    pdl_wait();
    pdl_trigger();
    __shared__ __align__(16) float cs[kRopeMaxGroup][2][kRopeMaxPairs];
    constexpr int U = kRopeAhead;
    const int t = threadIdx.x, row0 = blockIdx.x * a.group, rows = min(a.group, a.rows - row0);
    const int chunks = a.n / VE, per = (a.heads[0] + a.heads[1]) * chunks, items = rows * per;
    RopePiece<T, VE> lo[U], hi[U];
    auto at = [&](int i, int& r, int& c, int& which, int& h) {
        r = i / per;
        int x = i - r * per;
        h = x / chunks;
        c = (x - h * chunks) * VE;
        which = h >= a.heads[0];
        h -= which ? a.heads[0] : 0;
    };
    auto fetch = [&](int i0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * kRopeThreads;
            if (i >= items) break;
            int r, c, which, h;
            at(i, r, c, which, h);
            const T* p = static_cast<const T*>(a.src[which]) + (row0 + r) * a.src_stride[which] + h * a.hd + c;
            lo[u].load(p);
            hi[u].load(p + a.n);
        }
    };
    fetch(t);
    for (int i = t; i < rows * a.n; i += kRopeThreads) {
        const int r = i / a.n, p = i - r * a.n;
        const int pos = a.pos ? a.pos[a.axis[p] * a.pos_stride + row0 + r] : row_position(a, span, row0 + r);
        const float2 f = cos_sin((uint64_t)(int64_t)pos * a.freq[p]);
        cs[r][0][p] = f.x;
        cs[r][1][p] = f.y;
    }
    __syncthreads();
    for (int i0 = t; i0 < items;) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * kRopeThreads;
            if (i >= items) break;
            int r, c, which, h;
            at(i, r, c, which, h);
            float x[VE], y[VE];
            lo[u].get(x);
            hi[u].get(y);
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float v = x[e], z = y[e], co = cs[r][0][c + e], si = cs[r][1][c + e];
                x[e] = v * co - z * si;
                y[e] = z * co + v * si;
            }
            T* p = static_cast<T*>(a.dst[which]) + (row0 + r) * a.dst_stride[which] + h * a.hd + c;
            RopePiece<T, VE>::store(p, x);
            RopePiece<T, VE>::store(p + a.n, y);
        }
        i0 += U * kRopeThreads;
        fetch(i0);
    }
    if (a.rest) {
        const int left = a.hd - 2 * a.n, lp = left / VE, rest = rows * (a.heads[0] + a.heads[1]) * lp;
        for (int i = t; i < rest; i += kRopeThreads) {
            const int hr = i / lp, c = 2 * a.n + (i - hr * lp) * VE, r = hr / (a.heads[0] + a.heads[1]);
            int h = hr - r * (a.heads[0] + a.heads[1]);
            const int which = h >= a.heads[0];
            h -= which ? a.heads[0] : 0;
            RopePiece<T, VE> p;
            float x[VE];
            p.load(static_cast<const T*>(a.src[which]) + (row0 + r) * a.src_stride[which] + h * a.hd + c);
            p.get(x);
            RopePiece<T, VE>::store(static_cast<T*>(a.dst[which]) + (row0 + r) * a.dst_stride[which] + h * a.hd + c, x);
        }
    }
}

}  // namespace spec

using namespace spec;

extern "C" int spec_rope(const spec_rope_config* cfg, int32_t rows, const void* q, int64_t q_stride, void* q_out,
                         int64_t q_out_stride, const void* k, int64_t k_stride, void* k_out, int64_t k_out_stride,
                         const int32_t* positions, int64_t pos_stride, spec_kv* kv, int32_t batch, const int32_t* n_rows,
                         const int32_t* tree_parent, void* stream) {
    if (!cfg) return set_error(SPEC_ERR_ARG, "spec_rope: null pointer");
    const spec_rope_config c = *cfg;
    if (c.dtype != SPEC_DTYPE_F32 && c.dtype != SPEC_DTYPE_BF16) return set_error(SPEC_ERR_ARG, "spec_rope: unknown dtype");
    if (c.n_heads < 0 || c.n_kv_heads < 0 || c.n_heads + (int64_t)c.n_kv_heads < 1 || rows < 0)
        return set_error(SPEC_ERR_ARG, "spec_rope: bad sizes");
    if (c.head_dim < 2 || c.head_dim > 2 * kRopeMaxPairs || c.n_heads > 4096 || c.n_kv_heads > 4096)
        return set_error(SPEC_ERR_UNSUPPORTED, "spec_rope: head_dim must be in [2, 256], heads at most 4096");
    if (!(c.theta >= 1.0) || !(c.theta <= 1e30)) return set_error(SPEC_ERR_ARG, "spec_rope: theta must be in [1, 1e30]");
    if (c.axes < 1 || c.axes > kRopeMaxAxes) return set_error(SPEC_ERR_ARG, "spec_rope: axes must be in [1, 4]");
    int64_t n = 0;
    for (int x = 0; x < c.axes; ++x) {
        if (c.sections[x] < 0 || c.sections[x] > kRopeMaxPairs) return set_error(SPEC_ERR_ARG, "spec_rope: sections must be in [0, head_dim / 2]");
        n += c.sections[x];
    }
    if (n < 1 || 2 * n > c.head_dim) return set_error(SPEC_ERR_ARG, "spec_rope: sections must add up to 1 .. head_dim / 2");
    if ((positions && kv) || (!positions && !kv && rows > 0)) return set_error(SPEC_ERR_ARG, "spec_rope: positions or a cache, not both");
    if (kv && c.axes != 1) return set_error(SPEC_ERR_ARG, "spec_rope: a cache gives positions of one axis");
    if (positions && c.axes > 1 && pos_stride < rows) return set_error(SPEC_ERR_ARG, "spec_rope: pos_stride is shorter than the rows");
    const int64_t qd = (int64_t)c.n_heads * c.head_dim, kd = (int64_t)c.n_kv_heads * c.head_dim;
    if ((c.n_heads && (q_stride < qd || q_out_stride < qd)) || (c.n_kv_heads && (k_stride < kd || k_out_stride < kd)))
        return set_error(SPEC_ERR_ARG, "spec_rope: a row stride is shorter than its row");
    AttendSpan span{};
    RopeArgs a{};
    if (kv) {
        int dev = -1;
        SPEC_TRY(check_cuda(cudaGetDevice(&dev), "spec_rope: cudaGetDevice"));
        if (dev != kv->m->device) return set_error(SPEC_ERR_ARG, "spec_rope: the cache is on another device than the current one");
        SPEC_TRY(kv_check_prefix(kv, "spec_rope"));
        if (!n_rows) return set_error(SPEC_ERR_ARG, "spec_rope: null pointer");
        if (batch < 1 || batch > kv->batch) return set_error(SPEC_ERR_ARG, "spec_rope: bad batch");
        int64_t T = 0;
        int n_max = 0;
        for (int b = 0; b < batch; ++b) {
            if (n_rows[b] < 0 || n_rows[b] > kMaxSeqRows) return set_error(SPEC_ERR_ARG, "spec_rope: n_rows[b] must be in [0, 64]");
            T += n_rows[b];
            n_max = n_rows[b] > n_max ? n_rows[b] : n_max;
        }
        if (T != rows) return set_error(SPEC_ERR_ARG, "spec_rope: n_rows must add up to rows");
        if (tree_parent) {
            if (n_max > 0 && tree_parent[0] != -1) return set_error(SPEC_ERR_ARG, "tree_parent[0] must be -1");
            for (int i = 1; i < n_max; ++i)
                if (tree_parent[i] < 0 || tree_parent[i] >= i) return set_error(SPEC_ERR_ARG, "tree_parent[i] must be in [0, i)");
        }
        SPEC_TRY(make_span(&span, batch, n_rows, 0, tree_parent, nullptr));
        a.len = kv->len;
        if (kv->prefix) {
            a.pre_len = kv->prefix->len + kv->prefix_seq;
            a.pre_cap = kv->prefix->max_ctx;
        }
    }
    if (rows == 0) return SPEC_OK;
    if ((c.n_heads && (!q || !q_out)) || (c.n_kv_heads && (!k || !k_out))) return set_error(SPEC_ERR_ARG, "spec_rope: null pointer");
    a.src[0] = q;
    a.src[1] = k;
    a.dst[0] = q_out;
    a.dst[1] = k_out;
    a.src_stride[0] = q_stride;
    a.src_stride[1] = k_stride;
    a.dst_stride[0] = q_out_stride;
    a.dst_stride[1] = k_out_stride;
    a.heads[0] = c.n_heads;
    a.heads[1] = c.n_kv_heads;
    a.hd = c.head_dim;
    a.n = (int)n;
    a.rows = rows;
    a.pos = positions;
    a.pos_stride = pos_stride;
    // a pair's frequency in turns; its axis by sections, or the axes in turn while their sections last
    int32_t left[kRopeMaxAxes] = {};
    for (int x = 0; x < c.axes; ++x) left[x] = c.sections[x];
    const double step = -std::log2(c.theta) / (double)n;
    for (int i = 0, x = 0; i < n; ++i) {
        a.freq[i] = (uint64_t)std::ldexp(std::exp2(step * i) * 0.15915494309189535, 64);
        while (left[x] == 0) x = x + 1 < c.axes ? x + 1 : 0;
        a.axis[i] = (uint8_t)x;
        --left[x];
        if (c.interleaved) x = x + 1 < c.axes ? x + 1 : 0;
    }
    const int elem = c.dtype == SPEC_DTYPE_BF16 ? 2 : 4, ve = 16 / elem;
    bool vec = n % ve == 0 && c.head_dim % ve == 0, in_place = true;
    for (int w = 0; w < 2; ++w) {
        if (!a.heads[w]) continue;
        if (reinterpret_cast<uintptr_t>(a.src[w]) % elem || reinterpret_cast<uintptr_t>(a.dst[w]) % elem)
            return set_error(SPEC_ERR_ARG, "spec_rope: rows not aligned to their type");
        vec &= a.src_stride[w] % ve == 0 && a.dst_stride[w] % ve == 0 && reinterpret_cast<uintptr_t>(a.src[w]) % 16 == 0 &&
               reinterpret_cast<uintptr_t>(a.dst[w]) % 16 == 0;
        in_place &= a.src[w] == a.dst[w] && a.src_stride[w] == a.dst_stride[w];
    }
    a.rest = 2 * n < c.head_dim && !in_place;
    // rows a CTA: one, or as many as its threads hold at once where there are enough
    const int pieces = (c.n_heads + c.n_kv_heads) * (int)(vec ? n / ve : n);
    a.group = rows < 2048 ? 1 : std::max(1, std::min(kRopeMaxGroup, kRopeAhead * kRopeThreads / pieces));
    void (*f)(RopeArgs, AttendSpan) = elem == 2 ? (vec ? rope_kernel<__nv_bfloat16, 8> : rope_kernel<__nv_bfloat16, 1>)
                                                : (vec ? rope_kernel<float, 4> : rope_kernel<float, 1>);
    return check_cuda(launch_k(true, f, dim3((unsigned)((rows + a.group - 1) / a.group)), dim3(kRopeThreads), 0,
                               (cudaStream_t)stream, a, span), "spec_rope launch");
}
