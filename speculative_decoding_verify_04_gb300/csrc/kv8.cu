// 8-bit KV caches: rows quantised as they are written, and read back.
//
// Both directions are bound by memory (the arithmetic is a maximum over hd
// values, a shift of the exponent and one conversion a value): writing moves
// 2 bytes in and 1 out a value, reading back 1 in and 2 out, and one exponent
// byte a row.  32 layers x 2048 slots x 32 KV heads of 128 (1.6 GB) go in in
// 266 us (6.06 TB/s, 90 % of the measured copy rate) and out in 284 us (5.69);
// where they stay in L2 the conversions bound the way in (76 MB in 17.6 us, the
// issue slots 63 % used) and the latency of the loads the way out (12.7 us).
#include <algorithm>

#include "attend.cuh"

namespace spec {

// 8 bf16 values at p; one 16-byte load where the rows are aligned
SPEC_DEV uint4 load8(const __nv_bfloat16* p, bool vec) {
    if (vec) return *reinterpret_cast<const uint4*>(p);
    const unsigned short* s = reinterpret_cast<const unsigned short*>(p);
    return make_uint4(s[0] | (uint32_t)s[1] << 16, s[2] | (uint32_t)s[3] << 16, s[4] | (uint32_t)s[5] << 16,
                      s[6] | (uint32_t)s[7] << 16);
}
SPEC_DEV void floats8(const uint4& w, float (&x)[8]) {
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(a[i] << 16);
        x[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
    }
}

// New rows of a batch into one layer.  HD / 8 lanes hold a row, 8 values each
// (16-byte loads); the row's maximum goes around by shuffles.  8-bit caches
// get the quantised row, bf16 caches the row itself.  A call's rows are few (512 rows
// of 8 KV heads: 3.2 us), so this is one launch's latency.
struct AppendArgs {
    const __nv_bfloat16* src[2];
    long long stride[2];
    int vec[2];                     // rows and strides are 16-byte aligned
    void* cache[2];                 // first row of the layer
    uint8_t* exps[2];               // null: bf16 cache
    KVPages pages;
    const int* len;
    int cap, Hkv;
    int* err;
    AttendSpan span;
};

template <int HD>
__global__ void __launch_bounds__(128)
append_kernel(const __grid_constant__ AppendArgs a) {
    pdl_wait();
    pdl_trigger();
    constexpr int L = HD / 8;
    const int which = blockIdx.y;
    const int item = (blockIdx.x * 128 + threadIdx.x) / L, l = threadIdx.x % L;
    const bool in = item < a.span.T * a.Hkv;
    const int r = in ? item / a.Hkv : 0, h = in ? item % a.Hkv : 0;
    int lo = 0, hi = a.span.batch - 1;            // last sequence with row0 <= r
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.span.row0[mid] <= r) lo = mid; else hi = mid - 1;
    }
    uint4 w = make_uint4(0, 0, 0, 0);
    if (in) w = load8(a.src[which] + r * a.stride[which] + h * HD + l * 8, a.vec[which]);
    const int slot = a.len[lo] + a.span.extra + r - a.span.row0[lo];
    long long row = -1;
    if (in && slot < a.cap) row = kv_row_in_layer(a.pages, a.Hkv, lo, h, slot);
    if (in && row < 0 && l == 0) dev_error(a.err, SPEC_DEVERR_CAPACITY);
    if (a.exps[which]) {
        float x[8];
        floats8(w, x);
        float m = finite_amax(x);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const int e = kv8_exp(m);
        if (row >= 0) {
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.cache[which]) + row * HD + l * 8) = e4m3x8(x, kv8_inv_scale(e));
            if (l == 0) a.exps[which][row] = (uint8_t)e;
        }
    } else if (row >= 0) {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.cache[which]) + row * HD + l * 8) = w;
    }
}

// One sequence's rows [n_layers][n_slots][Hkv][hd] into or out of an 8-bit
// cache.  A warp takes 16 consecutive slots of one KV head (so the exponents
// leave as one 16-byte piece and the e4m3 rows as one run), neighbouring warps
// neighbouring heads (so the bf16 rows are read in runs too).
constexpr int kCopySlots = 16;

struct Kv8CopyArgs {
    __nv_bfloat16* rows[2];
    uint8_t* cache[2];
    uint8_t* exps[2];
    KVPages pages;
    int seq, Hkv, layer0, n_layers, slot0, n_slots, n_blk;
    int vec;
    int* err;
};

template <int HD, bool IN>
__global__ void __launch_bounds__(256)
kv8_copy_kernel(const __grid_constant__ Kv8CopyArgs a) {
    pdl_wait();
    pdl_trigger();
    constexpr int L = HD / 8, RPS = 32 / L, STEPS = kCopySlots / RPS;
    const int which = blockIdx.y, lane = threadIdx.x & 31, grp = lane / L, l = lane % L;
    const long long n_items = (long long)a.n_layers * a.n_blk * a.Hkv;
    for (long long it = blockIdx.x * 8ll + (threadIdx.x >> 5); it < n_items; it += gridDim.x * 8ll) {
        const int h = (int)(it % a.Hkv);
        const long long rest = it / a.Hkv;
        const int blk = (int)(rest % a.n_blk), layer = (int)(rest / a.n_blk);
        // blocks start at multiples of kCopySlots of the cache, so none crosses a page
        const int s_first = (a.slot0 / kCopySlots + blk) * kCopySlots;
        const int s0 = max(s_first, a.slot0), s1 = min(s_first + kCopySlots, a.slot0 + a.n_slots);
        const long long row0 = kv_row(a.pages, a.Hkv, a.layer0 + layer, a.seq, h, s_first);
        if (row0 < 0) {
            if (lane == 0) dev_error(a.err, SPEC_DEVERR_CAPACITY);
            continue;
        }
        __nv_bfloat16* rows = a.rows[which] + ((long long)layer * a.n_slots * a.Hkv + h) * HD + l * 8;
        uint8_t* cache = a.cache[which] + row0 * HD + l * 8;
        uint8_t* exps = a.exps[which] + row0;
        if (IN) {
            uint4 w[STEPS];
#pragma unroll
            for (int t = 0; t < STEPS; ++t) {
                const int s = s_first + t * RPS + grp;
                w[t] = make_uint4(0, 0, 0, 0);
                if (s >= s0 && s < s1) w[t] = load8(rows + (long long)(s - a.slot0) * a.Hkv * HD, a.vec);
            }
#pragma unroll
            for (int t = 0; t < STEPS; ++t) {
                const int s = s_first + t * RPS + grp;
                float x[8];
                floats8(w[t], x);
                float m = finite_amax(x);
#pragma unroll
                for (int o = L / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                const int e = kv8_exp(m);
                if (s >= s0 && s < s1) {
                    *reinterpret_cast<uint2*>(cache + (s - s_first) * HD) = e4m3x8(x, kv8_inv_scale(e));
                    if (l == 0) exps[s - s_first] = (uint8_t)e;
                }
            }
        } else {
#pragma unroll
            for (int t = 0; t < STEPS; ++t) {
                const int s = s_first + t * RPS + grp;
                if (s < s0 || s >= s1) continue;
                const uint2 w = *reinterpret_cast<const uint2*>(cache + (s - s_first) * HD);
                const float sc = kv8_scale(exps[s - s_first]);
                uint32_t o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = e4m3x2_f32((i < 2 ? w.x : w.y) >> (16 * (i & 1)));
                    o[i] = bf16x2(f.x * sc, f.y * sc);
                }
                __nv_bfloat16* dst = rows + (long long)(s - a.slot0) * a.Hkv * HD;
                if (a.vec) {
                    *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
                } else {
                    unsigned short* d = reinterpret_cast<unsigned short*>(dst);
#pragma unroll
                    for (int i = 0; i < 4; ++i) { d[2 * i] = (unsigned short)o[i]; d[2 * i + 1] = (unsigned short)(o[i] >> 16); }
                }
            }
        }
    }
}

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

int launch_kv8_copy(spec_kv* kv, int seq, int layer0, int n_layers, int slot0, int n_slots, void* k, void* v,
                    bool to_cache, cudaStream_t st) {
    spec_model* m = kv->m;
    const spec_model_config& c = m->cfg;
    Kv8CopyArgs a{};
    a.rows[0] = (__nv_bfloat16*)k; a.rows[1] = (__nv_bfloat16*)v;
    a.cache[0] = (uint8_t*)kv->k; a.cache[1] = (uint8_t*)kv->v;
    a.exps[0] = kv->ke; a.exps[1] = kv->ve;
    a.pages = kv->pages();
    a.seq = seq; a.Hkv = c.n_kv_heads; a.layer0 = layer0; a.n_layers = n_layers;
    a.slot0 = slot0; a.n_slots = n_slots;
    a.n_blk = (slot0 + n_slots - 1) / kCopySlots - slot0 / kCopySlots + 1;
    a.vec = aligned16(k) && aligned16(v);
    a.err = m->err;
    const long long items = (long long)n_layers * a.n_blk * c.n_kv_heads;
    const dim3 grid((unsigned)std::min<long long>((items + 7) / 8, 1 << 16), 2);
    void (*f)(Kv8CopyArgs) = c.head_dim == 128 ? (to_cache ? kv8_copy_kernel<128, true> : kv8_copy_kernel<128, false>)
                                               : (to_cache ? kv8_copy_kernel<64, true> : kv8_copy_kernel<64, false>);
    const cudaError_t e = launch_k(m->pdl, f, grid, dim3(256), 0, st, a);
    ++m->launches;
    return check_cuda(e, "8-bit cache copy launch");
}

int launch_append(spec_kv* kv, int layer, const AttendSpan& span, const void* k, long long k_stride, const void* v,
                  long long v_stride, cudaStream_t st) {
    spec_model* m = kv->m;
    const spec_model_config& c = m->cfg;
    const size_t off = (size_t)layer * kv->n_pages * c.n_kv_heads * kv->page;
    AppendArgs a{};
    a.src[0] = (const __nv_bfloat16*)k; a.src[1] = (const __nv_bfloat16*)v;
    a.stride[0] = k_stride; a.stride[1] = v_stride;
    for (int i = 0; i < 2; ++i) a.vec[i] = aligned16(a.src[i]) && a.stride[i] % 8 == 0;
    a.cache[0] = (char*)kv->k + off * c.head_dim * kv->elem;
    a.cache[1] = (char*)kv->v + off * c.head_dim * kv->elem;
    a.exps[0] = kv->q8 ? kv->ke + off : nullptr;
    a.exps[1] = kv->q8 ? kv->ve + off : nullptr;
    a.pages = kv->pages();
    a.len = kv->len;
    a.cap = kv->max_ctx;
    a.Hkv = c.n_kv_heads;
    a.err = m->err;
    a.span = span;
    const int per = 128 / (c.head_dim / 8);
    const dim3 grid((span.T * c.n_kv_heads + per - 1) / per, 2);
    cudaError_t e = launch_k(m->pdl, c.head_dim == 128 ? append_kernel<128> : append_kernel<64>, grid, dim3(128), 0, st, a);
    ++m->launches;
    return check_cuda(e, "cache append launch");
}

}  // namespace spec
