// Attention of a batch whose sequences may continue one shared prompt, and the
// 8-bit form of a KV cache: structures shared by the translation units.
//
// 8-bit form of one cached row x[hd] (a slot of one KV head, K or V): the
// exponent e is the least integer with max|x| <= 448 * 2^e (448: the largest
// e4m3 value), kept in [-124, 119]; the row is held as e4m3(x * 2^-e) (nearest,
// ties to even) and the byte e + 127, and stands for y * 2^e.  A power of two
// costs an e4m3 value nothing (only values below 2^-14 of the row's largest
// meet the format's subnormal end, at most one bit sooner than under an exact
// max/448 scale), and in this range of exponents every y * 2^e is a bf16
// number: reading back, and converting a tile for a bf16 matrix product, are
// exact.  Infinities count as no magnitude and saturate; NaN stays NaN.
#pragma once

#include "model.cuh"

namespace spec {

// The rows of one call: rows [row0[b], row0[b + 1]) are sequence b's, its row j
// in slot len[b] + extra + j.  Row j sees the sequence's slots below
// len[b] + extra and the rows of its mask.
struct AttendSpan {
    int batch, T, max_rows;
    int extra;
    int tree;                                  // 0 chain, 1 mask[] for every sequence, 2 parents on the device
    const int* dev_parent;                     // tree 2: [batch][kMaxSeqRows]
    short row0[kMaxPlanBatch + 1];
    unsigned long long mask[kMaxSeqRows];      // tree 1: bit x of mask[j]: row j sees row x
};

// One layer of one cache as the attention reads it.
struct CacheView {
    const void* k; const void* v;              // first row of the layer
    const uint8_t* ke; const uint8_t* ve;      // exponents (8-bit caches)
    KVPages pages;
    const int* len;
    int cap;                                   // slots a sequence can address
    int q8;
};

CacheView cache_view(const spec_kv* kv, int layer);
// span of a call with n_rows[b] rows of sequence b
int make_span(AttendSpan* s, int batch, const int* n_rows, int extra, const int* tree_parent, const int* dev_parent);

// Parameters of the attention kernels.  Ranges of keys leave partial states:
// the prompt's ranges first, then each sequence's own.
struct AttendArgs {
    const void* q;
    int q_f32;                        // f32 queries (else bf16)
    int q_vec;                        // bf16 queries: rows are 16-byte aligned
    long long q_stride;
    float c;                          // scale * log2(e)
    CacheView own, pre;
    int pre_seq;                      // sequence of the prompt in its cache
    int layer;
    int H, Hkv;
    AttendSpan span;
    int own_splits, pre_splits;       // key ranges; pre_splits is 0 where the tile kernel takes the prompt
    int tile_ctas;                    // the tile kernel's CTAs a pair of query tiles (at most: tile_ctas_at_work)
    int own_qb, pre_qb;               // query blocks of 16
    float* part_o;                    // [range][T * H][hd]
    float* part_ml;                   // [range][T * H][2]
    int own_range0;                   // first range of the own part
    int* err;
};

SPEC_DEV float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// two f32 lanes in one instruction
SPEC_DEV float2 fma2(float2 x, float2 y, float2 z) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, r;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 r, a, b, c;\n\tmov.b64 {%0, %1}, r;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
    return d;
}
SPEC_DEV float2 mul2(float2 x, float2 y) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, r;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 r, a, b;\n\tmov.b64 {%0, %1}, r;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
    return d;
}
SPEC_DEV float2 add2(float2 x, float2 y) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, r;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 r, a, b;\n\tmov.b64 {%0, %1}, r;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
    return d;
}

// attend_tile.cu: the prompt's part for lists of many query vectors
bool attend_tile_ok(const spec_kv* pre);
int attend_tile_ctas(const spec_model* m, const AttendSpan& span, bool q_f32, int prompt_cap);
int attend_tile_ranges(const spec_model* m, int ctas);      // most ranges of one KV head
// a / b of numbers >= 0; nearly always a division of 32 bits, a third of the other's instructions
SPEC_DEV long long quotient(long long a, long long b) {
    return ((a | b) >> 32) ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}
// CTAs that share W key tiles: the host's count, chosen for a full cache, or one a tile where the prompt
// has fewer tiles, so that none is without keys and every range that the join counts is written.
SPEC_DEV int tile_ctas_at_work(int ctas, long long W) { return W < ctas ? (int)W : ctas; }
// Of n <= W CTAs that share the W = Hkv KB key tiles of all heads evenly (CTA j from j W / n on),
// the one that holds head g's first.  Its range of the head is range 0, the next one's range 1, ...
SPEC_DEV int tile_first_cta(int g, int KB, long long W, int n) { return (int)quotient(((long long)g * KB + 1) * n - 1, W); }
SPEC_DEV int tile_range_count(int g, int KB, long long W, int n) {
    return KB == 0 ? 0 : (int)quotient((long long)(g + 1) * KB * n - 1, W) - tile_first_cta(g, KB, W, n) + 1;
}
int launch_attend_tile(const spec_kv* pre, const AttendArgs& a, cudaStream_t st);

// Where the attention's result goes: bf16 rows of the caller, or the model's
// O-projection input (hi rows, then lo rows at out_lo).
struct AttendOut { __nv_bfloat16* p; long long stride; size_t lo; };

// rows [T][Hkv][hd] (strides in elements) into layer `layer` of kv at their slots
int launch_append(spec_kv* kv, int layer, const AttendSpan& span, const void* k, long long k_stride, const void* v,
                  long long v_stride, cudaStream_t st);
// q: bf16 (q_f32 = 0) or f32 rows of [H][hd], stride in elements; scores are q.k * scale
int launch_attend(spec_kv* kv, int layer, const AttendSpan& span, const void* q, int q_f32, long long q_stride,
                  float scale, const AttendOut& out, cudaStream_t st);
// floats of workspace that launch_attend may use in a model of this shape
size_t attend_floats_needed(const spec_model* m);
// 8-bit cache <-> bf16 rows [n_layers][n_slots][Hkv][hd] of one sequence
int launch_kv8_copy(spec_kv* kv, int seq, int layer0, int n_layers, int slot0, int n_slots, void* k, void* v,
                    bool to_cache, cudaStream_t st);

// ---------------------------------------------------------------------------
// the 8-bit form

// largest finite magnitude of 8 values
SPEC_DEV float finite_amax(const float (&x)[8]) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float t = fabsf(x[i]);
        a = fmaxf(a, t <= 3.4028234e38f ? t : 0.f);
    }
    return a;
}
// exponent byte e + 127 of a row whose largest magnitude is amax
SPEC_DEV int kv8_exp(float amax) {
    const uint32_t b = __float_as_uint(amax);
    int e = (int)(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);   // biased; 448 = 1.75 * 2^8
    return min(max(e, 127 - 124), 127 + 119);
}
SPEC_DEV float kv8_scale(int ebyte) { return __uint_as_float((uint32_t)ebyte << 23); }            // 2^e
SPEC_DEV float kv8_inv_scale(int ebyte) { return __uint_as_float((uint32_t)(254 - ebyte) << 23); }  // 2^-e
SPEC_DEV uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
SPEC_DEV uint2 e4m3x8(const float (&x)[8], float inv) {
    uint2 r;
    r.x = e4m3x2(x[0] * inv, x[1] * inv) | (e4m3x2(x[2] * inv, x[3] * inv) << 16);
    r.y = e4m3x2(x[4] * inv, x[5] * inv) | (e4m3x2(x[6] * inv, x[7] * inv) << 16);
    return r;
}
// two e4m3 values as floats (exact)
SPEC_DEV float2 e4m3x2_f32(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    float2 f;
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
        : "=f"(f.x), "=f"(f.y) : "r"(h));
    return f;
}
// two e4m3 values as f16 (exact)
SPEC_DEV uint32_t e4m3x2_f16(uint32_t two) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
    return h;
}
SPEC_DEV uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
SPEC_DEV float f16_round(float x) {
    float r;
    asm("{\n\t.reg .b16 h;\n\tcvt.rn.f16.f32 h, %1;\n\tcvt.f32.f16 %0, h;\n\t}" : "=f"(r) : "f"(x));
    return r;
}
SPEC_DEV uint32_t f16x2_mul(uint32_t x, uint32_t y) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    return r;
}
// two floats to bf16x2, `lo` in the low half
SPEC_DEV uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

}  // namespace spec
