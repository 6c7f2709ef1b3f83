// Rows of logits: segments of a row as a warp reads them, shared by the kernels over the vocabulary.
#pragma once

#include "attend.cuh"

namespace spec {

constexpr int kLpSeg = 256;

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

// a cluster barrier in two halves
SPEC_DEV void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
SPEC_DEV void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

}  // namespace spec
