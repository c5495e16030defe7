// linear_simple.cuh -- the 16-bit products on the fp32 cores: any size, row
// stride and alignment.  One CTA computes 64 output rows x 64 columns with 256
// threads, 4 x 4 values each, over slabs of 16 terms staged in shared memory as
// fp32.  Bound by the fp32 pipes (two shared-memory reads per eight FMAs).
#pragma once
#include "linear_common.cuh"

namespace moe {

constexpr int kLsTile = 64, kLsSlab = 16;

// grid: (C tiles, row tiles over all groups (upper bound), wgrad: outputs * groups, else 1)
template <bool DUAL>
__global__ void __launch_bounds__(256) lin_simple_kernel(const LinArgs a) {
    __shared__ float As[kLsSlab][kLsTile + 4], Au[DUAL ? kLsSlab : 1][kLsTile + 4], Bs[kLsSlab][kLsTile + 4];
    __shared__ int find_s[4];
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x;
    const bool wg = a.kind == LIN_WGRAD;
    const int c0 = blockIdx.x * kLsTile;
    int e, r0, nrows, p0 = 0, p1 = 0, which = 0;
    if (wg) {
        e = blockIdx.z % a.E;
        which = blockIdx.z / a.E;
        if (!lin_group(a.offsets, a.rows, e, a.err, &p0, &p1)) return;
        r0 = blockIdx.y * kLsTile;
        nrows = min(kLsTile, a.out_n - r0);
    } else {
        if (tid == 0) {   // the group of row tile blockIdx.y
            int left = blockIdx.y;
            find_s[0] = -1;
            for (int g = 0; g < a.E; ++g) {
                int q0, q1;
                if (!lin_group(a.offsets, a.rows, g, a.err, &q0, &q1)) continue;
                const int t = (q1 - q0 + kLsTile - 1) / kLsTile;
                if (left < t) {
                    find_s[0] = g;
                    find_s[1] = q0 + left * kLsTile;
                    find_s[2] = min(kLsTile, q1 - find_s[1]);
                    break;
                }
                left -= t;
            }
        }
        __syncthreads();
        e = find_s[0];
        if (e < 0) return;
        r0 = find_s[1];
        nrows = find_s[2];
    }
    const int Q = wg ? p1 - p0 : a.Q;
    const int ncols = min(kLsTile, a.C - c0);
    const int tx = tid & 15, ty = tid >> 4;
    float acc[4][4] = {}, accu[DUAL ? 4 : 1][4] = {};
    const int parts = (a.kind == LIN_DGRAD && a.b[1]) ? 2 : 1;
    for (int part = 0; part < parts; ++part) {
        const void* pa = wg ? a.a[0] : a.a[part];
        const void* pb = wg ? a.b[which] : a.b[part];
        const size_t abase = wg ? 0 : static_cast<size_t>(e) * a.a_gstride;
        for (int q0 = 0; q0 < Q; q0 += kLsSlab) {
            for (int i = tid; i < kLsSlab * kLsTile; i += 256) {
                // walk the contiguous index of each operand fastest
                int q, c;
                if (a.kind == LIN_FWD) { q = i % kLsSlab; c = i / kLsSlab; } else { c = i % kLsTile; q = i / kLsTile; }
                const int qq = q0 + q;
                float v = 0.0f, u = 0.0f;
                if (qq < Q && c < ncols) {
                    if (a.kind == LIN_FWD) {
                        const size_t at = abase + static_cast<size_t>(c0 + c) * a.lda + qq;
                        v = lin_load(pa, at, a.type);
                        if (DUAL) u = lin_load(a.a[1], at, a.type);
                    } else if (a.kind == LIN_DGRAD) {
                        v = lin_load(pa, abase + static_cast<size_t>(qq) * a.lda + c0 + c, a.type);
                    } else {
                        const int src = lin_index(a.gather, a.gather_total, p0 + qq, a.err);
                        if (src >= 0) v = lin_load(pa, static_cast<size_t>(src) * a.lda + c0 + c, a.type);
                    }
                }
                As[q][c] = v;
                if (DUAL) Au[q][c] = u;
            }
            for (int i = tid; i < kLsSlab * kLsTile; i += 256) {
                int q, r;
                if (!wg) { q = i % kLsSlab; r = i / kLsSlab; } else { r = i % kLsTile; q = i / kLsTile; }
                const int qq = q0 + q;
                float v = 0.0f;
                if (qq < Q && r < nrows) {
                    if (wg) {
                        v = lin_load(pb, static_cast<size_t>(p0 + qq) * a.ldb + r0 + r, a.type);
                    } else {
                        const int src = a.kind == LIN_FWD ? lin_index(a.gather, a.gather_total, r0 + r, a.err) : r0 + r;
                        if (src >= 0) v = lin_load(pb, static_cast<size_t>(src) * a.ldb + qq, a.type);
                    }
                }
                Bs[q][r] = v;
            }
            __syncthreads();
#pragma unroll
            for (int q = 0; q < kLsSlab; ++q) {
                float av[4], uv[4], bv[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    av[i] = As[q][tx + 16 * i];
                    if (DUAL) uv[i] = Au[q][tx + 16 * i];
                    bv[i] = Bs[q][ty * 4 + i];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        acc[i][j] = fmaf(av[j], bv[i], acc[i][j]);
                        if (DUAL) accu[i][j] = fmaf(uv[j], bv[i], accu[i][j]);
                    }
            }
            __syncthreads();
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = ty * 4 + i;
        if (r >= nrows) continue;
        const int orow = wg ? 0 : lin_index(a.scatter, a.scatter_total, r0 + r, a.err);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = tx + 16 * j;
            if (c >= ncols) continue;
            if (wg) {
                const size_t o = static_cast<size_t>(e) * a.o_gstride + static_cast<size_t>(r0 + r) * a.ldo + c0 + c;
                float v = acc[i][j];
                if (a.accumulate) v += lin_load(a.out[which], o, a.out_type);
                lin_store(a.out[which], o, v, a.out_type);
            } else {
                lin_finish(a, e, r0 + r, orow, c0 + c, acc[i][j], DUAL ? accu[i][j] : 0.0f);
            }
        }
    }
}

}  // namespace moe
