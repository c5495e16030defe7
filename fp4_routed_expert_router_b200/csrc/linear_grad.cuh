// linear_grad.cuh -- the elementwise half of the backward pass: dz = dy act'(z)
// (SwiGLU: dz and dz_up) rounded once to 16 bits, and db = sum of dz over the
// rows of each group, taken before the rounding.
//
// Bound by memory: dy, z (z_up) read once, dz (dz_up) written once.  A CTA owns
// 64 columns and a strip of rows, each thread VEC = 8 consecutive columns (one
// 16-byte access per row; VEC = 1 when a base or row stride is not 16-byte
// aligned).  Column sums stay in the thread's fp32 registers, meet in shared
// memory in a fixed order and, when a group's rows are split over the CTAs of a
// cluster, in the first CTA's shared memory, again in a fixed order: no atomics
// and no workspace, and the same bits every time.
#pragma once
#include <cooperative_groups.h>

#include "linear_common.cuh"

namespace moe {

struct LinGradArgs {
    const int32_t* offsets;   // NULL: rows [0, rows)
    int E, rows, N, type, act;
    const int32_t* dy_rows;
    int dy_total, dy_type;
    const void* dy;
    long long lddy;
    const void* z[2];
    long long ldz;
    void* dz[2];              // may be NULL (only db is wanted)
    long long lddz;
    int packed;               // rows of dz at lin_packed, zeros behind each group up to the next multiple of 16
    float* db[2];
    int accumulate;
    int* err;
};

constexpr int kLgCols = 64, kLgThreads = 256;

template <int VEC>
__device__ __forceinline__ void lg_load(const void* p, size_t at, int type, float v[VEC]) {
    if constexpr (VEC == 1) {
        v[0] = lin_load(p, at, type);
    } else if (type == LIN_F32) {
        const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) {
            const float4 t = __ldcg(f + i);
            v[4 * i] = t.x; v[4 * i + 1] = t.y; v[4 * i + 2] = t.z; v[4 * i + 3] = t.w;
        }
    } else {
        const uint4 t = __ldcg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at));
        const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            const uint16_t lo = w[i] & 0xFFFF, hi = w[i] >> 16;
            v[2 * i] = type == LIN_BF16 ? bf16_to_f32(lo) : __half2float(__ushort_as_half(lo));
            v[2 * i + 1] = type == LIN_BF16 ? bf16_to_f32(hi) : __half2float(__ushort_as_half(hi));
        }
    }
}

template <int VEC>
__device__ __forceinline__ void lg_store(void* p, size_t at, int type, const float v[VEC]) {
    uint16_t* d = static_cast<uint16_t*>(p) + at;
    if constexpr (VEC == 1) {
        d[0] = lin_cvt16(v[0], type);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i)
            w[i] = static_cast<uint32_t>(lin_cvt16(v[2 * i], type)) |
                   (static_cast<uint32_t>(lin_cvt16(v[2 * i + 1], type)) << 16);
        *reinterpret_cast<uint4*>(d) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// grid (column blocks, row strips, groups); with db the strips of a group form one cluster.  Without db and without
// packing the rows of all groups are strips of one.
template <int VEC, bool UP>
__global__ void __launch_bounds__(kLgThreads) lin_grad_kernel(const LinGradArgs a) {
    namespace cg = cooperative_groups;
    constexpr int TX = kLgCols / VEC, TY = kLgThreads / TX;
    __shared__ float part[UP ? 2 : 1][kLgThreads * VEC];   // [row lane][column]
    __shared__ float sums[UP ? 2 : 1][kLgCols];
    pdl_wait();
    pdl_trigger();
    const int e = blockIdx.z, tx = threadIdx.x % TX, ty = threadIdx.x / TX;
    const int c = blockIdx.x * kLgCols + tx * VEC;
    const bool on = c < a.N;   // VEC divides N on the vector path
    const bool want_db = a.db[0] != nullptr || a.db[1] != nullptr;
    int p0, p1;
    bool ok = true;
    if (want_db || a.packed || !a.offsets) {
        ok = lin_group(a.offsets, a.rows, e, a.err, &p0, &p1);
    } else {   // the groups do not matter: the rows of all of them
        p0 = max(0, min(a.rows, __ldg(a.offsets)));
        p1 = max(p0, min(a.rows, __ldg(a.offsets + a.E)));
    }
    const int S = gridDim.y, strip = blockIdx.y;
    const int per = (p1 - p0 + S - 1) / S;
    const int r_lo = p0 + min(p1 - p0, strip * per), r_hi = min(p1, r_lo + per);
    // first row of the strip's rows in dz, from r = 0 on
    const long long g0 = a.packed ? static_cast<long long>(lin_packed(p0, e)) - p0 : 0;
    if (a.packed && ok && strip == 0 && on) {   // zeros behind the group
        const int end = p1 - p0 + ((p0 - p1) & 15);
        float zero[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) zero[i] = 0.0f;
        for (int r = p1 - p0 + ty; r < end; r += TY) {
            const size_t gi = static_cast<size_t>(g0 + p0 + r) * a.lddz + c;
            lg_store<VEC>(a.dz[0], gi, a.type, zero);
            if (UP) lg_store<VEC>(a.dz[1], gi, a.type, zero);
        }
    }
    float s0[VEC], s1[UP ? VEC : 1];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        s0[i] = 0.0f;
        if (UP) s1[i] = 0.0f;
    }
    constexpr int U = VEC == 1 ? 4 : 2;   // rows whose loads are in flight together
    for (int r0 = r_lo + ty; r0 < r_hi; r0 += U * TY) {
        float dy[U][VEC], z[U][VEC], u[UP ? U : 1][VEC];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int r = r0 + k * TY;
            const int src = r < r_hi ? lin_index(a.dy_rows, a.dy_total, r, a.err) : -1;
            const size_t zi = static_cast<size_t>(r) * a.ldz + c;
#pragma unroll
            for (int i = 0; i < VEC; ++i) dy[k][i] = z[k][i] = 0.0f;
            if (on && src >= 0) lg_load<VEC>(a.dy, static_cast<size_t>(src) * a.lddy + c, a.dy_type, dy[k]);
            if (on && r < r_hi && a.act != LACT_NONE) lg_load<VEC>(a.z[0], zi, a.type, z[k]);
            if (UP) {
                if (on && r < r_hi) lg_load<VEC>(a.z[1], zi, a.type, u[UP ? k : 0]);
            }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int r = r0 + k * TY;
            if (!on || r >= r_hi) continue;
            const size_t gi = static_cast<size_t>(g0 + r) * a.lddz + c;
            float g[VEC];
            if (UP) {
                float gu[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float sg = 1.0f / (1.0f + expf(-z[k][i]));
                    gu[i] = dy[k][i] * (z[k][i] * sg);
                    g[i] = dy[k][i] * u[UP ? k : 0][i] * (sg * (1.0f + z[k][i] * (1.0f - sg)));
                    s0[i] += g[i];
                    s1[UP ? i : 0] += gu[i];
                }
                if (a.dz[1]) lg_store<VEC>(a.dz[1], gi, a.type, gu);
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    g[i] = a.act == LACT_NONE ? dy[k][i] : dy[k][i] * lin_slope(a.act, z[k][i]);
                    s0[i] += g[i];
                }
            }
            if (a.dz[0]) lg_store<VEC>(a.dz[0], gi, a.type, g);
        }
    }
    if (!want_db) return;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        part[0][ty * kLgCols + tx * VEC + i] = s0[i];
        if constexpr (UP) part[1][ty * kLgCols + tx * VEC + i] = s1[i];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < (UP ? 2 : 1) * kLgCols; i += kLgThreads) {
        const int w = i / kLgCols, col = i % kLgCols;
        float t = 0.0f;
        for (int y = 0; y < TY; ++y) t += part[w][y * kLgCols + col];
        sums[w][col] = t;
    }
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();
    if (cl.block_rank() == 0 && ok) {
        for (int i = threadIdx.x; i < (UP ? 2 : 1) * kLgCols; i += kLgThreads) {
            const int w = i / kLgCols, col = i % kLgCols, cc = blockIdx.x * kLgCols + col;
            float t = 0.0f;
            for (unsigned k = 0; k < cl.num_blocks(); ++k) t += *cl.map_shared_rank(&sums[w][col], k);
            if (cc < a.N && a.db[w]) {
                float* d = a.db[w] + static_cast<size_t>(e) * a.N + cc;
                *d = a.accumulate ? *d + t : t;
            }
        }
    }
    cl.sync();   // the first CTA has read the others' sums
}

}  // namespace moe
