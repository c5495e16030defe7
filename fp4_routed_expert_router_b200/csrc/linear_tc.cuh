// linear_tc.cuh -- the 16-bit products on the 5th-generation tensor cores
// (tcgen05 + TMEM), dense and grouped by expert.
//
// out[row][c] = sum_q A(q, c) B(q, row) (linear_common.cuh).  c, the contiguous
// index of the output, is the M side of tcgen05.mma: 128 TMEM lanes; the rows
// are its N side, BN <= 256 columns.  A warp of the epilogue therefore holds
// 32 neighbouring c of a row in its lanes and writes them straight to memory,
// with bias and activation per lane, and a handful of rows (decode) costs an
// MMA of N = 16 instead of a 128-row tile that is mostly empty.
//
// Operands in shared memory, 64 terms (q) a stage, 128-byte swizzle:
//   forward  A = w    K-major  (row c, 64 q)       B = x   K-major  (row, 64 q)
//   dgrad    A = w    MN-major (row q, 64 c) x 2   B = dz  K-major
//   wgrad    A = x    MN-major (row q, 64 c) x 2   B = dz  MN-major (row q, 64 rows) x BN / 64
// Both majors are read by the tensor core as they lie in memory, so nothing is
// transposed anywhere.  SwiGLU's forward keeps two accumulators (w, w_up) fed
// by one B; its dgrad runs on through a second pair (dz_up, w_up).
//
// Groups: rows of a tile belong to one group; a tile that ends inside a group's
// last rows reads what lies behind them into columns that are not stored.  In
// wgrad the group is the sum: its last stage runs only the 16-term steps it
// needs, and the up to 15 foreign rows in the last step are zeroed in both
// operands first (0 * inf would not be 0).
//
// One persistent CTA per SM.  Warps: 0 loads (TMA; with x_rows one
// tile::gather4 per four rows and lane), 1 issues the MMAs, 4-11 epilogue
// (TMEM lane group warp % 4, 16-column units shared by two warps), 12-15 (only
// for operands TMA cannot take: a base that is not 16-byte aligned or rows
// that are not multiples of 8 values) load element by element.  Two
// accumulators, so the epilogue of a tile overlaps the next one's products.
// Every wait is bounded; the first that gives up ends the CTA's other waits
// and latches ETIMEOUT, after the copies in flight have landed.
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>

#include "linear_common.cuh"
#include "tc_prefill.cuh"
#include "tma.cuh"

namespace moe {

constexpr int kLtM = 128;            // c of a tile (TMEM lanes)
constexpr int kLtBK = 64;            // terms per stage: one 128-byte swizzle row
constexpr int kLtATile = kLtM * 128; // bytes of one A tile of a stage
constexpr int kLtEpiWarps = 8;
constexpr int kLtMaxStages = 12;
constexpr int kLtPromote = 10;       // fp32 outputs: stages summed in the tensor core before the sum moves to registers
constexpr int kLtRaster = 8;         // row tiles walked together, so that operands of neighbouring tiles meet in L2
__host__ __device__ constexpr int lt_threads(bool tma) { return (4 + kLtEpiWarps + (tma ? 0 : 4)) * 32; }

struct LtPlan {
    int bn;         // output rows of a tile
    int bbox;       // rows of one K-major B box
    int stages, stage_bytes, off_ring, smem;
    int n_ct;       // tiles along c
    int promote;    // stages per accumulation span (0: the whole sum)
    int tmem_cols;
    int grid;
};

struct LtMaps {
    CUtensorMap a0, a1, b0, b1;
};

__device__ __forceinline__ uint64_t lt_desc_mn(uint32_t smem_addr) {
    // MN-major, 128-byte swizzle: 64-element blocks 8,192 bytes apart (LBO), groups of 8 q 1,024 apart (SBO)
    return static_cast<uint64_t>((smem_addr >> 4) & 0x3FFF) | (static_cast<uint64_t>(8192 >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
           (static_cast<uint64_t>(2) << 61);
}

// D fp32 (bits 4-5), operand type in bits 7-9 and 10-12 (0 f16, 1 bf16), bit 15 / 16: A / B is MN-major,
// N >> 3 at bits 17-22, M >> 4 at bits 24-28.
__device__ __forceinline__ uint32_t lt_idesc(int type, bool a_mn, bool b_mn, int n) {
    const uint32_t t = type == LIN_BF16 ? 1u : 0u;
    return (1u << 4) | (t << 7) | (t << 10) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
           (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(kLtM >> 4) << 24);
}

__device__ __forceinline__ void lt_mma(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
        : "memory");
}

__device__ __forceinline__ void lt_tma3(void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::
            "r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
        : "memory");
}

// Four rows (any rows) x 64 values; the map's box is one row high.
__device__ __forceinline__ void lt_gather4(void* dst, const CUtensorMap* map, int c0, int4 r, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w), "r"(smem_u32(bar))
        : "memory");
}

struct LtTile {
    int e, which;   // group, output (wgrad: dw or dw_up)
    int c0;         // first c
    int r0, nrows;  // first output row (forward, dgrad: grouped row; wgrad: row of the group's output), rows
    int p0, nq;     // wgrad: the group's first row and row count
    int nkb;        // stages
};

template <int KIND, bool DUAL, bool TMA>
__global__ void __launch_bounds__(lt_threads(TMA), 1)
lin_tc_kernel(const LinArgs a, const LtPlan p, const __grid_constant__ LtMaps maps) {
    constexpr bool WG = KIND == LIN_WGRAD;
    constexpr bool A_MN = KIND != LIN_FWD;
    constexpr int NACC = DUAL ? 2 : 1;
    extern __shared__ __align__(1024) uint8_t lt_smem_raw[];
    uint8_t* smem = lt_smem_raw + ((1024u - (smem_u32(lt_smem_raw) & 1023u)) & 1023u);
    const int S = p.stages, BN = p.bn;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem);
    uint64_t* empty = full + kLtMaxStages;
    uint64_t* acc_full = empty + kLtMaxStages;
    uint64_t* acc_empty = acc_full + 2;
    int* tprefix = reinterpret_cast<int*>(smem + 512);   // [E+1] tiles before group e (forward, dgrad)
    __shared__ uint32_t tmem_base_s;
    __shared__ int abort_s;
    volatile int* abort_flag = &abort_s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], TMA ? 1 : 4);
            mbar_init(&empty[s], 1);
        }
        for (int q = 0; q < 2; ++q) {
            mbar_init(&acc_full[q], 1);
            mbar_init(&acc_empty[q], kLtEpiWarps);
        }
        abort_s = 0;
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base_s)),
                     "r"(static_cast<uint32_t>(p.tmem_cols)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    pdl_wait();
    if (!WG && warp == 0) {   // tiles before each group
        int work = 0;
        for (int base = 0; base < a.E; base += 32) {
            const int e = base + lane;
            int p0 = 0, p1 = 0;
            if (e < a.E) lin_group(a.offsets, a.rows, e, a.err, &p0, &p1);
            const int mine = (p1 - p0 + BN - 1) / BN * p.n_ct;
            int incl = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
                if (lane >= o) incl += v;
            }
            if (e < a.E) tprefix[e] = work + incl - mine;
            work += __shfl_sync(0xFFFFFFFFu, incl, 31);
        }
        if (lane == 0) tprefix[a.E] = work;
    }
    if (tid == 0) fence_barrier_init();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_trigger();
    const uint32_t tmem = tmem_base_s;
    const int n_rt_w = WG ? (a.out_n + BN - 1) / BN : 0;
    const int n_work = WG ? p.n_ct * n_rt_w * a.E * (a.b[1] ? 2 : 1) : tprefix[a.E];
    const int G = gridDim.x;

    // Tile w of the walk; false when its group is not sound (nothing is computed or written).
    auto tile_of = [&](int w, LtTile& t) -> bool {
        int v, n_rt;
        t.which = 0;
        if (WG) {
            const int per = p.n_ct * n_rt_w;
            const int ve = w / per;
            v = w - ve * per;
            t.e = ve % a.E;
            t.which = ve / a.E;
            n_rt = n_rt_w;
            int p1;
            if (!lin_group(a.offsets, a.rows, t.e, a.err, &t.p0, &p1)) return false;
            t.nq = p1 - t.p0;
            t.nkb = (t.nq + kLtBK - 1) / kLtBK;
        } else {
            int lo = 0, hi = a.E - 1;   // the last group that starts at or before w (empty groups start where they end)
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (tprefix[mid] <= w) lo = mid; else hi = mid - 1;
            }
            t.e = lo;
            v = w - tprefix[lo];
            n_rt = (tprefix[lo + 1] - tprefix[lo]) / p.n_ct;
            t.p0 = 0;
            t.nq = a.Q;
            t.nkb = (a.Q + kLtBK - 1) / kLtBK * (KIND == LIN_DGRAD && a.b[1] ? 2 : 1);
        }
        const int blk = v / (kLtRaster * p.n_ct);
        v -= blk * kLtRaster * p.n_ct;
        const int in_blk = min(kLtRaster, n_rt - blk * kLtRaster);
        t.c0 = v / in_blk * kLtM;
        const int rt = blk * kLtRaster + v % in_blk;
        if (WG) {
            t.r0 = rt * BN;
            t.nrows = min(BN, a.out_n - t.r0);
        } else {
            int p0 = 0, p1 = a.rows;
            if (a.offsets) {
                p0 = __ldg(a.offsets + t.e);
                p1 = __ldg(a.offsets + t.e + 1);
            }
            t.r0 = p0 + rt * BN;
            t.nrows = min(BN, p1 - t.r0);
        }
        return true;
    };
    auto stage_a = [&](int st) { return smem + p.off_ring + static_cast<size_t>(st) * p.stage_bytes; };
    auto stage_b = [&](int st) { return stage_a(st) + NACC * kLtATile; };
    const int half_kb = (a.Q + kLtBK - 1) / kLtBK;   // dgrad: stages of the first pair

    if (TMA && warp == 0) {
        // ------------------------------------------------------------ TMA producer
        int g = 0;
        bool stop = false;
        for (int w = blockIdx.x; w < n_work && !stop; w += G) {
            LtTile t;
            if (!tile_of(w, t)) continue;
            const int nbox = WG ? (t.nrows + 63) / 64 : (t.nrows + p.bbox - 1) / p.bbox;
            const int nquad = (t.nrows + 3) / 4;
            const bool gather = a.gather != nullptr && KIND != LIN_DGRAD;
            const uint32_t bytes =
                static_cast<uint32_t>(NACC * kLtATile + (WG ? nbox * 8192 : gather ? nquad * 512 : nbox * p.bbox * 128));
            int4 idx[2];
            if (KIND == LIN_FWD && gather) {   // rows 4 lane .. and 128 + 4 lane .. of the tile (clamped; not stored)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    int* ip = reinterpret_cast<int*>(&idx[h]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = t.r0 + min(t.nrows - 1, 128 * h + 4 * lane + j);
                        const int v = __ldg(a.gather + r);
                        ip[j] = v >= 0 && v < a.gather_total ? v : 0;
                    }
                }
            }
            for (int kb = 0; kb < t.nkb; ++kb, ++g) {
                const int st = g % S;
                int ok = 1;
                if (g >= S && lane == 0) ok = mbar_poll(&empty[st], ((g / S) - 1) & 1, abort_flag, a.timeout_ns);
                if (!__shfl_sync(0xFFFFFFFFu, ok, 0)) {
                    if (lane == 0) latch_error(a.err, ERR_ETIMEOUT, g, KID_LINEAR);
                    stop = true;
                    break;
                }
                uint8_t* sa = stage_a(st);
                uint8_t* sb = stage_b(st);
                if (lane == 0) {
                    mbar_arrive_expect_tx(&full[st], bytes);
                    if (KIND == LIN_FWD) {
                        lt_tma3(sa, &maps.a0, kb * kLtBK, t.c0, t.e, &full[st]);
                        if (DUAL) lt_tma3(sa + kLtATile, &maps.a1, kb * kLtBK, t.c0, t.e, &full[st]);
                        if (!gather)
                            for (int b = 0; b < nbox; ++b)
                                lt_tma3(sb + b * p.bbox * 128, &maps.b0, kb * kLtBK, t.r0 + b * p.bbox, 0, &full[st]);
                    } else if (KIND == LIN_DGRAD) {
                        const bool second = kb >= half_kb;
                        const int q = (second ? kb - half_kb : kb) * kLtBK;
                        const CUtensorMap* ma = second ? &maps.a1 : &maps.a0;
                        const CUtensorMap* mb = second ? &maps.b1 : &maps.b0;
                        lt_tma3(sa, ma, t.c0, q, t.e, &full[st]);
                        lt_tma3(sa + 8192, ma, t.c0 + 64, q, t.e, &full[st]);
                        for (int b = 0; b < nbox; ++b)
                            lt_tma3(sb + b * p.bbox * 128, mb, q, t.r0 + b * p.bbox, 0, &full[st]);
                    } else {
                        const CUtensorMap* mb = t.which ? &maps.b1 : &maps.b0;
                        if (!gather) {
                            lt_tma3(sa, &maps.a0, t.c0, t.p0 + kb * kLtBK, 0, &full[st]);
                            lt_tma3(sa + 8192, &maps.a0, t.c0 + 64, t.p0 + kb * kLtBK, 0, &full[st]);
                        }
                        for (int b = 0; b < nbox; ++b)
                            lt_tma3(sb + b * 8192, mb, t.r0 + b * 64, t.p0 + kb * kLtBK, 0, &full[st]);
                    }
                }
                __syncwarp();
                if (gather && KIND == LIN_FWD) {
                    if (lane < nquad) lt_gather4(sb + lane * 512, &maps.b0, kb * kLtBK, idx[0], &full[st]);
                    if (lane + 32 < nquad) lt_gather4(sb + (lane + 32) * 512, &maps.b0, kb * kLtBK, idx[1], &full[st]);
                } else if (gather && WG) {   // 16 quads of q rows x 2 blocks of 64 c: one per lane
                    int4 r;
                    int* ip = reinterpret_cast<int*>(&r);
                    const int quad = lane & 15, blk = lane >> 4;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int v = __ldg(a.gather + t.p0 + min(t.nq - 1, kb * kLtBK + 4 * quad + j));
                        const bool in = v >= 0 && v < a.gather_total;
                        if (!in) latch_error(a.err, ERR_EINVAL, v, KID_LINEAR);
                        ip[j] = in ? v : 0;
                    }
                    lt_gather4(sa + blk * 8192 + quad * 512, &maps.a0, t.c0 + 64 * blk, r, &full[st]);
                }
                __syncwarp();
            }
        }
        if (*abort_flag && lane == 0) {   // copies still in flight land before the CTA may exit
            volatile int fresh = 0;
            for (int st = 0; st < S && st < g; ++st) {
                const int last = st + ((g - 1 - st) / S) * S;
                fresh = 0;
                mbar_wait(&full[st], (last / S) & 1, &fresh);
            }
        }
    } else if (!TMA && warp >= 4 + kLtEpiWarps) {
        // ------------------------------------------------------------ element loader (128 threads)
        const int lt = tid - (4 + kLtEpiWarps) * 32;
        int g = 0;
        bool stop = false;
        for (int w = blockIdx.x; w < n_work && !stop; w += G) {
            LtTile t;
            if (!tile_of(w, t)) continue;
            for (int kb = 0; kb < t.nkb; ++kb, ++g) {
                const int st = g % S;
                int ok = 1;
                if (g >= S && lane == 0) ok = mbar_poll(&empty[st], ((g / S) - 1) & 1, abort_flag, a.timeout_ns);
                if (!__shfl_sync(0xFFFFFFFFu, ok, 0)) {
                    if (lane == 0) latch_error(a.err, ERR_ETIMEOUT, g, KID_LINEAR);
                    stop = true;
                    break;
                }
                const bool second = KIND == LIN_DGRAD && kb >= half_kb;
                const int q0 = (second ? kb - half_kb : kb) * kLtBK;
                const int nq = min(kLtBK, t.nq - q0);
                // a row of 64 contiguous values (zeros from n on; n <= 0 or no row: all zeros) into swizzled row `sr`
                // of a tile: half a warp per row, two rows a step
                auto put = [&](uint8_t* tile, int sr, int col, uint16_t v) {
                    *reinterpret_cast<uint16_t*>(tile + sr * 128 + (((col >> 3) ^ (sr & 7)) << 4) + (col & 7) * 2) = v;
                };
                auto fill = [&](uint8_t* tile, int rows, auto src_of, int n) {
                    for (int i = lt; i < rows * 64; i += 128) {
                        const int sr = i >> 6, col = i & 63;
                        const uint16_t* s = src_of(sr);
                        put(tile, sr, col, s && col < n ? __ldg(s + col) : static_cast<uint16_t>(0));
                    }
                };
                uint8_t* sa = stage_a(st);
                uint8_t* sb = stage_b(st);
                if (KIND == LIN_FWD) {
                    for (int m = 0; m < NACC; ++m) {
                        const uint16_t* base = static_cast<const uint16_t*>(a.a[m]) +
                                               static_cast<size_t>(t.e) * a.a_gstride + q0;
                        fill(sa + m * kLtATile, kLtM,
                             [&](int sr) -> const uint16_t* {
                                 return t.c0 + sr < a.C ? base + static_cast<size_t>(t.c0 + sr) * a.lda : nullptr;
                             }, nq);
                    }
                } else {
                    const uint16_t* base = static_cast<const uint16_t*>(a.a[second ? 1 : 0]) +
                                           (WG ? 0 : static_cast<size_t>(t.e) * a.a_gstride);
                    for (int blk = 0; blk < 2; ++blk) {
                        const int c = t.c0 + 64 * blk;
                        fill(sa + blk * 8192, kLtBK,
                             [&](int sr) -> const uint16_t* {
                                 if (sr >= nq) return nullptr;
                                 int row = q0 + sr;
                                 if (WG) row = lin_index(a.gather, a.gather_total, t.p0 + row, a.err);
                                 return row < 0 ? nullptr : base + static_cast<size_t>(row) * a.lda + c;
                             }, a.C - c);
                    }
                }
                const uint16_t* bb = static_cast<const uint16_t*>(a.b[WG ? t.which : second ? 1 : 0]);
                if (WG) {
                    for (int blk = 0; blk * 64 < t.nrows; ++blk)
                        fill(sb + blk * 8192, kLtBK,
                             [&](int sr) -> const uint16_t* {
                                 return sr < nq ? bb + static_cast<size_t>(t.p0 + q0 + sr) * a.ldb + t.r0 + 64 * blk
                                                : nullptr;
                             }, t.nrows - 64 * blk);
                } else {
                    fill(sb, t.nrows,
                         [&](int sr) -> const uint16_t* {
                             int row = t.r0 + sr;
                             if (KIND == LIN_FWD && a.gather) {
                                 const int v = __ldg(a.gather + row);
                                 row = v >= 0 && v < a.gather_total ? v : -1;
                             }
                             return row < 0 ? nullptr : bb + static_cast<size_t>(row) * a.ldb + q0;
                         }, nq);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[st]);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        int g = 0, acc = 0;
        for (int w = blockIdx.x; w < n_work; w += G) {
            LtTile t;
            if (!tile_of(w, t)) continue;
            const int n = (t.nrows + 15) / 16 * 16;
            const uint32_t idesc = lt_idesc(a.type, A_MN, WG, n);
            const int span = p.promote ? p.promote : t.nkb;
            for (int k0 = 0; k0 < t.nkb; k0 += span, ++acc) {
                const int ab = acc & 1;
                if (acc >= 2 && !mbar_poll(&acc_empty[ab], ((acc >> 1) - 1) & 1, abort_flag, a.timeout_ns) && lane == 0)
                    latch_error(a.err, ERR_ETIMEOUT, acc, KID_LINEAR);
                tc_fence_after();
                const uint32_t d = tmem + ab * (NACC * BN);
                const int k1 = min(t.nkb, k0 + span);
                for (int kb = k0; kb < k1; ++kb, ++g) {
                    const int st = g % S;
                    if (!mbar_poll(&full[st], (g / S) & 1, abort_flag, a.timeout_ns) && lane == 0)
                        latch_error(a.err, ERR_ETIMEOUT, g, KID_LINEAR);
                    int steps = kLtBK / 16;
                    if (WG) {
                        const int valid = t.nq - kb * kLtBK;
                        if (valid < kLtBK) {   // the group's last stage
                            steps = (valid + 15) / 16;
                            if (TMA && (valid & 15)) {   // foreign rows of the last step, in every 64-wide block
                                const int nz = steps * 16 - valid, blocks = 2 + (t.nrows + 63) / 64;
                                uint8_t* base = stage_a(st) + valid * 128;
                                for (int i = lane; i < blocks * nz * 8; i += 32)
                                    *reinterpret_cast<uint4*>(base + (i / (nz * 8)) * 8192 + (i % (nz * 8)) * 16) =
                                        make_uint4(0, 0, 0, 0);
                                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                                __syncwarp();
                            }
                        }
                    }
                    tc_fence_after();
                    if (lane == 0) {
                        const uint32_t sa = smem_u32(stage_a(st)), sb = smem_u32(stage_b(st));
                        const uint64_t ad = A_MN ? lt_desc_mn(sa) : umma_desc_sw128(sa);
                        const uint64_t bd = WG ? lt_desc_mn(sb) : umma_desc_sw128(sb);
                        for (int k = 0; k < steps; ++k) {   // 16 terms: 32 bytes of a K-major row, 16 rows of MN-major
                            const uint64_t ak = ad + static_cast<uint64_t>(A_MN ? 128 * k : 2 * k);
                            const uint64_t bk = bd + static_cast<uint64_t>(WG ? 128 * k : 2 * k);
                            const uint32_t on = kb > k0 || k > 0 ? 1u : 0u;
                            lt_mma(d, ak, bk, idesc, on);
                            if (DUAL) lt_mma(d + BN, ak + (kLtATile >> 4), bk, idesc, on);
                        }
                        umma_commit(&empty[st]);
                    }
                    __syncwarp();
                }
                if (lane == 0) umma_commit(&acc_full[ab]);
                __syncwarp();
            }
        }
        for (int k = 1; k <= 2; ++k)   // the last commits land before TMEM is released
            if (acc >= k && lane == 0) {
                volatile int fresh = 0;
                mbar_wait(&acc_full[(acc - k) & 1], ((acc - k) >> 1) & 1, &fresh);
            }
    } else if (warp >= 4 && warp < 4 + kLtEpiWarps) {
        // ------------------------------------------------------------ epilogue
        const int lg = warp & 3, uh = (warp - 4) >> 2;
        const uint32_t lane_addr = static_cast<uint32_t>(32 * lg) << 16;
        const bool pair_out = a.out_type != LIN_F32 && ((a.C | a.ldo | a.o_gstride) & 1) == 0 &&
                              (reinterpret_cast<uintptr_t>(a.out[0]) & 3) == 0 &&
                              (reinterpret_cast<uintptr_t>(a.out[1]) & 3) == 0;
        const bool pair_z = ((a.C | a.ldz) & 1) == 0 && (reinterpret_cast<uintptr_t>(a.z[0]) & 3) == 0 &&
                            (reinterpret_cast<uintptr_t>(a.z[1]) & 3) == 0;
        // 16 rows of this lane's c.  16-bit values of two rows are exchanged between neighbouring lanes so that a
        // store carries two values: 64 bytes of each of two rows per instruction.
        auto store16 = [&](void* ptr, long long ld, int type, bool pair, int row, int c, const float (&v)[16]) {
            const bool on = c < a.C;
            if (type == LIN_F32) {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int o = __shfl_sync(0xFFFFFFFFu, row, j);
                    if (o >= 0 && on) static_cast<float*>(ptr)[static_cast<size_t>(o) * ld + c] = v[j];
                }
            } else if (pair) {
                const bool odd = lane & 1;
#pragma unroll
                for (int j = 0; j < 16; j += 2) {
                    const float got = __shfl_xor_sync(0xFFFFFFFFu, odd ? v[j] : v[j + 1], 1);
                    const float lo = odd ? got : v[j], hi = odd ? v[j + 1] : got;
                    const int o = __shfl_sync(0xFFFFFFFFu, row, j + (odd ? 1 : 0));
                    const uint32_t u = static_cast<uint32_t>(lin_cvt16(lo, type)) |
                                       (static_cast<uint32_t>(lin_cvt16(hi, type)) << 16);
                    if (o >= 0 && on)
                        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(ptr) + static_cast<size_t>(o) * ld +
                                                     (c & ~1)) = u;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int o = __shfl_sync(0xFFFFFFFFu, row, j);
                    if (o >= 0 && on)
                        static_cast<uint16_t*>(ptr)[static_cast<size_t>(o) * ld + c] = lin_cvt16(v[j], type);
                }
            }
        };
        // Finish 16 rows (unit `un` of the tile).
        auto finish = [&](const LtTile& t, int un, float (&v)[16], float (&u)[16]) {
            const int c = t.c0 + 32 * lg + lane;
            const bool on = c < a.C;
            const int rr = un * 16 + (lane & 15);
            const bool have = rr < t.nrows;
            int grow = have ? t.r0 + rr : -1, orow = grow;
            if (!WG && have) orow = lin_index(a.scatter, a.scatter_total, grow, a.err);
            if (KIND == LIN_FWD) {
                const bool bad = a.gather && have && lin_index(a.gather, a.gather_total, grow, a.err) < 0;
                const uint32_t z = __ballot_sync(0xFFFFFFFFu, bad);
                if (z) {   // rows that an index outside x stands for count as zero
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (z >> j & 1) v[j] = u[j] = 0.0f;
                }
                const size_t bi = static_cast<size_t>(t.e) * a.C + c;
                if (a.bias[0] && on) {
                    const float b = lin_load(a.bias[0], bi, a.bias_type);
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] += b;
                }
                if (DUAL && a.bias[1] && on) {
                    const float b = lin_load(a.bias[1], bi, a.bias_type);
#pragma unroll
                    for (int j = 0; j < 16; ++j) u[j] += b;
                }
                if (a.z[0]) store16(a.z[0], a.ldz, a.type, pair_z, grow, c, v);
                if (DUAL && a.z[1]) store16(a.z[1], a.ldz, a.type, pair_z, grow, c, u);
                if (DUAL) lin_act16<LACT_SWIGLU>(v, u);
                else if (a.act == LACT_RELU) lin_act16<LACT_RELU>(v, u);
                else if (a.act == LACT_SILU) lin_act16<LACT_SILU>(v, u);
                else if (a.act == LACT_GELU) lin_act16<LACT_GELU>(v, u);
            }
            void* out = a.out[WG ? t.which : 0];
            if (WG) {
                const size_t skip = static_cast<size_t>(t.e) * a.o_gstride;
                out = a.out_type == LIN_F32 ? static_cast<void*>(static_cast<float*>(out) + skip)
                                            : static_cast<void*>(static_cast<uint16_t*>(out) + skip);
            }
            const void* res = WG ? (a.accumulate ? out : nullptr) : a.res;
            if (res) {
                const long long ldr = WG ? a.ldo : a.ldr;
                const int rt = WG ? a.out_type : a.res_type;
                float r[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int o = __shfl_sync(0xFFFFFFFFu, orow, j);
                    r[j] = o >= 0 && on ? lin_load(res, static_cast<size_t>(o) * ldr + c, rt) : 0.0f;
                }
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] += r[j];
                __syncwarp();   // a neighbour writes this lane's value below (res may be the output)
            }
            store16(out, a.ldo, a.out_type, pair_out, orow, c, v);
        };
        auto ld16 = [&](uint32_t addr, float (&v)[16]) {
            uint32_t r[16];
            tmem_ld16(addr, r);
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r[j]);
        };
        int acc = 0;
        for (int w = blockIdx.x; w < n_work; w += G) {
            LtTile t;
            if (!tile_of(w, t)) continue;
            const int units = (t.nrows + 15) / 16;
            auto take = [&](int ab) {
                if (!mbar_poll(&acc_full[ab], (acc >> 1) & 1, abort_flag, a.timeout_ns) && lane == 0)
                    latch_error(a.err, ERR_ETIMEOUT, acc, KID_LINEAR);
                tc_fence_after();
            };
            auto release = [&](int ab) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_empty[ab]);
            };
            if (t.nkb == 0) {   // an empty group's gradient
                for (int un = uh; un < units; un += 2) {
                    float v[16], u[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = u[j] = 0.0f;
                    finish(t, un, v, u);
                }
            } else if (!p.promote || t.nkb <= p.promote) {
                const int ab = acc & 1;
                take(ab);
                const uint32_t d = tmem + lane_addr + ab * (NACC * BN);
                for (int un = uh; un < units; un += 2) {
                    float v[16], u[16];
                    ld16(d + un * 16, v);
                    if (DUAL) ld16(d + BN + un * 16, u);
                    finish(t, un, v, u);
                }
                release(ab);
                ++acc;
            } else {   // fp32 output: at most 128 columns (64 of each accumulator), summed over spans in registers
                float v[4][16];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[i][j] = 0.0f;
                for (int k0 = 0; k0 < t.nkb; k0 += p.promote, ++acc) {
                    const int ab = acc & 1;
                    take(ab);
                    const uint32_t d = tmem + lane_addr + ab * (NACC * BN);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int un = DUAL ? uh + 2 * (i & 1) : uh + 2 * i;
                        if (un < units) {
                            float x[16];
                            ld16(d + (DUAL && i >= 2 ? BN : 0) + un * 16, x);
#pragma unroll
                            for (int j = 0; j < 16; ++j) v[i][j] += x[j];
                        }
                    }
                    release(ab);
                }
#pragma unroll
                for (int i = 0; i < (DUAL ? 2 : 4); ++i) {
                    const int un = uh + 2 * i;
                    if (un < units) finish(t, un, v[i], v[DUAL ? i + 2 : i]);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(static_cast<uint32_t>(p.tmem_cols)));
}

// ------------------------------------------------------------------ host side
// 16-bit tensor map with a 128-byte swizzle: up to three dimensions, innermost contiguous.
inline bool lt_encode(CUtensorMap* map, int type, const void* base, uint64_t d0, uint64_t d1, uint64_t d2, uint64_t s1,
                      uint64_t s2, uint32_t b1, bool rank2 = false) {
    static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    if (!encode) {
        cudaDriverEntryPointQueryResult q;
        void* f = nullptr;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return false;
        encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }
    const cuuint64_t dims[3] = {d0, d1, d2};
    const cuuint64_t strides[2] = {s1 * 2, s2 * 2};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(kLtBK), b1, 1}, es[3] = {1, 1, 1};
    return encode(map, type == LIN_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                  rank2 ? 2 : 3, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether TMA can read the operands as they lie: 16-byte aligned bases, strides of whole 16 bytes.
inline bool lt_tma_ok(const LinArgs& a) {
    auto base = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
    const bool groups = a.kind != LIN_WGRAD && a.E > 1;
    return base(a.a[0]) && base(a.a[1]) && base(a.b[0]) && base(a.b[1]) && a.lda % 8 == 0 && a.ldb % 8 == 0 &&
           (!groups || a.a_gstride % 8 == 0);
}

inline LtPlan lt_plan(const LinArgs& a, int sm_count, int smem_limit) {
    LtPlan p{};
    const bool dual = a.kind == LIN_FWD && a.a[1];
    const int nacc = dual ? 2 : 1;
    const bool f32 = a.out_type == LIN_F32;
    p.n_ct = (a.C + kLtM - 1) / kLtM;
    p.promote = f32 ? kLtPromote : 0;
    int most = 256 / nacc / (f32 ? 2 : 1);
    // rows a tile should hold: those of an average group
    const int want = a.kind == LIN_WGRAD ? a.out_n : (a.rows + a.E - 1) / a.E;
    p.bn = a.kind == LIN_WGRAD ? 64 : 16;
    while (p.bn < want && p.bn < most) p.bn *= 2;
    p.bbox = p.bn < 64 ? p.bn : 64;
    const int btile = p.bn * 128;
    p.stage_bytes = (nacc * kLtATile + btile + 1023) / 1024 * 1024;
    const int head = 512 + 4 * (a.E + 1);
    p.off_ring = (head + 1023) / 1024 * 1024;
    p.stages = (smem_limit - 1024 - p.off_ring) / p.stage_bytes;
    if (p.stages > kLtMaxStages) p.stages = kLtMaxStages;
    p.smem = p.off_ring + p.stages * p.stage_bytes + 1024;
    p.tmem_cols = 32;
    while (p.tmem_cols < 2 * nacc * p.bn) p.tmem_cols *= 2;
    long long tiles = static_cast<long long>(p.n_ct);
    if (a.kind == LIN_WGRAD) tiles *= static_cast<long long>((a.out_n + p.bn - 1) / p.bn) * a.E * (a.b[1] ? 2 : 1);
    else tiles *= a.rows / p.bn + a.E;
    p.grid = tiles < sm_count ? static_cast<int>(tiles) : sm_count;
    return p;
}

inline bool lt_maps(const LinArgs& a, const LtPlan& p, LtMaps* m) {
    const uint64_t R = static_cast<uint64_t>(a.rows > 0 ? a.rows : 1);
    const uint64_t C = a.C, Q = a.Q, E = a.E, lda = a.lda, ldb = a.ldb;
    const bool g = a.gather != nullptr;
    bool ok = true;
    if (a.kind == LIN_WGRAD) {   // A = x [rows, C], B = dz [rows, out_n]
        const uint64_t xr = g ? a.gather_total : R;
        ok = lt_encode(&m->a0, a.type, a.a[0], C, xr, 1, lda, lda * xr, g ? 1 : 64, g) &&
             lt_encode(&m->b0, a.type, a.b[0], a.out_n, R, 1, ldb, ldb * R, 64);
        m->a1 = m->a0;
        m->b1 = m->b0;
        return ok && (!a.b[1] || lt_encode(&m->b1, a.type, a.b[1], a.out_n, R, 1, ldb, ldb * R, 64));
    }
    const bool fwd = a.kind == LIN_FWD;
    const uint64_t inner = fwd ? Q : C, outer = fwd ? C : Q;
    const uint64_t gs = E > 1 ? static_cast<uint64_t>(a.a_gstride) : lda * outer;
    const uint64_t br = g && fwd ? a.gather_total : R;
    ok = lt_encode(&m->a0, a.type, a.a[0], inner, outer, E, lda, gs, fwd ? kLtM : 64) &&
         lt_encode(&m->b0, a.type, a.b[0], Q, br, 1, ldb, ldb * br, g && fwd ? 1 : p.bbox, g && fwd);
    m->a1 = m->a0;
    m->b1 = m->b0;
    if (a.a[1]) ok = ok && lt_encode(&m->a1, a.type, a.a[1], inner, outer, E, lda, gs, fwd ? kLtM : 64);
    if (a.b[1]) ok = ok && lt_encode(&m->b1, a.type, a.b[1], Q, br, 1, ldb, ldb * br, p.bbox);
    return ok;
}

}  // namespace moe
