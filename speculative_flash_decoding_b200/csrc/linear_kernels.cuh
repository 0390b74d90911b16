// Linear layer of a decode batch on the fifth-generation tensor cores:
// y = activation(x W^T + bias) + residual, bf16 operands, fp32 sums.
//
// The batch is small, so the operands change sides: 128 rows of W are the M
// of a tcgen05.mma, up to 256 rows of x its N, and the accumulator is
// y^T in TMEM (lane = feature, column = batch row).  W is read once from HBM
// while x comes from L2; TMA brings 64-column slices of both (128-byte
// swizzle) through a ring of up to 220 KB.  One warp's lane issues the
// copies, one the MMAs, then eight warps read the accumulator back for the
// epilogue.  When there are fewer tiles than SMs, the CTAs of a cluster
// split K and add their accumulators through distributed shared memory, each
// for its share of the batch rows, in rank order (the same bits every time).
// Bound by the bytes of W up to about 250 rows.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include <cstdint>
#include <type_traits>

#include "common.cuh"
#include "linear_plan.h"
#include "ptx.cuh"

namespace alspec {

constexpr int kLinThreads = 256;
constexpr int kLinK = 64;         // columns of a stage: 128 bytes
constexpr int kLinMaxN = 256;     // batch rows per tile
constexpr int kLinMaxStages = 12;
constexpr int kLinSmem = 224 * 1024;  // dynamic shared memory, at most
// Batch rows of a tile up to which parts of the sums are pushed to the CTA that
// finishes their rows, instead of read by it: one cluster barrier less, a
// buffer of split * slice * 512 bytes beside the ring more.  k = n = 4096, pushed
// against read: 9.9 and 10.9 us for 1 row, 9.7 and 10.5 for 32, 10.0 and 10.9
// for 48.  At 64 rows it still gains where K is split (11.0 and 11.3; 12.5 and
// 13.7 with k = 8192, n = 2048), but loses where it is hardly or not (27.9 and
// 27.4 with k = n = 8192, 16.0 and 14.8 with k = 2048, n = 16384).
constexpr int kLinPush = 48;
constexpr int kLinAhead = 8;      // blocks asked for before the kernel ahead has ended
// More than half of an SM's shared memory whatever the sizes, so that an SM
// holds one CTA and its TMEM allocation never waits for another's.
constexpr int kLinMinSmem = 120 * 1024;

struct LinearParams {
    // Views of W and x: 3-D (column in a block, row, whole 64-column block),
    // boxes of `group` blocks; and 2-D (column, row) for a last block of
    // fewer columns, filled up with zeros.
    CUtensorMap tw, tx, tw_end, tx_end;
    const __nv_bfloat16* bias;
    const void* residual;
    void* y;
    int rows, n, kblocks, whole;  // 64-column blocks of k, and those without a fill
    int nt;        // batch rows per tile: a multiple of 16
    int row_tiles, split, stages;
    int group;     // 64-column blocks a stage holds
    int tmem_cols;
    int sums, sum_cols;  // accumulators that the blocks go round, columns of each
    int out_bf16, act;
    int push;      // parts of the sums go to the CTA that finishes their rows
    int slice;     // batch rows that a CTA finishes, at most
    int vec;       // y and the residual can be taken four features at a time
    unsigned* err;
    unsigned long long timeout_ns;
};

__device__ __forceinline__ bool lin_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                         const LinearParams& p) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 31) == 0) {
            if (*abort) return false;
            if (global_ns() - t0 > p.timeout_ns) {
                *abort = 1;
                if (p.err) atomicOr(p.err, kErrTimeout);
                return false;
            }
        }
    }
}

// Shared-memory matrix descriptor: K-major rows of 128 bytes with 128-byte
// swizzle, groups of 8 rows 1024 bytes apart.
__device__ __forceinline__ uint64_t lin_desc(uint32_t addr) {
    return (uint64_t)((addr & 0x3ffffu) >> 4) | (1ull << 16) | (64ull << 32) | (1ull << 46) |
           (2ull << 61);
}

template <bool PAIR>
__device__ __forceinline__ void lin_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        bool add) {
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
            : "memory");
}

// Arrive on `bar` (PAIR: of both CTAs, `first` the pair's lower rank in the
// cluster) once the MMAs so far are done.
template <bool PAIR>
__device__ __forceinline__ void lin_commit(uint64_t* bar, int first) {
    if constexpr (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
            ".multicast::cluster.b64 [%0], %1;" ::"r"(smem_addr(bar)),
            "h"((uint16_t)(3 << first))
            : "memory");
    else
        asm volatile(
            "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                smem_addr(bar))
            : "memory");
}

// TMEM columns, for one warp of the CTA (PAIR: of each CTA of the pair).
template <bool PAIR>
__device__ __forceinline__ void lin_tmem_alloc(uint32_t* at, uint32_t columns) {
    if constexpr (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(at)),
                     "r"(columns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(at)),
                     "r"(columns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
}

template <bool PAIR>
__device__ __forceinline__ void lin_tmem_free(uint32_t tmem, uint32_t columns) {
    if constexpr (PAIR)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(columns)
                     : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(columns)
                     : "memory");
}

// 16 accumulator columns of this thread's lane, from the first accumulator.
__device__ __forceinline__ void lin_load16(uint32_t addr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(addr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// The same, all accumulators added: `used` of them, sum_cols columns apart.
__device__ __forceinline__ void lin_sum16(const LinearParams& p, uint32_t addr, int used,
                                          float (&v)[16]) {
    lin_load16(addr, v);
    for (int a = 1; a < used; ++a) {
        float w[16];
        lin_load16(addr + (uint32_t)(a * p.sum_cols), w);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] += w[i];
    }
}

// The activation of N sums: one branch on its kind, not one per sum.  SiLU
// takes the fast exponential, of x / 2 so that its square, and the quotient by
// a number in [1, 2], stay in range wherever the result does: within 2^-20 +
// |x| 2^-23 of the result.  (x over 1 + exp(-x) by the fast quotient is 0 from
// -87.4 down, where the result is a normal number until -92.)
template <int N>
__device__ __forceinline__ void lin_activate(float (&x)[N], int act) {
    if (act == 1) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = x[i] < 0.f ? 0.f : x[i];
    } else if (act == 2) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = 0.5f * x[i] * (1.f + erff(x[i] * 0.70710678118654752f));
    } else if (act == 3) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float t = __expf(-0.5f * fabsf(x[i]));
            x[i] = __fdividef(x[i] < 0.f ? x[i] * t * t : x[i], 1.f + t * t);
        }
    }
}

__device__ __forceinline__ float lin_value(const float* p) { return *p; }
__device__ __forceinline__ float lin_value(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void lin_put(float* p, float v) { *p = v; }
__device__ __forceinline__ void lin_put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Four neighbouring values, aligned to their size.
__device__ __forceinline__ void lin_put4(float* p, const float* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void lin_put4(__nv_bfloat16* p, const float* v) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
}

// The epilogue of batch rows [c0, c1) of a tile.  Their sums lie in shared
// memory, either one part in each of the cluster's CTAs (of its half, where
// CTAS is 2), [row][feature], or (PUSH) all parts here, [CTA][row - c0]
// [feature].  A warp takes a row at a time, a lane four features; a round of R
// rows is asked for (the residual, the first two parts) before the round ahead
// is finished (250 x 8192 x 8192 36.2 -> 35.7 us, 33 x 4096 x 6144 14.7 ->
// 14.5; large batches take rounds of eight rows, with four 36.1).
template <typename O, int R>
struct LinRound {
    alignas(16) O add[R][4];  // the residual
    float4 part[2][R];
};

template <typename O, bool PUSH, int CTAS, int R>
__device__ __forceinline__ void lin_epilogue(const LinearParams& p, uint32_t sums, int place,
                                             int c0, int c1, int r0, int n0) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kWarps = kLinThreads / 32;
    const int f = n0 + 4 * lane;
    const int nf = min(4, p.n - f);  // features of this lane
    if (nf <= 0) return;
    const O* res = static_cast<const O*>(p.residual);
    const long long step = (long long)kWarps * p.n;
    // Part s of row c + u * kWarps, u < R.
    auto load_part = [&](int c, int s, float4 (&part)[R]) {
        const uint32_t here = sums + (uint32_t)((PUSH ? c - c0 : c) * kLinM + 4 * lane) * 4;
        // This CTA's own part without the way through the cluster.
        if (PUSH || s == place / CTAS) {
            const uint32_t from = here + (uint32_t)(PUSH ? s * p.slice * kLinM * 4 : 0);
#pragma unroll
            for (int u = 0; u < R; ++u)
                if (c + u * kWarps < c1) part[u] = lds_v4(from + u * kWarps * kLinM * 4);
        } else {
            const uint32_t from = dsmem_addr(here, (uint32_t)(s * CTAS + place % CTAS));
#pragma unroll
            for (int u = 0; u < R; ++u)
                if (c + u * kWarps < c1) part[u] = ld_dsmem_v4(from + u * kWarps * kLinM * 4);
        }
    };
    auto load = [&](int c, LinRound<O, R>& r) {
        if (res) {
            const O* from = res + (long long)(r0 + c) * p.n + f;
#pragma unroll
            for (int u = 0; u < R; ++u) {
                if (c + u * kWarps >= c1) continue;
                if (p.vec) {
                    using V = typename std::conditional<sizeof(O) == 4, float4, uint2>::type;
                    *reinterpret_cast<V*>(r.add[u]) = *reinterpret_cast<const V*>(from + u * step);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i < nf) r.add[u][i] = from[u * step + i];
                }
            }
        }
        load_part(c, 0, r.part[0]);
        if (p.split > 1) load_part(c, 1, r.part[1]);
    };
    LinRound<O, R> now;
    if (c0 + warp < c1) load(c0 + warp, now);
    float bias[4] = {0.f, 0.f, 0.f, 0.f};
    if (p.bias) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < nf) bias[i] = __bfloat162float(p.bias[f + i]);
    }
    for (int c = c0 + warp; c < c1; c += kWarps * R) {
        LinRound<O, R> next;
        if (c + kWarps * R < c1) load(c + kWarps * R, next);
        float v[4 * R];
        auto add_part = [&](const float4 (&part)[R]) {
#pragma unroll
            for (int u = 0; u < R; ++u) {
                v[4 * u] += part[u].x, v[4 * u + 1] += part[u].y;
                v[4 * u + 2] += part[u].z, v[4 * u + 3] += part[u].w;
            }
        };
#pragma unroll
        for (int u = 0; u < R; ++u) {
            v[4 * u] = now.part[0][u].x, v[4 * u + 1] = now.part[0][u].y;
            v[4 * u + 2] = now.part[0][u].z, v[4 * u + 3] = now.part[0][u].w;
        }
        if (p.split > 1) add_part(now.part[1]);
        for (int s = 2; s < p.split; ++s) {
            float4 part[R];
            load_part(c, s, part);
            add_part(part);
        }
#pragma unroll
        for (int i = 0; i < 4 * R; ++i) v[i] += bias[i % 4];
        lin_activate(v, p.act);
        if (res) {
#pragma unroll
            for (int i = 0; i < 4 * R; ++i) v[i] += lin_value(&now.add[i / 4][i % 4]);
        }
        O* y = static_cast<O*>(p.y) + (long long)(r0 + c) * p.n + f;
#pragma unroll
        for (int u = 0; u < R; ++u) {
            if (c + u * kWarps >= c1) continue;
            if (p.vec) {
                lin_put4(y + u * step, v + 4 * u);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < nf) lin_put(y + u * step + i, v[4 * u + i]);
            }
        }
        now = next;
    }
}

// PAIR: two CTAs of a cluster (ranks 2 i and 2 i + 1) work as one on 256
// features: each brings its own 128 rows of W and half of the rows of x, the
// first issues MMAs of twice the M that read both CTAs' shared memory, and
// each keeps the sums of its own features.
template <bool PAIR>
__global__ void __launch_bounds__(kLinThreads, 1) linear_kernel(
    const __grid_constant__ LinearParams p) {
    extern __shared__ unsigned char lin_raw[];
    __shared__ uint64_t full[kLinMaxStages], empty[kLinMaxStages], done;
    __shared__ uint32_t tmem_base;
    __shared__ uint16_t owner[kLinPush];
    __shared__ int abort_flag;
    volatile int* abort = &abort_flag;
    unsigned char* ring = reinterpret_cast<unsigned char*>(
        (reinterpret_cast<uintptr_t>(lin_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kCtas = PAIR ? 2 : 1;  // that work on one tile's block of K
    const int place = (int)blockIdx.x % (kCtas * p.split);  // in the cluster
    const int tile = (int)blockIdx.x / (kCtas * p.split);
    const int rank = place / kCtas, half = place % kCtas;
    const int first = place - half;
    // Row tiles of one feature tile are neighbours: its W comes from L2 for
    // all but the first.
    const int n0 = (tile / p.row_tiles * kCtas + half) * kLinM, r0 = tile % p.row_tiles * p.nt;
    const int xr = p.nt / kCtas;  // rows of x that this CTA brings
    const int kb0 = (int)((long long)rank * p.kblocks / p.split);
    const int kb1 = (int)((long long)(rank + 1) * p.kblocks / p.split);
    const int stage_bytes = (kLinM + xr) * 128 * p.group;
    const int fills = (kb1 - kb0 + p.group - 1) / p.group;
    const int rows = min(p.nt, p.rows - r0);
    const int c0 = rank * rows / p.split, c1 = (rank + 1) * rows / p.split;  // this CTA finishes
    // Small batches: who finishes row c (low 4 bits), as which of its rows.
    float* exchange = reinterpret_cast<float*>(ring + p.stages * stage_bytes);
    if (p.push && (int)threadIdx.x < rows) {
        const int c = (int)threadIdx.x, r = ((c + 1) * p.split - 1) / rows;
        owner[c] = (uint16_t)(r | (c - r * rows / p.split) << 4);
    }

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        mbar_init(&done, 1);
        abort_flag = 0;
        fence_barrier_init();
        prefetch_tmap(&p.tw);
        prefetch_tmap(&p.tx);
        prefetch_tmap(&p.tw_end);
        prefetch_tmap(&p.tx_end);
    }
    if (warp == 2) {
        lin_tmem_alloc<PAIR>(&tmem_base, (uint32_t)p.tmem_cols);
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    }
    // (A pair's CTAs signal each other's barriers.)
    if constexpr (PAIR)
        cluster_sync();
    else
        __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = tmem_base;
    // Launched while the kernel ahead on the stream may still run: nothing is
    // read or written before it has completed, and only then may the next
    // one be launched.
    // (W's first stages are asked for in L2 meanwhile, which is coherent
    // whoever writes them: 16 x 8192 x 8192 back to back 25.9 -> 24.5 us.)
    if (warp == 0 && lane == 0 && n0 < p.n) {
        for (int i = 0; i < kLinAhead / p.group; ++i) {
            const int kb = kb0 + i * p.group;
            if (kb + p.group <= min(kb1, p.whole)) tma_prefetch_3d(&p.tw, 0, n0, kb);
        }
    }
    pdl_wait_prerequisite();
    pdl_launch_dependents();
    // Every CTA of the cluster has begun before one writes to another (waited
    // for there).
    if (p.push && p.split > 1) cluster_arrive_relaxed();

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t keep = l2_evict_normal_policy();
            const uint64_t policy = p.row_tiles == 1 ? l2_evict_first_policy() : keep;
            for (int i = 0; i < fills; ++i) {
                const int s = i % p.stages;
                if (i >= p.stages && !lin_wait(empty + s, (i / p.stages - 1) & 1, abort, p)) break;
                const int kb = kb0 + i * p.group;
                unsigned char* w = ring + s * stage_bytes;
                unsigned char* x = w + p.group * kLinM * 128;
                const int blocks = min(p.group, kb1 - kb), rx = r0 + half * xr;
                // The barrier of the CTA that issues the MMAs takes the bytes
                // of both.
                if (half == 0)
                    mbar_arrive_expect_tx(full + s,
                                          (uint32_t)(kCtas * blocks * (kLinM + xr) * 128));
                if constexpr (PAIR) {
                    const uint32_t bar = dsmem_addr(smem_addr(full + s), (uint32_t)first);
                    if (kb + p.group <= min(kb1, p.whole)) {
                        tma_load_3d_pair(w, &p.tw, 0, n0, kb, bar, policy);
                        tma_load_3d_pair(x, &p.tx, 0, rx, kb, bar, keep);
                    } else {
                        for (int g = 0; g < blocks; ++g) {
                            tma_load_2d_pair(w + g * kLinM * 128, &p.tw_end, (kb + g) * kLinK, n0,
                                             bar, policy);
                            tma_load_2d_pair(x + g * xr * 128, &p.tx_end, (kb + g) * kLinK, rx,
                                             bar, keep);
                        }
                    }
                } else if (kb + p.group <= min(kb1, p.whole)) {
                    tma_load_3d(w, &p.tw, 0, n0, kb, full + s, policy);
                    tma_load_3d(x, &p.tx, 0, rx, kb, full + s, keep);
                } else {  // the last blocks of this CTA, one at a time
                    for (int g = 0; g < blocks; ++g) {
                        tma_load_2d(w + g * kLinM * 128, &p.tw_end, (kb + g) * kLinK, n0, full + s,
                                    policy);
                        tma_load_2d(x + g * xr * 128, &p.tx_end, (kb + g) * kLinK, rx, full + s,
                                    keep);
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && half == 0) {
            // fp32 accumulator, bf16 operands, both K-major.
            const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) |
                                   ((uint32_t)(p.nt >> 3) << 17) | ((uint32_t)(kCtas * kLinM >> 4) << 24);
            int sum = 0;
            for (int i = 0; i < fills; ++i) {
                const int s = i % p.stages;
                if (!lin_wait(full + s, (i / p.stages) & 1, abort, p)) {
                    // Given up: let the copies in flight land (bounded).
                    const uint64_t t0 = global_ns();
                    for (int j = i; j < min(i + p.stages, fills); ++j)
                        while (!mbar_try_wait(full + j % p.stages, (j / p.stages) & 1))
                            if (global_ns() - t0 > p.timeout_ns) break;
                    break;
                }
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t a = smem_addr(ring + s * stage_bytes);
                const int blocks = min(p.group, kb1 - kb0 - i * p.group);
                for (int g = 0; g < blocks; ++g) {
                    const uint64_t da = lin_desc(a + g * kLinM * 128);
                    const uint64_t db = lin_desc(a + p.group * kLinM * 128 + g * xr * 128);
#pragma unroll
                    for (int k = 0; k < kLinK / 16; ++k)  // 32 bytes of every row a step
                        lin_mma<PAIR>(tmem + (uint32_t)(sum * p.sum_cols), da + 2 * k, db + 2 * k,
                                      idesc, k > 0 || i * p.group + g >= p.sums);
                    if (++sum == p.sums) sum = 0;
                }
                lin_commit<PAIR>(empty + s, first);
            }
            lin_commit<PAIR>(&done, first);
        }
    } else if (p.residual) {
        // Meanwhile the residual is asked for in L2.
        const int es = p.out_bf16 ? 2 : 4;
        const int lines = (kLinM * es + 127) / 128;
        const char* res = static_cast<const char*>(p.residual);
        for (int i = threadIdx.x - 64; i < (c1 - c0) * lines; i += kLinThreads - 64) {
            const int f = n0 + i % lines * (128 / es);
            if (f < p.n) prefetch_l2(res + ((long long)(r0 + c0 + i / lines) * p.n + f) * es);
        }
    }
    __syncwarp();
    // The accumulator is complete (each thread waits; bounded).
    const bool good = lin_wait(&done, 0, abort, p) && !*abort;
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    __syncthreads();

    // Warp w reads the 32 lanes of its quarter, the two halves of the warps
    // alternate groups of 16 columns.
    const int fl = (warp & 3) * 32 + lane;  // feature within the tile
    const uint32_t taddr = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    if (!PAIR && p.push) {
        // Small batches: a part goes straight to the CTA that finishes the
        // row, into a buffer beside the ring, and one cluster barrier later
        // every CTA is on its own.  (Reading the others' parts needs a second
        // barrier before anyone may leave: 1 x 4096 x 4096 10.1 us.)
        if (p.split > 1) cluster_wait();
        const uint32_t mine =
            smem_addr(exchange) + (uint32_t)(rank * p.slice * kLinM + fl) * 4;
        for (int c = 16 * (warp >> 2); c < rows; c += 32) {
            float v[16];
            lin_sum16(p, taddr + c, min(p.sums, kb1 - kb0), v);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if (c + i < rows) {
                    const int to = owner[c + i] & 15, at = owner[c + i] >> 4;
                    st_dsmem(dsmem_addr(mine + at * kLinM * 4, to), v[i]);
                }
            }
            __syncwarp();
        }
        if (p.split > 1)
            cluster_sync();
        else
            __syncthreads();
        if (good) {
            if (p.out_bf16)
                lin_epilogue<__nv_bfloat16, true, 1, 2>(p, smem_addr(exchange), place, c0, c1, r0,
                                                        n0);
            else
                lin_epilogue<float, true, 1, 2>(p, smem_addr(exchange), place, c0, c1, r0, n0);
        }
    } else {
        // Large batches: this CTA's parts, [batch row][feature], go where the
        // ring was, and every CTA reads those of the rows it finishes (a
        // pair's CTAs have features of their own: the ranks of one half).
        float* mine = reinterpret_cast<float*>(ring);
        for (int c = 16 * (warp >> 2); c < rows; c += 32) {
            float v[16];
            lin_sum16(p, taddr + c, min(p.sums, kb1 - kb0), v);
#pragma unroll
            for (int i = 0; i < 16; ++i) mine[(c + i) * kLinM + fl] = v[i];
        }
        if (p.split > 1)
            cluster_sync();
        else
            __syncthreads();
        if (good) {
            if (p.out_bf16)
                lin_epilogue<__nv_bfloat16, false, kCtas, 8>(p, smem_addr(mine), place, c0, c1,
                                                             r0, n0);
            else
                lin_epilogue<float, false, kCtas, 8>(p, smem_addr(mine), place, c0, c1, r0, n0);
        }
        if (PAIR || p.split > 1) cluster_sync();
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (warp == 2) lin_tmem_free<PAIR>(tmem, (uint32_t)p.tmem_cols);
}

}  // namespace alspec
