// Matrix products with a fused epilogue on the fifth-generation tensor cores, plain or grouped by
// expert:
//     y[r] = act(W x[r] + b) [* (U x[r] + c)] [+ residual[r]]
// x [rows][K] and the weights [N][K] (grouped: [E][N][K], rows offsets[e] .. offsets[e+1] take
// expert e's) are bf16 or fp16; products are summed in fp32 in tensor memory (TMEM), the epilogue
// runs in fp32, and y is rounded once (bf16, fp16) or stored as fp32.
//
// Orientation: the MMA's M = weight rows (128 per CTA), N = the tile's tokens, so an output
// feature is a TMEM lane: its bias is a per-thread constant, few tokens cost few MMA columns, and
// the outputs of a token are turned in shared memory into one run of features. With a gate (U given)
// a CTA holds 64 features: 64 rows of W and the same 64 rows of U, which meet in that turn.
//
// Variants:
//   CG = 2  two CTAs share one tile (256 weight rows x up to 256 tokens, cta_group::2): each loads
//           its 128 weight rows and half of the tokens, so a 64-wide K step moves 32 KB per SM for
//           512 cycles of MMA. For compute-bound sizes; persistent, one pair per two SMs.
//   CG = 1  one CTA per tile of 128 weight rows x up to 128 tokens. For weight-bound sizes. With
//           few tiles, a cluster of S CTAs splits K: every CTA sends its partial sums of token u
//           into the shared memory of CTA u mod S, which adds them up in rank order
//           (deterministic) before the epilogue.
//
// Roles (576 threads): warps 0-15 epilogue (four per TMEM lane quadrant; with eight, an epilogue of
// 256 tokens took longer than 2048 inputs' MMAs), warp 16 TMA loads (no multicast), warp 17 TMEM
// allocation and MMA issue. Two accumulators alternate, so that a tile's epilogue (or a K block's
// addition to the running sums) overlaps the next one's MMAs. Every wait is bounded: on a timeout the
// kernel records DPA_ERR_DEVICE_TIMEOUT and every role leaves its loop.
#pragma once
#include <climits>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "epilogue.cuh"
#include "kernels.h"
#include "tc.cuh"

namespace dpa {

// Maps of x for one load per stage: plain, boxes of a whole tile's rows (the first map); grouped,
// boxes of 16, 32, 64 and 128 rows, of which a tile takes the smallest that holds its rows. (Several
// boxes of 32 rows per stage cost more than the rows that a larger box reads in vain: 128 experts of
// 256 rows 218 against 196 us.)
constexpr int kRowMaps = 4;
struct RowMaps {
    CUtensorMap m[kRowMaps];
};

// A launch as launch_linear has prepared it.
struct LinearLaunch {
    bool pair, gated, f16, blocks;
    const CUtensorMap* wmaps;   // W, U
    const RowMaps* xmaps;
    int clusters;
    size_t smem;
};
template <bool VEC>   // out_features % 8 == 0
cudaError_t launch_linear_variant(const LinearArgs& a, const LinearLaunch& l, cudaStream_t stream);

namespace {

constexpr int kRowsA = 128;                      // weight rows per CTA (TMEM lanes)
constexpr int kStepK = 64;                       // K per stage: one 128-byte swizzle row of 16-bit values
constexpr int kATile = kRowsA * 128;             // 16 KB
constexpr int kEpiWarps = 16, kGroups = kEpiWarps / 4;   // a group is one warp per TMEM lane quadrant
constexpr int kChunk = 16;                       // tokens that a group finishes at a time
constexpr int kLoadWarp = kEpiWarps, kMmaWarp = kEpiWarps + 1;
constexpr int kThreads = (kEpiWarps + 2) * 32;   // 576
constexpr int kMaxStages = 12;
constexpr uint32_t kTmemCols = 512;
constexpr int kBlockedSteps = 4, kBlockedTokens = 160;   // K in blocks: steps per block, most tokens per tile
constexpr int kSmemMax = 232448;
constexpr int kOutBytes = kGroups * kChunk * kRowsA * 4;   // epilogue staging, one chunk per group
// full[stages], empty[stages], acc_full[2], acc_empty[2], done; then the TMEM address and abort flag
constexpr int kBarBytes = (2 * kMaxStages + 5) * 8 + 16;

struct Tile {
    int e, row0, n, ft;
};

// Rows of one token tile when n rows are cut into nt tiles: equal parts rounded up to `step` rows. With
// tiles of at most tn rows, a multiple of step, nt is n / tn rounded up, and so is n / the result.
__host__ __device__ __forceinline__ int tile_rows(int n, int nt, int step) {
    const int each = nt == 1 ? n : (n - 1) / nt + 1;
    return (each + step - 1) / step * step;
}
__host__ __device__ __forceinline__ int balanced_rows(int n, int tn, int step) {
    return tile_rows(n, (n - 1) / tn + 1, step);
}

__device__ __forceinline__ int group_edge(const LinearArgs& a, int e) {
    return min(max(__ldg(a.offsets + e), 0), a.rows);   // an edge outside the rows reads as the nearest row
}

// Groups' tables in shared memory (grouped): token tiles before each group and its first row, [E + 1]
// each, and the rows of its tiles, [E].
struct GroupTables {
    int *pref, *off, *rows;
};

// A warp's way through its cluster's tiles, every ncl-th one from `cid` on, features innermost.
// Divisions are left out of it: with few K steps a tile takes little longer than finding it did (128
// experts, 12 steps: 97 to 114 us with a division and a search through all groups per tile, 95 to 100 without).
struct TileCursor {
    int tt, ft, e;   // token tile, feature tile, group (of an earlier tile until find)

    __device__ __forceinline__ TileCursor(const LinearArgs& a, int cid)
        : tt(static_cast<int>(static_cast<unsigned>(cid) / static_cast<unsigned>(a.FT))), ft(cid - tt * a.FT), e(0) {}
    __device__ __forceinline__ void advance(const LinearArgs& a) {
        tt += a.step_t;
        ft += a.step_f;
        if (ft >= a.FT) {
            ft -= a.FT;
            ++tt;
        }
    }
    // Called by whole warps: the group is the last one whose first tile is not after the tile.
    __device__ __forceinline__ Tile find(const LinearArgs& a, const GroupTables& g, int lane) {
        Tile t;
        t.ft = ft;
        t.e = 0;
        if (a.E == 0) {   // plain: the launcher's TN is the tiles' size
            t.row0 = tt * a.TN;
            t.n = min(a.rows - t.row0, a.TN);
            return t;
        }
        for (int c = 32; c == 32;) {
            const int x = e + lane;
            c = __popc(__ballot_sync(0xffffffffu, x < a.E && g.pref[x] <= tt));   // at least one
            e += c - 1;
        }
        const int begin = g.off[e], n = g.off[e + 1] - begin, sz = g.rows[e], skip = (tt - g.pref[e]) * sz;
        t.e = e;
        t.row0 = begin + skip;
        t.n = min(n - skip, sz);
        return t;
    }
};

// Eight outputs (or residual values) of one token. VEC (N % 8 == 0): consecutive features, 16-byte
// aligned and wholly inside or outside N. Otherwise the first `cnt` of features `fs` apart, fs lanes
// side by side, so that a token's single elements still leave as runs (8 consecutive ones per lane
// took 161 us where this takes 91: 5025x696x5966 fp16 with a gate).
struct Out8 {
    uint4 lo, hi;   // 16-bit values: lo only; fp32: lo, hi
};
template <bool VEC>
__device__ __forceinline__ Out8 load_residual(const LinearArgs& a, int64_t at, int cnt, int fs) {
    Out8 r;
    if (a.res32) {
        const float* p = static_cast<const float*>(a.residual) + at;
        if (VEC) {
            r.lo = *reinterpret_cast<const uint4*>(p);
            r.hi = *reinterpret_cast<const uint4*>(p + 4);
        } else {
            uint32_t v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = i < cnt ? __float_as_uint(p[i * fs]) : 0u;
            r.lo = make_uint4(v[0], v[1], v[2], v[3]);
            r.hi = make_uint4(v[4], v[5], v[6], v[7]);
        }
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(a.residual) + at;
        if (VEC) {
            r.lo = *reinterpret_cast<const uint4*>(p);
        } else {
            uint32_t v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = (2 * i < cnt ? p[2 * i * fs] : 0u) |
                       (2 * i + 1 < cnt ? static_cast<uint32_t>(p[(2 * i + 1) * fs]) << 16 : 0u);
            r.lo = make_uint4(v[0], v[1], v[2], v[3]);
        }
    }
    return r;
}
template <bool F16>
__device__ __forceinline__ void add_residual(const LinearArgs& a, const Out8& r, float (&v)[8]) {
    const uint32_t w[8] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w, r.hi.x, r.hi.y, r.hi.z, r.hi.w};
    if (a.res32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += __uint_as_float(w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] += up16<F16>(static_cast<uint16_t>(w[i]));
            v[2 * i + 1] += up16<F16>(static_cast<uint16_t>(w[i] >> 16));
        }
    }
}
template <bool F16, bool VEC>
__device__ __forceinline__ void store_out(const LinearArgs& a, const float (&v)[8], int64_t at, int cnt, int fs) {
    if (a.out32) {
        float* p = static_cast<float*>(a.out) + at;
        if (VEC && a.out_wide) {   // one 32-byte store
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]),
                         "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                         : "memory");
        } else if (VEC) {
            *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < cnt) p[i * fs] = v[i];
        }
    } else {
        uint16_t* p = static_cast<uint16_t*>(a.out) + at;
        if (VEC) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = down16x2<F16>(v[2 * i], v[2 * i + 1]);
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < cnt) p[i * fs] = down16<F16>(v[i]);
        }
    }
}

// Barrier of the four warps of an epilogue group; `ok` comes back false if any of them brought false.
__device__ __forceinline__ bool group_agree(int grp, bool ok) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.and.aligned.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(ok)), "r"(1 + grp)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void group_sync(int grp) {
    asm volatile("barrier.cta.sync.aligned %0, 128;" ::"r"(1 + grp) : "memory");
}

// ---- pair (cta_group::2) forms of the tensor-core operations ----
template <int CG>
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t acc) {
    if constexpr (CG == 1) {
        tc_mma(d, ad, bd, idesc, acc);
    } else {
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(ad), "l"(bd), "r"(idesc), "r"(acc)
            : "memory");
    }
}
// arrival on the same barrier of every CTA of the tile
template <int CG>
__device__ __forceinline__ void commit(uint64_t* bar) {
    if constexpr (CG == 1) {
        tc_commit(bar);
    } else {
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                smem_u32(bar)),
            "h"(static_cast<uint16_t>(3))
            : "memory");
    }
}
// tensor loads into this CTA's shared memory, completing on `bar` (shared::cluster address; of the
// pair's first CTA with CG = 2)
template <int CG>
__device__ __forceinline__ void load2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    if constexpr (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
            " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
            : "memory");
}
template <int CG>
__device__ __forceinline__ void load3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    if constexpr (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
            " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// Eight biases of one group's features (zeros without a bias and behind the last feature), as loaded:
// turned into fp32 by biases() after the wait for the sums.
struct Bias8 {
    uint32_t w[4];
};
template <bool VEC>
__device__ __forceinline__ Bias8 load_bias(const void* b, int64_t at, int cnt, int fs) {
    Bias8 r = {};
    if (b && cnt > 0) {
        const uint16_t* p = static_cast<const uint16_t*>(b) + at;
        if (VEC) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
            r.w[0] = v.x;
            r.w[1] = v.y;
            r.w[2] = v.z;
            r.w[3] = v.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                r.w[i] = (2 * i < cnt ? __ldg(p + 2 * i * fs) : 0u) |
                         (2 * i + 1 < cnt ? static_cast<uint32_t>(__ldg(p + (2 * i + 1) * fs)) << 16 : 0u);
        }
    }
    return r;
}
template <bool F16>
__device__ __forceinline__ void biases(const Bias8& b, Two (&out)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        out[i] = two(up16<F16>(static_cast<uint16_t>(b.w[i])), up16<F16>(static_cast<uint16_t>(b.w[i] >> 16)));
}

// Bias, activation and gate of eight sums (g; m: the second product's).
template <bool GATED>
__device__ __forceinline__ void finish8(Two (&g)[4], const Two (&m)[4], const Two (&bias)[4], const Two (&bmul)[4], int act,
                                        float (&o)[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) g[e] = add2(g[e], bias[e]);
    act_many(g, act);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (GATED) g[e] = mul2(g[e], add2(m[e], bmul[e]));
        const float2 h = apart(g[e]);
        o[2 * e] = h.x;
        o[2 * e + 1] = h.y;
    }
}
// Where column R of a staged token lies: permuted within the row, 16-byte pieces kept whole, so that
// both the lanes of a quadrant (consecutive columns) and those of a token (8 columns each, or single
// ones) are free of bank conflicts.
__device__ __forceinline__ int staged(int R) { return R ^ (((R >> 5) & 1) * 4 + (R >> 6) * 16); }

// Eight sums FS columns apart.
template <int FS, bool SWIZZLED>
__device__ __forceinline__ void load_sums_apart(const float* row, int c, Two (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int c0 = c + 2 * i * FS, c1 = c0 + FS;
        v[i] = two(row[SWIZZLED ? staged(c0) : c0], row[SWIZZLED ? staged(c1) : c1]);
    }
}
__device__ __forceinline__ void load_sums(const float* p0, const float* p1, Two (&v)[4]) {
    const float4 x = *reinterpret_cast<const float4*>(p0), y = *reinterpret_cast<const float4*>(p1);
    v[0] = two(x.x, x.y);
    v[1] = two(x.z, x.w);
    v[2] = two(y.x, y.y);
    v[3] = two(y.z, y.w);
}

template <int CG, bool GATED, bool F16, bool BLOCKED, bool VEC>
__global__ void __launch_bounds__(kThreads, 1) linear_kernel(LinearArgs a, const __grid_constant__ CUtensorMap wmap,
                                                             const __grid_constant__ CUtensorMap umap,
                                                             const __grid_constant__ RowMaps xmaps) {
    constexpr int kFeat = GATED ? 64 : 128;   // output features per CTA
    constexpr int kAccCols = BLOCKED ? kBlockedTokens : 256;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                         ~static_cast<uintptr_t>(1023));
    const int stages = a.stages, btile = (a.TN / CG) * 128;
    unsigned char* sA = sm;
    unsigned char* sB = sm + stages * kATile;
    // epilogue staging [kGroups][kChunk][128]; K split: [splits][this CTA's tokens][128] partial sums
    float* s_out = reinterpret_cast<float*>(sB + stages * btile);
    unsigned char* tail = sB + stages * btile + a.out_bytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(tail);
    uint64_t* empty = full + kMaxStages;
    uint64_t* acc_full = empty + kMaxStages;
    uint64_t* acc_empty = acc_full + 2;
    uint64_t* done = acc_empty + 2;
    volatile uint32_t* s_tmem = reinterpret_cast<volatile uint32_t*>(done + 1);
    volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
    GroupTables groups;
    groups.pref = reinterpret_cast<int*>(tail + kBarBytes);
    groups.off = groups.pref + a.E + 1;
    groups.rows = groups.off + a.E + 1;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int S = a.splits;                                     // CTAs sharing K (CG = 1)
    const int rank = CG == 2 || S > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int csize = CG == 2 ? 2 : S;
    const int cid = static_cast<int>(blockIdx.x) / csize, ncl = static_cast<int>(gridDim.x) / csize;

    if (tid == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], kEpiWarps * CG);
        }
        mbar_init(done, 1);
        *s_abort = 0;
        fence_barrier_init();
    }
    if (warp == kLoadWarp && lane == 0) {
        prefetch_map(&wmap);
        if (GATED) prefetch_map(&umap);
        prefetch_map(&xmaps.m[0]);
    }
    if (CG == 1 && S > 1) cluster_arrive();   // waited for before the first access to another CTA's memory
    if (warp == kMmaWarp) {
        if constexpr (CG == 1) {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_u32(const_cast<uint32_t*>(s_tmem))),
                         "r"(kTmemCols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                             smem_u32(const_cast<uint32_t*>(s_tmem))),
                         "r"(kTmemCols)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        }
    }
    pdl_wait();
    // edges of the groups and token tiles before each: counted by all threads, added up by one warp
    if (a.E > 0) {
        for (int e = tid; e <= a.E; e += kThreads) {
            const int begin = group_edge(a, e), n = e < a.E ? group_edge(a, e + 1) - begin : 0;
            const int nt = n > 0 ? (n - 1) / a.TN + 1 : 0;
            groups.off[e] = begin;
            groups.pref[e] = nt;
            if (e < a.E) groups.rows[e] = nt > 0 ? tile_rows(n, nt, 16 * CG) : 0;
        }
        __syncthreads();
        if (warp == kLoadWarp) {
            const int each = a.E / 32 + 1, e0 = min(lane * each, a.E + 1), e1 = min(e0 + each, a.E + 1);
            // 64 bits: offsets out of order name rows many times over (1024 groups of 2^30 rows, 2^33 tiles)
            int64_t sum = 0;
            for (int e = e0; e < e1; ++e) sum += groups.pref[e];
            int64_t incl = sum;
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            int64_t before = incl - sum;
            for (int e = e0; e < e1; ++e) {
                const int c = groups.pref[e];
                groups.pref[e] = static_cast<int>(min(before, static_cast<int64_t>(INT_MAX)));
                before += c;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();   // the pair's barriers are initialised
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    // grouped: as many as the offsets name, but no more than there can be when they are in order (with K
    // split, one per cluster)
    int ntiles = a.ntiles;
    if (a.E > 0) ntiles = static_cast<int>(min(static_cast<int64_t>(groups.pref[a.E]) * a.FT, static_cast<int64_t>(ntiles)));
    // this CTA's K steps
    const int k0 = CG == 1 ? a.ksteps * rank / S : 0, k1 = CG == 1 ? a.ksteps * (rank + 1) / S : a.ksteps;

    if (warp == kLoadWarp) {
        // ================= loads =================
        // The whole warp runs the loop, so that its counters and addresses stay in uniform registers,
        // and one elected lane issues the copies (as a loop of one lane, the issue bound the kernel).
        {
            const bool leader = elect_one();
            const uint32_t full0 = CG == 2 ? mapa_shared(smem_u32(full), 0) : smem_u32(full);
            const uint32_t a0 = smem_u32(sA), b0 = smem_u32(sB);
            int s = 0, ph = 1;
            bool ok = true;
            TileCursor cursor(a, cid);
            for (int it = cid; it < ntiles && ok; it += ncl, cursor.advance(a)) {
                const Tile t = cursor.find(a, groups, lane);
                const int part = ((t.n + 16 * CG - 1) / (16 * CG)) * 16;   // token rows of this CTA
                int mi = 0, box = a.xbox;
                while (box < part) {   // grouped only: a plain tile's box holds it
                    box *= 2;
                    ++mi;
                }
                const CUtensorMap* xm = &xmaps.m[mi];
                const int f0 = (t.ft * CG + (CG == 2 ? rank : 0)) * kFeat;
                const int r0 = t.row0 + (CG == 2 ? rank * part : 0);
                const uint32_t bytes = static_cast<uint32_t>(CG) * (kATile + box * 128);
                for (int kc = k0; kc < k1; ++kc) {
                    if (!__all_sync(0xffffffffu, mbar_wait_abortable(&empty[s], ph, s_abort, a.hdr, 0x710))) {
                        ok = false;
                        break;
                    }
                    if (leader) {
                        const uint32_t bar = full0 + 8 * s, da = a0 + s * kATile;
                        if (CG == 1 || rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
                        load3d<CG>(da, &wmap, kc * kStepK, f0, t.e, bar);
                        if constexpr (GATED) load3d<CG>(da + kATile / 2, &umap, kc * kStepK, f0, t.e, bar);
                        load2d<CG>(b0 + s * btile, xm, kc * kStepK, r0, bar);
                    }
                    __syncwarp();
                    if (++s == stages) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
            // The last arrival on every stage's barrier lands before this CTA may end (the MMA warp of the
            // pair's first CTA sends them to both CTAs' shared memory).
            for (int i = 0; i < stages && ok; ++i) {
                ok = __all_sync(0xffffffffu, mbar_wait_abortable(&empty[s], ph, s_abort, a.hdr, 0x711));
                if (++s == stages) {
                    s = 0;
                    ph ^= 1;
                }
            }
            // So does the first CTA's last commit (waited for beside the last tile's epilogue; behind it,
            // 4096x768x2048 took 16.4 us against 16.25).
            if (CG == 2 && rank == 1) mbar_wait_bounded(done, 0, a.hdr, 0x723);
            if (*s_abort) {   // copies already issued land well within this time
                const uint64_t t0 = globaltimer();
                while (globaltimer() - t0 < 2000000ull) __nanosleep(10000);
            }
        }
        __syncwarp();
    } else if (warp == kMmaWarp) {
        // ================= MMA issue (the pair's first CTA) =================
        if (CG == 1 || rank == 0) {
            const bool leader = elect_one();
            const uint32_t a_base = smem_u32(sA), b_base = smem_u32(sB);
            const uint64_t dconst = smem_desc_sw128(0);
            int s = 0, ph = 0, j = 0;   // j: accumulators filled
            bool ok = true;
            TileCursor cursor(a, cid);
            for (int it = cid; it < ntiles && ok; it += ncl, cursor.advance(a)) {
                const Tile t = cursor.find(a, groups, lane);
                const int ncols = (t.n + 16 * CG - 1) / (16 * CG) * (16 * CG);
                const uint32_t idesc = instr_desc(F16 ? 0 : 1, ncols, 128 * CG);
                for (int kb = k0, kend; kb < k1 && ok; kb = kend, ++j) {
                    const int b = j & 1;
                    kend = BLOCKED ? min(kb + kBlockedSteps, k1) : k1;
                    const uint32_t td = tmem + static_cast<uint32_t>(b * kAccCols);
                    bool w_ok = mbar_wait_abortable(&acc_empty[b], ((j >> 1) & 1) ^ 1, s_abort, a.hdr, 0x720);
                    ok = __all_sync(0xffffffffu, w_ok);
                    for (int kc = kb; kc < kend && ok; ++kc) {
                        w_ok = mbar_wait_abortable(&full[s], ph, s_abort, a.hdr, 0x721);
                        if (!__all_sync(0xffffffffu, w_ok)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint64_t ad = dconst | ((a_base + static_cast<uint32_t>(s) * kATile) >> 4);
                        const uint64_t bd = dconst | ((b_base + static_cast<uint32_t>(s * btile)) >> 4);
                        if (leader) {
                            mma_f16<CG>(td, ad, bd, idesc, kc > kb ? 1u : 0u);
                            mma_f16<CG>(td, ad + 2, bd + 2, idesc, 1u);
                            mma_f16<CG>(td, ad + 4, bd + 4, idesc, 1u);
                            mma_f16<CG>(td, ad + 6, bd + 6, idesc, 1u);
                            commit<CG>(&empty[s]);
                            if (kc == kend - 1) commit<CG>(&acc_full[b]);
                        }
                        __syncwarp();
                        if (++s == stages) {
                            s = 0;
                            ph ^= 1;
                        }
                    }
                }
            }
            // every MMA issued has completed before TMEM is released
            if (leader) commit<CG>(done);
            __syncwarp();
            mbar_wait_bounded(done, 0, a.hdr, 0x722);
            __syncwarp();
        }
    } else {
        // ================= epilogue =================
        // The four warps of a group take every fourth chunk of 16 tokens. A chunk is read from TMEM
        // (lane = weight row) and turned through shared memory, so that each thread then finishes 8
        // features of a token and a token's features leave as one contiguous run.
        const int q = warp & 3, grp = warp >> 2, R = 32 * q + lane;
        const uint32_t lane_base = static_cast<uint32_t>(32 * q) << 16;
        float* stage = s_out + grp * (kChunk * kRowsA);
        float* put = stage + staged(R);
        // this thread's features and tokens of a chunk
        constexpr int kFeatGroups = kFeat / 8, kItems = kChunk * kFeatGroups / 128, kTokStep = kChunk / kItems;
        const int fg = R % kFeatGroups, tk0 = R / kFeatGroups;   // R is also the thread of the group
        const float* get0 = stage + staged(fg * 8);
        const float* get1 = stage + staged(fg * 8 + 4);
        const float* gum0 = stage + staged(fg * 8 + 64);   // the second product (GATED)
        const float* gum1 = stage + staged(fg * 8 + 68);
        uint32_t empty_bar[2] = {smem_u32(&acc_empty[0]), smem_u32(&acc_empty[1])};
        if (CG == 2) {
            empty_bar[0] = mapa_shared(empty_bar[0], 0);
            empty_bar[1] = mapa_shared(empty_bar[1], 0);
        }
        constexpr int fs = VEC ? 1 : kFeatGroups;
        if (CG == 1 && S > 1) cluster_wait();   // every CTA of the cluster has started
        auto release = [&](int b) {   // this warp has read its part of accumulator b
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (CG == 2) arrive_cluster(empty_bar[b]);
                else mbarrier_arrive(&acc_empty[b]);
            }
        };
        const bool blocked = BLOCKED && k1 - k0 > kBlockedSteps;
        const uint32_t sums = tmem + lane_base + static_cast<uint32_t>(2 * kAccCols);   // of a tile's K blocks
        int j = 0;
        TileCursor cursor(a, cid);
        for (int it = cid; it < ntiles; it += ncl, ++j, cursor.advance(a)) {
            const Tile t = cursor.find(a, groups, lane);
            const int f = (t.ft * CG + (CG == 2 ? rank : 0)) * kFeat + (VEC ? fg * 8 : fg);
            const int cnt = min(max((a.N - f + fs - 1) / fs, 0), 8);
            const int nch = (t.n + kChunk - 1) / kChunk;
            Bias8 bias_raw = {}, bmul_raw = {};
            Out8 res[kItems];
            if (CG == 2 || S == 1) {   // operands of the epilogue: loaded while the MMAs run
                const int64_t fb = static_cast<int64_t>(t.e) * a.N + f;
                bias_raw = load_bias<VEC>(a.bias, fb, cnt, fs);
                if (GATED) bmul_raw = load_bias<VEC>(a.bias_mul, fb, cnt, fs);
                if (a.residual && cnt > 0) {
#pragma unroll
                    for (int i = 0; i < kItems; ++i) {
                        const int tok = kChunk * grp + tk0 + i * kTokStep;
                        if (tok < t.n)
                            res[i] = load_residual<VEC>(a, (static_cast<int64_t>(t.row0) + tok) * a.N + f, cnt, fs);
                    }
                }
            }
            // every K block but the last: added to the running sums
            bool w_ok = true;
            for (int kb = k0; BLOCKED && kb + kBlockedSteps < k1; kb += kBlockedSteps, ++j) {
                w_ok = mbar_wait_abortable(&acc_full[j & 1], (j >> 1) & 1, s_abort, a.hdr, 0x731);
                w_ok = group_agree(grp, w_ok);
                if (!w_ok) break;
                tc_fence_after();
                const uint32_t acc = tmem + lane_base + static_cast<uint32_t>((j & 1) * kAccCols);
                for (int c = grp; c < nch; c += kGroups) {
                    uint32_t v[kChunk], w[kChunk];
                    tmem_ld16(acc + kChunk * c, v);
                    if (kb > k0) tmem_ld16(sums + kChunk * c, w);
                    tmem_wait_ld();
                    if (kb > k0) {
#pragma unroll
                        for (int u = 0; u < kChunk; ++u) v[u] = __float_as_uint(__uint_as_float(v[u]) + __uint_as_float(w[u]));
                    }
                    tmem_st16(sums + kChunk * c, v);
                }
                tmem_wait_st();
                release(j & 1);
            }
            if (!w_ok) break;
            const int b = j & 1;
            w_ok = mbar_wait_abortable(&acc_full[b], (j >> 1) & 1, s_abort, a.hdr, 0x730);
            w_ok = group_agree(grp, w_ok);   // the group leaves together (it synchronises below)
            if (!w_ok) break;
            tc_fence_after();
            const uint32_t acc = tmem + lane_base + static_cast<uint32_t>(b * kAccCols);
            auto read_sums = [&](int c, uint32_t (&v)[kChunk]) {
                tmem_ld16(acc + kChunk * c, v);
                if (BLOCKED && blocked) {
                    uint32_t w[kChunk];
                    tmem_ld16(sums + kChunk * c, w);
                    tmem_wait_ld();
#pragma unroll
                    for (int u = 0; u < kChunk; ++u) v[u] = __float_as_uint(__uint_as_float(v[u]) + __uint_as_float(w[u]));
                } else {
                    tmem_wait_ld();
                }
            };
            if (CG == 1 && S > 1) {
                // token u goes to CTA u mod S of the cluster: [this CTA's rank][u / S][128]
                const int slice = (t.n + S - 1) / S * kRowsA;
                const uint32_t dst = smem_u32(s_out) + static_cast<uint32_t>(rank * slice + R) * 4;
                for (int c = grp; c < nch; c += kGroups) {
                    uint32_t v[kChunk];
                    read_sums(c, v);
                    int place = kChunk * c / S, owner = kChunk * c - place * S;
#pragma unroll
                    for (int u = 0; u < kChunk; ++u) {
                        if (kChunk * c + u < t.n)
                            st_cluster_f32(mapa_shared(dst + static_cast<uint32_t>(place * kRowsA) * 4, owner), __uint_as_float(v[u]));
                        if (++owner == S) {
                            owner = 0;
                            ++place;
                        }
                    }
                }
                break;   // one tile per cluster
            }
            Two bias[4], bmul[4];
            biases<F16>(bias_raw, bias);
            if (GATED) biases<F16>(bmul_raw, bmul);
            for (int c = grp; c < nch; c += kGroups) {
                uint32_t v[kChunk];
                read_sums(c, v);
                if (c + kGroups >= nch) release(b);   // last read of this accumulator by this warp
                if (c > grp) group_sync(grp);   // the chunk before has been read out
#pragma unroll
                for (int u = 0; u < kChunk; ++u) put[u * kRowsA] = __uint_as_float(v[u]);
                group_sync(grp);
                if (cnt > 0) {
#pragma unroll
                    for (int i = 0; i < kItems; ++i) {
                        const int in = tk0 + i * kTokStep, tok = kChunk * c + in;
                        if (tok >= t.n) break;
                        const int64_t at = (static_cast<int64_t>(t.row0) + tok) * a.N + f;
                        Two g2[4], m2[4];
                        if constexpr (VEC) {
                            load_sums(get0 + in * kRowsA, get1 + in * kRowsA, g2);
                            if (GATED) load_sums(gum0 + in * kRowsA, gum1 + in * kRowsA, m2);
                        } else {
                            load_sums_apart<kFeatGroups, true>(stage + in * kRowsA, fg, g2);
                            if (GATED) load_sums_apart<kFeatGroups, true>(stage + in * kRowsA, fg + 64, m2);
                        }
                        float g[8];
                        finish8<GATED>(g2, m2, bias, bmul, a.act, g);
                        if (a.residual) {
                            add_residual<F16>(a, res[i], g);
                            if (tok + kChunk * kGroups < t.n)
                                res[i] = load_residual<VEC>(a, at + kChunk * kGroups * static_cast<int64_t>(a.N), cnt, fs);
                        }
                        store_out<F16, VEC>(a, g, at, cnt, fs);
                    }
                }
            }
            if (grp >= nch) release(b);   // this group had nothing to read
            group_sync(grp);   // read out before the next tile is staged
        }
    }
    __syncwarp();

    if (CG == 1 && S > 1) {
        if (warp >= kEpiWarps) cluster_wait();   // the first phase, which the epilogue has waited for
        __syncwarp();
        cluster_sync();                          // every partial sum has arrived
        if (cid < ntiles) {
            const Tile t = TileCursor(a, cid).find(a, groups, lane);
            const int slice = (t.n + S - 1) / S * kRowsA, mine = (t.n - rank + S - 1) / S;
            constexpr int kFeatGroups = kFeat / 8, fs = VEC ? 1 : kFeatGroups;
            for (int i = tid; i < mine * kFeatGroups; i += kThreads) {
                const int place = i / kFeatGroups, fg = i % kFeatGroups, c = VEC ? fg * 8 : fg, f = t.ft * kFeat + c;
                const int cnt = min(max((a.N - f + fs - 1) / fs, 0), 8);
                if (cnt == 0) continue;
                const int64_t fb = static_cast<int64_t>(t.e) * a.N + f;
                const int64_t at = (static_cast<int64_t>(t.row0) + place * S + rank) * a.N + f;
                Two bias[4], bmul[4], g[4], m[4];
                Out8 res;
                biases<F16>(load_bias<VEC>(a.bias, fb, cnt, fs), bias);
                if (GATED) biases<F16>(load_bias<VEC>(a.bias_mul, fb, cnt, fs), bmul);
                if (a.residual) res = load_residual<VEC>(a, at, cnt, fs);
                const float* src = s_out + place * kRowsA;
                auto sums = [&](int col, Two (&v)[4]) {
                    if constexpr (VEC) load_sums(src + col, src + col + 4, v);
                    else load_sums_apart<kFeatGroups, false>(src, col, v);
                };
                sums(c, g);
                if (GATED) sums(c + 64, m);
                for (int r = 1; r < S; ++r) {   // in rank order
                    Two x[4];
                    src += slice;
                    sums(c, x);
#pragma unroll
                    for (int e = 0; e < 4; ++e) g[e] = add2(g[e], x[e]);
                    if (GATED) {
                        sums(c + 64, x);
#pragma unroll
                        for (int e = 0; e < 4; ++e) m[e] = add2(m[e], x[e]);
                    }
                }
                float o[8];
                finish8<GATED>(g, m, bias, bmul, a.act, o);
                if (a.residual) add_residual<F16>(a, res, o);
                store_out<F16, VEC>(a, o, at, cnt, fs);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();   // both CTAs are done with the pair's barriers and TMEM
    if (warp == kMmaWarp) {
        tc_fence_after();
        if constexpr (CG == 1)
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
        else
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

template <int CG, bool GATED, bool F16, bool VEC>
cudaError_t launch_variant(const LinearArgs& in, bool blocks, const CUtensorMap* wmaps, const RowMaps& xmaps, int clusters,
                           size_t smem, cudaStream_t stream) {
    LinearArgs a = in;
    const void* fn = blocks ? reinterpret_cast<const void*>(linear_kernel<CG, GATED, F16, true, VEC>)
                            : reinterpret_cast<const void*>(linear_kernel<CG, GATED, F16, false, VEC>);
    const cudaError_t err = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    if (err != cudaSuccess) return err;
    const int csize = CG == 2 ? 2 : a.splits;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(clusters) * csize);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(csize);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = csize > 1 ? 2 : 1;
    void* args[] = {&a, const_cast<CUtensorMap*>(wmaps), const_cast<CUtensorMap*>(wmaps + 1), const_cast<RowMaps*>(&xmaps)};
    return cudaLaunchKernelExC(&cfg, fn, args);
}

}  // namespace

template <bool VEC>
cudaError_t launch_linear_variant(const LinearArgs& a, const LinearLaunch& l, cudaStream_t stream) {
    auto go = [&](auto cg, auto gated, auto f16) {
        return launch_variant<decltype(cg)::value, decltype(gated)::value, decltype(f16)::value, VEC>(
            a, l.blocks, l.wmaps, *l.xmaps, l.clusters, l.smem, stream);
    };
    using One = std::integral_constant<int, 1>;
    using Pair = std::integral_constant<int, 2>;
    auto types = [&](auto cg) {
        if (l.gated) return l.f16 ? go(cg, std::true_type{}, std::true_type{}) : go(cg, std::true_type{}, std::false_type{});
        return l.f16 ? go(cg, std::false_type{}, std::true_type{}) : go(cg, std::false_type{}, std::false_type{});
    };
    return l.pair ? types(Pair{}) : types(One{});
}

}  // namespace dpa
