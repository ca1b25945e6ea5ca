// Routed pairs sorted by expert, and the rows that travel with them.
//
// A batch of T tokens with K routed experts each has P = T*K pairs, pair p = t*K + k. A pair whose
// expert id lies outside [0, E) is not routed (a padded token, an expert held elsewhere).
//   sort       stable counting sort of the pairs by expert, unrouted pairs last:
//              order[i] = pair at place i, pos[p] = place of pair p (-1 if unrouted),
//              offsets[e] = places before expert e, e = 0..E (offsets[E] = routed pairs)
//   permute    out[pos[t,k]] = x[t]
//   unpermute  y[t] = residual[t] + sum_k w[t,k] z[pos[t,k]]
//   backward   dz[pos[t,k]] = w[t,k] dy[t],   dw[t,k] = <dy[t], z[pos[t,k]]>
// The gradient of permute is unpermute with unit weights. Every result is a gather or has one
// writer, so nothing here uses floating-point atomics and repeated runs agree bit for bit.
// Positions outside [0, P) are skipped, whatever their value.
#include <climits>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace dpa {
namespace {

// ---------------------------------------------------------------- sort

constexpr int kSortThreads = 1024;
constexpr int kSortOneBlock = 2048;   // pairs that one CTA sorts alone (one launch)
// Beyond that: 64 CTAs' chunks of at least 1024 pairs (131072 pairs: 10.5 us with 2048 each, 11.8 us
// with 1024), 128 chunks once a warp's keys would not stay in registers.
constexpr int kSortChunk = 1024;

__device__ __forceinline__ int pair_key(const int32_t* idx, int p, int E) {
    const int e = __ldcg(idx + p);   // from L2: sort_place_kernel starts before sort_count_kernel ends
    return static_cast<unsigned>(e) < static_cast<unsigned>(E) ? e : E;
}

// Lanes of the warp with this lane's key, from one ballot per key bit (`bits` covers 0 .. E; lanes
// without a pair have key -1, all ones). On 128 experts a round of 32 pairs takes a third of the
// time of the match instruction, which goes through the distinct keys one by one.
__device__ __forceinline__ unsigned same_key(int key, int bits) {
    unsigned same = __ballot_sync(0xffffffffu, key >= 0);
    if (key < 0) same = ~same;
    for (int b = 0; b < bits; ++b) {
        const bool set = (key >> b) & 1;
        const unsigned with = __ballot_sync(0xffffffffu, set);
        same &= set ? with : ~with;
    }
    return same;
}

// Pairs per expert of each CTA's chunk: hist[b][key], key = E for unrouted pairs.
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(SortArgs a) {
    extern __shared__ int32_t s_cnt[];
    const int E1 = a.E + 1;
    for (int i = threadIdx.x; i < E1; i += kSortThreads) s_cnt[i] = 0;
    __syncthreads();
    pdl_wait();
    pdl_trigger();   // the ids are final: sort_place_kernel may start on them
    const int p0 = blockIdx.x * a.chunk, p1 = min(a.P - p0, a.chunk) + p0;
    for (int p = p0 + threadIdx.x; p < p1; p += kSortThreads) atomicAdd(&s_cnt[pair_key(a.idx, p, a.E)], 1);
    __syncthreads();
    int32_t* h = a.hist + static_cast<size_t>(blockIdx.x) * E1;
    for (int i = threadIdx.x; i < E1; i += kSortThreads) h[i] = s_cnt[i];
}

// Places of one CTA's chunk. Each warp owns a contiguous run of the chunk and counts it by key
// (lanes of equal key found by ballots), the counts are scanned over warps, earlier chunks and
// keys, and every pair's place is its key's start plus its rank in the run. IT > 0: the run has at
// most IT rounds of 32 pairs, whose keys (all loaded at once) and ranks stay in registers; IT = 0:
// any length, read and ranked a second time.
// With several chunks the kernel starts beside sort_count_kernel (which lets it go once the ids are
// final) and waits for it only before it reads the other chunks' counts.
template <int IT>
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(SortArgs a) {
    extern __shared__ int32_t smem[];
    const int E1 = a.E + 1, nw = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t* s_warp = smem;               // [nw][E1] counts, later the first place
    int32_t* s_tot = smem + nw * E1;      // [E1] pairs of the key in all chunks, later the key's start
    int32_t* s_pre = s_tot + E1;          // [E1] pairs of the key in earlier chunks
    int32_t* s_sum = s_pre + E1;          // [32] totals of each warp's keys
    for (int i = threadIdx.x; i < (nw + 2) * E1; i += blockDim.x) smem[i] = 0;
    const bool alone = gridDim.x == 1;
    if (alone) pdl_wait();
    const int p0 = blockIdx.x * a.chunk, n = min(a.P - p0, a.chunk);
    const int run = (((n + nw - 1) / nw) + 31) & ~31;
    const int w0 = p0 + min(warp * run, n), w1 = p0 + min(warp * run + run, n);
    int32_t* mine = s_warp + warp * E1;
    const unsigned below = (1u << lane) - 1;
    const int bits = 32 - __clz(a.E);
    int key[IT > 0 ? IT : 1], rank[IT > 0 ? IT : 1];
    if constexpr (IT > 0) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int p = w0 + 32 * i + lane;
            key[i] = p < w1 ? pair_key(a.idx, p, a.E) : -1;
        }
    }
    __syncthreads();
    if constexpr (IT > 0) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            if (w0 + 32 * i < w1) {   // warp-uniform
                const unsigned same = same_key(key[i], bits);
                const int before = key[i] >= 0 ? mine[key[i]] : 0;
                rank[i] = before + __popc(same & below);
                __syncwarp();
                if (key[i] >= 0 && (same & below) == 0) mine[key[i]] = before + __popc(same);
                __syncwarp();
            }
        }
    } else {
        for (int b = w0; b < w1; b += 32) {
            const int p = b + lane;
            if (p < w1) atomicAdd(&mine[pair_key(a.idx, p, a.E)], 1);
        }
    }
    if (!alone) {
        pdl_wait();   // the counts of every chunk
        // the chunks are split over groups of threads that cover the keys once
        const int cover = (E1 + 31) & ~31, nb = static_cast<int>(gridDim.x);
        const int parts = max(1, min(static_cast<int>(blockDim.x) / cover, nb));
        for (int i = threadIdx.x; i < cover * parts; i += blockDim.x) {
            const int part = i / cover, e = i - part * cover;
            if (e >= E1) continue;
            const int b1 = nb * (part + 1) / parts;
            int tot = 0, pre = 0;
#pragma unroll 16
            for (int b = nb * part / parts; b < b1; ++b) {
                const int c = __ldcg(a.hist + static_cast<size_t>(b) * E1 + e);
                tot += c;
                pre += b < static_cast<int>(blockIdx.x) ? c : 0;
            }
            atomicAdd(&s_tot[e], tot);   // whole numbers: the order does not matter
            atomicAdd(&s_pre[e], pre);
        }
    }
    __syncthreads();
    // counts -> places before this warp's run, per key
    for (int e = threadIdx.x; e < E1; e += blockDim.x) {
        int acc = alone ? 0 : s_pre[e];
#pragma unroll 8
        for (int w = 0; w < nw; ++w) {
            const int c = s_warp[w * E1 + e];
            s_warp[w * E1 + e] = acc;
            acc += c;
        }
        if (alone) s_tot[e] = acc;
    }
    __syncthreads();
    // exclusive scan of the totals over the keys, `items` consecutive keys per thread
    const int items = (E1 + blockDim.x - 1) / blockDim.x, e0 = threadIdx.x * items;
    int sum = 0;
    for (int i = 0; i < items; ++i) sum += e0 + i < E1 ? s_tot[e0 + i] : 0;
    int incl = sum;
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    int start = incl - sum;
    for (int w = 0; w < warp; ++w) start += s_sum[w];
    for (int i = 0; i < items; ++i) {
        if (e0 + i < E1) {
            const int c = s_tot[e0 + i];
            s_tot[e0 + i] = start;
            if (blockIdx.x == 0) a.offsets[e0 + i] = start;   // key E: the routed pairs
            start += c;
        }
    }
    __syncthreads();
    if constexpr (IT > 0) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            if (key[i] >= 0) {
                const int p = w0 + 32 * i + lane, at = mine[key[i]] + s_tot[key[i]] + rank[i];
                a.pos[p] = key[i] < a.E ? at : -1;
                a.order[at] = p;
            }
        }
    } else {
        for (int b = w0; b < w1; b += 32) {
            const int p = b + lane;
            const int k = p < w1 ? pair_key(a.idx, p, a.E) : -1;
            const unsigned same = same_key(k, bits);
            const int before = k >= 0 ? mine[k] : 0;
            if (k >= 0) {
                const int at = before + s_tot[k] + __popc(same & below);
                a.pos[p] = k < a.E ? at : -1;
                a.order[at] = p;
            }
            __syncwarp();
            if (k >= 0 && (same & below) == 0) mine[k] = before + __popc(same);
            __syncwarp();
        }
    }
}

// All of sort_place_kernel's shared memory (none is static).
size_t sort_smem_bytes(int warps, int E) { return static_cast<size_t>(warps + 2) * (E + 1) * 4 + 32 * 4; }

// ---------------------------------------------------------------- rows

// Element types of the rows: conversion to and from fp32 (one rounding, to nearest even).
__device__ __forceinline__ float up(float v) { return v; }
__device__ __forceinline__ float up(__half v) { return __half2float(v); }
__device__ __forceinline__ float up(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T down(float v);
template <>
__device__ __forceinline__ float down<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half down<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 down<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// VEC consecutive elements, loaded and stored in 16-byte pieces (VEC = 1: one element).
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC < 16 ? sizeof(T) * VEC : 16) Pack {
    T v[VEC];
};

// Slots of one token, held one per lane (top_k <= 32): lane k has the place of slot k (UINT_MAX:
// unrouted or outside the rows) and its weight (0 then, whatever the weights hold there). Read
// once per warp, handed out by shuffles.
struct Slots {
    unsigned p;
    float w;
};
__device__ __forceinline__ Slots load_slots(const int32_t* pos, const void* weights, int wtype, int64_t t, int K,
                                            unsigned P, int lane) {
    Slots s{UINT_MAX, 0.f};
    if (lane < K) {
        const unsigned p = static_cast<unsigned>(__ldg(pos + t * K + lane));
        float w = 1.f;   // no weights
        if (wtype == DPA_DTYPE_FP64) w = static_cast<float>(__ldg(static_cast<const double*>(weights) + t * K + lane));
        if (wtype == DPA_DTYPE_FP32) w = __ldg(static_cast<const float*>(weights) + t * K + lane);
        if (p < P) {
            s.p = p;
            s.w = w;
        }
    }
    return s;
}

// A pack if `on`, else zeros. Written as predicated loads so that the loads of several rows stay
// together in front of the arithmetic (as branches they were moved to their uses, one at a time:
// 136 against 41 us for 4096 tokens of 8 rows of 2048 bf16). Outputs may lie on inputs (a residual, the
// rows' gradient): the compiler must not move a store in front of them, hence "memory".
template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load_if(const T* p, bool on) {
    constexpr int kBytes = sizeof(T) * VEC;
    Pack<T, VEC> out;
    if constexpr (kBytes % 16 == 0) {
        uint4 r[kBytes / 16];
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i)
            asm volatile(
                "{\n\t.reg .pred p;\n\t"
                "setp.ne.u32 p, %5, 0;\n\t"
                "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
                "@p ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
                : "=&r"(r[i].x), "=&r"(r[i].y), "=&r"(r[i].z), "=&r"(r[i].w)
                : "l"(reinterpret_cast<const char*>(p) + 16 * i), "r"(static_cast<uint32_t>(on))
                : "memory");
        memcpy(&out, r, kBytes);
    } else if constexpr (kBytes == 8) {
        uint2 r;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.u32 p, %3, 0;\n\t"
            "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\t"
            "@p ld.global.v2.b32 {%0, %1}, [%2];\n\t}"
            : "=&r"(r.x), "=&r"(r.y)
            : "l"(p), "r"(static_cast<uint32_t>(on))
            : "memory");
        memcpy(&out, &r, kBytes);
    } else if constexpr (kBytes == 4) {
        uint32_t r;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.u32 p, %2, 0;\n\t"
            "mov.b32 %0, 0;\n\t"
            "@p ld.global.b32 %0, [%1];\n\t}"
            : "=&r"(r)
            : "l"(p), "r"(static_cast<uint32_t>(on))
            : "memory");
        memcpy(&out, &r, kBytes);
    } else {
        uint16_t r;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.u32 p, %2, 0;\n\t"
            "mov.b16 %0, 0;\n\t"
            "@p ld.global.b16 %0, [%1];\n\t}"
            : "=&h"(r)
            : "l"(p), "r"(static_cast<uint32_t>(on))
            : "memory");
        memcpy(&out, &r, kBytes);
    }
    return out;
}

// Pieces that a lane works on together: four with single elements, so that narrow loads keep as
// many bytes in flight.
constexpr int pieces(int vec) { return vec == 1 ? 4 : vec == 2 ? 2 : 1; }

// One warp copies 32*U vectors of one token's row to each of its places. The copy moves bytes
// only: V is the widest vector that the row length allows.
template <typename V, int U>
__global__ void __launch_bounds__(256) permute_kernel(const V* x, const int32_t* pos, V* out, int T, int K, int nvec,
                                                      int nseg) {
    pdl_wait();
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    const int t = static_cast<int>(unit / nseg), c0 = static_cast<int>(unit % nseg) * (32 * U) + lane;
    if (t >= T) return;
    const unsigned P = static_cast<unsigned>(T) * K;
    const int mypos = lane < K ? __ldg(pos + static_cast<int64_t>(t) * K + lane) : -1;
    V v[U];
    const V* xr = x + static_cast<int64_t>(t) * nvec;
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (c0 + 32 * u < nvec) v[u] = xr[c0 + 32 * u];
    for (int k = 0; k < K; ++k) {
        const unsigned p = static_cast<unsigned>(__shfl_sync(0xffffffffu, mypos, k));
        if (p >= P) continue;
        V* o = out + static_cast<int64_t>(p) * nvec;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c0 + 32 * u < nvec) o[c0 + 32 * u] = v[u];
    }
}

// `wpt` warps per token (8 / wpt tokens per CTA), each over every wpt-th run of 32 * U packs. The
// rows of up to 8 slots are in flight together and are added in slot order in fp32. Weights in
// fp64 are rounded to fp32 first (2^-24 relative, below the fp32 products' own rounding); the
// result is rounded once.
template <typename ZT, typename YT, typename RT, int VEC>
__global__ void __launch_bounds__(256) unpermute_kernel(UnpermuteArgs a, int wpt) {
    constexpr int U = pieces(VEC);
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (8 / wpt) + warp / wpt;
    if (t >= a.T) return;
    const Slots s = load_slots(a.pos, a.weights, a.wtype, t, a.K, static_cast<unsigned>(a.T) * a.K, lane);
    const RT* res = a.residual ? static_cast<const RT*>(a.residual) + t * a.H : nullptr;
    YT* yr = static_cast<YT*>(a.y) + t * a.H;
    for (int c0 = (warp % wpt) * (32 * VEC * U); c0 < a.H; c0 += wpt * (32 * VEC * U)) {   // the warp stays together
        int c[U];
        bool in[U];
        Pack<RT, VEC> r[U];
        float acc[U][VEC];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            c[i] = c0 + (32 * i + lane) * VEC;
            in[i] = c[i] < a.H;
            r[i] = load_if<RT, VEC>(res + c[i], res && in[i]);
#pragma unroll
            for (int j = 0; j < VEC; ++j) acc[i][j] = 0.f;
        }
        for (int s0 = 0; s0 < a.K; s0 += 8) {
            Pack<ZT, VEC> z[8][U];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const unsigned p = __shfl_sync(0xffffffffu, s.p, (s0 + u) & 31);
                const bool on = s0 + u < a.K && p != UINT_MAX;
                const ZT* zr = static_cast<const ZT*>(a.z) + static_cast<int64_t>(on ? p : 0u) * a.H;
#pragma unroll
                for (int i = 0; i < U; ++i) z[u][i] = load_if<ZT, VEC>(zr + c[i], on && in[i]);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (s0 + u < a.K) {   // unrouted: weight 0 on a row of zeros
                    const float w = __shfl_sync(0xffffffffu, s.w, (s0 + u) & 31);
#pragma unroll
                    for (int i = 0; i < U; ++i)
#pragma unroll
                        for (int j = 0; j < VEC; ++j) acc[i][j] = fmaf(w, up(z[u][i].v[j]), acc[i][j]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (in[i]) {
                Pack<YT, VEC> y;
#pragma unroll
                for (int j = 0; j < VEC; ++j) y.v[j] = down<YT>(res ? up(r[i].v[j]) + acc[i][j] : acc[i][j]);
                *reinterpret_cast<Pack<YT, VEC>*>(yr + c[i]) = y;
            }
        }
    }
}

// The same sums for large batches: each warp takes a contiguous range of (token, run) items, a run
// being kStreamPieces times 32 packs, and keeps the next items' rows on their way into shared
// memory (asynchronous copies into a ring of its own, nothing shared between threads), so that the
// loads in flight do not depend on registers. An item's rows are its token's routed slots only,
// kStreamRows at a time. (Bound by latency with few warps and by copies in flight with small rings:
// 16384 tokens of 8 bf16 rows take 92 to 100 us over one to two runs of packs, two to four rows and
// two or three stages; where a third of the slots is routed, two rows at a time and seven CTAs per SM
// are 10% ahead of four rows and three CTAs.)
constexpr int kStreamThreads = 128, kStreamStages = 3, kStreamRows = 2, kStreamPieces = 2;
constexpr int kStreamPack = kStreamThreads * 16;
constexpr int kStreamRes = kStreamRows * kStreamPieces * kStreamPack;        // residual packs behind the rows'
constexpr int kStreamSmem = 227 * 1024, kStreamMaxCtas = 7;                     // per SM

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
    if constexpr (BYTES == 32) {
        copy_async<16>(dst, src);
        copy_async<16>(dst + 16, static_cast<const char*>(src) + 16);
    } else if constexpr (BYTES == 16) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    } else {
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
    }
}

// Position in a warp's items: token, run of the row, and which of the token's routed slots.
struct Cursor {
    int64_t t;
    int left;         // items to go, this one included
    int run, s0, n;   // n routed slots of the token
    Slots s;          // lane j: place and weight of the j-th routed slot

    __device__ __forceinline__ void token(const UnpermuteArgs& a, int lane) {
        s = load_slots(a.pos, a.weights, a.wtype, t, a.K, static_cast<unsigned>(a.T) * a.K, lane);
        unsigned m = __ballot_sync(0xffffffffu, s.p != UINT_MAX);
        n = __popc(m);
        if (n < a.K) {   // close the gaps, keeping the order
            for (int j = 0; j < lane && m; ++j) m &= m - 1;
            const int from = m ? __ffs(m) - 1 : 31;
            __syncwarp();
            s.p = __shfl_sync(0xffffffffu, s.p, from);
            s.w = __shfl_sync(0xffffffffu, s.w, from);
        }
    }
    __device__ __forceinline__ void advance(const UnpermuteArgs& a, int runs, int lane) {
        s0 += kStreamRows;
        if (s0 < n) return;
        s0 = 0;
        --left;
        if (++run < runs) return;
        run = 0;
        ++t;
        if (left > 0) token(a, lane);
    }
};

template <typename ZT, typename YT, typename RT>
__global__ void __launch_bounds__(kStreamThreads, kStreamMaxCtas) unpermute_stream_kernel(UnpermuteArgs a, int runs,
                                                                                          int stage_bytes) {
    constexpr int VEC = 16 / sizeof(ZT), kRes = VEC * sizeof(RT);
    extern __shared__ __align__(16) unsigned char ring[];
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t items = static_cast<int64_t>(a.T) * runs, warps = static_cast<int64_t>(gridDim.x) * (kStreamThreads / 32);
    const int64_t me = static_cast<int64_t>(blockIdx.x) * (kStreamThreads / 32) + (threadIdx.x >> 5);
    const int64_t i0 = items * me / warps, i1 = items * (me + 1) / warps;   // items <= 2^30 * 2^24
    if (i0 >= i1) return;
    const uint32_t base = smem_u32(ring);
    Cursor in, out;
    out.t = i0 / runs;
    out.run = static_cast<int>(i0 - out.t * runs);
    out.left = static_cast<int>(i1 - i0);
    out.s0 = 0;
    out.token(a, lane);
    in = out;
    auto issue = [&](int stage) {
        if (in.left > 0) {
            const int c = (in.run * kStreamPieces * 32 + lane) * VEC;
            const uint32_t dst = base + stage * stage_bytes;
#pragma unroll
            for (int u = 0; u < kStreamRows; ++u) {
                if (in.s0 + u < in.n) {
                    const unsigned p = __shfl_sync(0xffffffffu, in.s.p, (in.s0 + u) & 31);
                    const ZT* zr = static_cast<const ZT*>(a.z) + static_cast<int64_t>(p) * a.H + c;
#pragma unroll
                    for (int i = 0; i < kStreamPieces; ++i)
                        if (c + i * 32 * VEC < a.H)
                            copy_async<16>(dst + (u * kStreamPieces + i) * kStreamPack + threadIdx.x * 16, zr + i * 32 * VEC);
                }
            }
            if (a.residual && in.s0 + kStreamRows >= in.n) {
                const RT* rr = static_cast<const RT*>(a.residual) + in.t * a.H + c;
#pragma unroll
                for (int i = 0; i < kStreamPieces; ++i)
                    if (c + i * 32 * VEC < a.H)
                        copy_async<kRes>(dst + kStreamRes + (i * kStreamThreads + threadIdx.x) * kRes, rr + i * 32 * VEC);
            }
            in.advance(a, runs, lane);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int i = 0; i < kStreamStages - 1; ++i) issue(i);
    float acc[kStreamPieces][VEC];
#pragma unroll
    for (int i = 0; i < kStreamPieces; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) acc[i][j] = 0.f;
    for (int stage = 0; out.left > 0; stage = stage + 1 == kStreamStages ? 0 : stage + 1) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStreamStages - 2) : "memory");
        issue(stage == 0 ? kStreamStages - 1 : stage - 1);   // the stage used up by the last round
        const int c = (out.run * kStreamPieces * 32 + lane) * VEC;
        const unsigned char* src = ring + stage * stage_bytes;
#pragma unroll
        for (int u = 0; u < kStreamRows; ++u) {
            if (out.s0 + u < out.n) {
                const float w = __shfl_sync(0xffffffffu, out.s.w, (out.s0 + u) & 31);
#pragma unroll
                for (int i = 0; i < kStreamPieces; ++i) {   // lanes behind the row work on what the ring holds
                    const Pack<ZT, VEC> z = *reinterpret_cast<const Pack<ZT, VEC>*>(
                        src + (u * kStreamPieces + i) * kStreamPack + threadIdx.x * 16);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) acc[i][j] = fmaf(w, up(z.v[j]), acc[i][j]);
                }
            }
        }
        if (out.s0 + kStreamRows >= out.n) {
#pragma unroll
            for (int i = 0; i < kStreamPieces; ++i) {
                Pack<YT, VEC> y;
                if (a.residual) {
                    const Pack<RT, VEC> r = *reinterpret_cast<const Pack<RT, VEC>*>(
                        src + kStreamRes + (i * kStreamThreads + threadIdx.x) * kRes);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) acc[i][j] = up(r.v[j]) + acc[i][j];
                }
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    y.v[j] = down<YT>(acc[i][j]);
                    acc[i][j] = 0.f;
                }
                if (c + i * 32 * VEC < a.H)
                    *reinterpret_cast<Pack<YT, VEC>*>(static_cast<YT*>(a.y) + out.t * a.H + c + i * 32 * VEC) = y;
            }
        }
        out.advance(a, runs, lane);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// The same for rows that are not whole 16-byte pieces: a row starts anywhere in a 16-byte block, so a
// warp copies the aligned blocks that cover its run (the blocks' other elements are not used; behind
// the end of the tensor nothing is read) and takes single elements from shared memory, lanes side by
// side. (4096 tokens of 8 bf16 rows of 2047 and a residual take 91 us with loads of single
// elements and 39 with this; 16384 tokens of 2: 203 and 63.)
// Lanes are laid over whole 128-byte lines, so that a run asks for each of its lines once.
constexpr int kShiftRow = kStreamPieces * 32 * 16 + 128;   // a warp's bytes of one row

// Starts the copy of the 16-byte blocks that hold elements [at, at + n) of a tensor of `total` elements;
// element `at` comes to place line_offset(at) of dst.
template <typename T>
__device__ __forceinline__ int line_offset(int64_t at) {
    return static_cast<int>(at) & (128 / static_cast<int>(sizeof(T)) - 1);
}
template <int RUN, typename T>   // n <= RUN
__device__ __forceinline__ void copy_blocks(uint32_t dst, const T* src, int64_t at, int n, int64_t total, int lane) {
    constexpr int kPer = 16 / sizeof(T);
    const int m = line_offset<T>(at), end = m + n;   // elements, from the line's start
    const T* line = src + (at - m);
    const int64_t rest = total - (at - m);   // elements from the line's start on; the last block may be short
    const int left = rest < end + kPer ? static_cast<int>(rest) : end + kPer;
#pragma unroll
    for (int i = 0; i < (RUN / kPer + 31) / 32 + 1; ++i) {
        const int e = (i * 32 + lane) * kPer;   // the block's first element
        if (e + kPer > m && e < end)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + e * static_cast<int>(sizeof(T))), "l"(line + e),
                         "r"(min(16, (left - e) * static_cast<int>(sizeof(T))))
                         : "memory");
    }
}

template <typename ZT, typename YT, typename RT>
__global__ void __launch_bounds__(kStreamThreads, kStreamMaxCtas) unpermute_shift_kernel(UnpermuteArgs a, int runs,
                                                                                         int stage_bytes) {
    constexpr int kRun = kStreamPieces * 32 * (16 / sizeof(ZT)), kEach = kRun / 32;
    extern __shared__ __align__(16) unsigned char ring[];
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t items = static_cast<int64_t>(a.T) * runs, warps = static_cast<int64_t>(gridDim.x) * (kStreamThreads / 32);
    const int64_t me = static_cast<int64_t>(blockIdx.x) * (kStreamThreads / 32) + (threadIdx.x >> 5);
    const int64_t i0 = items * me / warps, i1 = items * (me + 1) / warps;   // items <= 2^30 * 2^24
    if (i0 >= i1) return;
    unsigned char* mine = ring + (threadIdx.x >> 5) * stage_bytes * kStreamStages;
    const uint32_t base = smem_u32(mine);
    const int64_t z_total = static_cast<int64_t>(a.T) * a.K * a.H, r_total = static_cast<int64_t>(a.T) * a.H;
    Cursor in, out;
    out.t = i0 / runs;
    out.run = static_cast<int>(i0 - out.t * runs);
    out.left = static_cast<int>(i1 - i0);
    out.s0 = 0;
    out.token(a, lane);
    in = out;
    auto issue = [&](int stage) {
        if (in.left > 0) {
            const int c = in.run * kRun, n = min(kRun, a.H - c);
            const uint32_t dst = base + stage * stage_bytes;
#pragma unroll
            for (int u = 0; u < kStreamRows; ++u) {
                if (in.s0 + u < in.n) {
                    const unsigned p = __shfl_sync(0xffffffffu, in.s.p, (in.s0 + u) & 31);
                    copy_blocks<kRun>(dst + u * kShiftRow, static_cast<const ZT*>(a.z), static_cast<int64_t>(p) * a.H + c,
                                      n, z_total, lane);
                }
            }
            if (a.residual && in.s0 + kStreamRows >= in.n)
                copy_blocks<kRun>(dst + kStreamRows * kShiftRow, static_cast<const RT*>(a.residual), in.t * a.H + c, n,
                                  r_total, lane);
            in.advance(a, runs, lane);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int i = 0; i < kStreamStages - 1; ++i) issue(i);
    float acc[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j) acc[j] = 0.f;
    for (int stage = 0; out.left > 0; stage = stage + 1 == kStreamStages ? 0 : stage + 1) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStreamStages - 2) : "memory");
        __syncwarp();   // every lane's copies are there, and every lane is done with the last round's stage
        issue(stage == 0 ? kStreamStages - 1 : stage - 1);
        const int c = out.run * kRun, n = a.H - c;
        const unsigned char* src = mine + stage * stage_bytes;
#pragma unroll
        for (int u = 0; u < kStreamRows; ++u) {
            if (out.s0 + u < out.n) {
                const float w = __shfl_sync(0xffffffffu, out.s.w, (out.s0 + u) & 31);
                const unsigned p = __shfl_sync(0xffffffffu, out.s.p, (out.s0 + u) & 31);
                const ZT* z = reinterpret_cast<const ZT*>(src + u * kShiftRow) +
                              line_offset<ZT>(static_cast<int64_t>(p) * a.H + c) + lane;
#pragma unroll
                for (int q = 0; q < kEach; q += 4) {
                    if (32 * q < n) {   // elements behind the row are whatever the ring holds, and not stored
#pragma unroll
                        for (int j = q; j < q + 4; ++j) acc[j] = fmaf(w, up(z[32 * j]), acc[j]);
                    }
                }
            }
        }
        if (out.s0 + kStreamRows >= out.n) {
            YT* y = static_cast<YT*>(a.y) + out.t * a.H + c + lane;
            const RT* r = reinterpret_cast<const RT*>(src + kStreamRows * kShiftRow) +
                          line_offset<RT>(out.t * a.H + c) + lane;
#pragma unroll
            for (int j = 0; j < kEach; ++j) {
                if (lane + 32 * j < n) y[32 * j] = down<YT>(a.residual ? up(r[32 * j]) + acc[j] : acc[j]);
                acc[j] = 0.f;
            }
        }
        out.advance(a, runs, lane);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// Sums of 8 values over the lanes of a warp; lane l returns the sum of value l & 7 (in the order of
// the butterfly, the same in every run): halves of the values are exchanged while there are several.
__device__ __forceinline__ float warp_sums8(const float (&v)[8], int lane) {
    float a[4], b[2], c;
    const bool h0 = lane & 4, h1 = lane & 2, h2 = lane & 1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float got = __shfl_xor_sync(0xffffffffu, h0 ? v[i] : v[i + 4], 4);
        a[i] = (h0 ? v[i + 4] : v[i]) + got;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float got = __shfl_xor_sync(0xffffffffu, h1 ? a[i] : a[i + 2], 2);
        b[i] = (h1 ? a[i + 2] : a[i]) + got;
    }
    {
        const float got = __shfl_xor_sync(0xffffffffu, h2 ? b[0] : b[1], 1);
        c = (h2 ? b[1] : b[0]) + got;
    }
    c += __shfl_xor_sync(0xffffffffu, c, 8);
    c += __shfl_xor_sync(0xffffffffu, c, 16);
    return c;
}

// `wpt` warps per token (8 / wpt tokens per CTA), SLOTS rows at a time (2, 4 or 8), and more pieces of
// them the fewer they are (16384 tokens of 2 rows of 2048 bf16 take 54 us, with 8 slots 71, with 2 and
// one piece 62; of 2047 74, 143 and 91). Each thread
// reads its part of dy and the same part of the slots' rows, writes the rows' gradients and adds to
// their dot products; the dot products are then summed over the lanes and, in order, over the token's
// warps.
// Three CTAs per SM: two of them leave too few loads in flight (4096 tokens of 8 rows of 2048: fp32 109
// against 93 us, bf16 50 against 49).
template <typename T, int VEC, int SLOTS>
__global__ void __launch_bounds__(256, 3) unpermute_bwd_kernel(UnpermuteBwdArgs a, int wpt) {
    constexpr int U = pieces(VEC) * (8 / SLOTS);
    __shared__ float s_dot[8][8];
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wt = warp % wpt;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (8 / wpt) + warp / wpt;
    const bool live = t < a.T;
    Slots s{UINT_MAX, 0.f};
    if (live) s = load_slots(a.pos, a.weights, a.wtype, t, a.K, static_cast<unsigned>(a.T) * a.K, lane);
    const T* dyr = static_cast<const T*>(a.dy) + t * a.H;
    for (int s0 = 0; s0 < a.K; s0 += SLOTS) {
        float dot[8] = {}, w[SLOTS];
        unsigned p[SLOTS];
#pragma unroll
        for (int u = 0; u < SLOTS; ++u) {
            p[u] = __shfl_sync(0xffffffffu, s.p, (s0 + u) & 31);
            w[u] = __shfl_sync(0xffffffffu, s.w, (s0 + u) & 31);
            if (s0 + u >= a.K) p[u] = UINT_MAX;
        }
        for (int c0 = wt * (32 * VEC * U); live && c0 < a.H; c0 += wpt * (32 * VEC * U)) {
            Pack<T, VEC> dy[U], z[SLOTS][U];
            int c[U];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                c[i] = c0 + (32 * i + lane) * VEC;
                dy[i] = load_if<T, VEC>(dyr + c[i], c[i] < a.H);
            }
#pragma unroll
            for (int u = 0; u < SLOTS; ++u) {
                const T* zr = static_cast<const T*>(a.z) + static_cast<int64_t>(p[u] != UINT_MAX ? p[u] : 0u) * a.H;
#pragma unroll
                for (int i = 0; i < U; ++i) z[u][i] = load_if<T, VEC>(zr + c[i], p[u] != UINT_MAX && c[i] < a.H);
            }
#pragma unroll
            for (int u = 0; u < SLOTS; ++u) {
                if (p[u] == UINT_MAX) continue;
                T* dzr = static_cast<T*>(a.dz) + static_cast<int64_t>(p[u]) * a.H;
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    Pack<T, VEC> g;
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        const float d = up(dy[i].v[j]);
                        dot[u] = fmaf(d, up(z[u][i].v[j]), dot[u]);
                        g.v[j] = down<T>(w[u] * d);
                    }
                    if (c[i] < a.H) *reinterpret_cast<Pack<T, VEC>*>(dzr + c[i]) = g;
                }
            }
        }
        __syncwarp();
        float d = warp_sums8(dot, lane);   // 0 for unrouted slots
        if (wpt > 1) {
            if (lane < 8) s_dot[warp][lane] = d;
            __syncthreads();
            if (wt == 0 && lane < 8) {
                d = 0.f;
                for (int v = 0; v < wpt; ++v) d += s_dot[warp + v][lane];
            }
            __syncthreads();
        }
        if (live && wt == 0 && lane < SLOTS && s0 + lane < a.K) a.dweights[t * a.K + s0 + lane] = d;
    }
}

// Warps per token: enough to fill the GPU (32 warps per SM), no more than the row has runs.
int warps_per_token(int T, int H, int run, int sms) {
    int w = 1;
    while (w < 8 && static_cast<int64_t>(T) * w < 32 * sms && w * run < H) w *= 2;
    return w;
}

// Elements per pack: the widest of 16 bytes (of the narrower type) that divides the row.
int pack_of(int H, int widest) {
    int v = widest;
    while (H % v) v /= 2;
    return v;
}

template <typename V>
cudaError_t permute_vec(const void* x, const int32_t* pos, void* out, int T, int K, int nvec, cudaStream_t stream,
                        int sms) {
    // four vectors per lane where that still leaves eight warps per SM, else one
    const bool wide = static_cast<int64_t>(T) * ((nvec + 127) / 128) >= 8 * sms;
    int nseg = wide ? (nvec + 127) / 128 : (nvec + 31) / 32;
    const int64_t blocks = (static_cast<int64_t>(T) * nseg + 7) / 8;
    if (blocks > INT_MAX) return cudaErrorInvalidValue;
    void* args[] = {&x, &pos, &out, &T, &K, &nvec, &nseg};
    const void* fn = wide ? reinterpret_cast<const void*>(permute_kernel<V, 4>)
                          : reinterpret_cast<const void*>(permute_kernel<V, 1>);
    return launch_pdl_raw(fn, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream, args);
}

template <typename ZT, typename YT, typename RT>
cudaError_t unpermute_types(const UnpermuteArgs& a, cudaStream_t stream, int sms) {
    constexpr int kWidest = sizeof(ZT) == 2 ? 8 : 4;
    const int vec = pack_of(a.H, kWidest);
    int wpt = warps_per_token(a.T, a.H, 32 * vec * pieces(vec), sms);
    UnpermuteArgs b = a;
    constexpr int kRun = kStreamPieces * 32 * kWidest;
    const int runs = (a.H - 1) / kRun + 1;
    const bool whole = vec == kWidest;
    int stage_bytes = whole ? kStreamRes : kStreamRows * kShiftRow;   // shifted: of one warp
    if (a.residual) stage_bytes += whole ? kRun * static_cast<int>(sizeof(RT)) * (kStreamThreads / 32)
                                         : kRun * static_cast<int>(sizeof(RT)) + 128;
    const int smem = kStreamStages * stage_bytes * (whole ? 1 : kStreamThreads / 32);
    int per_sm = kStreamSmem / (smem + 1024);   // the system takes 1 KB of each CTA's
    per_sm = per_sm < kStreamMaxCtas ? per_sm : kStreamMaxCtas;
    // two items per warp at least, and two CTAs per SM (8 rows of 2048 bf16 per token: at 512 tokens 5.5
    // us with the ring, 5.0 without; at 1024 tokens 8.0 and 13.2, at 4096 26.6 and 40.8)
    // Rows that start inside a block: full runs' worth of elements for four (8 rows per token; ring and
    // without: 4096 tokens of 321 bf16 17.6 and 11.5, of 513 19.5 and 22.8; 16384 tokens of 65 fp32 27.8
    // and 18.6, of 201 23.6 and 38.3).
    const int64_t fed = (whole ? static_cast<int64_t>(a.T) * runs : static_cast<int64_t>(a.T) * a.H / kRun) / (kStreamThreads / 32 * 2);
    if (fed >= (whole ? 2 : 4) * sms) {
        const int ctas = fed < per_sm * sms ? static_cast<int>(fed) : per_sm * sms;
        const void* fn = whole ? reinterpret_cast<const void*>(unpermute_stream_kernel<ZT, YT, RT>)
                               : reinterpret_cast<const void*>(unpermute_shift_kernel<ZT, YT, RT>);
        const cudaError_t err = allow_dynamic_smem(fn, static_cast<size_t>(smem));   // with or without a residual
        if (err != cudaSuccess) return err;
        int r = runs;
        void* sargs[] = {&b, &r, &stage_bytes};
        return launch_pdl_raw(fn, dim3(ctas), dim3(kStreamThreads), static_cast<size_t>(smem), stream, sargs);
    }
    void* args[] = {&b, &wpt};
    const void* fn = vec == kWidest ? reinterpret_cast<const void*>(unpermute_kernel<ZT, YT, RT, kWidest>)
                     : vec == 4     ? reinterpret_cast<const void*>(unpermute_kernel<ZT, YT, RT, 4>)
                     : vec == 2     ? reinterpret_cast<const void*>(unpermute_kernel<ZT, YT, RT, 2>)
                                    : reinterpret_cast<const void*>(unpermute_kernel<ZT, YT, RT, 1>);
    return launch_pdl_raw(fn, dim3((a.T - 1) / (8 / wpt) + 1), dim3(256), 0, stream, args);
}

// the residual has y's type or is fp32
template <typename ZT, typename YT>
cudaError_t unpermute_residual(const UnpermuteArgs& a, bool res32, cudaStream_t stream, int sms) {
    return res32 ? unpermute_types<ZT, YT, float>(a, stream, sms) : unpermute_types<ZT, YT, YT>(a, stream, sms);
}

template <typename T>
cudaError_t unpermute_bwd_type(const UnpermuteBwdArgs& a, cudaStream_t stream, int sms) {
    constexpr int kWidest = 16 / sizeof(T);
    const int vec = pack_of(a.H, kWidest);
    const int slots = a.K <= 2 ? 2 : a.K <= 4 ? 4 : 8;
    int wpt = warps_per_token(a.T, a.H, 32 * vec * pieces(vec) * (8 / slots), sms);
    UnpermuteBwdArgs b = a;
    void* args[] = {&b, &wpt};
    auto pick = [&](auto slots) {
        constexpr int S = decltype(slots)::value;
        return vec == kWidest ? reinterpret_cast<const void*>(unpermute_bwd_kernel<T, kWidest, S>)
               : vec == 4     ? reinterpret_cast<const void*>(unpermute_bwd_kernel<T, 4, S>)
               : vec == 2     ? reinterpret_cast<const void*>(unpermute_bwd_kernel<T, 2, S>)
                              : reinterpret_cast<const void*>(unpermute_bwd_kernel<T, 1, S>);
    };
    const void* fn = slots == 2   ? pick(std::integral_constant<int, 2>{})
                     : slots == 4 ? pick(std::integral_constant<int, 4>{})
                                  : pick(std::integral_constant<int, 8>{});
    return launch_pdl_raw(fn, dim3((a.T - 1) / (8 / wpt) + 1), dim3(256), 0, stream, args);
}

}  // namespace

int sort_chunk_pairs(int P) {
    if (P <= kSortOneBlock) return P;
    const int per = (P - 1) / 64 + 1 <= 8 * kSortThreads ? (P - 1) / 64 + 1 : (P - 1) / 128 + 1;
    return (per + kSortChunk - 1) / kSortChunk * kSortChunk;
}

// Counts of the chunks of any batch of up to P pairs.
size_t sort_hist_bytes(int P, int E) {
    if (P <= kSortOneBlock) return 0;
    const int nb = (P - 1) / kSortChunk + 1;
    return static_cast<size_t>(nb < 128 ? nb : 128) * (E + 1) * 4;
}

cudaError_t launch_sort_pairs(const SortArgs& a, cudaStream_t stream) {
    SortArgs b = a;
    b.chunk = sort_chunk_pairs(a.P);
    const int nb = (a.P - 1) / b.chunk + 1;
    int threads = kSortThreads;
    if (nb == 1) {
        // a warp per 32 pairs, and at least four for the scan over the experts
        threads = ((a.P + 31) / 32) * 32;
        threads = threads < 128 ? 128 : threads > kSortThreads ? kSortThreads : threads;
    }
    const int rounds = (((b.chunk < a.P ? b.chunk : a.P) + threads / 32 - 1) / (threads / 32) + 31) / 32;   // per warp
    const void* fn = rounds <= 1   ? reinterpret_cast<const void*>(sort_place_kernel<1>)
                     : rounds <= 4 ? reinterpret_cast<const void*>(sort_place_kernel<4>)
                     : rounds <= 8 ? reinterpret_cast<const void*>(sort_place_kernel<8>)
                                   : reinterpret_cast<const void*>(sort_place_kernel<0>);
    const size_t smem = sort_smem_bytes(threads / 32, a.E);
    if (smem > kDefaultDynamicSmem) {   // before the first launch: an error leaves nothing launched
        const cudaError_t err =
            cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(sort_smem_bytes(kSortThreads / 32, kSortMaxExperts)));
        if (err != cudaSuccess) return err;
    }
    void* args[] = {&b};
    if (nb > 1) {
        const cudaError_t err = launch_pdl_raw(reinterpret_cast<const void*>(sort_count_kernel), dim3(nb),
                                               dim3(kSortThreads), static_cast<size_t>(a.E + 1) * 4, stream, args);
        if (err != cudaSuccess) return err;
    }
    return launch_pdl_raw(fn, dim3(nb), dim3(threads), smem, stream, args);
}

cudaError_t launch_permute_pairs(int elem_bytes, const void* x, const int32_t* pos, int T, int K, int H, void* out,
                                 cudaStream_t stream, int sms) {
    const int64_t bytes = static_cast<int64_t>(H) * elem_bytes;
    const int width = bytes % 16 == 0 ? 16 : bytes % 8 == 0 ? 8 : bytes % 4 == 0 ? 4 : 2;
    const int nvec = static_cast<int>(bytes / width);
    switch (width) {
        case 16: return permute_vec<uint4>(x, pos, out, T, K, nvec, stream, sms);
        case 8: return permute_vec<uint2>(x, pos, out, T, K, nvec, stream, sms);
        case 4: return permute_vec<uint32_t>(x, pos, out, T, K, nvec, stream, sms);
        default: return permute_vec<uint16_t>(x, pos, out, T, K, nvec, stream, sms);
    }
}

cudaError_t launch_unpermute(const UnpermuteArgs& a, int ztype, int ytype, bool res32, cudaStream_t stream, int sms) {
    if (ztype == DPA_DTYPE_BF16 && ytype == DPA_DTYPE_BF16) return unpermute_residual<__nv_bfloat16, __nv_bfloat16>(a, res32, stream, sms);
    if (ztype == DPA_DTYPE_FP16 && ytype == DPA_DTYPE_FP16) return unpermute_residual<__half, __half>(a, res32, stream, sms);
    if (ztype == DPA_DTYPE_FP32 && ytype == DPA_DTYPE_FP32) return unpermute_residual<float, float>(a, res32, stream, sms);
    if (ztype == DPA_DTYPE_BF16 && ytype == DPA_DTYPE_FP32) return unpermute_residual<__nv_bfloat16, float>(a, res32, stream, sms);
    if (ztype == DPA_DTYPE_FP16 && ytype == DPA_DTYPE_FP32) return unpermute_residual<__half, float>(a, res32, stream, sms);
    if (ztype == DPA_DTYPE_FP32 && ytype == DPA_DTYPE_BF16) return unpermute_residual<float, __nv_bfloat16>(a, res32, stream, sms);
    if (ztype == DPA_DTYPE_FP32 && ytype == DPA_DTYPE_FP16) return unpermute_residual<float, __half>(a, res32, stream, sms);
    return cudaErrorInvalidValue;
}

cudaError_t launch_unpermute_bwd(const UnpermuteBwdArgs& a, int type, cudaStream_t stream, int sms) {
    switch (type) {
        case DPA_DTYPE_BF16: return unpermute_bwd_type<__nv_bfloat16>(a, stream, sms);
        case DPA_DTYPE_FP16: return unpermute_bwd_type<__half>(a, stream, sms);
        case DPA_DTYPE_FP32: return unpermute_bwd_type<float>(a, stream, sms);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace dpa
