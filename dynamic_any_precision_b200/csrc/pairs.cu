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
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace dpa {
namespace {

// ---------------------------------------------------------------- sort

constexpr int kSortThreads = 512;
constexpr int kSortOneBlock = 4096;   // pairs that one CTA sorts alone (one launch)

__device__ __forceinline__ int pair_key(const int32_t* idx, int p, int E) {
    const int e = __ldg(idx + p);
    return static_cast<unsigned>(e) < static_cast<unsigned>(E) ? e : E;
}

// Pairs per expert of each CTA's chunk: hist[b][key], key = E for unrouted pairs.
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(SortArgs a) {
    extern __shared__ int32_t s_cnt[];
    const int E1 = a.E + 1;
    for (int i = threadIdx.x; i < E1; i += kSortThreads) s_cnt[i] = 0;
    __syncthreads();
    pdl_wait();
    const int p0 = blockIdx.x * a.chunk, p1 = min(a.P - p0, a.chunk) + p0;
    for (int p = p0 + threadIdx.x; p < p1; p += kSortThreads) atomicAdd(&s_cnt[pair_key(a.idx, p, a.E)], 1);
    __syncthreads();
    int32_t* h = a.hist + static_cast<size_t>(blockIdx.x) * E1;
    for (int i = threadIdx.x; i < E1; i += kSortThreads) h[i] = s_cnt[i];
}

// Places of one CTA's chunk. Each warp owns a contiguous run of the chunk and counts it by key
// (lanes of equal key found with match), the counts are scanned over warps, earlier chunks and
// keys, and a second pass over the run hands out the places in order.
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(SortArgs a) {
    extern __shared__ int32_t smem[];
    const int E1 = a.E + 1, nw = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t* s_warp = smem;               // [nw][E1] counts, later the next place
    int32_t* s_tot = smem + nw * E1;      // [E1] pairs of the key in all chunks
    int32_t* s_pre = s_tot + E1;          // [E1] pairs of the key in earlier chunks
    __shared__ int32_t s_sum[32];
    for (int i = threadIdx.x; i < nw * E1; i += blockDim.x) s_warp[i] = 0;
    __syncthreads();
    pdl_wait();
    const int p0 = blockIdx.x * a.chunk, n = min(a.P - p0, a.chunk);
    const int run = (((n + nw - 1) / nw) + 31) & ~31;
    const int w0 = p0 + min(warp * run, n), w1 = p0 + min(warp * run + run, n);
    int32_t* mine = s_warp + warp * E1;
    for (int b = w0; b < w1; b += 32) {
        const int p = b + lane;
        const int key = p < w1 ? pair_key(a.idx, p, a.E) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, key);
        if (key >= 0 && lane == __ffs(same) - 1) mine[key] += __popc(same);
        __syncwarp();
    }
    if (gridDim.x > 1) {
        for (int e = threadIdx.x; e < E1; e += blockDim.x) {
            const int32_t* h = a.hist + e;
            int tot = 0, pre = 0;
#pragma unroll 8
            for (int b = 0; b < static_cast<int>(gridDim.x); ++b) {
                const int c = __ldcg(h + static_cast<size_t>(b) * E1);
                pre = b == static_cast<int>(blockIdx.x) ? tot : pre;
                tot += c;
            }
            s_tot[e] = tot;
            s_pre[e] = pre;
        }
    }
    __syncthreads();
    // counts -> places before this warp's run, per key
    for (int e = threadIdx.x; e < E1; e += blockDim.x) {
        int acc = gridDim.x > 1 ? s_pre[e] : 0;
#pragma unroll 4
        for (int w = 0; w < nw; ++w) {
            const int c = s_warp[w * E1 + e];
            s_warp[w * E1 + e] = acc;
            acc += c;
        }
        if (gridDim.x == 1) s_tot[e] = acc;
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
    for (int b = w0; b < w1; b += 32) {
        const int p = b + lane;
        const int key = p < w1 ? pair_key(a.idx, p, a.E) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, key);
        if (key >= 0) {
            const int at = mine[key] + s_tot[key] + __popc(same & ((1u << lane) - 1));
            a.pos[p] = key < a.E ? at : -1;
            a.order[at] = p;
        }
        __syncwarp();
        if (key >= 0 && lane == __ffs(same) - 1) mine[key] += __popc(same);
        __syncwarp();
    }
}

size_t sort_smem_bytes(int warps, int E) { return static_cast<size_t>(warps + 2) * (E + 1) * 4; }

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

__device__ __forceinline__ float load_weight(const void* w, int wtype, int64_t i) {
    if (wtype == DPA_DTYPE_FP64) return static_cast<float>(__ldg(static_cast<const double*>(w) + i));
    if (wtype == DPA_DTYPE_FP32) return __ldg(static_cast<const float*>(w) + i);
    return 1.f;   // no weights
}

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

// One thread per (token, VEC elements); the rows of up to 8 slots are in flight together and are
// added in slot order in fp32. Weights in fp64 are rounded to fp32 first (2^-24 relative, below
// the fp32 products' own rounding); the result is rounded once.
template <typename ZT, typename YT, int VEC>
__global__ void __launch_bounds__(256) unpermute_kernel(UnpermuteArgs a, int nvec) {
    pdl_wait();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t t = i / nvec;
    if (t >= a.T) return;
    const int64_t c = (i - t * nvec) * VEC;
    const unsigned P = static_cast<unsigned>(a.T) * a.K;
    float acc[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) acc[j] = 0.f;
    Pack<YT, VEC> r;
    if (a.residual) r = *reinterpret_cast<const Pack<YT, VEC>*>(static_cast<const YT*>(a.residual) + t * a.H + c);
    for (int s0 = 0; s0 < a.K; s0 += 8) {
        Pack<ZT, VEC> z[8];
        float w[8];
        bool on[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            on[u] = false;
            if (s0 + u < a.K) {
                const unsigned p = static_cast<unsigned>(__ldg(a.pos + t * a.K + s0 + u));
                on[u] = p < P;
                if (on[u]) {
                    w[u] = load_weight(a.weights, a.wtype, t * a.K + s0 + u);
                    z[u] = *reinterpret_cast<const Pack<ZT, VEC>*>(static_cast<const ZT*>(a.z) +
                                                                   static_cast<int64_t>(p) * a.H + c);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            if (on[u]) {
#pragma unroll
                for (int j = 0; j < VEC; ++j) acc[j] = fmaf(w[u], up(z[u].v[j]), acc[j]);
            }
        }
    }
    Pack<YT, VEC> y;
#pragma unroll
    for (int j = 0; j < VEC; ++j) y.v[j] = down<YT>(a.residual ? up(r.v[j]) + acc[j] : acc[j]);
    *reinterpret_cast<Pack<YT, VEC>*>(static_cast<YT*>(a.y) + t * a.H + c) = y;
}

// WPT warps per token (8 / WPT tokens per CTA). Each thread holds its part of dy, reads the same
// part of up to 8 slots' rows, writes their gradients and adds to their dot products; the dot
// products are then summed over the lanes by shuffles and over the warps in order.
template <typename T, int VEC, int WPT>
__global__ void __launch_bounds__(256) unpermute_bwd_kernel(UnpermuteBwdArgs a) {
    __shared__ float s_dot[8][8];
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, wt = warp % WPT;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * (8 / WPT) + warp / WPT;
    const bool live = t < a.T;
    const unsigned P = static_cast<unsigned>(a.T) * a.K;
    const T* dyr = static_cast<const T*>(a.dy) + t * a.H;
    for (int s0 = 0; s0 < a.K; s0 += 8) {
        float dot[8], w[8];
        unsigned p[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            dot[u] = 0.f;
            p[u] = UINT_MAX;
            if (live && s0 + u < a.K) {
                p[u] = static_cast<unsigned>(__ldg(a.pos + t * a.K + s0 + u));
                if (p[u] < P) w[u] = load_weight(a.weights, a.wtype, t * a.K + s0 + u);
            }
        }
        for (int c = (wt * 32 + lane) * VEC; live && c < a.H; c += 32 * WPT * VEC) {
            const Pack<T, VEC> dy = *reinterpret_cast<const Pack<T, VEC>*>(dyr + c);
            Pack<T, VEC> z[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (p[u] < P)
                    z[u] = *reinterpret_cast<const Pack<T, VEC>*>(static_cast<const T*>(a.z) +
                                                                  static_cast<int64_t>(p[u]) * a.H + c);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (p[u] < P) {
                    Pack<T, VEC> g;
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        const float d = up(dy.v[j]);
                        dot[u] = fmaf(d, up(z[u].v[j]), dot[u]);
                        g.v[j] = down<T>(w[u] * d);
                    }
                    *reinterpret_cast<Pack<T, VEC>*>(static_cast<T*>(a.dz) + static_cast<int64_t>(p[u]) * a.H + c) = g;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            for (int o = 16; o > 0; o >>= 1) dot[u] += __shfl_xor_sync(0xffffffffu, dot[u], o);
            if (lane == 0) s_dot[warp][u] = dot[u];
        }
        __syncthreads();
        if (live && wt == 0 && lane < 8 && s0 + lane < a.K) {
            float d = 0.f;
#pragma unroll
            for (int v = 0; v < WPT; ++v) d += s_dot[warp + v][lane];
            a.dweights[t * a.K + s0 + lane] = d;
        }
        __syncthreads();
    }
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

template <typename ZT, typename YT>
cudaError_t unpermute_types(const UnpermuteArgs& a, cudaStream_t stream) {
    constexpr int VEC = sizeof(ZT) < sizeof(YT) ? 16 / sizeof(YT) * 2 : 16 / sizeof(ZT);
    const bool vec = a.H % VEC == 0;
    int nvec = vec ? a.H / VEC : a.H;
    const int64_t blocks = (static_cast<int64_t>(a.T) * nvec + 255) / 256;
    if (blocks > INT_MAX) return cudaErrorInvalidValue;
    UnpermuteArgs b = a;
    void* args[] = {&b, &nvec};
    const void* fn = vec ? reinterpret_cast<const void*>(unpermute_kernel<ZT, YT, VEC>)
                         : reinterpret_cast<const void*>(unpermute_kernel<ZT, YT, 1>);
    return launch_pdl_raw(fn, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream, args);
}

template <typename T, int VEC>
cudaError_t unpermute_bwd_vec(const UnpermuteBwdArgs& a, cudaStream_t stream) {
    const int lanes = (a.H + VEC - 1) / VEC;
    UnpermuteBwdArgs b = a;
    void* args[] = {&b};
    auto go = [&](const void* fn, int wpt) {
        const int per = 8 / wpt;
        return launch_pdl_raw(fn, dim3((a.T - 1) / per + 1), dim3(256), 0, stream, args);
    };
    if (lanes <= 32) return go(reinterpret_cast<const void*>(unpermute_bwd_kernel<T, VEC, 1>), 1);
    if (lanes <= 64) return go(reinterpret_cast<const void*>(unpermute_bwd_kernel<T, VEC, 2>), 2);
    if (lanes <= 128) return go(reinterpret_cast<const void*>(unpermute_bwd_kernel<T, VEC, 4>), 4);
    return go(reinterpret_cast<const void*>(unpermute_bwd_kernel<T, VEC, 8>), 8);
}

template <typename T>
cudaError_t unpermute_bwd_type(const UnpermuteBwdArgs& a, cudaStream_t stream) {
    constexpr int VEC = 16 / sizeof(T);
    return a.H % VEC == 0 ? unpermute_bwd_vec<T, VEC>(a, stream) : unpermute_bwd_vec<T, 1>(a, stream);
}

}  // namespace

int sort_chunk_pairs(int P) {
    if (P <= kSortOneBlock) return P;
    const int per = (P - 1) / 128 + 1;   // at most 128 chunks
    return per <= 1024 ? 1024 : (per + 511) & ~511;
}

// Counts of the chunks of any batch of up to P pairs.
size_t sort_hist_bytes(int P, int E) {
    if (P <= kSortOneBlock) return 0;
    const int nb = (P - 1) / 1024 + 1;
    return static_cast<size_t>(nb < 128 ? nb : 128) * (E + 1) * 4;
}

cudaError_t launch_sort_pairs(const SortArgs& a, cudaStream_t stream) {
    SortArgs b = a;
    b.chunk = sort_chunk_pairs(a.P);
    const int nb = (a.P - 1) / b.chunk + 1;
    void* args[] = {&b};
    int threads = kSortThreads;
    if (nb > 1) {
        const cudaError_t err = launch_pdl_raw(reinterpret_cast<const void*>(sort_count_kernel), dim3(nb),
                                               dim3(kSortThreads), static_cast<size_t>(a.E + 1) * 4, stream, args);
        if (err != cudaSuccess) return err;
    } else {
        // a warp per 32 pairs, and at least four for the scan over the experts
        threads = ((a.P + 31) / 32) * 32;
        threads = threads < 128 ? 128 : threads > kSortThreads ? kSortThreads : threads;
    }
    const size_t smem = sort_smem_bytes(threads / 32, a.E);
    if (smem > 48 * 1024) {
        const cudaError_t err = cudaFuncSetAttribute(reinterpret_cast<const void*>(sort_place_kernel),
                                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     static_cast<int>(sort_smem_bytes(kSortThreads / 32, kSortMaxExperts)));
        if (err != cudaSuccess) return err;
    }
    return launch_pdl_raw(reinterpret_cast<const void*>(sort_place_kernel), dim3(nb), dim3(threads), smem, stream, args);
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

cudaError_t launch_unpermute(const UnpermuteArgs& a, int ztype, int ytype, cudaStream_t stream) {
    if (ztype == DPA_DTYPE_BF16 && ytype == DPA_DTYPE_BF16) return unpermute_types<__nv_bfloat16, __nv_bfloat16>(a, stream);
    if (ztype == DPA_DTYPE_FP16 && ytype == DPA_DTYPE_FP16) return unpermute_types<__half, __half>(a, stream);
    if (ztype == DPA_DTYPE_FP32 && ytype == DPA_DTYPE_FP32) return unpermute_types<float, float>(a, stream);
    if (ztype == DPA_DTYPE_BF16 && ytype == DPA_DTYPE_FP32) return unpermute_types<__nv_bfloat16, float>(a, stream);
    if (ztype == DPA_DTYPE_FP16 && ytype == DPA_DTYPE_FP32) return unpermute_types<__half, float>(a, stream);
    if (ztype == DPA_DTYPE_FP32 && ytype == DPA_DTYPE_BF16) return unpermute_types<float, __nv_bfloat16>(a, stream);
    if (ztype == DPA_DTYPE_FP32 && ytype == DPA_DTYPE_FP16) return unpermute_types<float, __half>(a, stream);
    return cudaErrorInvalidValue;
}

cudaError_t launch_unpermute_bwd(const UnpermuteBwdArgs& a, int type, cudaStream_t stream) {
    switch (type) {
        case DPA_DTYPE_BF16: return unpermute_bwd_type<__nv_bfloat16>(a, stream);
        case DPA_DTYPE_FP16: return unpermute_bwd_type<__half>(a, stream);
        case DPA_DTYPE_FP32: return unpermute_bwd_type<float>(a, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace dpa
