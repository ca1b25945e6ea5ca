// Host side of the dense matrix products: which kernel and which tiles a call takes, the tensor maps,
// and the launch. The tensor-memory kernel is in linear_tc.cuh, compiled here for output rows of whole
// 16-byte groups and in linear_tc_odd.cu for the others.
#include <mutex>

#include "linear_tc.cuh"

namespace dpa {

template cudaError_t launch_linear_variant<true>(const LinearArgs&, const LinearLaunch&, cudaStream_t);
extern template cudaError_t launch_linear_variant<false>(const LinearArgs&, const LinearLaunch&, cudaStream_t);

namespace {

// 16-bit [groups][rows][cols] tensor, boxes of 64 columns x box_rows, 128-byte swizzle, zero fill
bool encode_map(CUtensorMap* map, const void* base, bool f16, uint64_t cols, uint64_t rows, uint64_t groups,
                uint32_t box_rows, int rank) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {cols, rows, groups};
    const cuuint64_t strides[2] = {cols * 2, cols * rows * 2};
    const cuuint32_t box[3] = {kStepK, box_rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank,
              const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Clusters of S CTAs of the kernel that the current device holds at once (S <= 8; asked once per
// device). Fewer than its SMs / S: a cluster's SMs lie in one GPC (148 SMs: 45, 33, 26, 22, 15, 15
// clusters of 3 to 8).
int cluster_capacity(int S) {
    constexpr int kDevices = 64;
    static std::mutex mu;
    static int known[kDevices][9];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return 0;
    std::lock_guard<std::mutex> lock(mu);
    int& n = known[dev][S];
    if (n == 0) {
        const void* fn = reinterpret_cast<const void*>(linear_kernel<1, false, false, false, true>);
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(256 * S));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kSmemMax;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(S);
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess || n < 1) {
            n = -1;   // K is not split then
            (void)cudaGetLastError();
        }
    }
    return n;
}

// CTAs that share a tile's K: the most for which every tile's cluster runs at once. (64x2048x2048: 16
// tiles, 6.9 us with 6 each; with 8 each, of which 15 fit, 12.5 us.)
int split_k(int64_t tiles, int ksteps) {
    for (int S = ksteps < 8 ? ksteps : 8; S > 1; --S)
        if (tiles <= cluster_capacity(S)) return S;
    return 1;
}

// Rows per token tile, at most `most`, for pairs of CTAs: those for which the rounds of tiles over the
// GPU's pairs take the least time, about rounds x (tile rows + 100).
// Equal tiles of at most 256 alone leave pairs without work: 600x2048x4096 (48 tiles of 224 on 74 pairs)
// 16.3 us, as 64 of 160 13.7; 2048x2048x1408 with a gate (two rounds of 256) 27.2, of 160 21.3;
// 4819x1680x408 (one of 256) 15.9, of 160 13.0.
int pair_rows(int rows, int most, int FT, int pairs) {
    int best = 0;
    int64_t least = INT64_MAX;
    for (int tn = most; tn > 0; tn -= 32) {   // a multiple of 16 per CTA
        const int even = balanced_rows(rows, tn, 32);
        const int64_t tiles = static_cast<int64_t>((rows - 1) / even + 1) * FT;
        const int64_t cost = ((tiles - 1) / pairs + 1) * (even + 100);
        if (cost < least) {
            least = cost;
            best = even;
        }
    }
    return best;
}

// Whether the register kernel takes the call. Plain: up to 16 rows, and up to 32 where the weights are
// small, so that start-up counts (32 rows: 2048x2816 6.6 us against 6.9 here; gated 10.4 against 8.3).
// Grouped: up to 64 rows, 8 per group on average (8 tokens of top-8 through 128 experts of 2048x768
// gated: 54 us against 62 here; 16 tokens 81 against 84, and the down products 50 against 47). The average
// is over all groups, the empty ones included, for only the device knows the offsets: rows that all meet
// in one group take turns of 8 (64 rows in one of 8 groups of 2048x768 gated: 21.4 us against 12.7; spread
// over the 8 groups 8.5 against 11.9).
bool few_rows(const LinearArgs& a, bool gated) {
    if (a.E > 0) return a.rows <= 64 && a.rows <= 8 * a.E;
    return a.rows <= 16 || (a.rows <= 32 && static_cast<int64_t>(a.K) * a.N * (gated ? 2 : 1) <= 1 << 23);
}

}  // namespace

cudaError_t launch_linear(const LinearArgs& in, bool f16, const void* x, const void* w, const void* w_mul,
                          cudaStream_t stream, int sms) {
    if (few_rows(in, w_mul != nullptr)) return launch_linear_few(in, f16, x, w, w_mul, stream, sms);
    LinearArgs a = in;
    const bool gated = w_mul != nullptr;
    const int feat = gated ? 64 : 128;   // output features per CTA
    a.ksteps = (a.K - 1) / kStepK + 1;
    const int mean = a.E > 0 ? (a.rows - 1) / a.E + 1 : a.rows;   // rows per group
    const int groups = a.E > 0 ? a.E : 1;
    // a pair of CTAs per tile where tiles of 256 tokens are reasonably full and fill half the SMs
    const int64_t pair_tiles = static_cast<int64_t>(groups) * ((mean - 1) / 256 + 1) * ((a.N - 1) / (2 * feat) + 1);
    // (not where one CTA's features are all there are, which leaves the other none: 55 experts of 138
    // rows, 1192x43 with a gate, 14.3 us without pairs, 21.1 with)
    const bool pair = mean >= 64 && pair_tiles >= sms / 4 && a.N > feat;
    const int CG = pair ? 2 : 1;
    a.FT = (a.N - 1) / (feat * CG) + 1;
    a.splits = 1;
    int64_t clusters;
    // K blocks: the tensor cores drop the bits below the accumulator's last place at every step of 16
    // inputs, which takes about 1e-9 of the sum per input away (K = 8192: 9e-6; with a gate twice
    // that). 16-bit outputs see it in very long sums only (long_sums). For fp32 outputs blocks of 256
    // inputs are added in fp32 with rounding, from the length on where one accumulator's error would pass
    // 1e-6 of the outputs (root mean squares over random terms): at 768 inputs 9.5e-7, with an activation
    // at 512 7.7e-7 (it widens the error), with a gate at 256 6.4e-7. In blocks it is 3.4e-7 to 3.6e-7 up to
    // 8192 inputs, with a gate 6.3e-7 to 6.9e-7 (an fp32 product by the library 4.9e-7 at 768, 1.6e-6 at
    // 8192). Not from 256 on without a gate, for the running sums take time, and a third of tensor memory,
    // so that a tile has at most 160 tokens: 4096x768x2048 23.7 us against 18.4, 4096x512x2048 20.3 against
    // 16.9, the down products of 128 experts of 768 (2040 tokens) 122 against 95.
    const bool blocks =
        a.out32 ? a.ksteps > (gated ? 4 : a.act != DPA_ACT_NONE ? 8 : 12) : long_sums(a, gated);
    if (a.E > 0) {
        a.TN = pair && !blocks ? 256 : 128;
        a.xbox = 16;
        // most token tiles there can be: every full tile, and one more per non-empty group
        const int64_t tiles =
            (static_cast<int64_t>(a.rows) / a.TN + (a.rows < a.E ? a.rows : a.E)) * a.FT;
        if (tiles > INT32_MAX) return cudaErrorInvalidValue;
        a.ntiles = static_cast<int>(tiles);
        if (!pair) a.splits = split_k(tiles, a.ksteps);
        clusters = a.splits > 1 ? tiles : (sms / CG < tiles ? sms / CG : tiles);
    } else {
        a.TN = pair ? pair_rows(a.rows, blocks ? kBlockedTokens : 256, a.FT, sms / 2) : balanced_rows(a.rows, 128, 16);
        a.xbox = a.TN / CG;
        const int64_t tiles = static_cast<int64_t>((a.rows - 1) / a.TN + 1) * a.FT;
        if (tiles > INT32_MAX) return cudaErrorInvalidValue;
        a.ntiles = static_cast<int>(tiles);
        if (!pair) a.splits = split_k(tiles, a.ksteps);
        clusters = a.splits > 1 ? tiles : (sms / CG < tiles ? sms / CG : tiles);
    }
    a.step_t = static_cast<int>(clusters) / a.FT;
    a.step_f = static_cast<int>(clusters) % a.FT;
    a.out_wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;   // buffers are 16-byte aligned at least
    a.out_bytes = kOutBytes;
    if (a.splits > 1 && (a.TN + a.splits) * kRowsA * 4 > kOutBytes) a.out_bytes = (a.TN + a.splits) * kRowsA * 4;
    const int stage = kATile + a.TN / CG * 128, fixed = 1024 + a.out_bytes + kBarBytes + 3 * (a.E + 1) * 4;
    a.stages = (kSmemMax - fixed) / stage;
    if (a.stages > kMaxStages) a.stages = kMaxStages;
    const size_t smem = static_cast<size_t>(a.stages) * stage + fixed;
    alignas(64) CUtensorMap maps[2];
    alignas(64) RowMaps xmaps;
    const uint64_t E = static_cast<uint64_t>(groups);
    const uint32_t wbox = static_cast<uint32_t>(feat);
    if (!encode_map(&maps[0], w, f16, a.K, a.N, E, wbox, 3) ||
        !encode_map(&maps[1], gated ? w_mul : w, f16, a.K, a.N, E, wbox, 3))
        return cudaErrorInvalidValue;
    for (int i = 0; i < kRowMaps; ++i)
        if (!encode_map(&xmaps.m[i], x, f16, a.K, a.rows, 1, static_cast<uint32_t>(a.E > 0 ? a.xbox << i : a.xbox), 2))
            return cudaErrorInvalidValue;
    const LinearLaunch l{pair, gated, f16, blocks, maps, &xmaps, static_cast<int>(clusters), smem};
    return a.N % 8 == 0 ? launch_linear_variant<true>(a, l, stream) : launch_linear_variant<false>(a, l, stream);
}

}  // namespace dpa
