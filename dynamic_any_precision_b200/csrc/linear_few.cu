// The matrix products of dpa_linear and dpa_grouped_linear for few rows (one token up to a small decode
// batch): bound by reading the weights once, and at these sizes (8 MB: 1.3 us of memory time) by
// latency.
//
// A CTA computes 16 output features for all rows (grouped: for the rows of one non-empty group), its
// 4, 8 or 16 warps taking turns at blocks of 32 inputs. Each lane reads 16-byte pieces of two weight
// rows straight into registers, all of a warp's loads of a round in flight at once, with no shared
// memory, barrier or TMEM set-up in front of them. The
// products go through m16n8k16 MMAs with the weight rows as M and the tokens as N; the tensor rate
// does not matter here. The MMA's order of the 16 inputs is free as long as both operands use the
// same one, so a lane's 16-byte piece (8 inputs) feeds two MMAs as it is. The warps' partial sums
// are added in warp order in shared memory (the same in every run), then the epilogue runs.
#include "common.cuh"
#include "epilogue.cuh"
#include "kernels.h"

namespace dpa {
namespace {

constexpr int kFeat = 16, kBlockK = 32;

template <bool F16>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
    if constexpr (F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 load_weights(const uint16_t* p) {   // read once: kept out of L1
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// The i-th non-empty group and its rows; false if there are fewer. Every warp looks for itself, 32
// groups at a time.
__device__ __forceinline__ bool nonempty_group(const LinearArgs& a, int i, int lane, int& e, int& row0, int& n) {
    int seen = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
        int begin = 0, end = 0;
        if (e0 + lane < a.E) {
            begin = min(max(__ldg(a.offsets + e0 + lane), 0), a.rows);
            end = min(max(__ldg(a.offsets + e0 + lane + 1), 0), a.rows);
        }
        unsigned m = __ballot_sync(0xffffffffu, end > begin);
        const int c = __popc(m);
        if (i < seen + c) {
            for (int j = seen; j < i; ++j) m &= m - 1;
            const int src = __ffs(m) - 1;
            e = e0 + src;
            row0 = __shfl_sync(0xffffffffu, begin, src);
            n = __shfl_sync(0xffffffffu, end, src) - row0;
            return true;
        }
        seen += c;
    }
    return false;
}

// NT tiles of 8 tokens at a time; MATS weight matrices (2: gated). Grid: feature blocks, groups (at
// most as many as there are rows).
template <bool F16, int MATS, int NT, bool GROUPED, int kWarps, bool PRECISE>
__global__ void __launch_bounds__(kWarps * 32, kWarps == 16 ? 1 : (NT == 1 ? 3 : 2) * 8 / kWarps)
few_rows_kernel(LinearArgs a, const uint16_t* x, const uint16_t* w, const uint16_t* u) {
    __shared__ float s_part[kWarps][MATS][8 * NT][kFeat + 1];
    constexpr int kRound = MATS * NT >= 4 ? 2 : 4;   // blocks whose loads are in flight together
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int f0 = blockIdx.x * kFeat;
    const int nblk = (a.K + kBlockK - 1) / kBlockK;
    pdl_wait();
    int e = 0, row0 = 0, n = a.rows;
    if (GROUPED && !nonempty_group(a, blockIdx.y, lane, e, row0, n)) return;
    // rows behind the last feature read the last one, and are not stored
    const int64_t we = static_cast<int64_t>(e) * a.N;
    const int64_t r0 = (we + min(f0 + g, a.N - 1)) * a.K + 8 * c, r1 = (we + min(f0 + g + 8, a.N - 1)) * a.K + 8 * c;
    const uint16_t* mat[2] = {w, u};
    for (int t0 = 0; t0 < (GROUPED ? n : 1); t0 += 8 * NT) {   // plain: one turn
        const uint16_t* xt = x + static_cast<int64_t>(row0 + t0) * a.K + 8 * c;
        const int left = n - t0;
        float acc[MATS][NT][4];
#pragma unroll
        for (int m = 0; m < MATS; ++m)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][t][i] = 0.f;
        for (int b = warp; b < nblk; b += kWarps * kRound) {
            uint4 av[kRound][MATS][2], bv[kRound][NT];
#pragma unroll
            for (int i = 0; i < kRound; ++i) {
                const int k = (b + i * kWarps) * kBlockK;
                const bool in = k + 8 * c < a.K;   // K % 8 == 0: a piece is wholly inside or outside
#pragma unroll
                for (int m = 0; m < MATS; ++m) {
                    av[i][m][0] = in ? load_weights(mat[m] + r0 + k) : make_uint4(0, 0, 0, 0);
                    av[i][m][1] = in ? load_weights(mat[m] + r1 + k) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const int tok = 8 * t + g;
                    bv[i][t] = in && tok < left
                                   ? __ldg(reinterpret_cast<const uint4*>(xt + static_cast<int64_t>(tok) * a.K + k))
                                   : make_uint4(0, 0, 0, 0);
                }
            }
            auto multiply = [&](float (&sum)[MATS][NT][4]) {   // in the order of the loads
#pragma unroll
                for (int i = 0; i < kRound; ++i)
#pragma unroll
                    for (int m = 0; m < MATS; ++m)
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            const uint4 p = av[i][m][0], q = av[i][m][1], s = bv[i][t];
                            mma16<F16>(sum[m][t], p.x, q.x, p.y, q.y, s.x, s.y);
                            mma16<F16>(sum[m][t], p.z, q.z, p.w, q.w, s.z, s.w);
                        }
            };
            if constexpr (PRECISE) {
                // fp32 outputs, very long sums: a round's products are summed by themselves and added with rounding;
                // the MMA drops the bits below its accumulator's last place at every step, which
                // would grow with K
                float part[MATS][NT][4] = {};
                multiply(part);
#pragma unroll
                for (int m = 0; m < MATS; ++m)
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[m][t][i] += part[m][t][i];
            } else {
                multiply(acc);
            }
        }
        if (GROUPED && t0 > 0) __syncthreads();   // the last tile's sums have been read
#pragma unroll
        for (int m = 0; m < MATS; ++m)
#pragma unroll
            for (int t = 0; t < NT; ++t) {   // accumulator i: feature g + 8 (i / 2), token 2c + i % 2
                s_part[warp][m][8 * t + 2 * c][g] = acc[m][t][0];
                s_part[warp][m][8 * t + 2 * c + 1][g] = acc[m][t][1];
                s_part[warp][m][8 * t + 2 * c][g + 8] = acc[m][t][2];
                s_part[warp][m][8 * t + 2 * c + 1][g + 8] = acc[m][t][3];
            }
        __syncthreads();
        for (int i = threadIdx.x; i < min(left, 8 * NT) * kFeat; i += kWarps * 32) {
            const int tok = i / kFeat, fi = i % kFeat, f = f0 + fi;
            if (f >= a.N) continue;
            float v[MATS];
#pragma unroll
            for (int m = 0; m < MATS; ++m) {
                v[m] = 0.f;
#pragma unroll
                for (int q = 0; q < kWarps; ++q) v[m] += s_part[q][m][tok][fi];
            }
            float o = act_one(v[0] + bias_at<F16>(a.bias, we + f), a.act);
            if (MATS == 2) o *= v[MATS - 1] + bias_at<F16>(a.bias_mul, we + f);
            store_one<F16>(a, o, (static_cast<int64_t>(row0) + t0 + tok) * a.N + f);
        }
    }
}

template <bool F16, int MATS, int NT, bool GROUPED, int WARPS>
const void* pick_kernel(bool precise) {
    return precise ? reinterpret_cast<const void*>(few_rows_kernel<F16, MATS, NT, GROUPED, WARPS, true>)
                   : reinterpret_cast<const void*>(few_rows_kernel<F16, MATS, NT, GROUPED, WARPS, false>);
}

template <bool F16, int MATS, int WARPS>
const void* pick_tokens(bool grouped, int tokens, bool precise) {
    if constexpr (WARPS < 16) {
        // groups of so few rows have one or two each; more take turns
        if (grouped) return pick_kernel<F16, MATS, 1, true, WARPS>(precise);
        if (tokens > 16) return pick_kernel<F16, MATS, 4, false, WARPS>(precise);
    }
    return tokens <= 8 ? pick_kernel<F16, MATS, 1, false, WARPS>(precise)
                       : pick_kernel<F16, MATS, 2, false, WARPS>(precise);
}

template <bool F16, int MATS>
const void* pick(bool grouped, int tokens, int warps, bool precise) {
    return warps == 16  ? pick_tokens<F16, MATS, 16>(grouped, tokens, precise)
           : warps == 8 ? pick_tokens<F16, MATS, 8>(grouped, tokens, precise)
                        : pick_tokens<F16, MATS, 4>(grouped, tokens, precise);
}

}  // namespace

cudaError_t launch_linear_few(const LinearArgs& a, bool f16, const void* x, const void* w, const void* w_mul,
                              cudaStream_t stream, int sms) {
    const bool grouped = a.E > 0;
    const int blocks = (a.N - 1) / kFeat + 1, groups = !grouped ? 1 : a.rows < a.E ? a.rows : a.E;
    // More warps on a CTA's features while all CTAs run at once, so that more loads are in flight and
    // each CTA finishes sooner; fewer where CTAs wait for one another or K is short. (One token:
    // 2048x2048 2.6 us with sixteen, 2.9 with eight, 3.4 with four; 768x8192 3.4 with four, 3.8 with
    // eight.)
    const int64_t ctas = static_cast<int64_t>(blocks) * groups;
    int warps = ctas <= 3 * sms && a.K > 512 ? 8 : 4;
    if (!grouped && ctas <= sms && a.K > 1024 && a.rows <= 16) warps = 16;
    const bool precise = a.out32 || long_sums(a, w_mul != nullptr);
    const void* fn = w_mul ? (f16 ? pick<true, 2>(grouped, a.rows, warps, precise) : pick<false, 2>(grouped, a.rows, warps, precise))
                           : (f16 ? pick<true, 1>(grouped, a.rows, warps, precise) : pick<false, 1>(grouped, a.rows, warps, precise));
    LinearArgs b = a;
    void* args[] = {&b, &x, &w, &w_mul};
    return launch_pdl_raw(fn, dim3(blocks, groups), dim3(warps * 32), 0, stream, args);
}

}  // namespace dpa
