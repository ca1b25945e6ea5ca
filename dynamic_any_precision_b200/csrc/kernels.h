// Launch interfaces of the device kernels (internal to the library).
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "common.cuh"

namespace dpa {

struct RouteArgs {
    const uint16_t* x;        // [T][H] bf16
    const uint16_t* wr;       // [E][H] bf16
    int T, E, H, K, G, norm_topk;
    double* logits_user;      // [T][E] or nullptr
    double* logits_ws;        // [T][E] workspace copy
    int32_t* idx;             // [T][K]
    double* gate;             // [T][K]
    unsigned* counters;       // [T] zero between calls
    int8_t* xdig;             // [T][2][H] activation digits for the expert GEMV, or nullptr
    float* xscl;              // [T][ngp] group scales 2^(E-14) (ngp = H/G rounded up to 4)
    float* xfsx;              // [T][ngp] group sums of the fixed-point values times the scale
    WsHeader* hdr;
    int wpe;                  // warps per expert (set by the launcher)
    // large-batch path (nullptr: always the per-logit kernel): per-row exactness statistics
    int16_t* lsb_x;           // [T][H/64] lowest set bit over each 64-input block's nonzero elements
    int16_t* hb_x;            // [T][H/64] h with |x_b| < 2^h (Euclidean norm of the block)
    double* n2_x;             // [T] sum of squares
    int16_t* lsb_w;           // [E][H/64]
    int16_t* hb_w;            // [E][H/64]
    double* n2_w;             // [E]
    double* part;             // [ks][T][E] slice sums of the tiled logits
    int ks;                   // input slices (set by the launcher)
};
cudaError_t launch_route(const RouteArgs& a, cudaStream_t stream, int sms = 148);

// Tiling of the large-batch logits: token x expert CTA tiles, input slices to fill the SMs.
struct RouteTiling {
    int TT, TE, gx, gy, ks, kslice;
};
constexpr int kRouteMaxSms = 256;   // the partial-sum buffer is sized for up to this many SMs
RouteTiling route_tiling(int T, int E, int H, int sms);
bool route_tiled_path(int T, int H);
// doubles of the slice-sum buffer the tiled path needs for T tokens (0: the per-logit path)
size_t route_partial_doubles(int T, int E, int H);

// A token group of the expert GEMV: [0] expert, [1] kmax over the group, [2] tiles (<= 2),
// [4 + t] plane count of tile t, [6 + t] pairs in tile t (<= 4), [8 + 4t + q] grouped position
// (output row) of pair q of tile t, [16 + 4t + q] its token; unused slots hold -1.
constexpr int kVRecInts = 32;

struct AllocArgs {
    const double* rtable;     // [E][B]
    const int32_t* idx;       // [T][K]
    const double* gate;       // [T][K]
    const double* target;     // device scalar
    int T, K, E, B, kmin, kmax;
    uint8_t* k_out;           // [T][K]
    double* lambda_out;       // scalar or nullptr
    double* cbuf;             // [P][nk] workspace
    // grouping outputs (do_permute)
    int do_permute;
    int32_t* pair_pos;        // [P] position of each pair in the (expert, k)-grouped order
    int k_given;              // 1: k_out already holds the plane counts (grid-wide bisection ran)
    int4* gtiles;             // nullptr, or [P/kGemmTileTokens + E*nk] GEMM token tiles {e, k, pos0, n}
    int32_t* pos_tok;         // nullptr, or [P] token of each grouped position
    WsHeader* hdr;
    int policy;               // DPA_ALLOC_LAGRANGE, DPA_ALLOC_UNIFORM or DPA_ALLOC_THRESHOLD
    const double* threshold;  // device scalar (DPA_ALLOC_THRESHOLD)
    // work list of the pipelined expert GEMV (nullptr: not written): token groups of up to
    // vtiles_per_group (<= 2) tiles of up to 4 pairs of one (expert, k) class, as records of
    // kVRecInts ints (see kVRec*); count in hdr->n_vgroups
    int32_t* vrec;            // [P/4 + E*nk][kVRecInts]
    int vtiles_per_group;
    // per GEMV launch j (0: gate/up, 1: down), unless vstart[j] is nullptr: the first item of each
    // of its vgrid[j] CTAs over items (record, row block; vnrb[j] row blocks per record), with
    // equal shares of the estimated work; vstart[j][vgrid[j]] = the item count
    int32_t* vstart[2];
    int vgrid[2], vnrb[2];
    const uint8_t* expert_k;  // [E] plane count per expert (DPA_ALLOC_EXPERT_TABLE)
    const uint8_t* expert_width;   // nullptr, or [E] stored planes per expert: no pair reads more
};
// Counters of the grid-wide bisection (zeroed by the launcher before every call).
constexpr int kCoopRoundsMax = 16;
struct CoopSync {
    unsigned barrier;
    unsigned bad;
    unsigned long long mx_bits;
    int counts[kCoopRoundsMax][64][32];   // one 128-byte line per node: CTAs' atomics do not queue on one line
};
// coop: workspace counters for the grid-wide bisection of large batches (nullptr: single CTA).
cudaError_t launch_allocate(const AllocArgs& a, cudaStream_t stream, CoopSync* coop = nullptr, int sms = 0);
size_t allocate_smem_bytes(int P, int E, int nk, bool recs);
int allocate_threads(int P);

// Threshold calibration of the score-threshold policy: 64 bisection steps over n scores.
struct CalibArgs {
    const double* scores;     // [n]
    int n, kmin, kmax;
    const double* target;     // device scalar
    double* threshold_out;    // device scalar
    WsHeader* hdr;
};
cudaError_t launch_calibrate(const CalibArgs& a, cudaStream_t stream);

// Workload profile of a prefill and the per-expert read rates solved from it.
struct ProfileArgs {
    const uint16_t* x;        // [T][H] bf16 prefill activations
    const int32_t* idx;       // [T][K] routed experts
    int T, H, K, E;
    double* m;                // [H] mean square per input channel
    int32_t* counts;          // [E] routed pairs per expert
    WsHeader* hdr;
};
cudaError_t launch_profile(const ProfileArgs& a, cudaStream_t stream);
struct RatesArgs {
    const double* tdist;      // [E][B][H] distortion tensor
    const double* m;          // [H]
    const int32_t* counts;    // [E]
    const double* target;     // device scalar
    int E, B, H, kmin, kmax;
    uint8_t* k_table;         // [E]
    double* lambda_out;       // scalar or nullptr
    WsHeader* hdr;
};
cudaError_t launch_solve_rates(const RatesArgs& a, cudaStream_t stream);
size_t rates_smem_bytes(int E, int nk);

// Prefill expert FFN on tcgen05: grouped GEMMs over the GEMM token tiles of the allocation.
struct GemmArgs {
    const uint8_t* planes;    // encoded layer (uniform format)
    const uint8_t* meta;
    uint64_t planes_per_expert, meta_per_expert;
    uint64_t planes_mat_off[3], meta_mat_off[3];
    int H, I, B, G;
    int T, P;                 // tokens, routed pairs (rows of x and of hbuf)
    const int4* gtiles;       // {e, k, pos0, n}, count in hdr->n_gtiles
    const int32_t* pos_tok;   // [P] token of each grouped position
    const uint16_t* x;        // [T][H] bf16 activations
    uint16_t* xperm;          // [P][H] bf16 activations in grouped pair order (written by the permute)
    int E;
    uint16_t* hbuf;           // [P][I] fp16 SwiGLU outputs, grouped order
    float* out_pair;          // [P][H] per-pair expert outputs, grouped order
    WsHeader* hdr;
};
cudaError_t launch_permute_rows(const GemmArgs& a, cudaStream_t stream);
cudaError_t launch_gemm_gateup(const GemmArgs& a, cudaStream_t stream, int sms);
cudaError_t launch_gemm_down(const GemmArgs& a, cudaStream_t stream, int sms);
size_t gemm_tc_smem_bytes();

// Pipelined variable-plane expert GEMV (decode batches): one launch computes either gate and up
// with the SwiGLU epilogue (nmat = 2: out = h [P][R], R = inter) or down (nmat = 1: out =
// per-pair outputs [P][R], R = hidden) for every (token group, row block) item.
struct VpArgs {
    const uint8_t* planes;    // encoded layer
    const uint8_t* meta;
    uint64_t planes_per_expert, meta_per_expert;
    uint64_t planes_mat_off[3], meta_mat_off[3];
    int fmt, B, G;
    int R, K;                 // rows and columns of each matrix of this launch
    int mat0, nmat;           // first matrix (0: gate, up; 2: down) and the matrix count
    int tiles_per_group;      // 1 or 2 (the allocation's grouping)
    const int32_t* vrec;      // token group records [n_vgroups][kVRecInts], count in hdr->n_vgroups
    const int8_t* dig;        // activation digit rows [rows][2][K] (permuted 64-column blocks)
    const float* dscl;        // [rows][ngp] group scales 2^(E-14)
    const float* dfsx;        // [rows][ngp] group sums of the fixed-point values times the scale
    int dig_by_token;         // 1: the digit row of a pair is its token (x); 0: its position (h)
    float* out;               // [P][R] by grouped position
    WsHeader* hdr;
    int max_groups;           // host bound of the token groups
    const uint64_t* expert_off;   // nullptr (full layout), or [E][2] byte offsets of each expert's
                                  // planes and scale data in the compact layer of stored widths
    const uint8_t* expert_width;  // [E] stored planes per expert (with expert_off)
    const int32_t* vstart;    // nullptr (equal item counts per CTA), or [grid + 1] first item of each
                              // CTA, balanced by estimated work (written by the allocation)
    int vgrid;                // the grid vstart was written for (used only when the launch matches)
};
cudaError_t launch_vp_gemv(const VpArgs& a, cudaStream_t stream, int sms);
// The launch geometry of a variant, as launch_vp_gemv will use it: CTAs and rows per item.
int vp_grid(const VpArgs& a, int sms);
int vp_rows_per_item(const VpArgs& a);
// tiles per token group the layer's shapes allow (2 where the group slots fit, else 1)
int vp_tiles_per_group(int K_gateup, int K_down, int G, int fmt, int B);
// dynamic shared memory of one CTA of a variant
size_t vp_smem_bytes(int K, int G, int fmt, int B, int nmat, int tiles_per_group);
constexpr size_t kVpMaxSmem = 227 * 1024;

// Fixed-point digits of activation rows (x as bf16, or h as fp32), per group of G columns:
// X = rint(v * 2^(14 - E)) with |v| < 2^E, as digits d0 + 256 d1 in rows [rows][2][K] with each
// 64-column block permuted for the B operand; per group the scale 2^(E-14) and the scaled sum
// 2^(E-14) sum_j X_j (both exact in fp32), [rows][ngp], ngp = K/G rounded up to a multiple of 4.
struct DigitArgs {
    const uint16_t* x16;      // bf16 rows or nullptr
    const float* x32;         // fp32 rows (when x16 is nullptr)
    int rows, K, G;
    int8_t* dig;
    float* dscl;
    float* dfsx;
};
cudaError_t launch_digits(const DigitArgs& d, cudaStream_t stream);

struct CombineArgs {
    const float* out_pair;    // [P][H] by sorted position
    const int32_t* pair_pos;  // [P]
    const double* gate;       // [T][K]
    const float* shared_out;  // [T][H] or nullptr
    float* pair_out_user;     // [T][K][H] diagnostic copy or nullptr
    uint16_t* y;              // [T][H] bf16
    int T, K, H;
    WsHeader* hdr;
};
cudaError_t launch_combine(const CombineArgs& a, cudaStream_t stream);

struct SharedArgs {
    const uint16_t* x;        // [T][H] bf16
    const uint16_t* wg;       // [S][I][H]
    const uint16_t* wu;
    const uint16_t* wd;       // [S][H][I]
    float* h;                 // [T][S][I] workspace
    float* out;               // [T][H]
    int T, S, H, I;
};
cudaError_t launch_shared(const SharedArgs& a, cudaStream_t stream);

cudaError_t launch_residual_rmsnorm(const uint16_t* y, float* h, uint16_t* x, int T, int H, float eps,
                                    cudaStream_t stream);

// Routed pairs sorted by expert, and the rows that travel with them (pairs.cu).
constexpr int kSortMaxExperts = 1024;
struct SortArgs {
    const int32_t* idx;       // [P] expert of each pair; outside [0, E): not routed
    int P, E;
    int32_t* pos;             // [P] place of each pair, -1 if not routed
    int32_t* order;           // [P] pair at each place, unrouted pairs last
    int32_t* offsets;         // [E + 1] places before each expert
    int32_t* hist;            // [chunks][E + 1] workspace (several chunks only)
    int chunk;                // pairs per CTA (set by the launcher)
};
int sort_chunk_pairs(int P);
size_t sort_hist_bytes(int P, int E);
cudaError_t launch_sort_pairs(const SortArgs& a, cudaStream_t stream);

cudaError_t launch_permute_pairs(int elem_bytes, const void* x, const int32_t* pos, int T, int K, int H, void* out,
                                 cudaStream_t stream, int sms);

struct UnpermuteArgs {
    const void* z;            // [T*K][H] rows by place
    const int32_t* pos;       // [T][K]
    const void* weights;      // [T][K] fp32 or fp64, or nullptr (all 1)
    int wtype;                // DPA_DTYPE_FP32, DPA_DTYPE_FP64, or -1 without weights
    const void* residual;     // [T][H] in y's type or fp32, or nullptr
    void* y;                  // [T][H]
    int T, K, H;
};
cudaError_t launch_unpermute(const UnpermuteArgs& a, int ztype, int ytype, bool res32, cudaStream_t stream, int sms);

struct UnpermuteBwdArgs {
    const void* dy;           // [T][H]
    const void* z;            // [T*K][H]
    const int32_t* pos;       // [T][K]
    const void* weights;      // [T][K] fp32 or fp64
    int wtype;
    void* dz;                 // [T*K][H], rows without a pair are left as they were
    float* dweights;          // [T][K], 0 for unrouted pairs
    int T, K, H;
};
cudaError_t launch_unpermute_bwd(const UnpermuteBwdArgs& a, int type, cudaStream_t stream, int sms);

// Matrix products with a fused epilogue, plain or grouped by expert (linear_tc.cuh).
struct LinearArgs {
    int rows, K, N;           // rows of x, in and out features
    int E;                    // groups (0: plain)
    const int32_t* offsets;   // [E + 1] first row of each group
    const void* bias;         // [N] or [E][N], or nullptr
    const void* bias_mul;     // the same for the second product, or nullptr
    const void* residual;     // [rows][N] in the output's type or fp32, or nullptr
    void* out;                // [rows][N]
    int act, out32, res32;    // DPA_ACT_*; 1: fp32 output, fp32 residual
    WsHeader* hdr;
    // set by the launcher: K steps, feature tiles, most tokens per tile, CTAs sharing K, pipeline
    // stages, rows of the smallest token load, tiles (grouped: the most there can be), bytes of the
    // epilogue's shared memory, whether out is 32-byte aligned, and how far a cluster's next tile lies
    // (token tiles, then feature tiles)
    int ksteps, FT, TN, splits, stages, xbox, ntiles, out_bytes, out_wide, step_t, step_f;
};
// Sums so long that 16-bit outputs, too, would see what the tensor cores drop when they add without
// rounding (7e-10 of the sum per input, with a gate twice that: at this border a tenth of fp16's half unit
// 2^-11, at 2^20 inputs 1.5 of it, and 3 with a gate). They are added in blocks, as those of fp32 outputs.
inline bool long_sums(const LinearArgs& a, bool gated) {
    return a.K > (gated || a.act != DPA_ACT_NONE ? 1 << 15 : 1 << 16);
}
cudaError_t launch_linear(const LinearArgs& a, bool f16, const void* x, const void* w, const void* w_mul,
                          cudaStream_t stream, int sms);
// The products of few rows (linear_few.cu): at most 32 plain ones, or 64 that lie in few per group.
cudaError_t launch_linear_few(const LinearArgs& a, bool f16, const void* x, const void* w, const void* w_mul,
                              cudaStream_t stream, int sms);

}  // namespace dpa
