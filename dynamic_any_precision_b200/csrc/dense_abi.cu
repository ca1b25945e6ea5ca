// C ABI of the expert row sort and of the dense matrix products (include/dpa.h): validation and
// launches.
#include <atomic>
#include <initializer_list>
#include <cstdint>

#include <cuda_runtime.h>

#include "common.cuh"
#include "dpa.h"
#include "kernels.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool given16(const void* p) { return p && aligned16(p); }   // required, aligned
bool opt16(const void* p) { return !p || aligned16(p); }    // optional, aligned

constexpr int64_t kMaxPairs = 1 << 30;
constexpr int kMaxRowLength = 1 << 24;   // row calls: 32-bit positions inside a row
constexpr int kMaxSide = 1 << 30;        // products: rows and output features, in 32 bits with a tile's overhang
constexpr int kMaxInputs = 1 << 22;      // products: a tile's K loop stays far below the kernels' time limit

bool row_type(int t) { return t == DPA_DTYPE_BF16 || t == DPA_DTYPE_FP16 || t == DPA_DTYPE_FP32; }

// tokens, slots and row length of the row calls
dpa_status check_rows(int T, int K, int H) {
    if (T <= 0 || K <= 0 || H <= 0) return DPA_ERR_INVALID_ARG;
    if (K > 32 || H > kMaxRowLength || static_cast<int64_t>(T) * K > kMaxPairs) return DPA_ERR_UNSUPPORTED;
    return DPA_OK;
}

// the gate weights: none, or fp32 / fp64
bool check_weights(const void* w, int wtype) {
    return !w || (aligned16(w) && (wtype == DPA_DTYPE_FP32 || wtype == DPA_DTYPE_FP64));
}

// SMs of the current device, asked once per device
int sms_current() {
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices];
    int dev = 0, n = 148;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return n;
    if (dev < kDevices && known[dev].load(std::memory_order_relaxed) > 0) return known[dev].load(std::memory_order_relaxed);
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && dev < kDevices)
        known[dev].store(n, std::memory_order_relaxed);
    return n;
}

// Bytes that a call reads or writes (none if the pointer is null).
struct Span {
    const void* at;
    uint64_t bytes;
};
bool overlap(const Span& a, const Span& b) {
    if (!a.at || !b.at) return false;
    const uint64_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
    return x <= y ? y - x < a.bytes : x - y < b.bytes;
}
bool overlaps_any(const Span& out, std::initializer_list<Span> others) {
    for (const Span& s : others)
        if (overlap(out, s)) return true;
    return false;
}
// `in` may be `out` itself, element for element, but lie across it in no other way
bool lies_across(const Span& out, const Span& in) {
    return overlap(out, in) && !(out.at == in.at && out.bytes == in.bytes);
}
uint64_t width(int dtype) { return dtype == DPA_DTYPE_FP64 ? 8 : dtype == DPA_DTYPE_FP32 ? 4 : 2; }

dpa_status launched(cudaError_t e) { return e == cudaSuccess ? DPA_OK : DPA_ERR_CUDA; }

dpa_status run_linear(const dpa_linear_desc* d, int groups, const void* x, const int32_t* offsets, const void* w,
                      const void* bias, const void* w_mul, const void* bias_mul, const void* residual, void* out,
                      void* ws, size_t ws_bytes, void* stream) {
    if (!d || d->rows <= 0 || d->in_features <= 0 || d->out_features <= 0) return DPA_ERR_INVALID_ARG;
    if (d->dtype != DPA_DTYPE_BF16 && d->dtype != DPA_DTYPE_FP16) return DPA_ERR_INVALID_ARG;
    if (d->out_dtype != d->dtype && d->out_dtype != DPA_DTYPE_FP32) return DPA_ERR_INVALID_ARG;
    if (residual && d->residual_dtype != d->out_dtype && d->residual_dtype != DPA_DTYPE_FP32) return DPA_ERR_INVALID_ARG;
    if (d->act < DPA_ACT_NONE || d->act > DPA_ACT_SILU) return DPA_ERR_INVALID_ARG;
    if (!given16(x) || !given16(w) || !given16(out) || !given16(ws)) return DPA_ERR_INVALID_ARG;
    if (!opt16(bias) || !opt16(w_mul) || !opt16(bias_mul) || !opt16(residual)) return DPA_ERR_INVALID_ARG;
    if (bias_mul && !w_mul) return DPA_ERR_INVALID_ARG;
    // rows of whole 16-byte pieces (tensor loads)
    if (d->in_features % 8 || d->in_features > kMaxInputs) return DPA_ERR_UNSUPPORTED;
    if (d->rows > kMaxSide || d->out_features > kMaxSide) return DPA_ERR_UNSUPPORTED;
    if (ws_bytes < DPA_LINEAR_WORKSPACE_BYTES) return DPA_ERR_WORKSPACE;
    const uint64_t M = d->rows, K = d->in_features, N = d->out_features, E = groups > 0 ? groups : 1;
    const Span y{out, M * N * width(d->out_dtype)};
    if (overlaps_any(y, {{x, M * K * 2}, {w, E * N * K * 2}, {w_mul, E * N * K * 2}, {bias, E * N * 2}, {bias_mul, E * N * 2},
                         {offsets, (E + 1) * 4}, {ws, DPA_LINEAR_WORKSPACE_BYTES}}) ||
        lies_across(y, {residual, M * N * width(d->residual_dtype)}))
        return DPA_ERR_INVALID_ARG;
    dpa::LinearArgs a{};
    a.rows = d->rows;
    a.K = d->in_features;
    a.N = d->out_features;
    a.E = groups;
    a.offsets = offsets;
    a.bias = bias;
    a.bias_mul = bias_mul;
    a.residual = residual;
    a.out = out;
    a.act = d->act;
    a.out32 = d->out_dtype == DPA_DTYPE_FP32;
    a.res32 = d->residual_dtype == DPA_DTYPE_FP32;
    a.hdr = static_cast<dpa::WsHeader*>(ws);
    return launched(dpa::launch_linear(a, d->dtype == DPA_DTYPE_FP16, x, w, w_mul, static_cast<cudaStream_t>(stream),
                                       sms_current()));
}

}  // namespace

static_assert(sizeof(dpa::WsHeader) == DPA_LINEAR_WORKSPACE_BYTES, "the products use the workspace header only");

extern "C" {

size_t dpa_sort_workspace_size(int n_pairs, int n_experts) {
    if (n_pairs <= 0 || n_pairs > kMaxPairs || n_experts <= 0 || n_experts > dpa::kSortMaxExperts) return 0;
    return sizeof(dpa::WsHeader) + ((dpa::sort_hist_bytes(n_pairs, n_experts) + 255) & ~static_cast<size_t>(255));
}

dpa_status dpa_sort_pairs(const int32_t* idx, int n_pairs, int n_experts, int32_t* pos, int32_t* order,
                          int32_t* offsets, void* ws, size_t ws_bytes, void* stream) {
    if (n_pairs <= 0 || n_experts <= 0) return DPA_ERR_INVALID_ARG;
    if (!given16(idx) || !given16(pos) || !given16(order) || !given16(offsets) || !given16(ws))
        return DPA_ERR_INVALID_ARG;
    if (n_pairs > kMaxPairs || n_experts > dpa::kSortMaxExperts) return DPA_ERR_UNSUPPORTED;
    const size_t need = dpa_sort_workspace_size(n_pairs, n_experts);
    if (ws_bytes < need) return DPA_ERR_WORKSPACE;
    const uint64_t per = static_cast<uint64_t>(n_pairs) * 4;
    const Span in{idx, per}, place{pos, per}, pair{order, per}, work{ws, need};
    const Span edge{offsets, (static_cast<uint64_t>(n_experts) + 1) * 4};
    if (overlaps_any(place, {in, pair, edge, work}) || overlaps_any(pair, {in, edge, work}) ||
        overlaps_any(edge, {in, work}) || overlap(in, work))
        return DPA_ERR_INVALID_ARG;
    dpa::SortArgs a{};
    a.idx = idx;
    a.P = n_pairs;
    a.E = n_experts;
    a.pos = pos;
    a.order = order;
    a.offsets = offsets;
    a.hist = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + sizeof(dpa::WsHeader));
    return launched(dpa::launch_sort_pairs(a, static_cast<cudaStream_t>(stream)));
}

dpa_status dpa_permute_rows(int dtype, const void* x, const int32_t* pos, int n_tokens, int top_k, int hidden,
                            void* out, void* stream) {
    const dpa_status st = check_rows(n_tokens, top_k, hidden);
    if (st != DPA_OK) return st;
    if (!row_type(dtype) || !given16(x) || !given16(pos) || !given16(out)) return DPA_ERR_INVALID_ARG;
    const uint64_t T = n_tokens, P = T * top_k, row = hidden * width(dtype);
    if (overlaps_any({out, P * row}, {{x, T * row}, {pos, P * 4}})) return DPA_ERR_INVALID_ARG;
    return launched(dpa::launch_permute_pairs(dtype == DPA_DTYPE_FP32 ? 4 : 2, x, pos, n_tokens, top_k, hidden, out,
                                              static_cast<cudaStream_t>(stream), sms_current()));
}

dpa_status dpa_unpermute_rows(int dtype, const void* z, const int32_t* pos, const void* weights, int weight_dtype,
                              const void* residual, int residual_dtype, int out_dtype, int n_tokens, int top_k,
                              int hidden, void* y, void* stream) {
    const dpa_status st = check_rows(n_tokens, top_k, hidden);
    if (st != DPA_OK) return st;
    if (!row_type(dtype) || !row_type(out_dtype)) return DPA_ERR_INVALID_ARG;
    if (dtype != out_dtype && dtype != DPA_DTYPE_FP32 && out_dtype != DPA_DTYPE_FP32) return DPA_ERR_INVALID_ARG;
    if (residual && residual_dtype != out_dtype && residual_dtype != DPA_DTYPE_FP32) return DPA_ERR_INVALID_ARG;
    if (!given16(z) || !given16(pos) || !given16(y) || !opt16(residual) || !check_weights(weights, weight_dtype))
        return DPA_ERR_INVALID_ARG;
    const uint64_t T = n_tokens, P = T * top_k, H = hidden;
    const Span out{y, T * H * width(out_dtype)};
    if (overlaps_any(out, {{z, P * H * width(dtype)}, {pos, P * 4}, {weights, P * width(weight_dtype)}}) ||
        lies_across(out, {residual, T * H * width(residual_dtype)}))
        return DPA_ERR_INVALID_ARG;
    dpa::UnpermuteArgs a{};
    a.z = z;
    a.pos = pos;
    a.weights = weights;
    a.wtype = weights ? weight_dtype : -1;
    a.residual = residual;
    a.y = y;
    a.T = n_tokens;
    a.K = top_k;
    a.H = hidden;
    return launched(dpa::launch_unpermute(a, dtype, out_dtype, residual_dtype == DPA_DTYPE_FP32,
                                          static_cast<cudaStream_t>(stream), sms_current()));
}

dpa_status dpa_unpermute_rows_backward(int dtype, const void* dy, const void* z, const int32_t* pos,
                                       const void* weights, int weight_dtype, int n_tokens, int top_k, int hidden,
                                       void* dz, float* dweights, void* stream) {
    const dpa_status st = check_rows(n_tokens, top_k, hidden);
    if (st != DPA_OK) return st;
    if (!row_type(dtype) || !given16(dy) || !given16(z) || !given16(pos) || !given16(dz) || !given16(dweights))
        return DPA_ERR_INVALID_ARG;
    if (!weights || !check_weights(weights, weight_dtype)) return DPA_ERR_INVALID_ARG;
    const uint64_t T = n_tokens, P = T * top_k, row = hidden * width(dtype);
    const Span rows{dz, P * row}, gates{dweights, P * 4};
    const Span ins[] = {{dy, T * row}, {z, P * row}, {pos, P * 4}, {weights, P * width(weight_dtype)}};
    if (overlap(rows, gates) || overlaps_any(rows, {ins[0], ins[2], ins[3]}) || lies_across(rows, ins[1]) ||
        overlaps_any(gates, {ins[0], ins[1], ins[2], ins[3]}))
        return DPA_ERR_INVALID_ARG;
    dpa::UnpermuteBwdArgs a{};
    a.dy = dy;
    a.z = z;
    a.pos = pos;
    a.weights = weights;
    a.wtype = weight_dtype;
    a.dz = dz;
    a.dweights = dweights;
    a.T = n_tokens;
    a.K = top_k;
    a.H = hidden;
    return launched(dpa::launch_unpermute_bwd(a, dtype, static_cast<cudaStream_t>(stream), sms_current()));
}

dpa_status dpa_linear(const dpa_linear_desc* desc, const void* x, const void* w, const void* bias, const void* w_mul,
                      const void* bias_mul, const void* residual, void* out, void* ws, size_t ws_bytes,
                      void* stream) {
    return run_linear(desc, 0, x, nullptr, w, bias, w_mul, bias_mul, residual, out, ws, ws_bytes, stream);
}

dpa_status dpa_grouped_linear(const dpa_linear_desc* desc, int n_groups, const void* x, const int32_t* offsets,
                              const void* w, const void* bias, const void* w_mul, const void* bias_mul,
                              const void* residual, void* out, void* ws, size_t ws_bytes, void* stream) {
    if (n_groups <= 0 || !given16(offsets)) return DPA_ERR_INVALID_ARG;
    if (n_groups > dpa::kSortMaxExperts) return DPA_ERR_UNSUPPORTED;
    return run_linear(desc, n_groups, x, offsets, w, bias, w_mul, bias_mul, residual, out, ws, ws_bytes, stream);
}

}  // extern "C"
