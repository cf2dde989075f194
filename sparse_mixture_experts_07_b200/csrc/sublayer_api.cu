// The C ABI of the operators around the block: norms fused with the combine,
// gate and residual, their backward pass, and the gradient norm with clipping.
// Host-side validation and dispatch; no memory is allocated on the device.
#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "grad_norm.cuh"
#include "host_common.cuh"
#include "norm.cuh"

namespace {

using namespace moe::host;

moe_status check_norm(const moe_norm_spec* n) {
    if (n->kind < MOE_NORM_NONE || n->kind > MOE_NORM_LAYER) return MOE_ERR_INVALID_ARG;
    if (n->kind == MOE_NORM_NONE)
        return n->weight || n->bias ? MOE_ERR_INVALID_ARG : MOE_OK;
    return n->eps >= 0.f && std::isfinite(n->eps) ? MOE_OK : MOE_ERR_INVALID_ARG;
}

moe_status check_gate(int32_t kind, const float* gate, int64_t T) {
    if (kind < MOE_GATE_NONE || kind > MOE_GATE_CHANNEL) return MOE_ERR_INVALID_ARG;
    if ((kind == MOE_GATE_NONE) != (gate == nullptr) && T > 0) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

moe::NormDev norm_dev(const moe_norm_spec* n) {
    return n ? moe::NormDev{n->weight, n->bias, n->eps, n->kind}
             : moe::NormDev{nullptr, nullptr, 0.f, MOE_NORM_NONE};
}

moe_status check_norm_shape(const moe_shape* s) {
    const moe_status st = moe::check_shape(s);
    if (st != MOE_OK) return st;
    return s->H <= moe::kMaxNormH ? MOE_OK : MOE_ERR_UNSUPPORTED;
}

// Rows are read in 16-byte pieces when every one of them starts on such a
// boundary (bf16: required); float32 rows may start anywhere.
template <size_t N> bool all_aligned(const void* const (&ptrs)[N]) {
    for (const void* p : ptrs)
        if (!aligned16(p)) return false;
    return true;
}

// Buffers of a call.  A row's values are read before they are written by the
// same thread, so an output may be an input of its size; anything else that
// shares memory with it is refused.
struct Span {
    const void* p;
    size_t bytes;
};
bool apart(const Span& a, const Span& b) {
    const auto x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return !a.p || !b.p || x + a.bytes <= y || y + b.bytes <= x;
}
bool same_or_apart(const Span& a, const Span& b) { return a.p == b.p || apart(a, b); }

Span rows_span(const moe_shape* s, const void* p, int64_t rows) {
    return {p, static_cast<size_t>(rows) * static_cast<size_t>(s->H) * elem_bytes(*s)};
}

struct Interval {
    uintptr_t begin, end;
    bool operator<(const Interval& o) const { return begin < o.begin; }
};

moe_status check_grads(int32_t n, void* const* grads, const int64_t* numel, const int32_t* dtype) {
    if (n < 0 || (n > 0 && (!grads || !numel || !dtype))) return MOE_ERR_INVALID_ARG;
    std::vector<Interval> spans;
    try {
        spans.reserve(static_cast<size_t>(n));
    } catch (const std::bad_alloc&) {
        return MOE_ERR_UNSUPPORTED;
    }
    for (int32_t i = 0; i < n; ++i) {
        if (numel[i] < 0 || (dtype[i] != MOE_F32 && dtype[i] != MOE_BF16))
            return MOE_ERR_INVALID_ARG;
        if (numel[i] == 0) continue;
        if (!grads[i]) return MOE_ERR_INVALID_ARG;
        const uintptr_t eb = dtype[i] == MOE_BF16 ? 2 : 4;
        const uintptr_t at = reinterpret_cast<uintptr_t>(grads[i]);
        if (at % eb) return MOE_ERR_UNSUPPORTED;
        spans.push_back({at, at + static_cast<uintptr_t>(numel[i]) * eb});
    }
    std::sort(spans.begin(), spans.end());
    for (size_t i = 1; i < spans.size(); ++i)
        if (spans[i].begin < spans[i - 1].end) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

// Values per chunk: 64 KB of float32 amortise the search of the tensor when
// there is work for every resident CTA several times over; otherwise 16 KB, so
// that small lists spread over more SMs.
int32_t chunk_values(int32_t n, const int64_t* numel) {
    int64_t total = 0;
    for (int32_t i = 0; i < n; ++i) total += numel[i];
    return total >= (int64_t(1) << 26) ? 16384 : 4096;
}

moe::GradList grad_list(int32_t from, int32_t n, void* const* grads, const int64_t* numel,
                        const int32_t* dtype, int32_t chunk) {
    moe::GradList l{};
    l.chunk = chunk;
    for (int32_t i = from; i < n && l.n < moe::kGradsPerLaunch; ++i) {
        l.ptr[l.n] = grads[i];
        l.numel[l.n] = numel[i];
        l.dtype[l.n] = dtype[i];
        l.chunk_start[l.n + 1] = l.chunk_start[l.n] + (numel[i] + chunk - 1) / chunk;
        ++l.n;
    }
    return l;
}

// Partial sums, one per CTA: enough CTAs to keep every SM's loads in flight, no
// more than all tensors together have chunks.  (Every launch of 64 tensors has
// this many, so that each adds to the same partial sums; a CTA without a chunk
// leaves its own as it was.)
int grad_parts(int32_t n, const int64_t* numel, int32_t chunk) {
    int64_t chunks = 0;
    for (int32_t i = 0; i < n; ++i) chunks += (numel[i] + chunk - 1) / chunk;
    int64_t parts = static_cast<int64_t>(num_sms()) * 8;
    if (parts > moe::kGradParts) parts = moe::kGradParts;
    if (parts > chunks) parts = chunks;
    return static_cast<int>(parts > 0 ? parts : 1);
}

moe_status square_sum_parts(int32_t n, void* const* grads, const int64_t* numel,
                            const int32_t* dtype, int32_t chunk, double* part, int parts,
                            cudaStream_t cs) {
    for (int32_t from = 0; from == 0 || from < n; from += moe::kGradsPerLaunch) {
        const moe::GradList l = grad_list(from, n, grads, numel, dtype, chunk);
        if (moe::launch_grad_square_sum(l, from > 0, part, parts, cs) != cudaSuccess)
            return MOE_ERR_CUDA;
    }
    return MOE_OK;
}

moe_status scale_all(int32_t n, void* const* grads, const int64_t* numel, const int32_t* dtype,
                     int32_t chunk, const double* part, int parts, float max_norm, float* norm,
                     cudaStream_t cs) {
    // the last tensors first: the sum's pass ended with them
    int32_t from = n > 0 ? (n - 1) / moe::kGradsPerLaunch * moe::kGradsPerLaunch : 0;
    for (; from >= 0; from -= moe::kGradsPerLaunch) {
        const int32_t end = std::min(n, from + moe::kGradsPerLaunch);
        const moe::GradList l = grad_list(from, end, grads, numel, dtype, chunk);
        if (moe::launch_grad_scale(l, part, parts, max_norm, norm, num_sms(), cs) != cudaSuccess)
            return MOE_ERR_CUDA;
    }
    return MOE_OK;
}

bool good_max_norm(float m) { return m >= 0.f; }   // infinity: measures only

}  // namespace

extern "C" {

moe_status moe_norm_forward(const moe_shape* shape, const moe_norm_spec* norm, const void* x,
                            void* y, void* stream) {
    moe_status st = check_norm_shape(shape);
    if (st != MOE_OK) return st;
    if (!norm) return MOE_ERR_INVALID_ARG;
    st = check_norm(norm);
    if (st != MOE_OK) return st;
    if (shape->T == 0) return MOE_OK;
    if (!x || !y) return MOE_ERR_INVALID_ARG;
    // the combine of one "shared" row per token, without residual or post norm
    moe::CombineNormParams p{};
    p.y_slots = x;
    p.xn_out = y;
    p.next = norm_dev(norm);
    p.T = shape->T;
    p.H = shape->H;
    p.S = 1;
    p.scale = 1.f;
    const void* ptrs[] = {x, y, norm->weight, norm->bias};
    const bool vec = all_aligned(ptrs) && p.H % 4 == 0;
    const bool bf16 = shape->dtype == MOE_BF16;
    if (bf16 && !vec) return MOE_ERR_UNSUPPORTED;
    if (!same_or_apart(rows_span(shape, y, p.T), rows_span(shape, x, p.T)))
        return MOE_ERR_INVALID_ARG;
    return cuda_status(moe::launch_combine_norm(p, bf16, vec, num_sms(),
                                                static_cast<cudaStream_t>(stream)));
}

moe_status moe_combine_norm(const moe_shape* shape, const void* y_slots, const int32_t* inv,
                            const void* residual, const moe_norm_spec* post, int32_t gate_kind,
                            const float* gate, float scale, const moe_norm_spec* next,
                            void* y_out, void* h_out, void* xn_out, void* stream) {
    moe_status st = check_norm_shape(shape);
    if (st != MOE_OK) return st;
    if (post && (st = check_norm(post)) != MOE_OK) return st;
    if (next && (st = check_norm(next)) != MOE_OK) return st;
    if ((st = check_gate(gate_kind, gate, shape->T)) != MOE_OK) return st;
    if (shape->T == 0) return MOE_OK;
    if (!y_slots || !inv || !h_out || (next == nullptr) != (xn_out == nullptr))
        return MOE_ERR_INVALID_ARG;
    moe::CombineNormParams p{};
    p.y_slots = y_slots;
    p.inv = inv;
    p.residual = residual;
    p.gate = gate;
    p.y_out = y_out;
    p.h_out = h_out;
    p.xn_out = xn_out;
    p.post = norm_dev(post);
    p.next = norm_dev(next);
    p.T = shape->T;
    p.H = shape->H;
    p.k = shape->k;
    p.S = shape->n_shared;
    p.gate_kind = gate_kind;
    p.scale = scale;
    const void* ptrs[] = {y_slots, residual, y_out, h_out, xn_out, p.post.weight, p.post.bias,
                          p.next.weight, p.next.bias,
                          gate_kind == MOE_GATE_CHANNEL ? gate : nullptr};
    const bool vec = all_aligned(ptrs) && p.H % 4 == 0;
    const bool bf16 = shape->dtype == MOE_BF16;
    if (bf16 && !vec) return MOE_ERR_UNSUPPORTED;
    const Span slots = rows_span(shape, y_slots, p.T * (p.k + p.S));
    const Span res = rows_span(shape, residual, p.T);
    const Span outs[] = {rows_span(shape, h_out, p.T), rows_span(shape, xn_out, p.T),
                         rows_span(shape, y_out, p.T)};
    for (int i = 0; i < 3; ++i) {
        if (!apart(outs[i], slots) || !same_or_apart(outs[i], res)) return MOE_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (!apart(outs[i], outs[j])) return MOE_ERR_INVALID_ARG;
    }
    return cuda_status(moe::launch_combine_norm(p, bf16, vec, num_sms(),
                                                static_cast<cudaStream_t>(stream)));
}

moe_status moe_norm_backward_workspace_size(const moe_shape* shape, size_t* bytes) {
    const moe_status st = check_norm_shape(shape);
    if (st != MOE_OK) return st;
    if (!bytes) return MOE_ERR_INVALID_ARG;
    *bytes = align_up(static_cast<size_t>(moe::norm_backward_parts(shape->T, shape->H, num_sms())) *
                      2 * static_cast<size_t>(shape->H) * 4);
    return MOE_OK;
}

moe_status moe_norm_backward(const moe_shape* shape, const moe_norm_spec* norm, const void* x,
                             const void* dout, int32_t gate_kind, const float* gate, float scale,
                             const void* dadd, void* dx, float* dweight, float* dbias,
                             float* dgate, void* workspace, size_t workspace_bytes,
                             void* stream) {
    moe_status st = check_norm_shape(shape);
    if (st != MOE_OK) return st;
    if (!norm) return MOE_ERR_INVALID_ARG;
    if ((st = check_norm(norm)) != MOE_OK) return st;
    if ((st = check_gate(gate_kind, gate, shape->T)) != MOE_OK) return st;
    if (dgate && gate_kind == MOE_GATE_NONE) return MOE_ERR_INVALID_ARG;
    if (norm->kind == MOE_NORM_NONE && (dweight || dbias)) return MOE_ERR_INVALID_ARG;
    if (shape->T > 0 && (!x || !dout || !dx)) return MOE_ERR_INVALID_ARG;
    size_t need = 0;
    moe_norm_backward_workspace_size(shape, &need);
    const bool columns = dweight || dbias || (dgate && gate_kind == MOE_GATE_CHANNEL);
    if (columns && (!workspace || workspace_bytes < need)) return MOE_ERR_WORKSPACE;
    if (shape->T == 0 && !columns) return MOE_OK;
    if (shape->T == 0 && gate_kind == MOE_GATE_CHANNEL && !gate) return MOE_ERR_INVALID_ARG;
    moe::NormBackwardParams p{};
    p.x = x;
    p.dout = dout;
    p.dadd = dadd;
    p.gate = gate;
    p.dx = dx;
    p.dweight = dweight;
    p.dbias = dbias;
    p.dgate = dgate;
    p.part = columns ? static_cast<float*>(workspace) : nullptr;
    p.norm = norm_dev(norm);
    p.T = shape->T;
    p.H = shape->H;
    p.gate_kind = gate_kind;
    p.scale = scale;
    const void* ptrs[] = {x, dout, dadd, dx, norm->weight, norm->bias, p.part,
                          gate_kind == MOE_GATE_CHANNEL ? gate : nullptr};
    const bool vec = all_aligned(ptrs) && p.H % 4 == 0;
    const bool bf16 = shape->dtype == MOE_BF16;
    if (bf16 && !vec) return MOE_ERR_UNSUPPORTED;
    const Span out = rows_span(shape, dx, p.T);
    for (const void* in : {x, dout, dadd})
        if (!same_or_apart(out, rows_span(shape, in, p.T))) return MOE_ERR_INVALID_ARG;
    return cuda_status(moe::launch_norm_backward(p, bf16, vec, num_sms(),
                                                 static_cast<cudaStream_t>(stream)));
}

moe_status moe_grad_norm_workspace_size(size_t* bytes) {
    if (!bytes) return MOE_ERR_INVALID_ARG;
    *bytes = moe::kGradParts * sizeof(double);
    return MOE_OK;
}

moe_status moe_grad_square_sum(int32_t n, void* const* grads, const int64_t* numel,
                               const int32_t* dtype, double* total, void* workspace,
                               size_t workspace_bytes, void* stream) {
    moe_status st = check_grads(n, grads, numel, dtype);
    if (st != MOE_OK) return st;
    if (!total) return MOE_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < moe::kGradParts * sizeof(double)) return MOE_ERR_WORKSPACE;
    if (!aligned16(workspace) || reinterpret_cast<uintptr_t>(total) % 8) return MOE_ERR_UNSUPPORTED;
    const int32_t chunk = chunk_values(n, numel);
    double* part = static_cast<double*>(workspace);
    const int parts = grad_parts(n, numel, chunk);
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    st = square_sum_parts(n, grads, numel, dtype, chunk, part, parts, cs);
    if (st != MOE_OK) return st;
    return cuda_status(moe::launch_grad_total(part, parts, total, cs));
}

moe_status moe_clip_grads(int32_t n, void* const* grads, const int64_t* numel,
                          const int32_t* dtype, const double* total, float max_norm, float* norm,
                          void* stream) {
    const moe_status st = check_grads(n, grads, numel, dtype);
    if (st != MOE_OK) return st;
    if (!total || !good_max_norm(max_norm)) return MOE_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(total) % 8) return MOE_ERR_UNSUPPORTED;
    return scale_all(n, grads, numel, dtype, chunk_values(n, numel), total, 1, max_norm, norm,
                     static_cast<cudaStream_t>(stream));
}

moe_status moe_clip_grad_norm(int32_t n, void* const* grads, const int64_t* numel,
                              const int32_t* dtype, float max_norm, float* norm, void* workspace,
                              size_t workspace_bytes, void* stream) {
    moe_status st = check_grads(n, grads, numel, dtype);
    if (st != MOE_OK) return st;
    if (!good_max_norm(max_norm)) return MOE_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < moe::kGradParts * sizeof(double)) return MOE_ERR_WORKSPACE;
    if (!aligned16(workspace)) return MOE_ERR_UNSUPPORTED;
    const int32_t chunk = chunk_values(n, numel);
    double* part = static_cast<double*>(workspace);
    const int parts = grad_parts(n, numel, chunk);
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    st = square_sum_parts(n, grads, numel, dtype, chunk, part, parts, cs);
    if (st != MOE_OK) return st;
    return scale_all(n, grads, numel, dtype, chunk, part, parts, max_norm, norm, cs);
}

}  // extern "C"
