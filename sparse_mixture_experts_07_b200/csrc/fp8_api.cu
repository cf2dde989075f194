// The C ABI of the 8-bit expert path: host-side validation, workspace layout
// and dispatch.
#include "fp8.cuh"
#include "host_common.cuh"

namespace {

using namespace moe::host;

struct Fp8Layout {
    size_t xq, xs, hq, hs, hq_sh, hs_sh, inv, part, arrived, total;
};

Fp8Layout fp8_layout(const moe_shape& s) {
    Fp8Layout l{};
    const size_t Tk = static_cast<size_t>(s.T * s.k);
    const size_t rows = Tk + (s.n_shared > 0 ? static_cast<size_t>(s.T) : 0);
    const size_t ST = static_cast<size_t>(s.n_shared) * static_cast<size_t>(s.T);
    const size_t Is = s.n_shared > 0 ? static_cast<size_t>(s.I_shared) : 0;
    size_t off = 0;
    l.xq = off;
    off += align_up(rows * s.H);
    l.xs = off;
    off += align_up(rows * moe::fp8_scale_ld(s.H));
    l.hq = off;
    off += align_up(Tk * s.I);
    l.hs = off;
    off += align_up(Tk * moe::fp8_scale_ld(s.I));
    l.hq_sh = off;
    off += align_up(ST * Is);
    l.hs_sh = off;
    off += align_up(ST * moe::fp8_scale_ld(static_cast<int>(Is)));
    l.inv = off;
    if (moe::fp8_by_token(s)) off += align_up(Tk * 4);
    l.part = l.arrived = off;
    if (moe::fp8_is_split(s)) {
        off += align_up(static_cast<size_t>(num_sms()) * 2 * moe::fp8_part_rows(s) * 256 * 4);
        l.arrived = off;
        const moe::Fp8Tiles tiles = moe::fp8_tiles(s);
        off += align_up(static_cast<size_t>(tiles.gate_up + tiles.down) * 4);
    }
    l.total = off;
    return l;
}

// bf16 activations; rows of codes in whole 16-byte pieces, as TMA takes them.
moe_status check_fp8_shape(const moe_shape* s) {
    const moe_status st = moe::check_shape(s);
    if (st != MOE_OK) return st;
    if (s->dtype != MOE_BF16 || s->H % 16 || s->I % 16 || (s->n_shared > 0 && s->I_shared % 16))
        return MOE_ERR_UNSUPPORTED;
    // rows of the weight tensors are indexed in 32 bits
    constexpr int64_t kMaxRows = int64_t(1) << 31;
    if (int64_t(s->E) * 2 * s->I >= kMaxRows || int64_t(s->E) * s->H >= kMaxRows ||
        int64_t(s->n_shared) * 2 * s->I_shared >= kMaxRows ||
        int64_t(s->n_shared) * s->H >= kMaxRows)
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_fp8_quantize(int64_t n, int32_t rows, int32_t cols, const void* w, int32_t dtype,
                            uint8_t* q, float* s, void* stream) {
    if (n < 0 || rows < 0 || cols < 0 || (dtype != MOE_F32 && dtype != MOE_BF16))
        return MOE_ERR_INVALID_ARG;
    if (n == 0 || rows == 0 || cols == 0) return MOE_OK;
    if (!w || !q || !s) return MOE_ERR_INVALID_ARG;
    if (cols % 16 || !aligned16(w) || !aligned16(q) || reinterpret_cast<uintptr_t>(s) % 4)
        return MOE_ERR_UNSUPPORTED;
    const int64_t blocks = ((rows + int64_t(127)) / 128) * ((cols + int64_t(127)) / 128);
    if (n > 0x7fffffff / blocks) return MOE_ERR_UNSUPPORTED;
    return cuda_status(moe::launch_fp8_quantize_weights(w, dtype == MOE_BF16, n, rows, cols, q, s,
                                                        static_cast<cudaStream_t>(stream)));
}

moe_status moe_fp8_workspace_size(const moe_shape* shape, size_t* bytes) {
    const moe_status st = check_fp8_shape(shape);
    if (st != MOE_OK) return st;
    if (!bytes) return MOE_ERR_INVALID_ARG;
    *bytes = fp8_layout(*shape).total;
    return MOE_OK;
}

moe_status moe_forward_fp8(const moe_shape* shape, const void* x, const int32_t* offsets,
                           const int32_t* perm, const float* topk_w, const uint8_t* gate_up_q,
                           const float* gate_up_s, const uint8_t* down_q, const float* down_s,
                           const uint8_t* sh_gate_up_q, const float* sh_gate_up_s,
                           const uint8_t* sh_down_q, const float* sh_down_s, void* y_slots,
                           int32_t* err_flag, void* workspace, size_t workspace_bytes,
                           void* stream) {
    const moe_status st = check_fp8_shape(shape);
    if (st != MOE_OK) return st;
    const moe_shape& s = *shape;
    if (s.T == 0) return MOE_OK;
    if (!x || !offsets || !perm || !topk_w || !gate_up_q || !gate_up_s || !down_q || !down_s ||
        !y_slots)
        return MOE_ERR_INVALID_ARG;
    if (s.n_shared > 0 && (!sh_gate_up_q || !sh_gate_up_s || !sh_down_q || !sh_down_s))
        return MOE_ERR_INVALID_ARG;
    const Fp8Layout l = fp8_layout(s);
    if (!workspace || workspace_bytes < l.total) return MOE_ERR_WORKSPACE;
    const void* ptrs[] = {x, gate_up_q, down_q, y_slots, workspace};
    for (const void* p : ptrs)
        if (!aligned16(p)) return MOE_ERR_UNSUPPORTED;
    if (s.n_shared > 0 && (!aligned16(sh_gate_up_q) || !aligned16(sh_down_q)))
        return MOE_ERR_UNSUPPORTED;
    auto* ws = static_cast<uint8_t*>(workspace);
    const moe::Fp8Operands o{x, offsets, perm, topk_w, gate_up_q, gate_up_s, down_q, down_s,
                             sh_gate_up_q, sh_gate_up_s, sh_down_q, sh_down_s, y_slots, err_flag,
                             ws + l.xq, ws + l.xs, ws + l.hq, ws + l.hs, ws + l.hq_sh,
                             ws + l.hs_sh, reinterpret_cast<int32_t*>(ws + l.inv),
                             reinterpret_cast<float*>(ws + l.part),
                             reinterpret_cast<int32_t*>(ws + l.arrived)};
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    cudaError_t e = moe::launch_fp8_quantize_rows(s, o, num_sms(), cs);
    if (e != cudaSuccess) return MOE_ERR_CUDA;
    return cuda_status(moe::launch_ffn_fp8(s, o, num_sms(), cs));
}

}  // extern "C"
