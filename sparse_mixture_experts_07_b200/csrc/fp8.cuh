// Shared pieces of the 8-bit (E4M3) expert path: rounding to codes, block
// scales, and the launch functions' declarations.
//
// Values are codes times a scale per block of 128 along the contraction:
//   weights     one float32 scale per 128 x 128 block;
//   activations one power of two per row and 128 columns, stored as an E8M0
//               byte b (the scale is 2^(b - 127)): the smallest power of two
//               that brings the block's largest magnitude to at most 448, the
//               largest E4M3 value.  Dividing by a power of two is exact, so
//               a code is the once-rounded activation.
// A value that is not finite gets the NaN code and takes no part in its
// block's scale; its row's outputs are NaN.
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kFp8Block = 128;
constexpr float kE4M3Max = 448.f;

// Two floats to two E4M3 codes, nearest even (lo in the low byte); magnitudes
// past 448 saturate, NaN gives the NaN code.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}

// Magnitude bits of a finite value, 0 of one that is not: unsigned order is
// the order of magnitudes.
__device__ __forceinline__ uint32_t finite_mag(float v) {
    const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
    return b < 0x7f800000u ? b : 0u;
}

// E8M0 byte of a block whose largest magnitude has the float bits `mag`:
// 2^e >= amax / 448 = amax / (1.75 * 2^8) with e = exponent - 8, one more when
// the significand is above 1.75.  At least 1 (2^-126), so that the inverse is
// a normal float too.
__device__ __forceinline__ uint32_t e8m0_of(uint32_t mag) {
    const int e = static_cast<int>(mag >> 23) - 8 + ((mag & 0x7fffffu) > 0x600000u ? 1 : 0);
    return static_cast<uint32_t>(e < 1 ? 1 : e);
}
__device__ __forceinline__ float e8m0_value(uint32_t byte) { return __uint_as_float(byte << 23); }
__device__ __forceinline__ float e8m0_inverse(uint32_t byte) {
    return __uint_as_float((254u - byte) << 23);
}

// A value that is not finite as NaN (an infinity would saturate to a number).
__device__ __forceinline__ float nan_if_not_finite(float v) {
    return (__float_as_uint(v) & 0x7f800000u) == 0x7f800000u ? __uint_as_float(0x7fffffffu) : v;
}

// Rounds 8 consecutive bf16 values of a 128-column block that 16 neighbouring
// lanes hold (all 32 lanes call); `byte` is the block's E8M0 scale.
__device__ __forceinline__ uint2 e4m3_block_piece(const uint4& u, uint32_t& byte) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    const uint32_t half_mask = threadIdx.x & 16 ? 0xffff0000u : 0x0000ffffu;
    // the largest magnitude, two values at a time; NaN is skipped
    __nv_bfloat162 m = __float2bfloat162_rn(0.f);
    float v[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        m = __hmax2(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[e])));
        v[2 * e] = __uint_as_float(w[e] << 16);
        v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
    uint32_t mag = __float_as_uint(fmaxf(__low2float(m), __high2float(m)));
    mag = __reduce_max_sync(half_mask, mag);
    if (mag >= 0x7f800000u) {            // an infinity: NaN, and outside the maximum
        mag = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            mag = max(mag, finite_mag(v[e]));
            v[e] = nan_if_not_finite(v[e]);
        }
        mag = __reduce_max_sync(half_mask, mag);
    }
    byte = e8m0_of(mag);
    const float inv = e8m0_inverse(byte);
    return make_uint2(e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                      e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
}

// Bytes per row of E8M0 scales: one per 128 columns, rows 16-byte aligned.
__host__ __device__ inline int fp8_scale_ld(int cols) {
    return ((cols + kFp8Block - 1) / kFp8Block + 15) / 16 * 16;
}

// Operands of the expert FFNs on E4M3 weights.
struct Fp8Operands {
    const void* x;             // [T, H] bf16
    const int32_t* offsets;    // [E+1]
    const int32_t* perm;       // [T*k]
    const float* topk_w;       // [T*k]
    const uint8_t* gate_up;    // [E, 2I, H]
    const float* gate_up_s;    // [E, 2, ceil(I/128), ceil(H/128)]
    const uint8_t* down;       // [E, H, I]
    const float* down_s;       // [E, ceil(H/128), ceil(I/128)]
    const uint8_t* sh_gate_up; // [S, 2Is, H] and so on
    const float* sh_gate_up_s;
    const uint8_t* sh_down;
    const float* sh_down_s;
    void* y_slots;             // [T*k + S*T, H] bf16
    int32_t* err_flag;
    // workspace
    uint8_t* xq;               // [T*k + (S > 0 ? T : 0), H] codes, sorted slots then tokens
    uint8_t* xs;               // their E8M0 scales, fp8_scale_ld(H) per row
    uint8_t* hq;               // [T*k, I] codes of SwiGLU outputs
    uint8_t* hs;
    uint8_t* hq_sh;            // [S*T, Is]
    uint8_t* hs_sh;
    int32_t* inv;              // [T*k] sorted position of each slot (fp8_by_token)
    // small batches (fp8_is_split)
    float* part;               // [SMs, 2, fp8_part_rows, 256] sums of partial tiles
    int32_t* arrived;          // [tiles of both GEMMs] K-blocks whose sums are in part
};

// Batches whose K-blocks are shared out over the SMs rather than whole tiles:
// few rows per expert, so that what takes the time is reading the weights, and
// a tile's sums are small.  Both ways on one B200, us shared out / in whole tiles:
//                                        1 token  8 tokens  32 tokens  128 tokens
//   top-2 of 16, 4096 x 6400              42/68    129/146   237/243    257/253
//   top-8 of 256 + 1, 2048 x 1024         35/33     90/95    200/216    360/354
//   top-6 of 64 + 2, 2048 x 1024          42/38     80/75    107/93     115/97
// The rule looks at the tokens alone: the last line's tiles are short and many,
// and whole ones serve it better throughout.
constexpr int kFp8SplitRows = 32;      // rows of their tiles
inline bool fp8_is_split(const moe_shape& s) { return s.T <= kFp8SplitRows; }
// Batches whose activations are rounded once per token rather than once per
// slot, through the inverse permutation.
inline bool fp8_by_token(const moe_shape& s) { return !fp8_is_split(s) && s.k + s.n_shared > 1; }

// Most rows of one such tile with data.
inline int fp8_part_rows(const moe_shape& s) {
    return static_cast<int>(s.T * s.k < kFp8SplitRows ? s.T * s.k : kFp8SplitRows);
}

// At most this many tiles: every group may end in a partial m-tile.
struct Fp8Tiles {
    int64_t gate_up, down;
};
inline Fp8Tiles fp8_tiles(const moe_shape& s) {
    const int64_t slots = s.T * s.k;
    const int64_t rows = fp8_is_split(s) ? kFp8SplitRows : 128;
    const int64_t m = (slots + rows - 1) / rows + (s.E < slots ? s.E : slots);
    const int64_t ms = s.n_shared * ((s.T + rows - 1) / rows);
    const int64_t Is = s.n_shared > 0 ? s.I_shared : 0;
    return {m * ((s.I + 127) / 128) + ms * ((Is + 127) / 128), (m + ms) * ((s.H + 255) / 256)};
}

cudaError_t launch_fp8_quantize_weights(const void* w, bool bf16, int64_t n, int rows, int cols,
                                        uint8_t* q, float* s, cudaStream_t);
cudaError_t launch_fp8_quantize_rows(const moe_shape&, const Fp8Operands&, int num_sms,
                                     cudaStream_t);
cudaError_t launch_ffn_fp8(const moe_shape&, const Fp8Operands&, int num_sms, cudaStream_t);

}  // namespace moe
