// Rounding to E4M3 with block scales: expert weights (once, at load time) and
// the activations that enter the experts.
#include "fp8.cuh"

namespace moe {

namespace {

constexpr int kThreads = 512;

// Weights: one CTA per 128 x 128 block of a matrix.
//   s = amax|W| / 448 over the block's finite values (1 for a block of zeros,
//   at least 2^-126), code = e4m3(W / s), the division correctly rounded.
// Bound by memory: each value is read once, kept in registers over the CTA's
// maximum, and its code written once.  A thread holds pieces of 16 columns
// (bf16: two 16-byte loads, float32: four), so that a code store is 16 bytes.
template <typename T>
__global__ void __launch_bounds__(kThreads) fp8_quantize_weights_kernel(
    const T* __restrict__ w, int rows, int cols, int row_blocks, int col_blocks,
    uint8_t* __restrict__ q, float* __restrict__ s) {
    constexpr int kPieces = 2;              // 128 rows x 8 pieces of 16 over 512 threads
    __shared__ uint32_t red[kThreads / 32];
    const int64_t b = blockIdx.x;
    const int cb = static_cast<int>(b % col_blocks);
    const int rb = static_cast<int>(b / col_blocks % row_blocks);
    const int64_t n = b / col_blocks / row_blocks;
    float v[kPieces][16];
    int64_t at[kPieces];
    uint32_t mag = 0;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const int piece = threadIdx.x + i * kThreads;
        const int r = rb * 128 + piece / 8, c = cb * 128 + piece % 8 * 16;
        at[i] = r < rows && c < cols ? (n * rows + r) * cols + c : -1;
#pragma unroll
        for (int e = 0; e < 16; ++e) v[i][e] = 0.f;
        if (at[i] < 0) continue;
        if constexpr (sizeof(T) == 2) {
            const uint4* src = reinterpret_cast<const uint4*>(w + at[i]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint4 u = src[h];
                const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[i][8 * h + 2 * e] = __uint_as_float(x[e] << 16);
                    v[i][8 * h + 2 * e + 1] = __uint_as_float(x[e] & 0xffff0000u);
                }
            }
        } else {
            const float4* src = reinterpret_cast<const float4*>(w + at[i]);
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const float4 u = src[h];
                v[i][4 * h] = u.x; v[i][4 * h + 1] = u.y;
                v[i][4 * h + 2] = u.z; v[i][4 * h + 3] = u.w;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) mag = max(mag, finite_mag(v[i][e]));
    mag = __reduce_max_sync(0xffffffffu, mag);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = mag;
    __syncthreads();
    mag = __reduce_max_sync(0xffffffffu, red[threadIdx.x & (kThreads / 32 - 1)]);
    const float amax = __uint_as_float(mag);
    const float scale = mag == 0 ? 1.f : fmaxf(amax / kE4M3Max, 1.17549435e-38f);
    if (threadIdx.x == 0) s[b] = scale;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        if (at[i] < 0) continue;
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            o[e] = e4m3x4(nan_if_not_finite(v[i][4 * e]) / scale,
                          nan_if_not_finite(v[i][4 * e + 1]) / scale,
                          nan_if_not_finite(v[i][4 * e + 2]) / scale,
                          nan_if_not_finite(v[i][4 * e + 3]) / scale);
        *reinterpret_cast<uint4*>(q + at[i]) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// Activations: row p < T*k is x of the token of sorted slot p, rows past them
// (with shared experts) the T tokens in order.  16 lanes hold a row's 128
// columns, 8 values each.  For a small batch it also clears the counters on
// which the GEMMs' partial tiles arrive.
__global__ void __launch_bounds__(256) fp8_quantize_rows_kernel(
    const uint4* __restrict__ x, const int32_t* __restrict__ perm, int64_t slots, int64_t rows,
    int k, int H, uint8_t* __restrict__ xq, uint8_t* __restrict__ xs, int32_t* arrived,
    int counters) {
    const int blocks = (H + kFp8Block - 1) / kFp8Block;
    const int ld = fp8_scale_ld(H), vec = H / 8;
    const int lane = threadIdx.x & 15;
    const int64_t total = rows * blocks;
    pdl_wait();
    pdl_launch_dependents();     // after the wait: see the GEMM's prologue
    for (int i = blockIdx.x * 256 + threadIdx.x; i < counters; i += gridDim.x * 256) arrived[i] = 0;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4);
         i - (threadIdx.x >> 4) < total; i += static_cast<int64_t>(gridDim.x) * 16) {
        const int64_t row = i / blocks;
        const int b = static_cast<int>(i - row * blocks);
        int64_t token = -1;
        if (i < total) {
            if (row < slots) {
                const int64_t q = perm[row];
                // a plan with skipped slots (bad expert index) leaves holes
                if (q >= 0 && q < slots) token = q / k;
            } else {
                token = row - slots;
            }
        }
        const int c = b * 16 + lane;
        const bool in = token >= 0 && c < vec;
        const uint4 u = in ? x[token * vec + c] : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        float v[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[2 * e] = __uint_as_float(w[e] << 16);
            v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        }
        uint32_t byte;
        const uint2 codes = e4m3_block_piece(v, byte);
        if (in) *reinterpret_cast<uint2*>(xq + row * H + c * 8) = codes;
        if (lane == 0 && token >= 0) xs[row * ld + b] = static_cast<uint8_t>(byte);
    }
}

}  // namespace

cudaError_t launch_fp8_quantize_weights(const void* w, bool bf16, int64_t n, int rows, int cols,
                                        uint8_t* q, float* s, cudaStream_t st) {
    const int rb = (rows + 127) / 128, cb = (cols + 127) / 128;
    const int64_t blocks = n * rb * cb;
    if (blocks == 0) return cudaSuccess;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    if (bf16)
        fp8_quantize_weights_kernel<<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(
            static_cast<const __nv_bfloat16*>(w), rows, cols, rb, cb, q, s);
    else
        fp8_quantize_weights_kernel<<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(
            static_cast<const float*>(w), rows, cols, rb, cb, q, s);
    return cudaGetLastError();
}

cudaError_t launch_fp8_quantize_rows(const moe_shape& s, const Fp8Operands& o, int num_sms,
                                     cudaStream_t st) {
    const int64_t slots = s.T * s.k, rows = slots + (s.n_shared > 0 ? s.T : 0);
    const int64_t total = rows * ((s.H + kFp8Block - 1) / kFp8Block);
    const Fp8Tiles tiles = fp8_tiles(s);
    int64_t grid = (total + 15) / 16;
    if (grid > static_cast<int64_t>(num_sms) * 16) grid = static_cast<int64_t>(num_sms) * 16;
    return launch_pdl(fp8_quantize_rows_kernel, dim3(static_cast<unsigned>(grid)), dim3(256), 0, st,
                      static_cast<const uint4*>(o.x), o.perm, slots, rows, s.k, s.H, o.xq, o.xs, o.arrived,
                      fp8_is_split(s) ? static_cast<int>(tiles.gate_up + tiles.down) : 0);
}

}  // namespace moe
