// Rounding to E4M3 with block scales: expert weights (once, at load time) and
// the activations that enter the experts.
#include "fp8.cuh"

namespace moe {

namespace {

// Weights: one CTA per 128 x 128 block of a matrix.
//   s = amax|W| / 448 over the block's finite values (1 for a block of zeros,
//   at least 2^-126), code = e4m3(W / s), the division correctly rounded.
// Bound by memory: each value is read once, kept as it was read in registers
// over the CTA's maximum, and its code written once.  A thread holds pieces of
// 16 columns (bf16: four, of two 16-byte loads each; float32: two, of four), so
// that a code store is 16 bytes and 1024 resident threads keep 128 KB of loads
// in flight on an SM.  32 x 6400 x 4096 bf16 (2.5 GB): 392 to 433 us from card to
// card, 0.90 to 0.99 of the copy bandwidth; with a division per value the
// arithmetic took 785 us.
template <typename T> struct QuantPiece;
template <> struct QuantPiece<__nv_bfloat16> {
    static constexpr int LOADS = 2, PIECES = 4;
    // largest magnitude of the piece, NaN skipped, two values at a time
    __device__ __forceinline__ static float top(const uint4 (&u)[2]) {
        __nv_bfloat162 m = __float2bfloat162_rn(0.f);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t w[4] = {u[h].x, u[h].y, u[h].z, u[h].w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                m = __hmax2(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[e])));
        }
        return fmaxf(__low2float(m), __high2float(m));
    }
    __device__ __forceinline__ static float value(const uint4 (&u)[2], int e) {
        const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
        return __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
    }
};
template <> struct QuantPiece<float> {
    static constexpr int LOADS = 4, PIECES = 2;
    __device__ __forceinline__ static float top(const uint4 (&u)[4]) {
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) m = fmaxf(m, fabsf(value(u, e)));
        return m;
    }
    __device__ __forceinline__ static float value(const uint4 (&u)[4], int e) {
        const uint4& q = u[e / 4];
        return __uint_as_float(e % 4 == 0 ? q.x : e % 4 == 1 ? q.y : e % 4 == 2 ? q.z : q.w);
    }
};

// Maximum over the CTA.
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t (&red)[32]) {
    v = __reduce_max_sync(0xffffffffu, v);
    __syncthreads();                // the last use of red
    if (threadIdx.x < 32) red[threadIdx.x] = 0;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    return __reduce_max_sync(0xffffffffu, red[threadIdx.x & 31]);
}

template <typename T>
__global__ void __launch_bounds__(1024 / QuantPiece<T>::PIECES, QuantPiece<T>::PIECES) fp8_quantize_weights_kernel(
    const T* __restrict__ w, int rows, int cols, int row_blocks, int col_blocks,
    uint8_t* __restrict__ q, float* __restrict__ s) {
    using P = QuantPiece<T>;
    constexpr int THREADS = 1024 / P::PIECES;       // 128 rows x 8 pieces
    __shared__ uint32_t red[32];
    const int64_t b = blockIdx.x;
    const int cb = static_cast<int>(b % col_blocks);
    const int rb = static_cast<int>(b / col_blocks % row_blocks);
    const int64_t n = b / col_blocks / row_blocks;
    uint4 raw[P::PIECES][P::LOADS];
    int64_t at[P::PIECES];
#pragma unroll
    for (int i = 0; i < P::PIECES; ++i) {
        const int piece = threadIdx.x + i * THREADS;
        const int r = rb * 128 + piece / 8, c = cb * 128 + piece % 8 * 16;
        at[i] = r < rows && c < cols ? (n * rows + r) * cols + c : -1;
        const uint4* src = reinterpret_cast<const uint4*>(w + at[i]);
#pragma unroll
        for (int h = 0; h < P::LOADS; ++h)
            raw[i][h] = at[i] >= 0 ? __ldg(src + h) : make_uint4(0, 0, 0, 0);
    }
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < P::PIECES; ++i) top = fmaxf(top, P::top(raw[i]));
    uint32_t mag = __float_as_uint(top);
    mag = block_max(mag, red);
    const bool infinite = mag >= 0x7f800000u;
    if (infinite) {                                 // infinities take no part in the scale
        mag = 0;
#pragma unroll
        for (int i = 0; i < P::PIECES; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) mag = max(mag, finite_mag(P::value(raw[i], e)));
        mag = block_max(mag, red);
    }
    const float amax = __uint_as_float(mag);
    const float scale = mag == 0 ? 1.f : fmaxf(amax / kE4M3Max, 1.17549435e-38f);
    if (threadIdx.x == 0) s[b] = scale;
    // The correctly rounded quotient from the correctly rounded reciprocal
    // (Markstein, IBM J. Res. Dev. 34, 1990): q = w y, then q - (s q - w) y; the
    // residual is exact as long as it cannot underflow.
    const float y = 1.f / scale;
    const bool by_reciprocal = !infinite && scale > 7.8886091e-31f;     // 2^-100
    auto store = [&](auto quotient) {
#pragma unroll
        for (int i = 0; i < P::PIECES; ++i) {
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[e] = e4m3x4(quotient(P::value(raw[i], 4 * e)),
                              quotient(P::value(raw[i], 4 * e + 1)),
                              quotient(P::value(raw[i], 4 * e + 2)),
                              quotient(P::value(raw[i], 4 * e + 3)));
            if (at[i] >= 0)
                *reinterpret_cast<uint4*>(q + at[i]) = make_uint4(o[0], o[1], o[2], o[3]);
        }
    };
    if (by_reciprocal)
        store([&](float x) {
            const float t = x * y;
            return fmaf(-fmaf(scale, t, -x), y, t);
        });
    else
        store([&](float x) { return nan_if_not_finite(x) / scale; });
}

// Activations: row p < T*k of xq is x of the token of sorted slot p, rows past
// them (with shared experts) the T tokens in order.  A warp takes 8 blocks of
// 128 columns of a row of x, 16 lanes a block with 8 values each, its four
// loads in flight together.
//   BY_TOKEN: once per token, written to each of its slots' rows (inv: the
//     sorted position of each slot), for large batches: 16384 tokens x 2048
//     columns with 6 + 1 rows each take 130 us slot by slot, the rounding being
//     what bounds them.
//   else: once per row, without the inverse permutation (one launch less), for
//     small ones; also clears the counters on which their GEMMs' partial tiles
//     arrive.
constexpr int kRowLoads = 4;
constexpr int kRowBlocks = 2 * kRowLoads;

struct QuantRowsParams {
    const uint4* x;
    const int32_t* perm;
    const int32_t* inv;
    const int32_t* placed;     // offsets[E]: slots that the plan placed
    int64_t T, slots;
    int k, S, H;
    uint8_t* xq;
    uint8_t* xs;
    int32_t* arrived;
    int counters;
};

template <bool BY_TOKEN>
__global__ void __launch_bounds__(256) fp8_quantize_rows_kernel(const QuantRowsParams p) {
    const int blocks = (p.H + kFp8Block - 1) / kFp8Block;
    const int per_row = (blocks + kRowBlocks - 1) / kRowBlocks;
    const int ld = fp8_scale_ld(p.H), vec = p.H / 8;
    const int lane = threadIdx.x & 15, half = threadIdx.x >> 4 & 1;
    const int64_t total = (BY_TOKEN ? p.T : p.slots + (p.S > 0 ? p.T : 0)) * per_row;
    pdl_wait();
    pdl_launch_dependents();     // after the wait: see the GEMM's prologue
    const int placed = BY_TOKEN ? placed_slots(p.placed, p.slots) : 0;
    if (!BY_TOKEN)
        for (int i = blockIdx.x * 256 + threadIdx.x; i < p.counters; i += gridDim.x * 256)
            p.arrived[i] = 0;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); i < total;
         i += static_cast<int64_t>(gridDim.x) * 8) {
        const int64_t row = total <= 0xffffffffll
                                ? static_cast<uint32_t>(i) / static_cast<uint32_t>(per_row)
                                : i / per_row;
        const int first = static_cast<int>(i - row * per_row) * kRowBlocks + half;
        int64_t token = row;
        if (!BY_TOKEN) {
            token = row - p.slots;
            if (row < p.slots) {
                const int32_t q = p.perm[row];
                // a plan with skipped slots (bad expert index) leaves holes
                if (q < 0 || q >= p.slots) continue;
                token = q / p.k;
            }
        }
        uint4 u[kRowLoads];
#pragma unroll
        for (int n = 0; n < kRowLoads; ++n) {
            const int c = (first + 2 * n) * 16 + lane;
            u[n] = c < vec ? p.x[token * vec + c] : make_uint4(0, 0, 0, 0);
        }
        uint2 codes[kRowLoads];
        uint32_t byte[kRowLoads];
#pragma unroll
        for (int n = 0; n < kRowLoads; ++n) codes[n] = e4m3_block_piece(u[n], byte[n]);
        auto write = [&](int64_t to) {
#pragma unroll
            for (int n = 0; n < kRowLoads; ++n) {
                const int b = first + 2 * n, c = b * 16 + lane;
                if (c < vec) *reinterpret_cast<uint2*>(p.xq + to * p.H + c * 8) = codes[n];
                if (lane == 0 && b < blocks) p.xs[to * ld + b] = static_cast<uint8_t>(byte[n]);
            }
        };
        if (BY_TOKEN) {
            for (int j = 0; j < p.k; ++j) {
                const int64_t slot = token * p.k + j;
                const int32_t at = p.inv[slot];
                // a slot that the plan skipped has no entry: whatever is there
                // leads to no placed row, or to another slot's
                if (at >= 0 && at < placed && p.perm[at] == slot) write(at);
            }
            if (p.S > 0) write(p.slots + token);
        } else {
            write(row);
        }
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
        fp8_quantize_weights_kernel<<<static_cast<unsigned>(blocks), 256, 0, st>>>(
            static_cast<const __nv_bfloat16*>(w), rows, cols, rb, cb, q, s);
    else
        fp8_quantize_weights_kernel<<<static_cast<unsigned>(blocks), 512, 0, st>>>(
            static_cast<const float*>(w), rows, cols, rb, cb, q, s);
    return cudaGetLastError();
}

cudaError_t launch_fp8_quantize_rows(const moe_shape& s, const Fp8Operands& o, int num_sms,
                                     cudaStream_t st) {
    const Fp8Tiles tiles = fp8_tiles(s);
    const bool by_token = fp8_by_token(s);
    const QuantRowsParams p{static_cast<const uint4*>(o.x), o.perm, o.inv, o.offsets + s.E, s.T,
                            s.T * s.k, s.k, s.n_shared, s.H, o.xq, o.xs, o.arrived,
                            fp8_is_split(s) ? static_cast<int>(tiles.gate_up + tiles.down) : 0};
    const int64_t most = static_cast<int64_t>(num_sms) * 8;
    auto grid_for = [&](int64_t ctas) { return dim3(static_cast<unsigned>(ctas < most ? ctas : most)); };
    if (by_token) {
        const cudaError_t e = launch_invert_perm(o.perm, p.placed, o.inv, p.slots, num_sms, st);
        if (e != cudaSuccess) return e;
    }
    const int blocks = (s.H + kFp8Block - 1) / kFp8Block;
    const int64_t rows = by_token ? s.T : p.slots + (s.n_shared > 0 ? s.T : 0);
    const int64_t warps = rows * ((blocks + kRowBlocks - 1) / kRowBlocks);
    return launch_pdl(by_token ? fp8_quantize_rows_kernel<true> : fp8_quantize_rows_kernel<false>,
                      grid_for((warps + 7) / 8), dim3(256), 0, st, p);
}

}  // namespace moe
