// Norms before and after the block, fused with the combine, the gate and the
// scaled residual, and their backward pass.
//
// A decoder layer puts the block between norms and adds its output to the
// residual stream ("PhiMoE in Transformers", section 2: layer norms with
// weight and bias; GraniteMoeSWA decoder layer: RMS norms, the block's output
// times residual_multiplier added to the residual).  With
//   N(v) = (v - m) r w + b,  r = 1 / sqrt(mean((v - m)^2) + eps),
//   m = mean(v) for a layer norm, 0 for an RMS norm (kind none: N(v) = v),
// the kernels compute, per token t and hidden column c,
//   y = sum of the token's slot rows (moe_combine's sum, same order),
//   h = residual + scale * gate * N_post(y),        xn = N_next(h),
// in one pass: the row stays in registers from the slot loads to xn, so y, z
// and the second read of h never touch memory.  All arithmetic is float32;
// y, h and xn are each rounded once, when stored (xn is computed from the
// unrounded h).
//
// Bound by memory: (k + S + 1) rows read, 2 (3 with y) written.  One CTA owns
// one row at a time; what hides a row's load latency and its block-wide sums is
// the other CTAs of the SM, so registers are held to five CTAs of 256 threads:
// two 16-byte vectors per thread and at most 8 loads in flight.  Measured on a
// B200, 32768 tokens of 2048 columns, 6 + 1 slots (1.34 GB): 230 to 245 us from
// card to card, 0.85 to 0.90 of the copy bandwidth.  On the card with 230, one
// vector per thread: 260 us (twice the threads in every barrier); 88 registers and
// two CTAs less: 316 us; rows copied to shared memory two to four tokens ahead,
// two CTAs per SM: 303 us and more.
#include "norm.cuh"

namespace moe {

namespace {

// 16-byte (or, for float32 rows that are not 16-byte aligned, 4-byte) pieces.
template <typename T, int VEC> struct RowIO;
template <> struct RowIO<__nv_bfloat16, 8> {
    using Raw = uint4;
    __device__ __forceinline__ static void unpack(const Raw& u, float (&v)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            v[2 * q] = __uint_as_float(w[q] << 16);
            v[2 * q + 1] = __uint_as_float(w[q] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ static Raw pack(const float (&v)[8]) {
        return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                          pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    }
};
template <> struct RowIO<float, 4> {
    using Raw = float4;
    __device__ __forceinline__ static void unpack(const Raw& u, float (&v)[4]) {
        v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
    }
    __device__ __forceinline__ static Raw pack(const float (&v)[4]) {
        return make_float4(v[0], v[1], v[2], v[3]);
    }
};
template <> struct RowIO<float, 1> {
    using Raw = float;
    __device__ __forceinline__ static void unpack(const Raw& u, float (&v)[1]) { v[0] = u; }
    __device__ __forceinline__ static Raw pack(const float (&v)[1]) { return v[0]; }
};

// A load, zero when !ok: volatile PTX, so that a group of them stays ahead of the
// arithmetic and all of the group are in flight together.
__device__ __forceinline__ uint4 load_if(const uint4* p, bool ok) {
    uint4 v;
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@q ld.global.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
        : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
        : "l"(p), "r"(static_cast<int>(ok)));
    return v;
}
__device__ __forceinline__ float4 load_if(const float4* p, bool ok) {
    const uint4 u = load_if(reinterpret_cast<const uint4*>(p), ok);
    return make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z),
                       __uint_as_float(u.w));
}
__device__ __forceinline__ float load_if(const float* p, bool ok) {
    float v;
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\tmov.f32 %0, 0f00000000;\n\t"
        "@q ld.global.f32 %0, [%1];\n\t}"
        : "=f"(v)
        : "l"(p), "r"(static_cast<int>(ok)));
    return v;
}

// VEC float32 parameters of the columns of vector c.
template <int VEC>
__device__ __forceinline__ void load_params(const float* p, int c, float (&v)[VEC]) {
    if constexpr (VEC % 4 == 0) {
#pragma unroll
        for (int q = 0; q < VEC / 4; ++q) {
            const float4 u = reinterpret_cast<const float4*>(p)[c * (VEC / 4) + q];
            v[4 * q] = u.x; v[4 * q + 1] = u.y; v[4 * q + 2] = u.z; v[4 * q + 3] = u.w;
        }
    } else {
        v[0] = p[c];
    }
}

// Sums of N values over the CTA, in a fixed order.  One barrier per call: the
// calls alternate between two halves of `buf`, and a half is written again
// only after the barrier that follows its last read.
template <int N> struct BlockSum {
    float (*buf)[N][32];      // [2]
    int turn = 0;
    __device__ __forceinline__ void operator()(float (&v)[N]) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        const int warps = static_cast<int>(blockDim.x >> 5);
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) v[n] += __shfl_xor_sync(0xffffffffu, v[n], d);
        if (warps == 1) return;
        if (lane == 0)
#pragma unroll
            for (int n = 0; n < N; ++n) buf[turn][n][warp] = v[n];
        __syncthreads();
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float s = lane < warps ? buf[turn][n][lane] : 0.f;
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
            v[n] = s;
        }
        turn ^= 1;
    }
};

// v = N(v) over the row held by the CTA (columns past H hold 0 and stay out
// of every sum).  The variance is taken about the mean, in a second sum, so
// that rows far from zero lose nothing.
template <int VEC, int VPT>
__device__ __forceinline__ void normalise(float (&v)[VPT][VEC], const NormDev& n, int nvec,
                                          float inv_h, BlockSum<1>& sum) {
    if (n.kind == MOE_NORM_NONE) return;
    float m = 0.f;
    if (n.kind == MOE_NORM_LAYER) {
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) s[0] += v[i][e];
        sum(s);
        m = s[0] * inv_h;
    }
    float q[1] = {0.f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if (static_cast<int>(threadIdx.x + i * blockDim.x) >= nvec) continue;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            v[i][e] -= m;
            q[0] += v[i][e] * v[i][e];
        }
    }
    sum(q);
    const float r = rsqrtf(q[0] * inv_h + n.eps);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c >= nvec) continue;
        float w[VEC];
        if (n.weight) {
            load_params<VEC>(n.weight, c, w);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e) w[e] = 1.f;
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][e] = v[i][e] * r * w[e];
        if (n.bias) {
            load_params<VEC>(n.bias, c, w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[i][e] += w[e];
        }
    }
}

template <typename T, int VEC, int VPT, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? 5 : MAXT == 512 ? 2 : 1)
    combine_norm_kernel(const CombineNormParams p) {
    using IO = RowIO<T, VEC>;
    using Raw = typename IO::Raw;
    __shared__ float red[2][1][32];
    BlockSum<1> sum{red};
    const int nvec = p.H / VEC;
    const float inv_h = 1.f / static_cast<float>(p.H);
    const Raw* slots = static_cast<const Raw*>(p.y_slots);
    const Raw* residual = static_cast<const Raw*>(p.residual);
    const int64_t routed = p.T * p.k;
    const int nrows = p.k + p.S;
    const int lane = threadIdx.x & 31;
    pdl_launch_dependents();
    pdl_wait();
    // lane j holds the row of slot j, k + S <= 24 of them; the next token's are
    // fetched while this one is worked on.  -1: a slot that the plan skipped (bad
    // expert index), which adds nothing.
    auto slot_row = [&](int64_t t) {
        int64_t row = -1;
        if (t < p.T && lane < p.k) {
            row = p.inv[t * p.k + lane];
            if (row >= routed) row = -1;
        } else if (t < p.T && lane < nrows) {
            row = routed + (lane - p.k) * p.T + t;
        }
        return row;
    };
    int64_t mine = slot_row(blockIdx.x);
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        const int64_t rows = mine;
        float v[VPT][VEC];
        Raw res[VPT];
        mine = slot_row(t + gridDim.x);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            res[i] = load_if(residual + t * nvec + c, residual && c < nvec);
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[i][e] = 0.f;
        }
        // up to IN_FLIGHT rows' loads at once, summed in row order
        constexpr int LOADS = VEC == 1 ? 16 : 8;
        constexpr int IN_FLIGHT = VPT < LOADS ? LOADS / VPT : 1;
        for (int j = 0; j < nrows; j += IN_FLIGHT) {
            Raw u[IN_FLIGHT][VPT];
#pragma unroll
            for (int r = 0; r < IN_FLIGHT; ++r) {
                const int64_t row = __shfl_sync(0xffffffffu, rows, (j + r) & 31);
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    const int c = threadIdx.x + i * blockDim.x;
                    u[r][i] = load_if(slots + row * nvec + c,
                                      c < nvec && j + r < nrows && row >= 0);
                }
            }
#pragma unroll
            for (int r = 0; r < IN_FLIGHT; ++r)
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    float a[VEC];
                    IO::unpack(u[r][i], a);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) v[i][e] += a[e];
                }
        }
        if (p.y_out) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = threadIdx.x + i * blockDim.x;
                if (c < nvec) static_cast<Raw*>(p.y_out)[t * nvec + c] = IO::pack(v[i]);
            }
        }
        normalise<VEC, VPT>(v, p.post, nvec, inv_h, sum);
        const float gt = p.gate_kind == MOE_GATE_TOKEN ? p.scale * p.gate[t] : p.scale;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c >= nvec) continue;
            float a[VEC], g[VEC];
            IO::unpack(res[i], a);
            if (p.gate_kind == MOE_GATE_CHANNEL) {
                load_params<VEC>(p.gate, c, g);
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[i][e] *= g[e];
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[i][e] = a[e] + gt * v[i][e];
            if (p.h_out) static_cast<Raw*>(p.h_out)[t * nvec + c] = IO::pack(v[i]);
        }
        if (p.xn_out) {
            normalise<VEC, VPT>(v, p.next, nvec, inv_h, sum);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                const int c = threadIdx.x + i * blockDim.x;
                if (c < nvec) static_cast<Raw*>(p.xn_out)[t * nvec + c] = IO::pack(v[i]);
            }
        }
    }
}

// Backward of out = scale * gate * N(x) (and of the residual, as `dadd`).  With
// xc = x - m, xhat = xc r, D = scale gate dout:
//   dx = r (wD - [mean(wD)] - xhat mean(wD xhat)) + dadd   ([..]: layer norms)
//   column sums A = sum_t G xhat, B = sum_t G with G = dout (times the token's
//   gate): dw = scale gate A, db = scale gate B, and for a channel gate
//   dgate = scale (w A + b B); for a token gate dgate_t = scale sum_c dout N(x).
// The statistics are taken again from x (the row is in registers anyway), so
// the forward pass has nothing to keep but x.  r factors out of both row sums:
// an RMS norm needs one block-wide reduction per row, a layer norm two.
//
// Bound by memory: x, dout (and dadd) read once, dx written.  Each thread owns
// the same columns in every row of its CTA and keeps their weights and their
// sums A and B in registers; the next row's loads are issued before this row's
// reduction, and two CTAs share an SM so that one's loads and arithmetic fill
// the other's barrier.  PLAIN: an RMS norm (or none) without a bias, which
// needs two row sums instead of four and no B.
// The partial sums of the CTAs are added in CTA order by the second kernel:
// no atomics, the same result every time.  4096 x 4096 bf16 (134 MB), RMS with
// a channel gate: 30 us, 25 of them here (0.83 of the copy bandwidth; issue
// slots 0.73 used).
template <typename T, int VEC, int VPT, int MAXT, bool PLAIN>
__global__ void __launch_bounds__(MAXT, MAXT == 512 && VPT == 1 ? 2 : 1)
    norm_backward_kernel(const NormBackwardParams p) {
    using IO = RowIO<T, VEC>;
    using Raw = typename IO::Raw;
    constexpr int SUMS = PLAIN ? 2 : 4;
    // more columns per thread than registers for their parameters: loaded per row
    constexpr bool KEEP = VPT * VEC <= 8;
    __shared__ float red1[2][1][32];
    __shared__ float red[2][SUMS][32];
    BlockSum<1> sum1{red1};
    BlockSum<SUMS> sum{red};
    const int nvec = p.H / VEC;
    const Raw* X = static_cast<const Raw*>(p.x);
    const Raw* DO = static_cast<const Raw*>(p.dout);
    const Raw* DA = static_cast<const Raw*>(p.dadd);
    const bool has_norm = p.norm.kind != MOE_NORM_NONE;
    const bool layer = !PLAIN && p.norm.kind == MOE_NORM_LAYER;
    const bool token = p.gate_kind == MOE_GATE_TOKEN, channel = p.gate_kind == MOE_GATE_CHANNEL;
    const float inv_h = 1.f / static_cast<float>(p.H);
    pdl_launch_dependents();
    pdl_wait();
    Raw xr[VPT], dr[VPT], ar[VPT];
    auto fetch = [&](int64_t t) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            const bool in = t < p.T && c < nvec;
            xr[i] = load_if(X + t * nvec + c, in);
            dr[i] = load_if(DO + t * nvec + c, in);
            ar[i] = load_if(DA + t * nvec + c, in && DA);
        }
    };
    fetch(blockIdx.x);
    // weight times channel gate of vector c
    auto load_wg = [&](int c, float (&w)[VEC]) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) w[e] = 1.f;
        if (c >= nvec) return;
        if (p.norm.weight) load_params<VEC>(p.norm.weight, c, w);
        if (channel) {
            float g[VEC];
            load_params<VEC>(p.gate, c, g);
#pragma unroll
            for (int e = 0; e < VEC; ++e) w[e] *= g[e];
        }
    };
    float kept[KEEP ? VPT : 1][VEC];
    if (KEEP) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) load_wg(threadIdx.x + i * blockDim.x, kept[i]);
    }
    float A[VPT][VEC], B[PLAIN ? 1 : VPT][VEC];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            A[i][e] = 0.f;
            if (!PLAIN) B[i][e] = 0.f;
        }
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x) {
        float x[VPT][VEC], d[VPT][VEC];
        Raw add[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            IO::unpack(xr[i], x[i]);
            IO::unpack(dr[i], d[i]);
            add[i] = ar[i];
        }
        fetch(t + gridDim.x);
        const float gt = token ? p.gate[t] : 1.f;
        if (layer) {
            float s[1] = {0.f};
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int e = 0; e < VEC; ++e) s[0] += x[i][e];
            sum1(s);
            const float m = s[0] * inv_h;
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    if (static_cast<int>(threadIdx.x + i * blockDim.x) < nvec) x[i][e] -= m;
        }
        // row sums: xc^2, (w gate_c dout) xc, w gate_c dout, b dout
        float s[SUMS];
#pragma unroll
        for (int n = 0; n < SUMS; ++n) s[n] = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c >= nvec) continue;
            float w[VEC];
            if (!KEEP) load_wg(c, w);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float wd = (KEEP ? kept[KEEP ? i : 0][e] : w[e]) * d[i][e];
                s[0] += x[i][e] * x[i][e];
                s[1] += wd * x[i][e];
                if (!PLAIN) s[2] += wd;
            }
            if (!PLAIN && token && p.norm.bias) {
                load_params<VEC>(p.norm.bias, c, w);
#pragma unroll
                for (int e = 0; e < VEC; ++e) s[3] += w[e] * d[i][e];
            }
        }
        if (has_norm || token) sum(s);
        const float r = has_norm ? rsqrtf(s[0] * inv_h + p.norm.eps) : 1.f;
        const float f = p.scale * gt * r;
        const float mean_wd = layer ? s[PLAIN ? 0 : 2] * inv_h : 0.f;
        const float proj = has_norm ? s[1] * inv_h * r * r : 0.f;   // times xc: xhat mean(wD xhat)
        if (token && threadIdx.x == 0 && p.dgate)
            p.dgate[t] = p.scale * (r * s[1] + (PLAIN ? 0.f : s[PLAIN ? 0 : 3]));
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c >= nvec) continue;
            float w[VEC], o[VEC], a[VEC];
            if (!KEEP) load_wg(c, w);
            IO::unpack(add[i], a);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float wd = (KEEP ? kept[KEEP ? i : 0][e] : w[e]) * d[i][e];
                o[e] = f * (wd - mean_wd - proj * x[i][e]) + a[e];
                A[i][e] += gt * r * d[i][e] * x[i][e];
                if (!PLAIN) B[i][e] += gt * d[i][e];
            }
            static_cast<Raw*>(p.dx)[t * nvec + c] = IO::pack(o);
        }
    }
    if (!p.part) return;
    float* pa = p.part + static_cast<int64_t>(blockIdx.x) * 2 * p.H;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c >= nvec) continue;
        if constexpr (VEC % 4 == 0) {
#pragma unroll
            for (int q = 0; q < VEC / 4; ++q) {
                reinterpret_cast<float4*>(pa)[c * (VEC / 4) + q] =
                    make_float4(A[i][4 * q], A[i][4 * q + 1], A[i][4 * q + 2], A[i][4 * q + 3]);
                if constexpr (!PLAIN)
                    reinterpret_cast<float4*>(pa + p.H)[c * (VEC / 4) + q] = make_float4(
                        B[i][4 * q], B[i][4 * q + 1], B[i][4 * q + 2], B[i][4 * q + 3]);
            }
        } else {
            pa[c] = A[i][0];
            if constexpr (!PLAIN) pa[p.H + c] = B[i][0];
        }
    }
}

// The parameters' gradients from the CTAs' column sums: 32 columns per CTA,
// 32 warps each adding every 32nd partial row, then the warps in order.
__global__ void __launch_bounds__(1024) norm_params_kernel(const NormBackwardParams p, int parts,
                                                           bool plain) {
    __shared__ float sh[2][32][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x * 32 + lane;
    pdl_launch_dependents();
    pdl_wait();
    float a = 0.f, b = 0.f;
    if (c < p.H) {
#pragma unroll 8
        for (int i = warp; i < parts; i += 32) {
            const float* row = p.part + static_cast<int64_t>(i) * 2 * p.H;
            a += row[c];
            if (!plain) b += row[p.H + c];
        }
    }
    sh[0][warp][lane] = a;
    sh[1][warp][lane] = b;
    __syncthreads();
    if (warp != 0 || c >= p.H) return;
    a = b = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        a += sh[0][i][lane];
        b += sh[1][i][lane];
    }
    const bool channel = p.gate_kind == MOE_GATE_CHANNEL;
    const float f = p.scale * (channel ? p.gate[c] : 1.f);
    if (p.dweight) p.dweight[c] = f * a;
    if (p.dbias) p.dbias[c] = f * b;
    if (channel && p.dgate) {
        const float w = p.norm.weight ? p.norm.weight[c] : 1.f;
        const float bias = p.norm.bias ? p.norm.bias[c] : 0.f;
        p.dgate[c] = p.scale * (w * a + bias * b);
    }
}

// CTAs of `kern` that are resident at once on the current device (looked up
// once per device and block size).
template <typename K> int resident_ctas(K kern, int threads, int num_sms, int (&cache)[64][33]) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
    int& per_sm = cache[dev][threads / 32];
    if (per_sm <= 0 &&
        (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, 0) != cudaSuccess ||
         per_sm <= 0))
        per_sm = 1;
    return num_sms * per_sm;
}

int threads_for(int nvec, int vpt) { return (((nvec + vpt - 1) / vpt) + 31) / 32 * 32; }

template <typename T, int VEC, int VPT, int MAXT>
cudaError_t run_combine_norm(const CombineNormParams& p, int num_sms, cudaStream_t st) {
    const int threads = threads_for(p.H / VEC, VPT);
    auto kern = combine_norm_kernel<T, VEC, VPT, MAXT>;
    static int resident[64][33] = {};
    const int64_t cap = p.T <= num_sms ? num_sms : resident_ctas(kern, threads, num_sms, resident);
    return launch_pdl(kern, dim3(static_cast<unsigned>(p.T < cap ? p.T : cap)), dim3(threads), 0,
                      st, p);
}

template <typename T, int VEC, int VPT, int MAXT>
cudaError_t run_norm_backward(const NormBackwardParams& p, int num_sms, cudaStream_t st) {
    const int threads = threads_for(p.H / VEC, VPT);
    // without a bias neither db nor dgate needs the sums B
    const bool plain = p.norm.kind != MOE_NORM_LAYER && !p.norm.bias && !p.dbias;
    auto kern = plain ? norm_backward_kernel<T, VEC, VPT, MAXT, true>
                      : norm_backward_kernel<T, VEC, VPT, MAXT, false>;
    const int grid = norm_backward_parts(p.T, p.H, num_sms);
    cudaError_t e = launch_pdl(kern, dim3(grid), dim3(threads), 0, st, p);
    if (e != cudaSuccess || !p.part) return e;
    return launch_pdl(norm_params_kernel, dim3((p.H + 31) / 32), dim3(1024), 0, st, p, grid, plain);
}

}  // namespace

// Rows of partial column sums, one per CTA of the backward kernel.
int norm_backward_parts(int64_t T, int H, int num_sms) {
    const int64_t cap = static_cast<int64_t>(num_sms) * (H <= 1024 ? 8 : H <= 2048 ? 4 : 2);
    return static_cast<int>(T < cap ? (T > 0 ? T : 1) : cap);
}

// `vec16`: every row pointer 16-byte aligned and H a multiple of the vector.
cudaError_t launch_combine_norm(const CombineNormParams& p, bool bf16, bool vec16, int num_sms,
                                cudaStream_t st) {
    if (bf16) {
        if (p.H <= 4096) return run_combine_norm<__nv_bfloat16, 8, 2, 256>(p, num_sms, st);
        if (p.H <= 8192) return run_combine_norm<__nv_bfloat16, 8, 2, 512>(p, num_sms, st);
        return run_combine_norm<__nv_bfloat16, 8, 4, 1024>(p, num_sms, st);
    }
    if (vec16) {
        if (p.H <= 2048) return run_combine_norm<float, 4, 2, 1024>(p, num_sms, st);
        if (p.H <= 4096) return run_combine_norm<float, 4, 4, 1024>(p, num_sms, st);
        return run_combine_norm<float, 4, 8, 1024>(p, num_sms, st);
    }
    if (p.H <= 4096) return run_combine_norm<float, 1, 4, 1024>(p, num_sms, st);
    return run_combine_norm<float, 1, 32, 1024>(p, num_sms, st);
}

cudaError_t launch_norm_backward(const NormBackwardParams& p, bool bf16, bool vec16, int num_sms,
                                 cudaStream_t st) {
    if (bf16) {
        if (p.H <= 4096) return run_norm_backward<__nv_bfloat16, 8, 1, 512>(p, num_sms, st);
        if (p.H <= 8192) return run_norm_backward<__nv_bfloat16, 8, 1, 1024>(p, num_sms, st);
        return run_norm_backward<__nv_bfloat16, 8, 8, 512>(p, num_sms, st);
    }
    if (vec16) {
        if (p.H <= 2048) return run_norm_backward<float, 4, 1, 512>(p, num_sms, st);
        if (p.H <= 4096) return run_norm_backward<float, 4, 1, 1024>(p, num_sms, st);
        return run_norm_backward<float, 4, 16, 512>(p, num_sms, st);
    }
    if (p.H <= 4096) return run_norm_backward<float, 1, 4, 1024>(p, num_sms, st);
    return run_norm_backward<float, 1, 64, 512>(p, num_sms, st);
}

}  // namespace moe
