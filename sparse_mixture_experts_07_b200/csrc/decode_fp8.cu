// Expert FFNs on E4M3 codes for decode batches (T <= 8, so at most 8 rows per
// group): every active expert's codes are read once, front to back.
//
// As in the bf16 decode kernels, a CTA's 4 warps split the contraction of a
// unit of 16 weight rows and sum their fragments in shared memory; the
// products run on mma.sync m16n8k32 (E4M3, fp32 accumulate), weight rows being
// the 16 M rows and the group's token rows the 8 N columns, with the
// contraction permuted alike on both sides so that every load is 16 contiguous
// bytes: lane (g = lane/4, q = lane%4) holds columns [64 h + 16 q, + 16) of
// weight rows g and g+8 and of token row g.  A K-block of 128 is four MMAs;
// their sum times the block's two scales is added in float32.
//
//   decode_gate_up: unit = (group, 16 columns of h).  h is written in float32;
//     the last of the (up to 8) units of a 128-column block to arrive rounds
//     the block's rows to E4M3 (which unit that is changes nothing in the
//     result).
//   decode_down: unit = (group, 16 columns of y).
//
// Bound by memory: the active experts' codes.  A warp keeps two (gate_up) or
// four (down) K-blocks of its rows in flight, 8 KB.
#include "fp8.cuh"

namespace moe {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;

struct DecodeFp8Params {
    Fp8Operands o;
    int64_t T;
    int H, I, E, k, S, Is, h_blocks;
    float routed_scale;
};

// The groups that have rows: routed experts (ascending), then shared experts.
struct Active {
    int n;                       // routed experts with rows
    int gid[kMaxExperts];
};

// Built by warp 0, 32 experts at a time.
__device__ __forceinline__ void build_active_experts(Active& a, const int32_t* offsets, int E) {
    const int lane = threadIdx.x & 31;
    int n = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
        const int e = e0 + lane;
        const bool has = e < E && offsets[e + 1] > offsets[e];
        const uint32_t mask = __ballot_sync(0xffffffffu, has);
        if (has) a.gid[n + __popc(mask & ((1u << lane) - 1))] = e;
        n += __popc(mask);
    }
    if (lane == 0) a.n = n;
}

// Unit -> group and first row of 16; routed groups have ur units, shared us.
struct Unit {
    int g, i0, rows;
    bool routed;
    int64_t row0;                // first row of the group in h, and of y's slots
};
__device__ __forceinline__ Unit find_unit(const Active& a, const DecodeFp8Params& p, int unit,
                                          int ur, int us) {
    Unit u;
    const int routed_units = a.n * ur;
    u.routed = unit < routed_units;
    if (u.routed) {
        const int ai = unit / ur;
        u.g = a.gid[ai];
        u.i0 = (unit - ai * ur) * 16;
        u.row0 = p.o.offsets[u.g];
        u.rows = p.o.offsets[u.g + 1] - static_cast<int>(u.row0);
    } else {
        const int s = (unit - routed_units) / us;
        u.g = s;
        u.i0 = (unit - routed_units - s * us) * 16;
        u.row0 = static_cast<int64_t>(s) * p.T;
        u.rows = static_cast<int>(p.T);
    }
    return u;
}

// A predicated 16-byte load (zero when !ok), volatile so that all loads of an
// unrolled step stay ahead of the products.
__device__ __forceinline__ uint4 ld16(const uint8_t* p, bool ok) {
    uint4 v;
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@q ld.global.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
        : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
        : "l"(p), "r"(static_cast<int>(ok)));
    return v;
}
// Same, for weights that are read once: do not allocate them in L1.
__device__ __forceinline__ uint4 ld16_stream(const uint8_t* p, bool ok) {
    uint4 v;
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@q ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
        : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
        : "l"(p), "r"(static_cast<int>(ok)));
    return v;
}

__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// c += W[rows g, g+8] . X[row g]^T over 64 columns.
__device__ __forceinline__ void mma_step(float (&c)[4], const uint4& wa, const uint4& wb,
                                         const uint4& xv) {
    mma_e4m3(c, wa.x, wb.x, wa.y, wb.y, xv.x, xv.y);
    mma_e4m3(c, wa.z, wb.z, wa.w, wb.w, xv.z, xv.w);
}

// Adds NF floats per lane over the CTA's warps; the sum is in warp 0.
template <int NF>
__device__ __forceinline__ bool sum_over_warps(float (&v)[NF], float* red) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();             // the last use of red
#pragma unroll
    for (int j = 0; j < NF; ++j) red[(warp * NF + j) * 32 + lane] = v[j];
    __syncthreads();
    if (warp != 0) return false;
#pragma unroll
    for (int j = 0; j < NF; ++j) {
        v[j] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v[j] += red[(w * NF + j) * 32 + lane];
    }
    return true;
}

// Accumulates M sets of 16 weight rows (M = 2: gate and up) against the
// group's token rows over K-blocks [b0, b1), UNROLL blocks in flight.
template <int M, int UNROLL>
__device__ __forceinline__ void stream_rows(float (&acc)[M][4], const uint8_t* const (&w)[M],
                                            const float* const (&sw)[M], const uint8_t* x,
                                            const uint8_t* xs, int xs_ld, int rows, int K, int b0,
                                            int b1, bool r0_ok, bool r1_ok) {
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const bool tok_ok = g < rows;
    // scales of this lane's two token columns
    const uint8_t* xs0 = xs + static_cast<int64_t>(min(2 * q, rows - 1)) * xs_ld;
    const uint8_t* xs1 = xs + static_cast<int64_t>(min(2 * q + 1, rows - 1)) * xs_ld;
    const uint8_t* xrow = x + static_cast<int64_t>(tok_ok ? g : 0) * K;
    for (int b = b0; b < b1; b += UNROLL) {
        uint4 wa[UNROLL][M][2], wb[UNROLL][M][2], xv[UNROLL][2];
        float s[UNROLL][M], e0[UNROLL], e1[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int col = (b + u) * 128 + 64 * h + 16 * q;
                const bool in = b + u < b1 && col < K;
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    wa[u][m][h] = ld16_stream(w[m] + col, in && r0_ok);
                    wb[u][m][h] = ld16_stream(w[m] + static_cast<int64_t>(8) * K + col,
                                              in && r1_ok);
                }
                xv[u][h] = ld16(xrow + col, in && tok_ok);
            }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const bool in = b + u < b1;
#pragma unroll
            for (int m = 0; m < M; ++m) s[u][m] = in ? __ldg(sw[m] + b + u) : 0.f;
            e0[u] = in ? e8m0_value(xs0[b + u]) : 0.f;
            e1[u] = in ? e8m0_value(xs1[b + u]) : 0.f;
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u)
#pragma unroll
            for (int m = 0; m < M; ++m) {
                float c[4] = {0.f, 0.f, 0.f, 0.f};
                mma_step(c, wa[u][m][0], wb[u][m][0], xv[u][0]);
                mma_step(c, wa[u][m][1], wb[u][m][1], xv[u][1]);
                const float f0 = s[u][m] * e0[u], f1 = s[u][m] * e1[u];
                acc[m][0] = fmaf(f0, c[0], acc[m][0]);
                acc[m][1] = fmaf(f1, c[1], acc[m][1]);
                acc[m][2] = fmaf(f0, c[2], acc[m][2]);
                acc[m][3] = fmaf(f1, c[3], acc[m][3]);
            }
    }
}

// K-blocks of warp w.
__device__ __forceinline__ void split_blocks(int blocks, int w, int& b0, int& b1) {
    b0 = blocks * w / kWarps;
    b1 = blocks * (w + 1) / kWarps;
}

__global__ void __launch_bounds__(kThreads) fp8_decode_gate_up_kernel(const DecodeFp8Params p) {
    __shared__ Active act;
    __shared__ float red[kWarps * 8 * 32];
    __shared__ int last_sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    pdl_launch_dependents();
    pdl_wait();
    if (warp == 0) build_active_experts(act, p.o.offsets, p.E);
    __syncthreads();
    const int ur = (p.I + 15) / 16, us = (p.Is + 15) / 16;
    const int total = act.n * ur + p.S * us;
    const int kb = (p.H + 127) / 128, xs_ld = fp8_scale_ld(p.H);
    int b0, b1;
    split_blocks(kb, warp, b0, b1);
    for (int unit = blockIdx.x; unit < total; unit += gridDim.x) {
        const Unit u = find_unit(act, p, unit, ur, us);
        const int N = u.routed ? p.I : p.Is;
        const int nb = (N + 127) / 128;
        const int64_t e = u.g;
        const uint8_t* W = (u.routed ? p.o.gate_up : p.o.sh_gate_up) + e * 2 * N * p.H;
        const float* sw = (u.routed ? p.o.gate_up_s : p.o.sh_gate_up_s) + e * 2 * nb * kb;
        // token rows: the group's sorted slots, or (shared) the tokens behind them
        const int64_t xrow0 = u.routed ? u.row0 : p.T * p.k;
        const uint8_t* w0 = W + static_cast<int64_t>(u.i0 + g) * p.H;
        const uint8_t* const w[2] = {w0, w0 + static_cast<int64_t>(N) * p.H};
        const float* s0 = sw + static_cast<int64_t>(u.i0 / 128) * kb;
        const float* const s[2] = {s0, s0 + static_cast<int64_t>(nb) * kb};
        float acc[2][4] = {};
        stream_rows<2, 2>(acc, w, s, p.o.xq + xrow0 * p.H, p.o.xs + xrow0 * xs_ld, xs_ld, u.rows,
                          p.H, b0, b1, u.i0 + g < N, u.i0 + g + 8 < N);
        float c[8] = {acc[0][0], acc[0][1], acc[0][2], acc[0][3],
                      acc[1][0], acc[1][1], acc[1][2], acc[1][3]};
        float* h32 = p.o.h32 + (u.routed ? 0 : p.T * p.k * p.I);
        if (sum_over_warps<8>(c, red)) {
            // c[0], c[1]: weight row g, tokens 2q, 2q+1; c[2], c[3]: row g+8 (gate; up at +4)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = j < 2 ? g : g + 8, t = 2 * q + (j & 1);
                if (t < u.rows && u.i0 + r < N)
                    h32[(u.row0 + t) * N + u.i0 + r] = c[j] / (1.f + __expf(-c[j])) * c[4 + j];
            }
            __threadfence();
            __syncwarp();
            if (lane == 0) {
                const int block = u.i0 / 128;
                const int units = min(8, (N - block * 128 + 15) / 16);
                const int grp = u.routed ? u.g : p.E + u.g;
                const int before = atomicAdd(p.o.arrived + grp * p.h_blocks + block, 1);
                last_sh = before == units - 1;
                __threadfence();
            }
        }
        __syncthreads();
        if (!last_sh) continue;
        // 16 threads per row; every 32 lanes reach the shuffles
        const int t = threadIdx.x >> 4, col = u.i0 / 128 * 128 + (threadIdx.x & 15) * 8;
        const bool in = t < u.rows && col < N;
        float v[8];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const float4 f = in ? __ldcg(reinterpret_cast<const float4*>(
                                             h32 + (u.row0 + t) * N + col + 4 * half))
                                : make_float4(0.f, 0.f, 0.f, 0.f);
            v[4 * half] = f.x; v[4 * half + 1] = f.y;
            v[4 * half + 2] = f.z; v[4 * half + 3] = f.w;
        }
        uint32_t byte;
        const uint2 codes = e4m3_block_piece(v, byte);
        if (in) {
            *reinterpret_cast<uint2*>((u.routed ? p.o.hq : p.o.hq_sh) + (u.row0 + t) * N + col) =
                codes;
            if ((threadIdx.x & 15) == 0)
                (u.routed ? p.o.hs : p.o.hs_sh)[(u.row0 + t) * fp8_scale_ld(N) + col / 128] =
                    static_cast<uint8_t>(byte);
        }
    }
}

__global__ void __launch_bounds__(kThreads) fp8_decode_down_kernel(const DecodeFp8Params p) {
    __shared__ Active act;
    __shared__ float red[kWarps * 4 * 32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    pdl_launch_dependents();
    pdl_wait();
    if (warp == 0) build_active_experts(act, p.o.offsets, p.E);
    __syncthreads();
    const int units = (p.H + 15) / 16, nb = (p.H + 127) / 128;
    const int total = (act.n + p.S) * units;
    const int64_t slots = p.T * p.k;
    for (int unit = blockIdx.x; unit < total; unit += gridDim.x) {
        const Unit u = find_unit(act, p, unit, units, units);
        const int K = u.routed ? p.I : p.Is;
        const int kb = (K + 127) / 128, hs_ld = fp8_scale_ld(K);
        const int64_t e = u.g;
        const uint8_t* const w[1] = {(u.routed ? p.o.down : p.o.sh_down) +
                                     (e * p.H + u.i0 + g) * K};
        const float* const s[1] = {(u.routed ? p.o.down_s : p.o.sh_down_s) +
                                   (e * nb + u.i0 / 128) * kb};
        int b0, b1;
        split_blocks(kb, warp, b0, b1);
        float acc[1][4] = {};
        stream_rows<1, 4>(acc, w, s, (u.routed ? p.o.hq : p.o.hq_sh) + u.row0 * K,
                          (u.routed ? p.o.hs : p.o.hs_sh) + u.row0 * hs_ld, hs_ld, u.rows, K, b0,
                          b1, u.i0 + g < p.H, u.i0 + g + 8 < p.H);
        if (!sum_over_warps<4>(acc[0], red)) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = j < 2 ? g : g + 8, t = 2 * q + (j & 1);
            if (t >= u.rows || u.i0 + r >= p.H) continue;
            int64_t orow = u.row0 + t;
            float scale = 1.f;
            if (u.routed) {
                // a plan with skipped slots (bad expert index) leaves holes
                const int64_t slot = p.o.perm[orow];
                scale = slot >= 0 && slot < slots ? p.routed_scale * p.o.topk_w[slot] : 0.f;
            } else {
                orow += slots;
            }
            static_cast<__nv_bfloat16*>(p.o.y_slots)[orow * p.H + u.i0 + r] =
                __float2bfloat16_rn(scale * acc[0][j]);
        }
    }
}

template <typename K> int resident(K kern, int num_sms) {
    int per_sm = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kThreads, 0) != cudaSuccess ||
        per_sm <= 0)
        per_sm = 1;
    return num_sms * per_sm;
}

}  // namespace

// The experts on the quantised rows o.xq / o.xs, T <= 8.
cudaError_t launch_ffn_fp8_decode(const moe_shape& s, const Fp8Operands& o, int num_sms,
                                  cudaStream_t st) {
    if (!fp8_is_decode(s)) return cudaErrorInvalidValue;
    DecodeFp8Params p{};
    p.o = o;
    p.T = s.T;
    p.H = s.H;
    p.I = s.I;
    p.E = s.E;
    p.k = s.k;
    p.S = s.n_shared;
    p.Is = s.n_shared > 0 ? s.I_shared : 0;
    p.h_blocks = fp8_h_blocks(s);
    p.routed_scale = s.routed_scale;
    const int64_t active = s.T * s.k < s.E ? s.T * s.k : s.E;
    int64_t units = active * ((s.I + 15) / 16) + static_cast<int64_t>(p.S) * ((p.Is + 15) / 16);
    int64_t cap = resident(fp8_decode_gate_up_kernel, num_sms);
    cudaError_t e = launch_pdl(fp8_decode_gate_up_kernel,
                               dim3(static_cast<unsigned>(units < cap ? units : cap)),
                               dim3(kThreads), 0, st, p);
    if (e != cudaSuccess) return e;
    units = (active + p.S) * ((s.H + 15) / 16);
    cap = resident(fp8_decode_down_kernel, num_sms);
    return launch_pdl(fp8_decode_down_kernel,
                      dim3(static_cast<unsigned>(units < cap ? units : cap)), dim3(kThreads), 0,
                      st, p);
}

}  // namespace moe
