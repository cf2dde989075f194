// Grouped GEMMs of the expert FFNs on E4M3 codes with block scales.
//
//   D[m, n] = sum over K-blocks b of 128:  2^ea[m,b] sw[n/128, b] (A_b B_b^T)[m, n]
// where A_b, B_b are the codes of block b.  The tensor cores (tcgen05,
// kind::f8f6f4) multiply one K-block's codes into tensor memory; the epilogue
// warps read that 128-column product back, multiply it by the block's two
// scales and add it to float32 accumulators in registers.  (The scales cannot
// enter the MMA: its block scales are powers of two per 32 values, a
// checkpoint's weight scales are any float32.)  Two product buffers in tensor
// memory, 256 columns each, alternate: the tensor cores fill one while the
// epilogue drains the other.
//
// A tile is 128 rows x 256 MMA columns per CTA.  Eight epilogue warps each own
// 32 rows (their TMEM lanes) and half of the columns, 128 accumulators per
// thread.  GEMM 1 (kSwiGLU): 128 gate and the matching 128 up columns, so one
// tile holds a whole 128-column block of h: the two threads of a row exchange
// their maxima through shared memory and h is rounded to E4M3 in the epilogue,
// never stored wider.  GEMM 2 (kScaled): 256 columns of y, times the routing
// weight.
//
// PAIR: two CTAs of a cluster compute 256 x 256 with cta_group::2, each
// loading its own 128 rows of A and 128 of the 256 B rows; as in the bf16 pair
// kernel, without its folded half tiles.  One CTA alone otherwise (128 x 256),
// which wastes fewer rows on small groups.
#include "fp8.cuh"
#include "gemm_common.cuh"

namespace moe {

namespace fp8g {
constexpr int BM = 128;                    // rows per CTA
constexpr int BN = 256;
constexpr int BK = 128;                    // codes (bytes) per K-block
constexpr int UMMA_K = 32;
constexpr int TILE_BYTES = 128 * BK;       // 128 rows of A or of B: 16 KB
constexpr int TMEM_COLS = 512;
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 64 + EPI_WARPS * 32;
template <bool PAIR> struct Cfg {
    static constexpr int B_TILES = PAIR ? 1 : 2;              // of 128 rows each, per CTA
    static constexpr int STAGE_BYTES = TILE_BYTES * (1 + B_TILES);
    static constexpr int STAGES = PAIR ? 6 : 4;               // 192 KB
    static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + 1024 + 256;
};
}  // namespace fp8g

struct Fp8GemmParams {
    GemmParams g;
    const uint8_t* sa_routed;     // E8M0 scales of the A rows
    const uint8_t* sa_shared;
    const float* sw_routed;       // weight scales
    const float* sw_shared;
    uint8_t* hs_routed;           // kSwiGLU: E8M0 scales of h
    uint8_t* hs_shared;
};

__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate));
}
__device__ __forceinline__ void umma_e4m3_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                               uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate));
}

// Instruction descriptor, kind::f8f6f4: E4M3 A and B (format 0, K-major), fp32 D.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
    return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(M >> 4) << 24);
}

// Barrier of the 256 epilogue threads.
__device__ __forceinline__ void epilogue_sync() {
    asm volatile("bar.sync 1, 256;" ::: "memory");
}

template <int EPI, bool PAIR, int MAXG>
__global__ void __launch_bounds__(fp8g::THREADS, 1) grouped_gemm_fp8(
    const __grid_constant__ CUtensorMap map_a_routed,
    const __grid_constant__ CUtensorMap map_a_shared,
    const __grid_constant__ CUtensorMap map_b_routed,
    const __grid_constant__ CUtensorMap map_b_shared, const Fp8GemmParams fp) {
    using namespace fp8g;
    using C = Cfg<PAIR>;
    constexpr int STAGES = C::STAGES, STAGE_BYTES = C::STAGE_BYTES;
    constexpr int TILE_M = PAIR ? 2 * BM : BM;
    constexpr int n_cols_per_tile = (EPI == kSwiGLU) ? BN / 2 : BN;
    const GemmParams& p = fp.g;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ GroupTableT<MAXG> gt;
    __shared__ uint32_t tmem_base_sh;
    __shared__ uint32_t mag_sh[2][2][BM];       // [tile parity][column half][row]

    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * STAGE_BYTES);
    uint64_t* full = bars;                 // [STAGES] even CTA: TMA bytes (of both CTAs)
    uint64_t* empty = bars + STAGES;       // [STAGES] stage consumed
    uint64_t* tfull = bars + 2 * STAGES;   // [2]      K-block product ready
    uint64_t* tempty = tfull + 2;          // [2]      even CTA: product read by every epilogue warp
    uint64_t* drain = tempty + 2;          // [1]      all MMAs complete

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
    const int worker = PAIR ? static_cast<int>(cluster_id_x()) : static_cast<int>(blockIdx.x);
    const int workers = PAIR ? static_cast<int>(n_clusters_x()) : static_cast<int>(gridDim.x);
    const uint64_t deadline = global_ns() + p.timeout_ns;

    pdl_launch_dependents();
    pdl_wait();
    stage_offsets(gt.tile_start, p.offsets, p.E);
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], (PAIR ? 2 : 1) * EPI_WARPS);
        }
        mbar_init(drain, 1);
        fence_barrier_init();
        build_group_table(gt, p.E, p.S, p.T, TILE_M, p.n_tiles_routed, p.n_tiles_shared);
        tma_prefetch_desc(&map_a_routed);
        tma_prefetch_desc(&map_b_routed);
        if (p.S > 0) {
            tma_prefetch_desc(&map_a_shared);
            tma_prefetch_desc(&map_b_shared);
        }
    }
    if (warp == 1) {
        if (PAIR) {
            tmem_alloc_pair(&tmem_base_sh, TMEM_COLS);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(&tmem_base_sh, TMEM_COLS);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();    // both CTAs' barriers initialised before any remote use
    tc_fence_after();
    const uint32_t tmem_base = tmem_base_sh;
    const int total = gt.total_tiles;

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            const uint64_t pol_a = l2_policy_evict_last();
            const uint64_t pol_b = l2_policy_evict_normal();
            const uint32_t full_leader =
                PAIR ? mapa_shared(smem_u32(full), 0) : smem_u32(full);
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int tile = worker; tile < total && ok; tile += workers) {
                const TileCoord c = decode_tile(gt, p, tile, n_cols_per_tile, TILE_M);
                const CUtensorMap* ma = c.routed ? &map_a_routed : &map_a_shared;
                const CUtensorMap* mb = c.routed ? &map_b_routed : &map_b_shared;
                const int K = c.routed ? p.K_routed : p.K_shared;
                const int eidx = c.routed ? c.g : c.g - p.E;
                // routed -> sorted slot rows; shared GEMM 1 -> token rows; shared
                // GEMM 2 -> that expert's block of h
                const int a_row =
                    (EPI == kSwiGLU && !c.routed ? 0 : gt.row0[c.g]) + c.m0 + rank * BM;
                const int b_row = eidx * (c.routed ? p.b_rows_routed : p.b_rows_shared) + c.n0;
                const int second = EPI == kSwiGLU ? (c.routed ? p.half_routed : p.half_shared)
                                                  : BN / 2;
                const int num_kb = (K + BK - 1) / BK;
                for (int kb = 0; kb < num_kb; ++kb) {
                    if (!mbar_wait(&empty[stage], phase ^ 1u, deadline)) { ok = false; break; }
                    uint8_t* sa = smem + stage * STAGE_BYTES;
                    if (rank == 0)
                        mbar_arrive_expect_tx(&full[stage], (PAIR ? 2 : 1) * STAGE_BYTES);
                    const uint32_t bar = full_leader + stage * 8;
                    if (PAIR) {
                        tma_load_2d_pair_hint(sa, ma, bar, kb * BK, a_row, pol_a);
                        tma_load_2d_pair_hint(sa + TILE_BYTES, mb, bar, kb * BK,
                                              b_row + rank * second, pol_b);
                    } else {
                        tma_load_2d(sa, ma, &full[stage], kb * BK, a_row);
                        tma_load_2d(sa + TILE_BYTES, mb, &full[stage], kb * BK, b_row);
                        tma_load_2d(sa + 2 * TILE_BYTES, mb, &full[stage], kb * BK,
                                    b_row + second);
                    }
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
            }
            if (!ok) raise_error(p.err_flag, MOE_ERR_TIMEOUT);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA (even CTA)
        if (lane == 0 && rank == 0) {
            constexpr uint32_t idesc = idesc_e4m3_f32(TILE_M, BN);
            int stage = 0, buf = 0;
            uint32_t phase = 0, buf_phase = 0;
            bool ok = true;
            for (int tile = worker; tile < total && ok; tile += workers) {
                const TileCoord c = decode_tile(gt, p, tile, n_cols_per_tile, TILE_M);
                const int num_kb = ((c.routed ? p.K_routed : p.K_shared) + BK - 1) / BK;
                for (int kb = 0; kb < num_kb; ++kb) {
                    if (!mbar_wait(&tempty[buf], buf_phase ^ 1u, deadline) ||
                        !mbar_wait(&full[stage], phase, deadline)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d = tmem_base + static_cast<uint32_t>(buf * BN);
                    const uint32_t sa = smem_u32(smem + stage * STAGE_BYTES);
                    const uint32_t sb = sa + TILE_BYTES;
#pragma unroll
                    for (int kk = 0; kk < BK / UMMA_K; ++kk) {
                        const uint64_t da = smem_desc_sw128(sa + kk * UMMA_K);
                        const uint64_t db = smem_desc_sw128(sb + kk * UMMA_K);
                        if (PAIR) umma_e4m3_pair(d, da, db, idesc, kk != 0 ? 1u : 0u);
                        else umma_e4m3(d, da, db, idesc, kk != 0 ? 1u : 0u);
                    }
                    if (PAIR) {
                        umma_commit_pair(&empty[stage], 0x3);
                        umma_commit_pair(&tfull[buf], 0x3);
                    } else {
                        umma_commit(&empty[stage]);
                        umma_commit(&tfull[buf]);
                    }
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                    if (++buf == 2) { buf = 0; buf_phase ^= 1u; }
                }
            }
            if (!ok) raise_error(p.err_flag, MOE_ERR_TIMEOUT);
            // every issued MMA completes before the tensor memory is released
            if (PAIR) umma_commit_pair(drain, 0x1);
            else umma_commit(drain);
            if (!mbar_wait(drain, 0, deadline + 1000000000ull))
                raise_error(p.err_flag, MOE_ERR_TIMEOUT);
        }
    } else {
        // ------------------------------------------------------------ epilogue
        const int quarter = warp & 3;               // TMEM lane quarter of this warp
        const int half = (warp - 2) >> 2;           // column half
        const int row = quarter * 32 + lane;
        const uint32_t tempty_leader =
            PAIR ? mapa_shared(smem_u32(tempty), 0) : smem_u32(tempty);
        // first TMEM column of this thread's two runs of 64
        const int col0 = EPI == kSwiGLU ? 64 * half : 128 * half;
        const int col1 = EPI == kSwiGLU ? 128 + 64 * half : 128 * half + 64;
        int buf = 0, parity = 0;
        uint32_t buf_phase = 0;
        // after a wait that ran out, the loops still run to their end (the
        // epilogue barrier needs every warp) without waiting or storing
        bool ok = true;
        for (int tile = worker; tile < total; tile += workers) {
            const TileCoord c = decode_tile(gt, p, tile, n_cols_per_tile, TILE_M);
            const int K = c.routed ? p.K_routed : p.K_shared;
            const int N = c.routed ? p.N_routed : p.N_shared;
            const int num_kb = (K + BK - 1) / BK;
            const int eidx = c.routed ? c.g : c.g - p.E;
            const int m = c.m0 + rank * BM + row;
            const bool valid = m < c.rows;
            const bool any = m - lane < c.rows;      // of this warp's rows
            const int64_t a_row =
                (EPI == kSwiGLU && !c.routed ? 0 : static_cast<int64_t>(gt.row0[c.g])) +
                (valid ? m : c.rows - 1);
            const uint32_t* sa = reinterpret_cast<const uint32_t*>(
                (c.routed ? fp.sa_routed : fp.sa_shared) + a_row * fp8_scale_ld(K));
            // weight scales of the two runs: gate and up, or the same 128 columns
            const int row_blocks = (N + 127) / 128;
            const float* sw = c.routed ? fp.sw_routed : fp.sw_shared;
            const float *sw0, *sw1;
            if (EPI == kSwiGLU) {
                sw0 = sw + (static_cast<int64_t>(eidx) * 2 * row_blocks + c.n0 / 128) * num_kb;
                sw1 = sw0 + static_cast<int64_t>(row_blocks) * num_kb;
            } else {
                const int rb = min(c.n0 / 128 + half, row_blocks - 1);
                sw0 = sw + (static_cast<int64_t>(eidx) * row_blocks + rb) * num_kb;
                sw1 = sw0;
            }
            float acc0[64], acc1[64];
#pragma unroll
            for (int j = 0; j < 64; ++j) acc0[j] = acc1[j] = 0.f;
            uint32_t bytes = 0;
#pragma unroll 1
            for (int kb = 0; kb < num_kb; ++kb) {
                if ((kb & 3) == 0) bytes = sa[kb >> 2];
                const float ea = e8m0_value(bytes & 0xffu);
                bytes >>= 8;
                const float s0 = ea * sw0[kb];
                const float s1 = EPI == kSwiGLU ? ea * sw1[kb] : s0;
                if (ok && !mbar_wait(&tfull[buf], buf_phase, deadline)) {
                    raise_error(p.err_flag, MOE_ERR_TIMEOUT);
                    ok = false;
                }
                ok = __all_sync(0xffffffffu, ok);    // the loads below are the warp's
                tc_fence_after();
                if (any && ok) {
                    const uint32_t t = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                                       static_cast<uint32_t>(buf * BN);
#pragma unroll
                    for (int cc = 0; cc < 64; cc += 32) {
                        float v[32];
                        tmem_ld32(t + col0 + cc, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 32; ++j) acc0[cc + j] = fmaf(s0, v[j], acc0[cc + j]);
                    }
#pragma unroll
                    for (int cc = 0; cc < 64; cc += 32) {
                        float v[32];
                        tmem_ld32(t + col1 + cc, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int j = 0; j < 32; ++j) acc1[cc + j] = fmaf(s1, v[j], acc1[cc + j]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (PAIR) mbar_arrive_cluster(tempty_leader + buf * 8);
                    else mbar_arrive(&tempty[buf]);
                }
                if (++buf == 2) { buf = 0; buf_phase ^= 1u; }
            }
            if (EPI == kSwiGLU) {
                // h = silu(g) u, rounded to E4M3 with the scale of its 128 columns
                const int n = c.n0 + 64 * half;
                uint32_t mag = 0;
#pragma unroll
                for (int j = 0; j < 64; ++j) {
                    const float g = acc0[j];
                    const float h = __fdividef(g, 1.f + __expf(-g)) * acc1[j];
                    acc0[j] = nan_if_not_finite(n + j < N ? h : 0.f);
                    mag = max(mag, finite_mag(acc0[j]));
                }
                mag_sh[parity][half][row] = mag;
                epilogue_sync();
                mag = max(mag, mag_sh[parity][half ^ 1][row]);
                parity ^= 1;
                const uint32_t byte = e8m0_of(mag);
                const float inv = e8m0_inverse(byte);
                if (valid && ok) {
                    const int64_t orow = static_cast<int64_t>(gt.row0[c.g]) + m;
                    uint8_t* out = static_cast<uint8_t*>(c.routed ? p.out_routed : p.out_shared) +
                                   orow * N + n;
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        uint32_t o[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int j = 16 * v + 4 * e;
                            o[e] = e4m3x4(acc0[j] * inv, acc0[j + 1] * inv, acc0[j + 2] * inv,
                                          acc0[j + 3] * inv);
                        }
                        if (n + 16 * v < N)
                            *reinterpret_cast<uint4*>(out + 16 * v) =
                                make_uint4(o[0], o[1], o[2], o[3]);
                    }
                    if (half == 0)
                        (c.routed ? fp.hs_routed
                                  : fp.hs_shared)[orow * fp8_scale_ld(N) + c.n0 / 128] =
                            static_cast<uint8_t>(byte);
                }
            } else if (valid && ok) {
                float scale = 1.f;
                int64_t orow = static_cast<int64_t>(gt.row0[c.g]) + m;
                if (c.routed) {
                    const int64_t slot = p.perm[orow];
                    scale = slot >= 0 && slot < p.T * p.k ? p.routed_scale * p.topk_w[slot] : 0.f;
                } else {
                    orow += p.out_row0_shared;
                }
                const int n = c.n0 + 128 * half;
                __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out_routed) + orow * N + n;
#pragma unroll
                for (int v = 0; v < 16; ++v) {
                    uint32_t o[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = 8 * (v & 7) + 2 * e;
                        o[e] = v < 8 ? pack_bf16x2(scale * acc0[j], scale * acc0[j + 1])
                                     : pack_bf16x2(scale * acc1[j], scale * acc1[j + 1]);
                    }
                    if (n + 8 * v < N)
                        *reinterpret_cast<uint4*>(out + 8 * v) = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        if (PAIR) tmem_dealloc_pair(tmem_base, TMEM_COLS);
        else tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

namespace {

// Codes [rows, cols], box of 128 columns x 128 rows, 128-byte swizzle.
bool make_map_codes(CUtensorMap* map, const void* base, int64_t rows, int64_t cols) {
    EncodeTiledFn enc = get_encode_fn();
    if (!enc || rows <= 0 || cols <= 0) return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols)};
    cuuint32_t box[2] = {fp8g::BK, 128u};
    cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

template <int EPI, bool PAIR>
cudaError_t launch_gemm(const Fp8GemmParams& p, int64_t rows_routed, int num_sms,
                        const CUtensorMap& ar, const CUtensorMap& as, const CUtensorMap& br,
                        const CUtensorMap& bs, cudaStream_t st) {
    using C = fp8g::Cfg<PAIR>;
    constexpr int ctas = PAIR ? 2 : 1;
    constexpr int tile_m = ctas * fp8g::BM;
    const GemmParams& g = p.g;
    // at most this many tiles: every group may end in a partial m-tile
    const int64_t tiles = (ceil_div(rows_routed, tile_m) + (g.E < rows_routed ? g.E : rows_routed)) *
                              g.n_tiles_routed +
                          g.S * ceil_div(g.T, tile_m) * g.n_tiles_shared;
    const int64_t workers = num_sms / ctas < tiles ? num_sms / ctas : tiles;
    auto kern = grouped_gemm_fp8<EPI, PAIR, kMaxGroups>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(workers * ctas), 1, 1);
    cfg.blockDim = dim3(fp8g::THREADS, 1, 1);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = PAIR ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, ar, as, br, bs, p);
}

template <bool PAIR>
cudaError_t run_ffn(const moe_shape& s, const Fp8Operands& o, int num_sms, cudaStream_t st) {
    const int64_t Tk = s.T * s.k;
    const int S = s.n_shared, Is = S > 0 ? s.I_shared : s.I;
    CUtensorMap a1r, a1s, b1r, b1s, a2r, a2s, b2r, b2s;
    bool ok = make_map_codes(&a1r, o.xq, Tk, s.H);
    ok &= make_map_codes(&b1r, o.gate_up, static_cast<int64_t>(s.E) * 2 * s.I, s.H);
    ok &= make_map_codes(&a2r, o.hq, Tk, s.I);
    ok &= make_map_codes(&b2r, o.down, static_cast<int64_t>(s.E) * s.H, s.I);
    if (S > 0) {
        ok &= make_map_codes(&a1s, o.xq + Tk * s.H, s.T, s.H);
        ok &= make_map_codes(&b1s, o.sh_gate_up, static_cast<int64_t>(S) * 2 * Is, s.H);
        ok &= make_map_codes(&a2s, o.hq_sh, S * s.T, Is);
        ok &= make_map_codes(&b2s, o.sh_down, static_cast<int64_t>(S) * s.H, Is);
    } else {
        a1s = a1r; b1s = b1r; a2s = a2r; b2s = b2r;
    }
    if (!ok) return cudaErrorInvalidValue;

    Fp8GemmParams p{};
    GemmParams& g = p.g;
    g.offsets = o.offsets;
    g.perm = o.perm;
    g.topk_w = o.topk_w;
    g.T = s.T;
    g.E = s.E;
    g.S = S;
    g.k = s.k;
    g.routed_scale = s.routed_scale;
    g.group_m = PAIR ? 16 : 8;
    g.err_flag = o.err_flag;
    g.timeout_ns = 4000000000ull;

    // GEMM 1: h = silu(x Wg^T) * (x Wu^T), rounded to E4M3
    g.n_tiles_routed = static_cast<int>(ceil_div(s.I, fp8g::BN / 2));
    g.n_tiles_shared = static_cast<int>(ceil_div(Is, fp8g::BN / 2));
    g.K_routed = g.K_shared = s.H;
    g.N_routed = s.I;
    g.N_shared = Is;
    g.b_rows_routed = 2 * s.I;
    g.b_rows_shared = 2 * Is;
    g.half_routed = s.I;
    g.half_shared = Is;
    g.out_routed = o.hq;
    g.out_shared = o.hq_sh;
    p.sa_routed = o.xs;
    p.sa_shared = o.xs + Tk * fp8_scale_ld(s.H);
    p.sw_routed = o.gate_up_s;
    p.sw_shared = o.sh_gate_up_s;
    p.hs_routed = o.hs;
    p.hs_shared = o.hs_sh;
    cudaError_t e = launch_gemm<kSwiGLU, PAIR>(p, Tk, num_sms, a1r, a1s, b1r, b1s, st);
    if (e != cudaSuccess) return e;

    // GEMM 2: the slots' rows of y
    g.n_tiles_routed = g.n_tiles_shared = static_cast<int>(ceil_div(s.H, fp8g::BN));
    g.K_routed = s.I;
    g.K_shared = Is;
    g.N_routed = g.N_shared = s.H;
    g.b_rows_routed = g.b_rows_shared = s.H;
    g.out_routed = o.y_slots;
    g.out_row0_shared = Tk;
    p.sa_routed = o.hs;
    p.sa_shared = o.hs_sh;
    p.sw_routed = o.down_s;
    p.sw_shared = o.sh_down_s;
    return launch_gemm<kScaled, PAIR>(p, Tk, num_sms, a2r, a2s, b2r, b2s, st);
}

}  // namespace

// The experts on the quantised rows o.xq / o.xs.
cudaError_t launch_ffn_fp8(const moe_shape& s, const Fp8Operands& o, int num_sms,
                           cudaStream_t st) {
    constexpr int kPairMinRows = 256;    // average rows per expert for CTA pairs
    if (s.T * s.k >= static_cast<int64_t>(kPairMinRows) * s.E)
        return run_ffn<true>(s, o, num_sms, st);
    return run_ffn<false>(s, o, num_sms, st);
}

}  // namespace moe
