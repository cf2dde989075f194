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
// A tile is 128 rows x 256 MMA columns.  Eight epilogue warps each own 32 rows
// (their TMEM lanes) and half of the columns, 128 accumulators per thread.
// GEMM 1 (kSwiGLU): 128 gate and the matching 128 up columns, so one tile
// holds a whole 128-column block of h: the two threads of a row exchange their
// maxima through shared memory and h is rounded to E4M3 in the epilogue, never
// stored wider.  GEMM 2 (kScaled): 256 columns of y, times the routing weight.
//
// CTA pairs (cta_group::2, 256 x 256), which the bf16 kernel uses, were built
// and measured first: every buffer hand-over then crosses the cluster twice
// per K-block, and the Mixtral-shaped layer took 3.87 ms against 2.15 ms.
//
// Bounds, measured on a B200: 4096 tokens, 8 experts of 4096 x 14336 take
// 1.71 to 1.73 ms (1.68 PFLOP/s; 1.94 to 2.05 ms at the power cap; the bf16
// experts 2.31 and 2.66 ms).  Without the epilogue's work
// 1.34 ms: a K-block's operands cost one SM 48 KB of shared-memory writes and
// as many reads.  The rest is the epilogue, 128 multiply-adds per thread and
// K-block behind the tensor-memory loads.
//
// SPLIT (up to 32 tokens): reading the weights is what takes the time, and a
// tile per CTA leaves SMs idle, so that K-blocks are shared out instead (see
// Walk): one token on two of 16 experts of 4096 x 6400 takes 42 us for 157 MB,
// in whole tiles 68 us (fp8_is_split has both ways at other sizes).
#include "fp8.cuh"
#include "gemm_common.cuh"

namespace moe {

namespace fp8g {
constexpr int BM = 128;                    // MMA rows
constexpr int BN = 256;
constexpr int BK = 128;                    // codes (bytes) per K-block
constexpr int UMMA_K = 32;
constexpr int TILE_BYTES = 128 * BK;       // 128 rows of B: 16 KB
constexpr int TMEM_COLS = 512;
constexpr int EPI_WARPS = 8;
// One warpgroup for the producer and MMA warps (two of its warps idle), two for
// the epilogue; the epilogue's threads take the registers that the first does
// not need: 128 x 56 + 256 x 224 = 384 x 168, what the block is launched with.
constexpr int THREADS = 128 + EPI_WARPS * 32;
constexpr int REGS_FEW = 56, REGS_MANY = 224;
// Rows of a tile that hold data.  With SPLIT (few rows per expert) 32 of the
// MMA's 128: the others read what follows the A rows in the stage, and what
// they compute is not looked at.  A stage is then 36 KB, and six of them fit.
template <bool SPLIT> struct Cfg {
    static constexpr int ROWS = SPLIT ? kFp8SplitRows : BM;
    static constexpr int A_BYTES = ROWS * BK;
    static constexpr int STAGE_BYTES = A_BYTES + 2 * TILE_BYTES;   // A, 2 x 128 rows of B
    static constexpr int STAGES = SPLIT ? 6 : 4;                   // 216, 192 KB
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
    int wide;                     // output rows 32-byte aligned: 32-byte stores
    // SPLIT
    float* part;                  // [workers, 2, part_rows, 256] sums of a worker's partial tiles
    int part_rows;
    int32_t* arrived;             // [tiles] K-blocks whose sums are in part
};

__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate));
}
// Instruction descriptor, kind::f8f6f4: E4M3 A and B (format 0, K-major), fp32 D.
__host__ __device__ constexpr uint32_t idesc_e4m3_f32(int M, int N) {
    return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(M >> 4) << 24);
}

// Bounded wait that polls: the product buffers change hands every K-block, and
// a suspended thread's wake-up would be on that path.
__device__ __forceinline__ bool mbar_poll(uint64_t* bar, uint32_t parity, uint64_t deadline_ns) {
    for (uint32_t i = 1;; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        if (ok) return true;
        if ((i & 255u) == 0 && global_ns() > deadline_ns) return false;
    }
}

template <int N> __device__ __forceinline__ void give_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void take_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// Waits for this thread's tensor-memory loads; `v` is in the operand list so
// that no use of it can be moved above the wait.
__device__ __forceinline__ void tmem_ld_wait_for(float (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]),
                   "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]),
                   "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]),
                   "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
                   "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]),
                   "+f"(v[30]), "+f"(v[31])
                 :
                 : "memory");
}

// acc[AT .. AT + 32) += s * v.  (The packed two-float multiply-add was slower:
// 348 us against 296 for a 8192 x 2048 x 4096 layer.)
template <int AT> __device__ __forceinline__ void add_scaled(float (&acc)[128], float s,
                                                             const float (&v)[32]) {
#pragma unroll
    for (int j = 0; j < 32; ++j) acc[AT + j] = fmaf(s, v[j], acc[AT + j]);
}

// 2^x and 1/x to within 2 units in the last place, results below 2^-126 flushed
// to zero: one instruction each (__expf and a division handle subnormals, in
// several more).
__device__ __forceinline__ float exp2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 32 bytes of a row.  A thread writes its own row, so that a warp's store
// touches 32 rows: 32-byte stores fill whole sectors (16384 tokens, 64 experts
// of 2048 x 1024: 1153 us against 1235 us in pairs of 16 bytes).
__device__ __forceinline__ void store32(void* p, const uint32_t (&o)[8], bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(o[0]),
                     "r"(o[1]), "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                     : "memory");
    } else {
        static_cast<uint4*>(p)[0] = make_uint4(o[0], o[1], o[2], o[3]);
        static_cast<uint4*>(p)[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

// Barrier of the 256 epilogue threads.
__device__ __forceinline__ void epilogue_sync() {
    asm volatile("bar.sync 1, 256;" ::: "memory");
}

__device__ __forceinline__ float silu_mul(float g, float u) {
    return g * rcp_approx(1.f + exp2_approx(g * -1.44269504f)) * u;
}

// What a row of y is multiplied by (GEMM 2).  `hole`: an entry of perm outside
// the slots.  No token was rounded into such a row; it is written as zeros
// (a weight of 0 would keep the NaN that old codes and scales can stand for).
__device__ __forceinline__ float row_weight(const GemmParams& p, const TileCoord& c,
                                            int64_t row, bool& hole) {
    hole = false;
    if (!c.routed) return 1.f;
    const int64_t slot = p.perm[row];
    hole = slot < 0 || slot >= p.T * p.k;
    return hole ? 0.f : p.routed_scale * p.topk_w[slot];
}

// The tiles a CTA computes, in the order that its producer, MMA and epilogue
// warps all walk.  Without SPLIT: every workers-th tile, whole.  With SPLIT:
// the K-blocks of all tiles in a row, an equal share per CTA, which may begin
// and end inside a tile.
struct Segment {
    TileCoord c;
    int tile, num_kb, kb0, kb1;     // K-blocks [kb0, kb1) of num_kb
};

template <int EPI, bool SPLIT> struct Walk {
    const GroupTable& gt;
    const GemmParams& p;
    int worker, workers;
    int kb_routed, kb_shared;       // K-blocks of a tile
    int routed_tiles;
    int share, longer;              // SPLIT: K-blocks per CTA, one more in the first `longer`
    int pos, end;                   // SPLIT: K-blocks; else tiles
    __device__ __forceinline__ Walk(const GroupTable& gt, const GemmParams& p)
        : gt(gt), p(p), worker(blockIdx.x), workers(gridDim.x) {
        kb_routed = (p.K_routed + fp8g::BK - 1) / fp8g::BK;
        kb_shared = (p.K_shared + fp8g::BK - 1) / fp8g::BK;
        routed_tiles = gt.tile_start[p.E];
        if (SPLIT) {
            const int blocks = first_block(gt.total_tiles);
            share = blocks / workers;
            longer = blocks - share * workers;
            pos = begin_of(worker);
            end = begin_of(worker + 1);
        } else {
            pos = worker;
            end = gt.total_tiles;
        }
    }
    // first K-block of a tile, numbered through all tiles
    __device__ __forceinline__ int first_block(int tile) const {
        return min(tile, routed_tiles) * kb_routed + max(tile - routed_tiles, 0) * kb_shared;
    }
    // first K-block of CTA w
    __device__ __forceinline__ int begin_of(int w) const { return w * share + min(w, longer); }
    // CTA that computes K-block b
    __device__ __forceinline__ int worker_of(int b) const {
        const int in_longer = longer * (share + 1);
        return b < in_longer ? b / (share + 1) : longer + (b - in_longer) / share;
    }
    __device__ __forceinline__ bool next(Segment& s) {
        if (pos >= end) return false;
        if (SPLIT) {
            const int routed = routed_tiles * kb_routed;
            s.tile = pos < routed ? pos / kb_routed : routed_tiles + (pos - routed) / kb_shared;
            s.c = tile_coord(s.tile);
            s.num_kb = s.c.routed ? kb_routed : kb_shared;
            s.kb0 = pos - first_block(s.tile);
            s.kb1 = min(s.num_kb, s.kb0 + (end - pos));
            pos += s.kb1 - s.kb0;
        } else {
            s.tile = pos;
            s.c = tile_coord(s.tile);
            s.num_kb = s.kb1 = s.c.routed ? kb_routed : kb_shared;
            s.kb0 = 0;
            pos += workers;
        }
        return true;
    }
    __device__ __forceinline__ TileCoord tile_coord(int tile) const {
        return decode_tile(gt, p, tile, EPI == kSwiGLU ? fp8g::BN / 2 : fp8g::BN,
                           fp8g::Cfg<SPLIT>::ROWS);
    }
};

// Offsets that do not go up from 0 to at most the slots (no plan of moe_permute's):
// each is brought into that range and to the smallest behind it.  The groups'
// rows then lie side by side and end at offsets[E], as the rounding of x takes
// it, so that rows, tiles and the arrival counters stay within what the host
// sized, whatever the offsets say.  By one warp.
__device__ __forceinline__ void order_offsets(int32_t* offsets, int E, int slots) {
    if ((threadIdx.x & 31) == 0) {
        int least = slots;
        for (int g = E; g >= 0; --g) offsets[g] = least = max(min(offsets[g], least), 0);
    }
    __syncwarp();
}

// The group table, by one warp, 32 groups at a time, from the offsets that all
// threads have put in gt.tile_start[0..E] (an entry is read before the prefix
// takes its place).
__device__ __forceinline__ void build_table(GroupTable& gt, const GemmParams& p, int tile_rows) {
    const int lane = threadIdx.x & 31;
    int start = 0;
    for (int g0 = 0; g0 < p.E + p.S; g0 += 32) {
        const int g = g0 + lane;
        int rows = 0, row0 = 0;
        if (g < p.E) {
            row0 = gt.tile_start[g];
            rows = gt.tile_start[g + 1] - row0;
        } else if (g < p.E + p.S) {
            row0 = static_cast<int>((g - p.E) * p.T);
            rows = static_cast<int>(p.T);
        }
        const int tiles = (rows + tile_rows - 1) / tile_rows *
                          (g < p.E ? p.n_tiles_routed : p.n_tiles_shared);
        int sum = tiles;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int v = __shfl_up_sync(0xffffffffu, sum, d);
            if (lane >= d) sum += v;
        }
        __syncwarp();                  // this chunk's offsets are read
        if (g < p.E + p.S) {
            gt.rows[g] = rows;
            gt.row0[g] = row0;
            gt.tile_start[g] = start + sum - tiles;
        }
        __syncwarp();
        start += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) {
        gt.n_groups = p.E + p.S;
        gt.tile_start[p.E + p.S] = gt.total_tiles = start;
    }
}

// Rows of the operands of a tile.
struct TileSource {
    int a_row, b_row, b_row2;       // A; the two halves of B
};
template <int EPI>
__device__ __forceinline__ TileSource tile_source(const GemmParams& p, const GroupTable& gt,
                                                  const TileCoord& c) {
    TileSource t;
    const int eidx = c.routed ? c.g : c.g - p.E;
    // routed -> sorted slot rows; shared GEMM 1 -> token rows; shared GEMM 2 ->
    // that expert's block of h
    t.a_row = (EPI == kSwiGLU && !c.routed ? 0 : gt.row0[c.g]) + c.m0;
    t.b_row = eidx * (c.routed ? p.b_rows_routed : p.b_rows_shared) + c.n0;
    t.b_row2 = t.b_row + (EPI == kSwiGLU ? (c.routed ? p.half_routed : p.half_shared)
                                         : fp8g::BN / 2);
    return t;
}

// Adds up the parts of a tile in the order of their K-blocks (whichever CTA
// does it, the sum is the same) and writes the tile's rows, a warp per row:
// rows warp, warp + warps, ...
template <int EPI, bool SPLIT>
__device__ __forceinline__ void finish_parts(const Walk<EPI, SPLIT>& walk, const Segment& sg,
                                             const GroupTable& gt, const Fp8GemmParams& fp,
                                             int warp, int warps) {
    const GemmParams& p = fp.g;
    const TileCoord& c = sg.c;
    const int lane = threadIdx.x & 31;
    const int N = c.routed ? p.N_routed : p.N_shared;
    const int first = walk.first_block(sg.tile);
    const int w0 = walk.worker_of(first), w1 = walk.worker_of(first + sg.num_kb - 1);
    const int rows = min(c.rows - c.m0, fp8g::Cfg<SPLIT>::ROWS);
    // this lane's columns of the tile: 4 of gate and of up, or twice 4 of y
    const int ca = 4 * lane, cb = 128 + 4 * lane;
    for (int r = warp; r < rows; r += warps) {
        const int64_t orow = static_cast<int64_t>(gt.row0[c.g]) + c.m0 + r;
        bool hole = false;
        const float weight = EPI == kScaled ? row_weight(p, c, orow, hole) : 1.f;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
        for (int w = w0; w <= w1; w += 8) {
            // eight CTAs' parts in flight, added in order
            float4 va[8], vb[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                va[i] = vb[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (w + i > w1) continue;
                const int begin = walk.begin_of(w + i);
                const float* from = fp.part + ((static_cast<int64_t>(w + i) * 2 +
                                                (begin <= first)) * fp.part_rows + r) * fp8g::BN;
                va[i] = __ldcg(reinterpret_cast<const float4*>(from + ca));
                vb[i] = __ldcg(reinterpret_cast<const float4*>(from + cb));
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                a.x += va[i].x; a.y += va[i].y; a.z += va[i].z; a.w += va[i].w;
                b.x += vb[i].x; b.y += vb[i].y; b.z += vb[i].z; b.w += vb[i].w;
            }
        }
        if (EPI == kSwiGLU) {
            const int n = c.n0 + ca;
            float h[4] = {silu_mul(a.x, b.x), silu_mul(a.y, b.y), silu_mul(a.z, b.z),
                          silu_mul(a.w, b.w)};
            uint32_t mag = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h[j] = n < N ? nan_if_not_finite(h[j]) : 0.f;
                mag = max(mag, finite_mag(h[j]));
            }
            mag = __reduce_max_sync(0xffffffffu, mag);
            const uint32_t byte = e8m0_of(mag);
            const float inv = e8m0_inverse(byte);
            if (n < N)
                *reinterpret_cast<uint32_t*>(
                    static_cast<uint8_t*>(c.routed ? p.out_routed : p.out_shared) + orow * N + n) =
                    e4m3x4(h[0] * inv, h[1] * inv, h[2] * inv, h[3] * inv);
            if (lane == 0)
                (c.routed ? fp.hs_routed : fp.hs_shared)[orow * fp8_scale_ld(N) + c.n0 / 128] =
                    static_cast<uint8_t>(byte);
        } else {
            const float s = weight;
            if (hole) a = b = make_float4(0.f, 0.f, 0.f, 0.f);
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out_routed) +
                                 (orow + (c.routed ? 0 : p.out_row0_shared)) * N + c.n0;
            if (c.n0 + ca < N)
                *reinterpret_cast<uint2*>(out + ca) = make_uint2(pack_bf16x2(s * a.x, s * a.y),
                                                                 pack_bf16x2(s * a.z, s * a.w));
            if (c.n0 + cb < N)
                *reinterpret_cast<uint2*>(out + cb) = make_uint2(pack_bf16x2(s * b.x, s * b.y),
                                                                 pack_bf16x2(s * b.z, s * b.w));
        }
    }
}

template <int EPI, bool SPLIT>
__global__ void __launch_bounds__(fp8g::THREADS, 1) grouped_gemm_fp8(
    const __grid_constant__ CUtensorMap map_a_routed,
    const __grid_constant__ CUtensorMap map_a_shared,
    const __grid_constant__ CUtensorMap map_b_routed,
    const __grid_constant__ CUtensorMap map_b_shared, const Fp8GemmParams fp) {
    using namespace fp8g;
    using C = Cfg<SPLIT>;
    constexpr int ROWS = C::ROWS, A_BYTES = C::A_BYTES, STAGE_BYTES = C::STAGE_BYTES,
                  STAGES = C::STAGES;
    const GemmParams& p = fp.g;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ GroupTable gt;
    __shared__ uint32_t tmem_base_sh;
    __shared__ bool last_sh[2];                 // SPLIT: this CTA completes the tile
    __shared__ uint32_t mag_sh[2][2][BM];       // [tile parity][column half][row]

    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * STAGE_BYTES);
    uint64_t* full = bars;                 // [STAGES] TMA bytes of the stage
    uint64_t* empty = bars + STAGES;       // [STAGES] stage consumed
    uint64_t* tfull = bars + 2 * STAGES;   // [2]      K-block product ready
    uint64_t* tempty = tfull + 2;          // [2]      product read by every epilogue warp
    uint64_t* drain = tempty + 2;          // [1]      all MMAs complete

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // Every kernel of this chain lets the next one start only after its own
    // pdl_wait: what the kernels before the previous one wrote (the plan) and
    // the weights are there already, so the table is built and the first weight
    // tiles are loaded while the previous kernel still runs.
    // (The plan is read from L2: a line of an earlier one may still be in L1.)
    const int slots = static_cast<int>(p.T * p.k);
    bool disorder = false;
    for (int g = threadIdx.x; g <= p.E; g += THREADS) {
        const int at = __ldcg(p.offsets + g);
        const int next = g < p.E ? __ldcg(p.offsets + g + 1) : slots;
        disorder |= at < 0 || at > next || next > slots;
        gt.tile_start[g] = at;
    }
    if (threadIdx.x == 32) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], EPI_WARPS);
        }
        mbar_init(drain, 1);
        fence_barrier_init();
    }
    __syncwarp();
    if (warp == 1) {
        tmem_alloc(&tmem_base_sh, TMEM_COLS);
        tmem_relinquish();
    }
    if (threadIdx.x == 64) {
        tma_prefetch_desc(&map_a_routed);
        tma_prefetch_desc(&map_b_routed);
        if (p.S > 0) {
            tma_prefetch_desc(&map_a_shared);
            tma_prefetch_desc(&map_b_shared);
        }
    }
    tc_fence_before();
    const bool reorder = __syncthreads_or(disorder);
    tc_fence_after();
    if (warp == 0) {
        if (reorder) order_offsets(gt.tile_start, p.E, slots);
        build_table(gt, p, ROWS);
    }
    __syncthreads();
    const uint32_t tmem_base = tmem_base_sh;
    Walk<EPI, SPLIT> walk(gt, p);
    Segment sg;

    if (warp < 4) {
        give_registers<REGS_FEW>();
        if (warp == 0) {
            // ------------------------------------------------------------ producer
            if (lane == 0) {
                int stage = 0;
                uint32_t phase = 0;
                uint32_t filled = 0, parity = 0;   // per stage: loaded at all, phase of the last load
                bool ok = true;
                // the weight tiles of the first stages, before pdl_wait
                int ahead = 0;
                {
                    Walk<EPI, SPLIT> first = walk;
                    while (ahead < STAGES && first.next(sg)) {
                        const TileSource src = tile_source<EPI>(p, gt, sg.c);
                        const CUtensorMap* mb = sg.c.routed ? &map_b_routed : &map_b_shared;
                        for (int kb = sg.kb0; kb < sg.kb1 && ahead < STAGES; ++kb, ++ahead) {
                            uint8_t* sb = smem + ahead * STAGE_BYTES + A_BYTES;
                            mbar_arrive_expect_tx(&full[ahead], STAGE_BYTES);
                            tma_load_2d(sb, mb, &full[ahead], kb * BK, src.b_row);
                            tma_load_2d(sb + TILE_BYTES, mb, &full[ahead], kb * BK, src.b_row2);
                        }
                    }
                }
                pdl_wait();
                pdl_launch_dependents();
                const uint64_t deadline = global_ns() + p.timeout_ns;
                while (ok && walk.next(sg)) {
                    const TileSource src = tile_source<EPI>(p, gt, sg.c);
                    const CUtensorMap* ma = sg.c.routed ? &map_a_routed : &map_a_shared;
                    const CUtensorMap* mb = sg.c.routed ? &map_b_routed : &map_b_shared;
                    for (int kb = sg.kb0; kb < sg.kb1; ++kb) {
                        uint8_t* sa = smem + stage * STAGE_BYTES;
                        if (ahead > 0) {
                            --ahead;
                        } else {
                            if (!mbar_wait(&empty[stage], phase ^ 1u, deadline)) {
                                ok = false;
                                break;
                            }
                            mbar_arrive_expect_tx(&full[stage], STAGE_BYTES);
                            tma_load_2d(sa + A_BYTES, mb, &full[stage], kb * BK, src.b_row);
                            tma_load_2d(sa + A_BYTES + TILE_BYTES, mb, &full[stage], kb * BK,
                                        src.b_row2);
                        }
                        tma_load_2d(sa, ma, &full[stage], kb * BK, src.a_row);
                        filled |= 1u << stage;
                        parity = (parity & ~(1u << stage)) | (phase << stage);
                        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                    }
                }
                // no copy is in flight when the CTA ends
                for (int s = 0; s < STAGES; ++s)
                    if (filled >> s & 1u)
                        ok &= mbar_wait(&full[s], parity >> s & 1u, deadline + 1000000000ull);
                if (!ok) raise_error(p.err_flag, MOE_ERR_TIMEOUT);
            }
        } else if (warp == 1) {
            // ------------------------------------------------------------ MMA
            if (lane == 0) {
                constexpr uint32_t idesc = idesc_e4m3_f32(BM, BN);
                pdl_wait();
                const uint64_t deadline = global_ns() + p.timeout_ns;
                int stage = 0, buf = 0;
                uint32_t phase = 0, buf_phase = 0;
                bool ok = true;
                while (ok && walk.next(sg)) {
                    for (int kb = sg.kb0; kb < sg.kb1; ++kb) {
                        if (!mbar_poll(&tempty[buf], buf_phase ^ 1u, deadline) ||
                            !mbar_poll(&full[stage], phase, deadline)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t d = tmem_base + static_cast<uint32_t>(buf * BN);
                        const uint32_t sa = smem_u32(smem + stage * STAGE_BYTES);
                        const uint32_t sb = sa + A_BYTES;
#pragma unroll
                        for (int kk = 0; kk < BK / UMMA_K; ++kk)
                            umma_e4m3(d, smem_desc_sw128(sa + kk * UMMA_K),
                                      smem_desc_sw128(sb + kk * UMMA_K), idesc, kk != 0 ? 1u : 0u);
                        umma_commit(&empty[stage]);
                        umma_commit(&tfull[buf]);
                        if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                        if (++buf == 2) { buf = 0; buf_phase ^= 1u; }
                    }
                }
                if (!ok) raise_error(p.err_flag, MOE_ERR_TIMEOUT);
                // every issued MMA completes before the tensor memory is released
                umma_commit(drain);
                if (!mbar_wait(drain, 0, deadline + 1000000000ull))
                    raise_error(p.err_flag, MOE_ERR_TIMEOUT);
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue
        take_registers<REGS_MANY>();
        pdl_wait();
        const uint64_t deadline = global_ns() + p.timeout_ns;
        const int quarter = warp & 3;               // TMEM lane quarter of this warp
        const int half = (warp - 4) >> 2;           // column half
        const int row = quarter * 32 + lane;
        // first TMEM column of this thread's two runs of 64
        const int col0 = EPI == kSwiGLU ? 64 * half : 128 * half;
        const int col1 = EPI == kSwiGLU ? 128 + 64 * half : 128 * half + 64;
        int buf = 0, parity = 0;
        uint32_t buf_phase = 0;
        // after a wait that ran out, the loops still run to their end (the
        // epilogue barrier needs every warp) without waiting or storing
        bool ok = true;
        // tiles that this CTA has left a part of: one begun by another CTA, one
        // that another goes on with
        int pending[2] = {-1, -1};
        while (walk.next(sg)) {
            const TileCoord& c = sg.c;
            const int N = c.routed ? p.N_routed : p.N_shared;
            const int num_kb = sg.num_kb;
            const int eidx = c.routed ? c.g : c.g - p.E;
            const int m = c.m0 + row;
            const bool valid = row < ROWS && m < c.rows;
            // of this warp's rows
            const bool any = quarter * 32 < ROWS && m - lane < c.rows;
            const int64_t a_row =
                (EPI == kSwiGLU && !c.routed ? 0 : static_cast<int64_t>(gt.row0[c.g])) +
                (valid ? m : c.rows - 1);
            const uint32_t* sa = reinterpret_cast<const uint32_t*>(
                (c.routed ? fp.sa_routed : fp.sa_shared) + a_row * fp8_scale_ld(c.routed ? p.K_routed : p.K_shared));
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
            float acc[128];          // [0, 64) the first run of 64 columns, [64, 128) the second
#pragma unroll
            for (int j = 0; j < 128; ++j) acc[j] = 0.f;
            // scales one step ahead: words of four activation scales, and the
            // weight scales of the next K-block
            uint32_t word = sa[sg.kb0 >> 2];
            uint32_t next_word = (sg.kb0 | 3) + 1 < sg.kb1 ? sa[(sg.kb0 >> 2) + 1] : 0;
            float w0 = sw0[sg.kb0], w1 = sw1[sg.kb0];
#pragma unroll 1
            for (int kb = sg.kb0; kb < sg.kb1; ++kb) {
                const float ea = e8m0_value(word >> (8 * (kb & 3)) & 0xffu);
                if ((kb & 3) == 3) {
                    word = next_word;
                    if (kb + 5 < sg.kb1) next_word = sa[(kb >> 2) + 2];
                }
                const float s0 = ea * w0, s1 = ea * w1;
                if (kb + 1 < sg.kb1) {
                    w0 = sw0[kb + 1];
                    if (EPI == kSwiGLU) w1 = sw1[kb + 1];
                    else w1 = w0;
                }
                if (ok && !mbar_poll(&tfull[buf], buf_phase, deadline)) {
                    raise_error(p.err_flag, MOE_ERR_TIMEOUT);
                    ok = false;
                }
                ok = __all_sync(0xffffffffu, ok);    // the loads below are the warp's
                tc_fence_after();
                const bool work = any && ok;
                float va[32], vb[32];
                if (work) {
                    // each load is in flight while the columns before it are added
                    const uint32_t t = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                                       static_cast<uint32_t>(buf * BN);
                    tmem_ld32(t + col0, va);
                    tmem_ld_wait_for(va);
                    tmem_ld32(t + col0 + 32, vb);
                    add_scaled<0>(acc, s0, va);
                    tmem_ld_wait_for(vb);
                    tmem_ld32(t + col1, va);
                    add_scaled<32>(acc, s0, vb);
                    tmem_ld_wait_for(va);
                    tmem_ld32(t + col1 + 32, vb);
                    add_scaled<64>(acc, s1, va);
                    tmem_ld_wait_for(vb);
                }
                // the buffer is free once its last columns are in registers
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&tempty[buf]);
                if (work) add_scaled<96>(acc, s1, vb);
                if (++buf == 2) { buf = 0; buf_phase ^= 1u; }
            }
            if (SPLIT && sg.kb1 - sg.kb0 < num_kb) {
                // a part of the tile: leave its sums, in the tile's columns
                float* mine = fp.part + ((static_cast<int64_t>(walk.worker) * 2 + (sg.kb0 == 0)) *
                                             fp.part_rows + row) * BN;
                if (valid) {
#pragma unroll
                    for (int j = 0; j < 64; j += 4) {
                        *reinterpret_cast<float4*>(mine + col0 + j) =
                            make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
                        *reinterpret_cast<float4*>(mine + col1 + j) = make_float4(
                            acc[64 + j], acc[64 + j + 1], acc[64 + j + 2], acc[64 + j + 3]);
                    }
                }
                pending[sg.kb0 == 0] = sg.tile;
                continue;
            }
            if (EPI == kSwiGLU) {
                // h = silu(g) u, rounded to E4M3 with the scale of its 128 columns
                const int n = c.n0 + 64 * half;
                float top = 0.f;
#pragma unroll
                for (int j = 0; j < 64; ++j) acc[j] = silu_mul(acc[j], acc[64 + j]);
                if (n + 64 > N) {            // columns past the end take no part
#pragma unroll
                    for (int j = 0; j < 64; ++j)
                        if (n + j >= N) acc[j] = 0.f;
                }
#pragma unroll
                for (int j = 0; j < 64; ++j) top = fmaxf(top, fabsf(acc[j]));   // skips NaN
                if (top == __uint_as_float(0x7f800000u)) {
                    // an infinity would saturate: a NaN instead, outside the maximum
                    uint32_t mag = 0;
#pragma unroll
                    for (int j = 0; j < 64; ++j) {
                        mag = max(mag, finite_mag(acc[j]));
                        acc[j] = nan_if_not_finite(acc[j]);
                    }
                    top = __uint_as_float(mag);
                }
                uint32_t mag = __float_as_uint(top);
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
                    for (int v = 0; v < 2; ++v) {
                        uint32_t o[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const int j = 32 * v + 4 * e;
                            o[e] = e4m3x4(acc[j] * inv, acc[j + 1] * inv, acc[j + 2] * inv,
                                          acc[j + 3] * inv);
                        }
                        if (n + 32 * v + 16 < N)
                            store32(out + 32 * v, o, fp.wide);
                        else if (n + 32 * v < N)
                            *reinterpret_cast<uint4*>(out + 32 * v) =
                                make_uint4(o[0], o[1], o[2], o[3]);
                    }
                    if (half == 0)
                        (c.routed ? fp.hs_routed
                                  : fp.hs_shared)[orow * fp8_scale_ld(N) + c.n0 / 128] =
                            static_cast<uint8_t>(byte);
                }
            } else if (valid && ok) {
                int64_t orow = static_cast<int64_t>(gt.row0[c.g]) + m;
                bool hole;
                const float scale = row_weight(p, c, orow, hole);
                const uint32_t keep = hole ? 0u : 0xffffffffu;
                if (!c.routed) orow += p.out_row0_shared;
                const int n = c.n0 + 128 * half;
                __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out_routed) + orow * N + n;
#pragma unroll
                for (int v = 0; v < 8; ++v) {
                    uint32_t o[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int j = 16 * v + 2 * e;
                        o[e] = pack_bf16x2(scale * acc[j], scale * acc[j + 1]) & keep;
                    }
                    if (n + 16 * v < N) store32(out + 16 * v, o, fp.wide);
                }
            }
        }
        if (SPLIT) {
            // count the parts in, once for both tiles; whoever completes a tile
            // finishes it
            __threadfence();
            epilogue_sync();
            if (warp < 6 && lane == 0) {
                const int i = warp - 4;         // one tile each
                const int tile = pending[i];
                last_sh[i] = false;
                if (tile >= 0) {
                    const int first = walk.first_block(tile);
                    const int blocks = tile < walk.routed_tiles ? walk.kb_routed : walk.kb_shared;
                    const int n = min(first + blocks, walk.end) -
                                  max(first, walk.begin_of(walk.worker));
                    last_sh[i] = atomicAdd(fp.arrived + tile, n) + n == blocks;
                }
                __threadfence();
            }
            epilogue_sync();
            // two tiles: four warps each
            const bool both = last_sh[0] && last_sh[1];
            const int i = both ? (warp - 4) >> 2 : last_sh[0] ? 0 : 1;
            if (last_sh[i] && ok) {
                sg.tile = pending[i];
                sg.c = walk.tile_coord(sg.tile);
                sg.num_kb = sg.c.routed ? walk.kb_routed : walk.kb_shared;
                finish_parts<EPI, SPLIT>(walk, sg, gt, fp, both ? warp & 3 : warp - 4,
                                         both ? 4 : EPI_WARPS);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

namespace {

// Codes [rows, cols], box of 128 columns x box_rows rows, 128-byte swizzle.
bool make_map_codes(CUtensorMap* map, const void* base, int64_t rows, int64_t cols,
                    int box_rows = 128) {
    EncodeTiledFn enc = get_encode_fn();
    if (!enc || rows <= 0 || cols <= 0) return false;
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols)};
    cuuint32_t box[2] = {fp8g::BK, static_cast<cuuint32_t>(box_rows)};
    cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

template <int EPI, bool SPLIT>
cudaError_t launch_gemm(const Fp8GemmParams& p, int64_t tiles, int num_sms,
                        const CUtensorMap& ar, const CUtensorMap& as, const CUtensorMap& br,
                        const CUtensorMap& bs, cudaStream_t st) {
    using namespace fp8g;
    auto kern = grouped_gemm_fp8<EPI, SPLIT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         Cfg<SPLIT>::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    // the register split assumes what the block is launched with
    static const bool split_fits = [&] {
        cudaFuncAttributes a;
        return cudaFuncGetAttributes(&a, kern) == cudaSuccess &&
               a.numRegs * THREADS >= 128 * REGS_FEW + 256 * REGS_MANY;
    }();
    if (!split_fits) return cudaErrorLaunchOutOfResources;
    const int64_t grid = SPLIT || tiles > num_sms ? num_sms : tiles;
    return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(THREADS),
                      Cfg<SPLIT>::SMEM_BYTES, st, ar,
                      as, br, bs, p);
}

}  // namespace

// The experts on the quantised rows o.xq / o.xs.
cudaError_t launch_ffn_fp8(const moe_shape& s, const Fp8Operands& o, int num_sms,
                           cudaStream_t st) {
    const int64_t Tk = s.T * s.k;
    const int S = s.n_shared, Is = S > 0 ? s.I_shared : s.I;
    CUtensorMap a1r, a1s, b1r, b1s, a2r, a2s, b2r, b2s;
    const bool split = fp8_is_split(s);
    const int a_rows = split ? kFp8SplitRows : fp8g::BM;
    bool ok = make_map_codes(&a1r, o.xq, Tk, s.H, a_rows);
    ok &= make_map_codes(&b1r, o.gate_up, static_cast<int64_t>(s.E) * 2 * s.I, s.H);
    ok &= make_map_codes(&a2r, o.hq, Tk, s.I, a_rows);
    ok &= make_map_codes(&b2r, o.down, static_cast<int64_t>(s.E) * s.H, s.I);
    if (S > 0) {
        ok &= make_map_codes(&a1s, o.xq + Tk * s.H, s.T, s.H, a_rows);
        ok &= make_map_codes(&b1s, o.sh_gate_up, static_cast<int64_t>(S) * 2 * Is, s.H);
        ok &= make_map_codes(&a2s, o.hq_sh, S * s.T, Is, a_rows);
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
    g.group_m = 16;
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
    const Fp8Tiles tiles = fp8_tiles(s);
    p.part = o.part;
    p.part_rows = fp8_part_rows(s);
    p.arrived = o.arrived;
    auto aligned32 = [](const void* q) { return reinterpret_cast<uintptr_t>(q) % 32 == 0; };
    p.wide = s.I % 32 == 0 && Is % 32 == 0 && aligned32(o.hq) && (S == 0 || aligned32(o.hq_sh));
    cudaError_t e = split ? launch_gemm<kSwiGLU, true>(p, tiles.gate_up, num_sms, a1r, a1s, b1r,
                                                       b1s, st)
                          : launch_gemm<kSwiGLU, false>(p, tiles.gate_up, num_sms, a1r, a1s, b1r,
                                                        b1s, st);
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
    p.arrived = o.arrived + tiles.gate_up;
    p.wide = aligned32(o.y_slots);      // H is a multiple of 16
    return split ? launch_gemm<kScaled, true>(p, tiles.down, num_sms, a2r, a2s, b2r, b2s, st)
                 : launch_gemm<kScaled, false>(p, tiles.down, num_sms, a2r, a2s, b2r, b2s, st);
}

}  // namespace moe
