// The experts' BF16 matrix products over rows ordered by expert, with FP32
// accumulation on the tensor cores:
//   forward  y[r]  = x[r] w[e]^T                       (sum over K)
//   dgrad    dx[r] = dy[r] w[e]                        (sum over N)
//   wgrad    dw[e] = sum over e's rows dy[r]^T x[r]    (sum over the rows)
//
// All three are one kernel computing D[m][n] = sum_d A(m, d) B(n, d) in tiles
// of 256 x TN per pair of SMs (tcgen05.mma.cta_group::2, kind::f16; each SM
// holds 128 of the 256 rows of A and D and half of the TN rows of B):
//   forward  m: output column, A = w[e] (d contiguous);  n: row, B = x
//   dgrad    m: output column, A = w[e] (m contiguous);  n: row, B = dy
//   wgrad    m: N, A = dy (m contiguous);  n: K, B = x (n contiguous);  d: row
// The weights sit on the M side, so that the tile's row extent TN follows the
// experts' segment lengths: an expert with one row streams its weights past a
// 32-row tile.  An operand whose m or n is contiguous in memory is copied as
// it lies (64 x 128 boxes, 128-byte swizzle) and read by the MMA as an MN-major
// operand: no transposed copy of w, dy or x is ever made.
//
// Segments are ragged and unpadded.  forward / dgrad: rows of a tile past the
// segment's end hold another expert's values (or the copy's zero fill), which
// reach only their own columns of D and are not stored.  wgrad sums over the
// rows, so there the last block of a segment is cut: the MMA issues only the
// 16-row steps that hold rows, and the rows of the last step past the end are
// overwritten with zeros in shared memory before the MMA reads them (a factor
// of zero on one side alone would let a neighbour's NaN through).
//
// Roles per CTA: warp 0 producer of the copies, warp 1 tensor-memory
// allocation and, in rank 0, the MMA issuer, warp 3 the cutter of ragged ends
// (wgrad), the last four or eight warps the epilogue.  Two accumulators: the
// epilogue of one tile overlaps the main loop of the next.  The grid is
// persistent, one pair per two SMs; every CTA scans the experts' counts for
// its tile list, so nothing runs ahead of the kernel and the counts never
// leave the device.  Every wait is bounded (1 s); a timeout sets a status bit,
// marks both CTAs aborted, and all roles drain to the final pair barrier.
//
// Few tiles of a long depth (SPLIT): a cluster of two or four pairs per tile,
// each pair with its part of the depth.  The parts' FP32 sums are left in their
// CTAs' shared memory and every pair adds up and stores a share of the columns,
// the parts in order: no workspace, no atomics, the same result each time.
//
// Bound by HBM while the experts have few rows, by the tensor cores under the
// power limit with many.  Measured on GB300 (BF16, 6.8 TB/s copied, 1.7 PFLOP/s
// sustained by cuBLAS): 8 rows of 8 experts of 4096 x 7168 forward 72-75 us
// (6.3-6.5 TB/s); 2999 rows of 60 experts of 1536 x 2048 dgrad 65 (6.2 TB/s),
// wgrad 72 (5.6 TB/s of gradients written); 16384 rows of 16 experts of
// 4096 x 7168 forward 585-675 us, dgrad 580-625, wgrad 625-660 (1.43-1.65
// PFLOP/s, by the box and by what ran before; equal segments 550-580, 540-610 and
// 600-640, on cuBLAS 500-545, 515-570 and 530-570).
#include <cudaTypedefs.h>
#include <math.h>

#include "common.cuh"
#include "host.h"
#include "train_kernels.h"

namespace moe {

namespace {

constexpr int kHalfM = 128;                    // A rows per CTA
constexpr int kMGroup = 8;                     // m tiles walked together (L2 reuse)
constexpr int kMaxExperts = 1024;

struct ExpertParams {
    int m_extent;          // D rows that exist: output columns (forward, dgrad) or N (wgrad)
    int n_extent;          // wgrad: K
    int depth;             // forward, dgrad: reduction length
    int E;
    int64_t rows;
    const int* count;
    const int* offsets;
    __nv_bfloat16* out;
    unsigned int* status;  // may be null
    int half_m;            // D rows per CTA of a tile, up to kHalfM
    int box_n;             // forward, dgrad: B rows per copy
    int stages;            // of the ring: what fits of half_m rows of A and TN / 2 of B
    int split;             // pairs of a cluster that share a tile's depth: 1, 2 or 4
};

// DEPTH: reduction elements per stage.  Deep stages (64 KB a CTA at TN = 256)
// halve the barrier hand-offs per MMA; the shallow wgrad leaves room for wider
// stores (see kWgradDeepRows).
template <int PRODUCT, int TN, int DEPTH>
struct ExpertCfg {
    static constexpr bool kWgrad = PRODUCT == kExpertWgrad;
    static_assert(DEPTH == 128 || (DEPTH == 64 && kWgrad), "K-major rows come in two chunks of 64");
    static constexpr int kHalfN = TN / 2;                          // B rows per CTA
    static constexpr int kTileA = kHalfM * DEPTH * 2;              // bytes
    static constexpr int kTileB = kHalfN * DEPTH * 2;
    static constexpr int kChunkMn = DEPTH * 128;                   // bytes of an MN-major chunk
    static constexpr int kStages = DEPTH == 64 ? 5 : TN == 256 ? 3 : TN == 128 ? 4 : 5;
    static constexpr int kOutCols = DEPTH == 64 ? 64 : 32;         // wgrad: columns a warp stores at a time
    static constexpr int kOutRows = TN == 64 ? 16 : 32;            // forward, dgrad: rows a warp stores at a time
    static constexpr int kOutBytes = kWgrad ? 32 * kOutCols * 2 : kOutRows * 64;
    static constexpr int kEpiWarps = TN >= 64 ? 8 : 4;
    static constexpr int kThreads = (4 + kEpiWarps) * 32;
    static constexpr uint32_t kTmemCols = 2 * TN;
    // forward: more stages where the tiles are lower than kHalfM
    static constexpr int kMaxStages = PRODUCT == kExpertForward ? 10 : kStages;
    static constexpr int kBars = 3 * kMaxStages + 5;
    static constexpr int kOut = kEpiWarps * kOutBytes;
    static constexpr int kSmemBytes =
        1024 + kStages * (kTileA + kTileB) + kOut + 3 * kMaxExperts * 4 + kBars * 8 + 64;
    static_assert(kSmemBytes <= 232448, "shared memory budget");
};

__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// MN-major operand tile: chunks of 64 m (or n) elements, each [depth][128 B]
// with the 128-byte swizzle; `chunk` = bytes from chunk to chunk (the leading
// offset), 1024 bytes from one group of eight d to the next (the stride).
__device__ __forceinline__ uint64_t sdesc_mnmajor_sw128(uint32_t saddr, uint32_t chunk) {
    return sdesc(saddr, chunk, 1024, kSwizzle128B);
}

// Descriptor offset (16-byte units) of a stage's j-th 16 reduction elements:
// 16 rows of 128 bytes further in every chunk (MN-major), or 32 bytes further
// in the rows of the 64-element chunk j / 4 (K-major, `tile` bytes in two chunks).
template <bool MN>
__device__ __forceinline__ uint64_t operand_step(int j, int tile) {
    return MN ? (uint64_t)j * 128 : (uint64_t)((j >> 2) * (tile / 2 / 16) + (j & 3) * 2);
}

// Place of 16-byte chunk c of row r in a store buffer of COLS columns: the 128-
// or 64-byte swizzle of its tensor map, which keeps the writes of a warp's 32
// rows on different banks.
template <int COLS>
__device__ __forceinline__ int out_chunk(int r, int c) {
    return COLS == 64 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// Store of a shared-memory box (the part inside the map's extents).
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* smem, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(smem_u32(smem)), "r"(x), "r"(y), "r"(z)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void tma_store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void tma_store_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t cluster_addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(cluster_addr)
                 : "memory");
    return v;
}

// Bits 15 / 16 of the instruction descriptor: A / B is MN-major.
constexpr uint32_t kIdescAMn = 1u << 15, kIdescBMn = 1u << 16;

struct ExpertTile {
    int e, m0, n0;         // expert, first m of the pair's tile, first n
    int n;                 // columns of D that the MMAs compute, a multiple of 32 up to TN
    int first, count;      // the expert's segment
};

// Tiles of an expert along n.  forward / dgrad: the segment's 32-row units in
// nearly equal parts of at most TN (the MMAs' time follows N): 1030 rows are
// 33 units in tiles of 224, 224, 224, 192 and 192 rows.
template <int TN>
__device__ __forceinline__ int n_tiles(int extent) { return (extent + TN - 1) / TN; }

// The tile list: experts in order, an expert's tiles in groups of kMGroup m
// tiles, n outer and m inner, so that the pairs running at a time share both
// operands in L2.  s_end[e] = tiles of experts 0..e.
template <int TN, bool WGRAD>
__device__ __forceinline__ ExpertTile expert_tile(const ExpertParams& p, int tile, const int* s_end,
                                                  const int* s_first, const int* s_count) {
    int lo = 0, hi = p.E - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (tile < s_end[mid]) hi = mid;
        else lo = mid + 1;
    }
    ExpertTile t;
    t.e = lo;
    t.first = s_first[lo];
    t.count = s_count[lo];
    const int local = tile - (lo ? s_end[lo - 1] : 0);
    const int mt = (p.m_extent + 2 * p.half_m - 1) / (2 * p.half_m);
    const int extent = WGRAD ? p.n_extent : t.count;
    const int nt = n_tiles<TN>(extent);
    const int g = local / (kMGroup * nt), in = local % (kMGroup * nt);
    const int gm = min(kMGroup, mt - g * kMGroup);
    const int i = in / gm;
    if (WGRAD) {
        t.n0 = i * TN;
        t.n = min(TN, (extent - t.n0 + 31) / 32 * 32);
    } else {
        const int units = (extent + 31) / 32, per = units / nt, more = units % nt;
        t.n0 = 32 * (i * per + min(i, more));
        t.n = 32 * (per + (i < more ? 1 : 0));
    }
    t.m0 = (g * kMGroup + in % gm) * 2 * p.half_m;
    return t;
}

// SPLIT: a cluster of p.split pairs per tile, the depth divided.
template <int PRODUCT, int TN, int DEPTH, bool SPLIT>
__global__ void __launch_bounds__(ExpertCfg<PRODUCT, TN, DEPTH>::kThreads, 1)
    expert_linear_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                         const __grid_constant__ CUtensorMap tmC, const ExpertParams p) {
    using C = ExpertCfg<PRODUCT, TN, DEPTH>;
    constexpr bool kWgrad = PRODUCT == kExpertWgrad;
    constexpr bool kAMn = PRODUCT != kExpertForward;      // A's m contiguous
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* s_a = base;
    // bytes of a stage's A: its rows, in 128-byte chunks, or the full tile
    const int a_tile = kAMn ? C::kTileA : p.half_m * DEPTH * 2;
    const int stages = kAMn ? C::kStages : p.stages;
    uint8_t* s_b = s_a + stages * a_tile;
    uint8_t* s_out = s_a + C::kStages * (C::kTileA + C::kTileB);
    uint64_t* full = reinterpret_cast<uint64_t*>(s_out + C::kOut);                // rank 0: a stage of both CTAs
    uint64_t* empty = full + C::kMaxStages;                                       // both: the stage's MMAs are done
    uint64_t* landed = empty + C::kMaxStages;                                     // own copies of a stage to be cut
    uint64_t* acc_full = landed + C::kMaxStages;
    uint64_t* acc_empty = acc_full + 2;                                           // rank 0
    uint64_t* drain = acc_empty + 2;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort = reinterpret_cast<volatile int*>(tmem_holder + 1);
    int* s_end = reinterpret_cast<int*>(tmem_holder + 4);
    int* s_first = s_end + kMaxExperts;
    int* s_count = s_first + kMaxExperts;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t cta = cluster_cta_rank();
    const uint32_t rank = SPLIT ? cta & 1 : cta, leader = SPLIT ? cta & ~1u : 0;   // rank: in the pair
    const int slot = SPLIT ? blockIdx.x / (2 * p.split) : blockIdx.x >> 1;
    const int slots = SPLIT ? gridDim.x / (2 * p.split) : gridDim.x >> 1;
    volatile int no_abort = 0;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kMaxStages; ++i) {
            mbar_init(&full[i], 2);        // one arrival per CTA
            mbar_init(&empty[i], 1);
            mbar_init(&landed[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 2 * C::kEpiWarps);
        }
        mbar_init(drain, 1);
        *abort = 0;
        fence_mbar_init();
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmB);
        if (kWgrad) prefetch_tensormap(&tmC);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_holder, C::kTmemCols);
        tmem_relinquish_pair();
    }
    pdl_wait();
    {
        const int mt = (p.m_extent + 2 * p.half_m - 1) / (2 * p.half_m);
        for (int e = threadIdx.x; e < p.E; e += C::kThreads) {
            int64_t first = p.offsets[e], n = p.count[e];
            if (n < 0 || first < 0 || first + n > p.rows) {
                if (p.status && blockIdx.x == 0) atomicOr(p.status, kStatusBadRow);
                first = n = 0;
            }
            s_first[e] = (int)first;
            s_count[e] = (int)n;
            s_end[e] = mt * n_tiles<TN>(kWgrad ? p.n_extent : (int)n);
        }
        __syncthreads();
        if (warp == 0) {
            const int per = (p.E + 31) / 32, e0 = min(p.E, lane * per), e1 = min(p.E, e0 + per);
            int sum = 0;
            for (int e = e0; e < e1; ++e) sum += s_end[e];
            int incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int a = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += a;
            }
            int run = incl - sum;
            for (int e = e0; e < e1; ++e) {
                run += s_end[e];
                s_end[e] = run;
            }
        }
    }
    // both CTAs' barriers initialized and tensor memory allocated before any
    // cross-CTA copy, arrival or pair MMA
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    // a cluster that splits the depth has one tile at most (its ring holds the
    // sums then): the grid has room for every tile of counts that add up to rows
    const int total = SPLIT ? min(s_end[p.E - 1], slots) : s_end[p.E - 1];
    if (SPLIT && total < s_end[p.E - 1] && p.status && blockIdx.x == 0 && threadIdx.x == 0)
        atomicOr(p.status, kStatusBadRow);
    // this pair's part of a tile's depth, in whole stages
    auto part_of = [&](int depth, int& d0, int& d1) {
        d0 = 0;
        d1 = depth;
        if (SPLIT) {
            const int blocks = (depth + DEPTH - 1) / DEPTH, part = (int)cta >> 1;
            d0 = min(depth, blocks * part / p.split * DEPTH);
            d1 = min(depth, blocks * (part + 1) / p.split * DEPTH);
        }
    };
    // The tiles of wgrad are short (as deep as a segment has rows): its producer
    // and MMA issuer work out the next tile's place while a stage of the current
    // one is queued (64 ragged experts 77 -> 72 us; no gain for the others).
    auto tile_or_none = [&](int tile) {
        return tile < total ? expert_tile<TN, kWgrad>(p, tile, s_end, s_first, s_count) : ExpertTile{};
    };

    // the epilogue warps' parts of a tile
    const int q = warp & 3;                            // tensor-memory lane quadrant
    constexpr int kGroups = C::kEpiWarps / 4;
    constexpr int kCols = TN / kGroups;                // accumulator columns per warp
    const int group = (warp - 4) >> 2, col0 = group * kCols;
    auto row_of = [&](const ExpertTile& t) { return t.m0 + (int)rank * p.half_m + q * 32; };   // the warp's first D row
    auto limit_of = [&](const ExpertTile& t) {         // columns that exist
        return min(t.n, (kWgrad ? p.n_extent : t.count) - t.n0);
    };
    // wgrad: lane = row of dw[e], columns contiguous: kOutCols of them at a time
    // through shared memory, so that whole sectors or lines leave; the map's
    // extents cut what lies past N or K
    auto put_wgrad = [&](const ExpertTile& t, int c, int mw, auto fetch) {
        uint8_t* out = s_out + (warp - 4) * C::kOutBytes;
#pragma unroll
        for (int h = 0; h < C::kOutCols; h += 32) {
            float v[32];
            fetch(c + h, v);
            if (h == 0) {
                if (lane == 0) tma_store_wait_read();  // the buffer's last store has read it
                __syncwarp();
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float w[8] = {v[8 * j],     v[8 * j + 1], v[8 * j + 2], v[8 * j + 3],
                                    v[8 * j + 4], v[8 * j + 5], v[8 * j + 6], v[8 * j + 7]};
                *reinterpret_cast<uint4*>(out + out_chunk<C::kOutCols>(lane, h / 8 + j)) = pack_bf16x8(w);
            }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) tma_store_3d(&tmC, out, t.n0 + c, mw, t.e);
    };
    // forward, dgrad: lane = output column, accumulator column = row of the segment
    auto put_rows = [&](const ExpertTile& t, int c, int mw, int limit, bool m_there, const auto& v) {
        constexpr int kCount = sizeof(v) / sizeof(float);
        __nv_bfloat16* o = p.out + (size_t)(t.first + t.n0 + c) * p.m_extent + mw + lane;
        if (m_there) {
#pragma unroll
            for (int j = 0; j < kCount; ++j)
                if (c + j < limit) o[(size_t)j * p.m_extent] = __float2bfloat16_rn(v[j]);
        }
    };

    if (warp == 0) {
        if (lane == 0) {
            const uint64_t pol = policy_evict_normal();
            const uint32_t full0 = cluster_map(full, leader);
            const uint32_t landed_own = cluster_map(landed, cta);
            int stage = 0;
            uint32_t phase = 0;
            ExpertTile next{};
            if (kWgrad) next = tile_or_none(slot);
            for (int tile = slot; tile < total; tile += slots) {
                const ExpertTile t = kWgrad ? next : tile_or_none(tile);
                const int depth = kWgrad ? t.count : p.depth;
                int d0, d1;
                part_of(depth, d0, d1);
                if (kWgrad && d0 >= d1) next = tile_or_none(tile + slots);
                const int m0 = t.m0 + (int)rank * p.half_m, n0 = t.n0 + (int)rank * (t.n / 2);
                // forward, dgrad: a half of B with no row of the segment is
                // left as it is (its columns of D are not stored)
                const bool b1 = kWgrad || t.n0 + t.n / 2 < t.count;
                const bool b_mine = rank == 0 || b1;
                // MN-major chunks that hold an m (or n) of the tile; the others are left too
                const int a_pair = min(2 * (kHalfM / 64), (p.m_extent - t.m0 + 63) / 64);
                const int a_mine = max(0, min(kHalfM / 64, a_pair - (int)rank * (kHalfM / 64)));
                const int b_chunks = (t.n / 2 + 63) / 64;
                for (int d = d0; d < d1; d += DEPTH) {
                    // completed by rank 0's commit: acquire at cluster scope
                    if (!mbar_wait<true>(&empty[stage], phase ^ 1u, abort, p.status, kStatusTimeoutProducer)) goto done;
                    uint8_t* a_dst = s_a + stage * a_tile;
                    uint8_t* b_dst = s_b + stage * C::kTileB;
                    // a stage to be cut: counted on this CTA's own barrier,
                    // and warp 3 announces it
                    const bool cut = kWgrad && depth - d < DEPTH && (depth & 15) != 0;
                    const int chunks = depth - d > 64 ? 2 : 1;             // of K-major rows
                    const uint32_t a_both = kAMn ? a_pair * C::kChunkMn : 2 * chunks * p.half_m * 128;
                    const uint32_t b_bytes = kWgrad ? b_chunks * C::kChunkMn : chunks * p.box_n * 128;
                    const uint32_t bar = (cut ? landed_own : full0) + (uint32_t)stage * 8u;
                    if (cut) mbar_arrive_expect_tx(&landed[stage], a_mine * C::kChunkMn + b_bytes);
                    else if (rank == 0) mbar_arrive_expect_tx(&full[stage], a_both + (b1 ? 2u : 1u) * b_bytes);
                    else mbar_arrive_cluster(full0 + (uint32_t)stage * 8u);
                    if (kAMn) {
#pragma unroll
                        for (int j = 0; j < kHalfM / 64; ++j) {
                            if (j >= a_mine) break;
                            if (kWgrad) tma_load_2d_pair(a_dst + j * C::kChunkMn, &tmA, bar, m0 + 64 * j, t.first + d, pol);
                            else tma_load_3d_pair(a_dst + j * C::kChunkMn, &tmA, bar, m0 + 64 * j, d, t.e, pol);
                        }
                    } else {
                        for (int c = 0; c < chunks; ++c)
                            tma_load_3d_pair(a_dst + c * (a_tile / 2), &tmA, bar, d + 64 * c, m0, t.e, pol);
                    }
                    if (kWgrad) {
#pragma unroll
                        for (int j = 0; j < C::kHalfN / 64; ++j)
                            if (j < b_chunks) tma_load_2d_pair(b_dst + j * C::kChunkMn, &tmB, bar, n0 + 64 * j, t.first + d, pol);
                    } else if (b_mine) {
                        for (int c = 0; c < chunks; ++c)
                            tma_load_2d_pair(b_dst + c * (C::kTileB / 2), &tmB, bar, d + 64 * c, t.first + n0, pol);
                    }
                    if (++stage == stages) { stage = 0; phase ^= 1u; }
                    if (kWgrad && d == d0) next = tile_or_none(tile + slots);
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            constexpr uint32_t kMajor = (kAMn ? kIdescAMn : 0u) | (kWgrad ? kIdescBMn : 0u);
            int stage = 0, acc = 0;
            uint32_t phase = 0, acc_phase = 0;
            ExpertTile next{};
            if (kWgrad) next = tile_or_none(slot);
            for (int tile = slot; tile < total; tile += slots) {
                const ExpertTile t = kWgrad ? next : tile_or_none(tile);
                const int depth = kWgrad ? t.count : p.depth;
                int d0, d1;
                part_of(depth, d0, d1);
                if (d0 >= d1) {
                    if (kWgrad) next = tile_or_none(tile + slots);
                    continue;
                }
                if (!mbar_wait<true>(&acc_empty[acc], acc_phase ^ 1u, abort, p.status, kStatusTimeoutMma)) goto done;
                tc_fence_after();
                const uint32_t idesc = idesc_bf16(256, t.n) | kMajor;
                const uint32_t d_tmem = tmem_base + (uint32_t)acc * TN;
                for (int d = d0; d < d1; d += DEPTH) {
                    if (!mbar_wait<true>(&full[stage], phase, abort, p.status, kStatusTimeoutMma)) goto done;
                    tc_fence_after();
                    const uint32_t a_s = smem_u32(s_a + stage * a_tile), b_s = smem_u32(s_b + stage * C::kTileB);
                    const uint64_t adesc = kAMn ? sdesc_mnmajor_sw128(a_s, C::kChunkMn) : sdesc_kmajor_sw128(a_s);
                    const uint64_t bdesc = kWgrad ? sdesc_mnmajor_sw128(b_s, C::kChunkMn) : sdesc_kmajor_sw128(b_s);
                    if (depth - d >= DEPTH) {
#pragma unroll
                        for (int j = 0; j < DEPTH / 16; ++j)
                            tc_mma_bf16_pair(d_tmem, adesc + operand_step<kAMn>(j, a_tile),
                                             bdesc + operand_step<kWgrad>(j, C::kTileB), idesc, ((d - d0) | j) != 0);
                    } else {
                        for (int j = 0; j < (depth - d + 15) / 16; ++j)
                            tc_mma_bf16_pair(d_tmem, adesc + operand_step<kAMn>(j, a_tile),
                                             bdesc + operand_step<kWgrad>(j, C::kTileB), idesc, ((d - d0) | j) != 0);
                    }
                    tc_commit_pair_mc(&empty[stage], (uint16_t)(0x3 << leader));
                    if (++stage == stages) { stage = 0; phase ^= 1u; }
                    if (kWgrad && d == d0) next = tile_or_none(tile + slots);
                }
                tc_commit_pair_mc(&acc_full[acc], (uint16_t)(0x3 << leader));
                acc ^= 1;
                if (acc == 0) acc_phase ^= 1u;
            }
        }
    } else if (warp == 3) {
        if (kWgrad) {
            // the ragged ends: zeros from the segment's end to the end of its
            // last 16-row step, in this CTA's halves of both operands
            const uint32_t full0 = cluster_map(full, leader);
            int stage = 0;
            uint32_t phases = 0;           // bit s: parity of landed[s]
            for (int tile = slot; tile < total; tile += slots) {
                const ExpertTile t = expert_tile<TN, kWgrad>(p, tile, s_end, s_first, s_count);
                int d0, d1;
                part_of(t.count, d0, d1);
                const int blocks = (d1 - d0 + DEPTH - 1) / DEPTH;
                if ((t.count & 15) != 0 && d1 == t.count && d0 < d1) {
                    const int s = (stage + blocks - 1) % C::kStages;
                    if (!__all_sync(0xffffffffu, mbar_wait(&landed[s], (phases >> s) & 1u, abort, p.status,
                                                           kStatusTimeoutProducer)))
                        goto done;
                    phases ^= 1u << s;
                    const int r0 = t.count - d0 - (blocks - 1) * DEPTH, r1 = (r0 + 15) / 16 * 16;
                    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
                    // a row of a chunk is 128 bytes (the swizzle permutes within it)
                    for (int r = r0 + (lane >> 3); r < r1; r += 4) {
#pragma unroll
                        for (int j = 0; j < kHalfM / 64; ++j)
                            *reinterpret_cast<uint4*>(s_a + s * C::kTileA + j * C::kChunkMn + r * 128 + (lane & 7) * 16) = zero;
#pragma unroll
                        for (int j = 0; j < C::kHalfN / 64; ++j)
                            *reinterpret_cast<uint4*>(s_b + s * C::kTileB + j * C::kChunkMn + r * 128 + (lane & 7) * 16) = zero;
                    }
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) {
                        if (rank == 0) mbar_arrive(&full[s]);
                        else mbar_arrive_remote_cta_release(full0 + (uint32_t)s * 8u);
                    }
                }
                stage = (stage + blocks) % C::kStages;
            }
        }
    } else if (warp >= 4) {
        const uint32_t release0 = cluster_map(acc_empty, leader);
        int acc = 0;
        uint32_t acc_phase = 0;
        for (int tile = slot; tile < total; tile += slots) {
            const ExpertTile t = expert_tile<TN, kWgrad>(p, tile, s_end, s_first, s_count);
            int d0, d1;
            part_of(kWgrad ? t.count : p.depth, d0, d1);
            const int mw = row_of(t), limit = limit_of(t);
            const bool nothing = (kWgrad || SPLIT) && d0 >= d1;      // zeros, no accumulator
            if (!nothing) {
                // warp-uniform outcome: tcgen05.ld below is a warp-collective instruction
                if (!__all_sync(0xffffffffu, mbar_wait<true>(&acc_full[acc], acc_phase, abort, p.status,
                                                             kStatusTimeoutEpilogue)))
                    break;
                tc_fence_after();
            }
            const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)acc * TN;
            auto fetch = [&](int col, float (&v)[32]) {
                if (nothing) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = 0.0f;
                } else {
                    tmem_ld32(taddr + (uint32_t)col, v);
                    tmem_ld_wait();
                }
            };
            if constexpr (SPLIT) {
                // the sums of this part, [column / 4][row][4], over the ring: its
                // last stage has been read
                for (int c = col0; c < col0 + kCols && c < t.n; c += 32) {
                    float v[32];
                    fetch(c, v);
                    float4* sums = reinterpret_cast<float4*>(s_a) + c / 4 * kHalfM + q * 32 + lane;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        sums[j * kHalfM] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                }
            } else if constexpr (kWgrad) {
#pragma unroll 1
                for (int c = 0; c < kCols; c += C::kOutCols) {
                    if (col0 + c >= limit || mw >= p.m_extent) break;      // warp-uniform
                    put_wgrad(t, col0 + c, mw, fetch);
                }
            } else {
#pragma unroll 1
                for (int c = 0; c < kCols; c += 32) {
                    if (col0 + c >= limit) break;          // warp-uniform
                    float v[32];
                    tmem_ld32(taddr + (uint32_t)(col0 + c), v);
                    tmem_ld_wait();
                    // lane = output column, accumulator column = row of the segment:
                    // 32 columns of a row side by side, and 16 bytes of it a lane
                    // (8729 rows of 4152 x 640: 42.6 -> 39.3 us; 2047 of 760 x 96: 10.7 -> 7.9)
#pragma unroll
                    for (int h = 0; h < 32; h += C::kOutRows) {
                        uint8_t* out = s_out + (warp - 4) * C::kOutBytes;
#pragma unroll
                        for (int j = 0; j < C::kOutRows; ++j)
                            *reinterpret_cast<__nv_bfloat16*>(out + j * 64 + lane * 2) = __float2bfloat16_rn(v[h + j]);
                        __syncwarp();
                        const int at = (lane & 3) * 8;
                        const bool there = q * 32 + at < p.half_m && mw + at < p.m_extent;
#pragma unroll
                        for (int i = 0; i < C::kOutRows; i += 8) {
                            const int n = col0 + c + h + i + (lane >> 2);
                            if (there && n < limit)
                                *reinterpret_cast<uint4*>(p.out + (size_t)(t.first + t.n0 + n) * p.m_extent + mw + at) =
                                    *reinterpret_cast<const uint4*>(out + (i + (lane >> 2)) * 64 + at * 2);
                        }
                        __syncwarp();
                    }
                }
            }
            if (!nothing) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (rank == 0) mbar_arrive(&acc_empty[acc]);
                    else mbar_arrive_cluster(release0 + (uint32_t)acc * 8u);
                }
                acc ^= 1;
                if (acc == 0) acc_phase ^= 1u;
            }
        }
        if (kWgrad && lane == 0) tma_store_wait();
    }
done:
    if (*abort) {
        // tell the other CTA, let in-flight copies land and retire every
        // issued MMA before the memories go away
        st_cluster_u32(cluster_map((const void*)abort, cta ^ 1u), 1u);
        if (warp == 1 && lane == 0 && rank == 0) {
            tc_commit_pair(drain);
            mbar_wait(drain, 0, &no_abort, p.status, kStatusTimeoutMma);
        }
        for (int i = 0; i < 100; ++i) __nanosleep(10000);
    }
    if constexpr (SPLIT) {
        // all parts' sums lie in their CTAs' shared memory: each pair adds up and
        // stores its share of the columns, the parts in order
        __syncthreads();
        cluster_sync_all();
        if (warp >= 4 && slot < total) {
            const ExpertTile t = expert_tile<TN, kWgrad>(p, slot, s_end, s_first, s_count);
            auto fetch = [&](int col, auto& v) {
                constexpr int kCount = sizeof(v) / sizeof(float);
#pragma unroll
                for (int j = 0; j < kCount; ++j) v[j] = 0.0f;
#pragma unroll
                for (uint32_t s = 0; s < 4; ++s)
                    if (s < (uint32_t)p.split) {
                        const uint32_t from = cluster_map(s_a, 2 * s + rank) + (uint32_t)(col / 4 * kHalfM + q * 32 + lane) * 16u;
#pragma unroll
                        for (int j = 0; j < kCount / 4; ++j) {
                            const float4 w = ld_cluster_f32x4(from + (uint32_t)(j * kHalfM * 16));
                            v[4 * j] += w.x;
                            v[4 * j + 1] += w.y;
                            v[4 * j + 2] += w.z;
                            v[4 * j + 3] += w.w;
                        }
                    }
            };
            constexpr int kUnit = kWgrad ? C::kOutCols : 8;
            const int mw = row_of(t), limit = limit_of(t);
            const bool m_there = q * 32 + lane < p.half_m && mw + lane < p.m_extent;
            const int unit0 = ((int)cta >> 1) * kGroups + group;
#pragma unroll 1
            for (int c = unit0 * kUnit; c < limit; c += p.split * kGroups * kUnit) {
                if constexpr (kWgrad) {
                    if (mw < p.m_extent) put_wgrad(t, c, mw, fetch);
                } else {
                    float v[kUnit];
                    fetch(c, v);
                    put_rows(t, c, mw, limit, m_there, v);
                }
            }
            if (kWgrad && lane == 0) tma_store_wait();
        }
    }
    tc_fence_before();
    __syncthreads();
    // no CTA frees tensor memory or leaves before all are done
    cluster_sync_all();
    pdl_launch_dependents();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, C::kTmemCols);
    }
}

// No rows at all: a segment with some, or one that starts elsewhere than at 0,
// is reported as by the kernel above.
__global__ void __launch_bounds__(256) segment_check_kernel(int E, const int* count, const int* offsets,
                                                            unsigned int* status) {
    pdl_wait();
    for (int e = threadIdx.x; e < E; e += 256) {
        const int64_t first = offsets[e], n = count[e];
        if (n < 0 || first < 0 || first + n > 0) atomicOr(status, kStatusBadRow);
    }
    pdl_launch_dependents();
}

// Tensor map of a BF16 array: dims[0] contiguous, byte strides of the others,
// boxes as wide as the swizzle.
bool encode_bf16_map(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                     const cuuint32_t* box, CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
    const cuuint32_t step[3] = {1, 1, 1};
    return tensor_map_encoder()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box,
                                step, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int g_expert_grid[64] = {};
int g_expert_clusters[64][3] = {};     // clusters of 1, 2 and 4 pairs that run at a time

template <int PRODUCT, int TN, int DEPTH>
cudaError_t launch_tiles(const LaunchCtx& c, int grid, const CUtensorMap& a, const CUtensorMap& b,
                         const CUtensorMap& d, ExpertParams p) {
    // A's last chunk is read as 128 rows: what lies past its own is B's ring
    using C = ExpertCfg<PRODUCT, TN, DEPTH>;
    const int fit = C::kStages * (C::kTileA + C::kTileB) / (p.half_m * DEPTH * 2 + C::kTileB);
    p.stages = fit < C::kMaxStages ? fit : C::kMaxStages;
    // the shallow wgrad is not split: the deep one has the few tiles
    const auto kernel = p.split > 1 ? expert_linear_kernel<PRODUCT, TN, DEPTH, DEPTH == 128>
                                    : expert_linear_kernel<PRODUCT, TN, DEPTH, false>;
    return c.launch(kernel, dim3((unsigned)grid), dim3(C::kThreads), (size_t)C::kSmemBytes, a, b, d, p);
}

template <int PRODUCT, int TN, int DEPTH, bool SPLIT>
cudaError_t set_tiles() {
    return cudaFuncSetAttribute(expert_linear_kernel<PRODUCT, TN, DEPTH, SPLIT>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, ExpertCfg<PRODUCT, TN, DEPTH>::kSmemBytes);
}
template <int PRODUCT, bool SPLIT>
cudaError_t set_rows() {
    cudaError_t e;
    if ((e = set_tiles<PRODUCT, 32, 128, SPLIT>()) || (e = set_tiles<PRODUCT, 64, 128, SPLIT>()) ||
        (e = set_tiles<PRODUCT, 128, 128, SPLIT>()) || (e = set_tiles<PRODUCT, 256, 128, SPLIT>()))
        return e;
    return cudaSuccess;
}

template <int PRODUCT>
cudaError_t launch_rows(const LaunchCtx& c, int tn, int grid, const CUtensorMap& a, const CUtensorMap& b,
                        const ExpertParams& p) {
    switch (tn) {
        case 32: return launch_tiles<PRODUCT, 32, 128>(c, grid, a, b, b, p);
        case 64: return launch_tiles<PRODUCT, 64, 128>(c, grid, a, b, b, p);
        case 128: return launch_tiles<PRODUCT, 128, 128>(c, grid, a, b, b, p);
        default: return launch_tiles<PRODUCT, 256, 128>(c, grid, a, b, b, p);
    }
}

// Rows of a tile (its TN) for segments of `mean` rows on average.  Measured on
// GB300 (dgrad, 16 experts of 4096 x 7168; us at TN = 32, 64, 128, 256):
//   4 rows 138 138 139 186;  16 rows 147 140 141 152;  32 rows 186 147 143 149;
//   64 rows 316 195 151 150;  128 rows 542 300 194 161.
// Where the tiles leave pairs idle see Split.
int tile_rows(double mean) { return mean <= 8 ? 32 : mean <= 20 ? 64 : mean <= 80 ? 128 : 256; }

// Few tiles: their rows, and the pairs that share a tile's depth (1: none do).
struct Split {
    int tn, pairs;
};

// While the tiles leave pairs idle the time is one tile's: 5 us and then 0.44 us
// a stage of 128 (0.6 at 256 rows).  Lower tiles, and a cluster of two or four
// pairs for each, the depth divided, take what pairs there are; the join costs
// 1.5 us and more for the sums that cross the cluster.  The least of the times
// by these measured figures.  Measured on GB300 (us for 1, 2 and 4 pairs):
//   forward 64 rows of 1024 x 7168: 29.9 19.0 12.8;  2 x 291 rows of 120 x 3680:
//   17.8 13.3 11.0;  34 rows of 88 x 688: 7.4 7.7 7.1;  dgrad 64 rows of 7168 x
//   1024: 28.8 18.4 12.3;  wgrad 16384 rows of 256 x 256: 73 43 28;  2 x 912 rows
//   of 176 x 168: 11.1 11.3 12.0.
Split split_of(bool wgrad, int tn, int n_extent, double mean, int64_t rows, int64_t busy, int E, int m_tiles, int depth,
               const int* clusters) {
    Split best{tn, 1};
    double best_us = 1e30;
    const double stages = ceil(depth / 128.0);
    for (int i = 0; i < 3; ++i)
        for (int t = tn; t >= (wgrad ? 256 : 32); t /= 2) {
            // a split tile has a cluster of its own: as many as there can be
            const int64_t tiles = m_tiles * (wgrad ? E * (int64_t)((n_extent + 255) / 256)
                                             : i   ? busy + (rows - busy) / t
                                                   : busy * (int64_t)ceil(mean / t));
            if (tiles > clusters[i]) continue;
            const int width = wgrad && n_extent < 256 ? n_extent : t;
            double us = 0.44 + (width > 64 ? 0.0009 * (width - 64) : 0.0);
            if (t == 32 && i == 0 && tiles > clusters[0] / 2) us += 0.02;      // more copies of the weights at a time
            us *= ceil(stages / (1 << i));
            if (i) us += 1.4 + (wgrad ? 0.0045 * (1 << i) : 0.007) * width;
            if (us < best_us || (us == best_us && i == 0)) {
                best = Split{t, 1 << i};
                best_us = us;
            }
        }
    return best;
}

// Rows per busy expert from which wgrad takes the deep stages.  Measured on GB300
// (16 experts of 4096 x 7168; us shallow, deep): 4 rows 143 181;  128 rows 171
// 189;  256 rows 240 239;  384 rows 330 317;  1024 rows 665 652.  Also where the
// tiles leave pairs idle.
constexpr int kWgradDeepRows = 300;

// D rows per CTA (forward with narrow tiles, where the weights' bytes bound the
// time and an MMA row without a weight costs nothing): the height, in steps of
// eight rows, with the least work for the busiest pair if every busy expert
// has one tile of rows.  8 experts of 4096 rows on 76 pairs: 16 tiles of 256
// rows each are 128 tiles, two rounds of 128 rows per CTA; 19 tiles of 224
// are 152, two rounds of 112 (4096 x 7168: 88 -> 76 us).  A tile costs about a
// microsecond besides, the copies of kTileCost elements: 45 experts of 6520 x
// 416 took 77 us in 32 rounds of 64 rows.
constexpr int kTileCost = 22000;
int tile_height(int m_extent, int depth, int64_t row_tiles, int pairs) {
    int best = kHalfM;
    int64_t best_work = INT64_MAX;
    for (int h = kHalfM; h >= 64; h -= 8) {
        const int64_t tiles = row_tiles * ((m_extent + 2 * h - 1) / (2 * h));
        const int64_t work = (tiles + pairs - 1) / pairs * ((int64_t)h * depth + kTileCost);
        if (work < best_work) {
            best = h;
            best_work = work;
        }
    }
    return best;
}

}  // namespace

cudaError_t setup_expert_linear_kernels(int device, int num_sms) {
    cudaError_t e;
    if ((e = set_rows<kExpertForward, false>()) || (e = set_rows<kExpertForward, true>()) ||
        (e = set_rows<kExpertDgrad, false>()) || (e = set_rows<kExpertDgrad, true>()) ||
        (e = set_tiles<kExpertWgrad, 256, 128, false>()) || (e = set_tiles<kExpertWgrad, 256, 128, true>()) ||
        (e = set_tiles<kExpertWgrad, 256, 64, false>()))
        return e;
    // persistent grid: as many CTA pairs as can be resident at once
    if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
    for (int i = 0; i < 3; ++i) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(num_sms / (2 << i) * (2 << i)));
        cfg.blockDim = dim3(ExpertCfg<kExpertForward, 64, 128>::kThreads);
        cfg.dynamicSmemBytes = ExpertCfg<kExpertForward, 64, 128>::kSmemBytes;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2 << i;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int clusters = 0;
        if ((e = cudaOccupancyMaxActiveClusters(
                 &clusters, i ? expert_linear_kernel<kExpertForward, 64, 128, true>
                              : expert_linear_kernel<kExpertForward, 64, 128, false>, &cfg))) return e;
        g_expert_clusters[device][i] = clusters < num_sms / (2 << i) ? clusters : num_sms / (2 << i);
    }
    if (g_expert_clusters[device][0] < 1) return cudaErrorInvalidConfiguration;
    g_expert_grid[device] = 2 * g_expert_clusters[device][0];
    return cudaSuccess;
}

cudaError_t launch_expert_linear(const LaunchCtx& c, int product, int device, const ExpertArgs& a) {
    if (device < 0 || device >= 64 || g_expert_grid[device] < 2) return cudaErrorInvalidValue;
    if (a.rows == 0) {
        cudaError_t e = cudaSuccess;
        if (a.status) e = c.launch(segment_check_kernel, dim3(1), dim3(256), 0, a.E, a.count, a.offsets, a.status);
        if (e == cudaSuccess && product == kExpertWgrad)    // a gradient of zeros
            e = cudaMemsetAsync(a.out, 0, (size_t)a.E * a.N * a.K * 2, c.stream);
        return e;
    }
    const cuuint64_t N = (cuuint64_t)a.N, K = (cuuint64_t)a.K, R = (cuuint64_t)a.rows;
    const int64_t busy = a.rows < a.E ? a.rows : a.E;
    const double mean = (double)a.rows / (double)busy;
    const int pairs = g_expert_grid[device] / 2;
    const int m_tiles = ((product == kExpertDgrad ? a.K : a.N) + 255) / 256;
    const bool is_wgrad = product == kExpertWgrad;
    const Split sp = split_of(is_wgrad, is_wgrad ? 256 : tile_rows(mean), a.K, mean, a.rows, busy, a.E, m_tiles,
                              is_wgrad ? (int)ceil(mean) : product == kExpertDgrad ? a.N : a.K, g_expert_clusters[device]);
    const int tn = sp.tn;
    const bool wgrad_deep = mean >= kWgradDeepRows || busy * m_tiles * ((a.K + 255) / 256) <= pairs;
    ExpertParams p{};
    p.half_m = kHalfM;
    CUtensorMap ta, tb, td;
    bool ok;
    if (product == kExpertWgrad) {
        const cuuint64_t da[2] = {N, R}, sa[1] = {N * 2}, db[2] = {K, R}, sb[1] = {K * 2};
        const cuuint32_t box[2] = {64, wgrad_deep ? 128u : 64u};
        const cuuint64_t dd[3] = {K, N, (cuuint64_t)a.E}, sd[2] = {K * 2, N * K * 2};
        const cuuint32_t boxd[3] = {wgrad_deep ? 32u : 64u, 32, 1};
        ok = encode_bf16_map(&ta, a.a, 2, da, sa, box) && encode_bf16_map(&tb, a.b, 2, db, sb, box) &&
             encode_bf16_map(&td, a.out, 3, dd, sd, boxd,
                             wgrad_deep ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
    } else {
        const bool fwd = product == kExpertForward;
        const cuuint64_t dw[3] = {K, N, (cuuint64_t)a.E}, sw[2] = {K * 2, N * K * 2};
        if (fwd && sp.pairs > 1) p.half_m = (a.N + 16 * m_tiles - 1) / (16 * m_tiles) * 8;
        else if (fwd && tn < 256) p.half_m = tile_height(a.N, a.K, busy * (int64_t)ceil(mean / tn), pairs);
        // no more rows than there are: the copies of one token's rows are short
        p.box_n = (int)(a.rows < tn / 2 ? (a.rows + 7) / 8 * 8 : tn / 2);
        const cuuint32_t boxw[3] = {64, fwd ? (cuuint32_t)p.half_m : 128u, 1};
        const cuuint64_t dr[2] = {fwd ? K : N, R}, sr[1] = {(fwd ? K : N) * 2};
        const cuuint32_t boxr[2] = {64, (cuuint32_t)p.box_n};
        ok = encode_bf16_map(&ta, a.b, 3, dw, sw, boxw) && encode_bf16_map(&tb, a.a, 2, dr, sr, boxr);
    }
    if (!ok) return cudaErrorInvalidValue;
    p.m_extent = product == kExpertDgrad ? a.K : a.N;
    p.n_extent = a.K;
    p.depth = product == kExpertDgrad ? a.N : a.K;
    p.E = a.E;
    p.rows = a.rows;
    p.count = a.count;
    p.offsets = a.offsets;
    p.out = static_cast<__nv_bfloat16*>(a.out);
    p.status = a.status;
    p.split = sp.pairs;
    LaunchCtx cc = c;
    cc.cluster = 2 * sp.pairs;
    // a split tile has a cluster of its own
    const int64_t tiles = (int64_t)((p.m_extent + 2 * p.half_m - 1) / (2 * p.half_m)) *
                          (is_wgrad ? a.E * (int64_t)((a.K + 255) / 256) : busy + (a.rows - busy) / tn);
    const int grid = sp.pairs > 1 ? (int)(2 * sp.pairs * tiles) : g_expert_grid[device];
    if (product == kExpertForward) return launch_rows<kExpertForward>(cc, tn, grid, ta, tb, p);
    if (product == kExpertDgrad) return launch_rows<kExpertDgrad>(cc, tn, grid, ta, tb, p);
    return wgrad_deep ? launch_tiles<kExpertWgrad, 256, 128>(cc, grid, ta, tb, td, p)
                      : launch_tiles<kExpertWgrad, 256, 64>(cc, grid, ta, tb, td, p);
}

}  // namespace moe
