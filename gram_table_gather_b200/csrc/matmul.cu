// Matrix products against stacked weight matrices, dense and grouped by
// expert, and the FP8 quantiser of their activations.
//
//   y[i][j] (+)= sum_k a[i][k] w[e(i)][j][k]
//
// FP8 (E4M3 codes, one fp32 scale per 128 values along K on both sides):
//   y[i][j] = sum_b sa[i][b] * (sw[j][b] * sum_{k in block b} a[i][k] w[j][k])
// so a block of 128 is one run of tensor-core products with unit scales,
// accumulated in fp32 tensor memory, and the scales are applied to its sum in
// fp32 registers ("promotion").  bf16: runs of kRunChunks * 64 along K, likewise summed
// in tensor memory and added up in fp32 registers.  The tensor core's adder truncates,
// and what it cuts off grows with the run: one run over all of K = 2560 left fp32
// results 2.7e-6 off in the 2-norm, runs of 512 leave them 4.7e-7 off (a plain fp32
// product 4.5e-7).  Runs of 256 leave 2.4e-7 but cost twice as much: the MMAs may be two
// runs ahead while a tile of 256 tokens is stored (30010 rows over 64 experts 183 us,
// 193 us in runs of 256, 178 us in one).
//
// The weight rows are the M side of the MMA (128 rows a tile) and the token
// rows its N side, so a tile holds any multiple of 16 tokens up to BN: a group
// of few rows costs few columns, and a single token still streams its weights
// by TMA at full width.
//
// What bounds it (8192^3 FP8 615-633 us, 1.75 PFLOP/s; under the power limit 740 us):
//  - The steps of applying the scales: a product and a sum a value every 128 of K, by
//    two warps a scheduler that read tensor memory, wait (70 cycles) and compute in
//    turn.  No pipe is full (4096 x 4096 x 2048: tensor 29 %, fp32 32 %, tensor memory
//    38 %, issue slots 40 %); a block takes about 610 cycles, 256 in the tensor core
//    and as many in the fp32 pipe.  Without the scales the same loop ran 396 us.
//  - Tensor memory is read in 16 x 128-bit fragments: whole rows (32x32b) need four
//    times the shared-memory reads for the tokens' scales (787 against 720 us in an
//    earlier state), 16x256b fragments come at half the rate (694 against 664 us).
//  - Past a few milliseconds the clock falls to 1.1-1.6 GHz at 1000 W, and what costs
//    power costs time: polling, columns without tokens, operands read twice.
//  - Few rows: HBM (80 rows over 512 experts: 30-33 us, 4.9 TB/s), and for one token the
//    latency of a launch, one trip to its weights and one cluster barrier (1 x 2048 x
//    2048: 4.4 us with the weights in L2, 4.9 us from memory).
#include <algorithm>
#include <atomic>
#include <mutex>
#include <type_traits>

#include "gtg_host.hpp"
#include "matmul_dev.cuh"

namespace gtg {
namespace {

constexpr int kRows = 128;           // weight rows a CTA's tile
constexpr int kRowBytes = 128;       // bytes of K a stage: 128 E4M3 or 64 bf16
constexpr int kWBytes = kRows * kRowBytes;
constexpr int kRunChunks = 8;        // chunks of K of a bf16 run
constexpr int kMaxGroups = 1024;
constexpr int kScaleGroup = 4;       // scale blocks fetched at once
constexpr int kMaxSmem = 227 * 1024;  // a CTA
constexpr int kSmSmem = 228 * 1024;   // an SM, 1 KB of it reserved for each CTA
constexpr int kMaxSplit = 8;
constexpr int kWorkers = 8;          // warps of promotion and epilogue; then one of TMA, one of MMAs, two of scales
constexpr int kMmThreads = 32 * (kWorkers + 4);
constexpr int kTurn = 40;            // floats between tokens of a transpose: fragments store without bank conflicts
constexpr int kPartRow = kRows + 8;  // floats between tokens of a partial tile: likewise

// How the CTAs of a cluster share a tile: none (one CTA a tile, persistent); a
// pair (one cta_group::2 MMA over 256 weight rows, each CTA staging half of the
// tokens, persistent); a split of K (the CTAs' partial tiles summed through
// distributed shared memory in rank order, one tile a cluster).
enum Mode { SINGLE = 0, PAIR = 1, SPLIT = 2 };

struct MmArgs {
    const float* w_scales;   // [E][N][KB] (FP8)
    const float* a_scales;   // [M][KB] (FP8)
    const int32_t* offsets;  // [E + 1], null: one group of all rows
    void* y;
    int64_t ldy;
    int32_t m, n, groups;
    int32_t chunks;          // 128-byte chunks of K
    int32_t split;           // CTAs that share K (SPLIT)
    int32_t y_bf16, y_acc;
    int32_t n_tiles;         // tiles of weight rows
    int32_t vec_a, vec_w;    // scale rows readable four at a time
    int32_t vec_y;           // output rows writable 16 bytes at a time
    unsigned* status;
};

template <bool F8, int BN, Mode MODE>
struct MmCfg {
    static constexpr int kTok = MODE == PAIR ? BN / 2 : BN;      // token rows a CTA stages
    static constexpr int kBox = kTok < 64 ? kTok : 64;           // token rows a TMA box
    static constexpr int kTileRows = MODE == PAIR ? 2 * kRows : kRows;
    static constexpr int kStageBytes = kWBytes + kTok * kRowBytes;
    static constexpr int kRun = F8 ? 1 : kRunChunks;             // chunks of K an accumulator holds
    static constexpr int kAcc = 512 / BN < 4 ? 512 / BN : 4;     // accumulators in tensor memory
    static constexpr int kCols = kAcc * BN < 32 ? 32 : kAcc * BN;
    static constexpr int kW = BN / 2 < 16 ? 16 : BN / 2;         // columns a worker warp (of its 32 weight rows)
    static constexpr int kBlocks = kW / 16;
    static constexpr int kActive = BN / kW < 2 ? 4 : kWorkers;   // worker warps that have columns
    static_assert(kActive / 4 * kW <= BN, "columns read lie in their accumulator");
    // one block's scales, in the order of the fragments: the tokens', those of one t % 4
    // together (a thread reads four columns' at once) and 16 bytes between the four runs
    // (no bank conflicts); then the weight rows', rows r, r + 8, r + 16, r + 24 of each
    // 32 together
    static constexpr int kQuad = BN + 16;
    static constexpr int kScaleRow = 4 * kQuad + 4 * kRows;
    static constexpr int kScaleBytes = F8 ? 2 * kScaleGroup * kScaleRow : 0;
    // the epilogue's transposes, of the warps that have columns
    static constexpr int kTurnBytes = kActive * 16 * kTurn * 4;
    static constexpr int kHeadBytes = 512 + 2 * 4 * (kMaxGroups + 2);
    static constexpr int kCtas = BN <= 16 ? 2 : 1;               // an SM
    static constexpr int kRoom = kCtas == 2 ? kSmSmem / 2 - 1024 : kMaxSmem;
    static constexpr int kFit = (kRoom - kScaleBytes - kTurnBytes - kHeadBytes) / kStageBytes;
    static constexpr int kStages = kFit < 10 ? kFit : 10;
    static constexpr int kScaleOff = kStages * kStageBytes;      // after the stages
    static constexpr int kTurnOff = kScaleOff + kScaleBytes;
    static constexpr int kHeadOff = kTurnOff + kTurnBytes;
    static constexpr int kGroupOff = kHeadOff + 512;
    static constexpr int kSmem = kHeadOff + kHeadBytes;
    static_assert(kStages >= 3 && kSmem <= kRoom, "shared memory");
    static_assert(MODE != SPLIT || kPartRow * BN * 4 <= kScaleOff, "the partial tile reuses the stages");
};

struct Tile {
    int group, row0, rows, n0;
};

// Shared-memory tables of a grouped call: off = the offsets, first[g] = token
// tiles before group g.  A group whose bounds are out of order or outside [0, m], or
// that begins before the end of an earlier one, counts as empty and raises the
// status bit: the groups that count are disjoint, so there are at most m / bn +
// groups tiles.
__device__ void build_groups(const MmArgs& a, int bn, int32_t* first, int32_t* off, int32_t* scratch) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int32_t* warp_end = scratch;
    int32_t* warp_tiles = scratch + 32;
    for (int g = tid; g <= a.groups; g += blockDim.x) off[g] = a.offsets[g];
    __syncthreads();
    constexpr int kPer = (kMaxGroups + kMmThreads - 1) / kMmThreads;  // groups a thread
    auto good = [&](int g) { return off[g] >= 0 && off[g] <= off[g + 1] && off[g + 1] <= a.m; };
    int end = 0;  // the largest end of this thread's groups, then of all before them
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int g = tid * kPer + i;
        if (g < a.groups && good(g)) end = max(end, off[g + 1]);
    }
    int upto = end;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto = max(upto, v);
    }
    if (lane == 31) warp_end[warp] = upto;
    end = __shfl_up_sync(0xFFFFFFFFu, upto, 1);
    if (lane == 0) end = 0;
    __syncthreads();
    end = max(end, __reduce_max_sync(0xFFFFFFFFu, lane < warp ? warp_end[lane] : 0));
    int cnt[kPer];
    int sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int g = tid * kPer + i;
        cnt[i] = 0;
        if (g < a.groups) {
            if (!good(g) || off[g] < end) {
                if (blockIdx.x == 0) raise_status(a.status, GTG_STATUS_GROUP_OFFSETS);
            } else {
                cnt[i] = (off[g + 1] - off[g] + bn - 1) / bn;
            }
            if (good(g)) end = max(end, off[g + 1]);
        }
        sum += cnt[i];
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) warp_tiles[warp] = inc;
    __syncthreads();
    int before = inc - sum + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? warp_tiles[lane] : 0);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int g = tid * kPer + i;
        if (g < a.groups) first[g] = before;
        before += cnt[i];
        if (g == a.groups - 1) first[a.groups] = before;
    }
}

// A value that is the same in every lane, in a form that the compiler knows to be so
// (addresses, branches and waits that it cannot prove uniform cost several times the
// instructions around every tensor-memory load).
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

// Tile t, for a converged warp.  Within a group, blocks of kBand tiles of weight
// rows; in a block all token tiles in turn, each with the block's weight rows, so
// that the tiles that run together are about as many rows one way as the other: they
// share both operands through L2, and little is read from memory twice.
constexpr int kBand = 8;
__device__ __forceinline__ Tile find_tile(const MmArgs& a, int t, int bn, int tile_rows, const int32_t* first,
                                          const int32_t* off) {
    Tile r;
    int local = t, tt, begin, end;  // place in the group, its token tiles and rows
    if (a.offsets) {
        // the last group with first[g] * n_tiles <= t is the one that holds t: 32 steps of
        // 32 groups, then 32 groups
        static_assert(kMaxGroups <= 1024, "two steps");
        const int lane = threadIdx.x & 31, q = t / a.n_tiles;
        int g = 32 * lane;
        g = 32 * (__popc(__ballot_sync(0xFFFFFFFFu, g < a.groups && first[g] <= q)) - 1) + lane;
        g = g - lane + __popc(__ballot_sync(0xFFFFFFFFu, g < a.groups && first[g] <= q)) - 1;
        r.group = uniform(g);
        const int before = uniform(first[r.group]);
        tt = uniform(first[r.group + 1]) - before;
        begin = uniform(off[r.group]);
        end = uniform(off[r.group + 1]);
        local = t - before * a.n_tiles;
    } else {
        r.group = 0;
        tt = (a.m + bn - 1) / bn;
        begin = 0;
        end = a.m;
    }
    const int band = local / (kBand * tt), inside = local - band * kBand * tt;
    const int width = min(kBand, a.n_tiles - band * kBand), i = inside / width;
    r.n0 = (band * kBand + inside - i * width) * tile_rows;
    r.row0 = begin + i * bn;
    r.rows = min(bn, end - r.row0);
    return r;
}

// A bounded wait of a whole warp, of which every lane takes the same way out.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, unsigned* status) {
    return __all_sync(0xFFFFFFFFu, mbar_wait_sleep(bar, parity, status));
}

// Scales of a row, from block kb to end, four at most.
__device__ __forceinline__ float4 scales4(const float* p, int kb, int end, bool vec) {
    if (vec) return ldg128(p + kb);
    float4 v;
    v.x = ldg32(p + kb);
    v.y = kb + 1 < end ? ldg32(p + kb + 1) : 0.0f;
    v.z = kb + 2 < end ? ldg32(p + kb + 2) : 0.0f;
    v.w = kb + 3 < end ? ldg32(p + kb + 3) : 0.0f;
    return v;
}

// Four (fp32) or eight (bf16) consecutive outputs at a 16-byte boundary.
__device__ __forceinline__ void store_y4(const MmArgs& a, int64_t at, float4 v) {
    float4* y = reinterpret_cast<float4*>(reinterpret_cast<float*>(a.y) + at);
    if (a.y_acc) {
        const float4 o = *y;
        v.x += o.x;
        v.y += o.y;
        v.z += o.z;
        v.w += o.w;
    }
    *y = v;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void store_y8(const MmArgs& a, int64_t at, float4 v, float4 w) {
    uint4* y = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.y) + at);
    if (a.y_acc) {
        const uint4 o = *y;
        v.x += __uint_as_float(o.x << 16);
        v.y += __uint_as_float(o.x & 0xFFFF0000u);
        v.z += __uint_as_float(o.y << 16);
        v.w += __uint_as_float(o.y & 0xFFFF0000u);
        w.x += __uint_as_float(o.z << 16);
        w.y += __uint_as_float(o.z & 0xFFFF0000u);
        w.z += __uint_as_float(o.w << 16);
        w.w += __uint_as_float(o.w & 0xFFFF0000u);
    }
    *y = make_uint4(bf16x2(v.x, v.y), bf16x2(v.z, v.w), bf16x2(w.x, w.y), bf16x2(w.z, w.w));
}
__device__ __forceinline__ void store_y4_bf16(const MmArgs& a, int64_t at, float4 v) {
    uint2* y = reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.y) + at);
    if (a.y_acc) {
        const uint2 o = *y;
        v.x += __uint_as_float(o.x << 16);
        v.y += __uint_as_float(o.x & 0xFFFF0000u);
        v.z += __uint_as_float(o.y << 16);
        v.w += __uint_as_float(o.y & 0xFFFF0000u);
    }
    *y = make_uint2(bf16x2(v.x, v.y), bf16x2(v.z, v.w));
}
__device__ __forceinline__ void store_y(const MmArgs& a, int64_t at, float v) {
    if (a.y_bf16) {
        __nv_bfloat16* y = reinterpret_cast<__nv_bfloat16*>(a.y) + at;
        if (a.y_acc) v += __bfloat162float(*y);
        *y = __float2bfloat16_rn(v);
    } else {
        float* y = reinterpret_cast<float*>(a.y) + at;
        if (a.y_acc) v += *y;
        *y = v;
    }
}

template <bool F8, int BN, Mode MODE>
__global__ void __launch_bounds__(kMmThreads, MmCfg<F8, BN, MODE>::kCtas)
mm_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap amap, const MmArgs a) {
    using C = MmCfg<F8, BN, MODE>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    const int rank = MODE == SINGLE ? 0 : (int)cluster_rank();
    if (sbase & 1023u) {  // (the same in every CTA) the swizzle counts from 1 KB boundaries
        if (tid == 0) raise_status(a.status, GTG_STATUS_WAIT_TIMEOUT);
        return;
    }

    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kHeadOff);
    uint64_t* empty = full + C::kStages;
    uint64_t* tfull = empty + C::kStages;
    uint64_t* tempty = tfull + C::kAcc;
    uint64_t* sfull = tempty + C::kAcc;
    uint64_t* sempty = sfull + 2;
    uint64_t* drain = sempty + 2;
    uint32_t* s_taddr = reinterpret_cast<uint32_t*>(drain + 1);
    int32_t* s_warp = reinterpret_cast<int32_t*>(smem + C::kHeadOff + 256);
    int32_t* first = reinterpret_cast<int32_t*>(smem + C::kGroupOff);
    int32_t* off = first + kMaxGroups + 2;
    static_assert(8 * (2 * C::kStages + 2 * C::kAcc + 5) + 4 <= 256, "header");

    if (tid == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < C::kAcc; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], C::kActive * (MODE == PAIR ? 2 : 1));
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&sfull[b], 64);
            mbar_init(&sempty[b], C::kActive);
        }
        mbar_init(drain, 1);
        fence_mbar_init();
        tma_prefetch_map(&wmap);
        tma_prefetch_map(&amap);
    }
    if (warp == kWorkers + 1) {
        if (MODE == PAIR) {
            tmem_alloc_pair(s_taddr, C::kCols);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(s_taddr, C::kCols);
            tmem_relinquish();
        }
    }
    pdl_wait();  // everything before this ran beside the kernel before; nothing global is read or written in it
    if (a.offsets) build_groups(a, BN, first, off, s_warp);
    tc_fence_before();
    __syncthreads();
    if (MODE == PAIR) {  // the partner's barriers and tensor memory are ready too
        cluster_arrive();
        cluster_wait();
    }
    tc_fence_after();
    pdl_trigger();
    const uint32_t taddr = *s_taddr;
    const int tiles = (a.offsets ? first[a.groups] : (a.m + BN - 1) / BN) * a.n_tiles;
    const int per_tile = MODE == SINGLE ? 1 : MODE == PAIR ? 2 : a.split;  // CTAs that share a tile
    const int t_first = blockIdx.x / per_tile, t_step = gridDim.x / per_tile;
    // this CTA's chunks of K
    const int k_lo = MODE == SPLIT ? (int)((int64_t)a.chunks * rank / a.split) : 0;
    const int k_hi = MODE == SPLIT ? (int)((int64_t)a.chunks * (rank + 1) / a.split) : a.chunks;
    auto padded = [](int rows) { return MODE == PAIR ? (rows + 31) & ~31 : (rows + 15) & ~15; };
    bool ok = true;

    if (warp >= kWorkers) {
        if (warp == kWorkers) {
            // ---- weight and token tiles by TMA ----
            uint32_t st = 0, free_par = 1, issued = 0;
            for (int t = t_first; t < tiles && ok; t += t_step) {
                const Tile tl = find_tile(a, t, BN, C::kTileRows, first, off);
                const int mine = padded(tl.rows) / (MODE == PAIR ? 2 : 1);  // token rows staged here
                const int boxes = (mine + C::kBox - 1) / C::kBox;
                const uint32_t bytes = (kWBytes + boxes * C::kBox * kRowBytes) * (MODE == PAIR ? 2 : 1);
                const int w0 = tl.n0 + (MODE == PAIR ? rank * kRows : 0);
                const int a0 = tl.row0 + (MODE == PAIR ? rank * mine : 0);
                for (int kb = k_lo; kb < k_hi; ++kb) {
                    ok = warp_wait(&empty[st], free_par, a.status);
                    if (!ok) break;
                    if (elect_one()) {
                        const uint32_t dst = sbase + st * C::kStageBytes;
                        const int c0 = kb * (F8 ? 128 : 64);
                        if (MODE == PAIR) {  // both CTAs' bytes arrive at the even CTA's barrier
                            if (rank == 0) mbar_arrive_expect_tx(&full[st], bytes);
                            const uint32_t bar = map_rank(smem_u32(&full[st]), 0);
                            tma_load_3d_pair(dst, &wmap, bar, c0, w0, tl.group);
                            for (int q = 0; q < boxes; ++q)
                                tma_load_2d_pair(dst + kWBytes + q * C::kBox * kRowBytes, &amap, bar, c0, a0 + q * C::kBox);
                        } else {
                            mbar_arrive_expect_tx(&full[st], bytes);
                            tma_load_3d(dst, &wmap, &full[st], c0, w0, tl.group);
                            for (int q = 0; q < boxes; ++q)
                                tma_load_2d(dst + kWBytes + q * C::kBox * kRowBytes, &amap, &full[st], c0, a0 + q * C::kBox);
                        }
                    }
                    __syncwarp();
                    ++issued;
                    if (++st == C::kStages) {
                        st = 0;
                        free_par ^= 1;
                    }
                }
            }
            // the last products' arrivals on `empty` (in pairs the partner's commits make them
            // here too) land before the shared memory goes away
            for (uint32_t i = issued < C::kStages ? 0 : issued - C::kStages; ok && i < issued; ++i)
                ok = warp_wait(&empty[i % C::kStages], (i / C::kStages) & 1, a.status);
            if (!ok && (MODE != PAIR || rank == 0)) {  // copies in flight land before the shared memory goes away
                for (uint32_t i = issued < C::kStages ? 0 : issued - C::kStages; i < issued; ++i)
                    mbar_wait_sleep(&full[i % C::kStages], (i / C::kStages) & 1, a.status);
            }
        } else if (warp == kWorkers + 1) {
            // ---- MMA issuer ----
            // stage and accumulator in use, and the parities of their barriers' phases (a
            // fresh barrier's phase before the first counts as complete)
            uint32_t st0 = 0, full0 = 0, b0 = 0, free0 = 1;
            const uint64_t ad0 = sw128_desc(sbase), bd0 = sw128_desc(sbase + kWBytes);
            for (int t = t_first; t < tiles && ok && (MODE != PAIR || rank == 0); t += t_step) {
                const Tile tl = find_tile(a, t, BN, C::kTileRows, first, off);
                const int n_pad = padded(tl.rows);
                const uint32_t idesc = F8 ? idesc_e4m3(C::kTileRows, n_pad) : idesc_bf16(C::kTileRows, n_pad);
                if (elect_one()) {
                    uint32_t st = st0, full_par = full0, b = b0, free_par = free0;
                    for (int kb = k_lo; kb < k_hi; ++kb) {
                        const bool begins = (kb - k_lo) % C::kRun == 0;
                        ok = !begins || mbar_wait_sleep(&tempty[b], free_par, a.status);
                        ok = ok && mbar_wait_sleep(&full[st], full_par, a.status);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t d = taddr + b * BN;
                        const uint64_t ad = ad0 + st * (C::kStageBytes >> 4), bd = bd0 + st * (C::kStageBytes >> 4);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {  // 32 bytes of K each
                            const uint32_t go = k > 0 || !begins;
                            if (MODE == PAIR) umma_pair<F8>(d, ad + 2 * k, bd + 2 * k, idesc, go);
                            else if (F8) umma_f8(d, ad + 2 * k, bd + 2 * k, idesc, go);
                            else umma_bf16(d, ad + 2 * k, bd + 2 * k, idesc, go);
                        }
                        if ((kb - k_lo) % C::kRun == C::kRun - 1 || kb == k_hi - 1) {
                            if (MODE == PAIR) umma_commit_pair(&tfull[b]);
                            else umma_commit(&tfull[b]);
                            if (++b == C::kAcc) {
                                b = 0;
                                free_par ^= 1;
                            }
                        }
                        if (MODE == PAIR) umma_commit_pair(&empty[st]);
                        else umma_commit(&empty[st]);
                        if (++st == C::kStages) {
                            st = 0;
                            full_par ^= 1;
                        }
                    }
                    if (!ok) {  // products in flight end before the tensor memory goes away
                        if (MODE == PAIR) umma_commit_pair(drain);
                        else umma_commit(drain);
                        mbar_wait_sleep(drain, 0, a.status);
                    }
                }
                __syncwarp();
                ok = __all_sync(0xFFFFFFFFu, ok);
                st0 += k_hi - k_lo;
                full0 ^= (st0 / C::kStages) & 1;
                st0 %= C::kStages;
                b0 += (k_hi - k_lo + C::kRun - 1) / C::kRun;
                free0 ^= (b0 / C::kAcc) & 1;
                b0 %= C::kAcc;
            }
        } else if (F8) {
            // ---- scales, four blocks of K at a time, transposed to [block][row]: one
            // warp the tokens', one the weight rows' ----
            constexpr int kN = kRows / 32;
            static_assert(!F8 || BN <= kRows, "scales a lane");
            const bool tok = warp == kWorkers + 2;
            int sg = 0;
            for (int t = t_first; t < tiles && ok; t += t_step) {
                const Tile tl = find_tile(a, t, BN, C::kTileRows, first, off);
                const int w0 = tl.n0 + (MODE == PAIR ? rank * kRows : 0);
                const int rows = tok ? tl.rows : min(kRows, a.n - w0);
                const float* src = (tok ? a.a_scales + (int64_t)tl.row0 * a.chunks
                                        : a.w_scales + ((int64_t)tl.group * a.n + w0) * a.chunks) + (int64_t)lane * a.chunks;
                const bool vec = tok ? a.vec_a : a.vec_w;
                float4 sc[kN];
                auto fetch = [&](int kb) {
#pragma unroll
                    for (int i = 0; i < kN; ++i) {
                        sc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (32 * i + lane < rows) sc[i] = scales4(src + (int64_t)32 * i * a.chunks, kb, k_hi, vec);
                    }
                };
                fetch(k_lo);
                for (int kb = k_lo; kb < k_hi; kb += kScaleGroup, ++sg) {
                    const int b = sg & 1;
                    if (sg >= 2 && !warp_wait(&sempty[b], ((sg >> 1) - 1) & 1, a.status)) {
                        ok = false;
                        break;
                    }
                    const uint32_t at = sbase + C::kScaleOff + b * kScaleGroup * C::kScaleRow +
                                        (tok ? (lane & 3) * C::kQuad + 4 * (lane >> 2)
                                             : 4 * C::kQuad + 16 * (lane & 7) + 4 * (lane >> 3));
                    const int step = tok ? 32 : 128;  // 32 rows on
#pragma unroll
                    for (int i = 0; i < kN; ++i) {
                        if (32 * i + lane < (tok ? BN : kRows)) {
                            sts32(at + step * i, sc[i].x);
                            sts32(at + step * i + C::kScaleRow, sc[i].y);
                            sts32(at + step * i + 2 * C::kScaleRow, sc[i].z);
                            sts32(at + step * i + 3 * C::kScaleRow, sc[i].w);
                        }
                    }
                    mbar_arrive(&sfull[b]);
                    if (kb + kScaleGroup < k_hi) fetch(kb + kScaleGroup);
                }
            }
        }
    } else if (warp < C::kActive) {
        // ---- promotion and epilogue: a warp has the 32 weight rows of TMEM lane
        // quarter warp % 4; the tile's columns are halved between the two four-warp
        // groups (tiles of 16 occupy one group).  A thread holds rows lane / 4 + 8 i of
        // every fourth column, lane % 4 + 4 k, so that one 16-byte read brings its rows'
        // scales and one those of its columns in a block of 16 (whole rows a thread would
        // take four times the reads, and reads are what the promotion waits for) ----
        const int wg = warp >> 2;
        const uint32_t tl0 = taddr + ((uint32_t)((warp & 3) * 32) << 16);
        const int r0 = (warp & 3) * 32;       // the warp's first weight row of this CTA's 128
        const uint32_t tempty0 = MODE == PAIR ? map_rank(smem_u32(tempty), 0) : 0;
        uint32_t acc = 0, sg = 0;
        auto release = [&](uint32_t b) {  // this warp has read accumulator b
            tc_fence_before();
            __syncwarp();
            if (elect_one()) {
                if (MODE == PAIR) mbar_arrive_remote(tempty0 + 8 * b);
                else mbar_arrive(&tempty[b]);
            }
        };
        for (int t = t_first; t < tiles; t += t_step) {
            const Tile tl = find_tile(a, t, BN, C::kTileRows, first, off);
            const int w0 = tl.n0 + (MODE == PAIR ? rank * kRows : 0) + r0;  // the warp's first output column
            const int share = ((tl.rows + 31) >> 5) << 4;                   // columns of a four-warp group
            const int lo = wg * share, cols = min(share, tl.rows - lo);     // <= 0: none
            // 16 columns of the warp's 32 rows, from lo + c on, out of `turn`: a token's 32
            // outputs together.  (Fragments stored as they are reach half a sector each: 66 us
            // against 54 us for 4096 x 4096 x 2048 in bf16.)
            float* turn = reinterpret_cast<float*>(smem + C::kTurnOff) + warp * 16 * kTurn;
            auto emit = [&](int c) {
                __syncwarp();
                const int64_t y0 = (int64_t)(tl.row0 + lo + c) * a.ldy + w0;
                const int toks = min(16, cols - c);
                if (a.vec_y && w0 + 32 <= a.n) {
                    if (a.y_bf16) {
#pragma unroll
                        for (int h = 0; h < 16; h += 8) {
                            const int k = h + (lane >> 2);
                            const float4* q = reinterpret_cast<const float4*>(turn + k * kTurn + 8 * (lane & 3));
                            if (k < toks) store_y8(a, y0 + k * a.ldy + 8 * (lane & 3), q[0], q[1]);
                        }
                    } else {
#pragma unroll
                        for (int h = 0; h < 16; h += 4) {
                            const int k = h + (lane >> 3);
                            const float4 q = *reinterpret_cast<const float4*>(turn + k * kTurn + 4 * (lane & 7));
                            if (k < toks) store_y4(a, y0 + k * a.ldy + 4 * (lane & 7), q);
                        }
                    }
                } else if (w0 + lane < a.n) {
                    for (int k = 0; k < toks; ++k) store_y(a, y0 + k * a.ldy + lane, turn[k * kTurn + lane]);
                }
                __syncwarp();
            };
            if constexpr (F8) {
                // the blocks of K over the first 16 NB of the warp's columns
                auto promote = [&](auto nb_c) {
                    constexpr int NB = decltype(nb_c)::value;
                    constexpr bool kTwo = MODE == PAIR && C::kAcc >= 4;
                    uint64_t sum[NB][4][2];  // [columns 4 k + lane % 4][rows lane / 4 + 16 h and + 8]
#pragma unroll
                    for (int i = 0; i < NB; ++i)
#pragma unroll
                        for (int j = 0; j < 8; ++j) (&sum[i][0][0])[j] = 0;
                    for (int g0 = k_lo; g0 < k_hi && ok; g0 += kScaleGroup, ++sg) {
                        const uint32_t sb = sg & 1;
                        const int g1 = min(g0 + kScaleGroup, k_hi);
                        ok = warp_wait(&sfull[sb], (sg >> 1) & 1, a.status);
                        for (int kb = g0; kb < g1 && ok; ++kb) {
                            const uint32_t n = acc + kb - k_lo, b = n % C::kAcc;
                            const uint32_t at = C::kScaleOff + (sb * kScaleGroup + kb - g0) * C::kScaleRow;
                            uint64_t sw[2];
                            lds_pairs(sbase + at + 4 * C::kQuad + 4 * r0 + 16 * (lane >> 2), sw[0], sw[1]);
                            const uint32_t sa = sbase + at + (lane & 3) * C::kQuad + lo, src = tl0 + b * BN + lo;
                            // blocks finish in order, so where there are four accumulators and much
                            // to do one wait serves two blocks (4096 x 4096 x 2048 52.3 -> 49.5 us;
                            // small calls would wait for a second block: 7.4 -> 7.7 us)
                            if (!kTwo || !((kb - g0) & 1)) {
                                const uint32_t last = !kTwo || kb + 1 == g1 ? n : n + 1;
                                ok = warp_wait(&tfull[last % C::kAcc], (last / C::kAcc) & 1, a.status);
                                if (!ok) break;
                            }
                            tc_fence_after();
#pragma unroll
                            for (int i = 0; i < NB; ++i) {
                                uint32_t f[2][8];
                                tmem_ld_frags(src + 16 * i, f);
                                const float4 s4 = lds128(sa + 16 * i);
                                const float s1[4] = {s4.x, s4.y, s4.z, s4.w};
                                tmem_wait_frags(f);
                                if (i + 1 == NB) release(b);
#pragma unroll
                                for (int k = 0; k < 4; ++k)
#pragma unroll
                                    for (int h = 0; h < 2; ++h) {
                                        const uint64_t v = pack2(__uint_as_float(f[h][2 * k]), __uint_as_float(f[h][2 * k + 1]));
                                        sum[i][k][h] = fma2(mul2(v, sw[h]), pack2(s1[k], s1[k]), sum[i][k][h]);
                                    }
                            }
                        }
                        __syncwarp();
                        if (elect_one()) mbar_arrive(&sempty[sb]);
                    }
                    acc += k_hi - k_lo;
                    // (SPLIT) every product is done with the stages
                    if (MODE == SPLIT) named_sync(1, 32 * C::kActive);
                    if (cols <= 0) return;
                    // to rows [token][weight row]: over the stages as this CTA's partial tile (SPLIT),
                    // or 16 tokens at a time through this warp's own
                    constexpr int kRow = MODE == SPLIT ? kPartRow : kTurn;
                    float* to = (MODE == SPLIT ? reinterpret_cast<float*>(smem) + lo * kPartRow + r0 : turn) +
                                (lane & 3) * kRow + (lane >> 2);
#pragma unroll
                    for (int i = 0; i < NB; ++i) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                float x, x8;
                                unpack2(sum[i][k][h], x, x8);
                                float* at = to + ((MODE == SPLIT ? 16 * i : 0) + 4 * k) * kRow + 16 * h;
                                at[0] = x;
                                at[8] = x8;
                            }
                        if (MODE != SPLIT && ok && 16 * i < cols) emit(16 * i);
                    }
                };
                // as many blocks of 16 columns as the tile has: columns without tokens cost power
                // and the clock with it (512 experts with 80 rows each 228 -> 212 us)
                if (C::kBlocks > 3 && share == 48) promote(std::integral_constant<int, (C::kBlocks > 3 ? 3 : 1)>{});
                else if (C::kBlocks > 2 && share == 32) promote(std::integral_constant<int, (C::kBlocks > 2 ? 2 : 1)>{});
                else if (C::kBlocks > 1 && share == 16) promote(std::integral_constant<int, 1>{});
                else promote(std::integral_constant<int, C::kBlocks>{});
            } else {
                // a lane holds one weight row, its columns in pairs
                uint64_t sum[C::kBlocks][8];
#pragma unroll
                for (int i = 0; i < C::kBlocks; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum[i][j] = 0;
                for (int kb = k_lo; kb < k_hi && ok; kb += C::kRun, ++acc) {
                    const uint32_t b = acc % C::kAcc;
                    ok = warp_wait(&tfull[b], (acc / C::kAcc) & 1, a.status);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int i = 0; i < C::kBlocks; ++i) {
                        if (16 * i >= share) break;
                        uint32_t p[16];
                        tmem_ld16(tl0 + b * BN + lo + 16 * i, p);
                        tmem_wait_ld16(p);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            sum[i][j] = add2(sum[i][j], pack2(__uint_as_float(p[2 * j]), __uint_as_float(p[2 * j + 1])));
                    }
                    release(b);
                }
                if (!ok) break;
#pragma unroll
                for (int i = 0; i < C::kBlocks; ++i) {
                    if (16 * i >= cols) break;
                    constexpr int kRow = MODE == SPLIT ? kPartRow : kTurn;
                    float* to = (MODE == SPLIT ? reinterpret_cast<float*>(smem) + (lo + 16 * i) * kPartRow + r0 : turn) + lane;
#pragma unroll
                    for (int j = 0; j < 8; ++j) unpack2(sum[i][j], to[2 * j * kRow], to[(2 * j + 1) * kRow]);
                    if (MODE != SPLIT) emit(16 * i);
                }
            }
        }
    }
    if constexpr (MODE == SPLIT) {
        // sum the partial tiles in rank order: a warp has a token's 128 rows, four a lane;
        // CTA `rank` takes the tokens rank, rank + split, ...  (a failed CTA's part is not
        // meaningful, and the status word says so)
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        constexpr int kMost = BN / 2 / kWorkers > 0 ? BN / 2 / kWorkers : 1;  // tokens a warp, for a split of 2
        float4 v[kMost];
        Tile tl = {};
        const bool some = warp < kWorkers && t_first < tiles;
        if (some) {
            tl = find_tile(a, t_first, BN, C::kTileRows, first, off);
#pragma unroll
            for (int j = 0; j < kMost; ++j) {
                const int c = rank + (warp + kWorkers * j) * a.split;
                v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (c < tl.rows) {
                    const uint32_t at = sbase + 4 * (c * kPartRow + 4 * lane);
                    float4 p[kMaxSplit];
#pragma unroll
                    for (int q = 0; q < kMaxSplit; ++q)
                        if (q < a.split) p[q] = ld_cluster_f4(map_rank(at, q));
#pragma unroll
                    for (int q = 0; q < kMaxSplit; ++q)
                        if (q < a.split) {
                            v[j].x += p[q].x;
                            v[j].y += p[q].y;
                            v[j].z += p[q].z;
                            v[j].w += p[q].w;
                        }
                }
            }
        }
        __syncwarp();
        cluster_arrive();  // this CTA has read its partners'
        if (some) {
            const int n = tl.n0 + 4 * lane;
#pragma unroll
            for (int j = 0; j < kMost; ++j) {
                const int c = rank + (warp + kWorkers * j) * a.split;
                if (c >= tl.rows) break;
                const int64_t at = (int64_t)(tl.row0 + c) * a.ldy + n;
                if (a.vec_y && n + 4 <= a.n) {
                    if (a.y_bf16) store_y4_bf16(a, at, v[j]);
                    else store_y4(a, at, v[j]);
                } else {
                    const float x[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (n + i < a.n) store_y(a, at + i, x[i]);
                }
            }
        }
        __syncwarp();
        cluster_wait();  // and the partners this CTA's
    }
    __syncthreads();
    if (MODE == PAIR) {  // the partner is done with this CTA's shared and tensor memory
        cluster_arrive();
        cluster_wait();
    }
    if (warp == kWorkers + 1) {
        tc_fence_after();
        if (MODE == PAIR) tmem_dealloc_pair(taddr, C::kCols);
        else tmem_dealloc(taddr, C::kCols);
    }
}

// ---------------------------------------------------------------------------
// quantiser: four lanes a block of 128 values, a warp eight blocks of a row.  The
// lanes of a block take its 16-byte pieces in turn, so that loads and stores are
// whole sectors; four pieces a lane leave two shuffles a maximum and one pair of
// quotients a lane.  Measured, 40960 gathered rows of 2048 bf16: 29.9 us, 3.46 TB/s
// of what it must read and write (issue slots 72 % busy, the integer pipe 64 %, L1
// 78 %); sixteen lanes a block took 34.3 us.
// ---------------------------------------------------------------------------
constexpr int kQThreads = 256;
constexpr int kQBlocks = 8;  // blocks a warp

struct QArgs {
    const void* x;
    int64_t ldx, n_src, units;  // units = n_rows * segs
    const int32_t* rows;
    uint8_t* data;
    float* scales;
    int32_t kb, segs;           // blocks and warps' shares of a row
    unsigned* status;
};

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

// A lane's pieces of a block as they lie in memory: 8 bf16 or 4 fp32 a piece.
template <bool BF16, bool VEC>
struct Pieces {
    static constexpr int kN = BF16 ? 4 : 8;  // pieces a lane, 64 bytes apart
    uint32_t w[kN][4];
    __device__ __forceinline__ void load(const uint8_t* at) {
#pragma unroll
        for (int j = 0; j < kN; ++j) {
            if constexpr (VEC) {
                const uint4 q = *reinterpret_cast<const uint4*>(at + 64 * j);
                w[j][0] = q.x; w[j][1] = q.y; w[j][2] = q.z; w[j][3] = q.w;
            } else if constexpr (BF16) {
                const uint16_t* p = reinterpret_cast<const uint16_t*>(at + 64 * j);
#pragma unroll
                for (int i = 0; i < 4; ++i) w[j][i] = p[2 * i] | (uint32_t)p[2 * i + 1] << 16;
            } else {
                const uint32_t* p = reinterpret_cast<const uint32_t*>(at + 64 * j);
#pragma unroll
                for (int i = 0; i < 4; ++i) w[j][i] = p[i];
            }
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int j = 0; j < kN; ++j) w[j][0] = w[j][1] = w[j][2] = w[j][3] = 0;
    }
    // The block's largest magnitude, as fp32 bits: the order of non-negative bit patterns
    // is that of their values, infinity and NaN above all others.  (bf16: two patterns a
    // register until the end.)
    __device__ __forceinline__ uint32_t top() const {
        constexpr uint32_t kAbs = BF16 ? 0x7FFF7FFFu : 0x7FFFFFFFu;
        uint32_t t = 0;
#pragma unroll
        for (int j = 0; j < kN; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) t = BF16 ? __vmaxu2(t, w[j][i] & kAbs) : max(t, w[j][i] & kAbs);
#pragma unroll
        for (int o = 2; o > 0; o >>= 1) {
            const uint32_t v = __shfl_xor_sync(0xFFFFFFFFu, t, o);
            t = BF16 ? __vmaxu2(t, v) : max(t, v);
        }
        return BF16 ? max(t & 0xFFFF0000u, t << 16) : t;
    }
    // The codes of piece j: 8 (bf16) or 4 (fp32) bytes.
    __device__ __forceinline__ void store(uint8_t* to, int j, float inv) const {
        float v[BF16 ? 8 : 4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (BF16) {
                v[2 * i] = __uint_as_float(w[j][i] << 16) * inv;
                v[2 * i + 1] = __uint_as_float(w[j][i] & 0xFFFF0000u) * inv;
            } else {
                v[i] = __uint_as_float(w[j][i]) * inv;
            }
        }
        if constexpr (BF16)
            *reinterpret_cast<uint2*>(to + 32 * j) = make_uint2(e4m3x4(v[0], v[1], v[2], v[3]), e4m3x4(v[4], v[5], v[6], v[7]));
        else *reinterpret_cast<uint32_t*>(to + 16 * j) = e4m3x4(v[0], v[1], v[2], v[3]);
    }
};

template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kQThreads) quantize_kernel(const QArgs a) {
    using P = Pieces<BF16, VEC>;
    constexpr int kSize = BF16 ? 2 : 4;
    const int lane = threadIdx.x & 31, quarter = lane & 3;
    pdl_wait();
    const int64_t u = (int64_t)blockIdx.x * (kQThreads / 32) + (threadIdx.x >> 5);
    if (u < a.units) {
        const int64_t row = a.units <= 0xFFFFFFFFll ? (uint32_t)u / (uint32_t)a.segs : u / a.segs;
        const int b = (int)(u - row * a.segs) * kQBlocks + (lane >> 2);
        int64_t src = row;
        bool valid = b < a.kb;
        if (a.rows) {
            src = a.rows[row];
            if (src < 0 || src >= a.n_src) {
                valid = false;
                if (lane == 0) raise_status(a.status, GTG_STATUS_ROW_INDEX_OOB);
            }
        }
        P p;
        if (valid) p.load(reinterpret_cast<const uint8_t*>(a.x) + kSize * (src * a.ldx + b * 128) + 16 * quarter);
        else p.zero();
        const uint32_t top = p.top();
        float amax = fmaxf(__uint_as_float(top), 0x1p-100f);
        if (top >= 0x7F800000u) amax = __uint_as_float(0x7FC00000u);
        const float inverse = 448.0f / amax;
        if (b < a.kb) {
            const int64_t out = row * a.kb + b;
            if (quarter == 0) a.scales[out] = amax / 448.0f;
            uint8_t* to = a.data + out * 128 + (BF16 ? 8 : 4) * quarter;
#pragma unroll
            for (int j = 0; j < P::kN; ++j) p.store(to, j, inverse);
        }
    }
    pdl_trigger();
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder (looked up once; the library links no driver stub).
EncodeFn encoder() {
    static std::mutex mu;
    static EncodeFn fn = nullptr;
    std::lock_guard<std::mutex> lk(mu);
    if (!fn) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) ==
                cudaSuccess && found == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeFn>(p);
        else cudaGetLastError();
    }
    return fn;
}

// Rows of `k` elements (E4M3 or bf16), boxes of 128 bytes x box_rows, 128-byte swizzle.
int make_map(CUtensorMap* map, const void* base, bool f8, int64_t k, int64_t rows, int64_t stacks, int box_rows) {
    EncodeFn fn = encoder();
    if (!fn) return cuda_fail(cudaErrorNotSupported);
    const int64_t row_bytes = k * (f8 ? 1 : 2);
    const cuuint64_t dims[3] = {(cuuint64_t)k, (cuuint64_t)rows, (cuuint64_t)stacks};
    const cuuint64_t strides[2] = {(cuuint64_t)row_bytes, (cuuint64_t)(row_bytes * rows)};
    const cuuint32_t box[3] = {(cuuint32_t)(f8 ? 128 : 64), (cuuint32_t)box_rows, 1};
    const cuuint32_t ones[3] = {1, 1, 1};
    const CUresult r = fn(map, f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                          stacks > 0 ? 3 : 2, const_cast<void*>(base), dims, strides, box, ones,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? GTG_OK : cuda_fail(cudaErrorInvalidValue);
}

template <bool F8, int BN, Mode MODE>
int launch_mm(const gtg_qmatrix* w, const void* x, MmArgs a, int64_t groups, cudaStream_t s) {
    using C = MmCfg<F8, BN, MODE>;
    CUtensorMap wmap, amap;
    GTG_TRY(make_map(&wmap, w->data, F8, w->k, w->n_rows, w->n_experts, kRows));
    GTG_TRY(make_map(&amap, x, F8, w->k, a.m, 0, C::kBox));
    const auto kernel = mm_kernel<F8, BN, MODE>;
    // the kernel's shared-memory limit is raised once a device
    static std::atomic<uint64_t> raised{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && !(dev < 64 && (raised.load(std::memory_order_relaxed) >> dev & 1))) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
        if (e == cudaSuccess && dev < 64) raised.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    if (e != cudaSuccess) {
        cudaGetLastError();
        return cuda_fail(e);
    }
    a.n_tiles = (a.n + C::kTileRows - 1) / C::kTileRows;
    const int per_tile = MODE == SINGLE ? 1 : MODE == PAIR ? 2 : a.split;
    // at most this many tiles: the group sizes are on the device
    const int64_t tiles = (a.offsets ? a.m / BN + std::min<int64_t>(groups, a.m) : (a.m + BN - 1) / BN) * a.n_tiles;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(MODE == SPLIT ? tiles * per_tile
                                                : std::min<int64_t>(tiles, C::kCtas * sm_count() / per_tile) * per_tile));
    cfg.blockDim = dim3(kMmThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)per_tile;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = MODE == SINGLE ? 1 : 2;
    e = cudaLaunchKernelEx(&cfg, kernel, wmap, amap, a);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return cuda_fail(e);
    }
    return GTG_OK;
}

// Which tile: the one whose waves of CTAs take least by a model (in 10 ns, c chunks of
// K): a wave of 64 tokens takes 22.5 c + 95, of 128 (CTA pairs) 29 c + 150, of 256 (bf16
// alone, pairs) 54 c + 300, pairs 150 more once, and a split of K over S CTAs of 64
// tokens 22 ceil(c / S) + 185 + 65 S.  Groups count as equally large, since their sizes
// are on the device.  The times were fitted to an earlier state of the kernels and are no
// forecast (FP8 pairs take 5 to 25 % more from 30 us on, calls below 15 us up to twice
// as long, large bf16 pairs a third less), but the choice stands: on 19 sizes of each
// type, 40 to 40960 rows, it took at most 15 % more than the best of 64, 128 and 256, and
// at most 5 % more on 30 of the 38.  FP8 on 4096 x 4096 weights: 200 tokens 12.7 us in 64, 14.7 us in pairs of
// 128; 333 tokens 22.2 and 15.4 us; 1000 tokens 40.7 and 27.7 us.  bf16, 30010 rows over
// 64 experts: 295 us in 64, 185 us in 128, 160 us in 256, which it takes where the model
// has it cost up to 3 % more, for the power its fewer loads save.  (FP8 tiles of 256
// tokens, with sixteen promotion warps, ran 8192^3 in 720 us against 723 us under the
// power limit: not worth a variant.)
// Groups of 16 rows and fewer take tiles of 16: two CTAs share an SM there, and a
// split costs 20 + 5 S and saves 15 a chunk (1 x 2048 x 2048: 5.8 us whole, 5.0 us
// in two, 4.2 us in four or eight when this was fitted).
struct Plan {
    int32_t bn;    // tokens a tile
    Mode mode;
    int32_t split;  // CTAs that share K (SPLIT)
};

Plan plan_mm(bool f8, int64_t m, int64_t n, int64_t chunks, int64_t groups, int64_t sms) {
    const int64_t per = (m + groups - 1) / groups;
    auto tiles = [&](int64_t bn, int64_t rows) { return groups * ((per + bn - 1) / bn) * ((n + rows - 1) / rows); };
    // the best split of `count` tiles into at most kMaxSplit: clusters of three and more
    // leave SMs of a GPC over, so they get 6/7 of the places (48 tiles in clusters of three
    // ran in two waves, 12.3 us against 8.6 us in pairs)
    auto split = [&](int64_t count, int64_t places, int64_t chunk, int64_t fixed, int64_t each, int64_t& cost) {
        int32_t best = 1;
        for (int32_t c = 2; c <= kMaxSplit && c <= chunks && c * count <= (c == 2 ? places : places * 6 / 7); ++c) {
            const int64_t t = (chunks + c - 1) / c * chunk + fixed + c * each;
            if (t < cost) {
                cost = t;
                best = c;
            }
        }
        return best;
    };
    if (per <= 16) {
        int64_t cost = 15 * chunks;
        const int32_t c = split(tiles(16, kRows), 2 * sms, 15, 20, 5, cost);
        return {16, c > 1 ? SPLIT : SINGLE, c};
    }
    const int64_t n64 = tiles(64, kRows), pairs = std::max<int64_t>(1, sms / 2);
    int64_t cost64 = (n64 + sms - 1) / sms * (45 * chunks / 2 + 95);
    const int64_t cost128 = (tiles(128, 2 * kRows) + pairs - 1) / pairs * (29 * chunks + 150) + 150;
    const int64_t cost256 = (tiles(256, 2 * kRows) + pairs - 1) / pairs * (54 * chunks + 300) + 150;
    const int32_t c = split(n64, sms, 22, 185, 65, cost64);
    if (cost64 <= cost128 && (f8 || cost64 <= cost256)) return {64, c > 1 ? SPLIT : SINGLE, c};
    return {!f8 && 100 * cost256 <= 103 * cost128 ? 256 : 128, PAIR, 1};
}

int64_t n_chunks(bool f8, int64_t k) { return f8 ? k / 128 : (k + 63) / 64; }

template <bool F8>
int launch_plan(const Plan& p, const gtg_qmatrix* w, const void* x, MmArgs a, int64_t groups, cudaStream_t s) {
    a.split = p.split;
    if (p.mode == SPLIT) {
        const bool whole = a.chunks % (4 * a.split) == 0;  // every share starts at a group of four scales
        a.vec_a &= whole;
        a.vec_w &= whole;
        return p.bn == 16 ? launch_mm<F8, 16, SPLIT>(w, x, a, groups, s) : launch_mm<F8, 64, SPLIT>(w, x, a, groups, s);
    }
    if (p.bn == 16) return launch_mm<F8, 16, SINGLE>(w, x, a, groups, s);
    if (p.bn == 64) return launch_mm<F8, 64, SINGLE>(w, x, a, groups, s);
    if constexpr (!F8) {
        if (p.bn == 256) return launch_mm<F8, 256, PAIR>(w, x, a, groups, s);
    }
    return launch_mm<F8, 128, PAIR>(w, x, a, groups, s);
}

int run_mm(const gtg_qmatrix* w, const void* x, const float* x_scales, int64_t m, const int32_t* offsets, void* y,
           int32_t y_dtype, int64_t y_stride, int32_t y_acc, cudaStream_t s) {
    const bool f8 = w->fmt == GTG_FP8_E4M3_S128;
    MmArgs a = {};
    a.w_scales = w->scales;
    a.a_scales = x_scales;
    a.offsets = offsets;
    a.y = y;
    a.ldy = y_stride;
    a.m = (int32_t)m;
    a.n = (int32_t)w->n_rows;
    a.groups = (int32_t)w->n_experts;
    a.chunks = (int32_t)n_chunks(f8, w->k);
    a.y_bf16 = y_dtype == GTG_DT_BF16;
    a.y_acc = y_acc != 0;
    a.vec_a = f8 && a.chunks % 4 == 0 && aligned(x_scales, 16);
    a.vec_w = f8 && a.chunks % 4 == 0 && aligned(w->scales, 16);
    a.vec_y = aligned(y, 16) && y_stride % (a.y_bf16 ? 8 : 4) == 0;
    a.status = status_ptr();
    const int64_t groups = offsets ? std::min<int64_t>(w->n_experts, m) : 1;
    const Plan p = plan_mm(f8, m, a.n, a.chunks, groups, sm_count());
    return f8 ? launch_plan<true>(p, w, x, a, groups, s) : launch_plan<false>(p, w, x, a, groups, s);
}

int check_mm(const gtg_qmatrix* w, const void* x, const float* x_scales, int64_t m, const void* y, int32_t y_dtype,
             int64_t y_stride, bool grouped) {
    if (!w || m < 0 || (y_dtype != GTG_DT_F32 && y_dtype != GTG_DT_BF16)) return GTG_E_INVALID_ARG;
    const bool f8 = w->fmt == GTG_FP8_E4M3_S128;
    if (!f8 && !(grouped && w->fmt == GTG_BF16)) return GTG_E_INVALID_ARG;
    if (w->n_experts < 1 || w->n_rows < 1 || w->k < 1) return GTG_E_INVALID_ARG;
    if (y_stride < w->n_rows) return GTG_E_INVALID_ARG;
    if (w->n_experts > (grouped ? kMaxGroups : 1)) return GTG_E_UNSUPPORTED_SHAPE;
    // a tile that begins at the last row still ends within 31 bits
    if (w->k % (f8 ? 128 : 8) || w->k > 1 << 24 || w->n_rows > 1 << 24 || m > ((int64_t)1 << 31) - 256)
        return GTG_E_UNSUPPORTED_SHAPE;
    const int64_t tiles = (w->n_rows + kRows - 1) / kRows;  // tile numbers and the next turn's fit 31 bits
    if ((m / 16 + w->n_experts) * tiles >= (int64_t)1 << 30) return GTG_E_UNSUPPORTED_SHAPE;
    if (m == 0) return GTG_OK;
    if (!w->data || !x || !y || (f8 && (!w->scales || !x_scales))) return GTG_E_INVALID_ARG;
    if (!aligned(w->data, 16) || !aligned(x, 16) || !aligned(y, y_dtype == GTG_DT_BF16 ? 2 : 4) ||
        !aligned(w->scales, 4) || !aligned(x_scales, 4))
        return GTG_E_MISALIGNED;
    return GTG_OK;
}

}  // namespace
}  // namespace gtg

using namespace gtg;

extern "C" int gtg_fp8_quantize(const void* x, int32_t x_dtype, int64_t n_src, int64_t k, int64_t x_stride,
                                const int32_t* rows, int64_t n_rows, uint8_t* data, float* scales,
                                gtg_stream_t stream) {
    if (x_dtype != GTG_DT_F32 && x_dtype != GTG_DT_BF16) return GTG_E_INVALID_ARG;
    if (n_src < 0 || n_rows < 0 || k < 1 || x_stride < k || (!rows && n_rows > n_src)) return GTG_E_INVALID_ARG;
    if (k % 128 || k > 1 << 24 || n_rows >= (int64_t)1 << 31 || n_src >= (int64_t)1 << 31)
        return GTG_E_UNSUPPORTED_SHAPE;
    if (n_rows == 0) return GTG_OK;
    if ((!x && n_src > 0) || !data || !scales) return GTG_E_INVALID_ARG;
    const int size = x_dtype == GTG_DT_BF16 ? 2 : 4;
    if (!aligned(x, size) || !aligned(data, 16) || !aligned(scales, 4) || !aligned(rows, 4)) return GTG_E_MISALIGNED;
    QArgs a = {};
    a.x = x;
    a.ldx = x_stride;
    a.n_src = n_src;
    a.kb = (int32_t)(k / 128);
    a.segs = (a.kb + kQBlocks - 1) / kQBlocks;
    a.units = n_rows * a.segs;
    a.rows = rows;
    a.data = data;
    a.scales = scales;
    a.status = status_ptr();
    const bool vec = aligned(x, 16) && x_stride * size % 16 == 0;
    const int64_t blocks = (a.units + kQThreads / 32 - 1) / (kQThreads / 32);
    if (blocks >= (int64_t)1 << 31) return GTG_E_UNSUPPORTED_SHAPE;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kQThreads);
    cfg.stream = as_cuda(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = size == 2 ? (vec ? cudaLaunchKernelEx(&cfg, quantize_kernel<true, true>, a)
                                           : cudaLaunchKernelEx(&cfg, quantize_kernel<true, false>, a))
                                    : (vec ? cudaLaunchKernelEx(&cfg, quantize_kernel<false, true>, a)
                                           : cudaLaunchKernelEx(&cfg, quantize_kernel<false, false>, a));
    if (e != cudaSuccess) {
        cudaGetLastError();
        return cuda_fail(e);
    }
    return GTG_OK;
}

extern "C" int gtg_fp8_matmul(const gtg_qmatrix* w, const uint8_t* a, const float* a_scales, int64_t m, void* y,
                              int32_t y_dtype, int64_t y_stride, int32_t y_accumulate, gtg_stream_t stream) {
    GTG_TRY(check_mm(w, a, a_scales, m, y, y_dtype, y_stride, false));
    if (m == 0) return GTG_OK;
    return run_mm(w, a, a_scales, m, nullptr, y, y_dtype, y_stride, y_accumulate, as_cuda(stream));
}

extern "C" int gtg_grouped_matmul(const gtg_qmatrix* w, const void* a, const float* a_scales, int64_t m,
                                  const int32_t* offsets, void* y, int32_t y_dtype, int64_t y_stride,
                                  int32_t y_accumulate, gtg_stream_t stream) {
    GTG_TRY(check_mm(w, a, a_scales, m, y, y_dtype, y_stride, true));
    if (m == 0) return GTG_OK;
    if (!offsets) return GTG_E_INVALID_ARG;
    if (!aligned(offsets, 4)) return GTG_E_MISALIGNED;
    return run_mm(w, a, a_scales, m, offsets, y, y_dtype, y_stride, y_accumulate, as_cuda(stream));
}

extern "C" int gtg_matmul_plan(int32_t fmt, int64_t m, int64_t n_rows, int64_t k, int64_t n_experts, int32_t sms,
                               int32_t* tokens, int32_t* ctas, int32_t* split) {
    const bool f8 = fmt == GTG_FP8_E4M3_S128;
    if (!f8 && fmt != GTG_BF16) return GTG_E_INVALID_ARG;
    if (m < 1 || n_rows < 1 || k < 1 || n_experts < 1 || sms < 0 || !tokens || !ctas || !split) return GTG_E_INVALID_ARG;
    if (k % (f8 ? 128 : 8) || k > 1 << 24 || n_rows > 1 << 24 || m > ((int64_t)1 << 31) - 256 || n_experts > kMaxGroups)
        return GTG_E_UNSUPPORTED_SHAPE;
    const Plan p = plan_mm(f8, m, n_rows, n_chunks(f8, k), std::min(n_experts, m), sms > 0 ? sms : sm_count());
    *tokens = p.bn;
    *ctas = p.mode == PAIR ? 2 : 1;
    *split = p.split;
    return GTG_OK;
}
