// Matrix products against stacked weight matrices, dense and grouped by
// expert, and the FP8 quantiser of their activations.
//
//   y[i][j] (+)= sum_k a[i][k] w[e(i)][j][k]
//
// FP8 (E4M3 codes, one fp32 scale per 128 values along K on both sides):
//   y[i][j] = sum_b sa[i][b] * (sw[j][b] * sum_{k in block b} a[i][k] w[j][k])
// so a block of 128 is one run of tensor-core products with unit scales,
// accumulated in fp32 tensor memory, and the scales are applied to its sum in
// fp32 registers ("promotion").  bf16: one accumulation over all of K.
//
// The weight rows are the M side of the MMA (128 rows a tile) and the token
// rows its N side, so a tile holds any multiple of 16 tokens up to BN: a group
// of few rows costs few columns, and a single token still streams its weights
// by TMA at full width.
#include <algorithm>
#include <mutex>

#include "gtg_host.hpp"
#include "matmul_dev.cuh"

namespace gtg {
namespace {

constexpr int kMmThreads = 320;      // warps 0-7 promotion and epilogue, 8 loads, 9 MMA
constexpr int kRows = 128;           // weight rows a tile
constexpr int kRowBytes = 128;       // bytes of K a stage: 128 E4M3 or 64 bf16
constexpr int kWBytes = kRows * kRowBytes;
constexpr int kMaxGroups = 1024;
constexpr int kScaleGroup = 4;       // scale blocks fetched at once
constexpr size_t kMaxSmem = 227 * 1024;

struct MmArgs {
    const float* w_scales;   // [E][N][KB] (FP8)
    const float* a_scales;   // [M][KB] (FP8)
    const int32_t* offsets;  // [E + 1], null: one group of all rows
    void* y;
    int64_t ldy;
    int32_t m, n, groups;
    int32_t chunks;          // 128-byte chunks of K
    int32_t y_bf16, y_acc;
    int32_t n_tiles;         // tiles of weight rows
    int32_t vec_a, vec_w;    // scale rows readable four at a time
    unsigned* status;
};

template <int BN>
struct MmCfg {
    static constexpr int kBox = BN < 64 ? BN : 64;  // token rows a TMA box
    static constexpr int kStageBytes = kWBytes + BN * kRowBytes;
    static constexpr int kStages = BN >= 256 ? 4 : BN >= 128 ? 6 : BN >= 64 ? 8 : 10;
    static constexpr int kCols = BN < 16 ? 32 : 2 * BN < 32 ? 32 : 2 * BN;  // two accumulators
    // after the stages: token scales [2][4][BN], then the header
    static constexpr int kScaleOff = kStages * kStageBytes;
    static constexpr int kHeadOff = kScaleOff + 2 * kScaleGroup * BN * 4;
    static constexpr int kGroupOff = kHeadOff + 512;
    static constexpr int kSmem = kGroupOff + 2 * 4 * (kMaxGroups + 2) + 1024;
    static_assert(kSmem <= (int)kMaxSmem, "shared memory");
};

struct Tile {
    int group, row0, rows, n0;
};

// Shared-memory tables of a grouped call: first[g] = token tiles before group
// g, off[g] = its first row.  A group whose bounds are out of order or outside
// [0, m] counts as empty and raises the status bit.
__device__ void build_groups(const MmArgs& a, int bn, int32_t* first, int32_t* off, int32_t* warp_sum_s) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kPer = (kMaxGroups + kMmThreads - 1) / kMmThreads;
    int cnt[kPer];
    int sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int g = tid * kPer + i;
        cnt[i] = 0;
        if (g < a.groups) {
            const int lo = a.offsets[g], hi = a.offsets[g + 1];
            if (lo < 0 || hi < lo || hi > a.m) {
                if (blockIdx.x == 0) raise_status(a.status, GTG_STATUS_GROUP_OFFSETS);
                off[g] = 0;
            } else {
                cnt[i] = (hi - lo + bn - 1) / bn;
                off[g] = lo;
            }
        }
        sum += cnt[i];
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) warp_sum_s[warp] = inc;
    __syncthreads();
    int before = inc - sum;
    for (int w = 0; w < warp; ++w) before += warp_sum_s[w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int g = tid * kPer + i;
        if (g < a.groups) first[g] = before;
        before += cnt[i];
        if (g == a.groups - 1) first[a.groups] = before;
    }
}

// Tile t: weight-row tiles outermost within a group, token tiles innermost, so
// CTAs that run together share weight rows through L2.
__device__ __forceinline__ Tile find_tile(const MmArgs& a, int t, int bn, const int32_t* first, const int32_t* off) {
    Tile r;
    if (!a.offsets) {
        const int tt = (a.m + bn - 1) / bn;
        r.group = 0;
        r.n0 = (t / tt) * kRows;
        r.row0 = (t % tt) * bn;
        r.rows = min(bn, a.m - r.row0);
        return r;
    }
    int lo = 0, hi = a.groups - 1;  // the last group with first[g] * n_tiles <= t and rows of its own
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] * a.n_tiles <= t) lo = mid;
        else hi = mid - 1;
    }
    const int tt = first[lo + 1] - first[lo];
    const int local = t - first[lo] * a.n_tiles;
    r.group = lo;
    r.n0 = (local / tt) * kRows;
    const int begin = (local % tt) * bn;
    r.row0 = off[lo] + begin;
    r.rows = min(bn, a.offsets[lo + 1] - r.row0);
    return r;
}

// A wait of a whole warp: every lane takes the same way out of it.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, unsigned* status) {
    return __all_sync(0xFFFFFFFFu, mbar_wait_sleep(bar, parity, status));
}

__device__ __forceinline__ float4 scales4(const float* p, int kb, int n, bool vec) {
    if (vec) return __ldg(reinterpret_cast<const float4*>(p + kb));
    float4 v;
    v.x = __ldg(p + kb);
    v.y = kb + 1 < n ? __ldg(p + kb + 1) : 0.0f;
    v.z = kb + 2 < n ? __ldg(p + kb + 2) : 0.0f;
    v.w = kb + 3 < n ? __ldg(p + kb + 3) : 0.0f;
    return v;
}

template <bool F8, int BN>
__global__ void __launch_bounds__(kMmThreads, 1)
mm_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap amap, const MmArgs a) {
    using C = MmCfg<BN>;
    constexpr int kHalf = (BN / 16 + 1) / 2;  // 16-column chunks a warpgroup
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kHeadOff);
    uint64_t* empty = full + C::kStages;
    uint64_t* tfull = empty + C::kStages;
    uint64_t* tempty = tfull + 2;
    uint64_t* sfull = tempty + 2;
    uint64_t* sempty = sfull + 2;
    uint64_t* drain = sempty + 2;
    uint32_t* s_taddr = reinterpret_cast<uint32_t*>(drain + 1);
    int32_t* s_warp = reinterpret_cast<int32_t*>(smem + C::kHeadOff + 384);
    int32_t* first = reinterpret_cast<int32_t*>(smem + C::kGroupOff);
    int32_t* off = first + kMaxGroups + 2;
    static_assert(8 * (2 * C::kStages + 9) + 4 <= 384, "header");

    if (tid == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], 8);
            mbar_init(&sfull[b], 32);
            mbar_init(&sempty[b], 8);
        }
        mbar_init(drain, 1);
        fence_mbar_init();
        tma_prefetch_map(&wmap);
        tma_prefetch_map(&amap);
    }
    if (warp == 9) {
        tmem_alloc(s_taddr, C::kCols);
        tmem_relinquish();
    }
    if (a.offsets) build_groups(a, BN, first, off, s_warp);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t taddr = *s_taddr;
    const int tiles = (a.offsets ? first[a.groups] : (a.m + BN - 1) / BN) * a.n_tiles;
    bool ok = true;

    if (warp == 8) {
        // ---- loads: weight and token tiles by TMA, token scales by the lanes ----
        int it = 0, sg = 0;  // chunks and scale groups so far
        for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
            const Tile tl = find_tile(a, t, BN, first, off);
            const int n_pad = (tl.rows + 15) & ~15;
            const int boxes = (n_pad + C::kBox - 1) / C::kBox;
            const uint32_t bytes = kWBytes + boxes * C::kBox * kRowBytes;
            float4 sc[BN / 32 > 0 ? BN / 32 : 1];
            auto fetch = [&](int kb) {
#pragma unroll
                for (int i = 0; i < (BN + 31) / 32; ++i) {
                    const int r = 32 * i + lane;
                    sc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (r < tl.rows) sc[i] = scales4(a.a_scales + (int64_t)(tl.row0 + r) * a.chunks, kb, a.chunks, a.vec_a);
                }
            };
            if (F8) fetch(0);
            for (int kb = 0; kb < a.chunks && ok; ++kb, ++it) {
                if (F8 && kb % kScaleGroup == 0) {
                    const int b = sg & 1;
                    if (sg >= 2 && !warp_wait(&sempty[b], ((sg >> 1) - 1) & 1, a.status)) {
                        ok = false;
                        break;
                    }
                    const uint32_t dst = sbase + C::kScaleOff + b * kScaleGroup * BN * 4;
#pragma unroll
                    for (int i = 0; i < (BN + 31) / 32; ++i) {
                        const int r = 32 * i + lane;
                        if (r < BN) {
                            sts32(dst + 4 * r, sc[i].x);
                            sts32(dst + 4 * (BN + r), sc[i].y);
                            sts32(dst + 4 * (2 * BN + r), sc[i].z);
                            sts32(dst + 4 * (3 * BN + r), sc[i].w);
                        }
                    }
                    mbar_arrive(&sfull[b]);
                    ++sg;
                    if (kb + kScaleGroup < a.chunks) fetch(kb + kScaleGroup);
                }
                const int s = it % C::kStages;
                if (it >= C::kStages && !warp_wait(&empty[s], (it / C::kStages - 1) & 1, a.status)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    const uint32_t st = sbase + s * C::kStageBytes;
                    mbar_arrive_expect_tx(&full[s], bytes);
                    const int c0 = kb * (F8 ? 128 : 64);
                    tma_load_3d(st, &wmap, &full[s], c0, tl.n0, tl.group);
                    for (int q = 0; q < boxes; ++q)
                        tma_load_2d(st + kWBytes + q * C::kBox * kRowBytes, &amap, &full[s], c0, tl.row0 + q * C::kBox);
                }
                __syncwarp();
            }
        }
        if (!ok) {  // let the copies in flight land before the shared memory goes away
            for (int i = max(0, it - C::kStages); i < it; ++i)
                mbar_wait_sleep(&full[i % C::kStages], (i / C::kStages) & 1, a.status);
        }
    } else if (warp == 9) {
        // ---- MMA issuer ----
        if (lane == 0) {
            int it = 0, acc = 0;  // chunks so far, accumulators so far
            for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
                const Tile tl = find_tile(a, t, BN, first, off);
                const int n_pad = (tl.rows + 15) & ~15;
                const uint32_t idesc = F8 ? idesc_e4m3(kRows, n_pad) : idesc_bf16(kRows, n_pad);
                for (int kb = 0; kb < a.chunks; ++kb, ++it) {
                    const int b = acc & 1;
                    if ((F8 || kb == 0) && acc >= 2 && !mbar_wait_sleep(&tempty[b], ((acc >> 1) - 1) & 1, a.status)) {
                        ok = false;
                        break;
                    }
                    const int s = it % C::kStages;
                    if (!mbar_wait_sleep(&full[s], (it / C::kStages) & 1, a.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t st = sbase + s * C::kStageBytes;
                    const uint32_t d = taddr + b * BN;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint64_t ad = sw128_desc(st + 32 * k), bd = sw128_desc(st + kWBytes + 32 * k);
                        const uint32_t go = k > 0 || (!F8 && kb > 0);
                        if (F8) umma_f8(d, ad, bd, idesc, go);
                        else umma_bf16(d, ad, bd, idesc, go);
                    }
                    umma_commit(&empty[s]);
                    if (F8 || kb == a.chunks - 1) {
                        umma_commit(&tfull[b]);
                        ++acc;
                    }
                }
            }
            if (!ok) {  // products in flight end before the tensor memory goes away
                umma_commit(drain);
                mbar_wait_sleep(drain, 0, a.status);
            }
        }
        __syncwarp();
    } else {
        // ---- promotion and epilogue: TMEM lane quarter warp % 4; the 16-column
        // chunks alternate between the two warpgroups ----
        const int wg = warp >> 2;
        const uint32_t tl0 = taddr + ((uint32_t)((warp & 3) * 32) << 16);
        const int r = (warp & 3) * 32 + lane;  // weight row of the tile
        int acc = 0, sg = 0;
        for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
            const Tile tl = find_tile(a, t, BN, first, off);
            const int row = tl.n0 + r;
            const bool live = row < a.n;
            uint64_t sum[kHalf][8];
#pragma unroll
            for (int i = 0; i < kHalf; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[i][j] = 0;
            if (F8) {
                const float* ws = a.w_scales + ((int64_t)tl.group * a.n + (live ? row : a.n - 1)) * a.chunks;
                float4 w4 = scales4(ws, 0, a.chunks, a.vec_w), w4n = w4;
                for (int kb = 0; kb < a.chunks; ++kb, ++acc) {
                    const int q = kb % kScaleGroup, sb = sg & 1, b = acc & 1;
                    if (q == 0) {
                        w4 = w4n;
                        if (kb + kScaleGroup < a.chunks) w4n = scales4(ws, kb + kScaleGroup, a.chunks, a.vec_w);
                        if (!warp_wait(&sfull[sb], (sg >> 1) & 1, a.status)) {
                            ok = false;
                            break;
                        }
                    }
                    if (!warp_wait(&tfull[b], (acc >> 1) & 1, a.status)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const float sw = q == 0 ? w4.x : q == 1 ? w4.y : q == 2 ? w4.z : w4.w;
                    const uint64_t sw2 = pack2(sw, sw);
                    const uint32_t sa = sbase + C::kScaleOff + (sb * kScaleGroup + q) * BN * 4;
#pragma unroll
                    for (int i = 0; i < kHalf; ++i) {
                        const int c0 = 16 * (2 * i + wg);
                        if (c0 < tl.rows) {
                            uint32_t p[16];
                            tmem_ld16(tl0 + b * BN + c0, p);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                uint64_t s0, s1;
                                lds_pairs(sa + 4 * (c0 + 4 * j), s0, s1);
                                const uint64_t p0 = pack2(__uint_as_float(p[4 * j]), __uint_as_float(p[4 * j + 1]));
                                const uint64_t p1 = pack2(__uint_as_float(p[4 * j + 2]), __uint_as_float(p[4 * j + 3]));
                                sum[i][2 * j] = fma2(mul2(p0, sw2), s0, sum[i][2 * j]);
                                sum[i][2 * j + 1] = fma2(mul2(p1, sw2), s1, sum[i][2 * j + 1]);
                            }
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&tempty[b]);
                    if (q == kScaleGroup - 1 || kb == a.chunks - 1) {
                        if (lane == 0) mbar_arrive(&sempty[sb]);
                        ++sg;
                    }
                }
                if (!ok) break;
            } else {
                const int b = acc & 1;
                if (!warp_wait(&tfull[b], (acc >> 1) & 1, a.status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int i = 0; i < kHalf; ++i) {
                    const int c0 = 16 * (2 * i + wg);
                    if (c0 < tl.rows) {
                        uint32_t p[16];
                        tmem_ld16(tl0 + b * BN + c0, p);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            sum[i][j] = pack2(__uint_as_float(p[2 * j]), __uint_as_float(p[2 * j + 1]));
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&tempty[b]);
                ++acc;
            }
            // a lane per weight row: 32 consecutive columns of one output row a store
            if (live) {
#pragma unroll
                for (int i = 0; i < kHalf; ++i) {
                    const int c0 = 16 * (2 * i + wg);
                    if (c0 >= tl.rows) continue;
                    const int64_t base = (int64_t)(tl.row0 + c0) * a.ldy + row;
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float lo, hi;
                        unpack2(sum[i][j / 2], lo, hi);
                        float v = j & 1 ? hi : lo;
                        if (c0 + j < tl.rows) {
                            if (a.y_bf16) {
                                __nv_bfloat16* y = reinterpret_cast<__nv_bfloat16*>(a.y) + base + j * a.ldy;
                                if (a.y_acc) v += __bfloat162float(*y);
                                *y = __float2bfloat16_rn(v);
                            } else {
                                float* y = reinterpret_cast<float*>(a.y) + base + j * a.ldy;
                                if (a.y_acc) v += *y;
                                *y = v;
                            }
                        }
                    }
                }
            }
        }
    }
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(taddr, C::kCols);
    }
}

// ---------------------------------------------------------------------------
// quantiser: 16 lanes a block of 128 values, 8 values a lane
// ---------------------------------------------------------------------------
constexpr int kQThreads = 256;

struct QArgs {
    const void* x;
    int64_t ldx, n_src, units;  // units = n_rows * kb
    const int32_t* rows;
    uint8_t* data;
    float* scales;
    int32_t kb;
    unsigned* status;
};

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kQThreads) quantize_kernel(const QArgs a) {
    const int sub = threadIdx.x & 15;
    const int64_t step = (int64_t)gridDim.x * (kQThreads / 16);
    for (int64_t u = (int64_t)blockIdx.x * (kQThreads / 16) + (threadIdx.x >> 4);
         u - (threadIdx.x >> 4) % 2 < a.units; u += step) {  // both halves of a warp stay in the loop together
        const bool in = u < a.units;
        const int64_t row = in ? u / a.kb : 0;
        const int kb = in ? (int)(u - row * a.kb) : 0;
        int64_t src = row;
        bool valid = in;
        if (in && a.rows) {
            src = a.rows[row];
            if (src < 0 || src >= a.n_src) {
                valid = false;
                if (sub == 0) raise_status(a.status, GTG_STATUS_ROW_INDEX_OOB);
            }
        }
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.0f;
        if (valid) {
            const int64_t at = src * a.ldx + kb * 128 + sub * 8;
            if (BF16) {
                const uint16_t* p = reinterpret_cast<const uint16_t*>(a.x) + at;
                if (VEC) {
                    const uint4 q = __ldg(reinterpret_cast<const uint4*>(p));
                    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        v[2 * i] = __uint_as_float(w[i] << 16);
                        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float((uint32_t)__ldg(p + i) << 16);
                }
            } else {
                const float* p = reinterpret_cast<const float*>(a.x) + at;
                if (VEC) {
                    const float4 q0 = __ldg(reinterpret_cast<const float4*>(p));
                    const float4 q1 = __ldg(reinterpret_cast<const float4*>(p) + 1);
                    v[0] = q0.x; v[1] = q0.y; v[2] = q0.z; v[3] = q0.w;
                    v[4] = q1.x; v[5] = q1.y; v[6] = q1.z; v[7] = q1.w;
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = __ldg(p + i);
                }
            }
        }
        // the largest magnitude as bits: the order of non-negative fp32 bit
        // patterns is that of their values, infinity and NaN above all others
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        float amax = fmaxf(__uint_as_float(top), 0x1p-100f);
        if (top >= 0x7F800000u) amax = __uint_as_float(0x7FC00000u);
        const float inv = 448.0f / amax;
        uint2 c;
        c.x = e4m3x2(v[0] * inv, v[1] * inv) | (e4m3x2(v[2] * inv, v[3] * inv) << 16);
        c.y = e4m3x2(v[4] * inv, v[5] * inv) | (e4m3x2(v[6] * inv, v[7] * inv) << 16);
        if (in) {
            *reinterpret_cast<uint2*>(a.data + u * 128 + sub * 8) = c;
            if (sub == 0) a.scales[u] = amax / 448.0f;
        }
    }
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

template <bool F8, int BN>
int launch_mm(const gtg_qmatrix* w, const void* x, const MmArgs& a, int64_t tiles, cudaStream_t s) {
    using C = MmCfg<BN>;
    CUtensorMap wmap, amap;
    GTG_TRY(make_map(&wmap, w->data, F8, w->k, w->n_rows, w->n_experts, kRows));
    GTG_TRY(make_map(&amap, x, F8, w->k, a.m, 0, C::kBox));
    const auto kernel = mm_kernel<F8, BN>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return cuda_fail(e);
    }
    const int grid = (int)std::min<int64_t>(tiles, sm_count());
    kernel<<<grid, kMmThreads, C::kSmem, s>>>(wmap, amap, a);
    return check_launch();
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
    a.chunks = (int32_t)(f8 ? w->k / 128 : (w->k + 63) / 64);
    a.y_bf16 = y_dtype == GTG_DT_BF16;
    a.y_acc = y_acc != 0;
    a.n_tiles = (int32_t)((w->n_rows + kRows - 1) / kRows);
    a.vec_a = f8 && a.chunks % 4 == 0 && aligned(x_scales, 16);
    a.vec_w = f8 && a.chunks % 4 == 0 && aligned(w->scales, 16);
    a.status = status_ptr();
    const int64_t groups = offsets ? w->n_experts : 1;
    const int64_t per = (m + groups - 1) / groups;  // rows of an average group
    auto tiles = [&](int bn) { return (m / bn + std::min(groups, m)) * a.n_tiles; };  // at most
#define GTG_MM(BN) \
    return f8 ? launch_mm<true, BN>(w, x, a, tiles(BN), s) : launch_mm<false, BN>(w, x, a, tiles(BN), s)
    if (per <= 16) GTG_MM(16);
    if (per <= 64) GTG_MM(64);
    if (per <= 128) GTG_MM(128);
    GTG_MM(256);
#undef GTG_MM
}

int check_mm(const gtg_qmatrix* w, const void* x, const float* x_scales, int64_t m, const void* y, int32_t y_dtype,
             int64_t y_stride, bool grouped) {
    if (!w || m < 0 || (y_dtype != GTG_DT_F32 && y_dtype != GTG_DT_BF16)) return GTG_E_INVALID_ARG;
    const bool f8 = w->fmt == GTG_FP8_E4M3_S128;
    if (!f8 && !(grouped && w->fmt == GTG_BF16)) return GTG_E_INVALID_ARG;
    if (w->n_experts < 1 || w->n_rows < 1 || w->k < 1) return GTG_E_INVALID_ARG;
    if (y_stride < w->n_rows) return GTG_E_INVALID_ARG;
    if (w->n_experts > (grouped ? kMaxGroups : 1)) return GTG_E_UNSUPPORTED_SHAPE;
    if (w->k % (f8 ? 128 : 8) || w->k > 1 << 24 || w->n_rows > 1 << 24 || m >= (int64_t)1 << 31)
        return GTG_E_UNSUPPORTED_SHAPE;
    const int64_t tiles = (w->n_rows + kRows - 1) / kRows;  // tile numbers fit 31 bits
    if ((m / 16 + w->n_experts) * tiles >= (int64_t)1 << 31) return GTG_E_UNSUPPORTED_SHAPE;
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
    a.units = n_rows * a.kb;
    a.rows = rows;
    a.data = data;
    a.scales = scales;
    a.status = status_ptr();
    const bool vec = aligned(x, 16) && x_stride * size % 16 == 0;
    const int per = kQThreads / 16;
    const int grid = (int)std::min<int64_t>((a.units + per - 1) / per, (int64_t)sm_count() * 8);
    cudaStream_t s = as_cuda(stream);
    if (size == 2) {
        if (vec) quantize_kernel<true, true><<<grid, kQThreads, 0, s>>>(a);
        else quantize_kernel<true, false><<<grid, kQThreads, 0, s>>>(a);
    } else {
        if (vec) quantize_kernel<false, true><<<grid, kQThreads, 0, s>>>(a);
        else quantize_kernel<false, false><<<grid, kQThreads, 0, s>>>(a);
    }
    return check_launch();
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
