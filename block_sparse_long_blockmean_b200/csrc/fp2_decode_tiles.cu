// fp2_decode_tiles.cu -- fp2_decode for several new tokens a sequence (drafts that
// are checked at once): tiles of 128 keys against up to 32 packed query rows on
// the 5th-generation tensor core, head dimension 128.
//
// Mathematics as in fp2_decode.cu, with the keys as the product's 128 rows:
//   S^T (128 keys x 32 rows)  = K (128 x d) Q^T           both K-major
//   O^T (128 d x 32 rows)    += V^T (d x 128 keys) P^T    both MN-major, as stored
// so that neither K nor V is transposed or converted; a thread owns one key's
// logits and, at the end, one d of the outputs.
//
// The weights P need more than one 8-bit (or bf16) operand to keep their
// precision.  e4m3 caches: w is rounded to fp16 (11 bits; as in fp2_decode.cu) and cut
// into three e5m2 terms, each what is left rounded to 3 bits.  e5m2 is fp16's upper half,
// so a term is an addition and a mask, and the rest an exact subtraction.  What is left is
// multiplied by 16 before the next term, and that term's accumulators by 1/16 when the
// segment ends: of a value in [2^e, 2^(e+1)) the rest is at most 2^(e-3), so 2^(e+1) after
// it, no term overflows, and the least of the third is 2^-24, fp16's own.  The terms sum to
// the fp16 value, whatever it is in 0 .. 2^15.  (Unscaled terms end at e5m2's least, 2^-16,
// where a key 17 below the row's largest logit is lost, and with it a whole tail beside one
// key, a sink, that lies so far above the rest: 4 drafts on 256K keys 102.4 us, scaled 104.8.)
// bf16 caches: two bf16 terms.  The terms are columns of one product, so V is read once; their
// accumulators are added when the segment ends.
//
// Keys that only some of the tile's tokens see (at most 15, the new ones) stay out
// of the second product, where a weight of 0 would not keep a value that is not
// finite out of the other rows' sums: their logits and values are set aside as their
// tile passes, and added row by row when the segment ends.
//
// Warpgroups of four warps take the softmax, a thread a key; one more warp copies,
// one issues the products.  They meet in mbarriers only, so that the copies run on
// into the next segment.
//
// Bound by the cache's bytes and, some 8 us above them, by the softmax's instructions: 4
// tokens x 8 heads on 262144 e4m3 keys with factors (537 MB) 105 us, 5.1 TB/s (the
// copies and products alone, with no softmax, 93); on 2 x 32768 bf16 keys (268 MB) 53 us.  A
// run of seconds reaches the power limit and 1.64 GHz: 120 us.  On short keys a segment's end
// counts, where the rows pass through shared memory between barriers: 28 live sequences of
// 2048 e4m3 keys (119 MB) 45 us, of 500 bf16 keys (59 MB) 27.  K and V in one ring, when it was
// split: 133 us where two took 105 (a value's place stays taken until its product, a key's only
// until its logits).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp2_decode.cuh"

namespace fp2 {

namespace {

constexpr int kTileKeys = 128, kTileRows = 32;
constexpr float kTermScale = 16.f;  // between an e4m3 cache's terms of a weight

template <bool FP8>
struct Tile {
    static constexpr int DH = 128;
    static constexpr int RB = DH * (FP8 ? 1 : 2);
    static constexpr int HALVES = RB / 128;               // 128-byte columns of a row
    static constexpr int HALF = kTileKeys * 128;          // bytes of one
    static constexpr int STAGE = HALVES * HALF;           // a tile of K or of V
    // e4m3 tiles arrive faster than a warpgroup takes their softmax: two CTAs on each
    // SM (262144 keys at the time: 133 us; one, whose rows two warpgroups share, 141).  bf16
    // stages leave room for one CTA, and two warpgroups help it (2 x 32768 keys at the time:
    // 58 us, one warpgroup 78).
    static constexpr int PER_SM = FP8 ? 2 : 1;
    static constexpr int WGS = FP8 ? 1 : 2;               // softmax warpgroups
    static constexpr int H = kTileRows / WGS;             // rows of one
    static constexpr int WARPS = 4 * WGS + 2, THREADS = 32 * WARPS;
    // K is free once its logits are there, V only after its product
    static constexpr int K_STAGES = FP8 ? 2 : 3, V_STAGES = 3;
    static constexpr int TERMS = FP8 ? 3 : 2;             // operand terms of a weight
    static constexpr int PV_N = TERMS * kTileRows;        // columns of the second product, in 128 bytes a key
    static constexpr int KSTEP = FP8 ? 32 : 16;           // k of one product
    static constexpr int OFF_V = K_STAGES * STAGE;
    static constexpr int OFF_P = OFF_V + V_STAGES * STAGE;
    static constexpr int OFF_Q = OFF_P + HALF;
    static constexpr int SMEM = OFF_Q + HALVES * kTileRows * 128;
    static constexpr int O_COL = 64;                      // TMEM: S twice, then O
    static constexpr uint32_t TMEM = FP8 ? 256 : 128;
    static constexpr int CTAS = 148 * PER_SM;
    static_assert(O_COL + PV_N <= (int)TMEM && PER_SM * (SMEM + 9 * 1024) <= 228 * 1024, "on-chip memory");
};

enum { T_K_FULL = 0, T_K_EMPTY = 3, T_V_FULL = 6, T_V_EMPTY = 9, T_S_FULL = 12, T_S_FREE = 14, T_P_READY = 16, T_O_DONE = 18, T_Q_READY = 20, T_MEET, T_DRAIN, T_COUNT };
enum { kDetTileCopy = kDetWaitBase + 8, kDetTileMma, kDetTileSoftmax };

// Instruction descriptor with fp32 accumulation: operand formats a, b (kind::f16:
// 1 = bf16; kind::f8f6f4: 0 = e4m3, 1 = e5m2), MN-major operands, 128 x n.
__host__ __device__ constexpr uint32_t tile_idesc(uint32_t a, uint32_t b, bool mn_major, int n) {
    return (1u << 4) | (a << 7) | (b << 10) | ((mn_major ? 3u : 0u) << 15) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

// Barrier of a softmax warpgroup, and whether `x` holds in any of its threads.
__device__ __forceinline__ void softmax_sync(int wg) { asm volatile("bar.sync %0, 128;" ::"r"(1 + wg) : "memory"); }
__device__ __forceinline__ bool softmax_any(int wg, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x), "r"(1 + wg)
        : "memory");
    return r != 0;
}

// The largest of a value over the warp's lanes, in all of them.
__device__ __forceinline__ float warp_max(float x) {
    float y;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

// 32 lanes x 16 consecutive 32-bit TMEM columns.
__device__ __forceinline__ void tmem_ld16f(uint32_t at, float* f) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7]), "=f"(f[8]),
          "=f"(f[9]), "=f"(f[10]), "=f"(f[11]), "=f"(f[12]), "=f"(f[13]), "=f"(f[14]), "=f"(f[15])
        : "r"(at));
}
__device__ __forceinline__ void tmem_st16f(uint32_t at, const float* f) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(at),
        "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]), "f"(f[8]), "f"(f[9]), "f"(f[10]),
        "f"(f[11]), "f"(f[12]), "f"(f[13]), "f"(f[14]), "f"(f[15])
        : "memory");
}
template <int H>
__device__ __forceinline__ void tmem_load(uint32_t at, float (&f)[H]) {
    if constexpr (H == 32) tmem_ld32f(at, f);
    else tmem_ld16f(at, f);
    tmem_wait_ld();
}

__device__ __forceinline__ float2 e4m3_pair(uint16_t x) {
    uint32_t y;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(y) : "h"(x));
    return __half22float2(*reinterpret_cast<__half2*>(&y));
}
template <bool FP8>
__global__ void __launch_bounds__(Tile<FP8>::THREADS, Tile<FP8>::PER_SM)
    decode_tiles_kernel(const __grid_constant__ DecodeParams D, const __grid_constant__ DecodeMaps maps) {
    using C = Tile<FP8>;
    constexpr int R = kTileRows, H = C::H, WGS = C::WGS, DH = C::DH, RB = C::RB;
    constexpr int COPY_WARP = 4 * WGS, MMA_WARP = COPY_WARP + 1;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ __align__(8) uint64_t bars[T_COUNT];
    __shared__ uint32_t tmem_at;
    __shared__ int aborted;
    __shared__ float sm_red[4 * WGS][H], sm_m[R], sm_l[R], sm_f[R];
    // the keys that not every row sees: logits, then weights; value factors; values
    __shared__ float sm_w[16][R], sm_tf[16];
    __shared__ __align__(16) uint8_t sm_tv[16][RB];
    __shared__ __align__(16) float sm_sc[R], sm_nm[R];
    const KParams& p = D.p;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // adjacent CTAs take the heads of a group over the same keys, so that a token's
    // rows of both are read at about the same time
    const int c = blockIdx.y, hs = blockIdx.x;
    const uint32_t base = smem_u32(smem);
    if (threadIdx.x == 0) {
        for (int i = 0; i < T_COUNT; ++i)
            mbar_init(&bars[i], (i >= T_S_FREE && i < T_O_DONE) || i == T_Q_READY || i == T_MEET ? 4 * WGS : 1);
        fence_mbar_init();
        aborted = 0;
        prefetch_tmap(&maps.k);
        prefetch_tmap(&maps.v);
    }
    wait_previous();
    __shared__ Share found;
    Share x;
    if (!find_share<R, kTileKeys, C::WARPS>(D, c, gridDim.y, 0, hs == 0, found, x)) return;
    if (warp == MMA_WARP) {
        tmem_alloc(&tmem_at, C::TMEM);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_at;
    Segment g;
    int t = 0;  // tiles before the present one, over all segments: stages and phases follow it

    if (warp == COPY_WARP) {
        // ------------------------------------------------------------ copies ---
        bool ok = true;
        int k_copies = 0;  // t, or one more if V's copy failed
        while (ok && next_segment<R, kTileKeys>(D, x, g)) {
            const int hk = g.group * D.hc + hs, n_tiles = g.x1 - g.x0;
            // lane 8 i + j: cache row of box j of tile 4 k + i, the next round of 4 tiles on
            // its way, unchecked; a box is a page, or a tile where pages are larger
            const int lane_key = (lane >> 3) * kTileKeys + (lane & 7) * D.box;
            auto key_of = [&](int n) { return (g.x0 + n) * kTileKeys + lane_key; };
            auto wanted = [&](int n) {
                return n + (lane >> 3) < n_tiles && (lane & 7) * D.box < kTileKeys && key_of(n) < g.seen_any;
            };
            int now = -1, next = wanted(0) ? raw_row(D, x.s, x.b, key_of(0)) : 0;
            for (int n = 0; n < n_tiles; ++n, ++t) {
                if ((n & 3) == 0) {
                    now = wanted(n) ? checked_row(D, next, key_of(n)) : -1;
                    if (wanted(n + 4)) next = raw_row(D, x.s, x.b, key_of(n + 4));
                }
                const bool withheld = n + 1 == p.withhold_k_item;  // (tests of the waits' limit)
                const bool mine = (lane >> 3) == (n & 3) && now >= 0 && !withheld;
                const int bytes = __popc(__ballot_sync(~0u, mine)) * D.box * RB;
                // one of the tile's operands into its ring
                auto copy = [&](const CUtensorMap* map, int stages, int offset, int full, int empty) {
                    const int st = t % stages;
                    if (t >= stages && !__all_sync(~0u, mbar_wait(&bars[empty + st], (t / stages - 1) & 1, &aborted, p.wait_limit_ns)))
                        return false;
                    if (lane == 0 && !withheld) mbar_arrive_expect_tx(&bars[full + st], bytes);
                    __syncwarp();
                    if (mine) {
                        const uint32_t dst = base + offset + st * C::STAGE + (lane & 7) * D.box * 128;
#pragma unroll
                        for (int h = 0; h < C::HALVES; ++h)
                            tma_load_3d(dst + h * C::HALF, map, &bars[full + st], h * (FP8 ? 128 : 64), hk, now);
                    }
                    return true;
                };
                ok = copy(&maps.k, C::K_STAGES, 0, T_K_FULL, T_K_EMPTY);
                if (ok) {
                    ++k_copies;
                    ok = copy(&maps.v, C::V_STAGES, C::OFF_V, T_V_FULL, T_V_EMPTY);
                }
                if (!ok) {
                    if (lane == 0) set_error(p.err, kErrTimeout, kDetTileCopy);
                    break;
                }
            }
            x.u = g.item_at + g.x1;
        }
        // never leave with copies in flight
        int ignore = 0;
        for (int i = max(0, k_copies - C::K_STAGES); i < k_copies; ++i)
            mbar_wait(&bars[T_K_FULL + i % C::K_STAGES], (i / C::K_STAGES) & 1, &ignore, kDrainNs);
        for (int i = max(0, t - C::V_STAGES); i < t; ++i)
            mbar_wait(&bars[T_V_FULL + i % C::V_STAGES], (i / C::V_STAGES) & 1, &ignore, kDrainNs);
    } else if (warp == MMA_WARP) {
        // ---------------------------------------------------------- products ---
        if (lane == 0) {
            constexpr uint32_t fmt = FP8 ? 0u : 1u;
            constexpr uint32_t idesc_qk = tile_idesc(fmt, fmt, false, R);
            constexpr uint32_t idesc_pv = tile_idesc(fmt, 1u, true, C::PV_N);  // e4m3 x e5m2, bf16 x bf16
            // descriptors of the first stage; others differ in the address field (16 bytes a
            // unit), which no sum below carries out of: one thread issues everything, so
            // its own instructions count
            const uint64_t dk = sw128_desc(base, 16, 1024), dq = sw128_desc(base + C::OFF_Q, 16, 1024);
            const uint64_t dv = sw128_desc(base + C::OFF_V, C::HALF, 1024), dp = sw128_desc(base + C::OFF_P, C::HALF, 1024);
            bool ok = true;
            int k_stage = 0, k_phase = 0, v_stage = 0, v_phase = 0;
            for (int seg = 0; ok && next_segment<R, kTileKeys>(D, x, g); ++seg) {
                const int n_tiles = g.x1 - g.x0;
                ok = mbar_wait(&bars[T_Q_READY], seg & 1, &aborted, p.wait_limit_ns);
                for (int n = 0; ok && n <= n_tiles; ++n) {
                    if (n < n_tiles) {
                        const int i = t + n, buf = i & 1;
                        ok = mbar_wait(&bars[T_K_FULL + k_stage], k_phase, &aborted, p.wait_limit_ns) &&
                             (i < 2 || mbar_wait(&bars[T_S_FREE + buf], (i / 2 - 1) & 1, &aborted, p.wait_limit_ns));
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t at = dk + (uint32_t)(k_stage * (C::STAGE >> 4));
#pragma unroll
                        for (int ks = 0; ks < DH / C::KSTEP; ++ks) {  // 32 bytes of d each
                            const uint64_t ad = at + (uint32_t)((ks >> 2) * (C::HALF >> 4) + (ks & 3) * 2);
                            const uint64_t bd = dq + (uint32_t)((ks >> 2) * (R * 128 >> 4) + (ks & 3) * 2);
                            if constexpr (FP8) mma_f8_ss(tmem + buf * R, ad, bd, idesc_qk, ks > 0);
                            else mma_bf16_ss(tmem + buf * R, ad, bd, idesc_qk, ks > 0);
                        }
                        mma_commit(&bars[T_S_FULL + buf]);
                        mma_commit(&bars[T_K_EMPTY + k_stage]);
                        if (++k_stage == C::K_STAGES) {
                            k_stage = 0;
                            k_phase ^= 1;
                        }
                    }
                    if (n >= 1) {
                        const int i = t + n - 1;
                        ok = mbar_wait(&bars[T_V_FULL + v_stage], v_phase, &aborted, p.wait_limit_ns) &&
                             mbar_wait(&bars[T_P_READY + (i & 1)], (i >> 1) & 1, &aborted, p.wait_limit_ns);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t at = dv + (uint32_t)(v_stage * (C::STAGE >> 4));
#pragma unroll
                        for (int ks = 0; ks < kTileKeys / C::KSTEP; ++ks) {  // KSTEP keys each
                            const uint64_t ad = at + (uint32_t)(ks * C::KSTEP * 8), bd = dp + (uint32_t)(ks * C::KSTEP * 8);
                            const uint32_t acc = n > 1 || ks > 0;
                            if constexpr (FP8) mma_f8_ss(tmem + C::O_COL, ad, bd, idesc_pv, acc);
                            else mma_bf16_ss(tmem + C::O_COL, ad, bd, idesc_pv, acc);
                        }
                        mma_commit(&bars[T_O_DONE + (i & 1)]);
                        mma_commit(&bars[T_V_EMPTY + v_stage]);
                        if (++v_stage == C::V_STAGES) {
                            v_stage = 0;
                            v_phase ^= 1;
                        }
                    }
                }
                t += n_tiles;
                x.u = g.item_at + g.x1;
            }
            if (!ok) set_error(p.err, kErrTimeout, kDetTileMma);
            // every product is done before TMEM is given back
            mma_commit(&bars[T_DRAIN]);
            int ignore = 0;
            mbar_wait(&bars[T_DRAIN], 0, &ignore, 100 * kDrainNs);
        }
    } else {
        // ----------------------------------------------------------- softmax ---
        const int wg = warp >> 2, w4 = warp & 3, first = wg * H;  // rows first .. first + H - 1
        const int tid = threadIdx.x & 127;  // key of the tile, TMEM lane; d of the output
        const uint32_t lanes = (uint32_t)(w4 * 32) << 16;
        float(*const red)[H] = sm_red + 4 * wg;
        // one arrival a warp: 32 on one barrier would queue
        auto arrive = [&](uint64_t* bar) {
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        // the product of tile i has read its weights and values
        auto product_done = [&](int i) { return mbar_wait(&bars[T_O_DONE + (i & 1)], (i >> 1) & 1, &aborted, p.wait_limit_ns); };
        bool ok = true, dead = false;  // this thread's waits; the warps' common verdict
        int meets = 0;                 // of the two warpgroups
        auto meet = [&] {
            arrive(&bars[T_MEET]);
            ok = mbar_wait(&bars[T_MEET], meets++ & 1, &aborted, p.wait_limit_ns) && ok;
            __syncwarp();
        };
        Lens s;                        // of the segment in hand
        int b = 0, hk = 0, n_tiles = 0;
        float l[H];
        auto token = [&](int r) { return token_of(D, g.tile * R + r); };
        auto head = [&](int r) { return hk * p.G + head_of(D, g.tile * R + r); };
        for (bool begun = false;; begun = true) {
            // the next segment's queries before this one's result: their place is free, all
            // logits are there, and the products go on meanwhile
            Segment next;
            const bool more = next_segment<R, kTileKeys>(D, x, next);
            if (more) {
                const int head0 = (next.group * D.hc + hs) * p.G;
                for (int i = tid; i < H * RB / 16; i += 128) {  // swizzled, rows past the last 0
                    const int r = first + i / (RB / 16), ch = i % (RB / 16), at = next.tile * R + r;
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (r < next.rows)
                        v = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(D.q) + ch * 16 +
                                                            ((long long)(x.s.q0 + token_of(D, at)) * p.Hq + head0 + head_of(D, at)) * RB);
                    *reinterpret_cast<uint4*>(smem + C::OFF_Q + (ch >> 3) * R * 128 + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) = v;
                }
                fence_proxy_async_smem();
                arrive(&bars[T_Q_READY]);
            }
            if (begun) {
                // ------------------------------------------ the segment's result ---
                // (code that runs once or twice is fetched as it runs, at 30 cycles an
                // instruction: what can be is a loop here)
                ok = product_done(t - 1) && ok;
                __syncwarp();
                if (softmax_any(wg, !ok)) {
                    dead = true;
                    break;
                }
                tc_fence_after();
                float o[H];
                tmem_load(tmem + lanes + C::O_COL + first, o);
                float down = 1.f;
#pragma unroll 1
                for (int k = 1; k < C::TERMS; ++k) {
                    float y[H];
                    tmem_load(tmem + lanes + C::O_COL + k * R + first, y);
                    down *= FP8 ? 1.f / kTermScale : 1.f;
#pragma unroll
                    for (int i = 0; i < H; ++i) o[i] = fmaf(y[i], down, o[i]);
                }
                tc_fence_before();
                // the weights' place in shared memory takes the rows: its last reader is done
                float* const rows = reinterpret_cast<float*>(smem + C::OFF_P) + first * DH;
#pragma unroll
                for (int i = 0; i < H; ++i) rows[i * DH + tid] = l[i];
                // the keys set aside in this segment: [from, to) of them
                const int from = max(0, g.x0 * kTileKeys - g.seen_all);
                const int to = min(g.seen_any, g.x1 * kTileKeys) - g.seen_all;
                softmax_sync(wg);
                if (WGS > 1 && to > from) {  // (the other warpgroup holds half of the values)
                    meet();
                    if (softmax_any(wg, !ok)) {
                        dead = true;
                        break;
                    }
                }
                {
                    constexpr int TPR = 128 / H;  // threads that add up a row, H keys each
                    const int r = first + tid / TPR;
                    float sum = 0.f;
#pragma unroll 2
                    for (int i = 0; i < H; i += 4) {
                        const float4 y = *reinterpret_cast<const float4*>(&rows[tid * H + (i + tid * 4) % H]);
                        sum += (y.x + y.y) + (y.z + y.w);
                    }
#pragma unroll
                    for (int i = 1; i < TPR; i <<= 1) sum += __shfl_xor_sync(~0u, sum, i);
                    if (tid % TPR == 0) {
                        const float m = -sm_nm[r];
                        float most = m;
                        for (int k = from; k < to; ++k) most = fmaxf(most, sm_w[k][r]);
                        const float f = ex2(m - most);
                        sum *= f;
#pragma unroll 1
                        for (int k = from; k < to; ++k) {
                            const float w = ex2(sm_w[k][r] - most);
                            sum += w;
                            sm_w[k][r] = FP8 ? w * sm_tf[k] : w;
                        }
                        sm_m[r] = most;
                        sm_l[r] = sum;
                        sm_f[r] = f;
                    }
                }
                softmax_sync(wg);
#pragma unroll
                for (int i = 0; i < H; ++i) rows[i * DH + tid] = o[i];
                softmax_sync(wg);
                const int slot = 2 * c + (g.x0 == 0 ? 1 : 0);
#pragma unroll 1
                for (int y = tid; y < min(H, g.rows - first) * (DH / 4); y += 128) {
                    const int col = y % (DH / 4) * 4, r = first + y / (DH / 4);
                    float4 O = scaled(*reinterpret_cast<const float4*>(&rows[(r - first) * DH + col]), sm_f[r]);
                    // the keys set aside that the row sees: the row's token is the last
                    const int seen_to = min(to, token(r) - g.t_first);
#pragma unroll 1
                    for (int k = from; k < seen_to; ++k) {
                        const uint8_t* v = sm_tv[k] + col * (FP8 ? 1 : 2);
                        float4 V;
                        if constexpr (FP8) {
                            const uint32_t u = *reinterpret_cast<const uint32_t*>(v);
                            const float2 lo = e4m3_pair((uint16_t)u), hi = e4m3_pair((uint16_t)(u >> 16));
                            V = make_float4(lo.x, lo.y, hi.x, hi.y);
                        } else {
                            const uint2 u = *reinterpret_cast<const uint2*>(v);
                            V = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                                            __uint_as_float(u.y & 0xFFFF0000u));
                        }
                        O = plus(O, V, sm_w[k][r]);
                    }
                    if (g.whole()) {
                        put_out<FP8>(D, s.q0 + token(r), head(r), col, O, sm_l[r]);
                        if (D.lse && col == 0) D.lse[(long long)(s.q0 + token(r)) * p.Hq + head(r)] = lse_of(sm_m[r], sm_l[r]);
                    } else {
                        const size_t at = ((size_t)slot * D.hc + hs) * R + r;
                        *reinterpret_cast<float4*>(D.part + at * DH + col) = O;
                        if (col == 0) *reinterpret_cast<float2*>(D.part_ml + at * 2) = make_float2(sm_m[r], sm_l[r]);
                    }
                }
                if (threadIdx.x == 0 && hs == 0) put_record(D, x, s.q0, b, g, c);
                // sm_* and P are free for the next segment
                if constexpr (WGS > 1) meet();
                else softmax_sync(wg);
            }
            if (!more) break;
            g = next;
            s = x.s;
            b = x.b;
            hk = g.group * D.hc + hs;
            n_tiles = g.x1 - g.x0;
#pragma unroll
            for (int i = 0; i < H; ++i) l[i] = 0.f;
            if (tid < H) {
                sm_nm[first + tid] = FLT_MAX;  // minus the row's reference
                // a logit's factor: rows differ by their head's scale
                if (FP8) sm_sc[first + tid] = D.qk_scale * p.k_scale[hk] * p.q_scale[head(min(first + tid, g.rows - 1))];
            }
            softmax_sync(wg);
            auto factors = [&](int n) {  // of tile n's key block; used a tile later
                if (!FP8 || !p.kb_fac || n >= n_tiles) return make_float2(1.f, 1.f);
                const size_t at = ((size_t)b * p.nkb_max + g.x0 + n) * p.Hkv + hk;
                return make_float2(p.kb_fac[at], p.vb_fac[at]);
            };
            float2 fac_next = factors(0);
            for (int n = 0; n < n_tiles; ++n, ++t) {
                const int buf = t & 1, j0 = (g.x0 + n) * kTileKeys;
                float2 fac = fac_next;
                fac_next = factors(n + 1);
                if (FP8 && !(fac.x > 0.f && fac.x <= 1.f && fac.y > 0.f && fac.y <= 1.f)) {
                    set_error(p.err, kErrInvalid, kDetFactor);
                    fac = make_float2(1.f, 1.f);
                }
                ok = mbar_wait(&bars[T_S_FULL + buf], (t >> 1) & 1, &aborted, p.wait_limit_ns) && ok;
                __syncwarp();
                tc_fence_after();
                const bool seen = j0 + tid < g.seen_all;
                const bool edge = j0 + kTileKeys > g.seen_all;  // some of the tile's keys are not seen
                // the logits' factors and minus the references of rows 4 i .. 4 i + 3
                auto exponents = [&](float (&w)[H]) {
#pragma unroll
                    for (int i = 0; i < H; i += 4) {
                        const float4 m = *reinterpret_cast<const float4*>(&sm_nm[first + i]);
                        float4 f = make_float4(D.qk_scale, D.qk_scale, D.qk_scale, D.qk_scale);
                        if constexpr (FP8) {
                            f = *reinterpret_cast<const float4*>(&sm_sc[first + i]);
                            if (p.kb_fac) f = scaled(f, fac.x);
                        }
                        const float2 a = ffma2(make_float2(w[i], w[i + 1]), make_float2(f.x, f.y), make_float2(m.x, m.y));
                        const float2 b = ffma2(make_float2(w[i + 2], w[i + 3]), make_float2(f.z, f.w), make_float2(m.z, m.w));
                        w[i] = a.x;
                        w[i + 1] = a.y;
                        w[i + 2] = b.x;
                        w[i + 3] = b.y;
                    }
                };
                auto factor = [&](int i) { return FP8 ? sm_sc[first + i] * fac.x : D.qk_scale; };
                const uint32_t s_at = tmem + lanes + buf * R + first;
                const float room = FP8 && p.kb_fac ? room_of(fac.y) : 0.f;
                float w[H], top = -FLT_MAX;
                tmem_load(s_at, w);
                exponents(w);
#pragma unroll
                for (int i = 0; i < H; i += 2) top = max3f(top, w[i], w[i + 1]);
                if (softmax_any(wg, (seen && top > kRoof + room) || !ok)) {
                    if (softmax_any(wg, !ok)) {
                        dead = true;
                        break;
                    }
                    // the references move: each row's largest z over the tile's keys
                    tmem_load(s_at, w);
#pragma unroll
                    for (int i = 0; i < H; ++i) w[i] = seen ? w[i] * factor(i) : -INFINITY;
                    float top_of = 0.f;  // row `lane`'s
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        const float y = warp_max(w[i]);
                        if (lane == i) top_of = y;
                    }
                    if (lane < H) red[w4][lane] = top_of;
                    softmax_sync(wg);
                    if (tid < H) {
                        const float most = fmaxf(fmaxf(red[0][tid], red[1][tid]), fmaxf(red[2][tid], red[3][tid]));
                        const float least = fminf(fminf(red[0][tid], red[1][tid]), fminf(red[2][tid], red[3][tid]));
                        const float lift = lift_of<FP8>(most, least) + room;
                        const float old = sm_nm[first + tid];
                        const bool moves = most + old > kRoof + room;
                        sm_f[first + tid] = moves ? ex2(lift - most - old) : 1.f;
                        if (moves) sm_nm[first + tid] = lift - most;
                    }
                    softmax_sync(wg);
#pragma unroll
                    for (int i = 0; i < H; ++i) l[i] *= sm_f[first + i];
                    if (n > 0) {
                        ok = product_done(t - 1) && ok;
                        __syncwarp();
                        tc_fence_after();
#pragma unroll 1
                        for (int k = 0; k < C::TERMS; ++k) {
                            const uint32_t o_at = tmem + lanes + C::O_COL + k * R + first;
                            tmem_load(o_at, w);
#pragma unroll
                            for (int i = 0; i < H; ++i) w[i] *= sm_f[first + i];
#pragma unroll
                            for (int i = 0; i < H; i += 16) tmem_st16f(o_at + i, w + i);
                        }
                        tmem_wait_st();
                    }
                    tmem_load(s_at, w);
                    exponents(w);
                }
                // a key of the tile that is set aside: its place among them
                const int aside = j0 + tid < g.seen_any ? j0 + tid - g.seen_all : -1;
                if (edge) {
                    float z[H];
                    tmem_load(s_at, z);
                    if (aside >= 0) {
                        if (wg == 0) sm_tf[aside] = fac.y;
#pragma unroll
                        for (int i = 0; i < H; ++i)
                            sm_w[aside][first + i] = j0 + tid <= s.P + token(first + i) ? z[i] * factor(i) : -INFINITY;
                    }
                }
                tc_fence_before();
                arrive(&bars[T_S_FREE + buf]);
#pragma unroll
                for (int i = 0; i < H; ++i) w[i] = ex2(w[i]);
                if (edge && !seen) {
#pragma unroll
                    for (int i = 0; i < H; ++i) w[i] = 0.f;
                }
#pragma unroll
                for (int i = 0; i < H; i += 2) {
                    const float2 x = fadd2(make_float2(l[i], l[i + 1]), make_float2(w[i], w[i + 1]));
                    l[i] = x.x;
                    l[i + 1] = x.y;
                }
                // the operand terms: columns 32 k + row of the key's 128 bytes of P
                constexpr int CHUNKS = (FP8 ? C::TERMS : 4) * H / 16;
                uint4 out[CHUNKS];
                int chunk[CHUNKS];
                if constexpr (FP8) {
                    uint32_t left[H / 2];  // fp16 pairs: what the terms so far leave
#pragma unroll
                    for (int i = 0; i < H / 2; ++i) {
                        if (p.kb_fac) {
                            w[2 * i] *= fac.y;
                            w[2 * i + 1] *= fac.y;
                        }
                        asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(left[i]) : "f"(w[2 * i]), "f"(w[2 * i + 1]));
                    }
#pragma unroll
                    for (int k = 0; k < C::TERMS; ++k) {
                        uint32_t cut[H / 2];
#pragma unroll
                        for (int i = 0; i < H / 2; ++i) {
                            cut[i] = (left[i] + 0x00800080u) & 0xFF00FF00u;
                            if (k + 1 < C::TERMS)  // (x 16, kTermScale)
                                asm("{\n\t.reg .b32 r;\n\tsub.f16x2 r, %0, %1;\n\tmul.f16x2 %0, r, %2;\n\t}"
                                    : "+r"(left[i]) : "r"(cut[i]), "r"(0x4C004C00u));
                        }
#pragma unroll
                        for (int h = 0; h < H / 16; ++h) {
                            uint32_t v[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) v[e] = __byte_perm(cut[8 * h + 2 * e], cut[8 * h + 2 * e + 1], 0x7531);
                            out[k * (H / 16) + h] = make_uint4(v[0], v[1], v[2], v[3]);
                            chunk[k * (H / 16) + h] = 2 * k + first / 16 + h;
                        }
                    }
                } else {
#pragma unroll
                    for (int h = 0; h < H / 8; ++h) {
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float a = w[8 * h + 2 * e], b = w[8 * h + 2 * e + 1];
                            hi[e] = pack_bf16x2(a, b);
                            lo[e] = pack_bf16x2(a - __uint_as_float(hi[e] << 16), b - __uint_as_float(hi[e] & 0xFFFF0000u));
                        }
                        out[2 * h] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        out[2 * h + 1] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                        chunk[2 * h] = first / 8 + h;
                        chunk[2 * h + 1] = 4 + first / 8 + h;
                    }
                }
                if (n >= 1) {  // the weights' last reader
                    ok = product_done(t - 1) && ok;
                    __syncwarp();
                }
                uint8_t* const p_row = smem + C::OFF_P + tid * 128;
#pragma unroll
                for (int k = 0; k < CHUNKS; ++k) *reinterpret_cast<uint4*>(p_row + ((chunk[k] ^ (tid & 7)) << 4)) = out[k];
                if (edge) {
                    ok = mbar_wait(&bars[T_V_FULL + t % C::V_STAGES], (t / C::V_STAGES) & 1, &aborted, p.wait_limit_ns) && ok;
                    __syncwarp();
                }
                if (edge && !seen) {
                    // rows of V that are not every row's values: set aside, then 0
                    uint8_t* v = smem + C::OFF_V + (t % C::V_STAGES) * C::STAGE + tid * 128;
#pragma unroll
                    for (int h = 0; h < C::HALVES; ++h)
#pragma unroll
                        for (int e = wg * (8 / WGS); e < (wg + 1) * (8 / WGS); ++e) {
                            uint4* const at = reinterpret_cast<uint4*>(v + h * C::HALF + ((e ^ (tid & 7)) << 4));
                            if (aside >= 0) *reinterpret_cast<uint4*>(&sm_tv[aside][h * 128 + e * 16]) = *at;
                            *at = make_uint4(0u, 0u, 0u, 0u);
                        }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                arrive(&bars[T_P_READY + (t & 1)]);
            }
            if (dead) break;
            x.u = g.item_at + g.x1;
        }
        if (dead && lane == 0) set_error(p.err, kErrTimeout, kDetTileSoftmax);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM);
    }
    if (aborted && threadIdx.x == 0 && hs == 0) drop_records<R, kTileKeys>(D, found, x, c);
}

template <bool FP8>
cudaError_t launch(DecodeParams D, cudaStream_t s) {
    using C = Tile<FP8>;
    static std::atomic<unsigned long long> ready{0};
    cudaError_t e = allow_smem(decode_tiles_kernel<FP8>, C::SMEM, ready);
    if (e != cudaSuccess) return e;
    DecodeMaps maps;
    const bool wide = D.hc * C::RB >= 256 || D.p.Hkv == 1;
    D.box = D.p.paged && D.p.page_size < kTileKeys ? D.p.page_size : kTileKeys;
    if (!make_row_maps(D.p, D.k, D.v, D.box, wide, &maps.k, &maps.v)) return cudaErrorInvalidValue;
    return launch_early(decode_tiles_kernel<FP8>, dim3(D.hc, C::CTAS / D.hc), C::THREADS, C::SMEM, s, D, maps);
}

}  // namespace

cudaError_t launch_decode_tiles(const DecodeParams& D, cudaStream_t s) {
    return D.p.fp8 ? launch<true>(D, s) : launch<false>(D, s);
}
int decode_tile_ctas(bool fp8) { return fp8 ? Tile<true>::CTAS : Tile<false>::CTAS; }

}  // namespace fp2
