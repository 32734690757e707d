// fp2_decode.cu -- fp2_decode: exact attention of a few new tokens per sequence
// over the whole KV cache, split over the cache's length and joined.
//
// Mathematics: for a packed query row (token x head of a KV group) over keys
// j, with z_j = q . k_j / sqrt(d) in units of log2: m a reference near max z_j,
// l = sum 2^(z_j - m), o = sum 2^(z_j - m) v_j, taken in one pass with a running
// (m, l, o).  Two disjoint key ranges join by m = max(m1, m2), l = l1 2^(m1-m)
// + l2 2^(m2-m), o likewise; out = o / l, lse = ln 2 (m + log2 l).
//
// Split: the unit of work is 16 keys of one (sequence, group of hc adjacent KV
// heads, row tile).  All units, in that order, are cut into equal shares, so lengths
// may differ at will; every CTA finds its own share from the lengths.  A share is
// taken by hc / hw CTAs side by side, hw heads each.  An item (sequence, head group,
// tile) that lies in one share is finished there; one that spans several leaves a
// partial (m, l, o) per share in the workspace and a join kernel reduces them.
//
// Products: both on the tensor core with the keys (or the head dimension) as
// the 16 rows of an m16n8 product and 8 packed query rows as its columns:
//   S^T (16 keys x 8 rows)  = K (16 x d) Q^T (d x 8)
//   O^T (d x 8 rows)       += V^T (d x 16 keys) P^T (16 keys x 8 rows)
// so that a tile of one token and 8 group heads wastes nothing, and a lane holds the
// same two rows of S^T and O^T: the softmax's scaling never crosses lanes.
//
// Bound by the cache's bytes, each read once for up to 32 packed rows (more are several row
// tiles, items of their own, each of which reads the keys again: 8 tokens x 8 heads on
// 131072 e4m3 keys 108 us where 4 tokens take 60).  One sequence of 131072 bf16 keys, 32
// heads over 8 (537 MB): 87 us, 6.2 TB/s; 128 ragged ones to 8191 keys (2.13 GB): 316 us, 6.7
// TB/s; 8 e4m3 ones of 4K to 64K (486 MB): 85 us, 5.7 TB/s; 8 ragged bf16 ones to 4097 (73
// MB): 22 us, of which 4 pass before the first keys are there and 5 in the join; one of 1024:
// 6.8 us, the two launches; head dimension 64, 131072 keys (268 MB): 54 us, 5.0 TB/s, 128
// ragged (1.06 GB): 170 us, 6.3 TB/s.  Loads alone reach 6.55 TB/s in pieces of 256 bytes and
// 5.7 in pieces of 128.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp2_decode.cuh"

namespace fp2 {

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;  // (4: a CTA of hw = 1, 2 heads has 1 << (3 - hw) warps a head)
constexpr int kUnit = kDecBox;  // keys of a unit: one copy
constexpr int kWithheld = -2;   // instead of a row: a copy that does not come (tests of the waits' limit)
constexpr int kHeadBytes = 2048;  // of the heads' rows of a token that are read together

// Shared memory and shares of a variant: rows of RB bytes, R = 8 NT packed rows.
// Four warps a CTA, each with a ring of its own: a CTA of 8 warps on each SM leaves it
// idle at a segment's end (512 sequences of 500 e4m3 keys: 231 us where two of 4 warps took
// 177, before later steps brought them to 101).
// One tiled copy a unit, head and 128 bytes; a bulk copy per row took 134 us where
// this takes 95 (128-byte rows: the copies' number counts).
// A stage of a warp's ring holds the K and V rows of one unit and head, each as
// RB / 128 tiles of 16 rows x 128 bytes in the 128-byte swizzle (16-byte chunk c
// of row r at c ^ (r & 7)), as the tiled copies write them.
template <int DH, bool FP8, int NT>
struct Variant {
    static constexpr int R = 8 * NT;
    static constexpr int RB = DH * (FP8 ? 1 : 2);
    static constexpr int TILE = kUnit * 128;
    static constexpr int STAGE = 2 * kUnit * RB;
    static constexpr int STAGES = RB == 256 ? 3 : NT == 4 ? 5 : 4;
    static constexpr int RING = STAGES * STAGE;             // of one warp
    static constexpr bool Q_SMEM = NT == 4;                 // queries: shared memory or registers
    static constexpr int Q_BYTES = Q_SMEM ? R * DH * 2 : 0; // of one head
    static constexpr int SMEM = kWarps * RING + kDecHeads * Q_BYTES;
    static constexpr int PER_SM = RB == 256 || NT > 1 ? 2 : 3;  // CTAs (shared memory and registers)
    static constexpr int CTAS = 148 * PER_SM;
    static constexpr int OS = DH + 4;                       // row stride of the warps' join
    static_assert(R * OS * 4 <= RING, "a warp's partial rows fit its ring");
    static_assert(CTAS <= kDecCtas && R <= kDecRows, "workspace");
};
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
// Two 16 x 16 byte matrices, transposed: register 2 k + i of lane l holds bytes
// 4 (l % 4) .. + 3 of column l / 4 + 8 i of matrix k.
__device__ __forceinline__ void ldsm_bytes_t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool FP8>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (FP8) mma_f16(c, a, b0, b1);
    else mma_bf16(c, a, b0, b1);
}
// Two e4m3 -> two fp16, exact.
__device__ __forceinline__ uint32_t f16_of(uint32_t x, bool high) {
    uint32_t y;
    if (high)
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(y) : "r"(x));
    else
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(d) : "f"(a), "f"(b));
    return d;
}

// e4m3 values enter the products as fp16, converted here (the type's own mma.sync
// form runs as two fp16 products and converts both operands inside, one of them
// anew for every row tile: 4 drafted tokens on 2 x 131072 keys 199 us, so 172).
// A 32-bit register of four e4m3 values gives two 16-bit operand registers, so
// the products' k runs over the values (first product) or keys (second) in the
// order 0 1 | 4 5 | 8 9 | 12 13 | 2 3 | 6 7 | 10 11 | 14 15 of each 16.  The queries
// are laid out in that order; V's rows are loaded so that it comes out natural:
__device__ __forceinline__ int v_key(int i) {  // row i of the byte transpose
    return (i & 2) ? 8 + 2 * (i >> 2) + (i & 1) : 2 * (i >> 2) + (i & 1);
}

template <int DH, bool FP8, int NT>
__global__ void __launch_bounds__(kThreads, Variant<DH, FP8, NT>::PER_SM)
    decode_kernel(const __grid_constant__ DecodeParams D, const __grid_constant__ DecodeMaps maps) {
    using V = Variant<DH, FP8, NT>;
    constexpr int R = V::R, RB = V::RB, OS = V::OS, STAGES = V::STAGES;
    constexpr int QC = DH / 16;      // k-steps of 16 of the first product
    constexpr int MT = DH / 16;      // row blocks of the second
    extern __shared__ __align__(1024) uint8_t ring[];
    __shared__ int aborted;
    __shared__ float sm_m[kWarps][R], sm_l[kWarps][R];
    __shared__ float2 sm_fac[kWarps][STAGES];  // K, V scale factors of the unit in a stage
    __shared__ __align__(8) uint64_t full[kWarps][STAGES];
    const KParams& p = D.p;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t4 = lane & 3;
    // warp = head of the CTA + hw * (which of the kw warps that share its units)
    const int hw = D.hw, hs = warp & (hw - 1), kw = kWarps >> (hw - 1);
    uint8_t* const my_ring = ring + warp * V::RING;
    const uint32_t my_smem = smem_u32(my_ring);
    // adjacent CTAs take the heads of a group over the same keys
    const int c = blockIdx.y, h0 = blockIdx.x * hw;
    if (lane == 0) {
        for (int i = 0; i < STAGES; ++i) mbar_init(&full[warp][i], 1);
        fence_mbar_init();
        if (warp == 0) {
            aborted = 0;
            prefetch_tmap(&maps.k);
            prefetch_tmap(&maps.v);
        }
    }
    uint32_t phases = 0;  // parity of each stage's next completion
    wait_previous();

    __shared__ Share found;
    Share share;  // a share is at least one unit of each warp
    if (!find_share<R, kUnit, kWarps>(D, c, gridDim.y, 3 - hw, h0 == 0, found, share)) return;
    const Lens& s = share.s;
    Segment seg;
    while (next_segment<R, kUnit>(D, share, seg)) {
        const int b = share.b, group = seg.group, tile = seg.tile, rows = seg.rows;
        const int hk = group * D.hc + h0 + hs;
        const int x0 = seg.x0, x1 = seg.x1, t_first = seg.t_first, t_last = seg.t_last;
        const int seen_all = seg.seen_all, seen_any = seg.seen_any;

        // ---- the copies of this warp: its units are kw apart ----
        const int first = x0 + (warp >> (hw - 1));
        const int steps = x1 > first ? (x1 - first + kw - 1) >> (3 - hw) : 0;
        // lane i: cache row where unit 32 k + i of this warp starts, and the
        // unit's factors; the next round of 32 units is on its way, unchecked
        int row_now = -1, raw_next = 0;
        float2 fac_now = make_float2(1.f, 1.f), fac_next = fac_now;
        auto key_at = [&](int n) { return (first + n * kw) * kUnit; };
        auto fetch_round = [&](int n0) {
            const int n = n0 + lane;
            if (n >= steps) return;
            raw_next = raw_row(D, s, b, key_at(n));
            if (FP8 && p.kb_fac) {
                const size_t f = ((size_t)b * p.nkb_max + key_at(n) / kFactorKeys) * p.Hkv + hk;
                fac_next = make_float2(p.kb_fac[f], p.vb_fac[f]);
            }
        };
        auto begin_round = [&](int n0) {
            row_now = n0 + lane < steps ? checked_row(D, raw_next, key_at(n0 + lane)) : -1;
            if (n0 + lane + 1 == p.withhold_k_item) row_now = kWithheld;
            fac_now = fac_next;
            if (FP8 && p.kb_fac && !(fac_now.x > 0.f && fac_now.x <= 1.f && fac_now.y > 0.f && fac_now.y <= 1.f)) {
                set_error(p.err, kErrInvalid, kDetFactor);
                fac_now = make_float2(1.f, 1.f);
            }
            fetch_round(n0 + 32);
        };
        fetch_round(0);
        // the queries and their scales, on their way together with the page ids (a
        // row past the last repeats it: its results are not stored)
        auto q_row = [&](int hx, int r) {
            const int i = tile * R + min(r, rows - 1);
            return static_cast<const uint8_t*>(D.q) +
                   ((long long)(s.q0 + token_of(D, i)) * p.Hq + (group * D.hc + h0 + hx) * p.G + head_of(D, i)) * RB;
        };
        uint32_t q_raw[V::Q_SMEM ? 1 : NT][FP8 ? QC : 2 * QC];
        float q_scale[NT][2], k_scale = 1.f;
        if constexpr (!V::Q_SMEM) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const uint8_t* q = q_row(hs, nt * 8 + g) + 4 * t4;
#pragma unroll
                for (int i = 0; i < (FP8 ? QC : 2 * QC); ++i) q_raw[nt][i] = *reinterpret_cast<const uint32_t*>(q + 16 * i);
            }
        }
        if constexpr (FP8) {
            k_scale = p.k_scale[hk];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    q_scale[nt][e] = p.q_scale[hk * p.G + head_of(D, tile * R + min(nt * 8 + 2 * t4 + e, rows - 1))];
        }
        begin_round(0);
        auto issue = [&](int i, int stage) {
            if (i >= steps) return;
            if (i > 0 && (i & 31) == 0) begin_round(i);
            if (FP8 && p.kb_fac && lane == (i & 31)) sm_fac[warp][stage] = fac_now;
            const int row0 = __shfl_sync(~0u, row_now, i & 31);
            if (lane == 0) {
                uint64_t* bar = &full[warp][stage];
                const uint32_t dst = my_smem + stage * V::STAGE;
                if (row0 < 0) {  // a page id out of range, recorded: nothing is read
                    if (row0 != kWithheld) mbar_arrive(bar);
                } else {
                    mbar_arrive_expect_tx(bar, V::STAGE);
#pragma unroll
                    for (int h = 0; h < RB / 128; ++h) {
                        tma_load_3d(dst + h * V::TILE, &maps.k, bar, h * (FP8 ? 128 : 64), hk, row0);
                        tma_load_3d(dst + V::STAGE / 2 + h * V::TILE, &maps.v, bar, h * (FP8 ? 128 : 64), hk, row0);
                    }
                }
            }
        };
#pragma unroll 1
        for (int i = 0; i < STAGES - 1; ++i) issue(i, i);

        // ---- this warp's query columns, running (m, l, o) ----
        uint8_t* const q_smem = ring + kWarps * V::RING;
        if constexpr (V::Q_SMEM) {
            // [head][row][RB bytes], 16-byte chunk x at x ^ (row & 7) of each 8
            static_assert(!FP8, "16-bit queries");
            for (int y = threadIdx.x; y < hw * R * (RB / 16); y += kThreads) {
                const int ch = y % (RB / 16), r = y / (RB / 16) % R, hx = y / (RB / 16) / R;
                *reinterpret_cast<uint4*>(q_smem + hx * V::Q_BYTES + r * RB + ((ch ^ (r & 7)) << 4)) =
                    *reinterpret_cast<const uint4*>(q_row(hx, r) + ch * 16);
            }
            __syncthreads();
        }
        // operand registers of each 16-value step: two pairs of values
        uint32_t qf[V::Q_SMEM ? 1 : NT][QC][2];
        float sc[NT][2], neg_m[NT][2], l[NT][2], o[NT][MT][4];
        int last[NT][2];  // last visible key of rows 2 t4, 2 t4 + 1 of the tile
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if constexpr (!V::Q_SMEM) {
#pragma unroll
                for (int ch = 0; ch < QC; ++ch) {
                    qf[nt][ch][0] = FP8 ? f16_of(q_raw[nt][ch], false) : q_raw[nt][2 * ch];
                    qf[nt][ch][1] = FP8 ? f16_of(q_raw[nt][ch], true) : q_raw[nt][2 * ch + 1];
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = min(nt * 8 + 2 * t4 + e, rows - 1);
                last[nt][e] = s.P + token_of(D, tile * R + r);
                sc[nt][e] = D.qk_scale * (FP8 ? q_scale[nt][e] * k_scale : 1.f);
                neg_m[nt][e] = FLT_MAX;
                l[nt][e] = 0.f;
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nt][mt][e] = 0.f;
        }
        // lane parts of the matrix loads' addresses
        const uint32_t k_lane = ((lane & 7) + ((lane >> 3) & 1) * 8) * 128 + (((lane >> 4) ^ (lane & 7)) << 4);
        const int v_row = FP8 ? v_key(lane & 15) : (lane & 7) + (lane >> 4) * 8;
        const uint32_t v_lane = V::STAGE / 2 + v_row * 128 + (((FP8 ? lane >> 4 : (lane >> 3) & 1) ^ (v_row & 7)) << 4);
        const uint32_t q_lane = smem_u32(q_smem) + hs * V::Q_BYTES + ((lane & 7) + (lane >> 4) * 8) * DH * 2 +
                                ((((lane >> 3) & 1) ^ (lane & 7)) << 4);

        int stage = 0, fill = STAGES - 1;
        for (int i = 0; i < steps; ++i) {
            // (the warp's lanes go on or give up together)
            if (!__all_sync(~0u, mbar_wait(&full[warp][stage], (phases >> stage) & 1, &aborted, p.wait_limit_ns))) break;
            phases ^= 1u << stage;
            __syncwarp();
            issue(i + STAGES - 1, fill);
            fill = fill + 1 == STAGES ? 0 : fill + 1;
            const uint32_t at0 = my_smem + stage * V::STAGE;
            const int j0 = (first + i * kw) * kUnit;
            float z[NT][4];  // S^T: key g (+ 8 for 2, 3), rows 2 t4, 2 t4 + 1
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) z[nt][e] = 0.f;
            // one load: 16 keys x 32 bytes, a k-step of bf16 values or two of e4m3
#pragma unroll
            for (int ks = 0; ks < RB / 32; ++ks) {
                uint32_t x[4];
                ldsm4(x, ((at0 + k_lane) ^ ((ks & 3) << 5)) + (ks >> 2) * V::TILE);
#pragma unroll
                for (int half = 0; half < (FP8 ? 2 : 1); ++half) {
                    const int ch = FP8 ? 2 * ks + half : ks;
                    uint32_t a[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if constexpr (FP8) a[e] = f16_of(x[2 * half + (e & 1)], e >= 2);
                        else a[e] = x[e];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        if constexpr (!V::Q_SMEM) {
                            mma16<FP8>(z[nt], a, qf[nt][ch][0], qf[nt][ch][1]);
                        } else if (nt % 2 == 0) {
                            uint32_t q[4];
                            ldsm4(q, (q_lane ^ ((ch & 3) << 5)) + (ch >> 2) * 128 + nt * 8 * DH * 2);
                            mma16<FP8>(z[nt], a, q[0], q[1]);
                            mma16<FP8>(z[nt + 1], a, q[2], q[3]);
                        }
                    }
                }
            }
            float2 fac = make_float2(1.f, 1.f);
            float room = 0.f;
            if (FP8 && p.kb_fac) {
                fac = sm_fac[warp][stage];
                room = room_of(fac.y);
            }
            auto clear = [&](int from) {  // V rows from..15 of the stage
                for (int y = max(0, from) * 8 + lane; y < kUnit * 8; y += 32)
#pragma unroll
                    for (int h = 0; h < RB / 128; ++h)
                        *reinterpret_cast<uint4*>(my_ring + stage * V::STAGE + V::STAGE / 2 + h * V::TILE + y * 16) = make_uint4(0u, 0u, 0u, 0u);
                __syncwarp();
            };
            auto mask = [&](float (&x)[NT][4]) {  // keys that a row does not see
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (j0 + g + (e >> 1) * 8 > last[nt][e & 1]) x[nt][e] = -INFINITY;
            };
            if (j0 + kUnit > seen_all) mask(z);
            // exponents of the weights; m moves when one passes the roof
            float w[NT][4], top = -FLT_MAX;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float2 f = make_float2(sc[nt][0], sc[nt][1]);
                if (FP8 && p.kb_fac) f = make_float2(f.x * fac.x, f.y * fac.x);
                const float2 shift = make_float2(neg_m[nt][0], neg_m[nt][1]);
                const float2 x = ffma2(make_float2(z[nt][0], z[nt][1]), f, shift), y = ffma2(make_float2(z[nt][2], z[nt][3]), f, shift);
                w[nt][0] = x.x;
                w[nt][1] = x.y;
                w[nt][2] = y.x;
                w[nt][3] = y.y;
                top = max3f(max3f(top, x.x, x.y), y.x, y.y);
            }
            const bool grow = top > kRoof + room;
            if (__any_sync(~0u, grow)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float f = FP8 ? sc[nt][e] * fac.x : sc[nt][e];
                        float y = fmaxf(z[nt][e] * f, z[nt][e + 2] * f);
                        float least = y;  // of pairs of keys
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) {
                            y = fmaxf(y, __shfl_xor_sync(~0u, y, o));
                            if (FP8) least = fminf(least, __shfl_xor_sync(~0u, least, o));
                        }
                        if (y + neg_m[nt][e] > kRoof + room) {
                            const float lift = lift_of<FP8>(y, least) + room, shrink = ex2(lift - y - neg_m[nt][e]);
                            neg_m[nt][e] = lift - y;
                            l[nt][e] *= shrink;
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt) {
                                o[nt][mt][e] *= shrink;
                                o[nt][mt][e + 2] *= shrink;
                            }
                        }
                        w[nt][e] = fmaf(z[nt][e], f, neg_m[nt][e]);
                        w[nt][e + 2] = fmaf(z[nt][e + 2], f, neg_m[nt][e]);
                    }
            }
            // (again: a scale of 0, which stands for a head of zeros, or one whose product
            // with a factor is 0 has made NaN of -inf; the maxima above pass over it)
            if (FP8 && j0 + kUnit > seen_all) mask(w);
            {
                // weights as the 16-bit operand: fp16 (11 bits) beside e4m3 values; beside
                // bf16 ones two bf16 terms (16 bits).  Either rounding stays far below the
                // output's: against 64 bits the output is off by 0.0017 of its size with
                // 32-bit weights and with these.  (A second fp16 term: 512 sequences of 500
                // e4m3 keys 101 -> 105 us, 2 tokens on 2 x 32768 41 -> 45.)
                uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[nt][e] = ex2(w[nt][e]);
                    const float2 both = fadd2(make_float2(l[nt][0], l[nt][1]),
                                              fadd2(make_float2(w[nt][0], w[nt][1]), make_float2(w[nt][2], w[nt][3])));
                    l[nt][0] = both.x;
                    l[nt][1] = both.y;
                    if (FP8 && p.kb_fac) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) w[nt][e] *= fac.y;
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float x = w[nt][2 * e], y = w[nt][2 * e + 1];
                        if constexpr (FP8) {
                            hi[nt][e] = transpose8(pack_f16x2(x, y));
                        } else {
                            const uint32_t h = pack_bf16x2(x, y);
                            hi[nt][e] = transpose8(h);
                            lo[nt][e] = transpose8(
                                pack_bf16x2(x - __uint_as_float(h << 16), y - __uint_as_float(h & 0xFFFF0000u)));
                        }
                    }
                }
                uint32_t pair[4];  // e4m3: one load covers two products
                auto values = [&](int mt, uint32_t (&a)[4]) {  // V^T rows of product mt
                    if constexpr (FP8) {
                        if ((mt & 1) == 0) ldsm_bytes_t(pair, (at0 + v_lane) ^ (mt << 4));
#pragma unroll
                        for (int e = 0; e < 4; ++e) a[e] = f16_of(pair[2 * (mt & 1) + (e & 1)], e >= 2);
                    } else {
                        ldsm4_t(a, ((at0 + v_lane) ^ ((mt & 3) << 5)) + (mt >> 2) * V::TILE);
                    }
                };
                // rows of V past the last key that the tile sees: what the cache
                // holds there is no value of this sequence
                if (j0 + kUnit > seen_any) clear(seen_any - j0);
                if (t_first == t_last || j0 + kUnit <= seen_all) {
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        uint32_t a[4];
                        values(mt, a);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if constexpr (FP8) {
                                mma_f16(o[nt][mt], a, hi[nt][0], hi[nt][1]);
                            } else {
                                mma_bf16(o[nt][mt], a, hi[nt][0], hi[nt][1]);
                                mma_bf16(o[nt][mt], a, lo[nt][0], lo[nt][1]);
                            }
                        }
                    }
                } else {
                    // keys that only the later tokens of the tile see: a weight of 0
                    // would not keep a value that is not finite out of a product,
                    // so token by token, from the last, with the rows it does not
                    // see cleared
                    for (int tok = t_last; tok >= t_first; --tok) {
                        clear(s.P + tok + 1 - j0);
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            uint32_t a[4];
                            values(mt, a);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                float part[4] = {0.f, 0.f, 0.f, 0.f};
                                if constexpr (FP8) {
                                    mma_f16(part, a, hi[nt][0], hi[nt][1]);
                                } else {
                                    mma_bf16(part, a, hi[nt][0], hi[nt][1]);
                                    mma_bf16(part, a, lo[nt][0], lo[nt][1]);
                                }
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (last[nt][e & 1] == s.P + tok) o[nt][mt][e] += part[e];
                            }
                        }
                        __syncwarp();
                    }
                }
                // (generic writes before the next copy into the stage)
                if (j0 + kUnit > seen_all) fence_proxy_async_smem();
            }
            stage = stage + 1 == STAGES ? 0 : stage + 1;
        }
        if (*const_cast<volatile int*>(&aborted)) {
            // a copy did not come: recorded; the others' are waited for and the CTA ends
            if (lane == 0) set_error(p.err, kErrTimeout, kDetWaitBase);
            for (int i = 0; i < STAGES; ++i) {
                int ignore = 0;
                mbar_wait(&full[warp][i], (phases >> i) & 1, &ignore, kDrainNs);
            }
        }
        __syncwarp();

        // ---- the warps' parts of this segment, joined in shared memory ----
        float* mine = reinterpret_cast<float*>(my_ring);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float y = l[nt][e];
                y += __shfl_xor_sync(~0u, y, 4);
                y += __shfl_xor_sync(~0u, y, 8);
                y += __shfl_xor_sync(~0u, y, 16);
                const int r = nt * 8 + 2 * t4 + e;
                if (g == 0) {
                    sm_m[warp][r] = -neg_m[nt][e];
                    sm_l[warp][r] = y;
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    mine[r * OS + 16 * mt + g] = o[nt][mt][e];
                    mine[r * OS + 16 * mt + 8 + g] = o[nt][mt][e + 2];
                }
            }
        __syncthreads();
        if (aborted) {
            if (threadIdx.x == 0 && h0 == 0) drop_records<R, kUnit>(D, found, share, c);
            return;
        }
        const bool whole = seg.whole();
        const int slot = 2 * c + (x0 == 0 ? 1 : 0);
        for (int y = threadIdx.x; y < hw * rows * (DH / 4); y += kThreads) {
            const int col = y % (DH / 4) * 4, r = y / (DH / 4) % rows, hx = y / (DH / 4) / rows;
            float M = -FLT_MAX, L = 0.f;
            float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int w = hx; w < kWarps; w += hw) M = fmaxf(M, sm_m[w][r]);
            for (int w = hx; w < kWarps; w += hw) {
                const float f = ex2(sm_m[w][r] - M);
                L += f * sm_l[w][r];
                O = plus(O, *reinterpret_cast<const float4*>(ring + w * V::RING + (r * OS + col) * 4), f);
            }
            if (whole) {
                const int tok = token_of(D, tile * R + r), hkv = group * D.hc + h0 + hx, h = hkv * p.G + head_of(D, tile * R + r);
                put_out<FP8>(D, s.q0 + tok, h, col, O, L);
                if (D.lse && col == 0) D.lse[(long long)(s.q0 + tok) * p.Hq + h] = lse_of(M, L);
            } else {
                const size_t at = ((size_t)slot * D.hc + h0 + hx) * R + r;
                *reinterpret_cast<float4*>(D.part + at * DH + col) = O;
                if (col == 0) *reinterpret_cast<float2*>(D.part_ml + at * 2) = make_float2(M, L);
            }
        }
        if (threadIdx.x == 0 && h0 == 0) put_record(D, share, s.q0, b, seg, c);
        fence_proxy_async_smem();  // the ring held the warps' parts; copies come next
        __syncthreads();
        share.u = seg.item_at + x1;
    }
}

// What a join kernel reads of one item: part i of row r of the group's head hx
// lies in share first + i, in that share's second slot if the item starts there.
struct Item {
    int4 a, b;
    __device__ __forceinline__ int parts() const { return a.x; }
    __device__ __forceinline__ int rows() const { return b.x; }
    template <int R>
    __device__ __forceinline__ size_t at(const DecodeParams& D, int i, int hx, int r) const {
        return ((size_t)(2 * (b.y + i) + (i == 0 ? 1 : 0)) * D.hc + hx) * R + r;
    }
};
// Parts first, first + step, ... of a packed row, VEC columns a lane; BATCH of
// them are loaded at once, so that their latencies overlap.
template <int DH, int R, int VEC, int BATCH>
__device__ __forceinline__ void add_parts(const DecodeParams& D, const Item& item, int hx, int r, int first, int step, int lane,
                                          float& M, float& L, float (&O)[VEC]) {
    M = -FLT_MAX;
    L = 0.f;
#pragma unroll
    for (int e = 0; e < VEC; ++e) O[e] = 0.f;
    for (int i0 = first; i0 < item.parts(); i0 += BATCH * step) {
        float2 ml[BATCH];
        float part[BATCH][VEC];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int i = i0 + k * step;
            const bool on = i < item.parts();
            const size_t at = item.at<R>(D, i, hx, r);
            ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int e = 0; e < VEC; ++e) part[k][e] = 0.f;
            if (on) {
                ml[k] = *reinterpret_cast<const float2*>(D.part_ml + 2 * at);
                const float* from = D.part + at * DH + lane * VEC;
                if constexpr (VEC == 4) {
                    const float4 x = *reinterpret_cast<const float4*>(from);
                    part[k][0] = x.x;
                    part[k][1] = x.y;
                    part[k][2] = x.z;
                    part[k][3] = x.w;
                } else {
                    const float2 x = *reinterpret_cast<const float2*>(from);
                    part[k][0] = x.x;
                    part[k][1] = x.y;
                }
            }
        }
        float mn = M;
#pragma unroll
        for (int k = 0; k < BATCH; ++k) mn = fmaxf(mn, ml[k].x);
        const float old = ex2(M - mn);
        M = mn;
        L *= old;
#pragma unroll
        for (int e = 0; e < VEC; ++e) O[e] *= old;
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const float f = ex2(ml[k].x - mn);
            L += ml[k].y * f;
#pragma unroll
            for (int e = 0; e < VEC; ++e) O[e] += part[k][e] * f;
        }
    }
}
template <bool FP8, int R>
__device__ __forceinline__ void finish_row(const DecodeParams& D, const Item& item, int hx, int r, int col, float4 O, float M, float L) {
    const KParams& p = D.p;
    const int hkv = item.a.z * D.hc + hx, t = token_of(D, item.a.w * R + r), h = hkv * p.G + head_of(D, item.a.w * R + r);
    put_out<FP8>(D, item.a.y + t, h, col, O, L);
    if (D.lse && col == 0) D.lse[(long long)(item.a.y + t) * p.Hq + h] = lse_of(M, L);
}

constexpr int kJoinWarps = 16;

// Few items, each of many parts: grid (items, hc * packed rows), a CTA per row,
// whose warps add up every kJoinWarps-th part.  About 5 us, most of them its launch, two
// loads that wait for one another and code that is fetched as it runs: batches of
// 8 parts and unrolled sums over the warps took 0.7 us more.
template <int DH, bool FP8, int NT>
__global__ void __launch_bounds__(32 * kJoinWarps) join_rows_kernel(const __grid_constant__ DecodeParams D) {
    constexpr int R = 8 * NT, E = DH / 32;
    __shared__ __align__(16) float sm_o[kJoinWarps][DH];
    __shared__ float sm_m[kJoinWarps], sm_l[kJoinWarps];
    wait_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int hx = blockIdx.y % D.hc, r = blockIdx.y / D.hc;
    const Item item{D.record[2 * blockIdx.x], D.record[2 * blockIdx.x + 1]};
    if (item.parts() == 0 || r >= item.rows()) return;
    float M, L, O[E];
    add_parts<DH, R, E, 2>(D, item, hx, r, warp, kJoinWarps, lane, M, L, O);
#pragma unroll
    for (int e = 0; e < E; ++e) sm_o[warp][lane * E + e] = O[e];
    if (lane == 0) {
        sm_m[warp] = M;
        sm_l[warp] = L;
    }
    __syncthreads();
    const int col = threadIdx.x * 4;
    if (col >= DH) return;
    M = -FLT_MAX;
    L = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int w = 0; w < kJoinWarps; ++w) M = fmaxf(M, sm_m[w]);
#pragma unroll 4
    for (int w = 0; w < kJoinWarps; ++w) {
        const float f = ex2(sm_m[w] - M);
        L += f * sm_l[w];
        o = plus(o, *reinterpret_cast<const float4*>(&sm_o[w][col]), f);
    }
    finish_row<FP8, R>(D, item, hx, r, col, o, M, L);
}

// Many items, most of two or three parts: grid (shares, hc), the item that
// starts in share c and ends in a later one, a warp per row.
constexpr int kShareWarps = 8;
template <int DH, bool FP8, int NT>
__global__ void __launch_bounds__(32 * kShareWarps) join_shares_kernel(const __grid_constant__ DecodeParams D) {
    constexpr int R = 8 * NT;
    wait_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, hx = blockIdx.y;
    const Item item{D.record[2 * blockIdx.x], D.record[2 * blockIdx.x + 1]};
    if (item.parts() == 0) return;
    for (int r = warp; r < item.rows(); r += kShareWarps) {
        float M, L, O[4];
        const bool on = lane * 4 < DH;
        add_parts<DH, R, 4, 4>(D, item, hx, r, 0, 1, on ? lane : 0, M, L, O);
        if (on) finish_row<FP8, R>(D, item, hx, r, lane * 4, make_float4(O[0], O[1], O[2], O[3]), M, L);
    }
}

template <int DH, bool FP8, int NT>
cudaError_t launch(DecodeParams D, cudaStream_t s) {
    using V = Variant<DH, FP8, NT>;
    // more than 16 packed rows at head dimension 128: tiles on the 5th-generation tensor
    // core (4 tokens x 8 heads on 262144 e4m3 keys: 105 us, in this kernel's form of 32 rows
    // 169 when it was left).  Up to 16 rows here: 2 tokens x 8 heads, 98 live sequences of 500
    // keys, bf16 52.9 us, as tiles 57.4, e4m3 45.0 and 55.5; one of 200, 10.2 and 10.9, 10.6
    // and 12.2; 98 of 2500, 170 and 182, 116 and 118.  One long sequence is the better for
    // tiles (131072 keys: 93.8 and 86.8, 60.3 and 57.1), but the host does not know the lengths.
    constexpr bool TILES = DH == 128 && NT == 4;
    // (at least one: lengths above a limit of 0 have to be recorded)
    const int packed = D.p.max_seqlen_q > 0 ? D.p.max_seqlen_q * D.p.G : 1;
    // KV heads of an item: those whose rows of a token are 2 KB together, two of them in
    // a CTA where warps take its products, the others in the CTAs beside it, so that
    // the DRAM reads a token's heads at about the same time (128 ragged bf16 sequences:
    // 318 us, with 1 KB 321, with 512 bytes 338; 4 tokens on 2 x 32768 e4m3 keys: 42.6, 42.4
    // and 45.8)
    D.hw = TILES || D.p.Hkv % 2 ? 1 : 2;
    D.hc = kHeadBytes / V::RB;
    while (D.p.Hkv % D.hc || D.hc % D.hw) --D.hc;
    D.groups = D.p.Hkv / D.hc;
    D.tiles_max = (packed + V::R - 1) / V::R;
    const long long items = (long long)D.p.num_seqs * D.groups * D.tiles_max;
    const int shares = (TILES ? decode_tile_ctas(FP8) : V::CTAS) / (D.hc / D.hw);
    // join by item where an item spans some shares: its parts are shared out over 16 warps
    // a row (131072 keys: 87.8 us, by share 100.0); else by share, most of 2 or 3 parts
    // (64 sequences of 1024: 48.6 us, by item 55.0)
    D.few = items * 4 <= shares && D.p.num_seqs <= kThreads;
    cudaError_t e;
    if constexpr (TILES) {
        e = launch_decode_tiles(D, s);
    } else {
        static std::atomic<unsigned long long> ready{0};
        e = allow_smem(decode_kernel<DH, FP8, NT>, V::SMEM, ready);
        if (e != cudaSuccess) return e;
        DecodeMaps maps;
        // L2 fetches in pieces of 256 bytes where the item reads both halves
        const bool wide = D.hc * V::RB >= 256 || D.p.Hkv == 1;
        if (!make_row_maps(D.p, D.k, D.v, kUnit, wide, &maps.k, &maps.v)) return cudaErrorInvalidValue;
        e = launch_early(decode_kernel<DH, FP8, NT>, dim3(D.hc / D.hw, shares), kThreads, V::SMEM, s, D, maps);
    }
    if (e != cudaSuccess) return e;
    if (D.few)
        return launch_early(join_rows_kernel<DH, FP8, NT>, dim3((unsigned)items, D.hc * (packed < V::R ? packed : V::R)),
                            32 * kJoinWarps, 0, s, D);
    return launch_early(join_shares_kernel<DH, FP8, NT>, dim3(shares, D.hc), 32 * kShareWarps, 0, s, D);
}

template <int DH, bool FP8>
cudaError_t launch_rows(const DecodeParams& D, cudaStream_t s) {
    // the smallest tile that holds the rows of the longest sequence, up to 32
    const int rows = D.p.max_seqlen_q * D.p.G;
    return rows <= 8 ? launch<DH, FP8, 1>(D, s) : rows <= 16 ? launch<DH, FP8, 2>(D, s) : launch<DH, FP8, 4>(D, s);
}

}  // namespace

cudaError_t launch_decode(const DecodeParams& D, cudaStream_t s) {
    if (D.p.d == 128) return D.p.fp8 ? launch_rows<128, true>(D, s) : launch_rows<128, false>(D, s);
    return launch_rows<64, false>(D, s);
}

}  // namespace fp2
