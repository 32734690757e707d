// fp2_decode.cu -- fp2_decode: exact attention of a few new tokens per sequence
// over the whole KV cache, split over the cache's length and joined.
//
// Mathematics: for a packed query row (token x head of a KV group) over keys
// j, with z_j = q . k_j / sqrt(d) in units of log2: m a reference near max z_j,
// l = sum 2^(z_j - m), o = sum 2^(z_j - m) v_j, taken in one pass with a running
// (m, l, o).  Two disjoint key ranges join by m = max(m1, m2), l = l1 2^(m1-m)
// + l2 2^(m2-m), o likewise; out = o / l, lse = ln 2 (m + log2 l).
//
// Split: the unit of work is 16 keys of one (sequence, KV head, row tile).  All
// units, in that order, are cut into equal shares, one per CTA, so lengths may
// differ at will; every CTA finds its own share from the lengths.  An item
// (sequence, head, tile) that lies in one share is finished there; one that
// spans several leaves a partial (m, l, o) per share in the workspace and the
// join kernel reduces them.
//
// Products: both on the tensor core with the keys (or the head dimension) as
// the 16 rows of an m16n8 product and 8 packed query rows as its columns:
//   S^T (16 keys x 8 rows)  = K (16 x d) Q^T (d x 8)
//   O^T (d x 8 rows)       += V^T (d x 16 keys) P^T (16 keys x 8 rows)
// so that a tile of one token and at most 8 group heads wastes nothing, and a
// lane holds the same two rows of S^T and O^T: the softmax's scaling never
// crosses lanes.  Decoding reads each K and V byte once for at most 4 tiles of
// 8 rows; it is bound by the cache's bytes, not by these products.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <float.h>

#include "fp2_launch.cuh"
#include "fp2_seq.cuh"

namespace fp2 {

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kUnit = 16;  // keys of a unit: a unit never crosses a page

// Shared memory and shares of a variant: rows of RB bytes, R = 8 NT packed rows.
// A stage of a warp's ring holds the K and V rows of one unit.
template <int DH, bool FP8, int NT>
struct Variant {
    static constexpr int R = 8 * NT;
    static constexpr int RB = DH * (FP8 ? 1 : 2);
    static constexpr int STAGE = 2 * kUnit * RB;
    static constexpr int STAGES = RB == 256 ? 3 : NT == 4 ? 5 : 4;
    static constexpr int RING = STAGES * STAGE;             // of one warp
    static constexpr int SMEM = kWarps * RING;
    static constexpr int PER_SM = RB == 256 || NT > 1 ? 2 : 3;  // CTAs (shared memory and registers)
    static constexpr int CTAS = 148 * PER_SM;
    static constexpr int OS = DH + 4;                       // row stride of the warps' join
    static_assert(R * OS * 4 <= RING, "a warp's partial rows fit its ring");
    static_assert(CTAS <= kDecCtas && R <= kDecRows, "workspace");
};

// Weights are taken relative to m = (largest z when m was set) - kLift and may
// grow to 2^kRoof before m moves: no maximum has to be found in most steps.
// fp16 weights then span 2^kRoof (its largest is just under 2^16) down to
// 2^-24, that is 2^-31 of the row's largest.
constexpr float kLift = 7.f, kRoof = 15.f;

struct Shape {
    long long units;  // of the sequence
    int per_item;     // units of one item: ceil(Lk / kUnit)
    int tiles;        // row tiles per head
};
template <int R>
__device__ __forceinline__ Shape seq_shape(const KParams& p, const SeqInfo& s) {
    Shape x;
    x.per_item = (s.Lk + kUnit - 1) / kUnit;
    x.tiles = (s.Lq * p.G + R - 1) / R;
    x.units = (long long)x.per_item * x.tiles * p.Hkv;
    return x;
}
template <int R>
__device__ __forceinline__ long long seq_units(const KParams& p, int b) {
    SeqInfo s;
    if (!load_seq(p, b, s) || s.Lq == 0) return 0;
    return seq_shape<R>(p, s).units;
}

// Sum of x over the CTA and the exclusive prefix of the calling thread.
__device__ __forceinline__ long long block_prefix(long long x, long long& total, long long* sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long y = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(~0u, y, o);
        if (lane >= o) y += u;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = y;
    __syncthreads();
    long long before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
    }
    return before + y - x;
}

// Output of one packed row: o (unnormalised) over l, rounded once.
__device__ __forceinline__ void put_out(const DecodeParams& D, long long row, int h, int col, float x) {
    const KParams& p = D.p;
    const long long at = (row * p.Hq + h) * p.d + col;
    if (p.out_fp8) {
        const float sc = p.out_scale ? p.out_scale[h] : p.v_scale[h / p.G];
        const uint32_t b = pack_e4m3x4(x / sc, 0.f, 0.f, 0.f);
        static_cast<uint8_t*>(D.out)[at] = (uint8_t)b;
    } else {
        static_cast<__nv_bfloat16*>(D.out)[at] = __float2bfloat16(x);
    }
}
__device__ __forceinline__ float lse_of(float m, float l) { return (m + log2f(l)) * 0.69314718055994531f; }

// 16 bytes to shared memory, zeros where !on (then nothing is read).
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
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
__device__ __forceinline__ void mma_e4m3(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two e4m3 -> two fp16, exact.
__device__ __forceinline__ uint32_t f16_of(uint16_t x) {
    uint32_t y;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(y) : "h"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float a, float b) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(d) : "f"(a), "f"(b));
    return d;
}

// The rows of V^T that product mt of O^T covers: bf16 16 consecutive ones in
// natural order; e4m3 (two values per 16-bit element of the transposing load)
// the even ones first.  Column of the head for accumulator pair i (0: rows
// 0-7 of the product, 1: rows 8-15) of lane group g.
template <bool FP8>
__device__ __forceinline__ int out_col(int mt, int i, int g) {
    return 16 * mt + (FP8 ? 2 * g + i : 8 * i + g);
}

template <int DH, bool FP8, int NT>
__global__ void __launch_bounds__(kThreads, Variant<DH, FP8, NT>::PER_SM) decode_kernel(DecodeParams D) {
    using V = Variant<DH, FP8, NT>;
    constexpr int R = V::R, RB = V::RB, OS = V::OS, STAGES = V::STAGES;
    constexpr int CPR = RB / 16;                    // 16-byte chunks of a row
    constexpr int QS = RB / 32;                     // k-steps of the first product
    constexpr int MT = DH / 16;                     // row blocks of the second
    constexpr int LROWS = 32 / CPR;                 // rows that a warp copies at once
    extern __shared__ __align__(1024) uint8_t ring[];
    __shared__ long long sums[kWarps];
    __shared__ int start_seq;
    __shared__ long long start_base, chunk_end;
    __shared__ float sm_m[kWarps][R], sm_l[kWarps][R];
    __shared__ float2 sm_fac[kWarps][STAGES];       // K, V scale factors of the unit in a stage
    const KParams& p = D.p;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t4 = lane & 3;
    uint8_t* const my_ring = ring + warp * V::RING;
    const uint32_t my_smem = smem_u32(my_ring);
    wait_previous();
    allow_next();

    // total units, this CTA's share of them, and the sequence that holds its first
    const int c = blockIdx.x;
    if (threadIdx.x == 0) D.record[2 * c] = make_int4(0, 0, 0, 0);
    long long total = 0, n = threadIdx.x < p.num_seqs ? seq_units<R>(p, threadIdx.x) : 0;
    long long at = block_prefix(n, total, sums);
    for (int b0 = kThreads; b0 < p.num_seqs; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        long long t;
        block_prefix(b < p.num_seqs ? seq_units<R>(p, b) : 0, t, sums);
        total += t;
    }
    // a share is at least one unit of each warp
    const long long want = (total + kWarps - 1) / kWarps;
    const int ctas = (int)(want < gridDim.x ? (want > 0 ? want : 1) : gridDim.x);
    if (c >= ctas || total == 0) return;
    auto share = [&](int i) { return total * i / ctas; };
    long long u = share(c);
    const long long u_end = share(c + 1);
    for (int b0 = 0;;) {
        if (n > 0 && at <= u && u < at + n) {
            start_seq = b0 + threadIdx.x;
            start_base = at;
        }
        if ((b0 += kThreads) >= p.num_seqs) break;
        const int b = b0 + threadIdx.x;
        // (the next chunk's sequences start where this chunk's end)
        if (threadIdx.x == kThreads - 1) chunk_end = at + n;
        __syncthreads();
        const long long base = chunk_end;
        long long t;
        n = b < p.num_seqs ? seq_units<R>(p, b) : 0;
        at = base + block_prefix(n, t, sums);
    }
    __syncthreads();
    int b = start_seq;
    long long seq_at = start_base;

    while (u < u_end && b < p.num_seqs) {
        SeqInfo s;
        if (!load_seq(p, b, s) || s.Lq == 0) {
            ++b;
            continue;
        }
        const Shape sh = seq_shape<R>(p, s);
        if (u >= seq_at + sh.units) {
            seq_at += sh.units;
            ++b;
            continue;
        }
        const int item = (int)((u - seq_at) / sh.per_item);
        const long long item_at = seq_at + (long long)item * sh.per_item;
        const int hk = item / sh.tiles, tile = item % sh.tiles;
        const int x0 = (int)(u - item_at);
        const int x1 = (int)min((long long)sh.per_item, u_end - item_at);

        // packed rows of the tile: row r is token (tile * R + r) / G, head r % G
        const int rows = min(R, s.Lq * p.G - tile * R);
        const int t_first = tile * R / p.G, t_last = (tile * R + rows - 1) / p.G;
        const int seen_all = s.P + t_first + 1;  // keys that every row of the tile sees
        const int seen_any = s.P + t_last + 1;   // keys past it are not read

        // ---- the copies of this warp: its units are kWarps apart ----
        const int first = x0 + warp;
        const int steps = x1 > first ? (x1 - first + kWarps - 1) / kWarps : 0;
        // lane i: cache row where unit 32 k + i of this warp starts, and the
        // unit's factors; loaded a round of 32 units ahead of their use
        int row_now, row_next;
        float2 fac_now, fac_next;
        auto load_round = [&](int n0, int& row, float2& fac) {
            const int x = first + (n0 + lane) * kWarps;
            const bool on = x < x1 && x * kUnit < seen_any;
            row = on ? (int)key_row(p, s, b, x * kUnit) : -1;
            fac = make_float2(1.f, 1.f);
            if (FP8 && p.kb_fac && on) {
                const size_t f = ((size_t)b * p.nkb_max + x * kUnit / p.B) * p.Hkv + hk;
                fac = make_float2(p.kb_fac[f], p.vb_fac[f]);
            }
        };
        load_round(0, row_now, fac_now);
        load_round(32, row_next, fac_next);
        const uint8_t* kbase = static_cast<const uint8_t*>(D.k) + (size_t)hk * RB + (lane % CPR) * 16;
        const uint8_t* vbase = static_cast<const uint8_t*>(D.v) + (size_t)hk * RB + (lane % CPR) * 16;
        const long long token = (long long)p.Hkv * RB;  // bytes between two tokens' rows
        const long long lane_row = (lane / CPR) * token;
        auto issue = [&](int i, int stage) {
            if (i < steps) {
                if (i > 0 && (i & 31) == 0) {
                    row_now = row_next;
                    fac_now = fac_next;
                    load_round(i + 32, row_next, fac_next);
                }
                const uint32_t dst = my_smem + stage * V::STAGE;
                const int row0 = __shfl_sync(~0u, row_now, i & 31);
                const int valid = row0 < 0 ? 0 : seen_any - (first + i * kWarps) * kUnit;
                if (FP8 && p.kb_fac && lane == (i & 31)) {
                    if (!(fac_now.x > 0.f && fac_now.x <= 1.f && fac_now.y > 0.f && fac_now.y <= 1.f)) {
                        set_error(p.err, kErrInvalid, kDetFactor);
                        fac_now = make_float2(1.f, 1.f);
                    }
                    sm_fac[warp][stage] = fac_now;
                }
                const long long from = (long long)max(row0, 0) * token + lane_row;
#pragma unroll
                for (int r0 = 0; r0 < kUnit; r0 += LROWS) {
                    const int r = r0 + lane / CPR;
                    const uint32_t to = dst + r * RB + (((lane % CPR) ^ (r & 7)) << 4);
                    const bool on = r < valid;
                    const long long off = on ? from + r0 * token : 0;
                    copy16(to, kbase + off, on);
                    copy16(to + V::STAGE / 2, vbase + off, on);
                }
            }
            copies_commit();
        };
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i) issue(i, i);

        // ---- this warp's query columns, running (m, l, o) ----
        uint32_t qf[NT][QS][2];
        float sc[NT][2], m[NT][2], l[NT][2], o[NT][MT][4];
        int last[NT][2];  // last visible key of rows 2 t4, 2 t4 + 1 of the tile
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int rq = nt * 8 + g;
            const int tok = (tile * R + rq) / p.G, h = hk * p.G + (tile * R + rq) % p.G;
            const uint8_t* q = static_cast<const uint8_t*>(D.q) + ((long long)(s.q0 + tok) * p.Hq + h) * RB + 4 * t4;
#pragma unroll
            for (int ks = 0; ks < QS; ++ks) {
                qf[nt][ks][0] = rq < rows ? *reinterpret_cast<const uint32_t*>(q + 32 * ks) : 0u;
                qf[nt][ks][1] = rq < rows ? *reinterpret_cast<const uint32_t*>(q + 32 * ks + 16) : 0u;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = min(nt * 8 + 2 * t4 + e, rows - 1);
                last[nt][e] = s.P + (tile * R + r) / p.G;
                sc[nt][e] = D.qk_scale;
                if constexpr (FP8) sc[nt][e] *= p.q_scale[hk * p.G + (tile * R + r) % p.G] * p.k_scale[hk];
                m[nt][e] = -FLT_MAX;
                l[nt][e] = 0.f;
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[nt][mt][e] = 0.f;
        }

        int stage = 0, fill = STAGES - 1;
        for (int i = 0; i < steps; ++i) {
            copies_wait<STAGES - 2>();
            __syncwarp();
            issue(i + STAGES - 1, fill);
            fill = fill + 1 == STAGES ? 0 : fill + 1;
            const uint32_t ks0 = my_smem + stage * V::STAGE, vs0 = ks0 + V::STAGE / 2;
            const int j0 = (first + i * kWarps) * kUnit;
            float z[NT][4];  // S^T: key g (+ 8 for 2, 3), rows 2 t4, 2 t4 + 1
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) z[nt][e] = 0.f;
            {
                const int r = (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
                for (int ks = 0; ks < QS; ++ks) {
                    uint32_t a[4];
                    ldsm4(a, ks0 + r * RB + (((2 * ks + (lane >> 4)) ^ (r & 7)) << 4));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        if constexpr (FP8) mma_e4m3(z[nt], a, qf[nt][ks][0], qf[nt][ks][1]);
                        else mma_bf16(z[nt], a, qf[nt][ks][0], qf[nt][ks][1]);
                    }
                }
            }
            float2 fac = make_float2(1.f, 1.f);
            if (FP8 && p.kb_fac) fac = sm_fac[warp][stage];
            if (j0 + kUnit > seen_all) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (j0 + g + (e >> 1) * 8 > last[nt][e & 1]) z[nt][e] = -INFINITY;
            }
            // exponents of the weights; m moves when one passes the roof
            float w[NT][4];
            bool grow = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[nt][e] = fmaf(z[nt][e], FP8 ? sc[nt][e & 1] * fac.x : sc[nt][e & 1], -m[nt][e & 1]);
                    grow |= w[nt][e] > kRoof;
                }
            if (__any_sync(~0u, grow)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float f = FP8 ? sc[nt][e] * fac.x : sc[nt][e];
                        float y = fmaxf(z[nt][e] * f, z[nt][e + 2] * f);
                        y = fmaxf(y, __shfl_xor_sync(~0u, y, 4));
                        y = fmaxf(y, __shfl_xor_sync(~0u, y, 8));
                        y = fmaxf(y, __shfl_xor_sync(~0u, y, 16));
                        if (y - m[nt][e] > kRoof) {
                            const float shrink = ex2(m[nt][e] - (y - kLift));
                            m[nt][e] = y - kLift;
                            l[nt][e] *= shrink;
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt) {
                                o[nt][mt][e] *= shrink;
                                o[nt][mt][e + 2] *= shrink;
                            }
                        }
                        w[nt][e] = fmaf(z[nt][e], f, -m[nt][e]);
                        w[nt][e + 2] = fmaf(z[nt][e + 2], f, -m[nt][e]);
                    }
            }
            {
                // weights as the 16-bit operand: fp16 (11 bits) beside e4m3 values;
                // beside bf16 ones two bf16 terms (16 bits), so that the weights'
                // rounding stays far below the output's
                uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[nt][e] = ex2(w[nt][e]);
                    l[nt][0] += w[nt][0] + w[nt][2];
                    l[nt][1] += w[nt][1] + w[nt][3];
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
                auto values = [&](int mt, uint32_t (&a)[4]) {  // V^T rows of product mt
                    if constexpr (FP8) {
                        // one load covers two products: 16 keys x 32 values
                        uint32_t v[4];
                        const int r = (lane & 7) + ((lane >> 3) & 1) * 8;
                        ldsm4_t(v, vs0 + r * RB + ((((mt & ~1) + (lane >> 4)) ^ (r & 7)) << 4));
                        const uint32_t x = __byte_perm(v[2 * (mt & 1)], 0, 0x3120), y = __byte_perm(v[2 * (mt & 1) + 1], 0, 0x3120);
                        a[0] = f16_of((uint16_t)x);
                        a[1] = f16_of((uint16_t)(x >> 16));
                        a[2] = f16_of((uint16_t)y);
                        a[3] = f16_of((uint16_t)(y >> 16));
                    } else {
                        const int r = (lane & 7) + (lane >> 4) * 8;
                        ldsm4_t(a, vs0 + r * RB + (((2 * mt + ((lane >> 3) & 1)) ^ (r & 7)) << 4));
                    }
                };
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
                        const int clear = max(0, s.P + tok + 1 - j0);
                        for (int y = clear * CPR + lane; y < kUnit * CPR; y += 32)
                            *reinterpret_cast<uint4*>(my_ring + (vs0 - my_smem) + y * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                        __syncwarp();
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
            }
            stage = stage + 1 == STAGES ? 0 : stage + 1;
        }
        copies_wait<0>();
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
                    sm_m[warp][r] = m[nt][e];
                    sm_l[warp][r] = y;
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    mine[r * OS + out_col<FP8>(mt, 0, g)] = o[nt][mt][e];
                    mine[r * OS + out_col<FP8>(mt, 1, g)] = o[nt][mt][e + 2];
                }
            }
        __syncthreads();
        const bool whole = x0 == 0 && x1 == sh.per_item;
        const int slot = 2 * c + (x0 == 0 ? 1 : 0);
        for (int y = threadIdx.x; y < rows * DH; y += kThreads) {
            const int r = y / DH, col = y % DH;
            float M = -FLT_MAX, L = 0.f, O = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w][r]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = ex2(sm_m[w][r] - M);
                L += f * sm_l[w][r];
                O += f * reinterpret_cast<const float*>(ring + w * V::RING)[r * OS + col];
            }
            const int tok = (tile * R + r) / p.G, h = hk * p.G + (tile * R + r) % p.G;
            if (whole) {
                put_out(D, s.q0 + tok, h, col, O * ((FP8 ? p.v_scale[hk] : 1.f) / L));
                if (D.lse && col == 0) D.lse[(long long)(s.q0 + tok) * p.Hq + h] = lse_of(M, L);
            } else {
                D.part[((size_t)slot * R + r) * DH + col] = O;
                if (col == 0) {
                    D.part_ml[((size_t)slot * R + r) * 2] = M;
                    D.part_ml[((size_t)slot * R + r) * 2 + 1] = L;
                }
            }
        }
        if (!whole && x0 == 0 && threadIdx.x == 0) {
            // the item goes on to the share that holds its last unit
            const long long end = item_at + sh.per_item - 1;
            int c1 = c + 1;
            while (share(c1 + 1) <= end) ++c1;
            D.record[2 * c] = make_int4(c1 - c + 1, s.q0, hk, tile);
            D.record[2 * c + 1] = make_int4(rows, 0, 0, 0);
        }
        __syncthreads();
        u = item_at + x1;
    }
}

// grid (shares, R): row r of the item that starts in share c and ends in a
// later one.  A warp adds up every kJoinWarps-th part, DH / 32 columns a lane.
constexpr int kJoinWarps = 8;
template <int DH, bool FP8, int NT>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(DecodeParams D) {
    constexpr int R = 8 * NT, E = DH / 32;
    __shared__ float sm_o[kJoinWarps][DH], sm_m[kJoinWarps], sm_l[kJoinWarps];
    wait_previous();
    allow_next();
    const KParams& p = D.p;
    const int c = blockIdx.x, r = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int4 rec = D.record[2 * c];
    if (rec.x == 0) return;
    if (r >= D.record[2 * c + 1].x) return;
    auto slot = [&](int i) { return ((size_t)(i == 0 ? 2 * c + 1 : 2 * (c + i)) * R + r); };
    float M = -FLT_MAX, L = 0.f, O[E];
#pragma unroll
    for (int e = 0; e < E; ++e) O[e] = 0.f;
#pragma unroll 4
    for (int i = warp; i < rec.x; i += kJoinWarps) {
        const float2 ml = *reinterpret_cast<const float2*>(D.part_ml + 2 * slot(i));
        const float* part = D.part + slot(i) * DH + lane * E;
        const float mn = fmaxf(M, ml.x), old = ex2(M - mn), f = ex2(ml.x - mn);
        M = mn;
        L = L * old + ml.y * f;
#pragma unroll
        for (int e = 0; e < E; ++e) O[e] = O[e] * old + part[e] * f;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sm_o[warp][lane * E + e] = O[e];
    if (lane == 0) {
        sm_m[warp] = M;
        sm_l[warp] = L;
    }
    __syncthreads();
    const int col = threadIdx.x;
    if (col >= DH) return;
    M = -FLT_MAX;
    L = 0.f;
    float o = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) M = fmaxf(M, sm_m[w]);
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
        const float f = ex2(sm_m[w] - M);
        L += f * sm_l[w];
        o += f * sm_o[w][col];
    }
    const int t = (rec.w * R + r) / p.G, h = rec.z * p.G + (rec.w * R + r) % p.G;
    put_out(D, rec.y + t, h, col, o * ((FP8 ? p.v_scale[rec.z] : 1.f) / L));
    if (D.lse && col == 0) D.lse[(long long)(rec.y + t) * p.Hq + h] = lse_of(M, L);
}

template <int DH, bool FP8, int NT>
cudaError_t launch(const DecodeParams& D, cudaStream_t s) {
    using V = Variant<DH, FP8, NT>;
    static std::atomic<unsigned long long> ready{0};
    cudaError_t e = allow_smem(decode_kernel<DH, FP8, NT>, V::SMEM, ready);
    if (e == cudaSuccess) e = launch_early(decode_kernel<DH, FP8, NT>, dim3(V::CTAS), kThreads, V::SMEM, s, D);
    if (e == cudaSuccess) e = launch_early(join_kernel<DH, FP8, NT>, dim3(V::CTAS, V::R), 32 * kJoinWarps, 0, s, D);
    return e;
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
