// fp2_decode.cu -- fp2_decode: exact attention of a few new tokens per sequence
// over the whole KV cache, split over the cache's length and joined.
//
// Mathematics: for a packed query row (token x head of a KV group) over keys
// j, with z_j = q . k_j / sqrt(d) in units of log2: m = max z_j, l = sum
// 2^(z_j - m), o = sum 2^(z_j - m) v_j, taken in one pass with a running
// (m, l, o).  Two disjoint key ranges join by m = max(m1, m2), l = l1 2^(m1-m)
// + l2 2^(m2-m), o likewise; out = o / l, lse = ln 2 (m + log2 l).
//
// Split: the unit of work is 16 keys of one (sequence, KV head, row tile).  All
// units, in that order, are cut into equal shares, one per CTA, so lengths may
// differ at will; every CTA finds its own share from the lengths.  An item
// (sequence, head, tile) that lies in one share is finished there; one that
// spans several leaves a partial (m, l, o) per share in the workspace and the
// join kernel reduces them.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "fp2_seq.cuh"

namespace fp2 {

namespace {

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kUnit = 16;  // keys of a unit: a unit never crosses a page
constexpr int R = kDecRows;

struct Shape {
    long long units;  // of the sequence
    int per_item;     // units of one item: ceil(Lk / kUnit)
    int tiles;        // row tiles per head
};
__device__ __forceinline__ Shape seq_shape(const KParams& p, const SeqInfo& s) {
    Shape x;
    x.per_item = (s.Lk + kUnit - 1) / kUnit;
    x.tiles = (s.Lq * p.G + R - 1) / R;
    x.units = (long long)x.per_item * x.tiles * p.Hkv;
    return x;
}
__device__ __forceinline__ long long seq_units(const KParams& p, int b) {
    SeqInfo s;
    if (!load_seq(p, b, s) || s.Lq == 0) return 0;
    return seq_shape(p, s).units;
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

template <int DH, bool FP8>
__device__ __forceinline__ void load_row(const void* base, long long row, float* x) {
    // DH / 32 consecutive values of a row for this lane
    constexpr int E = DH / 32;
    const long long at = row * DH + (threadIdx.x & 31) * E;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if constexpr (FP8) {
            const uint8_t b = static_cast<const uint8_t*>(base)[at + e];
            x[e] = __half2float(__half(__nv_cvt_fp8_to_halfraw(b, __NV_E4M3)));
        } else {
            x[e] = __bfloat162float(static_cast<const __nv_bfloat16*>(base)[at + e]);
        }
    }
}

template <int DH, bool FP8>
__global__ void __launch_bounds__(kThreads) decode_kernel(DecodeParams D) {
    constexpr int E = DH / 32;
    const KParams& p = D.p;
    __shared__ long long sums[kWarps];
    __shared__ int start_seq;
    __shared__ long long start_base;
    __shared__ float sm_o[kWarps][R][DH];
    __shared__ float sm_m[kWarps][R], sm_l[kWarps][R];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

    // total units, and this CTA's share of them
    long long total = 0;
    for (int b0 = 0; b0 < p.num_seqs; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        long long t;
        block_prefix(b < p.num_seqs ? seq_units(p, b) : 0, t, sums);
        total += t;
    }
    // a share is at least one unit per warp
    const long long want = (total + kWarps - 1) / kWarps;
    const int ctas = (int)(want < gridDim.x ? (want > 0 ? want : 1) : gridDim.x);
    const int c = blockIdx.x;
    if (threadIdx.x == 0 && c < (int)gridDim.x) D.record[2 * c] = make_int4(0, 0, 0, 0);
    if (c >= ctas || total == 0) return;
    auto share = [&](int i) { return total * i / ctas; };
    long long u = share(c);
    const long long u_end = share(c + 1);

    // the sequence that holds unit u
    long long base = 0;
    for (int b0 = 0; b0 < p.num_seqs; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        long long t;
        const long long n = b < p.num_seqs ? seq_units(p, b) : 0;
        const long long at = base + block_prefix(n, t, sums);
        if (n > 0 && at <= u && u < at + n) {
            start_seq = b;
            start_base = at;
        }
        base += t;
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
        const Shape sh = seq_shape(p, s);
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
        float q[R][E], o[R][E], m[R], l[R];
        int last[R];  // the row's last visible key
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int t = (tile * R + r) / p.G, h = hk * p.G + (tile * R + r) % p.G;
            last[r] = r < rows ? s.P + t : -1;
            m[r] = -INFINITY;
            l[r] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) q[r][e] = o[r][e] = 0.f;
            if (r < rows) {
                load_row<DH, FP8>(D.q, (long long)(s.q0 + t) * p.Hq + h, q[r]);
                const float sc = D.qk_scale * (FP8 ? p.q_scale[h] * p.k_scale[hk] : 1.f);
#pragma unroll
                for (int e = 0; e < E; ++e) q[r][e] *= sc;
            }
        }
        for (int x = x0 + warp; x < x1; x += kWarps) {
            const int j0 = x * kUnit;
            const long long row0 = key_row(p, s, b, j0);
            if (row0 < 0) continue;
            float fk = 1.f, fv = 1.f;
            if (FP8 && p.kb_fac) {
                const size_t at = ((size_t)b * p.nkb_max + j0 / p.B) * p.Hkv + hk;
                fk = p.kb_fac[at];
                fv = p.vb_fac[at];
                if (!(fk > 0.f && fk <= 1.f && fv > 0.f && fv <= 1.f)) {
                    set_error(p.err, kErrInvalid, kDetFactor);
                    continue;
                }
            }
            for (int j = j0; j < min(s.Lk, j0 + kUnit); ++j) {
                float k[E], v[E];
                load_row<DH, FP8>(D.k, (row0 + j - j0) * p.Hkv + hk, k);
                load_row<DH, FP8>(D.v, (row0 + j - j0) * p.Hkv + hk, v);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    if (j > last[r]) continue;
                    float z = 0.f;
#pragma unroll
                    for (int e = 0; e < E; ++e) z += q[r][e] * k[e];
#pragma unroll
                    for (int w = 16; w > 0; w >>= 1) z += __shfl_xor_sync(~0u, z, w);
                    z *= fk;
                    const float mn = fmaxf(m[r], z), old = ex2(m[r] - mn), w = ex2(z - mn);
                    m[r] = mn;
                    l[r] = l[r] * old + w;
#pragma unroll
                    for (int e = 0; e < E; ++e) o[r][e] = o[r][e] * old + w * fv * v[e];
                }
            }
        }
        // the warps' parts of this segment, joined in shared memory
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
            for (int e = 0; e < E; ++e) sm_o[warp][r][lane * E + e] = o[r][e];
            if (lane == 0) {
                sm_m[warp][r] = m[r];
                sm_l[warp][r] = l[r];
            }
        }
        __syncthreads();
        const bool whole = x0 == 0 && x1 == sh.per_item;
        const int slot = 2 * c + (x0 == 0 ? 1 : 0);
        for (int r = warp; r < rows; r += kWarps) {
            float M = -INFINITY, L = 0.f, O[E];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w][r]);
#pragma unroll
            for (int e = 0; e < E; ++e) O[e] = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = sm_m[w][r] == -INFINITY ? 0.f : ex2(sm_m[w][r] - M);
                L += f * sm_l[w][r];
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (f != 0.f) O[e] += f * sm_o[w][r][lane * E + e];
            }
            const int t = (tile * R + r) / p.G, h = hk * p.G + (tile * R + r) % p.G;
            if (whole) {
                const float inv = (FP8 ? p.v_scale[hk] : 1.f) / L;
#pragma unroll
                for (int e = 0; e < E; ++e) put_out(D, s.q0 + t, h, lane * E + e, O[e] * inv);
                if (D.lse && lane == 0)
                    D.lse[(long long)(s.q0 + t) * p.Hq + h] = (M + log2f(L)) * 0.69314718055994531f;
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) D.part[((size_t)slot * R + r) * DH + lane * E + e] = O[e];
                if (lane == 0) {
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

// grid (shares, R), DH threads: row r of the item that starts in share c and
// ends in a later one.
template <int DH, bool FP8>
__global__ void __launch_bounds__(DH) join_kernel(DecodeParams D) {
    const KParams& p = D.p;
    const int c = blockIdx.x, r = blockIdx.y, col = threadIdx.x;
    const int4 rec = D.record[2 * c];
    if (rec.x == 0) return;
    if (r >= D.record[2 * c + 1].x) return;
    auto slot = [&](int i) { return ((size_t)(i == 0 ? 2 * c + 1 : 2 * (c + i)) * R + r); };
    float M = -INFINITY, L = 0.f, O = 0.f;
    for (int i = 0; i < rec.x; ++i) M = fmaxf(M, D.part_ml[2 * slot(i)]);
    for (int i = 0; i < rec.x; ++i) {
        const float m = D.part_ml[2 * slot(i)];
        if (m == -INFINITY) continue;
        const float f = ex2(m - M);
        L += f * D.part_ml[2 * slot(i) + 1];
        O += f * D.part[slot(i) * DH + col];
    }
    const int t = (rec.w * R + r) / p.G, h = rec.z * p.G + (rec.w * R + r) % p.G;
    put_out(D, rec.y + t, h, col, O * ((FP8 ? p.v_scale[rec.z] : 1.f) / L));
    if (D.lse && col == 0)
        D.lse[(long long)(rec.y + t) * p.Hq + h] = (M + log2f(L)) * 0.69314718055994531f;
}

template <int DH, bool FP8>
cudaError_t launch(const DecodeParams& D, cudaStream_t s) {
    const int ctas = 296;
    decode_kernel<DH, FP8><<<ctas, kThreads, 0, s>>>(D);
    join_kernel<DH, FP8><<<dim3(ctas, R), DH, 0, s>>>(D);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode(const DecodeParams& D, cudaStream_t s) {
    if (D.p.d == 128) return D.p.fp8 ? launch<128, true>(D, s) : launch<128, false>(D, s);
    return launch<64, false>(D, s);
}

}  // namespace fp2
