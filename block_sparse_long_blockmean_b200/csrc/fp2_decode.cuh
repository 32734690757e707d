// fp2_decode.cuh -- what the two decode kernels share: the split of the keys
// into shares, the output of a row, the records for the join.
#pragma once

#include <float.h>

#include "fp2_device.cuh"
#include "fp2_launch.cuh"

namespace fp2 {

constexpr uint64_t kDrainNs = 20000000ull;      // 20 ms per copy in flight after a wait has run out
constexpr int kFactorKeys = 128;                // keys that share their scale factors (e4m3's only block)
constexpr int kDecBox = 16;                     // rows of a copy: they never cross a page

// Weights are taken relative to m = (largest z when m was set) - kLift and may
// grow to 2^kRoof before m moves: no maximum has to be found in most steps.
// e4m3 caches: a weight times its value's factor is rounded to fp16, 11 bits down to
// 2^-14 and fewer below, to 2^-24.  Where the largest of the keys at hand lies far above
// others of them (`least`: the largest of some of them that it is not among), later keys
// will hardly pass it, while all of them may lie as far below: the room to grow is given
// up, bit for bit, for weights that keep their 11 bits down to 2^-(14 + kMostLift), 19.4
// in logits, below the largest.  (A lift of 12 for all: 2 drafted tokens on 2 x 32768
// e4m3 keys 40.6 -> 45.2 us, 4 on 2 x 131072 104 -> 126, as m moves more often.)
constexpr float kLift = 7.f, kMostLift = 14.f, kRoof = 15.f;
constexpr float kSpread = 12.f;  // of keys that lie together
template <bool FP8>
__device__ __forceinline__ float lift_of(float most, float least) {
    return FP8 ? fminf(kMostLift, kLift + fmaxf(0.f, most - least - kSpread)) : kLift;
}
// What is rounded is the product of the weight and its block's value factor f: it is kept in
// the range above, by moving the range of the weight (fp32, as are its sums) by 1 / f, so
// that blocks of small values keep their bits too.  Beyond 2^-60 they lose them.
__device__ __forceinline__ float room_of(float f) { return fminf(-__log2f(f), 60.f); }

struct DecodeMaps {
    CUtensorMap k, v;  // [rows][Hkv][d], boxes of some rows x 128 bytes of one head
};

// A sequence's lengths.  load_lens() checks them against the call's limits and records
// the error if they are bad.  Offsets are compared as they are, and differences taken
// without a sign: a signed one may be taken not to wrap, and the comparison dropped.
// (Short, like all code before the first copy: it is fetched as it runs, at about
// 30 cycles an instruction.)
struct Lens {
    int q0, Lq, Lk, k0, P;  // first query row, new tokens, keys, first key row, keys before the tokens
};
__device__ __forceinline__ bool load_lens(const DecodeParams& D, int b, Lens& s) {
    const KParams& p = D.p;
    const int q1 = p.cu_q[b + 1];
    s.q0 = p.cu_q[b];
    s.Lq = (int)((unsigned)q1 - (unsigned)s.q0);
    s.Lk = p.seqlens_k ? p.seqlens_k[b] : s.Lq;
    s.k0 = p.paged ? 0 : p.cu_k[b];
    s.P = (int)((unsigned)s.Lk - (unsigned)s.Lq);
    const bool lens_ok = s.q0 >= 0 && q1 >= s.q0 && q1 <= p.total_q && s.Lq <= p.max_seqlen_q && s.Lk >= s.Lq && s.Lk <= p.max_seqlen_k;
    const bool keys_ok = p.paged ? s.Lk <= (long long)p.max_pages * p.page_size : s.k0 >= 0 && s.Lk <= p.total_k - s.k0;
    if (lens_ok && keys_ok) return true;
    set_error(p.err, lens_ok ? kErrBounds : kErrInvalid, kDetSeqLen);
    return false;
}

struct Shape {
    long long units;  // of the sequence
    int per_item;     // units of one item: ceil(Lk / UNIT)
    int tiles;        // row tiles per head group
};
template <int R, int UNIT>
__device__ __forceinline__ Shape seq_shape(const DecodeParams& D, const Lens& s) {
    Shape x;
    x.per_item = (s.Lk + UNIT - 1) / UNIT;
    x.tiles = ((s.Lq << D.g_shift) + R - 1) / R;
    x.units = (long long)x.per_item * x.tiles * D.groups;
    return x;
}
// Sequence b's lengths and its units; 0 units if it rests or its lengths are bad.
template <int R, int UNIT>
__device__ __forceinline__ long long seq_units(const DecodeParams& D, int b, Lens& s) {
    if (!load_lens(D, b, s) || s.Lq == 0) return 0;
    return seq_shape<R, UNIT>(D, s).units;
}
// Packed row i of a sequence and KV head: its token, its query head within the group.
__device__ __forceinline__ int token_of(const DecodeParams& D, int i) { return i >> D.g_shift; }
__device__ __forceinline__ int head_of(const DecodeParams& D, int i) { return i & (D.p.G - 1); }
// a / b of values that mostly fit 32 bits.
__device__ __forceinline__ long long quotient(long long a, long long b) {
    if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
    return a / b;
}

// Cache row of key `key` in two steps, so that a page id can be on its way while
// other work is done: what has to be loaded, and the row, -1 (recorded) if it is bad.
__device__ __forceinline__ int raw_row(const DecodeParams& D, const Lens& s, int b, int key) {
    return D.p.paged ? D.p.page_table[(size_t)b * D.p.max_pages + (key >> D.page_shift)] : s.k0 + key;
}
__device__ __forceinline__ int checked_row(const DecodeParams& D, int raw, int key) {
    if (!D.p.paged) return raw;
    if (raw < 0 || raw >= D.p.num_pages) {
        set_error(D.p.err, kErrBounds, kDetPage);
        return -1;
    }
    return (raw << D.page_shift) + (key & (D.p.page_size - 1));
}

// Sum of x over the CTA of W warps and the exclusive prefix of the calling thread.
template <int W>
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
    for (int w = 0; w < W; ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
    }
    return before + y - x;
}

// Share c of `shares` at most: units [u, u_end) of `total` cut into `parts` equal
// shares, the first `more` of them with `each` + 1 units, the others with `each`;
// starting in sequence b, whose units start at seq_at and whose lengths are s (`found`, in
// shared memory, keeps these three).  False (for the whole CTA) if the share is empty.  The
// shares have about 2^least units or more.  With `records` also clears those that nobody
// else will write.
struct Share {
    long long u, u_end, seq_at, each, more;
    __device__ __forceinline__ long long start(int c) const { return c * each + (c < more ? c : more); }
    int b;
    Lens s;
    // the share that holds unit x
    __device__ __forceinline__ int of_unit(long long x) const {
        const long long large = more * (each + 1);
        return (int)(x < large ? quotient(x, each + 1) : more + quotient(x - large, each));
    }
};
template <int R, int UNIT, int W>
__device__ __forceinline__ bool find_share(const DecodeParams& D, int c, int shares, int least, bool records, Share& found, Share& x) {
    __shared__ long long sums[W];
    __shared__ long long chunk_end;
    const KParams& p = D.p;
    constexpr int T = 32 * W;
    Lens s;
    long long total = 0, n = (int)threadIdx.x < p.num_seqs ? seq_units<R, UNIT>(D, threadIdx.x, s) : 0;
    long long at = block_prefix<W>(n, total, sums);
    for (int b0 = T; b0 < p.num_seqs; b0 += T) {
        const int b = b0 + threadIdx.x;
        long long t;
        Lens y;
        block_prefix<W>(b < p.num_seqs ? seq_units<R, UNIT>(D, b, y) : 0, t, sums);
        total += t;
    }
    if (!records) {
    } else if (!D.few) {
        if (threadIdx.x == 0) D.record[2 * c] = make_int4(0, 0, 0, 0);
    } else if (c == 0 && (int)threadIdx.x < p.num_seqs) {
        // (few: a record per item, at most as many sequences as threads; the
        // tiles that this sequence does not have)
        const int tiles = n > 0 ? seq_shape<R, UNIT>(D, s).tiles : 0;
        for (int i = 0; i < D.groups; ++i)
            for (int j = tiles; j < D.tiles_max; ++j)
                D.record[2 * ((threadIdx.x * D.groups + i) * D.tiles_max + j)] = make_int4(0, 0, 0, 0);
    }
    const long long want = (total + (1 << least) - 1) >> least;
    const int parts = (int)(want < shares ? want : shares);
    if (c >= parts) return false;
    x.each = quotient(total, parts);
    x.more = total - x.each * parts;
    x.u = x.start(c);
    x.u_end = x.u + x.each + (c < x.more ? 1 : 0);
    for (int b0 = 0;;) {
        if (n > 0 && at <= x.u && x.u < at + n) {
            found.b = b0 + threadIdx.x;
            found.seq_at = at;
            found.s = s;
        }
        if ((b0 += T) >= p.num_seqs) break;
        const int b = b0 + threadIdx.x;
        // (the next chunk's sequences start where this chunk's end)
        if (threadIdx.x == T - 1) chunk_end = at + n;
        __syncthreads();
        const long long base = chunk_end;
        long long t;
        n = b < p.num_seqs ? seq_units<R, UNIT>(D, b, s) : 0;
        at = base + block_prefix<W>(n, t, sums);
    }
    __syncthreads();
    x.b = found.b;
    x.seq_at = found.seq_at;
    x.s = found.s;
    return true;
}

// A segment: units [x0, x1) of one item, the part of it that lies in the share.
struct Segment {
    long long item_at;
    int per_item, group, tile, x0, x1;
    int rows, t_first, t_last;  // packed rows of the tile and the tokens they span
    int seen_all, seen_any;     // keys that every row sees, that some row sees
    __device__ __forceinline__ bool whole() const { return x0 == 0 && x1 == per_item; }
};
// The segment that starts at unit x.u; false at the share's end.
template <int R, int UNIT>
__device__ __forceinline__ bool next_segment(const DecodeParams& D, Share& x, Segment& g) {
    if (x.u >= x.u_end) return false;
    const KParams& p = D.p;
    Shape sh = seq_shape<R, UNIT>(D, x.s);
    while (x.u >= x.seq_at + sh.units) {  // on to the sequence that holds u
        x.seq_at += sh.units;
        do
            if (++x.b >= p.num_seqs) return false;
        while (!load_lens(D, x.b, x.s) || x.s.Lq == 0);
        sh = seq_shape<R, UNIT>(D, x.s);
    }
    const int item = (int)quotient(x.u - x.seq_at, sh.per_item);
    g.item_at = x.seq_at + (long long)item * sh.per_item;
    g.per_item = sh.per_item;
    g.group = sh.tiles == 1 ? item : item / sh.tiles;
    g.tile = item - g.group * sh.tiles;
    g.x0 = (int)(x.u - g.item_at);
    g.x1 = (int)min((long long)sh.per_item, x.u_end - g.item_at);
    g.rows = min(R, (x.s.Lq << D.g_shift) - g.tile * R);
    g.t_first = token_of(D, g.tile * R);
    g.t_last = token_of(D, g.tile * R + g.rows - 1);
    g.seen_all = x.s.P + g.t_first + 1;
    g.seen_any = x.s.P + g.t_last + 1;
    return true;
}
// One thread: what the join has to do for an item that starts in this segment.
__device__ __forceinline__ void put_record(const DecodeParams& D, const Share& x, int q0, int b, const Segment& g, int c) {
    if (g.x0 != 0 || !(D.few || !g.whole())) return;
    const int parts = g.whole() ? 0 : x.of_unit(g.item_at + g.per_item - 1) - c + 1;
    const int at = 2 * (D.few ? (b * D.groups + g.group) * D.tiles_max + g.tile : c);
    D.record[at] = make_int4(parts, q0, g.group, g.tile);
    D.record[at + 1] = make_int4(g.rows, c, 0, 0);
}

__device__ __forceinline__ float lse_of(float m, float l) { return (m + log2f(l)) * 0.69314718055994531f; }
__device__ __forceinline__ float4 scaled(float4 x, float f) { return make_float4(x.x * f, x.y * f, x.z * f, x.w * f); }
__device__ __forceinline__ float4 plus(float4 a, float4 b, float f) {  // a + b f
    return make_float4(fmaf(b.x, f, a.x), fmaf(b.y, f, a.y), fmaf(b.z, f, a.z), fmaf(b.w, f, a.w));
}

// One thread of a CTA that gave up a wait: nothing is to be joined of the items that start
// in its share.  (By share: its one record was cleared at the start, and its last segment
// alone writes it.)  Their records would else be an earlier call's, with rows and shares of
// its own; the error word cannot tell the join, as it keeps the first error.
template <int R, int UNIT>
__device__ __forceinline__ void drop_records(const DecodeParams& D, const Share& found, Share x, int c) {
    if (!D.few) return;
    x.u = x.start(c);
    x.b = found.b;
    x.seq_at = found.seq_at;
    x.s = found.s;
    Segment g;
    while (next_segment<R, UNIT>(D, x, g)) {
        if (g.x0 == 0) D.record[2 * ((x.b * D.groups + g.group) * D.tiles_max + g.tile)] = make_int4(0, 0, 0, 0);
        x.u = g.item_at + g.x1;
    }
}

// Four columns of one packed row's output, o / l, rounded once.  e4m3 without scales of
// its own holds the stored values' units, as o does: the value scale, which may be 0,
// stays out.
template <bool FP8>
__device__ __forceinline__ void put_out(const DecodeParams& D, long long row, int h, int col, float4 o, float l) {
    const KParams& p = D.p;
    const long long at = (row * p.Hq + h) * p.d + col;
    const bool stored = p.out_fp8 && !p.out_scale;
    float4 x = scaled(o, (FP8 && !stored ? p.v_scale[h >> D.g_shift] : 1.f) / l);
    if (p.out_fp8) {
        const float sc = stored ? 1.f : p.out_scale[h];
        x = sc == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(x.x / sc, x.y / sc, x.z / sc, x.w / sc);
        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(D.out) + at) = pack_e4m3x4(x.x, x.y, x.z, x.w);
    } else {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(D.out) + at) =
            make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
    }
}
// Multi-token tiles of head dimension 128 (fp2_decode_tiles.cu): the shares'
// partial rows and records, as decode_kernel leaves them for 32 rows a tile.
cudaError_t launch_decode_tiles(const DecodeParams& D, cudaStream_t s);
int decode_tile_ctas(bool fp8);

}  // namespace fp2
