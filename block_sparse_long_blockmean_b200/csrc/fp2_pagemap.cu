// fp2_pagemap.cu -- fp2_page_map: cumulative lengths, new pages, positions and
// cache slots of a serving step from the request lengths, in one launch.
//
// Mathematics: two exclusive sums over the sequences (new tokens, new pages);
// token i belongs to the sequence b with cu[b] <= i < cu[b + 1], new page j
// likewise.  Every CTA takes both sums over all sequences for itself, in shared
// memory (they are a few KB and come from L2), and then maps its share of the
// tokens and pages by binary search, so that no CTA waits for another.
//
// Bound by its launch and three loads that wait for one another: 64 sequences of one
// token 2.9 us, 1000 of up to 511 tokens 5.2, 8 of 32768 3.8 (2.1 MB: 0.3 us of bytes).
#include "fp2_device.cuh"
#include "fp2_launch.cuh"

namespace fp2 {

constexpr int kMapThreads = 512;

namespace {

// Exclusive sums of (a, b) over the CTA's threads; totals in ta, tb.
__device__ __forceinline__ void block_scan2(long long& a, long long& b, long long& ta, long long& tb,
                                            longlong2* warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int W = kMapThreads / 32;
    long long x = a, y = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(~0u, x, o), v = __shfl_up_sync(~0u, y, o);
        if (lane >= o) {
            x += u;
            y += v;
        }
    }
    if (lane == 31) warp_sums[warp] = make_longlong2(x, y);
    __syncthreads();
    long long px = 0, py = 0;
    ta = tb = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        const longlong2 s = warp_sums[w];
        if (w < warp) {
            px += s.x;
            py += s.y;
        }
        ta += s.x;
        tb += s.y;
    }
    a = px + x - a;
    b = py + y - b;
}

// The b in [0, n) with v[b] <= i < v[b + 1] (v ascending, v[0] <= i < v[n]).
__device__ __forceinline__ int owner(const int* v, int n, int i) {
    int lo = 0, hi = n;  // v[lo] <= i < v[hi]
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (v[m] <= i) lo = m;
        else hi = m;
    }
    return lo;
}

// TOKENS consecutive tokens a thread.
template <int TOKENS>
__global__ void __launch_bounds__(kMapThreads) page_map_kernel(const __grid_constant__ MapParams p) {
    extern __shared__ int map_smem[];
    __shared__ longlong2 warp_sums[kMapThreads / 32];
    __shared__ int bad_len, bad_pages;
    const int S = p.num_seqs;
    int* cu = map_smem;          // [S + 1] exclusive sums of new tokens
    int* pc = cu + S + 1;        // [S + 1] exclusive sums of new pages
    int* had = pc + S + 1;       // [S] tokens that were there
    if (threadIdx.x == 0) bad_len = bad_pages = 0;
    wait_previous();
    __syncthreads();
    // a thread takes `per` consecutive sequences
    const int per = (S + kMapThreads - 1) / kMapThreads;
    const int b0 = min(S, (int)threadIdx.x * per), b1 = min(S, b0 + per);
    auto pages = [&](int n) { return (n >> p.page_shift) + ((n & (p.page_size - 1)) != 0); };
    auto read = [&](int b, int& pre, int& n) {
        pre = p.prefix[b];
        n = p.fresh[b];
        if (n < 0 || n > p.max_seqlen_q || pre < 0 || pre > p.max_seqlen_k - n) {
            bad_len = 1;
            pre = n = 0;
        } else if (((long long)pre + n + p.page_size - 1) >> p.page_shift > p.max_pages) {
            bad_pages = 1;
            pre = n = 0;
        }
    };
    long long nt = 0, np = 0, all_t, all_p;
    for (int b = b0; b < b1; ++b) {
        int pre, n;
        read(b, pre, n);
        nt += n;
        np += pages(pre + n) - pages(pre);
    }
    block_scan2(nt, np, all_t, all_p, warp_sums);
    const int head = *p.free_head;
    // the barrier inside the scan has ordered the flags
    const bool lens_ok = !bad_len && all_t <= p.total_q;
    const bool table_ok = !bad_pages;
    const bool free_ok = head >= 0 && (long long)head + all_p <= p.num_free;
    const bool ok = lens_ok && table_ok && free_ok;
    if (ok) {
        for (int b = b0; b < b1; ++b) {
            int pre, n;
            read(b, pre, n);
            cu[b] = (int)nt;
            pc[b] = (int)np;
            had[b] = pre;
            nt += n;
            np += pages(pre + n) - pages(pre);
        }
        if (threadIdx.x == 0) {
            cu[S] = (int)all_t;
            pc[S] = (int)all_p;
        }
    }
    __syncthreads();
    if (blockIdx.x == 0) {
        for (int b = threadIdx.x; b <= S; b += kMapThreads) {
            p.cu[b] = ok ? cu[b] : 0;
            if (b < S) p.seqlens_k[b] = p.prefix[b] + (ok ? p.fresh[b] : 0);
        }
        if (threadIdx.x == 0) {
            *p.free_head_out = ok ? head + (int)all_p : head;
            if (!lens_ok) set_error(p.err, kErrInvalid, kDetSeqLen);
            else if (!table_ok) set_error(p.err, kErrBounds, kDetSeqLen);
            else if (!free_ok) set_error(p.err, kErrBounds, kDetFree);
        }
    }
    const int live = ok ? (int)all_t : 0, fresh = ok ? (int)all_p : 0;
    const int first = blockIdx.x * kMapThreads + threadIdx.x, step = gridDim.x * kMapThreads;
    auto checked = [&](int id) {  // a page id, -1 if it is bad
        if (id < 0 || id >= p.num_pages) {
            set_error(p.err, kErrBounds, kDetPage);
            return -1;
        }
        return id;
    };
    // tokens, TOKENS consecutive ones a thread: one search, then a walk
    const bool wide = ((reinterpret_cast<uintptr_t>(p.positions) | reinterpret_cast<uintptr_t>(p.slots)) & 15) == 0;
    for (long long i0 = (long long)first * TOKENS; i0 < p.total_q; i0 += (long long)step * TOKENS) {
        int pos[TOKENS], slot[TOKENS], id[TOKENS];
        int b = i0 < live ? owner(cu, S, (int)i0) : S - 1;
#pragma unroll
        for (int e = 0; e < TOKENS; ++e) {
            pos[e] = 0;
            id[e] = -1;
            if (i0 + e < live) {
                const int i = (int)i0 + e;
                while (i >= cu[b + 1]) ++b;
                pos[e] = had[b] + (i - cu[b]);
                const int k = pos[e] >> p.page_shift, old = pages(had[b]);
                // the prefix's last page, not full, or one of the step's new ones
                id[e] = k < old ? p.table[(size_t)b * p.max_pages + k] : p.free_pages[head + pc[b] + (k - old)];
            }
        }
#pragma unroll
        for (int e = 0; e < TOKENS; ++e) {
            slot[e] = -1;
            if (i0 + e < live && checked(id[e]) >= 0) slot[e] = (id[e] << p.page_shift) + (pos[e] & (p.page_size - 1));
        }
        if (TOKENS == 4 && wide && i0 + 4 <= p.total_q) {
            *reinterpret_cast<int4*>(p.positions + i0) = make_int4(pos[0], pos[1 % TOKENS], pos[2 % TOKENS], pos[3 % TOKENS]);
            *reinterpret_cast<int4*>(p.slots + i0) = make_int4(slot[0], slot[1 % TOKENS], slot[2 % TOKENS], slot[3 % TOKENS]);
        } else {
#pragma unroll
            for (int e = 0; e < TOKENS; ++e)
                if (i0 + e < p.total_q) {
                    p.positions[i0 + e] = pos[e];
                    p.slots[i0 + e] = slot[e];
                }
        }
    }
    for (int j = first; j < fresh; j += step) {
        const int b = owner(pc, S, j);
        p.table[(size_t)b * p.max_pages + pages(had[b]) + (j - pc[b])] = checked(p.free_pages[head + j]);
    }
}

}  // namespace

template <int TOKENS>
static cudaError_t launch(const MapParams& p, cudaStream_t s) {
    const size_t smem = (3 * (size_t)p.num_seqs + 2) * sizeof(int);
    if (smem > 40 * 1024) {
        static std::atomic<unsigned long long> ready{0};
        const cudaError_t e = allow_smem(page_map_kernel<TOKENS>, (3 * 16384 + 2) * (int)sizeof(int), ready);
        if (e != cudaSuccess) return e;
    }
    const int per_cta = TOKENS * kMapThreads;
    int ctas = (int)(((long long)p.total_q + per_cta - 1) / per_cta);
    ctas = ctas < 1 ? 1 : ctas > 296 ? 296 : ctas;
    return launch_early(page_map_kernel<TOKENS>, dim3(ctas), kMapThreads, smem, s, p);
}

cudaError_t launch_page_map(const MapParams& p, cudaStream_t s) {
    // a token a thread while that takes at most one CTA on each of 148 SMs
    // (64 single tokens: 2.8 us, with four a thread 3.7); more tokens share their
    // CTA's sums and searches (254K tokens of 1000 sequences: 7.3 and 5.3 us)
    return p.total_q <= 148 * kMapThreads ? launch<1>(p, s) : launch<4>(p, s);
}

}  // namespace fp2
