// fp2_pagemap.cu -- fp2_page_map: cumulative lengths, new pages, positions and
// cache slots of a serving step from the request lengths, in one launch.
//
// Mathematics: two exclusive sums over the sequences (new tokens, new pages);
// token i belongs to the sequence b with cu[b] <= i < cu[b + 1], new page j
// likewise.  Every CTA takes both sums over all sequences for itself, in shared
// memory (they are a few KB and come from L2), and then maps its share of the
// tokens and pages by binary search, so that no CTA waits for another.
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

__global__ void __launch_bounds__(kMapThreads) page_map_kernel(const __grid_constant__ MapParams p) {
    extern __shared__ int map_smem[];
    __shared__ longlong2 warp_sums[kMapThreads / 32];
    __shared__ int bad_len, bad_pages;
    const int S = p.num_seqs;
    int* cu = map_smem;          // [S + 1] exclusive sums of new tokens
    int* pc = map_smem + S + 1;  // [S + 1] exclusive sums of new pages
    if (threadIdx.x == 0) bad_len = bad_pages = 0;
    wait_previous();
    __syncthreads();
    // a thread takes `per` consecutive sequences
    const int per = (S + kMapThreads - 1) / kMapThreads;
    const int b0 = min(S, (int)threadIdx.x * per), b1 = min(S, b0 + per);
    auto pages = [&](int n) { return (n + p.page_size - 1) >> p.page_shift; };
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
    auto free_page = [&](int j) {  // page j of the step's new ones, -1 if its id is bad
        const int id = p.free_pages[head + j];
        if (id < 0 || id >= p.num_pages) {
            set_error(p.err, kErrBounds, kDetPage);
            return -1;
        }
        return id;
    };
    for (int j = first; j < fresh; j += step) {
        const int b = owner(pc, S, j);
        p.table[(size_t)b * p.max_pages + pages(p.prefix[b]) + (j - pc[b])] = free_page(j);
    }
    for (int i = first; i < p.total_q; i += step) {
        int pos = 0, slot = -1;
        if (i < live) {
            const int b = owner(cu, S, i);
            const int pre = p.prefix[b];
            pos = pre + (i - cu[b]);
            const int k = pos >> p.page_shift, old = pages(pre);
            int id;
            if (k < old) {  // the prefix's last page, not full
                id = p.table[(size_t)b * p.max_pages + k];
                if (id < 0 || id >= p.num_pages) {
                    set_error(p.err, kErrBounds, kDetPage);
                    id = -1;
                }
            } else {
                id = free_page(pc[b] + (k - old));
            }
            if (id >= 0) slot = (id << p.page_shift) + (pos & (p.page_size - 1));
        }
        p.positions[i] = pos;
        p.slots[i] = slot;
    }
}

}  // namespace

cudaError_t launch_page_map(const MapParams& p, cudaStream_t s) {
    const size_t smem = 2 * ((size_t)p.num_seqs + 1) * sizeof(int);
    if (smem > 40 * 1024) {
        static std::atomic<unsigned long long> ready{0};
        const cudaError_t e = allow_smem(page_map_kernel, 2 * (16384 + 1) * (int)sizeof(int), ready);
        if (e != cudaSuccess) return e;
    }
    const int tokens_per_cta = 4 * kMapThreads;
    int ctas = (p.total_q + tokens_per_cta - 1) / tokens_per_cta;
    if (ctas < 1) ctas = 1;
    if (ctas > 296) ctas = 296;
    return launch_early(page_map_kernel, dim3(ctas), kMapThreads, smem, s, p);
}

}  // namespace fp2
