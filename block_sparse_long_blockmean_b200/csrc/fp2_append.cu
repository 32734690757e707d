// fp2_append.cu -- fp2_append: per-head RMS norm of q and k, position rotation,
// and the write of q and of the cache rows of k and v, one pass over the
// projection's rows.
//
// A head of a token is held by D / 8 lanes with 8 values each, as two groups
// of 4 that rotate with each other: values a..a+3 and b..b+3 with b = a +
// rot/2 for the half-split pairing, so that no value crosses lanes; only the
// mean square of a norm is summed over the head's lanes.
#include <cuda_bf16.h>

#include "fp2_device.cuh"
#include "fp2_internal.h"

namespace fp2 {

namespace {

constexpr int kAppThreads = 256;

__device__ __forceinline__ void load4(const void* base, long long at, float* x) {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + at);
    x[0] = __uint_as_float(w.x << 16);
    x[1] = __uint_as_float(w.x & 0xFFFF0000u);
    x[2] = __uint_as_float(w.y << 16);
    x[3] = __uint_as_float(w.y & 0xFFFF0000u);
}

// The one rounding: to bf16, or to e4m3 of x * (1 / scale).  The product
// with the reciprocal is off by under 2^-22 relative, far below e4m3's 2^-4.
template <bool FP8>
__device__ __forceinline__ void store4(void* base, long long at, const float* x, float inv_scale) {
    if constexpr (FP8) {
        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(base) + at) =
            pack_e4m3x4(x[0] * inv_scale, x[1] * inv_scale, x[2] * inv_scale, x[3] * inv_scale);
    } else {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + at) =
            make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
    }
}

// grid (ceil(T / warps), head chunks): a warp takes one token and a chunk of
// its Hq + 2 Hkv heads, 32 / (D / 8) heads at a time.
template <int D, bool FP8>
__global__ void __launch_bounds__(kAppThreads) append_kernel(AppendParams p, int chunk) {
    constexpr int HL = D / 8, HPW = 32 / HL;
    const int lane = threadIdx.x & 31, l = lane % HL;
    const int tok = blockIdx.x * (kAppThreads / 32) + (threadIdx.x >> 5);
    if (tok >= p.total_q) return;
    const int heads = p.Hq + 2 * p.Hkv, rot = p.rot;
    const bool rotates = l < rot / 8;
    // this lane's two groups of four values
    const int ia = rotates ? 4 * l : rot + 4 * (l - rot / 8);
    const int ib = rotates ? rot / 2 + 4 * l : ia + (D - rot) / 2;
    float cs[4], sn[4];
    if (rotates) {
        const double pos = (double)p.positions[tok];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            // pair (a[e], b[e]) of the half-split form turns with frequency
            // 4l + e; the interleaved pairs sit inside the groups
            const int f = !p.interleaved ? 4 * l + e : (e < 2 ? ia / 2 + e : ib / 2 + e - 2);
            // turns = position * frequency / 2 pi in 64 bits (a float holds no
            // far position's angle), of which only the fraction matters
            const double turns = pos * (double)p.inv_freq[f] * 0.15915494309189533577;
            float s, c;
            sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
            cs[e] = c * p.rope_scale;
            sn[e] = s * p.rope_scale;
        }
    }
    int slot = p.slots[tok];
    if (slot >= p.cache_rows) {
        if (lane == 0 && blockIdx.y == 0) set_error(p.err, kErrBounds, kDetRow);
        slot = -1;
    }
    const int h_end = min(heads, (int)(blockIdx.y + 1) * chunk);
    for (int h0 = blockIdx.y * chunk; h0 < h_end; h0 += HPW) {
        const int hh = h0 + lane / HL;
        const bool on = hh < h_end;
        const int kind = hh < p.Hq ? 0 : hh < p.Hq + p.Hkv ? 1 : 2;  // q, k, v
        const int h = kind == 0 ? hh : kind == 1 ? hh - p.Hq : hh - p.Hq - p.Hkv;
        float a[4] = {0.f, 0.f, 0.f, 0.f}, b[4] = {0.f, 0.f, 0.f, 0.f};
        if (on) {
            const void* src = kind == 0 ? p.q : kind == 1 ? p.k : p.v;
            const long long row = (long long)tok * (kind == 0 ? p.q_stride : kind == 1 ? p.k_stride : p.v_stride) + h * D;
            load4(src, row + ia, a);
            load4(src, row + ib, b);
        }
        const float* w = kind == 0 ? p.q_weight : kind == 1 ? p.k_weight : nullptr;
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) ss += a[e] * a[e] + b[e] * b[e];
#pragma unroll
        for (int o = HL / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
        if (!on) continue;
        if (w) {
            const float r = rsqrtf(ss * (1.0f / D) + p.eps);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                a[e] = a[e] * r * w[ia + e];
                b[e] = b[e] * r * w[ib + e];
            }
        }
        if (kind < 2 && rotates) {
            if (!p.interleaved) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float x = a[e], y = b[e];
                    a[e] = x * cs[e] - y * sn[e];
                    b[e] = y * cs[e] + x * sn[e];
                }
            } else {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = a[2 * e], y = a[2 * e + 1];
                    a[2 * e] = x * cs[e] - y * sn[e];
                    a[2 * e + 1] = y * cs[e] + x * sn[e];
                    x = b[2 * e];
                    y = b[2 * e + 1];
                    b[2 * e] = x * cs[2 + e] - y * sn[2 + e];
                    b[2 * e + 1] = y * cs[2 + e] + x * sn[2 + e];
                }
            }
        }
        if (kind != 0 && slot < 0) continue;
        void* dst = kind == 0 ? p.q_out : kind == 1 ? p.k_cache : p.v_cache;
        const long long at = kind == 0 ? ((long long)tok * p.Hq + h) * D : ((long long)slot * p.Hkv + h) * D;
        const float inv = FP8 ? 1.0f / (kind == 0 ? p.q_scale : kind == 1 ? p.k_scale : p.v_scale)[h] : 1.0f;
        store4<FP8>(dst, at + ia, a, inv);
        store4<FP8>(dst, at + ib, b, inv);
    }
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, cudaStream_t s) {
    const int heads = p.Hq + 2 * p.Hkv, hpw = 32 / (p.d / 8);
    const int warps = kAppThreads / 32;
    const dim3 grid((p.total_q + warps - 1) / warps, 1);
    const int chunk = (heads + hpw - 1) / hpw * hpw;
    if (p.d == 128) {
        if (p.fp8) append_kernel<128, true><<<grid, kAppThreads, 0, s>>>(p, chunk);
        else append_kernel<128, false><<<grid, kAppThreads, 0, s>>>(p, chunk);
    } else {
        if (p.fp8) append_kernel<64, true><<<grid, kAppThreads, 0, s>>>(p, chunk);
        else append_kernel<64, false><<<grid, kAppThreads, 0, s>>>(p, chunk);
    }
    return cudaGetLastError();
}

}  // namespace fp2
