// fp2_append.cu -- fp2_append: per-head RMS norm of q and k, position rotation,
// and the write of q and of the cache rows of k and v, one pass over the
// projection's rows.
//
// Mathematics: with r = 1 / sqrt(mean(x^2) + eps) and the norm's weight w, every
// stored value is r (x_i C_i + x_j S_i), j its partner in the rotated pair:
// C = w cos, S = -+ w_j sin.  C and S are the same for all heads of a token, so a
// warp takes them once and then streams heads: two packed products a pair, the
// square sum over the head's lanes, one rounding.
//
// A head of a token is held by D / 8 lanes with 8 values each, as two groups
// of 4, values a..a+3 and b..b+3 with b = a + rot/2, so that a half-split pair
// (i, i + rot/2) and an adjacent pair (2i, 2i + 1) both stay inside a lane.
//
// Bound by the rows' bytes.  A lane copies its own 8-byte groups a step ahead into
// shared memory: no lane waits for another's, 8-byte rows of any stride will do, and
// no register holds a row on its way.  32768 tokens of 64 + 2 x 8 heads of 128, bf16 to
// e4m3 (1007 MB): 156 us, 6.43 TB/s (in a run of seconds at the power limit 180); the rows
// in registers, loaded as they were needed: 178 us; a step ahead in registers: 242 us.
// Steps of 4 groups, two of them in shared memory, 6 CTAs on an SM: 155 us when these were
// compared; 3 steps of 4: 159; 4 of 4: 196 (the rest of the L1 cache is too small); 4 of 2:
// 164; 2 of 3: 164; 2 of 6: 165.
// Small calls are bound by their launch (64 tokens: 2.4 us).
#include <cuda_bf16.h>

#include <type_traits>

#include "fp2_device.cuh"
#include "fp2_launch.cuh"

namespace fp2 {

namespace {

constexpr int kAppThreads = 128, kAppWarps = kAppThreads / 32;
constexpr int kAppDepth = 4;   // groups of heads of a step
constexpr int kAppStages = 2;  // steps in shared memory or on their way there

struct Quad {
    float2 x, y;
};
__device__ __forceinline__ Quad unpack(uint2 w) {
    return {make_float2(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u)),
            make_float2(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u))};
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 swapped(float2 a) { return make_float2(a.y, a.x); }

// 8 bytes to shared memory, for this thread alone to read after wait_copies().
__device__ __forceinline__ void copy8(uint32_t to, const void* from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void end_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>  // all but the N latest groups of copies
__device__ __forceinline__ void wait_copies() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// The one rounding: to bf16, or to e4m3 (the caller has divided by the scale).
template <bool FP8>
__device__ __forceinline__ void store4(uint8_t* to, Quad v) {
    if constexpr (FP8) {
        *reinterpret_cast<uint32_t*>(to) = pack_e4m3x4(v.x.x, v.x.y, v.y.x, v.y.y);
    } else {
        *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(v.x.x, v.x.y), pack_bf16x2(v.y.x, v.y.y));
    }
}

// grid (ceil(T / warps), chunks): a warp takes one token and a chunk of its
// groups of 32 / (D / 8) heads (q's, then k's, then v's).
template <int D, bool FP8, bool ADJACENT>
__global__ void __launch_bounds__(kAppThreads, 6) append_kernel(const __grid_constant__ AppendParams p) {
    constexpr int HL = D / 8, HPW = 32 / HL;
    const int lane = threadIdx.x & 31, l = lane % HL;
    const int tok = blockIdx.x * kAppWarps + (threadIdx.x >> 5);
    wait_previous();
    if (tok >= p.total_q) return;
    const int rot = p.rot;
    const bool rotates = l < rot / 8;
    int slot = p.slots[tok];
    const double pos = rotates ? (double)p.positions[tok] : 0.;
    // this lane's two groups of four values
    const int ia = rotates ? 4 * l : rot + 4 * (l - rot / 8);
    const int ib = rotates ? rot / 2 + 4 * l : ia + (D - rot) / 2;
    // steps of kAppDepth groups: q's, then k's, then v's
    const int nq = (p.Hq + HPW - 1) / HPW, nk = (p.Hkv + HPW - 1) / HPW;
    const int g0 = blockIdx.y * p.chunk, g1 = min(g0 + p.chunk, nq + 2 * nk);
    const int k_from = max(g0, nq) - nq, v_from = max(g0, nq + nk) - nq - nk;
    const int q_to = min(g1, nq), k_to = min(g1, nq + nk) - nq, v_to = g1 - nq - nk;
    auto steps_of = [](int from, int to) { return to > from ? (to - from + kAppDepth - 1) / kAppDepth : 0; };
    const int q_steps = steps_of(g0, q_to), qk_steps = q_steps + steps_of(k_from, k_to), steps = qk_steps + steps_of(v_from, v_to);
    // a lane's own 16 bytes of each group, so that no lane waits for another's
    __shared__ __align__(16) uint4 rows[kAppStages][kAppDepth][kAppThreads];
    auto fetch = [&](int n) {
        if (n < steps) {
            const bool is_q = n < q_steps, is_k = !is_q && n < qk_steps;
            const int g = is_q ? g0 + n * kAppDepth : is_k ? k_from + (n - q_steps) * kAppDepth : v_from + (n - qk_steps) * kAppDepth;
            const int to = is_q ? q_to : is_k ? k_to : v_to, heads = is_q ? p.Hq : p.Hkv;
            const uint16_t* src = static_cast<const uint16_t*>(is_q ? p.q : is_k ? p.k : p.v) +
                                  (long long)tok * (is_q ? p.q_stride : is_k ? p.k_stride : p.v_stride) + (g * HPW + lane / HL) * D;
            const uint32_t dst = smem_u32(&rows[n % kAppStages][0][threadIdx.x]);
#pragma unroll
            for (int i = 0; i < kAppDepth; ++i)
                if (g + i < to && (g + i) * HPW + lane / HL < heads) {
                    copy8(dst + i * (kAppThreads * 16), src + i * HPW * D + ia);
                    copy8(dst + i * (kAppThreads * 16) + 8, src + i * HPW * D + ib);
                }
        }
        end_copies();
    };
#pragma unroll
    for (int n = 0; n < kAppStages - 1; ++n) fetch(n);
    int now = 0;
    Quad ca = {{1.f, 1.f}, {1.f, 1.f}}, cb = ca, sa = {{0.f, 0.f}, {0.f, 0.f}}, sb = sa;  // cos, -+ sin
    if (rotates) {
        float c[4], s[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            // pair (a[e], b[e]) turns with frequency 4 l + e; adjacent pairs sit
            // inside the groups
            const int f = !ADJACENT ? 4 * l + e : (e < 2 ? ia / 2 + e : ib / 2 + e - 2);
            // turns = position * frequency / 2 pi in 64 bits (a float holds no
            // far position's angle), of which only the fraction matters
            const double turns = pos * (double)p.inv_freq[f] * 0.15915494309189533577;
            sincospif(2.0f * (float)(turns - rint(turns)), &s[e], &c[e]);
            c[e] *= p.rope_scale;
            s[e] *= p.rope_scale;
        }
        if constexpr (!ADJACENT) {
            ca = cb = {{c[0], c[1]}, {c[2], c[3]}};
            sb = {{s[0], s[1]}, {s[2], s[3]}};
            sa = {{-s[0], -s[1]}, {-s[2], -s[3]}};
        } else {
            ca = {{c[0], c[0]}, {c[1], c[1]}};
            cb = {{c[2], c[2]}, {c[3], c[3]}};
            sa = {{-s[0], s[0]}, {-s[1], s[1]}};
            sb = {{-s[2], s[2]}, {-s[3], s[3]}};
        }
    }
    if (slot >= p.cache_rows) {
        if (lane == 0 && blockIdx.y == 0) set_error(p.err, kErrBounds, kDetRow);
        slot = -1;
    }

    // groups [from, to) of one kind; TURN: norm and rotation, else as they are
    auto stream = [&](auto turn, int from, int to, void* dst, long long row, int heads,
                      const float* weight, const float* scale) {
        constexpr bool TURN = decltype(turn)::value;
        if (from >= to) return;
        const long long out = row * heads * D;
        Quad wca = ca, wcb = cb, wsa = sa, wsb = sb;
        if (TURN && weight) {
            const float4 x = *reinterpret_cast<const float4*>(weight + ia), y = *reinterpret_cast<const float4*>(weight + ib);
            const Quad wa = {{x.x, x.y}, {x.z, x.w}}, wb = {{y.x, y.y}, {y.z, y.w}};
            wca = {mul2(ca.x, wa.x), mul2(ca.y, wa.y)};
            wcb = {mul2(cb.x, wb.x), mul2(cb.y, wb.y)};
            if constexpr (!ADJACENT) {
                wsa = {mul2(sa.x, wb.x), mul2(sa.y, wb.y)};
                wsb = {mul2(sb.x, wa.x), mul2(sb.y, wa.y)};
            } else {
                wsa = {mul2(sa.x, swapped(wa.x)), mul2(sa.y, swapped(wa.y))};
                wsb = {mul2(sb.x, swapped(wb.x)), mul2(sb.y, swapped(wb.y))};
            }
        }
        const bool norm = TURN && weight;
        // where this lane's values of the present step go; a group is GS values on
        constexpr int GS = HPW * D, ES = FP8 ? 1 : 2;
        uint8_t* wa = static_cast<uint8_t*>(dst) + (out + (from * HPW + lane / HL) * D + ia) * ES;
        uint8_t* wb = wa + (ib - ia) * ES;
        [[maybe_unused]] const float* sp = FP8 ? scale + from * HPW + lane / HL : nullptr;
        auto step = [&](auto full, int g) {
            constexpr bool FULL = decltype(full)::value;  // kAppDepth whole groups
            float inv[kAppDepth];
            fetch(now + kAppStages - 1);
            auto on = [&](int i) { return FULL || (g + i < to && (g + i) * HPW + lane / HL < heads); };
#pragma unroll
            for (int i = 0; i < kAppDepth; ++i) {
                inv[i] = 1.f;
                if (FP8 && on(i)) inv[i] = sp[i * HPW];
            }
            wait_copies<kAppStages - 1>();
            const uint4* mine = &rows[now % kAppStages][0][threadIdx.x];
#pragma unroll
            for (int i = 0; i < kAppDepth; ++i) {
                if (!FULL && g + i >= to) break;
                uint4 raw = make_uint4(0u, 0u, 0u, 0u);
                if (on(i)) raw = mine[i * kAppThreads];
                Quad a = unpack(make_uint2(raw.x, raw.y)), b = unpack(make_uint2(raw.z, raw.w));
                // (the reciprocal is off by 2^-23 of its value, far below e4m3's 2^-4)
                // a scale of 0 stands for a head of zeros, here as in fp2_decode
                float r = !FP8 ? 1.f : inv[i] == 0.f ? 0.f : __fdividef(1.f, inv[i]);
                if constexpr (TURN) {
                    if (norm) {
                        float2 q = ffma2(a.y, a.y, mul2(a.x, a.x));
                        q = ffma2(b.y, b.y, ffma2(b.x, b.x, q));
                        float ss = q.x + q.y;
#pragma unroll
                        for (int o = HL / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
                        r *= rsqrtf(ss * (1.0f / D) + p.eps);
                    }
                    Quad x = {mul2(a.x, wca.x), mul2(a.y, wca.y)}, y = {mul2(b.x, wcb.x), mul2(b.y, wcb.y)};
                    if (rotates) {
                        if constexpr (!ADJACENT) {
                            x = {ffma2(b.x, wsa.x, x.x), ffma2(b.y, wsa.y, x.y)};
                            y = {ffma2(a.x, wsb.x, y.x), ffma2(a.y, wsb.y, y.y)};
                        } else {
                            x = {ffma2(swapped(a.x), wsa.x, x.x), ffma2(swapped(a.y), wsa.y, x.y)};
                            y = {ffma2(swapped(b.x), wsb.x, y.x), ffma2(swapped(b.y), wsb.y, y.y)};
                        }
                    }
                    a = x;
                    b = y;
                }
                if (TURN || FP8) {
                    const float2 rr = make_float2(r, r);
                    a = {mul2(a.x, rr), mul2(a.y, rr)};
                    b = {mul2(b.x, rr), mul2(b.y, rr)};
                }
                if (on(i) && row >= 0) {
                    store4<FP8>(wa + i * GS * ES, a);
                    store4<FP8>(wb + i * GS * ES, b);
                }
            }
            ++now;
            wa += kAppDepth * GS * ES;
            wb += kAppDepth * GS * ES;
            if constexpr (FP8) sp += kAppDepth * HPW;
        };
        int g = from;
        if (heads % HPW == 0)
            for (; g + kAppDepth <= to; g += kAppDepth) step(std::true_type{}, g);
        for (; g < to; g += kAppDepth) step(std::false_type{}, g);
    };
    stream(std::true_type{}, g0, q_to, p.q_out, tok, p.Hq, p.q_weight, p.q_scale);
    stream(std::true_type{}, k_from, k_to, p.k_cache, slot, p.Hkv, p.k_weight, p.k_scale);
    stream(std::false_type{}, v_from, v_to, p.v_cache, slot, p.Hkv, nullptr, p.v_scale);
}

template <int D, bool FP8>
cudaError_t launch(AppendParams p, cudaStream_t s) {
    constexpr int HPW = 32 / (D / 8);
    const int groups = (p.Hq + HPW - 1) / HPW + 2 * ((p.Hkv + HPW - 1) / HPW);
    // all heads of a token in one warp once the tokens alone fill the machine
    // (16 warps on each of 148 SMs), fewer and fewer below that
    long long chunk = ((long long)p.total_q * groups + 148 * 16 - 1) / (148 * 16);
    p.chunk = (int)(chunk < groups ? chunk : groups);
    const dim3 grid((p.total_q + kAppWarps - 1) / kAppWarps, (groups + p.chunk - 1) / p.chunk);
    return p.interleaved ? launch_early(append_kernel<D, FP8, true>, grid, kAppThreads, 0, s, p)
                         : launch_early(append_kernel<D, FP8, false>, grid, kAppThreads, 0, s, p);
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, cudaStream_t s) {
    if (p.d == 128) return p.fp8 ? launch<128, true>(p, s) : launch<128, false>(p, s);
    return launch<64, false>(p, s);  // (e4m3 is head dimension 128 only)
}

}  // namespace fp2
