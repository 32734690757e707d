// fp2_serve.cu -- host side of the serving-step calls of include/fp2.h
// (fp2_page_map, fp2_append, fp2_decode): argument checks, workspace layout
// and launches, in the manner of fp2_api.cu.
#include <cmath>
#include <cstring>

#include "fp2.h"
#include "fp2_launch.cuh"

namespace {

bool is_pow2(int x) { return x > 0 && (x & (x - 1)) == 0; }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
fp2_status cuda_status(cudaError_t e) { return e == cudaSuccess ? FP2_OK : FP2_ERR_CUDA; }
cudaStream_t stream_of(const fp2_params* P) { return static_cast<cudaStream_t>(P->stream); }

fp2_status check_workspace(const fp2_params* P, size_t need) {
    if (!P->workspace || !aligned(P->workspace, 256) || P->workspace_bytes < need)
        return FP2_ERR_WORKSPACE;
    return FP2_OK;
}

fp2_status check_pages(const fp2_params* P) {
    if (!is_pow2(P->page_size) || P->page_size < 16 || P->page_size > 256)
        return FP2_ERR_UNSUPPORTED;
    if (P->num_pages < 1) return FP2_ERR_INVALID_ARG;
    if ((long long)P->num_pages * P->page_size > INT32_MAX) return FP2_ERR_UNSUPPORTED;
    return FP2_OK;
}

fp2_status check_heads(const fp2_params* P) {
    if (P->num_q_heads < 1 || P->num_kv_heads < 1 || P->total_q < 0) return FP2_ERR_INVALID_ARG;
    if (P->num_q_heads % P->num_kv_heads != 0) return FP2_ERR_INVALID_ARG;
    const int G = P->num_q_heads / P->num_kv_heads;
    if (G != 1 && G != 2 && G != 4 && G != 8) return FP2_ERR_UNSUPPORTED;
    if (P->head_dim != 64 && P->head_dim != 128) return FP2_ERR_UNSUPPORTED;
    return FP2_OK;
}

// Bytes [a, a + n) and [b, b + m) share a byte.
bool overlap(const void* a, size_t n, const void* b, size_t m) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + m && y < x + n;
}

fp2_status check_decode(const fp2_params* P) {
    if (!P) return FP2_ERR_INVALID_ARG;
    if (P->num_seqs < 1 || P->max_seqlen_q < 0 || P->max_seqlen_k < P->max_seqlen_q ||
        P->max_seqlen_k < 1 || P->debug_withhold_k_item < 0)
        return FP2_ERR_INVALID_ARG;
    fp2_status st = check_heads(P);
    if (st != FP2_OK) return st;
    return P->max_seqlen_q > FP2_DECODE_MAX_Q ? FP2_ERR_UNSUPPORTED : FP2_OK;
}

struct DecodeLayout {
    size_t part, part_ml, record, total;
};
DecodeLayout decode_layout(const fp2_params* P) {
    DecodeLayout L;
    // (the same for any number of new tokens: a server alternates between them)
    const size_t slots = 2 * (size_t)fp2::kDecCtas * fp2::kDecHeads * fp2::kDecRows;
    L.part = 256;  // after the error word
    L.part_ml = L.part + slots * P->head_dim * sizeof(float);
    L.record = L.part_ml + slots * 2 * sizeof(float);
    L.total = L.record + (size_t)fp2::kDecCtas * 2 * sizeof(int4);
    return L;
}

}  // namespace

namespace fp2 {

bool make_row_maps(const KParams& p, const void* k, const void* v, int rows, bool wide, CUtensorMap* mk, CUtensorMap* mv) {
    using Encode = decltype(&cuTensorMapEncodeTiled);
    static const Encode encode = [] {
        void* at = nullptr;
        cudaDriverEntryPointQueryResult found;
        const bool ok = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &at, cudaEnableDefault, &found) == cudaSuccess &&
                        found == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<Encode>(at) : nullptr;
    }();
    if (!encode) return false;
    const cuuint64_t row = (cuuint64_t)p.d * (p.fp8 ? 1 : 2);
    const cuuint64_t dims[3] = {(cuuint64_t)p.d, (cuuint64_t)p.Hkv,
                                p.paged ? (cuuint64_t)p.num_pages * p.page_size : (cuuint64_t)p.total_k};
    const cuuint64_t strides[2] = {row, p.Hkv * row};
    const cuuint32_t box[3] = {p.fp8 ? 128u : 64u, 1, (cuuint32_t)rows}, steps[3] = {1, 1, 1};
    auto map = [&](CUtensorMap* m, const void* base) {
        return encode(m, p.fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims,
                      strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                      wide ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    return map(mk, k) && map(mv, v);
}

}  // namespace fp2

extern "C" {

fp2_status fp2_page_map(const int32_t* prefix_lens, const int32_t* new_lens,
                        const int32_t* free_pages, int num_free, const int32_t* free_head,
                        int32_t* page_table, int32_t* cu_seqlens, int32_t* seqlens_k,
                        int32_t* positions, int32_t* slot_map, int32_t* free_head_out,
                        const fp2_params* params) {
    if (!params) return FP2_ERR_INVALID_ARG;
    const fp2_params* P = params;
    if (P->num_seqs < 1 || P->total_q < 0 || num_free < 0 || P->max_pages_per_seq < 1 ||
        P->max_seqlen_q < 0 || P->max_seqlen_k < P->max_seqlen_q || P->max_seqlen_k < 1)
        return FP2_ERR_INVALID_ARG;
    if (P->num_seqs > 16384) return FP2_ERR_UNSUPPORTED;
    fp2_status st = check_pages(P);
    if (st != FP2_OK) return st;
    if ((st = check_workspace(P, 256)) != FP2_OK) return st;
    if (!prefix_lens || !new_lens || !free_head || !page_table || !cu_seqlens || !seqlens_k ||
        !free_head_out || (num_free > 0 && !free_pages) ||
        (P->total_q > 0 && (!positions || !slot_map)))
        return FP2_ERR_INVALID_ARG;
    const size_t S = (size_t)P->num_seqs, T = (size_t)P->total_q;
    const struct { const void* p; size_t n; } in[] = {{prefix_lens, 4 * S}, {new_lens, 4 * S},
                                                      {free_pages, 4 * (size_t)num_free},
                                                      {free_head, 4}},
        out[] = {{page_table, 4 * S * P->max_pages_per_seq}, {cu_seqlens, 4 * (S + 1)},
                 {seqlens_k, 4 * S}, {positions, 4 * T}, {slot_map, 4 * T}, {free_head_out, 4}};
    for (const auto& o : out) {
        if (!aligned(o.p, 4)) return FP2_ERR_INVALID_ARG;
        for (const auto& i : in)
            if (!aligned(i.p, 4) || overlap(o.p, o.n, i.p, i.n)) return FP2_ERR_INVALID_ARG;
        for (const auto& x : out)
            if (&x != &o && overlap(o.p, o.n, x.p, x.n)) return FP2_ERR_INVALID_ARG;
    }
    fp2::MapParams m;
    m.num_seqs = P->num_seqs;
    m.total_q = P->total_q;
    m.page_size = P->page_size;
    m.page_shift = __builtin_ctz((unsigned)P->page_size);
    m.max_pages = P->max_pages_per_seq;
    m.num_pages = P->num_pages;
    m.max_seqlen_q = P->max_seqlen_q;
    m.max_seqlen_k = P->max_seqlen_k;
    m.num_free = num_free;
    m.prefix = prefix_lens;
    m.fresh = new_lens;
    m.free_pages = free_pages;
    m.free_head = free_head;
    m.table = page_table;
    m.cu = cu_seqlens;
    m.seqlens_k = seqlens_k;
    m.positions = positions;
    m.slots = slot_map;
    m.free_head_out = free_head_out;
    m.err = static_cast<uint32_t*>(P->workspace);
    return cuda_status(fp2::launch_page_map(m, stream_of(P)));
}

fp2_status fp2_append(const fp2_append_io* io, fp2_dtype dtype, const fp2_params* params) {
    if (!io || !params) return FP2_ERR_INVALID_ARG;
    const fp2_params* P = params;
    fp2_status st = check_heads(P);
    if (st != FP2_OK) return st;
    if (dtype != FP2_BF16 && dtype != FP2_FP8_E4M3) return FP2_ERR_INVALID_ARG;
    const bool fp8 = dtype == FP2_FP8_E4M3;
    if (P->k_block_factor || P->v_block_factor) return FP2_ERR_UNSUPPORTED;
    if (fp8 && P->head_dim != 128) return FP2_ERR_UNSUPPORTED;
    if (fp8 && (!P->q_scale || !P->k_scale || !P->v_scale)) return FP2_ERR_INVALID_ARG;
    if (P->page_size != 0) {
        if ((st = check_pages(P)) != FP2_OK) return st;
    } else if (P->total_k < 0) {
        return FP2_ERR_INVALID_ARG;
    }
    if ((st = check_workspace(P, 256)) != FP2_OK) return st;
    const int d = P->head_dim;
    if (io->rotary_dim < 0 || io->rotary_dim > d || !(io->eps >= 0.f) || std::isinf(io->eps) ||
        !std::isfinite(io->rope_scale) || (io->interleaved != 0 && io->interleaved != 1))
        return FP2_ERR_INVALID_ARG;
    if (io->rotary_dim % 8 != 0) return FP2_ERR_UNSUPPORTED;
    if (io->rotary_dim > 0 && !io->inv_freq) return FP2_ERR_INVALID_ARG;
    if (P->total_q == 0) return FP2_OK;
    if (!io->q || !io->k || !io->v || !io->q_out || !io->k_cache || !io->v_cache || !io->slot_map ||
        (io->rotary_dim > 0 && !io->positions))
        return FP2_ERR_INVALID_ARG;
    const long long wq = (long long)P->num_q_heads * d, wk = (long long)P->num_kv_heads * d;
    if (io->q_stride < wq || io->k_stride < wk || io->v_stride < wk || io->q_stride % 4 ||
        io->k_stride % 4 || io->v_stride % 4)
        return FP2_ERR_INVALID_ARG;
    if (!aligned(io->q, 8) || !aligned(io->k, 8) || !aligned(io->v, 8) || !aligned(io->q_out, 16) ||
        !aligned(io->k_cache, 16) || !aligned(io->v_cache, 16) || !aligned(io->q_weight, 16) ||
        !aligned(io->k_weight, 16) || !aligned(io->inv_freq, 4) || !aligned(io->positions, 4) ||
        !aligned(io->slot_map, 4))
        return FP2_ERR_INVALID_ARG;
    // extents, for the overlap checks: the strided rows' hull and the outputs
    const size_t T = (size_t)P->total_q, elt = fp8 ? 1 : 2;
    const size_t rows = P->page_size ? (size_t)P->num_pages * P->page_size : (size_t)P->total_k;
    const size_t nq = 2 * ((T - 1) * io->q_stride + wq), nk = 2 * ((T - 1) * io->k_stride + wk),
                 nv = 2 * ((T - 1) * io->v_stride + wk), no = T * wq * elt, nc = rows * wk * elt;
    const bool in_place = io->q_out == io->q && !fp8 && io->q_stride == wq;
    if ((!in_place && overlap(io->q_out, no, io->q, nq)) || overlap(io->q_out, no, io->k, nk) ||
        overlap(io->q_out, no, io->v, nv) || overlap(io->q_out, no, io->k_cache, nc) ||
        overlap(io->q_out, no, io->v_cache, nc) || overlap(io->k_cache, nc, io->v_cache, nc))
        return FP2_ERR_INVALID_ARG;
    for (const void* c : {(const void*)io->k_cache, (const void*)io->v_cache})
        if (overlap(c, nc, io->q, nq) || overlap(c, nc, io->k, nk) || overlap(c, nc, io->v, nv))
            return FP2_ERR_INVALID_ARG;
    fp2::AppendParams a = {};
    a.q = io->q;
    a.k = io->k;
    a.v = io->v;
    a.q_stride = io->q_stride;
    a.k_stride = io->k_stride;
    a.v_stride = io->v_stride;
    a.q_weight = io->q_weight;
    a.k_weight = io->k_weight;
    a.inv_freq = io->inv_freq;
    a.positions = io->positions;
    a.slots = io->slot_map;
    a.q_out = io->q_out;
    a.k_cache = io->k_cache;
    a.v_cache = io->v_cache;
    a.q_scale = P->q_scale;
    a.k_scale = P->k_scale;
    a.v_scale = P->v_scale;
    a.eps = io->eps;
    a.rope_scale = io->rope_scale;
    a.total_q = P->total_q;
    a.Hq = P->num_q_heads;
    a.Hkv = P->num_kv_heads;
    a.d = d;
    a.rot = io->rotary_dim;
    a.interleaved = io->interleaved;
    a.cache_rows = (int)rows;
    a.fp8 = fp8;
    a.err = static_cast<uint32_t*>(P->workspace);
    return cuda_status(fp2::launch_append(a, stream_of(P)));
}

size_t fp2_decode_workspace_size(const fp2_params* params) {
    return check_decode(params) == FP2_OK ? decode_layout(params).total : 0;
}

fp2_status fp2_decode(const void* q, const void* k_cache, const void* v_cache,
                      const int32_t* page_table, const int32_t* cu_seqlens, int block,
                      fp2_dtype dtype, void* out, float* lse, const fp2_params* params) {
    fp2_status st = check_decode(params);
    if (st != FP2_OK) return st;
    const fp2_params* P = params;
    if (block != 64 && block != 128) return FP2_ERR_UNSUPPORTED;
    if (dtype != FP2_BF16 && dtype != FP2_FP8_E4M3) return FP2_ERR_INVALID_ARG;
    if (P->out_dtype != FP2_BF16 && P->out_dtype != FP2_FP8_E4M3) return FP2_ERR_INVALID_ARG;
    const bool fp8 = dtype == FP2_FP8_E4M3;
    if (fp8) {
        if (P->head_dim != 128 || block != 128) return FP2_ERR_UNSUPPORTED;
        if (!P->q_scale || !P->k_scale || !P->v_scale) return FP2_ERR_INVALID_ARG;
        if (!P->k_block_factor != !P->v_block_factor) return FP2_ERR_INVALID_ARG;
    } else {
        if (P->k_block_factor || P->v_block_factor) return FP2_ERR_INVALID_ARG;
        if (P->out_dtype == FP2_FP8_E4M3 && !P->out_scale) return FP2_ERR_INVALID_ARG;
    }
    if (page_table) {
        if ((st = check_pages(P)) != FP2_OK) return st;
        if (P->max_pages_per_seq < 1) return FP2_ERR_INVALID_ARG;
    } else if (P->total_k < 0) {
        return FP2_ERR_INVALID_ARG;
    }
    if (!cu_seqlens) return FP2_ERR_INVALID_ARG;
    const DecodeLayout L = decode_layout(P);
    if ((st = check_workspace(P, L.total)) != FP2_OK) return st;
    if (!q || !k_cache || !v_cache || !out) return FP2_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
        !aligned(lse, 4))
        return FP2_ERR_INVALID_ARG;
    if (P->total_q == 0) return FP2_OK;
    if (!page_table && P->total_k == 0) return FP2_ERR_INVALID_ARG;
    // shares read queries, keys and values while others already write their rows
    const size_t nq = (size_t)P->total_q * P->num_q_heads * P->head_dim,
                 rows = page_table ? (size_t)P->num_pages * P->page_size : (size_t)P->total_k,
                 nc = rows * P->num_kv_heads * P->head_dim * (fp8 ? 1 : 2);
    const struct { const void* p; size_t n; } in[] = {{q, nq * (fp8 ? 1 : 2)}, {k_cache, nc}, {v_cache, nc}},
        outs[] = {{out, nq * (P->out_dtype == FP2_FP8_E4M3 ? 1 : 2)},
                  {lse, lse ? (size_t)P->total_q * P->num_q_heads * sizeof(float) : 0}};
    for (const auto& o : outs)
        for (const auto& i : in)
            if (o.n && overlap(o.p, o.n, i.p, i.n)) return FP2_ERR_INVALID_ARG;
    if (outs[1].n && overlap(lse, outs[1].n, out, outs[0].n)) return FP2_ERR_INVALID_ARG;

    uint8_t* ws = static_cast<uint8_t*>(P->workspace);
    fp2::DecodeParams D;
    std::memset(&D, 0, sizeof(D));
    fp2::KParams& kp = D.p;
    kp.num_seqs = P->num_seqs;
    kp.Hq = P->num_q_heads;
    kp.Hkv = P->num_kv_heads;
    kp.d = P->head_dim;
    kp.G = kp.Hq / kp.Hkv;
    kp.B = block;
    kp.total_q = P->total_q;
    kp.total_k = P->total_k;
    kp.paged = page_table ? 1 : 0;
    kp.page_size = page_table ? P->page_size : 0;
    kp.max_pages = page_table ? P->max_pages_per_seq : 0;
    kp.num_pages = page_table ? P->num_pages : 0;
    kp.max_seqlen_q = P->max_seqlen_q;
    // (lengths are rounded up to whole tiles in 32 bits)
    kp.max_seqlen_k = P->max_seqlen_k <= INT32_MAX - 256 ? P->max_seqlen_k : INT32_MAX - 256;
    kp.nkb_max = (int)(((long long)P->max_seqlen_k + block - 1) / block);
    kp.fp8 = fp8;
    kp.uses_kv = 1;
    kp.wait_limit_ns = P->debug_wait_limit_us ? P->debug_wait_limit_us * 1000ull : 2000000000ull;
    kp.withhold_k_item = P->debug_withhold_k_item;
    kp.out_fp8 = P->out_dtype == FP2_FP8_E4M3;
    kp.out_scale = P->out_scale;
    kp.kb_fac = P->k_block_factor;
    kp.vb_fac = P->v_block_factor;
    kp.cu_q = cu_seqlens;
    kp.cu_k = P->cu_seqlens_k ? P->cu_seqlens_k : cu_seqlens;
    kp.seqlens_k = P->seqlens_k;
    kp.page_table = page_table;
    kp.q_scale = P->q_scale;
    kp.k_scale = P->k_scale;
    kp.v_scale = P->v_scale;
    kp.err = reinterpret_cast<uint32_t*>(ws);
    D.q = q;
    D.k = k_cache;
    D.v = v_cache;
    D.out = out;
    D.lse = lse;
    D.part = reinterpret_cast<float*>(ws + L.part);
    D.part_ml = reinterpret_cast<float*>(ws + L.part_ml);
    D.record = reinterpret_cast<int4*>(ws + L.record);
    D.g_shift = __builtin_ctz((unsigned)kp.G);
    D.page_shift = page_table ? __builtin_ctz((unsigned)kp.page_size) : 0;
    D.qk_scale = 1.4426950408889634f / std::sqrt((float)kp.d);
    return cuda_status(fp2::launch_decode(D, stream_of(P)));
}

}  // extern "C"
