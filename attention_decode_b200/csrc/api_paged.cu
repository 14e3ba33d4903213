// C ABI of the paged 8-bit cache: argument validation and kernel launches.
#include <math.h>

#include "paged.cuh"

namespace {

using nsnq::set_error;

nsnq_status ok() {
    set_error(NSNQ_OK, "%s", "");
    return NSNQ_OK;
}
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Checks that both entry points share; fills the sequences' arguments.
nsnq_status check_paged(const nsnq_paged_cache& c, const int32_t* cu_rows, const int32_t* seq_lens,
                        const int32_t* table, int64_t table_cols, int64_t table_stride, int64_t n_rows,
                        int B, int Hq, int Hkv, int D, nsnq::PagedSeqs& s) {
    if (D != nsnq::kHeadDim) return set_error(NSNQ_ERR_UNSUPPORTED, "D = %d (only 128 is supported)", D);
    if (B < 0 || n_rows < 0 || Hkv <= 0 || Hq <= 0 || Hq % Hkv)
        return set_error(NSNQ_ERR_INVALID_ARG,
                         "need B, n_rows >= 0 and Hq a positive multiple of Hkv (B=%d n_rows=%lld Hq=%d Hkv=%d)",
                         B, (long long)n_rows, Hq, Hkv);
    if (B > 65535 || Hq > 65535) return set_error(NSNQ_ERR_UNSUPPORTED, "B or Hq above 65535");
    if (n_rows >= ((int64_t)1 << 31) / Hq)
        return set_error(NSNQ_ERR_UNSUPPORTED, "n_rows * Hq = %lld * %d (limit 2^31)", (long long)n_rows, Hq);
    if (!cu_rows && n_rows != B)
        return set_error(NSNQ_ERR_INVALID_ARG, "cu_rows is NULL but n_rows = %lld differs from B = %d",
                         (long long)n_rows, B);
    if (c.page_size != 16 && c.page_size != 32 && c.page_size != 64 && c.page_size != 128)
        return set_error(NSNQ_ERR_UNSUPPORTED, "cache.page_size = %d (16, 32, 64 or 128 supported)", c.page_size);
    if (c.heads != Hkv)
        return set_error(NSNQ_ERR_INVALID_ARG, "cache.heads = %d differs from Hkv = %d", c.heads, Hkv);
    if (c.num_pages <= 0)
        return set_error(NSNQ_ERR_INVALID_ARG, "cache.num_pages = %lld (at least 1)", (long long)c.num_pages);
    if (c.num_pages >= ((int64_t)1 << 31) / Hkv)
        return set_error(NSNQ_ERR_UNSUPPORTED, "cache.num_pages * heads = %lld * %d (limit 2^31)",
                         (long long)c.num_pages, Hkv);
    if (table_cols < 0 || table_stride < table_cols)
        return set_error(NSNQ_ERR_INVALID_ARG, "need 0 <= table_cols <= table_stride (%lld, %lld)",
                         (long long)table_cols, (long long)table_stride);
    if (!c.k || !c.v || !c.k_scales || !c.v_scales)
        return set_error(NSNQ_ERR_INVALID_ARG, "cache has a NULL buffer");
    if (!aligned(c.k, 128) || !aligned(c.v, 128))
        return set_error(NSNQ_ERR_INVALID_ARG, "cache.k and cache.v must be 128-byte aligned");
    if (!aligned(c.k_scales, 4) || !aligned(c.v_scales, 4) || !aligned(c.status, 4))
        return set_error(NSNQ_ERR_INVALID_ARG, "cache scales and status must be 4-byte aligned");
    if (c.k == c.v || c.k_scales == c.v_scales)
        return set_error(NSNQ_ERR_INVALID_ARG, "keys and values of the cache share a buffer");
    if (B > 0 && n_rows > 0) {
        if (!seq_lens || (table_cols > 0 && !table))
            return set_error(NSNQ_ERR_INVALID_ARG, "seq_lens or page_table is NULL");
        if (!aligned(seq_lens, 4) || !aligned(cu_rows, 4) || !aligned(table, 4))
            return set_error(NSNQ_ERR_INVALID_ARG, "cu_rows, seq_lens and page_table must be 4-byte aligned");
    }
    s.cu_rows = cu_rows;
    s.seq_lens = seq_lens;
    s.table = table;
    s.table_stride = table_stride;
    // positions are int32: a longer row is usable up to 2^31 - 129 tokens
    const int64_t most = ((int64_t)1 << 31) - 129;
    s.capacity = table_cols > most / c.page_size ? most : table_cols * c.page_size;
    s.n_rows = n_rows;
    s.B = B;
    s.status = c.status;
    return NSNQ_OK;
}

// (the stride of a dimension of one element is never used, and may be any)
nsnq_status check_rows(const void* p, const char* name, int64_t n_rows, int heads, int64_t st, int64_t sh, int64_t esz) {
    if (n_rows == 1) st = 0;
    if (heads == 1) sh = 0;
    if (!p) return set_error(NSNQ_ERR_INVALID_ARG, "%s is NULL", name);
    if (!aligned(p, 16) || (st * esz) % 16 || (sh * esz) % 16)
        return set_error(NSNQ_ERR_INVALID_ARG, "%s and its strides must be 16-byte aligned", name);
    if (st < 0 || sh < 0) return set_error(NSNQ_ERR_INVALID_ARG, "%s has a negative stride", name);
    return NSNQ_OK;
}

// Whether row tensor p (strides in elements of esz bytes) and the contiguous
// output o have bytes in common. Blocks write rows while others still read.
bool overlap(const void* p, int64_t n_rows, int heads, int64_t st, int64_t sh, int64_t esz, const void* o, int64_t rows,
             int Ho, int64_t osz) {
    const uintptr_t p0 = reinterpret_cast<uintptr_t>(p), o0 = reinterpret_cast<uintptr_t>(o);
    const uintptr_t p1 = p0 + ((n_rows - 1) * st + (heads - 1) * sh + nsnq::kHeadDim) * esz;
    return p0 < o0 + rows * Ho * nsnq::kHeadDim * osz && o0 < p1;
}

}  // namespace

extern "C" {

nsnq_status nsnq_paged_append(const void* k, const void* v, const void* q, void* q_out,
                              nsnq_dtype dtype, int64_t n_rows, int64_t k_stride_t,
                              int64_t k_stride_h, int64_t v_stride_t, int64_t v_stride_h,
                              int64_t q_stride_t, int64_t q_stride_h, const int32_t* cu_rows,
                              const int32_t* seq_lens, int B, int Hq, int Hkv, int D,
                              double rope_base, nsnq_paged_cache cache, const int32_t* page_table,
                              int64_t table_cols, int64_t table_stride, nsnq_stream stream) {
    if (dtype != NSNQ_F32 && dtype != NSNQ_BF16)
        return set_error(NSNQ_ERR_UNSUPPORTED, "dtype must be NSNQ_F32 or NSNQ_BF16");
    if (rope_base != 0.0 && (!isfinite(rope_base) || !(rope_base > 1.0)))
        return set_error(NSNQ_ERR_INVALID_ARG, "rope_base = %g must be 0, or finite and > 1", rope_base);
    if (!q) Hq = Hkv;
    nsnq::PagedAppendArgs a{};
    nsnq_status s = check_paged(cache, cu_rows, seq_lens, page_table, table_cols, table_stride, n_rows, B, Hq,
                                Hkv, D, a.seqs);
    if (s != NSNQ_OK) return s;
    if (B == 0 || n_rows == 0) return ok();
    const int64_t esz = dtype == NSNQ_BF16 ? 2 : 4;
    s = check_rows(k, "k", n_rows, Hkv, k_stride_t, k_stride_h, esz);
    if (s == NSNQ_OK) s = check_rows(v, "v", n_rows, Hkv, v_stride_t, v_stride_h, esz);
    if (s == NSNQ_OK && q) s = check_rows(q, "q", n_rows, Hq, q_stride_t, q_stride_h, esz);
    if (s != NSNQ_OK) return s;
    if (q && (!q_out || !aligned(q_out, 16)))
        return set_error(NSNQ_ERR_INVALID_ARG, "q_out is NULL or not 16-byte aligned");
    if (q && q == q_out && ((n_rows > 1 && q_stride_t != (int64_t)Hq * D) || (Hq > 1 && q_stride_h != D)))
        return set_error(NSNQ_ERR_INVALID_ARG, "q_out may equal q only if q is contiguous");
    if (q && (overlap(k, n_rows, Hkv, k_stride_t, k_stride_h, esz, q_out, n_rows, Hq, esz) ||
              overlap(v, n_rows, Hkv, v_stride_t, v_stride_h, esz, q_out, n_rows, Hq, esz) ||
              (q != q_out && overlap(q, n_rows, Hq, q_stride_t, q_stride_h, esz, q_out, n_rows, Hq, esz))))
        return set_error(NSNQ_ERR_INVALID_ARG, "q_out overlaps k, v or (other than as a whole) q");
    a.k = k; a.v = v; a.q = q; a.q_out = q_out;
    a.k_st = k_stride_t; a.k_sh = k_stride_h;
    a.v_st = v_stride_t; a.v_sh = v_stride_h;
    a.q_st = q_stride_t; a.q_sh = q_stride_h;
    a.Hq = Hq; a.Hkv = Hkv;
    a.rope = rope_base != 0.0;
    a.kc = cache.k; a.vc = cache.v; a.ks = cache.k_scales; a.vs = cache.v_scales;
    a.num_pages = cache.num_pages; a.page = cache.page_size;
    // a sequence of n rows touches at most n / page + 2 pages
    a.items = n_rows / a.page + 2 * (int64_t)B;
    for (int i = 0; i < D / 2 && a.rope; ++i) {
        a.freq[i] = pow(rope_base, -2.0 * i / D);
        a.turns[i] = a.freq[i] / 6.283185307179586476925;
    }
    const cudaError_t e = nsnq::launch_paged_append(a, dtype == NSNQ_BF16, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return set_error(NSNQ_ERR_CUDA, "paged append launch: %s", cudaGetErrorString(e));
    return ok();
}

size_t nsnq_paged_attn_workspace(int64_t n_rows, int B, int Hq, int Hkv, int D, int64_t max_rows) {
    if (n_rows < 0 || B < 0 || B > 65535 || Hq <= 0 || Hq > 65535 || Hkv <= 0 || Hq % Hkv ||
        D != nsnq::kHeadDim || max_rows < 0 || n_rows >= ((int64_t)1 << 31) / Hq)
        return 0;
    return nsnq::paged_attn_workspace(n_rows, B, Hq, Hkv, max_rows);
}

nsnq_status nsnq_paged_attn(const void* q, nsnq_dtype q_dtype, int64_t n_rows, int64_t q_stride_t,
                            int64_t q_stride_h, const int32_t* cu_rows, int64_t max_rows,
                            const int32_t* seq_lens, int B, int Hq, int Hkv, int D,
                            nsnq_paged_cache cache, const int32_t* page_table, int64_t table_cols,
                            int64_t table_stride, int64_t window, int64_t sinks,
                            float softmax_scale, void* out, nsnq_dtype out_dtype, void* workspace,
                            size_t workspace_bytes, nsnq_stream stream) {
    if ((q_dtype != NSNQ_F32 && q_dtype != NSNQ_BF16) || (out_dtype != NSNQ_F32 && out_dtype != NSNQ_BF16))
        return set_error(NSNQ_ERR_UNSUPPORTED, "q/out dtype must be NSNQ_F32 or NSNQ_BF16");
    nsnq::PagedAttnArgs a{};
    nsnq_status s = check_paged(cache, cu_rows, seq_lens, page_table, table_cols, table_stride, n_rows, B, Hq,
                                Hkv, D, a.seqs);
    if (s != NSNQ_OK) return s;
    if (window < 0 || sinks < 0)
        return set_error(NSNQ_ERR_INVALID_ARG, "window = %lld and sinks = %lld must not be negative",
                         (long long)window, (long long)sinks);
    if (max_rows < 0) return set_error(NSNQ_ERR_INVALID_ARG, "max_rows = %lld < 0", (long long)max_rows);
    if (!isfinite(softmax_scale)) return set_error(NSNQ_ERR_INVALID_ARG, "softmax_scale is not finite");
    if (B == 0 || n_rows == 0 || max_rows == 0) return ok();
    s = check_rows(q, "q", n_rows, Hq, q_stride_t, q_stride_h, q_dtype == NSNQ_BF16 ? 2 : 4);
    if (s != NSNQ_OK) return s;
    if (!out || !aligned(out, 16)) return set_error(NSNQ_ERR_INVALID_ARG, "out is NULL or not 16-byte aligned");
    const size_t need = nsnq::paged_attn_workspace(n_rows, B, Hq, Hkv, max_rows);
    if (!workspace || workspace_bytes < need)
        return set_error(NSNQ_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                         workspace ? workspace_bytes : (size_t)0);
    if (!aligned(workspace, nsnq::kWsAlign))
        return set_error(NSNQ_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    if (overlap(q, n_rows, Hq, q_stride_t, q_stride_h, q_dtype == NSNQ_BF16 ? 2 : 4, out, n_rows, Hq,
                out_dtype == NSNQ_BF16 ? 2 : 4))
        return set_error(NSNQ_ERR_INVALID_ARG, "out overlaps q");
    a.q = q; a.q_bf16 = q_dtype == NSNQ_BF16;
    a.q_st = q_stride_t; a.q_sh = q_stride_h;
    a.max_rows = max_rows;
    a.Hq = Hq; a.Hkv = Hkv;
    a.kc = cache.k; a.vc = cache.v; a.ks = cache.k_scales; a.vs = cache.v_scales;
    a.num_pages = cache.num_pages; a.page = cache.page_size;
    // positions are below 2^31: larger windows and sinks mean the same
    const int64_t most = ((int64_t)1 << 31) - 1;
    a.window = (int)(window < most ? window : most);
    a.sinks = window ? (int)(sinks < most ? sinks : most) : 0;
    const float scale = softmax_scale == 0.f ? 1.0f / sqrtf((float)D) : softmax_scale;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.out = out; a.out_bf16 = out_dtype == NSNQ_BF16;
    a.G = nsnq::make_fastdiv((uint32_t)(Hq / Hkv));
    a.workspace = workspace;
    const cudaError_t e = nsnq::launch_paged_attn(a, reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return set_error(NSNQ_ERR_CUDA, "paged attention launch: %s", cudaGetErrorString(e));
    return ok();
}

}  // extern "C"
