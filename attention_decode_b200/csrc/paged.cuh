// Shared by the kernels of the paged 8-bit cache: launch arguments, the rows
// and length of a sequence as the device arrays give them, e4m3 conversions.
#pragma once

#include <stdint.h>

#include "common.cuh"
#include "internal.h"

namespace nsnq {

// The sequences of a call: packed rows, lengths and page table, on the device.
struct PagedSeqs {
    const int32_t* cu_rows;   // [B + 1] or NULL (one row per sequence)
    const int32_t* seq_lens;  // [B]
    const int32_t* table;     // [B][table_cols], rows table_stride apart
    int64_t table_stride;
    int64_t capacity;         // tokens a table row can hold (at most 2^31 - 1)
    int64_t n_rows;
    int B;
    uint32_t* status;         // or NULL
};

struct PagedAppendArgs {
    PagedSeqs seqs;
    const void* k;
    const void* v;
    const void* q;
    void* q_out;
    int64_t k_st, k_sh, v_st, v_sh, q_st, q_sh;
    int Hq, Hkv;
    int rope;
    uint8_t* kc;
    uint8_t* vc;
    float* ks;
    float* vs;
    int64_t num_pages;
    int page;
    int64_t items;       // page slots the grid covers (an upper bound of those written)
    int heads;            // heads a block takes (set by the launcher)
    double freq[kD / 2];  // rope_base^(-2i/D): radians a token
    double turns[kD / 2];  // the same in turns
};
cudaError_t launch_paged_append(PagedAppendArgs a, bool bf16, cudaStream_t s);

struct PagedAttnArgs {
    PagedSeqs seqs;
    const void* q;
    int q_bf16;
    int64_t q_st, q_sh;
    int64_t max_rows;
    int Hq, Hkv;
    const uint8_t* kc;
    const uint8_t* vc;
    const float* ks;
    const float* vs;
    int64_t num_pages;
    int page;
    int window;  // 0: none
    int sinks;
    float scale_log2;
    void* out;
    int out_bf16;
    FastDiv G;                // query heads per kv-head
    void* workspace;
    struct PagedSeam* seams;  // set by the launchers: one per CTA, then the parts
    float* part;
};
size_t paged_attn_workspace(int64_t n_rows, int B, int Hq, int Hkv, int64_t max_rows);
cudaError_t launch_paged_attn(const PagedAttnArgs& a, cudaStream_t s);

#ifdef __CUDACC__

constexpr uint32_t kBadPage = NSNQ_PAGED_BAD_PAGE, kBadLength = NSNQ_PAGED_BAD_LENGTH, kTimeout = NSNQ_PAGED_TIMEOUT;

__device__ __forceinline__ void paged_report(const PagedSeqs& s, uint32_t bits) {
    if (s.status && bits) atomicOr(s.status, bits);
}

// Sequence b: its first row, its row count and its tokens with those rows.
// A length that the table row cannot hold, or rows outside [0, n_rows] (clamped
// into it), make the sequence empty of tokens (len = 0): where its tokens are is
// not known, and nothing of it is stored or attended.
struct PagedSeq {
    int row0, rows, len;
    uint32_t bad;
};
__device__ __forceinline__ PagedSeq paged_seq(const PagedSeqs& s, int b) {
    PagedSeq r;
    int64_t lo = b, hi = b + 1;
    if (s.cu_rows) {
        lo = s.cu_rows[b];
        hi = s.cu_rows[b + 1];
    }
    const int64_t clo = lo < 0 ? 0 : (lo > s.n_rows ? s.n_rows : lo);
    const int64_t chi = hi < clo ? clo : (hi > s.n_rows ? s.n_rows : hi);
    r.row0 = (int)clo;
    r.rows = (int)(chi - clo);
    r.len = s.seq_lens[b];
    r.bad = (clo != lo || chi != hi) ? kBadLength : 0u;
    if (r.bad || r.len < 0 || r.len > s.capacity) {
        r.len = 0;
        r.bad = kBadLength;
    }
    if (r.len < r.rows) r.bad = kBadLength;
    return r;
}

// Sixteen bits of two e4m3 codes from two values (nearest, ties to even,
// held at +-448; NaN stays NaN); the low byte holds a.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}
// Two e4m3 codes as fp16 (exact), low byte in the low half.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t c) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)c));
    return r;
}
__device__ __forceinline__ float f16_lo(uint32_t h) {
    float r;
    asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;}" : "=f"(r) : "r"(h));
    return r;
}
__device__ __forceinline__ float f16_hi(uint32_t h) {
    float r;
    asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, h;}" : "=f"(r) : "r"(h));
    return r;
}

#endif  // __CUDACC__

}  // namespace nsnq
