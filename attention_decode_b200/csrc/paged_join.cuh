// Shared by the two paged attention kernels: their arguments, the parts that
// a CTA leaves in the workspace for a unit it did not finish, and the kernel
// that joins them.
#pragma once

#include "attn_split.cuh"
#include "paged_plan.cuh"
#include "umma.cuh"

namespace nsnq {

// Prompt rows: paged_rows.cu.
cudaError_t launch_paged_rows(const PagedAttnArgs& a, cudaStream_t s);
size_t paged_rows_workspace();

// A part of a unit of RC rows: [RC][128] sums, [RC] m, [RC] l. A CTA leaves at
// most two: slot 2c for the unit its range begins in, 2c + 1 for a later one.
template <int RC>
__host__ __device__ constexpr int64_t part_stride() { return RC * (kD + 2); }

struct MapPair {
    CUtensorMap k, v;
};

#ifdef __CUDACC__

__device__ __forceinline__ void store_out(const PagedAttnArgs& a, int64_t row, int d, float v) {
    if (a.out_bf16) reinterpret_cast<__nv_bfloat16*>(a.out)[row * kD + d] = __float2bfloat16_rn(v);
    else reinterpret_cast<float*>(a.out)[row * kD + d] = v;
}

// Waits until a limit; once a wait has failed, the kernel goes through the
// motions without waiting (every index is still in bounds) and the call's
// results are void: it reports that.
struct Waiter {
    bool good = true;
    __device__ __forceinline__ void operator()(uint32_t bar, uint32_t parity) {
        if (good) good = mbar_wait(bar, parity);
    }
};

constexpr int kJoinThreads = 128;  // one per channel

// Block (c, y), c < grid: if a unit crosses from CTA c - 1 into CTA c and began
// in c - 1, joins its rows y, y + gridDim.y, ... Block (grid + b, y): zeros for
// the rows of sequence b that lie in front of its first token.
template <int RC>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const __grid_constant__ PagedAttnArgs a, int grid) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int d = threadIdx.x;
    if ((int)blockIdx.x >= grid) {
        const PagedSeq s = paged_seq(a.seqs, blockIdx.x - grid);
        const int64_t rows = s.rows < a.max_rows ? s.rows : a.max_rows;
        const int64_t blind = s.rows - s.len < rows ? s.rows - s.len : rows;
        for (int64_t i = blockIdx.y; i < blind * a.Hq; i += gridDim.y)
            store_out(a, (int64_t)s.row0 * a.Hq + i, d, 0.f);
        return;
    }
    const int c = blockIdx.x;
    PagedWalk<RC> walk(a);
    const int64_t total = walk.total();
    const int ctas = plan_ctas(total, grid);
    if (c == 0 || c >= ctas) return;
    const int64_t x = plan_begin(total, ctas, c);
    const int j = walk.seek(x);
    const PagedUnit u = walk.u;
    const int64_t u0 = x - j, u1 = u0 + u.n;
    if (j == 0 || u0 < plan_begin(total, ctas, c - 1)) return;
    const int c1 = plan_cta(total, ctas, u1 - 1);
    const int G = walk.G;
    auto part = [&](int k) {
        return a.part + (2 * k + (plan_begin(total, ctas, k) >= u0 ? 0 : 1)) * part_stride<RC>();
    };
    for (int r = blockIdx.y; r < u.rows; r += gridDim.y) {
        float top = -INFINITY;
        for (int k = c - 1; k <= c1; ++k) {
            const float* p = part(k) + RC * kD + r;
            if (p[RC] != 0.f) top = fmaxf(top, p[0]);
        }
        float sum = 0.f, acc = 0.f;
        for (int k = c - 1; k <= c1; ++k) {
            const float* p = part(k);
            const float l = p[RC * kD + RC + r];
            if (l == 0.f) continue;
            const float f = exp2_approx(p[RC * kD + r] - top);
            sum = fmaf(f, l, sum);
            acc = fmaf(f, p[r * kD + d], acc);
        }
        const int rr = u.r0 + r, i = rr / G;
        store_out(a, (int64_t)(u.row0 + i) * a.Hq + u.h * G + rr - i * G, d, sum == 0.f ? 0.f : acc / sum);
    }
}

template <int RC>
cudaError_t launch_paged_join(const PagedAttnArgs& a, int grid, cudaStream_t s) {
    static std::atomic<unsigned long long> ready{0};
    return launch_smem_pdl(paged_join_kernel<RC>, ready, dim3(grid + a.seqs.B, RC < 32 ? RC : 32),
                           dim3(kJoinThreads), 0, s, a, grid);
}

#endif  // __CUDACC__

}  // namespace nsnq
