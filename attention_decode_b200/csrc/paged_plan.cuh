// How the paged attention kernels divide their work. A unit is a group of at
// most RC (query row, head) pairs of one sequence and kv-head; its work is
// the 128-token tiles that some row of it sees. The units' tiles, laid end to
// end (sequence, kv-head, group), are cut into equal ranges, one per CTA: no
// CTA waits for a longer one, whatever the lengths, and a long context is
// split by itself. Each unit counts kSetup tiles more, in front of its own,
// for what a CTA spends on a unit besides its tiles. A unit inside one range
// is finished by its CTA; parts of a unit that spans ranges go to the
// workspace and are joined by a second kernel. Lengths are on the device, so
// a warp of each CTA derives its range.
#pragma once

#include "paged.cuh"

namespace nsnq {

constexpr int kTile = 128;  // tokens per tile

#ifdef __CUDACC__

// What the rows of a unit see. Row r of the unit is row r0 + r of the
// sequence's rows x G (head fastest).
struct PagedUnit {
    int row0;        // first packed row of the sequence
    int first_pos;   // position of the sequence's row 0 (may be negative)
    int rows;        // (query row, head) pairs of the unit
    int r0;
    int p0, p1;      // least and largest position
    int lo_tok;      // first token of p0's window
    int lo;          // tiles: `sink_tiles` of the sinks, then those from lo on
    int sink_tiles;
    int n;           // tiles in all
    __device__ __forceinline__ int tile(int j) const { return j < sink_tiles ? j : j - sink_tiles + lo; }
};

// Where a CTA's range begins and ends, and the unit it begins in.
struct PagedRange {
    int64_t begin, end;
    int b, h, g, at;  // at: where in the unit the range begins, setup tiles counted
};

// A unit that crosses from CTA c - 1 into CTA c and began in c - 1 (kept by c):
// its parts are slot `first`, then 2k of CTAs k = c .. last.
struct PagedSeam {
    int live, first, last;
    int row0, r0, rows, h;
    int pad;
};

template <int RC>
__device__ __forceinline__ int paged_groups(const PagedAttnArgs& a, const PagedSeq& q) {
    const int r = q.rows < a.max_rows ? q.rows : (int)a.max_rows;
    return (int)((r * (int64_t)a.G.d + RC - 1) / RC);
}

template <int RC>
__device__ __forceinline__ PagedUnit paged_unit(const PagedAttnArgs& a, const PagedSeq& q, int g) {
    PagedUnit v;
    const int G = (int)a.G.d;
    const int r = q.rows < a.max_rows ? q.rows : (int)a.max_rows;
    v.r0 = g * RC;  // n_rows * Hq < 2^31
    v.rows = r * G - v.r0 < RC ? r * G - v.r0 : RC;
    v.row0 = q.row0;
    v.first_pos = q.len - q.rows;
    v.p0 = v.first_pos + (int)fdiv((uint32_t)v.r0, a.G);
    v.p1 = v.first_pos + (int)fdiv((uint32_t)(v.r0 + v.rows - 1), a.G);
    const int hi = v.p1 >= 0 && q.len > 0 ? v.p1 / kTile + 1 : 0;
    v.lo_tok = a.window && v.p0 >= a.window ? v.p0 - a.window + 1 : 0;
    v.lo = v.lo_tok / kTile;
    const int st = a.sinks / kTile + (a.sinks % kTile != 0);
    v.sink_tiles = st < v.lo ? st : v.lo;
    v.n = hi > v.lo ? v.sink_tiles + hi - v.lo : 0;
    return v;
}

// The segments of a CTA's range: tiles [j0, j1) of a unit, one after the other.
//   for (PagedWalk<RC, kSetup> w(a, range); w.live(); w.next()) ...
template <int RC, int kSetup>
struct PagedWalk {
    const PagedAttnArgs& a;
    PagedSeq s;
    int b, h, g, groups;
    int j0, j1;
    bool first;      // the range began in this unit
    int64_t left;    // of the range, this unit's share included
    PagedUnit u;

    __device__ __forceinline__ PagedWalk(const PagedAttnArgs& args, const PagedRange& r)
        : a(args), b(r.b), h(r.h), g(r.g), first(true), left(r.end - r.begin) {
        if (left <= 0) return;
        s = paged_seq(a.seqs, b);
        groups = paged_groups<RC>(a, s);
        u = paged_unit<RC>(a, s, g);
        share(r.at);
        if (j0 >= j1) next();
    }
    __device__ __forceinline__ bool live() const { return left > 0; }
    __device__ __forceinline__ bool complete() const { return j0 == 0 && j1 == u.n; }
    __device__ __forceinline__ void next() {
        do {
            left -= taken;
            first = false;
            if (left <= 0) return;
            next_unit();
            if (u.n == 0) left = 0;  // the lengths changed under the call
            share(0);
        } while (left > 0 && j0 >= j1);
    }

private:
    int taken;
    __device__ __forceinline__ void share(int at) {
        const int end = left < u.n + kSetup - at ? at + (int)left : u.n + kSetup;
        taken = end - at;
        j0 = at > kSetup ? at - kSetup : 0;
        j1 = end > kSetup ? end - kSetup : 0;
    }
    // The next unit that has tiles; past the last one, u.n = 0.
    __device__ __forceinline__ void next_unit() {
        do {
            if (++g >= groups) {
                g = 0;
                if (++h >= a.Hkv) {
                    h = 0;
                    do {
                        if (++b >= a.seqs.B) {
                            u.n = 0;
                            return;
                        }
                        s = paged_seq(a.seqs, b);
                        groups = paged_groups<RC>(a, s);
                    } while (groups == 0);
                }
            }
            u = paged_unit<RC>(a, s, g);
        } while (u.n == 0);
    }
};

template <int kSetup>
__device__ __forceinline__ int paged_length(const PagedUnit& u) { return u.n ? u.n + kSetup : 0; }

// The tiles of this lane's sequence of chunk b0 .. b0 + 31, for one kv-head.
// Every lane of the warp calls it together. Sequences of a few groups are
// summed by their lane, longer ones by the warp (a prompt has tens of groups
// and may be the only sequence).
template <int RC, int kSetup>
__device__ __noinline__ int64_t paged_head_tiles(const PagedAttnArgs& a, int b0) {
    constexpr int kFew = 2;
    const int lane = lane_id();
    PagedSeq q{};
    int n = 0;
    if (b0 + lane < a.seqs.B) {
        q = paged_seq(a.seqs, b0 + lane);
        n = paged_groups<RC>(a, q);
    }
    int64_t t = 0;
#pragma unroll 1
    for (int i = 0; i < n && n <= kFew; ++i) t += paged_length<kSetup>(paged_unit<RC>(a, q, i));
#pragma unroll 1
    for (unsigned many = __ballot_sync(kFull, n > kFew); many; many &= many - 1) {
        const int src = __ffs(many) - 1;
        PagedSeq o{};
        o.rows = __shfl_sync(kFull, q.rows, src);
        o.len = __shfl_sync(kFull, q.len, src);
        const int m = __shfl_sync(kFull, n, src);
        int64_t part = 0;
#pragma unroll 1
        for (int i = lane; i < m; i += 32) part += paged_length<kSetup>(paged_unit<RC>(a, o, i));
#pragma unroll
        for (int k = 16; k; k >>= 1) part += __shfl_xor_sync(kFull, part, k);
        if (lane == src) t = part;
    }
    return t;
}

__device__ __forceinline__ int64_t warp_prefix(int64_t v) {  // inclusive
    const int lane = lane_id();
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int64_t o = __shfl_up_sync(kFull, v, m);
        if (lane >= m) v += o;
    }
    return v;
}

// The range of CTA c of `grid`, and the seam in front of it. With fewer tiles
// than CTAs, the first `total` take one each. Every lane of one warp calls it
// together; all get the result.
template <int RC, int kSetup>
__device__ __noinline__ PagedRange paged_plan(const PagedAttnArgs& a, int grid, int c) {
    const int lane = lane_id();
    PagedRange r{};
    int64_t total = 0, first_chunk = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < a.seqs.B; b0 += 32) {
        const int64_t mine = paged_head_tiles<RC, kSetup>(a, b0);
        if (b0 == 0) first_chunk = mine;
        total += mine;
    }
#pragma unroll
    for (int m = 16; m; m >>= 1) total += __shfl_xor_sync(kFull, total, m);
    total *= a.Hkv;
    const int n = total < grid ? (int)total : grid;
    // CTA k takes tiles [total * k / n, total * (k + 1) / n)
    int64_t edge = 0;  // lanes 0-2: edges c - 1, c, c + 1
    if (c < n && lane < 3 && c + lane > 0) edge = total * (c + lane - 1) / n;
    const int64_t prev = __shfl_sync(kFull, edge, 0);
    r.begin = __shfl_sync(kFull, edge, 1);
    r.end = __shfl_sync(kFull, edge, 2);
    PagedSeam seam{};
    if (c < n) {
        int64_t x = r.begin, before = 0, per_head = 1;
#pragma unroll 1
        for (int b0 = 0; b0 < a.seqs.B; b0 += 32) {
            const int64_t mine = b0 ? paged_head_tiles<RC, kSetup>(a, b0) : first_chunk;
            const int64_t incl = warp_prefix(mine * a.Hkv);
            const unsigned hit = __ballot_sync(kFull, x < before + incl);
            if (hit) {
                const int src = __ffs(hit) - 1;
                r.b = b0 + src;
                per_head = __shfl_sync(kFull, mine, src);
                x -= before + __shfl_sync(kFull, incl, src) - per_head * a.Hkv;
                break;
            }
            before += __shfl_sync(kFull, incl, 31);
        }
        const PagedSeq s = paged_seq(a.seqs, r.b);
        const int groups = paged_groups<RC>(a, s);
        r.h = (int)(x / per_head);
        x -= r.h * per_head;
#pragma unroll 1
        for (int g0 = 0; g0 < groups; g0 += 32) {
            const int64_t mine = g0 + lane < groups ? paged_length<kSetup>(paged_unit<RC>(a, s, g0 + lane)) : 0;
            const int64_t incl = warp_prefix(mine);
            const unsigned hit = __ballot_sync(kFull, x < incl);
            if (hit) {
                const int src = __ffs(hit) - 1;
                r.g = g0 + src;
                x -= __shfl_sync(kFull, incl - mine, src);
                break;
            }
            x -= __shfl_sync(kFull, incl, 31);
        }
        r.at = (int)x;
        const PagedUnit u = paged_unit<RC>(a, s, r.g);
        const int64_t u0 = r.begin - r.at;
        // CTA c - 1 holds the unit's first tile, and this one a later one
        if (c > 0 && r.at > kSetup && prev <= u0 + kSetup) {
            seam.live = 1;
            seam.first = 2 * (c - 1) + (prev >= u0 ? 0 : 1);
            // the CTA of the unit's last tile x: the last k with edge(k) <= x
            seam.last = (int)(((u0 + u.n + kSetup) * n - 1) / total);
            seam.row0 = u.row0;
            seam.r0 = u.r0;
            seam.rows = u.rows;
            seam.h = r.h;
        }
    }
    if (lane == 0) a.seams[c] = seam;
    return r;
}

#endif  // __CUDACC__

}  // namespace nsnq
