// How the paged attention kernels divide their work. A unit is a group of at
// most RC (query row, head) pairs of one sequence and kv-head; its work is
// the 128-token tiles that some row of it sees. The units' tiles, laid end to
// end (sequence, kv-head, group), are cut into equal ranges, one per CTA: no
// CTA waits for a longer one, whatever the lengths, and a long context is
// split by itself. A unit inside one range is finished by its CTA; pieces of
// a unit that spans ranges are joined by a second kernel. Lengths are on the
// device, so every warp derives its range itself.
#pragma once

#include "paged.cuh"

namespace nsnq {

constexpr int kTile = 128;  // tokens per tile

#ifdef __CUDACC__

// What the rows of a unit see. Row r of the unit is row r0 + r of the
// sequence's rows x G (head fastest).
struct PagedUnit {
    int b, h, g;
    int row0;        // first packed row of the sequence
    int first_pos;   // position of the sequence's row 0 (may be negative)
    int rows;        // (query row, head) pairs of the unit
    int r0;
    int p0, p1;      // least and largest position
    int lo_tok;      // first token of p0's window
    int lo, hi;      // tiles of the windows: [lo, hi)
    int sink_tiles;  // tiles of the sinks in front of them
    int n;           // tiles in all
    __device__ __forceinline__ int tile(int j) const { return j < sink_tiles ? j : j - sink_tiles + lo; }
};

template <int RC>
struct PagedWalk {
    const PagedAttnArgs& a;
    PagedSeq s;
    int G, b = 0, h = 0, g = 0, groups = 0;
    int64_t first_chunk = 0;  // this lane's sequence of the first 32: its tiles for one kv-head
    PagedUnit u;

    __device__ __forceinline__ explicit PagedWalk(const PagedAttnArgs& args) : a(args), G(args.Hq / args.Hkv) {}

    __device__ __forceinline__ int group_count(const PagedSeq& q) const {
        const int64_t r = q.rows < a.max_rows ? q.rows : a.max_rows;
        return (int)((r * G + RC - 1) / RC);
    }
    __device__ __forceinline__ PagedUnit unit(const PagedSeq& q, int gi) const {
        PagedUnit v;
        const int64_t all = (q.rows < a.max_rows ? q.rows : a.max_rows) * (int64_t)G;
        v.r0 = gi * RC;
        v.rows = (int)(all - v.r0 < RC ? all - v.r0 : RC);
        v.row0 = q.row0;
        v.first_pos = q.len - q.rows;
        v.p0 = v.first_pos + v.r0 / G;
        v.p1 = v.first_pos + (v.r0 + v.rows - 1) / G;
        v.hi = v.p1 >= 0 && q.len > 0 ? v.p1 / kTile + 1 : 0;
        v.lo_tok = a.window && v.p0 >= a.window ? v.p0 - a.window + 1 : 0;
        v.lo = v.lo_tok / kTile;
        const int st = a.sinks / kTile + (a.sinks % kTile != 0);
        v.sink_tiles = st < v.lo ? st : v.lo;
        v.n = v.hi > v.lo ? v.sink_tiles + v.hi - v.lo : 0;
        v.b = b;
        v.h = h;
        v.g = gi;
        return v;
    }
    // This lane's sequence of chunk b0 .. b0 + 31: the tiles of its units for one
    // kv-head. Every lane of the warp calls it together. Sequences of a few
    // groups are summed by their lane, longer ones by the warp (a prompt has
    // tens of groups and may be the only sequence).
    __device__ __forceinline__ int64_t head_tiles(int b0) const {
        constexpr int kFew = 2;
        const int lane = lane_id();
        PagedSeq q{};
        int n = 0;
        if (b0 + lane < a.seqs.B) {
            q = paged_seq(a.seqs, b0 + lane);
            n = group_count(q);
        }
        int64_t t = 0;
        if (n <= kFew)
            for (int i = 0; i < n; ++i) t += unit(q, i).n;
        for (unsigned many = __ballot_sync(kFull, n > kFew); many; many &= many - 1) {
            const int src = __ffs(many) - 1;
            PagedSeq o;
            o.row0 = 0;
            o.rows = __shfl_sync(kFull, q.rows, src);
            o.len = __shfl_sync(kFull, q.len, src);
            const int m = __shfl_sync(kFull, n, src);
            int64_t part = 0;
            for (int i = lane; i < m; i += 32) part += unit(o, i).n;
#pragma unroll
            for (int k = 16; k; k >>= 1) part += __shfl_xor_sync(kFull, part, k);
            if (lane == src) t = part;
        }
        return t;
    }
    // Tiles of all sequences. Every lane of the warp calls it together.
    __device__ __forceinline__ int64_t total() {
        int64_t t = 0;
        for (int b0 = 0; b0 < a.seqs.B; b0 += 32) {
            const int64_t mine = head_tiles(b0);
            if (b0 == 0) first_chunk = mine;
            t += mine;
        }
#pragma unroll
        for (int m = 16; m; m >>= 1) t += __shfl_xor_sync(kFull, t, m);
        return t * a.Hkv;
    }
    // Goes to the unit that holds tile x < total(), which was called before;
    // returns the tile's number in it. Every lane of the warp calls it together.
    __device__ __forceinline__ int seek(int64_t x) {
        const int lane = lane_id();
        int64_t before = 0, per_head = 1;
        b = 0;
        for (int b0 = 0; b0 < a.seqs.B; b0 += 32) {
            const int64_t mine = b0 ? head_tiles(b0) : first_chunk;
            int64_t incl = mine * a.Hkv;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const int64_t o = __shfl_up_sync(kFull, incl, m);
                if (lane >= m) incl += o;
            }
            const unsigned hit = __ballot_sync(kFull, x < before + incl);
            if (hit) {
                const int src = __ffs(hit) - 1;
                b = b0 + src;
                per_head = __shfl_sync(kFull, mine, src);
                x -= before + __shfl_sync(kFull, incl, src) - per_head * a.Hkv;
                break;
            }
            before += __shfl_sync(kFull, incl, 31);
        }
        s = paged_seq(a.seqs, b);
        groups = group_count(s);
        h = (int)(x / per_head);
        x -= h * per_head;
        for (int g0 = 0; g0 < groups; g0 += 32) {
            const int mine = g0 + lane < groups ? unit(s, g0 + lane).n : 0;
            int64_t incl = mine;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const int64_t o = __shfl_up_sync(kFull, incl, m);
                if (lane >= m) incl += o;
            }
            const unsigned hit = __ballot_sync(kFull, x < incl);
            if (hit) {
                const int src = __ffs(hit) - 1;
                g = g0 + src;
                x -= __shfl_sync(kFull, incl, src) - __shfl_sync(kFull, mine, src);
                break;
            }
            x -= __shfl_sync(kFull, incl, 31);
        }
        u = unit(s, g);
        return (int)x;
    }
    // The next unit that has tiles; past the last one, u.n = 0.
    __device__ __forceinline__ void next() {
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
                        groups = group_count(s);
                    } while (groups == 0);
                }
            }
            u = unit(s, g);
        } while (u.n == 0);
    }
};

// CTA c of n = plan_ctas takes tiles [plan_begin(c), plan_begin(c + 1)) of
// total, at least one; tile x belongs to CTA plan_cta(x).
__device__ __forceinline__ int plan_ctas(int64_t total, int grid) { return total < grid ? (int)total : grid; }
__device__ __forceinline__ int64_t plan_begin(int64_t total, int n, int c) { return total * c / n; }
__device__ __forceinline__ int plan_cta(int64_t total, int n, int64_t x) { return (int)(((x + 1) * n - 1) / total); }

#endif  // __CUDACC__

}  // namespace nsnq
