// The line of key tiles that the tensor-memory kernel of attention with modified scores shares out (kvc_mod_tc.cuh):
// which CTA takes which tiles of which unit, which units it finishes, and where the pieces of the others lie.
// Integer arithmetic only, for host and device alike: the attention kernel writes by it, the merge reads by it, and a
// CPU test walks it.
//
// Every unit of every head has kMtStart places (its start and end) and then one place per tile; CTA c of G takes places
// [c W / G, (c + 1) W / G) of the W in all.  A unit whose tiles all lie in one CTA is finished there.  So a CTA leaves
// pieces of two units at most: its first segment may be the rest of a unit that an earlier CTA began, its last the
// beginning of one that a later CTA ends, and every segment between them is a whole unit.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace kvc {

constexpr int kMtUnits = 2048;                     // most units (per head) of one launch
constexpr int kMtStart = 8;                        // a unit's start and end, in tiles: 9 us at 1.1 us a tile (4 instead: within
                                                   // 3 % either way for chunks of 5 to 2 048 queries)

// Units (per head) of one launch: at most kMtUnits, and so few that a head's places stay inside 32 bits however long its
// units are (2 048 units of 16 million positions would pass them).
inline int units_per_launch(int64_t longest_unit)
{
    const int64_t n = 0x7FFFFFFF / (longest_unit + kMtStart);
    return static_cast<int>(n < 1 ? 1 : (n < kMtUnits ? n : kMtUnits));
}

// A run of key tiles [k0, k1) of (head, unit).
struct Segment {
    int head, unit, k0, k1, tiles;
    bool ok;
    // the CTA holds the whole unit
    __host__ __device__ __forceinline__ bool all() const { return k0 == 0 && k1 == tiles; }
};

// The CTA that has place w of a line of W shared by G: the last c with c W / G <= w.
__host__ __device__ __forceinline__ int cta_of(int64_t w, int64_t W, int64_t G)
{
    const int64_t num = (w + 1) * G - 1;
    if (W * G < 0x7FFFFFFF) return static_cast<int>(static_cast<uint32_t>(num) / static_cast<uint32_t>(W));
    return static_cast<int>(num / W);
}

// Walks a CTA's share of the line; every role makes the same walk.  prefix: [units + 1] places of a head's units.
struct Walk {
    const int32_t *prefix;
    int units, per_head;
    int64_t at, end;      // whole: unit counters instead of places
    int64_t W, G;
    bool whole;
    int stride;

    __host__ __device__ __forceinline__ Walk(const int32_t *prefix_, int units_, int heads, int cta, int ctas, bool whole_)
        : prefix(prefix_), units(units_), per_head(whole_ ? 1 : prefix_[units_]), whole(whole_), stride(ctas)
    {
        W = static_cast<int64_t>(heads) * per_head;
        G = ctas < W ? ctas : W;
        if (whole) {   // unit after unit, dealt in turn
            at = cta;
            end = static_cast<int64_t>(heads) * units;
        } else {
            at = cta < G ? cta * W / G : 0;
            end = cta < G ? (cta + 1) * W / G : 0;
        }
    }

    __host__ __device__ __forceinline__ Segment next()
    {
        Segment s;
        s.ok = at < end;
        if (!s.ok) return s;
        if (whole) {
            s.head = static_cast<int>(at / units);
            s.unit = static_cast<int>(at % units);
            s.k0 = 0;
            s.tiles = s.k1 = 0;   // the caller's, from the unit's view
            at += stride;
            return s;
        }
        s.head = static_cast<int>(at / per_head);
        const int r = static_cast<int>(at - static_cast<int64_t>(s.head) * per_head);
        int lo = 0, hi = units;   // prefix[lo] <= r < prefix[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (prefix[mid] <= r) lo = mid;
            else hi = mid;
        }
        s.unit = lo;
        s.tiles = prefix[lo + 1] - prefix[lo] - kMtStart;
        const int64_t first = static_cast<int64_t>(s.head) * per_head + prefix[lo] + kMtStart;   // place of its tile 0
        s.k0 = at > first ? static_cast<int>(at - first) : 0;
        s.k1 = s.tiles < end - first ? s.tiles : static_cast<int>(end - first);
        s.ok = s.k1 > s.k0;   // else the share ends before the unit's first tile
        at = first + s.k1;
        return s;
    }
};

// Where a piece of a cut unit goes: CTA `cta`'s first segment into its first slot, a later one (the last) into its second.
__host__ __device__ __forceinline__ int64_t piece_slot(int cta, int segment) { return 2 * static_cast<int64_t>(cta) + (segment > 0 ? 1 : 0); }

// The pieces of a unit that lies at places [a, b): in CTAs first .. first + ctas - 1 (1 CTA: no pieces, it finished the
// unit), the first one's in slot0, every later one's in that CTA's first slot.
struct Pieces {
    int first, ctas, slot0;
};
__host__ __device__ __forceinline__ Pieces pieces_of(int64_t a, int64_t b, int64_t W, int64_t G)
{
    Pieces p;
    p.first = cta_of(a + kMtStart, W, G);   // of the unit's first tile
    p.ctas = cta_of(b - 1, W, G) - p.first + 1;
    p.slot0 = 2 * p.first + (a > 0 && cta_of(a - 1, W, G) == p.first ? 1 : 0);   // places before the unit: not its first segment
    return p;
}

}  // namespace kvc
