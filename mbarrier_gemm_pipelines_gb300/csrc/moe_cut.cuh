// moe_cut.cuh -- how the expert layer's work is cut over the SMs: which hidden
// columns of which expert each CTA runs, what fits in its shared memory, and
// how many rows of scratch the parts can take.  Host and device share it: the
// kernel's roles walk it, the host plans with it, and a host-only test checks
// that every unit is run once and that no routing takes more rows.
#pragma once
#include <cstdint>

#include "operators.h"

namespace gbr {
namespace moe {

constexpr uint32_t kSliceBytes = 64 * 128;              // 64 weight rows x 64 columns
constexpr int kMaxStages = 12;
constexpr uint32_t kXStages = 4;
constexpr int kUnit = 64;                               // hidden columns of a unit

// floor(a b / c), in 32 bits where the product fits.
__host__ __device__ __forceinline__ int32_t mul_div(int32_t a, int32_t b, int32_t c) {
    const uint64_t p = uint64_t(uint32_t(a)) * uint32_t(b);
    return int32_t((p >> 32) == 0 ? uint32_t(p) / uint32_t(c) : uint32_t(p / uint32_t(c)));
}

struct CutSizes {
    int32_t units;                                      // of an expert
    int32_t max_units;                                  // of a part, that fit in shared memory
    int32_t sms;
};

// The cut of the list of units, the same in every CTA.  It is made in grains
// of one unit, or of two where that leaves the largest part no larger: two
// units fill a 128-column tile, one costs the tensor core as much.  Where that
// leaves the largest part no larger either, every expert gets its own equal
// number of parts; else parts run on from one expert into the next.
struct Cut {
    int32_t grain;                                      // units
    int32_t per_expert;                                 // grains of an expert
    int32_t total;                                      // grains of all chosen experts
    int32_t parts;
    int32_t own;                                        // parts of each expert, 0: running on
    __host__ __device__ __forceinline__ int32_t begin(int32_t v) const {
        if (own == 0) return mul_div(v, total, parts);
        const int32_t x = v / own;
        return x * per_expert + mul_div(v - x * own, per_expert, own);
    }
    // The parts of the x-th chosen expert: the first, and how many.
    __host__ __device__ __forceinline__ int32_t first(int32_t x) const {
        return own ? x * own : part_of(x * per_expert);
    }
    __host__ __device__ __forceinline__ int32_t count(int32_t x) const {
        return own ? own : part_of((x + 1) * per_expert - 1) - part_of(x * per_expert) + 1;
    }
    // No expert of `active` has more parts.  Running on, an expert is the
    // stretch [x, x + 1) parts / active of the line on which every part has
    // length one, and meets at most one part more than that is long, rounded up.
    __host__ __device__ __forceinline__ int32_t most(int32_t active) const {
        return own ? own : (parts + active - 1) / active + 1;
    }

private:
    // Running on: the part that holds grain u, the last v with begin(v) <= u.
    __host__ __device__ __forceinline__ int32_t part_of(int32_t u) const {
        const uint64_t p = (uint64_t(uint32_t(u)) + 1) * uint32_t(parts) + uint32_t(total) - 1;
        return int32_t((p >> 32) == 0 ? uint32_t(p) / uint32_t(total) : uint32_t(p / uint32_t(total))) - 1;
    }
};

__host__ __device__ __forceinline__ Cut make_cut(const CutSizes& s, int32_t active) {
    Cut c;
    const int32_t twos = (s.units + 1) / 2;
    const int32_t per1 = (active * s.units + s.sms - 1) / s.sms, per2 = 2 * ((active * twos + s.sms - 1) / s.sms);
    c.grain = s.max_units >= 2 && per2 <= per1 ? 2 : 1;
    c.per_expert = c.grain == 2 ? twos : s.units;
    c.total = active * c.per_expert;
    const int32_t per = c.grain == 2 ? per2 : per1;
    const int32_t rounds = (per + s.max_units - 1) / s.max_units, most = s.sms * rounds;
    c.parts = most < c.total ? most : c.total;
    c.own = most / active < c.per_expert ? most / active : c.per_expert;
    const int32_t largest = c.own > 0 ? (c.per_expert + c.own - 1) / c.own * c.grain : per + 1;
    if (largest <= per && largest <= s.max_units) c.parts = active * c.own;
    else c.own = 0;
    return c;
}

// One run of units of one expert inside a part.
struct Segment {
    int32_t index;                                      // of the expert among the chosen
    int32_t u0, n;                                      // first unit within the expert, units
    int32_t part;
};

// Walks the segments of a CTA's parts in order.
struct Walk {
    int32_t v, v_end, at, end;
    __host__ __device__ __forceinline__ Walk(const Cut& c, int32_t cta, int32_t sms) {
        v = mul_div(cta, c.parts, sms);
        v_end = mul_div(cta + 1, c.parts, sms);
        at = end = 0;
        if (v < v_end) {
            at = c.begin(v);
            end = c.begin(v + 1);
        }
    }
    __host__ __device__ __forceinline__ bool next(const Cut& c, int32_t units, Segment& s) {
        if (v >= v_end) return false;
        s.index = at / c.per_expert;
        const int32_t first = at - s.index * c.per_expert, rest = c.per_expert - first;
        const int32_t n = end - at < rest ? end - at : rest;
        s.u0 = first * c.grain;
        s.n = n * c.grain < units - s.u0 ? n * c.grain : units - s.u0;
        s.part = v;
        at += n;
        if (at >= end && ++v < v_end) {
            at = c.begin(v);
            end = c.begin(v + 1);
        }
        return true;
    }
};

struct ExpertPlan {
    int32_t t_pad, units, max_units, stages, ksub;
    size_t smem;
};

inline ExpertPlan plan_experts(const MoeArgs& a, int32_t sms, int32_t smem_optin) {
    auto cdiv = [](int64_t x, int64_t y) { return (x + y - 1) / y; };
    auto least = [](int64_t x, int64_t y) { return x < y ? x : y; };
    ExpertPlan p;
    p.t_pad = int32_t(cdiv(a.T, 16) * 16);
    p.units = int32_t(cdiv(a.F, kUnit));
    const int64_t budget = int64_t(smem_optin) - 1024 - 10 * 1024;   // alignment; tables and barriers
    const int64_t block = p.t_pad * 128, slice = 2 * int64_t(kSliceBytes);
    const int64_t experts = least(a.E, int64_t(a.T) * a.top_k);
    // Room for a part's hidden columns if every expert that can be chosen is,
    // as long as a ring of 80 KiB remains beside it.
    const int64_t want = cdiv(experts * p.units, sms);
    const int64_t xring = int64_t(kXStages) * block;
    const int64_t fit = least(want, (budget - xring - 80 * 1024) / block);
    p.max_units = int32_t(fit > 1 ? fit : 1);
    if (p.max_units > 1) p.max_units = (p.max_units + 1) / 2 * 2;   // grains of two fit whole
    // Stages of 128 weight rows where four of them fit, else of 64: a stage
    // costs its handshakes, whatever its size.
    p.ksub = (budget - p.max_units * block - 2 * xring) / (2 * slice) >= 4 ? 2 : 1;
    const int64_t rest = budget - p.max_units * block - p.ksub * xring;
    p.stages = int32_t(least(kMaxStages, rest / (p.ksub * slice)));
    p.smem = size_t(1024 + p.max_units * block + p.ksub * xring + p.stages * p.ksub * slice);
    return p;
}

// Rows of the parts' buffer that suffice whatever the routing: a token and
// choice takes one row for each part that the chosen expert meets.  Every token
// has top_k experts, so at least that many are chosen.
inline int64_t most_part_rows(const MoeArgs& a, const CutSizes& s) {
    const int64_t pairs = int64_t(a.T) * a.top_k;
    const int32_t most = int32_t(pairs < a.E ? pairs : a.E);
    int64_t rows = 0;
    for (int32_t active = a.top_k; active <= most; ++active) {
        const Cut c = make_cut(s, active);
        // The pairs all on experts with the most parts; or T tokens on every
        // expert, whose parts are those of the cut and one more at each seam.
        const int64_t by_pairs = pairs * c.most(active);
        const int64_t by_experts = int64_t(a.T) * (c.own ? c.parts : c.parts + active - 1);
        const int64_t here = by_pairs < by_experts ? by_pairs : by_experts;
        if (here > rows) rows = here;
    }
    return rows;
}

}  // namespace moe
}  // namespace gbr
