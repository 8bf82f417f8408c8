// qb_clip.h -- internal launchers of the global gradient norm and of clipping by it.
#pragma once
#include "qb_launch.h"

namespace qb {

// Gradients of one launch, passed by value: no table is copied to the device, so that the
// calls may be captured into a graph and need no host memory afterwards (3.6 KB of
// kernel arguments).  size[i]: elements << 2 | dtype; tiles: of all of them.
constexpr int kNormGrads = 224, kScaleGrads = 150;

struct NormTable {
    const void* g[kNormGrads];
    uint64_t size[kNormGrads];
    int32_t count, tiles;
};
struct ScaleTable {
    const void* g[kScaleGrads];
    void* out[kScaleGrads];
    uint64_t size[kScaleGrads];
    int32_t count, tiles;
};
static_assert(sizeof(NormTable) <= 3700 && sizeof(ScaleTable) <= 3700, "kernel arguments are at most 4 KB");

// A tile is a wave's 8 accesses of 16 bytes a lane.
constexpr int64_t grad_tile_elems(int dt) { return 64 * 8 * (dt == 0 ? 4 : 8); }

// Workgroups of a norm launch at most: one partial sum each.
constexpr int kNormGroups = 1024;
// Tiles up to which one workgroup takes them all and writes the norm itself.
constexpr int kNormFewTiles = 64;

// part[0 .. groups) = the sums of squares of the workgroups of one launch; returns their
// number.  norm != nullptr: one workgroup, which writes sqrt of its sum there.
hipError_t launch_grad_squares(const NormTable& t, double* part, int* groups, float* norm, hipStream_t s);
// norm[0] = sqrt(sum of part), in order.
hipError_t launch_grad_norm(const double* part, int count, float* norm, hipStream_t s);
// out = g * min(1, max_norm / (norm[0] + 1e-6)), every gradient from its end (the table
// lists the gradients from the last on).
hipError_t launch_grad_scale(const ScaleTable& t, double max_norm, const float* norm, hipStream_t s);

}  // namespace qb
