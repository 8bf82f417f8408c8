// qb_clip.hip -- the global norm of many gradients, and clipping by it.
//
//   norm = sqrt(sum over gradients and elements of g^2),
//   out = g * min(1, max_norm / (norm + 1e-6)).
// Squares and sums are binary64: no square of a binary32 value leaves its range, and the
// order of the sums does not show in the norm's binary32 digits (it is fixed all the same:
// the same bits on every run).  Two passes over the gradients, bound by HBM; the second one
// walks them backwards, so that it begins with what the last-level cache still holds.
// 0.54e9 bf16 gradients (1.07 GB): norm 173 us, 6.2 TB/s; clip 360 us, 6.0 TB/s.  Every XCD
// walks a contiguous eighth of the tiles (570 -> 555 us together; tiles in turn before), the
// second pass reads and writes with non-temporal accesses (ordinary loads 574, stores 606),
// the first one not (566).  448 gradients of 65536 binary32: 73 us in five launches, 60 in three where
// they are neighbours.
#include "qb_clip.h"
#include "qb_device.h"

namespace qb {

namespace {

// Gradients are often views of a bucket: they begin at any element.
typedef u32x4 __attribute__((aligned(2))) u32x4_e2;

constexpr int kAcc = 8;                  // accesses of a lane and tile

__device__ __forceinline__ float word_value(int dt, const u32x4& w, int j)
{
    if (dt == DT_F32) return ffrom(w[j & 3]);
    const uint32_t h = w[(j >> 1) & 3];
    if (dt == DT_BF16) return (j & 1) ? bf16_hi(h) : bf16_lo(h);
    return (j & 1) ? f16_hi(h) : f16_lo(h);
}

template <int DT>
__device__ __forceinline__ double squares(const u32x4 w)
{
    double s = 0.0;
#pragma unroll
    for (int j = 0; j < (DT == DT_F32 ? 4 : 8); ++j) {
        const double v = (double)word_value(DT, w, j);
        s = __builtin_fma(v, v, s);
    }
    return s;
}

// This lane's accesses of a tile of `left` elements from p on (more than a tile, or the
// gradient's rest).
template <int DT>
struct Share {
    static constexpr int E = DT == DT_F32 ? 4 : 8;
    static constexpr int kTile = (int)grad_tile_elems(DT);
    const char* p;
    int64_t offset;                      // bytes from the gradient's beginning
    int left, lane;

    __device__ __forceinline__ Share(const void* base, int64_t n, int64_t local)
    {
        const int64_t first = local * kTile;
        lane = threadIdx.x & 63;
        left = n - first < kTile ? (int)(n - first) : kTile;
        offset = first * (16 / E);
        p = static_cast<const char*>(base) + offset;
    }
    __device__ __forceinline__ bool whole() const { return left == kTile; }       // uniform
    __device__ __forceinline__ bool has(int i) const { return (i * 64 + lane + 1) * E <= left; }
    __device__ __forceinline__ uint32_t at(int i) const { return (uint32_t)(i * 64 + lane) * 16; }
    // the element of this lane behind the whole accesses, or -1
    __device__ __forceinline__ int rest() const
    {
        const int e = left / E * E + lane;
        return e < left ? e : -1;
    }
    template <bool NT>
    __device__ __forceinline__ u32x4 load(uint32_t at) const
    {
        const QB_G u32x4_e2* const q = (const QB_G u32x4_e2*)(p + at);
        if constexpr (NT) return __builtin_nontemporal_load(q);
        else return *q;
    }
};

// The sum of squares over this lane's share of a tile.
template <int DT>
__device__ __forceinline__ double tile_squares(const void* g, int64_t n, int64_t local)
{
    const Share<DT> t(g, n, local);
    double s = 0.0;
    if (t.whole()) {
        u32x4 w[kAcc];
#pragma unroll
        for (int i = 0; i < kAcc; ++i) w[i] = t.template load<false>(t.at(i));
#pragma unroll
        for (int i = 0; i < kAcc; ++i) s += squares<DT>(w[i]);
        return s;
    }
    const int rest = t.rest();
    if (rest >= 0) {
        const double v = (double)load1<DT>(t.p, rest);
        s = v * v;
    }
    for (int i = 0; i * 64 * Share<DT>::E + Share<DT>::E <= t.left; ++i)
        if (t.has(i)) s += squares<DT>(t.template load<false>(t.at(i)));
    return s;
}

template <int DT>
__device__ __forceinline__ u32x4 scaled(const u32x4 w, float scale)
{
    if constexpr (DT == DT_F32) {
        return u32x4{fbits(ffrom(w.x) * scale), fbits(ffrom(w.y) * scale), fbits(ffrom(w.z) * scale),
                     fbits(ffrom(w.w) * scale)};
    } else {
        u32x4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = pack2<DT>(half_lo<DT>(w[j]) * scale, half_hi<DT>(w[j]) * scale);
        return o;
    }
}

template <int DT>
__device__ __forceinline__ void tile_scale(const void* g, void* out, int64_t n, int64_t local, float scale)
{
    const Share<DT> t(g, n, local);
    char* const q = static_cast<char*>(out) + t.offset;
    if (t.whole()) {
        u32x4 w[kAcc];
#pragma unroll
        for (int i = 0; i < kAcc; ++i) w[i] = t.template load<true>(t.at(i));
#pragma unroll
        for (int i = 0; i < kAcc; ++i) __builtin_nontemporal_store(scaled<DT>(w[i], scale), (QB_G u32x4_e2*)(q + t.at(i)));
        return;
    }
    const int rest = t.rest();
    if (rest >= 0) store1<DT>(q, rest, load1<DT>(t.p, rest) * scale);
    for (int i = 0; i * 64 * Share<DT>::E + Share<DT>::E <= t.left; ++i)
        if (t.has(i)) *(QB_G u32x4_e2*)(q + t.at(i)) = scaled<DT>(t.template load<false>(t.at(i)), scale);
}

// Sum over a workgroup, in lane and wave order (valid in thread 0).
template <int NT>
__device__ __forceinline__ double group_sum64(double v)
{
    __shared__ double s_wave[NT / 64];
#pragma unroll
    for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
    if ((threadIdx.x & 63) == 0) s_wave[threadIdx.x >> 6] = v;
    __syncthreads();
    double sum = 0.0;
    if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 0; w < NT / 64; ++w) sum += s_wave[w];
    }
    return sum;
}

// The launch's table in LDS.  Kernel arguments lie in host memory: all of them are fetched at
// once, not entry by entry on the way to a tile (each launch over 120 of 448 gradients of
// 65536 binary32 took 5 us longer then).  The tiles' beginnings are added up here, which leaves
// room for more gradients.
template <int CAP, bool OUT>
struct LdsTable {
    const void* g[CAP];
    void* out[OUT ? CAP : 1];
    uint64_t size[CAP];
    int32_t tile_begin[CAP + 1];
    int32_t wave_tiles[4];
};

template <class Table, int CAP, bool OUT>
__device__ __forceinline__ void stage_table(LdsTable<CAP, OUT>& s, const Table& t)
{
    static_assert(CAP <= 256, "four waves hold the table");
    const int i = threadIdx.x, wave = i >> 6;
    int tiles = 0;
    if (i < t.count) {
        const uint64_t size = t.size[i];
        s.g[i] = t.g[i];
        if constexpr (OUT) s.out[i] = t.out[i];
        s.size[i] = size;
        const int log2_tile = (size & 3) == DT_F32 ? 11 : 12;
        static_assert(grad_tile_elems(DT_F32) == 1 << 11 && grad_tile_elems(DT_F16) == 1 << 12, "tiles");
        tiles = (int)(((size >> 2) + (1u << log2_tile) - 1) >> log2_tile);
    }
    int sum = tiles;                                     // of the wave's lanes up to this one
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int v = __shfl_up(sum, d);
        if ((i & 63) >= d) sum += v;
    }
    if (wave < 4 && (i & 63) == 63) s.wave_tiles[wave] = sum;
    __syncthreads();
    if (i < t.count) {
        for (int w = 0; w < wave; ++w) sum += s.wave_tiles[w];
        s.tile_begin[i + 1] = sum;
    }
    if (i == 0) s.tile_begin[0] = 0;
    __syncthreads();
}

// The gradient that holds `tile` (not before gradient `lo`): uniform.
template <class Lds>
__device__ __forceinline__ int find_grad(const Lds& s, int count, int tile, int lo)
{
    int hi = count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__builtin_amdgcn_readfirstlane(s.tile_begin[mid]) <= tile) lo = mid;
        else hi = mid;
    }
    return lo;
}

// A wave's gradient: its entry, uniform.
struct Grad {
    const void* g;
    void* out;
    int64_t n;
    int begin, end, dt;
};

__device__ __forceinline__ const void* uniform_pointer(const void* p)
{
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return reinterpret_cast<const void*>((uint64_t)hi << 32 | lo);
}

template <int CAP, bool OUT>
__device__ __forceinline__ Grad grad_at(const LdsTable<CAP, OUT>& s, int i)
{
    Grad a;
    a.g = uniform_pointer(s.g[i]);
    a.out = OUT ? const_cast<void*>(uniform_pointer(s.out[i])) : nullptr;
    const uint64_t size = reinterpret_cast<uint64_t>(uniform_pointer(reinterpret_cast<const void*>(s.size[i])));
    a.n = (int64_t)(size >> 2);
    a.dt = (int)(size & 3);
    a.begin = __builtin_amdgcn_readfirstlane(s.tile_begin[i]);
    a.end = __builtin_amdgcn_readfirstlane(s.tile_begin[i + 1]);
    return a;
}

// A wave's tiles: the workgroups of an XCD (every eighth) walk one eighth of the tiles.
struct Range {
    int begin, end, step;

    __device__ __forceinline__ Range(int total, int waves, int wave)
    {
        const int groups = gridDim.x >= 8 ? 8 : 1, per = (total + groups - 1) / groups;
        const int x = blockIdx.x % groups, in_group = (gridDim.x - x + groups - 1) / groups;
        begin = x * per + (int)(blockIdx.x / groups) * waves + wave;
        end = (x + 1) * per < total ? (x + 1) * per : total;
        step = in_group * waves;
    }
};

constexpr int kNormThreads = 512;

__global__ __launch_bounds__(kNormThreads) void k_grad_squares(const NormTable t, double* __restrict__ part,
                                                               float* __restrict__ norm)
{
    __shared__ LdsTable<kNormGrads, false> s_table;
    stage_table(s_table, t);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int total = t.tiles;
    double sum = 0.0;
    int i = 0;
    Grad a{};
    const Range range(total, kNormThreads / 64, wave);
    for (int tile = range.begin; tile < range.end; tile += range.step) {
        if (tile >= a.end) {
            i = find_grad(s_table, t.count, tile, i);
            a = grad_at(s_table, i);
        }
        const int64_t local = tile - a.begin;
        sum += a.dt == DT_F32   ? tile_squares<DT_F32>(a.g, a.n, local)
               : a.dt == DT_F16 ? tile_squares<DT_F16>(a.g, a.n, local)
                                : tile_squares<DT_BF16>(a.g, a.n, local);
    }
    sum = group_sum64<kNormThreads>(sum);
    if (threadIdx.x == 0) {
        if (norm) norm[0] = (float)sqrt(sum);
        else part[blockIdx.x] = sum;
    }
}

__global__ __launch_bounds__(1024) void k_grad_norm(const double* __restrict__ part, int count, float* __restrict__ norm)
{
    double sum = 0.0;
    for (int i = threadIdx.x; i < count; i += 1024) sum += part[i];
    sum = group_sum64<1024>(sum);
    if (threadIdx.x == 0) norm[0] = (float)sqrt(sum);
}

__global__ __launch_bounds__(256) void k_grad_scale(const ScaleTable t, double max_norm, const float* __restrict__ norm)
{
    __shared__ LdsTable<kScaleGrads, true> s_table;
    const double s = max_norm / ((double)norm[0] + 1e-6);
    const float scale = s >= 1.0 ? 1.0f : (float)s;      // (a NaN stays one)
    stage_table(s_table, t);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int total = t.tiles;
    int i = 0;
    Grad a{};
    const Range range(total, 4, wave);
    for (int tile = range.begin; tile < range.end; tile += range.step) {
        if (tile >= a.end) {
            i = find_grad(s_table, t.count, tile, i);
            a = grad_at(s_table, i);
        }
        if (scale == 1.0f && a.g == a.out) continue;     // nothing to change
        const int64_t local = a.end - 1 - tile;          // the gradient's tiles from its end
        if (a.dt == DT_F32) tile_scale<DT_F32>(a.g, a.out, a.n, local, scale);
        else if (a.dt == DT_F16) tile_scale<DT_F16>(a.g, a.out, a.n, local, scale);
        else tile_scale<DT_BF16>(a.g, a.out, a.n, local, scale);
    }
}

}  // namespace

hipError_t launch_grad_squares(const NormTable& t, double* part, int* groups, float* norm, hipStream_t s)
{
    const int total = t.tiles, per = kNormThreads / 64;
    const int grid = norm ? 1 : (total + per - 1) / per < kNormGroups ? (total + per - 1) / per : kNormGroups;
    if (groups) *groups = grid;
    return launch_kernel_nt(k_grad_squares, grid, kNormThreads, s, t, part, norm);
}

hipError_t launch_grad_norm(const double* part, int count, float* norm, hipStream_t s)
{
    return launch_kernel_nt(k_grad_norm, 1, 1024, s, part, count, norm);
}

hipError_t launch_grad_scale(const ScaleTable& t, double max_norm, const float* norm, hipStream_t s)
{
    const int total = t.tiles;
    const int grid = (total + 3) / 4 < 8192 ? (total + 3) / 4 : 8192;
    return launch_kernel(k_grad_scale, grid, s, t, max_norm, norm);
}

}  // namespace qb
