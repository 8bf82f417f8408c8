// qb_rows.h -- device helpers of the row-wise layers (embedding lookup, layer
// norm): rows are cut into units of 8 elements, one unit per lane and step.
#pragma once
#include "qb_device.h"
#include "qb_layers.h"

namespace qb {

// Rows start at any multiple of the element size (dim may be odd), so units are
// accessed through vector types of element alignment: the GLOBAL instructions
// take them as they are (gfx950 runs in unaligned-access mode), and an aligned
// row costs the same as through aligned types.
typedef u32x4 __attribute__((aligned(2))) u32x4_a2;
typedef f32x4 __attribute__((aligned(4))) f32x4_a4;

// The raw bits of one unit: 16 bytes of a 16-bit type, 32 of binary32.
template <int DT>
struct Unit {
    uint32_t w[DT == DT_F32 ? 8 : 4];
};

constexpr int elem_bytes(int dt) { return dt == DT_F32 ? 4 : 2; }

// NT: non-temporal accesses for data read or written once, 16-bit types only: a
// binary32 unit takes two instructions that touch the same cache lines, and
// with the non-temporal hint the second one went to memory again (gradient of 5003
// ragged rows of 1001 elements: 38 us against 28 us).
template <int DT, bool NT>
__device__ __forceinline__ Unit<DT> load_unit8(const void* row, int64_t elem)
{
    Unit<DT> u;
    const char* p = static_cast<const char*>(row) + elem * elem_bytes(DT);
#pragma unroll
    for (int h = 0; h < (DT == DT_F32 ? 2 : 1); ++h) {
        const QB_G u32x4_a2* q = (const QB_G u32x4_a2*)(p + 16 * h);
        u32x4 v;
        if constexpr (NT && DT != DT_F32) v = __builtin_nontemporal_load(q);
        else v = *q;
        u.w[4 * h] = v.x; u.w[4 * h + 1] = v.y; u.w[4 * h + 2] = v.z; u.w[4 * h + 3] = v.w;
    }
    return u;
}

template <int DT>
__device__ __forceinline__ float unit_at(const Unit<DT>& u, int j)
{
    if constexpr (DT == DT_F32) return ffrom(u.w[j]);
    else return (j & 1) ? half_hi<DT>(u.w[j >> 1]) : half_lo<DT>(u.w[j >> 1]);
}

// The unit of a row's last `left` (1 .. 7) elements; the others are zero.
template <int DT>
__device__ __forceinline__ Unit<DT> load_part8(const void* row, int64_t elem, int left)
{
    Unit<DT> u;
#pragma unroll
    for (int j = 0; j < (DT == DT_F32 ? 8 : 4); ++j) u.w[j] = 0u;
    const char* p = static_cast<const char*>(row) + elem * elem_bytes(DT);
#pragma unroll
    for (int j = 0; j < 7; ++j) {
        if (j < left) {
            if constexpr (DT == DT_F32) u.w[j] = gld<uint32_t>(p + 4 * j);
            else u.w[j >> 1] |= (uint32_t)gld<uint16_t>(p + 2 * j) << (16 * (j & 1));
        }
    }
    return u;
}

// Elements `by` (0 .. 7) and up of a unit, moved to the front; zeros follow.
template <int DT>
__device__ __forceinline__ void shift_unit(Unit<DT>& u, int by)
{
    constexpr int W = DT == DT_F32 ? 8 : 4;
    const int words = DT == DT_F32 ? by : by >> 1;
#pragma unroll
    for (int step = W / 2; step > 0; step /= 2)
#pragma unroll
        for (int j = 0; j < W; ++j) u.w[j] = (words & step) ? (j + step < W ? u.w[j + step] : 0u) : u.w[j];
    if constexpr (DT != DT_F32) {
#pragma unroll
        for (int j = 0; j < W; ++j) u.w[j] = __builtin_amdgcn_alignbit(j + 1 < W ? u.w[j + 1] : 0u, u.w[j], (by & 1) * 16);
    }
}

// What the last unit of a row is: whole, partial, or the row's only one of fewer
// than 8 elements.
constexpr int kWhole = 0, kPartial = 1, kShort = 2;
constexpr int tail_of(int64_t dim) { return dim < 8 ? kShort : dim % 8 ? kPartial : kWhole; }

// Unit number `unit` of a row of `dim` elements.  A unit beyond the row (unit >=
// ceil(dim / 8)) reads unit 0 instead (its caller masks it), and a partial last
// unit is read as the row's last 8 elements and shifted, so that no load is under a
// branch and a wave's loads are in flight together.  (Read element by element, the
// one lane that holds the partial unit took a chain of up to 7 loads while its wave
// waited; with a branch for rows of fewer than 8 elements every load was waited for
// before the next.)
template <int DT, int TAIL, bool NT>
__device__ __forceinline__ Unit<DT> load_row_unit(const void* row, int unit, int units, int dim)
{
    const int e = (unit < units ? unit : 0) * 8;
    if constexpr (TAIL == kWhole) {
        return load_unit8<DT, NT>(row, e);
    } else if constexpr (TAIL == kPartial) {
        const int at = e < dim - 8 ? e : dim - 8;
        Unit<DT> u = load_unit8<DT, NT>(row, at);
        shift_unit<DT>(u, e - at);
        return u;
    } else {
        return load_part8<DT>(row, 0, dim);
    }
}

// Two values in one word, rounded to nearest even (bf16: one instruction for both).
template <int DT>
__device__ __forceinline__ uint32_t pack_pair(float a, float b)
{
    if constexpr (DT == DT_BF16) {
        typedef float f32x2 __attribute__((ext_vector_type(2)));
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        const bf16x2 h = __builtin_convertvector((f32x2){a, b}, bf16x2);
        uint32_t u;
        __builtin_memcpy(&u, &h, 4);
        return u;
    } else {
        return pack2<DT>(a, b);
    }
}

template <int DT, bool NT>
__device__ __forceinline__ void store_unit8(void* row, int64_t elem, const float* v)
{
    char* p = static_cast<char*>(row) + elem * elem_bytes(DT);
    if constexpr (DT == DT_F32) {
        f32x4 a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
        QB_G f32x4_a4* q = (QB_G f32x4_a4*)p;
        q[0] = a;
        q[1] = b;
    } else {
        u32x4 a = {pack_pair<DT>(v[0], v[1]), pack_pair<DT>(v[2], v[3]), pack_pair<DT>(v[4], v[5]),
                   pack_pair<DT>(v[6], v[7])};
        QB_G u32x4_a2* q = (QB_G u32x4_a2*)p;
        if constexpr (NT) __builtin_nontemporal_store(a, q);
        else *q = a;
    }
}

// Stores unit `unit` of a row (nothing beyond the row, a partial last unit element by element).
template <int DT, int TAIL, bool NT>
__device__ __forceinline__ void store_row_unit(void* row, int unit, int units, int dim, const float* v)
{
    if (unit >= units) return;
    if constexpr (TAIL) {
        const int left = dim - unit * 8;
        if (left < 8) {
#pragma unroll
            for (int j = 0; j < 7; ++j)
                if (j < left) store1<DT>(row, (int64_t)unit * 8 + j, v[j]);
            return;
        }
    }
    store_unit8<DT, NT>(row, (int64_t)unit * 8, v);
}

// The same with the type known at run time only (uniform).  Both 16-bit types
// share the stores: these calls sit in loops whose code a few waves run once, bound by
// the fetch of its instructions.
template <int TAIL, bool NT>
__device__ __forceinline__ void store_row_unit_rt(int dt, void* row, int unit, int units, int dim, const float* v)
{
    if (dt == DT_F32) {
        store_row_unit<DT_F32, TAIL, NT>(row, unit, units, dim, v);
        return;
    }
    u32x4 a;
    if (dt == DT_BF16)
        a = u32x4{pack_pair<DT_BF16>(v[0], v[1]), pack_pair<DT_BF16>(v[2], v[3]), pack_pair<DT_BF16>(v[4], v[5]),
                  pack_pair<DT_BF16>(v[6], v[7])};
    else
        a = u32x4{pack_pair<DT_F16>(v[0], v[1]), pack_pair<DT_F16>(v[2], v[3]), pack_pair<DT_F16>(v[4], v[5]),
                  pack_pair<DT_F16>(v[6], v[7])};
    if (unit >= units) return;
    char* const p = static_cast<char*>(row) + (int64_t)unit * 16;
    if (TAIL && dim - unit * 8 < 8) {
        const int left = dim - unit * 8;
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (j < left) gst<uint16_t>(p + 2 * j, (uint16_t)(a[j >> 1] >> (16 * (j & 1))));
        return;
    }
    QB_G u32x4_a2* const q = (QB_G u32x4_a2*)p;
    if constexpr (NT) __builtin_nontemporal_store(a, q);
    else *q = a;
}

// v += unit `unit` of a row whose type is known at run time only.
template <int TAIL>
__device__ __forceinline__ void add_row_unit_rt(int dt, const void* row, int unit, int units, int dim, float* v)
{
    if (dt == DT_F32) {
        const Unit<DT_F32> u = load_row_unit<DT_F32, TAIL, false>(row, unit, units, dim);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += unit_at<DT_F32>(u, j);
    } else {
        // (the 16-bit loads do not depend on which of the two types it is)
        const Unit<DT_BF16> u = load_row_unit<DT_BF16, TAIL, false>(row, unit, units, dim);
        Unit<DT_F16> h;
#pragma unroll
        for (int j = 0; j < 4; ++j) h.w[j] = u.w[j];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += dt == DT_BF16 ? unit_at<DT_BF16>(u, j) : unit_at<DT_F16>(h, j);
    }
}

__device__ __forceinline__ float load1_rt(int dt, const void* p, int64_t i)
{
    return dt == DT_F32 ? load1<DT_F32>(p, i) : dt == DT_F16 ? load1<DT_F16>(p, i) : load1<DT_BF16>(p, i);
}

__device__ __forceinline__ void store1_rt(int dt, void* p, int64_t i, float v)
{
    if (dt == DT_F32) store1<DT_F32>(p, i, v);
    else if (dt == DT_F16) store1<DT_F16>(p, i, v);
    else store1<DT_BF16>(p, i, v);
}

// Number of elements of unit `unit` that lie in the row: 8, or fewer at its end, or none beyond it.
__device__ __forceinline__ int unit_count(int unit, int dim)
{
    const int left = dim - unit * 8;
    return left < 0 ? 0 : left > 8 ? 8 : left;
}

// Token id number t (32- or 64-bit ids) as 64 bits.
__device__ __forceinline__ int64_t load_id(const void* ids, int id64, int64_t t)
{
    return id64 ? gld<int64_t>(static_cast<const int64_t*>(ids) + t)
                : (int64_t)gld<int32_t>(static_cast<const int32_t*>(ids) + t);
}

// Sum over aligned groups of L lanes (16 or 64), the same bits in every lane
// of the group.  All 64 lanes must be active.  Four steps leave a row of 16
// lanes its sum in every lane; two more carry the rows' sums into lane 63, in
// row order.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ float dpp_add(float v)
{
    return v + ffrom((uint32_t)__builtin_amdgcn_update_dpp(0, (int)fbits(v), CTRL, ROWS, 0xF, ROWS == 0xF));
}

template <int L>
__device__ __forceinline__ float lanes_sum(float v)
{
    static_assert(L == 16 || L == 64, "row of 16 lanes or whole wave");
    v = dpp_add<0xB1>(v);            // quad_perm [1,0,3,2]
    v = dpp_add<0x4E>(v);            // quad_perm [2,3,0,1]
    v = dpp_add<0x141>(v);           // row_half_mirror
    v = dpp_add<0x140>(v);           // row_mirror
    if constexpr (L == 64) {
        v = dpp_add<0x142, 0xA>(v);  // row_bcast:15 into rows 1 and 3
        v = dpp_add<0x143, 0xC>(v);  // row_bcast:31 into rows 2 and 3
        v = ffrom((uint32_t)__builtin_amdgcn_readlane((int)fbits(v), 63));
    }
    return v;
}

// Sum over aligned groups of W lanes (a power of two up to 16), the same bits in
// every lane of the group.
template <int W>
__device__ __forceinline__ float group_sum(float v)
{
    if constexpr (W >= 2) v = dpp_add<0xB1>(v);
    if constexpr (W >= 4) v = dpp_add<0x4E>(v);
    if constexpr (W >= 8) v = dpp_add<0x141>(v);
    if constexpr (W >= 16) v = dpp_add<0x140>(v);
    return v;
}

// Workgroup barrier that orders LDS accesses only: global loads and stores stay in flight across it.
__device__ __forceinline__ void lds_barrier()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

}  // namespace qb
