// qb_stable_grad.hip -- the gradients of the stable embedding (layer norm of an
// embedding's rows).
//
// All tokens of one id v share the row x = scale * W[v] and with it mean, rstd and
// h = (x - mean) * rstd, and the layer norm's gradient is linear in dy.  With S_v = sum of dy_t over the tokens of v and g = S_v * gamma:
//   dW[v]  = scale * rstd * (g - mean(g) - h * mean(g h)),
//   dgamma = sum_v S_v h,  dbeta = sum_v S_v.
// So dy is read once and summed by id first, every used row of W is read once,
// the norm's backward pass runs once per used id instead of once per token, and
// no [tokens, dim] intermediate is written: the bytes are those of the plain
// embedding's gradient plus the used rows of W.  16384 tokens, [32000, 4096] binary32
// with bf16 gradients: 127 us for 473 MB in five launches (ordering 12, k_prepare_grad
// 54, joined chunks 5, k_stable_grad 55, partial rows 5).
#include <type_traits>

#include "qb_norm_kernels.h"
#include "qb_token_sums.h"

namespace qb {

namespace {

constexpr int kStableParts = 512;        // workgroups of the gradient: two of 512 threads are all a CU holds

struct StableGradArgs {
    const void* dy;
    const float* chunk_part;
    const void* table;
    const void* gamma;
    void* dtable;
    float* part;
    int64_t pad;
    float scale, eps;
    int32_t wdt, ddt, accumulate;
};

// Work on single ids by a whole workgroup: TPR threads, unit k * TPR + tid in
// register k, the sums of dgamma and dbeta over the workgroup's ids.
template <int GDT, int TDT, int TPR, int VPT, int TAIL>
struct StableRows {
    const IdArgs& a;
    const StableGradArgs& p;
    float* slot;
    const int dim, units, tid;
    const RowShape<TPR, VPT> shape;
    float gam[VPT][8], accg[VPT][8] = {}, accb[VPT][8] = {};

    __device__ __forceinline__ StableRows(const IdArgs& a_, const StableGradArgs& p_, float* slot_)
        : a(a_), p(p_), slot(slot_), dim(a_.dim), units((a_.dim + 7) >> 3), tid(threadIdx.x),
          shape(threadIdx.x, a_.dim)
    {
        if (!p.gamma) {
#pragma unroll
            for (int k = 0; k < VPT; ++k)
#pragma unroll
                for (int j = 0; j < 8; ++j) gam[k][j] = 1.0f;
        } else if (p.wdt == DT_F32) {
            load_gamma<DT_F32>();
        } else {
            load_gamma<TDT>();
        }
    }

    template <int WDT>
    __device__ __forceinline__ void load_gamma()
    {
        Unit<WDT> u[VPT];
#pragma unroll
        for (int k = 0; k < VPT; ++k) u[k] = load_row_unit<WDT, TAIL, false>(p.gamma, k * TPR + tid, units, dim);
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) gam[k][j] = unit_at<WDT>(u[k], j);
    }

    __device__ __forceinline__ void load_table(Unit<TDT> (&w)[VPT], int64_t v)
    {
        const char* const row = static_cast<const char*>(p.table) + v * dim * elem_bytes(TDT);
#pragma unroll
        for (int k = 0; k < VPT; ++k) w[k] = load_row_unit<TDT, TAIL, true>(row, k * TPR + tid, units, dim);
    }

    // The id's row and its sum S_v: adds to dgamma and dbeta, writes dtable[v].
    __device__ __forceinline__ void finish(int64_t v, const Unit<TDT> (&w)[VPT], float (&sum)[VPT][8])
    {
        float x[VPT][8];
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[k][j] = unit_at<TDT>(w[k], j) * p.scale;
            if (!whole_step<TPR>(k, dim) && k * TPR + tid >= units) {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[k][j] = sum[k][j] = 0.0f;
            }
        }
        float mean, rstd;
        row_stats<TPR, VPT>(x, shape, tid, dim, p.eps, slot, &mean, &rstd);
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            // h is zero beyond the row, where (0 - mean) * rstd may overflow
            const bool whole = whole_step<TPR>(k, dim);
            const float rk = TAIL != kWhole || whole || k * TPR + tid < units ? rstd : 0.0f;
            const int cnt = unit_count(k * TPR + tid, dim);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float d = sum[k][j], g = d * gam[k][j];
                float h = (x[k][j] - mean) * rk;
                if (TAIL != kWhole && !whole) h = j < cnt ? h : 0.0f;
                sum[k][j] = g;
                x[k][j] = h;
                accg[k][j] = __builtin_fmaf(d, h, accg[k][j]);
                accb[k][j] += d;
                s1 += g;
                s2 = __builtin_fmaf(g, h, s2);
            }
        }
        row_sum2<TPR>(s1, s2, slot + row_slot_words(TPR));
        if (v == p.pad) return;                        // its row takes no gradient
        const float c1 = s1 * shape.inv_dim, c2 = s2 * shape.inv_dim, f = p.scale * rstd;
        char* const row = static_cast<char*>(p.dtable) + v * dim * (p.ddt == DT_F32 ? 4 : 2);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int unit = k * TPR + tid;
            float out[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) out[j] = f * (sum[k][j] - __builtin_fmaf(x[k][j], c2, c1));
            if (p.accumulate) add_row_unit_rt<TAIL>(p.ddt, row, unit, units, dim, out);
            store_row_unit_rt<TAIL, true>(p.ddt, row, unit, units, dim, out);
        }
    }

    __device__ __forceinline__ void load8f(const float* q, float (&v)[8])
    {
        const f32x4 lo = gld<f32x4>(q), hi = gld<f32x4>(q + 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = lo[j];
            v[4 + j] = hi[j];
        }
    }

    __device__ __forceinline__ void store8f(float* q, const float (&v)[8])
    {
        gst<f32x4>(q, f32x4{v[0], v[1], v[2], v[3]});
        gst<f32x4>(q + 4, f32x4{v[4], v[5], v[6], v[7]});
    }

    // The workgroup's partial sums.
    __device__ __forceinline__ void put_parts(int64_t wg)
    {
        const int64_t padded = (int64_t)units * 8;
        float* const out = p.part + wg * 2 * padded;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int unit = k * TPR + tid;
            if (unit >= units) continue;
            float* const q = out + (int64_t)unit * 8;
            store8f(q, accg[k]);
            store8f(q + padded, accb[k]);
        }
    }
};

// TPR threads (one workgroup) to a listed id; a workgroup walks the list by
// the grid, looks its next 64 ids up at once (lane l the l-th), and reads the
// next id's row and first token before it works on the current one.  Bound by the
// latency of an id's chain (row and token, two barriers, further tokens), at 54% of the
// vector ALU, and hidden no further because of the registers: 115 to 127 VGPRs let two
// workgroups of 512 threads reside on a CU, 512 in all; 768 or 1024 of them queue, and each
// leaves a partial row (136 to 140 us for the whole gradient against 133 then).  Ragged rows
// with binary32 dy take 129 to 143 VGPRs (rows of 2049 to 4096 elements: one workgroup a
// CU), with a binary32 table too 36 bytes a lane of scratch beyond 4096 elements; rows of
// 8193 to 16384 spill 152 to 348 bytes.  None of these is tuned.  (Two ids at a time, sharing the barriers, spilled or halved the resident workgroups: 60 to 65 us
// against 55 for 4300 ids of 4096 elements.)
template <int GDT, int TDT, int TPR, int VPT, int TAIL>
__global__ __launch_bounds__(TPR) void k_stable_grad(IdArgs a, OrderArgs o, StableGradArgs p)
{
    __shared__ float s_slot[2 * row_slot_words(TPR)];
    StableRows<GDT, TDT, TPR, VPT, TAIL> r(a, p, s_slot);
    const int lane = threadIdx.x % 64;
    const int64_t padded = (int64_t)r.units * 8;
    const int32_t count = o.count[0], step = (int32_t)gridDim.x;
    for (int64_t i0 = blockIdx.x; i0 < count; i0 += 64 * (int64_t)step) {
        const int64_t at = i0 + lane * (int64_t)step;
        int32_t id = 0, lo = 0, hi = 0, head = 0;
        if (at < count) {
            const u32x4 entry = gld<u32x4>(o.list + 4 * at);
            id = (int32_t)entry.x;
            lo = (int32_t)entry.y;
            hi = (int32_t)entry.z;
            head = (int32_t)entry.w;
        }
        const int todo = count - i0 > 63 * (int64_t)step ? 64 : (int)((count - i0 + step - 1) / step);
        Unit<TDT> wnext[VPT];
        Unit<GDT> dnext[VPT];
        auto load_next = [&](int i) {
            r.load_table(wnext, __builtin_amdgcn_readlane(id, i));
            const char* const row =
                static_cast<const char*>(p.dy) + (int64_t)__builtin_amdgcn_readlane(head, i) * r.dim * elem_bytes(GDT);
#pragma unroll
            for (int k = 0; k < VPT; ++k)
                dnext[k] = load_row_unit<GDT, TAIL, true>(row, k * TPR + r.tid, r.units, r.dim);
        };
        load_next(0);
        for (int i = 0; i < todo; ++i) {
            const int64_t v = __builtin_amdgcn_readlane(id, i);
            const int32_t first = __builtin_amdgcn_readlane(lo, i), last = __builtin_amdgcn_readlane(hi, i);
            Unit<TDT> w[VPT];
            float sum[VPT][8];
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                w[k] = wnext[k];
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[k][j] = unit_at<GDT>(dnext[k], j);
            }
            if (i + 1 < todo) load_next(i + 1);
            // S_v
            if (last - first > o.chunk) {              // joined before, in the slot of its first chunk
                const float* const q = p.chunk_part + chunk_slot(first / o.chunk, first, o.chunk) * padded;
#pragma unroll
                for (int k = 0; k < VPT; ++k)
                    r.load8f(q + (int64_t)(k * TPR + r.tid < r.units ? k * TPR + r.tid : 0) * 8, sum[k]);
            } else {
                sum_tokens<GDT, TAIL, TPR, VPT, 4>(o.order, first + 1, last, p.dy, r.tid, r.units, r.dim, sum);
            }
            r.finish(v, w, sum);
        }
    }
    r.put_parts(blockIdx.x);
}

// Few tokens: workgroup t works if token t is the first of its id, and writes
// partial sums in any case; workgroups beyond the tokens' write zero rows.
template <int GDT, int TDT, int TPR, int VPT, int TAIL>
__global__ __launch_bounds__(TPR) void k_stable_grad_direct(IdArgs a, StableGradArgs p)
{
    __shared__ float s_slot[2 * row_slot_words(TPR)];
    const DirectIds ids(a);
    if (blockIdx.x >= a.n) {
        zero_unnamed<TAIL, TPR>(a, ids, (blockIdx.x - a.n) * kZeroRows, p.pad, p.dtable, p.ddt);
        return;
    }
    StableRows<GDT, TDT, TPR, VPT, TAIL> r(a, p, s_slot);
    const int t = (int)blockIdx.x;
    const int32_t v = ids.of(t);
    const unsigned long long m0 = ids.tokens(0, v), m1 = ids.tokens(1, v);
    if (v >= 0 && (m0 ? __builtin_ctzll(m0) : 64 + __builtin_ctzll(m1)) == t) {
        Unit<TDT> w[VPT];
        r.load_table(w, v);
        float sum[VPT][8] = {};
        sum_masked<GDT, TAIL, TPR, VPT, 4>(m0, 0, p.dy, r.tid, r.units, r.dim, sum);
        sum_masked<GDT, TAIL, TPR, VPT, 4>(m1, 1, p.dy, r.tid, r.units, r.dim, sum);
        r.finish(v, w, sum);
    }
    r.put_parts(t);
}

template <int GDT, int TDT, int TPR, int VPT, int TAIL>
hipError_t stable_grad_tpr(const IdArgs& a, const OrderArgs* o, const StableGradArgs& p, int parts, hipStream_t s)
{
    if (!o)
        return launch_kernel_nt(k_stable_grad_direct<GDT, TDT, TPR, VPT, TAIL>,
                                (int)(a.n + direct_zero_wgs(a.rows, p.accumulate != 0)), TPR, s, a, p);
    return launch_kernel_nt(k_stable_grad<GDT, TDT, TPR, VPT, TAIL>, parts, TPR, s, a, *o, p);
}

// One unit per thread up to 8192 elements: a workgroup of many waves hides the
// latency of its reads with the few registers of each.  o nullptr: few tokens.
template <int GDT, int TDT, int TAIL>
hipError_t stable_grad_as(const IdArgs& a, const OrderArgs* o, const StableGradArgs& p, int parts, hipStream_t s)
{
    const int units = (a.dim + 7) / 8;
    if (units <= 64) return stable_grad_tpr<GDT, TDT, 64, 1, TAIL>(a, o, p, parts, s);
    if constexpr (TAIL != kShort) {
        if (units <= 256) return stable_grad_tpr<GDT, TDT, 256, 1, TAIL>(a, o, p, parts, s);
        if (units <= 512) return stable_grad_tpr<GDT, TDT, 512, 1, TAIL>(a, o, p, parts, s);
        if (units <= 1024) return stable_grad_tpr<GDT, TDT, 1024, 1, TAIL>(a, o, p, parts, s);
        if (units <= 2048) return stable_grad_tpr<GDT, TDT, 1024, 2, TAIL>(a, o, p, parts, s);
    }
    return hipErrorInvalidValue;
}

template <int GDT>
hipError_t stable_grad_t(const IdArgs& a, const OrderArgs* o, const StableGradArgs& p, int parts, int tdt,
                         hipStream_t s)
{
    auto with = [&](auto tdt_c) {
        constexpr int TDT = decltype(tdt_c)::value;
        const int tail = tail_of(a.dim);
        return tail == kWhole     ? stable_grad_as<GDT, TDT, kWhole>(a, o, p, parts, s)
               : tail == kPartial ? stable_grad_as<GDT, TDT, kPartial>(a, o, p, parts, s)
                                  : stable_grad_as<GDT, TDT, kShort>(a, o, p, parts, s);
    };
    if (tdt == DT_F32) return with(std::integral_constant<int, DT_F32>{});
    if (tdt == DT_F16) return with(std::integral_constant<int, DT_F16>{});
    return with(std::integral_constant<int, DT_BF16>{});
}

}  // namespace

// No more workgroups than ids that can have tokens; one per token where these are few.
int stable_parts(int64_t n, int64_t rows)
{
    if (takes_direct(n, rows)) return rows > 0 ? (int)n : 0;
    const int64_t most = n < rows ? n : rows;
    return (int)(most < kStableParts ? most : kStableParts);
}

template <typename... Args>
static hipError_t stable_grad_g(int gdt, Args... args)
{
    if (gdt == DT_F32) return stable_grad_t<DT_F32>(args...);
    if (gdt == DT_F16) return stable_grad_t<DT_F16>(args...);
    return stable_grad_t<DT_BF16>(args...);
}

hipError_t launch_stable_grad(const IdArgs& a, const OrderArgs& o, const void* dy, int gdt, const float* chunk_part,
                              const void* table, int tdt, float scale, const NormArgs& w, int64_t pad,
                              bool accumulate, void* dtable, int ddt, float* part, int parts, hipStream_t s)
{
    if (parts == 0) return hipSuccess;
    const StableGradArgs p{dy, chunk_part, table, w.gamma, dtable, part, pad, scale, w.eps,
                           w.wdt, ddt, accumulate ? 1 : 0};
    return stable_grad_g(gdt, a, &o, p, parts, tdt, s);
}

hipError_t launch_stable_grad_direct(const IdArgs& a, const void* dy, int gdt, const void* table, int tdt, float scale,
                                     const NormArgs& w, int64_t pad, bool accumulate, void* dtable, int ddt,
                                     float* part, hipStream_t s)
{
    const StableGradArgs p{dy, nullptr, table, w.gamma, dtable, part, pad, scale, w.eps, w.wdt, ddt, accumulate ? 1 : 0};
    return stable_grad_g(gdt, a, (const OrderArgs*)nullptr, p, (int)a.n, tdt, s);
}

}  // namespace qb
