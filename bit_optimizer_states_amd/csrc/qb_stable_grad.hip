// qb_stable_grad.hip -- the gradients of the stable embedding (layer norm of an
// embedding's rows).
//
// All tokens of one id v share the row x = scale * W[v] and with it mean, rstd and h = (x - mean) * rstd, and the layer norm's gradient is linear in
// dy.  With S_v = sum of dy_t over the tokens of v and g = S_v * gamma:
//   dW[v]  = scale * rstd * (g - mean(g) - h * mean(g h)),
//   dgamma = sum_v S_v h,  dbeta = sum_v S_v.
// So dy is read once and summed by id first, every used row of W is read once,
// the norm's backward pass runs once per used id instead of once per token, and
// no [tokens, dim] intermediate is written: the bytes are those of the plain
// embedding's gradient plus the used rows of W.
#include <type_traits>

#include "qb_norm_kernels.h"
#include "qb_token_sums.h"

namespace qb {

namespace {

constexpr int kStableParts = 512;        // workgroups of the gradient, two per CU

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

// TPR threads (one workgroup) to a listed id; a workgroup walks the list by
// the grid, looks its next 64 ids up at once (lane l the l-th), and reads the
// next id's row and first token before it works on the current one.
template <int GDT, int TDT, int TPR, int VPT, bool TAIL>
__global__ __launch_bounds__(TPR) void k_stable_grad(IdArgs a, OrderArgs o, StableGradArgs p)
{
    __shared__ float s_slot[2 * row_slot_words(TPR)];
    const int dim = a.dim, units = (dim + 7) >> 3;
    const int64_t padded = (int64_t)units * 8;
    const int tid = threadIdx.x, lane = tid % 64;
    const int32_t count = o.count[0], step = (int32_t)gridDim.x;
    float gam[VPT][8], accg[VPT][8] = {}, accb[VPT][8] = {};
    auto load_gamma = [&](auto wdt) {
        constexpr int WDT = decltype(wdt)::value;
        Unit<WDT> u[VPT];
#pragma unroll
        for (int k = 0; k < VPT; ++k) u[k] = load_row_unit<WDT, TAIL, false>(p.gamma, k * TPR + tid, units, dim);
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) gam[k][j] = unit_at<WDT>(u[k], j);
    };
    if (!p.gamma) {
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) gam[k][j] = 1.0f;
    } else if (p.wdt == DT_F32) {
        load_gamma(std::integral_constant<int, DT_F32>{});
    } else {
        load_gamma(std::integral_constant<int, TDT>{});
    }

    const RowShape<TPR, VPT> shape(tid, dim);
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
        // an id's row and its first token's dy
        auto load_next = [&](int i) {
            const char* const wrow =
                static_cast<const char*>(p.table) + (int64_t)__builtin_amdgcn_readlane(id, i) * dim * elem_bytes(TDT);
            const char* const drow =
                static_cast<const char*>(p.dy) + (int64_t)__builtin_amdgcn_readlane(head, i) * dim * elem_bytes(GDT);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                wnext[k] = load_row_unit<TDT, TAIL, true>(wrow, k * TPR + tid, units, dim);
                dnext[k] = load_row_unit<GDT, TAIL, true>(drow, k * TPR + tid, units, dim);
            }
        };
        load_next(0);
        for (int i = 0; i < todo; ++i) {
            const int64_t v = __builtin_amdgcn_readlane(id, i);
            const int32_t first = __builtin_amdgcn_readlane(lo, i), last = __builtin_amdgcn_readlane(hi, i);
            Unit<TDT> wu[VPT];
            float sum[VPT][8];
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                wu[k] = wnext[k];
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[k][j] = unit_at<GDT>(dnext[k], j);
            }
            if (i + 1 < todo) load_next(i + 1);
            // S_v
            if (last - first > o.chunk) {              // joined before, in the slot of its first chunk
                const float* const q = p.chunk_part + chunk_slot(first / o.chunk, first, o.chunk) * padded;
#pragma unroll
                for (int k = 0; k < VPT; ++k) {
                    const int64_t c = (int64_t)(k * TPR + tid < units ? k * TPR + tid : 0) * 8;
                    const f32x4 lo4 = gld<f32x4>(q + c), hi4 = gld<f32x4>(q + c + 4);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        sum[k][j] = lo4[j];
                        sum[k][4 + j] = hi4[j];
                    }
                }
            } else {
                sum_tokens<GDT, TAIL, TPR, VPT, 4>(o.order, first + 1, last, p.dy, tid, units, dim, sum);
            }
            // the statistics of its norm
            float x[VPT][8];
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[k][j] = unit_at<TDT>(wu[k], j) * p.scale;
                if (!whole_step<TPR>(k, dim) && k * TPR + tid >= units) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[k][j] = sum[k][j] = 0.0f;
                }
            }
            float mean, rstd;
            row_stats<TPR, VPT, TDT == DT_F32>(x, shape, tid, dim, p.eps, s_slot, &mean, &rstd);

            float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
            for (int k = 0; k < VPT; ++k)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float d = sum[k][j];
                    const float h = (x[k][j] - mean) * rstd, g = d * gam[k][j];
                    sum[k][j] = g;
                    x[k][j] = h;
                    accg[k][j] = __builtin_fmaf(d, h, accg[k][j]);
                    accb[k][j] += d;
                    s1 += g;
                    s2 = __builtin_fmaf(g, h, s2);
                }
            row_sum2<TPR>(s1, s2, s_slot + row_slot_words(TPR));
            if (v == p.pad) continue;                  // its row takes no gradient
            const float c1 = s1 * shape.inv_dim, c2 = s2 * shape.inv_dim, f = p.scale * rstd;
            char* const row = static_cast<char*>(p.dtable) + v * dim * (p.ddt == DT_F32 ? 4 : 2);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int unit = k * TPR + tid;
                float out[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) out[j] = f * (sum[k][j] - __builtin_fmaf(x[k][j], c2, c1));
                if (p.accumulate) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j < unit_count(unit, dim)) out[j] += load1_rt(p.ddt, row, (int64_t)unit * 8 + j);
                }
                store_row_unit_rt<TAIL, true>(p.ddt, row, unit, units, dim, out);
            }
        }
    }
    float* const out = p.part + (int64_t)blockIdx.x * 2 * padded;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int unit = k * TPR + tid;
        if (unit < units) {
            float* const q = out + (int64_t)unit * 8;
            gst<f32x4>(q, f32x4{accg[k][0], accg[k][1], accg[k][2], accg[k][3]});
            gst<f32x4>(q + 4, f32x4{accg[k][4], accg[k][5], accg[k][6], accg[k][7]});
            gst<f32x4>(q + padded, f32x4{accb[k][0], accb[k][1], accb[k][2], accb[k][3]});
            gst<f32x4>(q + padded + 4, f32x4{accb[k][4], accb[k][5], accb[k][6], accb[k][7]});
        }
    }
}

template <int GDT, int TDT, bool TAIL>
hipError_t stable_grad_as(const IdArgs& a, const OrderArgs& o, const StableGradArgs& p, int parts, hipStream_t s)
{
    const int units = (a.dim + 7) / 8;
    auto go = [&](auto kernel, int threads) { return launch_kernel_nt(kernel, parts, threads, s, a, o, p); };
    if (units <= 64) return go(k_stable_grad<GDT, TDT, 64, 1, TAIL>, 64);
    if (units <= 256) return go(k_stable_grad<GDT, TDT, 256, 1, TAIL>, 256);
    if (units <= 512) return go(k_stable_grad<GDT, TDT, 512, 1, TAIL>, 512);
    if (units <= 1024) return go(k_stable_grad<GDT, TDT, 1024, 1, TAIL>, 1024);
    if (units <= 2048) return go(k_stable_grad<GDT, TDT, 1024, 2, TAIL>, 1024);
    return hipErrorInvalidValue;
}

template <int GDT>
hipError_t stable_grad_t(const IdArgs& a, const OrderArgs& o, const StableGradArgs& p, int parts, int tdt,
                         hipStream_t s)
{
    if (a.dim % 8) {
        if (tdt == DT_F32) return stable_grad_as<GDT, DT_F32, true>(a, o, p, parts, s);
        if (tdt == DT_F16) return stable_grad_as<GDT, DT_F16, true>(a, o, p, parts, s);
        return stable_grad_as<GDT, DT_BF16, true>(a, o, p, parts, s);
    }
    if (tdt == DT_F32) return stable_grad_as<GDT, DT_F32, false>(a, o, p, parts, s);
    if (tdt == DT_F16) return stable_grad_as<GDT, DT_F16, false>(a, o, p, parts, s);
    return stable_grad_as<GDT, DT_BF16, false>(a, o, p, parts, s);
}

}  // namespace

// No more workgroups than ids that can have tokens.
int stable_parts(int64_t n, int64_t rows)
{
    const int64_t most = n < rows ? n : rows;
    return (int)(most < kStableParts ? most : kStableParts);
}

hipError_t launch_stable_grad(const IdArgs& a, const OrderArgs& o, const void* dy, int gdt, const float* chunk_part,
                              const void* table, int tdt, float scale, const NormArgs& w, int64_t pad,
                              bool accumulate, void* dtable, int ddt, float* part, int parts, hipStream_t s)
{
    if (parts == 0) return hipSuccess;
    const StableGradArgs p{dy, chunk_part, table, w.gamma, dtable, part, pad, scale, w.eps,
                           w.wdt, ddt, accumulate ? 1 : 0};
    if (gdt == DT_F32) return stable_grad_t<DT_F32>(a, o, p, parts, tdt, s);
    if (gdt == DT_F16) return stable_grad_t<DT_F16>(a, o, p, parts, tdt, s);
    return stable_grad_t<DT_BF16>(a, o, p, parts, tdt, s);
}

}  // namespace qb
