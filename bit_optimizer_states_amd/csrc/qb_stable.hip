// qb_stable.hip -- the stable embedding: layer norm of an embedding's rows, in
// one kernel forward, and its gradients.
//
// Backward.  All tokens of one id v share the row x = scale * W[v] and with it
// mean, rstd and h = (x - mean) * rstd, and the layer norm's gradient is linear in
// dy.  With S_v = sum of dy_t over the tokens of v and g = S_v * gamma:
//   dW[v]  = scale * rstd * (g - mean(g) - h * mean(g h)),
//   dgamma = sum_v S_v h,  dbeta = sum_v S_v.
// So dy is read once and summed by id first, every used row of W is read once,
// the norm's backward pass runs once per used id instead of once per token, and
// no [tokens, dim] intermediate is written: the bytes are those of the plain
// embedding's gradient plus the used rows of W.
#include "qb_norm_kernels.h"
#include "qb_token_sums.h"

namespace qb {

namespace {

template <int TDT, int YDT>
hipError_t stable_as(const IdArgs& a, const void* table, float scale, const NormArgs& w, void* y, hipStream_t s)
{
    if (w.wdt == DT_F32) return norm_dim<TDT, YDT, DT_F32, true>(table, a, scale, w, y, nullptr, nullptr, s);
    if (w.wdt != TDT) return hipErrorInvalidValue;
    return norm_dim<TDT, YDT, TDT, true>(table, a, scale, w, y, nullptr, nullptr, s);
}

template <int TDT>
hipError_t stable_y(const IdArgs& a, const void* table, float scale, const NormArgs& w, void* y, int ydt,
                    hipStream_t s)
{
    if (ydt == DT_F32) return stable_as<TDT, DT_F32>(a, table, scale, w, y, s);
    if (ydt == DT_F16) return stable_as<TDT, DT_F16>(a, table, scale, w, y, s);
    return stable_as<TDT, DT_BF16>(a, table, scale, w, y, s);
}

// Rows per zero-filling workgroup.
constexpr int kZeroRows = 16;

struct StableGradArgs {
    const void* dy;
    const float* chunk_part;
    const void* table;
    const void* gamma;
    void* dtable;
    float* part;
    int64_t pad;
    float scale, eps;
    int32_t chunk, wdt, ddt, accumulate, parts;
};

// The first `parts` workgroups take the ids that have tokens, TPR threads to a
// row: workgroup p the classes p, p + parts, ... (or, with more workgroups than
// classes, every (parts / classes)-th used id of class p % classes), so frequent
// ids, which have neighbouring numbers, are spread over workgroups.  The
// others write the zero rows of ids without tokens, kZeroRows each (none of
// these with accumulate).
template <int GDT, int TDT, int TPR, int VPT, bool TAIL>
__global__ __launch_bounds__(TPR) void k_stable_grad(IdArgs a, OrderArgs o, StableGradArgs p)
{
    const int dim = a.dim, units = (dim + 7) >> 3;
    const int64_t padded = (int64_t)units * 8;
    const int tid = threadIdx.x;
    const int ddt_bytes = p.ddt == DT_F32 ? 4 : 2;
    if ((int)blockIdx.x >= p.parts) {
        const int64_t v0 = ((int64_t)blockIdx.x - p.parts) * kZeroRows;
        const float zero[8] = {};
        for (int i = 0; i < kZeroRows && v0 + i < a.rows; ++i) {
            const int64_t s = slot_of(v0 + i, o);
            if (o.start[s] != o.start[s + 1]) continue;
            char* const row = static_cast<char*>(p.dtable) + (v0 + i) * dim * ddt_bytes;
            for (int unit = tid; unit < units; unit += TPR)
                store_row_unit_rt<TAIL, true>(p.ddt, row, unit, units, dim, zero);
        }
        return;
    }

    __shared__ float s_slot[2 * row_slot_words(TPR)];
    float gam[VPT][8], accg[VPT][8] = {}, accb[VPT][8] = {};
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = (k * TPR + tid) * 8 + j;
            gam[k][j] = c >= dim ? 0.0f : p.gamma ? load1_rt(p.wdt, p.gamma, c) : 1.0f;
        }

    const int32_t classes = 1 << o.log2g;
    const int32_t share = p.parts > classes ? p.parts / classes : 1;         // workgroups per class
    const int32_t step = p.parts > classes ? classes : p.parts;
    const int32_t turn = (int32_t)blockIdx.x / step;
    for (int32_t cls = (int32_t)blockIdx.x % step; cls < classes && turn < share; cls += step) {
        const int32_t* const start = o.start + (int64_t)cls * o.per;
        int32_t seen = 0;
        for (int32_t e0 = 0; e0 < o.per; e0 += 64) {
            const int32_t e = e0 + tid % 64;
            const int32_t lo = e < o.per ? gld<int32_t>(start + e) : 0, hi = e < o.per ? gld<int32_t>(start + e + 1) : 0;
            unsigned long long used = __ballot(lo != hi);
            while (used) {
                const int lead = __builtin_ctzll(used);
                used &= used - 1;
                if (seen++ % share != turn) continue;
                const int32_t first = __builtin_amdgcn_readlane(lo, lead), last = __builtin_amdgcn_readlane(hi, lead);
                const int64_t v = ((int64_t)(e0 + lead) << o.log2g) + cls;

                // the id's row and the statistics of its norm
                float x[VPT][8];
                const char* const wrow = static_cast<const char*>(p.table) + v * dim * elem_bytes(TDT);
                Unit<TDT> wu[VPT];
#pragma unroll
                for (int k = 0; k < VPT; ++k)
                    wu[k] = load_row_unit<TDT, TAIL, true>(wrow, k * TPR + tid, units, dim);
                // S_v
                float sum[VPT][8] = {};
#pragma unroll
                for (int k = 0; k < VPT; ++k) {
                    if (last - first > p.chunk)
                        sum_chunks<4>(p.chunk_part, p.chunk, first, last, k * TPR + tid, units, padded, sum[k]);
                    else
                        sum_tokens<GDT, TAIL, 4>(o.order, first, last, p.dy, k * TPR + tid, units, dim, sum[k]);
                }
#pragma unroll
                for (int k = 0; k < VPT; ++k)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        x[k][j] = k * TPR + tid < units ? unit_at<TDT>(wu[k], j) * p.scale : 0.0f;
                float mean, rstd;
                row_stats<TPR, VPT>(x, tid, dim, p.eps, s_slot, &mean, &rstd);

                float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
                for (int k = 0; k < VPT; ++k)
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float d = k * TPR + tid < units ? sum[k][j] : 0.0f;
                        const float h = (x[k][j] - mean) * rstd, g = d * gam[k][j];
                        sum[k][j] = g;
                        x[k][j] = h;
                        accg[k][j] = __builtin_fmaf(d, h, accg[k][j]);
                        accb[k][j] += d;
                        s1 += g;
                        s2 = __builtin_fmaf(g, h, s2);
                    }
                row_sum2<TPR>(s1, s2, s_slot + row_slot_words(TPR));
                const float c1 = s1 / (float)dim, c2 = s2 / (float)dim, f = v == p.pad ? 0.0f : p.scale * rstd;
                if (p.accumulate && v == p.pad) continue;
                char* const row = static_cast<char*>(p.dtable) + v * dim * ddt_bytes;
#pragma unroll
                for (int k = 0; k < VPT; ++k) {
                    const int unit = k * TPR + tid;
                    float out[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        out[j] = v == p.pad ? 0.0f : f * (sum[k][j] - __builtin_fmaf(x[k][j], c2, c1));
                    if (p.accumulate) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (j < unit_count(unit, dim)) out[j] += load1_rt(p.ddt, row, (int64_t)unit * 8 + j);
                    }
                    store_row_unit_rt<TAIL, true>(p.ddt, row, unit, units, dim, out);
                }
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
hipError_t stable_grad_as(const IdArgs& a, const OrderArgs& o, const StableGradArgs& p, hipStream_t s)
{
    const int units = (a.dim + 7) / 8;
    const int64_t grid = p.parts + (p.accumulate ? 0 : (a.rows + kZeroRows - 1) / kZeroRows);
    if (grid >= (int64_t(1) << 23)) return hipErrorInvalidValue;
    auto go = [&](auto kernel, int threads) { return launch_kernel_nt(kernel, (int)grid, threads, s, a, o, p); };
    if (units <= 64) return go(k_stable_grad<GDT, TDT, 64, 1, TAIL>, 64);
    if (units <= 256) return go(k_stable_grad<GDT, TDT, 256, 1, TAIL>, 256);
    if (units <= 512) return go(k_stable_grad<GDT, TDT, 256, 2, TAIL>, 256);
    if (units <= 1024) return go(k_stable_grad<GDT, TDT, 512, 2, TAIL>, 512);
    if (units <= 2048) return go(k_stable_grad<GDT, TDT, 1024, 2, TAIL>, 1024);
    return hipErrorInvalidValue;
}

template <int GDT>
hipError_t stable_grad_t(const IdArgs& a, const OrderArgs& o, const StableGradArgs& p, int tdt, hipStream_t s)
{
    const bool tail = a.dim % 8 != 0;
    if (tdt == DT_F32) return tail ? stable_grad_as<GDT, DT_F32, true>(a, o, p, s) : stable_grad_as<GDT, DT_F32, false>(a, o, p, s);
    if (tdt == DT_F16) return tail ? stable_grad_as<GDT, DT_F16, true>(a, o, p, s) : stable_grad_as<GDT, DT_F16, false>(a, o, p, s);
    return tail ? stable_grad_as<GDT, DT_BF16, true>(a, o, p, s) : stable_grad_as<GDT, DT_BF16, false>(a, o, p, s);
}

}  // namespace

hipError_t launch_stable_embedding(const IdArgs& a, const void* table, int tdt, float scale, const NormArgs& w,
                                   void* y, int ydt, hipStream_t s)
{
    if (tdt == DT_F32) return stable_y<DT_F32>(a, table, scale, w, y, ydt, s);
    if (tdt == DT_F16) return stable_y<DT_F16>(a, table, scale, w, y, ydt, s);
    return stable_y<DT_BF16>(a, table, scale, w, y, ydt, s);
}

// Two workgroups per class where there are enough tokens to occupy them; no
// more than there are tokens or classes of ids.
int stable_parts(int64_t n, int64_t rows)
{
    const int64_t classes = int64_t(1) << order_log2g(rows);
    const int64_t most = 2 * classes < kNormPartsMax ? 2 * classes : kNormPartsMax;
    const int64_t g = classes < kNormPartsMax && n <= classes ? classes : most;
    return (int)(rows == 0 ? 0 : g);
}

hipError_t launch_stable_grad(const IdArgs& a, const OrderArgs& o, const void* dy, int gdt, const float* chunk_part,
                              const void* table, int tdt, float scale, const NormArgs& w, int64_t pad,
                              bool accumulate, void* dtable, int ddt, float* part, int parts, hipStream_t s)
{
    const StableGradArgs p{dy, chunk_part, table, w.gamma, dtable, part, pad, scale, w.eps,
                           chunk_tokens(a.n), w.wdt, ddt, accumulate ? 1 : 0, parts};
    if (gdt == DT_F32) return stable_grad_t<DT_F32>(a, o, p, tdt, s);
    if (gdt == DT_F16) return stable_grad_t<DT_F16>(a, o, p, tdt, s);
    return stable_grad_t<DT_BF16>(a, o, p, tdt, s);
}

}  // namespace qb
