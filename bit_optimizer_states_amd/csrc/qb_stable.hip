// qb_stable.hip -- the stable embedding: layer norm of an embedding's rows in one
// kernel (k_norm's gathering form).  Its gradients: qb_stable_grad.hip.
#include "qb_norm_kernels.h"

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

}  // namespace

hipError_t launch_stable_embedding(const IdArgs& a, const void* table, int tdt, float scale, const NormArgs& w,
                                   void* y, int ydt, hipStream_t s)
{
    if (tdt == DT_F32) return stable_y<DT_F32>(a, table, scale, w, y, ydt, s);
    if (tdt == DT_F16) return stable_y<DT_F16>(a, table, scale, w, y, ydt, s);
    return stable_y<DT_BF16>(a, table, scale, w, y, ydt, s);
}

}  // namespace qb
