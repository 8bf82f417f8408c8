// qb_embedding.hip -- embedding lookup from dense and from quantized tables, and
// the gradient of the table by sorted tokens.
//
// Lookup: y_t = scale * W[id_t], one binary32 multiply and one rounding.  Bound
// by HBM: the rows that are used are read, y is written.
//
// Gradient: dW[v] = scale * (sum of dy_t over the tokens t with id_t = v), in
// three launches (four for large tables).  The tokens are ordered by id (k_order), so that every sum is
// taken in ascending order of the tokens: no atomics on floating-point values,
// the same bits on every run.  Then every wave streams one chunk of the ordered
// tokens: it writes the rows of the ids that begin there, and a partial row for an
// id that has more tokens than a chunk; the same launch writes the zero rows of the
// table (k_table_grad).  The last launch adds the partial rows (k_long_rows).
// Up to 128 tokens take one launch without ordering (k_table_grad_direct).  The
// stable embedding's gradient shares the ordering and prepares its sums of long ids
// and its zero rows with k_prepare_grad and k_join_chunks.
#include <type_traits>

#include "qb_token_sums.h"

namespace qb {

namespace {

// ---------------------------------------------------------------------------
// lookup
// ---------------------------------------------------------------------------

// `lanes` (a power of two) threads share a token, 256 / lanes tokens a workgroup;
// the id is the only read that others wait for.  Bound by HBM: 16384 tokens of
// natural frequencies from [32000, 4096] binary32 to bf16 in 44 us (134 MB of output and
// the 90 MB of rows that are used: 5.0 TB/s); 16 tokens 2.6 us, the latency of two
// dependent reads.
template <int TDT, int YDT, int TAIL>
__global__ __launch_bounds__(256) void k_embedding(IdArgs a, const void* __restrict__ table, float scale,
                                                   void* __restrict__ y, int log2lanes)
{
    const int lane = threadIdx.x & ((1 << log2lanes) - 1);
    const int64_t t = ((int64_t)blockIdx.x << (8 - log2lanes)) + (threadIdx.x >> log2lanes);
    if (t >= a.n) return;
    const int dim = a.dim, units = (dim + 7) >> 3;
    const int64_t id = load_id(a.ids, a.id64, t);
    const bool found = (uint64_t)id < (uint64_t)a.rows;
    const char* const row = static_cast<const char*>(table) + (found ? id : 0) * dim * elem_bytes(TDT);
    char* const yrow = static_cast<char*>(y) + t * dim * elem_bytes(YDT);
    const int step = 1 << log2lanes;
    for (int unit = lane; unit < units; unit += 2 * step) {
        float o[2][8] = {};
        if (found) {
            Unit<TDT> u[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) u[q] = load_row_unit<TDT, TAIL, false>(row, unit + q * step, units, dim);
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int j = 0; j < 8; ++j) o[q][j] = unit_at<TDT>(u[q], j) * scale;
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) store_row_unit<YDT, TAIL, true>(yrow, unit + q * step, units, dim, o[q]);
    }
}

// Threads that share a token: enough for one unit each, at most a workgroup.
int lanes_log2(int units)
{
    int k = 3;
    while (k < 8 && (1 << k) < units) ++k;
    return k;
}

template <int TDT, int YDT>
hipError_t embedding_as(const IdArgs& a, const void* table, float scale, void* y, hipStream_t s)
{
    const int k = lanes_log2((a.dim + 7) / 8);
    return launch_rows(a.n, 256 >> k, [&](int64_t t0, int64_t m, int grid) {
        const IdArgs b = ids_from(a, t0, m);
        void* const out = static_cast<char*>(y) + t0 * a.dim * elem_bytes(YDT);
        auto go = [&](auto kernel) { return launch_kernel(kernel, grid, s, b, table, scale, out, k); };
        const int tail = tail_of(a.dim);
        return tail == kWhole     ? go(k_embedding<TDT, YDT, kWhole>)
               : tail == kPartial ? go(k_embedding<TDT, YDT, kPartial>)
                                  : go(k_embedding<TDT, YDT, kShort>);
    });
}

template <int TDT>
hipError_t embedding_y(const IdArgs& a, const void* table, float scale, void* y, int ydt, hipStream_t s)
{
    if (ydt == DT_F32) return embedding_as<TDT, DT_F32>(a, table, scale, y, s);
    if (ydt == DT_F16) return embedding_as<TDT, DT_F16>(a, table, scale, y, s);
    return embedding_as<TDT, DT_BF16>(a, table, scale, y, s);
}

// ---------------------------------------------------------------------------
// lookup in a quantized table
// ---------------------------------------------------------------------------

// The table [rows, dim] is quantized as one flat tensor, so a block may span
// rows.  TAIL: dim is no multiple of 8, rows may begin inside a byte or a
// block, and every element finds its own code and block; otherwise a unit of 8
// elements is 4 or 8 aligned bytes of codes with one scale (blocks hold 64
// elements or more).  Bound by the writes of y: 16384 tokens of 4096, NF4 with nested
// constants to bf16, 24 us (5.6 TB/s of 134 MB); 32 tokens 3.3 us.
template <int BITS, int YDT, bool DQ, int TAIL>
__global__ __launch_bounds__(256) void k_dequant_embedding(IdArgs a, DequantDesc d, int log2B, int log2B2, int code4,
                                                           const QbTables* __restrict__ tab, float scale,
                                                           void* __restrict__ y, int log2lanes)
{
    __shared__ float s_val[BITS == 8 ? 256 : 16];
    __shared__ float s_dyn[DQ && BITS == 4 ? 256 : 1];
    if constexpr (BITS == 8) s_val[threadIdx.x] = tab->dyn8[threadIdx.x];
    else if (threadIdx.x < 16) s_val[threadIdx.x] = (code4 == 0 ? tab->nf4 : tab->fp4)[threadIdx.x];
    if constexpr (DQ && BITS == 4) s_dyn[threadIdx.x] = tab->dyn8[threadIdx.x];
    const float mu = DQ ? gld<float>(d.offset) : 0.0f;
    __syncthreads();

    const int lane = threadIdx.x & ((1 << log2lanes) - 1);
    const int64_t t = ((int64_t)blockIdx.x << (8 - log2lanes)) + (threadIdx.x >> log2lanes);
    if (t >= a.n) return;
    const int dim = a.dim, units = (dim + 7) >> 3;
    const int64_t id = load_id(a.ids, a.id64, t);
    const bool found = (uint64_t)id < (uint64_t)a.rows;
    const int64_t first = (found ? id : 0) * dim;
    char* const yrow = static_cast<char*>(y) + t * dim * elem_bytes(YDT);
    auto block_scale = [&](int64_t b) -> float {
        if constexpr (DQ) {
            const float c = (BITS == 8 ? s_val : s_dyn)[gld<uint8_t>(d.c2 + b)];
            return c * gld<float>(d.absmax2 + (b >> log2B2)) + mu;
        } else {
            return gld<float>(d.absmax + b);
        }
    };
    for (int unit = lane; unit < units; unit += 1 << log2lanes) {
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = 0.0f;
        const int64_t e = first + (int64_t)unit * 8;
        if (found) {
            if constexpr (!TAIL) {
                const float sc = block_scale(e >> log2B);
                uint32_t w0, w1 = 0;
                if constexpr (BITS == 8) {
                    const u32x2 w = gld<u32x2>(d.codes + e);
                    w0 = w.x;
                    w1 = w.y;
                } else {
                    w0 = gld<uint32_t>(d.codes + (e >> 1));
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    uint32_t c;
                    if constexpr (BITS == 8) c = ((j < 4 ? w0 : w1) >> (8 * (j & 3))) & 0xFFu;
                    else c = (w0 >> (8 * (j >> 1) + ((j & 1) ? 0 : 4))) & 15u;      // element 2k in the high nibble
                    o[j] = s_val[c] * sc * scale;
                }
            } else {
                const int left = dim - unit * 8;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (j < left) {
                        const int64_t i = e + j;
                        uint32_t c;
                        if constexpr (BITS == 8) c = gld<uint8_t>(d.codes + i);
                        else c = (gld<uint8_t>(d.codes + (i >> 1)) >> ((i & 1) ? 0 : 4)) & 15u;
                        o[j] = s_val[c] * block_scale(i >> log2B) * scale;
                    }
                }
            }
        }
        store_row_unit<YDT, TAIL, true>(yrow, unit, units, dim, o);
    }
}

int log2_of(int v)
{
    int k = 0;
    while ((1 << k) < v) ++k;
    return k;
}

template <int BITS, int YDT, bool DQ>
hipError_t dequant_embedding_as(const IdArgs& a, const DequantDesc& d, int code4, int B, int B2, const QbTables* tab,
                                float scale, void* y, hipStream_t s)
{
    const int k = lanes_log2((a.dim + 7) / 8);
    return launch_rows(a.n, 256 >> k, [&](int64_t t0, int64_t m, int grid) {
        const IdArgs b = ids_from(a, t0, m);
        void* const out = static_cast<char*>(y) + t0 * a.dim * elem_bytes(YDT);
        return a.dim % 8 ? launch_kernel(k_dequant_embedding<BITS, YDT, DQ, true>, grid, s, b, d, log2_of(B),
                                         log2_of(B2), code4, tab, scale, out, k)
                         : launch_kernel(k_dequant_embedding<BITS, YDT, DQ, false>, grid, s, b, d, log2_of(B),
                                         log2_of(B2), code4, tab, scale, out, k);
    });
}

template <int BITS, bool DQ>
hipError_t dequant_embedding_y(const IdArgs& a, const DequantDesc& d, int code4, int B, int B2, const QbTables* tab,
                               float scale, void* y, int ydt, hipStream_t s)
{
    if (ydt == DT_F32) return dequant_embedding_as<BITS, DT_F32, DQ>(a, d, code4, B, B2, tab, scale, y, s);
    if (ydt == DT_F16) return dequant_embedding_as<BITS, DT_F16, DQ>(a, d, code4, B, B2, tab, scale, y, s);
    return dequant_embedding_as<BITS, DT_BF16, DQ>(a, d, code4, B, B2, tab, scale, y, s);
}

// ---------------------------------------------------------------------------
// order of the tokens by id
// ---------------------------------------------------------------------------

// One workgroup per class of ids (OrderArgs).  It goes through all n ids twice:
// the first time it counts its own entries, per wave (each wave owns one
// contiguous stretch of the tokens), and the tokens of lower classes, whose number
// is where its part of the list begins; the second time it places its tokens.  A wave
// takes the tokens of its stretch in order and gives equal ids of one step
// consecutive places by their lane, so the order is stable and no workgroup waits
// for another.  The ids are read from L2 by every workgroup, n * classes reads in
// exchange for one launch and no atomics in memory; up to 16384 tokens a wave
// keeps its stretch in registers for the second time.  Bound by the chain load -
// count - scan - place of one workgroup per CU, not by bytes: 16384 ids of 32000 in 12
// us, 5003 in 8 us.  (Writing the zero rows beside it does not pay: their place is
// known only after it, and zeros under rows that are written again later took it from
// 11 to 17 us and the whole call with it.)
//
// With parts (order_in_parts) the same steps run twice: over all tokens with ranges of
// classes in the place of classes (kDeal), then per class over its part's tokens
// (kInPart).
enum OrderStep { kAll, kDeal, kInPart };

template <bool ID64, OrderStep STEP>
__global__ __launch_bounds__(kOrderWaves * 64) void k_order(IdArgs a, OrderArgs o)
{
    extern __shared__ int32_t s_cnt[];                 // [kOrderWaves][per]
    __shared__ int32_t s_below[kOrderWaves], s_wave[kOrderWaves], s_used[2][kOrderWaves];
    constexpr int UN = 16;                             // loads in flight per lane
    const int wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    const int32_t cls = (int32_t)blockIdx.x, mask = (1 << o.log2g) - 1, per = STEP == kDeal ? 1 : o.per;
    const int32_t shift = o.log2g - kOrderPartBits;
    auto class_of = [&](int32_t id) { return STEP == kDeal ? (id & mask) >> shift : id & mask; };
    auto entry_of = [&](int32_t id) { return STEP == kDeal ? 0 : id >> o.log2g; };

    // the tokens gone through: all, or the part's
    const int64_t begin = STEP == kInPart ? o.part_start[cls >> shift] : 0;
    const int64_t end = STEP == kInPart ? o.part_start[(cls >> shift) + 1] : a.n;
    const int64_t stretch = ((end - begin + kOrderWaves - 1) / kOrderWaves + 63) / 64 * 64;
    const int64_t first = begin + wave * stretch;
    const int64_t last = first + stretch < end ? first + stretch : end;
    int32_t* const cnt = s_cnt + wave * per;
    // ids of the tokens t0 + k * 64 + lane; -1 beyond the stretch or outside the table
    int32_t id[UN];
    auto load_ids = [&](int64_t t0) {
        int64_t raw[UN];
#pragma unroll
        for (int k = 0; k < UN; ++k) {
            const int64_t t = t0 + k * 64 + lane;
            const int64_t at = t < last ? t : last - 1;
            if constexpr (STEP == kInPart) raw[k] = gld<int32_t>(o.part_id + at);
            else if constexpr (ID64) raw[k] = gld<int64_t>(static_cast<const int64_t*>(a.ids) + at);
            else raw[k] = gld<int32_t>(static_cast<const int32_t*>(a.ids) + at);
        }
#pragma unroll
        for (int k = 0; k < UN; ++k)
            id[k] = t0 + k * 64 + lane < last && (uint64_t)raw[k] < (uint64_t)a.rows ? (int32_t)raw[k] : -1;
    };
    const bool once = stretch <= 64 * UN;              // uniform: the stretch fits in registers
    if (once && first < last) load_ids(first);
    for (int i = threadIdx.x; i < kOrderWaves * per; i += kOrderWaves * 64) s_cnt[i] = 0;
    __syncthreads();

    int32_t below = 0;
    for (int64_t t0 = first; t0 < last; t0 += 64 * UN) {
        if (!once) load_ids(t0);
#pragma unroll
        for (int k = 0; k < UN; ++k) {
            if (k % 4 == 0 && t0 + k * 64 >= last) break;      // uniform: few tokens run little of this code
            if (id[k] >= 0) {
                const int32_t c = class_of(id[k]);
                below += c < cls ? 1 : 0;
                if (c == cls) atomicAdd(&cnt[entry_of(id[k])], 1);
            }
        }
    }
    for (int step = 1; step < 64; step *= 2) below += __shfl_xor(below, step);
    if (lane == 0) s_below[wave] = below;
    __syncthreads();

    // exclusive scan over the entries: thread j owns entry j (per <= kOrderPerMax)
    int32_t base = (int32_t)begin;
#pragma unroll
    for (int w = 0; w < kOrderWaves; ++w) base += s_below[w];
    const int j = threadIdx.x;
    int32_t total = 0, of_wave[kOrderWaves];
#pragma unroll
    for (int w = 0; w < kOrderWaves; ++w) {
        of_wave[w] = j < per ? s_cnt[w * per + j] : 0;
        total += of_wave[w];
    }
    int32_t incl = total;
    for (int step = 1; step < 64; step *= 2) {
        const int32_t up = __shfl_up(incl, step);
        if (lane >= step) incl += up;
    }
    const unsigned long long some = __ballot(total > 0), many = __ballot(total > o.chunk);
    if (lane == 63) {
        s_wave[wave] = incl;
        s_used[0][wave] = (int32_t)__popcll(some);
        s_used[1][wave] = (int32_t)__popcll(many);
    }
    __syncthreads();
    int32_t before = 0;
    for (int w = 0; w < wave; ++w) before += s_wave[w];
    if (j < per) {
        int32_t run = base + before + incl - total;
        int32_t* const start = (STEP == kDeal ? o.part_start : o.start) + (int64_t)cls * per;
        start[j] = run;
#pragma unroll
        for (int w = 0; w < kOrderWaves; ++w) {
            s_cnt[w * per + j] = run;
            run += of_wave[w];
        }
        if (cls == (int32_t)gridDim.x - 1 && j == per - 1) start[per] = run;
    }
    if (STEP != kDeal && cls == 0 && j == 0) o.count[1] = 0;       // k_table_grad counts long ids in it
    if (STEP != kDeal && j < 2) {
        int32_t used = 0;
        for (int w = 0; w < kOrderWaves; ++w) used += s_used[j][w];
        o.used[2 * (int64_t)cls + j] = used;
    }
    __syncthreads();

    for (int64_t t0 = first; t0 < last; t0 += 64 * UN) {
        if (!once) load_ids(t0);
#pragma unroll
        for (int k = 0; k < UN; ++k) {
            if (k % 4 == 0 && t0 + k * 64 >= last) break;
            const bool mine = id[k] >= 0 && class_of(id[k]) == cls;
            unsigned long long todo = __ballot(mine);
            while (todo) {
                const int lead = __builtin_ctzll(todo);
                const int32_t e = __builtin_amdgcn_readlane(id[k], lead);
                const bool equal = mine && (STEP == kDeal || id[k] == e);
                const unsigned long long same = __ballot(equal);
                int32_t at = 0;
                if (lane == lead) at = atomicAdd(&cnt[entry_of(e)], (int32_t)__popcll(same));
                at = __builtin_amdgcn_readlane(at, lead);
                if (equal) {
                    const int32_t p = at + (int32_t)__popcll(same & ((1ull << lane) - 1));
                    const int64_t t = t0 + k * 64 + lane;
                    (STEP == kDeal ? o.part_pos : o.order)[p] = STEP == kInPart ? gld<int32_t>(o.part_pos + t) : (int32_t)t;
                    (STEP == kDeal ? o.part_id : o.key)[p] = id[k];
                }
                todo &= ~same;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// gradient of the table
// ---------------------------------------------------------------------------

// The lists of used and of long ids: one wave per class, which begins where the
// lower classes' counts end.
__device__ __forceinline__ void list_used(const OrderArgs& o, int64_t cls)
{
    const int lane = threadIdx.x % 64;
    const int64_t classes = int64_t(1) << o.log2g;
    if (cls >= classes) return;
    int32_t base = 0, lbase = 0;
    for (int64_t c = lane; c < cls; c += 64) {
        const u32x2 u = gld<u32x2>(o.used + 2 * c);
        base += (int32_t)u.x;
        lbase += (int32_t)u.y;
    }
    for (int step = 1; step < 64; step *= 2) {
        base += __shfl_xor(base, step);
        lbase += __shfl_xor(lbase, step);
    }
    const int32_t* const start = o.start + cls * o.per;
    for (int32_t e0 = 0; e0 < o.per; e0 += 64) {
        const int32_t e = e0 + lane;
        const int32_t k = e < o.per ? gld<int32_t>(start + e + 1) - gld<int32_t>(start + e) : 0;
        const unsigned long long some = __ballot(k > 0), many = __ballot(k > o.chunk), below = (1ull << lane) - 1;
        const int32_t v = (int32_t)(((int64_t)e << o.log2g) + cls);
        if (k > 0) {
            const int32_t lo = gld<int32_t>(start + e);
            const u32x4 entry = {(uint32_t)v, (uint32_t)lo, (uint32_t)(lo + k), gld<uint32_t>(o.order + lo)};
            gst<u32x4>(o.list + 4 * ((int64_t)base + __popcll(some & below)), entry);
        }
        if (k > o.chunk) o.longs[lbase + __popcll(many & below)] = v;
        base += (int32_t)__popcll(some);
        lbase += (int32_t)__popcll(many);
    }
    if (cls == classes - 1 && lane == 0) {
        o.count[0] = base;
        o.count[1] = lbase;
    }
}

// One wave: a chunk's tokens, 64 units.  Only the first and the last id of a chunk
// can have more tokens than a chunk.
template <int GDT, int TAIL>
__device__ __forceinline__ void chunk_sums(const IdArgs& a, const OrderArgs& o, const void* dy, float* part,
                                           int64_t c, int unit)
{
    const int32_t chunk = o.chunk;
    const int32_t found = o.start[(int64_t(1) << o.log2g) * o.per];        // tokens inside the table
    if (c * chunk >= found) return;
    const int32_t b = (int32_t)(c * chunk), e = found - b < chunk ? found : b + chunk;
    const int dim = a.dim, units = (dim + 7) >> 3;
    const int64_t padded = (int64_t)units * 8;
    // both sides' look-ups at once: each is a chain of three dependent reads
    const int32_t t0 = o.order[b], t1 = o.order[e - 1];
    const int64_t id[2] = {load_id(a.ids, a.id64, t0), load_id(a.ids, a.id64, t1)};
    const int64_t s[2] = {slot_of(id[0], o), slot_of(id[1], o)};
    const int32_t lo[2] = {o.start[s[0]], o.start[s[1]]}, hi[2] = {o.start[s[0] + 1], o.start[s[1] + 1]};
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        if (side == 1 && id[1] == id[0]) break;
        const int32_t v0 = lo[side], v1 = hi[side];
        if (v1 - v0 <= chunk) continue;
        float sums[1][8] = {};
        sum_tokens<GDT, TAIL, 64, 1, 8>(o.order, v0 > b ? v0 : b, v1 < e ? v1 : e, dy, unit, units, dim, sums);
        if (unit < units) {
            float* const p = part + (2 * c + (v0 > b ? 1 : 0)) * padded + (int64_t)unit * 8;
            gst<f32x4>(p, f32x4{sums[0][0], sums[0][1], sums[0][2], sums[0][3]});
            gst<f32x4>(p + 4, f32x4{sums[0][4], sums[0][5], sums[0][6], sums[0][7]});
        }
    }
}

// One workgroup of 256 threads: zeros into the empty ones of kZeroRows rows at a
// time, workgroup wg of wgs.
template <int TAIL>
__device__ __forceinline__ void zero_rows(const IdArgs& a, const OrderArgs& o, int64_t wg, int64_t wgs, int64_t pad,
                                          void* dtable, int ddt)
{
    const int lane = threadIdx.x % 64, dim = a.dim, units = (dim + 7) >> 3;
    const float zero[8] = {};
    for (int64_t v0 = wg * kZeroRows; v0 < a.rows; v0 += wgs * kZeroRows) {
        const int64_t mine = v0 + lane;
        bool empty = false;
        if (lane < kZeroRows && mine < a.rows) {
            const int64_t s = slot_of(mine, o);
            empty = mine == pad || gld<int32_t>(o.start + s) == gld<int32_t>(o.start + s + 1);
        }
        for (unsigned long long todo = __ballot(empty); todo; todo &= todo - 1) {
            char* const row = static_cast<char*>(dtable) + (v0 + __builtin_ctzll(todo)) * dim * (ddt == DT_F32 ? 4 : 2);
            for (int unit = threadIdx.x; unit < units; unit += 256)
                store_row_unit_rt<TAIL, true>(ddt, row, unit, units, dim, zero);
        }
    }
}

// The work with the longest chains of reads first.  Bound by HBM: 54 us for the case of
// k_table_grad, where 217 MB of zeros are written beside the long ids' tokens.
template <int GDT, int TAIL>
__global__ __launch_bounds__(256) void k_prepare_grad(IdArgs a, OrderArgs o, const void* __restrict__ dy,
                                                      float* __restrict__ part, int32_t slices, int32_t list_wgs,
                                                      int32_t chunk_wgs, int64_t pad,
                                                      void* __restrict__ dtable, int ddt)
{
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x % 64;
    int64_t wg = blockIdx.x;
    if (wg < list_wgs) {
        list_used(o, wg * 4 + wave);
        return;
    }
    wg -= list_wgs;
    if (wg < chunk_wgs) {
        for (int64_t w = wg * 4 + wave; w / slices * o.chunk < a.n; w += (int64_t)chunk_wgs * 4)
            chunk_sums<GDT, TAIL>(a, o, dy, part, w / slices, (int)(w % slices) * 64 + lane);
        return;
    }
    wg -= chunk_wgs;
    zero_rows<TAIL>(a, o, wg, (int64_t)gridDim.x - list_wgs - chunk_wgs, pad, dtable, ddt);
}

// Joined sums of the long ids, 64 columns a wave, into the slot of the first
// chunk (which no other wave reads in these columns); 4.8 us as k_long_rows.
__global__ __launch_bounds__(kJoinWaves * 64) void k_join_chunks(OrderArgs o, float* __restrict__ part, int64_t padded)
{
    join_long_ids(o, part, padded, [&](int64_t, int32_t first, int64_t col, float sum) {
        part[chunk_slot(first / o.chunk, first, o.chunk) * padded + col] = sum;
    });
}

struct TableGradArgs {
    const void* dy;
    float* part;
    void* dtable;
    int64_t pad;
    float scale;
    int32_t accumulate, ddt, slices, work, zeros;
};

// One wave: the ordered tokens from c * chunk on, 64 units.  It sums, in order,
//  - the ids whose tokens begin in its chunk and are no more than a chunk: their rows
//    are written when their last token is added (up to one chunk further on);
//  - the chunk's tokens of long ids, into the chunk's partial rows.
// Lane l holds token c * chunk + l (two chunks are at most the 64 lanes) with the
// range of its id; UN tokens' units are in flight while UN are added, whatever
// ids they belong to (4 instead of 8 of 16 bits: 97 us against 93 for 16384 tokens of
// 4096).  The code that ends an id is there UN times: once, in a loop over the
// pieces of ids among the UN tokens, made calls of 300 to 4000 tokens 2 to 3 us slower.
template <int GDT, int TAIL>
__device__ __forceinline__ void sum_chunk_rows(const IdArgs& a, const OrderArgs& o, const TableGradArgs& p, int64_t c,
                                               int slice)
{
    constexpr int UN = GDT == DT_F32 ? 4 : 8;
    const int lane = threadIdx.x % 64, dim = a.dim, units = (dim + 7) >> 3, unit = slice * 64 + lane;
    const int32_t found = o.start[(int64_t(1) << o.log2g) * o.per];
    if (c * o.chunk >= found) return;
    const int32_t b = (int32_t)(c * o.chunk), at = b + lane;
    const bool valid = at < found && lane < 2 * o.chunk;
    const int32_t t = valid ? gld<int32_t>(o.order + at) : 0, id = valid ? gld<int32_t>(o.key + at) : 0;
    int32_t lo = 0, hi = 0;
    if (valid) {
        const int64_t s = slot_of(id, o);
        lo = gld<int32_t>(o.start + s);
        hi = gld<int32_t>(o.start + s + 1);
    }
    const bool is_long = hi - lo > o.chunk;
    const int32_t stop = is_long && hi > b + o.chunk ? b + o.chunk : hi;      // end of the id's tokens here
    const bool mine = valid && (is_long ? at < b + o.chunk : lo >= b && lo < b + o.chunk);
    const unsigned long long todo = __ballot(mine), ends = __ballot(mine && at == stop - 1);
    const unsigned long long longs = __ballot(mine && is_long);
    if (slice == 0 && mine && is_long && lo == at) o.longs[atomicAdd(&o.count[1], 1)] = id;
    if (!todo) return;
    const int i1 = 64 - __builtin_clzll(todo);
    int i = __builtin_ctzll(todo);
    Unit<GDT> u[UN];
    auto load = [&](int k) {
#pragma unroll
        for (int q = 0; q < UN; ++q) {
            // (a token beyond the last is read as the last: no branch, the same lines)
            const int32_t row = __builtin_amdgcn_readlane(t, k + q < i1 ? k + q : i1 - 1);
            u[q] = load_row_unit<GDT, TAIL, true>(static_cast<const char*>(p.dy) + (int64_t)row * dim * elem_bytes(GDT),
                                                  unit, units, dim);
        }
    };
    load(i);
    // an id's last token was added: its row, or the chunk's partial row
    float sum[8] = {};
    auto end_id = [&](int l) {
        if ((longs >> l) & 1) {
            const int64_t padded = (int64_t)units * 8;
            float* const out = p.part + chunk_slot((int32_t)c, __builtin_amdgcn_readlane(lo, l), o.chunk) * padded +
                               (int64_t)unit * 8;
            if (unit < units) {
                gst<f32x4>(out, f32x4{sum[0], sum[1], sum[2], sum[3]});
                gst<f32x4>(out + 4, f32x4{sum[4], sum[5], sum[6], sum[7]});
            }
        } else {
            const int64_t v0 = __builtin_amdgcn_readlane(id, l);
            if (v0 != p.pad) {
                char* const row = static_cast<char*>(p.dtable) + v0 * dim * (p.ddt == DT_F32 ? 4 : 2);
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[j] *= p.scale;
                if (p.accumulate) add_row_unit_rt<TAIL>(p.ddt, row, unit, units, dim, sum);
                store_row_unit_rt<TAIL, true>(p.ddt, row, unit, units, dim, sum);
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
    };
    for (; i < i1; i += UN) {
        Unit<GDT> v[UN];
#pragma unroll
        for (int q = 0; q < UN; ++q) v[q] = u[q];
        if (i + UN < i1) load(i + UN);
#pragma unroll
        for (int q = 0; q < UN; ++q) {
            if (i + q >= i1) break;
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j] += unit_at<GDT>(v[q], j);
            if ((ends >> (i + q)) & 1) end_id(i + q);
        }
    }
}

// p.work workgroups that sum (four waves each), then p.zeros that write zero
// rows: the summing waves, which wait for chains of reads, start first and the
// writes fill the time around them (16384 tokens of natural frequencies into [32000,
// 4096] bf16: 75 to 80 us; taking turns 86, in two launches 54 + 33).  Bound by HBM
// with rows in scattered order: 383 MB to move, 5 TB/s.
template <int GDT, int TAIL>
__global__ __launch_bounds__(256) void k_table_grad(IdArgs a, OrderArgs o, TableGradArgs p)
{
    const int64_t b = blockIdx.x;
    if (b >= p.work) {
        zero_rows<TAIL>(a, o, b - p.work, p.zeros, p.pad, p.dtable, p.ddt);
    } else {
        for (int64_t w = b * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / 64); w / p.slices * o.chunk < a.n;
             w += (int64_t)p.work * 4)
            sum_chunk_rows<GDT, TAIL>(a, o, p, w / p.slices, (int)(w % p.slices));
    }
}

// The rows of the long ids, one wave per 64 columns: 4.8 us, mostly the launch and
// the chain count - range - partial rows.
__global__ __launch_bounds__(kJoinWaves * 64) void k_long_rows(OrderArgs o, int dim, TableGradArgs p)
{
    join_long_ids(o, p.part, (dim + 7) / 8 * 8, [&](int64_t v, int32_t, int64_t col, float sum) {
        if (v == p.pad || col >= dim) return;
        sum *= p.scale;
        char* const row = static_cast<char*>(p.dtable) + v * dim * (p.ddt == DT_F32 ? 4 : 2);
        if (p.accumulate) sum += load1_rt(p.ddt, row, col);
        store1_rt(p.ddt, row, col, sum);
    });
}

template <int GDT>
hipError_t prepare_grad_as(const IdArgs& a, const OrderArgs& o, const void* dy, float* part, int64_t pad,
                           bool accumulate, void* dtable, int ddt, hipStream_t s)
{
    const int32_t slices = (int32_t)chunk_slices(a.dim);
    const int64_t most = int64_t(1) << 22;
    const int64_t list = ((int64_t(1) << o.log2g) + 3) / 4;
    int64_t chunks = (chunk_count(a.n, o.chunk) * slices + 3) / 4;
    int64_t zeros = accumulate ? 0 : (a.rows + kZeroRows - 1) / kZeroRows;
    if (chunks > most) chunks = most;
    if (zeros > most) zeros = most;
    auto go = [&](auto kernel) {
        return launch_kernel(kernel, (int)(list + chunks + zeros), s, a, o, dy, part, slices, (int32_t)list,
                             (int32_t)chunks, pad, dtable, ddt);
    };
    const int tail = tail_of(a.dim);
    return tail == kWhole     ? go(k_prepare_grad<GDT, kWhole>)
           : tail == kPartial ? go(k_prepare_grad<GDT, kPartial>)
                              : go(k_prepare_grad<GDT, kShort>);
}

// Few tokens: workgroup (t, slice) of 256 units works if token t is the first of
// its id; workgroups beyond the tokens' write zero rows.  A call is bound by its launch
// on the host: 8.2 us, against 12 to 15 with the ordering.
template <int GDT, int TAIL>
__global__ __launch_bounds__(256) void k_table_grad_direct(IdArgs a, const void* __restrict__ dy, float scale, int64_t pad,
                                                           int accumulate, void* __restrict__ dtable, int ddt,
                                                           int32_t slices)
{
    const DirectIds ids(a);
    const int dim = a.dim, units = (dim + 7) >> 3;
    const int64_t work = a.n * slices;
    if (blockIdx.x >= work) {
        zero_unnamed<TAIL, 256>(a, ids, (blockIdx.x - work) * kZeroRows, pad, dtable, ddt);
        return;
    }
    const int t = (int)(blockIdx.x / slices), unit = (int)(blockIdx.x % slices) * 256 + threadIdx.x;
    const int32_t v = ids.of(t);
    const unsigned long long m0 = ids.tokens(0, v), m1 = ids.tokens(1, v);
    if (v < 0 || v == pad || (m0 ? __builtin_ctzll(m0) : 64 + __builtin_ctzll(m1)) != t) return;
    float sum[1][8] = {};
    sum_masked<GDT, TAIL, 256, 1, 8>(m0, 0, dy, unit, units, dim, sum);
    sum_masked<GDT, TAIL, 256, 1, 8>(m1, 1, dy, unit, units, dim, sum);
    char* const row = static_cast<char*>(dtable) + (int64_t)v * dim * (ddt == DT_F32 ? 4 : 2);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[0][j] *= scale;
    if (accumulate) add_row_unit_rt<TAIL>(ddt, row, unit, units, dim, sum[0]);
    store_row_unit_rt<TAIL, true>(ddt, row, unit, units, dim, sum[0]);
}

// Workgroups for the columns of the long ids, 4 per CU at most.
int long_wgs(const IdArgs& a, const OrderArgs& o)
{
    const int64_t wgs = (a.n / o.chunk * ((a.dim + 63) / 64) + kJoinWaves - 1) / kJoinWaves;
    return (int)(wgs < 2048 ? wgs : 2048);
}

template <int GDT>
hipError_t table_grad_as(const IdArgs& a, const OrderArgs& o, TableGradArgs p, hipStream_t s)
{
    const int64_t most = int64_t(1) << 22;
    p.slices = (int32_t)chunk_slices(a.dim);
    int64_t work = (chunk_count(a.n, o.chunk) * p.slices + 3) / 4;
    int64_t zeros = p.accumulate ? 0 : (a.rows + kZeroRows - 1) / kZeroRows;
    if (work > most) work = most;
    if (zeros > most) zeros = most;
    p.work = (int32_t)work;
    p.zeros = (int32_t)zeros;
    if (work + zeros == 0) return hipSuccess;
    auto go = [&](auto kernel) { return launch_kernel(kernel, (int)(work + zeros), s, a, o, p); };
    const int tail = tail_of(a.dim);
    const hipError_t e = tail == kWhole     ? go(k_table_grad<GDT, kWhole>)
                         : tail == kPartial ? go(k_table_grad<GDT, kPartial>)
                                            : go(k_table_grad<GDT, kShort>);
    if (e != hipSuccess || a.n <= o.chunk) return e;       // no id can be long
    return launch_kernel_nt(k_long_rows, long_wgs(a, o), kJoinWaves * 64, s, o, a.dim, p);
}

}  // namespace

hipError_t launch_embedding(const IdArgs& a, const void* table, int tdt, float scale, void* y, int ydt, hipStream_t s)
{
    if (tdt == DT_F32) return embedding_y<DT_F32>(a, table, scale, y, ydt, s);
    if (tdt == DT_F16) return embedding_y<DT_F16>(a, table, scale, y, ydt, s);
    return embedding_y<DT_BF16>(a, table, scale, y, ydt, s);
}

hipError_t launch_dequant_embedding(const IdArgs& a, const DequantDesc& t, int bits, int code4, int B, int B2,
                                    float scale, void* y, int ydt, hipStream_t s)
{
    const QbTables* tab = device_tables();
    if (!tab) return hipErrorNotInitialized;
    const bool dq = t.c2 != nullptr;
    if (bits == 8)
        return dq ? dequant_embedding_y<8, true>(a, t, code4, B, B2, tab, scale, y, ydt, s)
                  : dequant_embedding_y<8, false>(a, t, code4, B, B2, tab, scale, y, ydt, s);
    return dq ? dequant_embedding_y<4, true>(a, t, code4, B, B2, tab, scale, y, ydt, s)
              : dequant_embedding_y<4, false>(a, t, code4, B, B2, tab, scale, y, ydt, s);
}

hipError_t launch_order(const IdArgs& a, const OrderArgs& o, hipStream_t s)
{
    const size_t lds = (size_t)kOrderWaves * o.per * sizeof(int32_t);
    const int threads = kOrderWaves * 64;
    if (!o.part_start)
        return launch_kernel_lds(a.id64 ? k_order<true, kAll> : k_order<false, kAll>, 1 << o.log2g, threads, lds, s, a, o);
    const hipError_t e = launch_kernel_lds(a.id64 ? k_order<true, kDeal> : k_order<false, kDeal>, kOrderParts, threads,
                                           kOrderWaves * sizeof(int32_t), s, a, o);
    return e != hipSuccess ? e : launch_kernel_lds(k_order<false, kInPart>, 1 << o.log2g, threads, lds, s, a, o);
}

hipError_t launch_prepare_grad(const IdArgs& a, const OrderArgs& o, const void* dy, int gdt, float* part, int64_t pad,
                               bool accumulate, void* dtable, int ddt, hipStream_t s)
{
    if (gdt == DT_F32) return prepare_grad_as<DT_F32>(a, o, dy, part, pad, accumulate, dtable, ddt, s);
    if (gdt == DT_F16) return prepare_grad_as<DT_F16>(a, o, dy, part, pad, accumulate, dtable, ddt, s);
    return prepare_grad_as<DT_BF16>(a, o, dy, part, pad, accumulate, dtable, ddt, s);
}

hipError_t launch_table_grad_direct(const IdArgs& a, const void* dy, int gdt, float scale, int64_t pad,
                                    bool accumulate, void* dtable, int ddt, hipStream_t s)
{
    const int64_t slices = (a.dim + 2047) / 2048, grid = a.n * slices + direct_zero_wgs(a.rows, accumulate);
    auto go = [&](auto kernel) {
        return launch_kernel(kernel, (int)grid, s, a, dy, scale, pad, accumulate ? 1 : 0, dtable, ddt, (int32_t)slices);
    };
    auto with = [&](auto gdt_c) {
        constexpr int GDT = decltype(gdt_c)::value;
        const int tail = tail_of(a.dim);
        return tail == kWhole     ? go(k_table_grad_direct<GDT, kWhole>)
               : tail == kPartial ? go(k_table_grad_direct<GDT, kPartial>)
                                  : go(k_table_grad_direct<GDT, kShort>);
    };
    if (gdt == DT_F32) return with(std::integral_constant<int, DT_F32>{});
    if (gdt == DT_F16) return with(std::integral_constant<int, DT_F16>{});
    return with(std::integral_constant<int, DT_BF16>{});
}

hipError_t launch_join_chunks(const IdArgs& a, const OrderArgs& o, float* part, hipStream_t s)
{
    if (a.n <= o.chunk) return hipSuccess;             // no id can be long
    return launch_kernel_nt(k_join_chunks, long_wgs(a, o), kJoinWaves * 64, s, o, part, padded_dim(a.dim));
}

hipError_t launch_table_grad(const IdArgs& a, const OrderArgs& o, const void* dy, int gdt, float* part, float scale,
                             int64_t pad, bool accumulate, void* dtable, int ddt, hipStream_t s)
{
    const TableGradArgs p{dy, part, dtable, pad, scale, accumulate ? 1 : 0, ddt, 0, 0, 0};
    if (gdt == DT_F32) return table_grad_as<DT_F32>(a, o, p, s);
    if (gdt == DT_F16) return table_grad_as<DT_F16>(a, o, p, s);
    return table_grad_as<DT_BF16>(a, o, p, s);
}

}  // namespace qb
