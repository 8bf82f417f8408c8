// qb_layers.h -- internal launchers of the row-wise layers: embedding lookup
// (dense and quantized tables) and its gradient, layer norm, and the stable
// embedding that joins them.  Argument checks are done by the callers in
// qb_layers_api.cpp.
#pragma once
#include "qb_launch.h"

namespace qb {

// Longest row of the kernels that hold a row in registers (1024 threads x 2
// units x 8 elements).
constexpr int64_t kRowRegMax = 16384;

// Token ids of a lookup: n ids of 32 or 64 bits into a table of `rows` rows of
// `dim` elements.
struct IdArgs {
    const void* ids;
    int64_t n;
    int64_t rows;
    int32_t id64;
    int32_t dim;
};

// Order of the tokens of a gradient.  Ids are dealt into 2^log2g classes, class
// = id mod 2^log2g, entry = id >> log2g (`per` entries a class): frequent
// tokens have small ids in common vocabularies, and neighbouring ids land in
// different classes.  start[class * per + entry] .. start[... + 1] is the range of
// the id's tokens in `order`, which lists their positions in ascending order;
// `key` lists their ids.
// Where there are many classes (order_in_parts), the tokens are dealt into
// kOrderParts ranges of classes first: part p is part_pos / part_id[part_start[p] ..
// part_start[p + 1]), in ascending order of the positions, and a class goes through
// its part only.
// `list` holds the count[0] ids that have tokens, each as {id, begin, end, first
// position}, `longs` the count[1] ids that have more than `chunk` tokens.
struct OrderArgs {
    int32_t* start;      // [classes * per + 1]
    int32_t* order;      // [n]
    int32_t* key;        // [n]
    int32_t* used;       // [2 * classes] ids with tokens, and with more than a chunk, per class
    int32_t* count;      // [2]
    int32_t* list;       // [4 * min(n, rows)]
    int32_t* longs;      // [n / chunk + 1]
    int32_t log2g;
    int32_t per;
    int32_t chunk;
    int32_t* part_start; // [kOrderParts + 1], nullptr: without parts
    int32_t* part_pos;   // [n]
    int32_t* part_id;    // [n]
};

constexpr int kOrderWaves = 16;            // waves of the ordering kernel
constexpr int kOrderPerMax = 1000;         // entries of a class: one per thread, 16 x 1000 counters in 64 KB of LDS

// Classes for a table of `rows` rows: 256 (one workgroup per CU), more where a
// class would hold over kOrderPerMax entries, fewer for tiny tables.
constexpr int32_t order_log2g(int64_t rows)
{
    int32_t g = 0;
    while (g < 8 && (int64_t(1) << g) < rows) ++g;
    while (((rows + (int64_t(1) << g) - 1) >> g) > kOrderPerMax) ++g;
    return g;
}
constexpr int64_t order_per(int64_t rows) { return (rows + (int64_t(1) << order_log2g(rows)) - 1) >> order_log2g(rows); }

// Whether the ordering deals the tokens into parts first.  Every class's workgroup
// reads all tokens' ids otherwise, n * 2^log2g reads: minutes for 2^30 tokens and the
// 2^17 classes of 2^26 rows.  In parts it is n * (256 + 2^(log2g - 8)) and a launch more.
// Up to 512 classes are resident at once, and the launch pays for many tokens only;
// beyond that nearly always (whole gradient of rows of 8 elements in us, without / with
// parts: 300000 rows, 16384 tokens 37.1 / 42.7, 49152 68.5 / 67.5, 2^20 886 / 666; 600000
// rows, 300 tokens 31.0 / 34.1, 1024 39.9 / 38.7, 49152 102.6 / 72.8; 2^20 rows, 300 tokens
// 47.0 / 46.9, 2^20 2617 / 745; 2^24 rows, 2^20 tokens 36400 / 1500).
constexpr int kOrderPartBits = 8, kOrderParts = 1 << kOrderPartBits;
constexpr bool order_in_parts(int64_t n, int64_t rows)
{
    const int32_t log2g = order_log2g(rows);
    return log2g > 10 || (log2g == 10 && n >= 1024) || (log2g == 9 && n >= 49152);
}

// Tokens per chunk of the ordered list: an id with more tokens than this is
// summed chunk by chunk, then joined.  Two chunks fit the lanes of a wave.  A wave
// takes a chunk's share of 512 columns.  Short chunks give few tokens the more waves
// (16 against 32 tokens a chunk: 300 tokens of 704 elements 14.6 against 18.2 us, 5003 of
// 1001 binary32 25.1 against 30.6); beyond about 12 waves a CU the chip is full and they
// only leave more partial rows.  Both, in us for natural frequencies over 8191 and 32000
// rows of bf16: 16384 x 64 24.9/28.2 and 26.0/29.6, 65536 x 64 55.4/57.0 and 57.8/57.3,
// 131072 x 64 93.4/89.6 and 92.5/91.3; 16384 x 1024 30.0/30.9 and 35.8/38.4, 32768 x 1024
// 51.6/47.4 and 53.2/53.5; 5003 x 4096 37.5/38.2 and 71.1/72.3, 12000 x 4096 52.3/50.3 and
// 86.3/84.5.  Ids even over the table cross at twice the tokens; a batch of a single id
// is 10 to 15% faster with 32 throughout.
constexpr int32_t kChunkShort = 16, kChunkLong = 32;
constexpr int64_t kChunkWaves = 12 * 256;
constexpr int64_t chunk_count(int64_t n, int64_t chunk = kChunkLong) { return (n + chunk - 1) / chunk; }
constexpr int64_t chunk_slices(int64_t dim) { return (dim + 511) / 512; }
constexpr int32_t chunk_tokens(int64_t n, int64_t dim)
{
    return chunk_count(n, kChunkShort) * chunk_slices(dim) <= kChunkWaves ? kChunkShort : kChunkLong;
}
constexpr int64_t padded_dim(int64_t dim) { return (dim + 7) / 8 * 8; }

// Workgroups whose partial sums of the norm's weight gradients are joined.
constexpr int kNormPartsMax = 256;

// Workgroups of T threads for a kernel that walks `tiles` tiles by the grid: as
// many as are resident at once.
template <int T, class Kernel>
int persistent_grid_of(Kernel kernel, int64_t tiles)
{
    auto query = [](const void* k) -> int {
        int per_cu = 0;
        if (hipOccupancyMaxActiveBlocksPerMultiprocessor(&per_cu, reinterpret_cast<Kernel>(const_cast<void*>(k)), T, 0) !=
                hipSuccess || per_cu < 1)
            per_cu = 1;
        return per_cu;
    };
    const int cap = persistent_grid_cap(reinterpret_cast<const void*>(kernel), query);
    return (int)(tiles < cap ? tiles : cap);
}

// Rows [t0, t0 + m) of n in one launch each: a launch holds at most 2^21
// workgroups (workgroups times threads stay below 2^32), `per_wg` rows apiece.
template <class Launch>
hipError_t launch_rows(int64_t n, int64_t per_wg, Launch launch)
{
    const int64_t most = per_wg << 21;
    for (int64_t t0 = 0; t0 < n; t0 += most) {
        const int64_t m = n - t0 < most ? n - t0 : most;
        const hipError_t e = launch(t0, m, (int)((m + per_wg - 1) / per_wg));
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// The ids from token t0 on.
inline IdArgs ids_from(const IdArgs& a, int64_t t0, int64_t m)
{
    IdArgs b = a;
    if (a.ids) b.ids = static_cast<const char*>(a.ids) + t0 * (a.id64 ? 8 : 4);
    b.n = m;
    return b;
}

hipError_t launch_embedding(const IdArgs& a, const void* table, int tdt, float scale, void* y, int ydt,
                            hipStream_t s);

// Table as codes (bits 8: dynamic code; 4: code4 0 NF4, 1 FP4) with block size
// B, and absmax (plain) or c2 / absmax2 / offset (nested, block size B2).
hipError_t launch_dequant_embedding(const IdArgs& a, const DequantDesc& t, int bits, int code4, int B, int B2,
                                    float scale, void* y, int ydt, hipStream_t s);

// start, order, key of the ids.
hipError_t launch_order(const IdArgs& a, const OrderArgs& o, hipStream_t s);

// Joins the chunks' sums of the long ids, each into the slot of its first chunk.
hipError_t launch_join_chunks(const IdArgs& a, const OrderArgs& o, float* part, hipStream_t s);

// The second step of a stable embedding's gradient, one launch of three kinds of
// workgroups:
//  - the list of the ids that have tokens;
//  - sums of dy over the chunks' tokens of ids that have more tokens than a
//    chunk: part[2 * chunk] for an id whose tokens begin at or before the chunk's
//    first, part[2 * chunk + 1] for one whose tokens begin inside the chunk (rows of
//    padded_dim binary32);
//  - zeros into the rows of dtable whose ids take no gradient: those without
//    tokens, and pad (none with accumulate).
hipError_t launch_prepare_grad(const IdArgs& a, const OrderArgs& o, const void* dy, int gdt, float* part, int64_t pad,
                               bool accumulate, void* dtable, int ddt, hipStream_t s);

// dtable[v] = scale * sum of dy over the tokens of v (+ dtable[v] with
// accumulate), zeros for the other rows: one launch, and one that joins the long
// ids' sums (part as above).
hipError_t launch_table_grad(const IdArgs& a, const OrderArgs& o, const void* dy, int gdt, float* part, float scale,
                             int64_t pad, bool accumulate, void* dtable, int ddt, hipStream_t s);

// Up to kDirectTokens tokens take no ordering: one launch, in which the first token
// of each id sums the id's tokens (a wave holds all ids in two registers a lane).
// A call of few tokens is bound by its launches, about 2.5 us each on the host.
constexpr int64_t kDirectTokens = 128;
constexpr bool takes_direct(int64_t n, int64_t rows) { return n > 0 && n <= kDirectTokens && rows < (int64_t(1) << 24); }
hipError_t launch_table_grad_direct(const IdArgs& a, const void* dy, int gdt, float scale, int64_t pad,
                                    bool accumulate, void* dtable, int ddt, hipStream_t s);

struct NormArgs {
    const void* gamma;      // nullptr: ones
    const void* beta;       // nullptr: zeros
    int wdt;
    float eps;
};

hipError_t launch_layer_norm(const void* x, int xdt, int64_t n, int64_t dim, const NormArgs& w, void* y, float* mean,
                             float* rstd, hipStream_t s);
hipError_t launch_stable_embedding(const IdArgs& a, const void* table, int tdt, float scale, const NormArgs& w,
                                   void* y, int ydt, hipStream_t s);

// Workgroups (and partial sums) of the backward passes.
int layer_norm_parts(int64_t n, int64_t dim);
int stable_parts(int64_t n, int64_t rows);

// dx, and the partial sums part[g][2][padded_dim] of dgamma and dbeta over
// layer_norm_parts(n, dim) workgroups (part nullptr: not wanted).
hipError_t launch_layer_norm_grad(const void* dy, const void* x, int xdt, int64_t n, int64_t dim, const void* gamma,
                                  int wdt, const float* mean, const float* rstd, void* dx, float* part,
                                  hipStream_t s);

// As launch_table_grad for the table below a layer norm, with the partial sums of dgamma and dbeta.
hipError_t launch_stable_grad(const IdArgs& a, const OrderArgs& o, const void* dy, int gdt, const float* chunk_part,
                              const void* table, int tdt, float scale, const NormArgs& w, int64_t pad,
                              bool accumulate, void* dtable, int ddt, float* part, int parts, hipStream_t s);

// The same for up to kDirectTokens tokens, with one partial sum per token.
hipError_t launch_stable_grad_direct(const IdArgs& a, const void* dy, int gdt, const void* table, int tdt, float scale,
                                     const NormArgs& w, int64_t pad, bool accumulate, void* dtable, int ddt,
                                     float* part, hipStream_t s);

// dgamma, dbeta (either may be nullptr) = the sum of `parts` partial sums.
hipError_t launch_join_parts(const float* part, int parts, int64_t dim, bool accumulate, void* dgamma, void* dbeta,
                             int wdt, hipStream_t s);

}  // namespace qb
