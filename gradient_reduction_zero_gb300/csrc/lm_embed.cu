// Embedding lookup with scaling, and its gradient by sorted tokens.
#include <algorithm>

#include "bulk.cuh"
#include "device.cuh"
#include "internal.h"
#include "lm.h"

namespace dpz {

namespace {

// One access unit of a row: W = 8 or 4 elements in one word of 8 to 32 bytes
// (rows aligned to W elements whose length is a multiple of W), or W = 1
// element.
template <int DT, int W>
struct Unit;

template <>
struct Unit<DPZ_F32, 4> {
    using Raw = uint4;
    static __device__ __forceinline__ Raw load(const char* p) { return ld16(p); }
    static __device__ __forceinline__ void unpack(const Raw& r, float x[4])
    {
        x[0] = __uint_as_float(r.x);
        x[1] = __uint_as_float(r.y);
        x[2] = __uint_as_float(r.z);
        x[3] = __uint_as_float(r.w);
    }
    static __device__ __forceinline__ void store(char* p, const float x[4])
    {
        st16(p, make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                           __float_as_uint(x[3])));
    }
};

template <>
struct Unit<DPZ_BF16, 4> {
    using Raw = uint2;
    static __device__ __forceinline__ Raw load(const char* p)
    {
        Raw r;
        asm volatile("ld.global.L2::256B.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
        return r;
    }
    static __device__ __forceinline__ void unpack(const Raw& r, float x[4])
    {
        x[0] = bf16_lo(r.x);
        x[1] = bf16_hi(r.x);
        x[2] = bf16_lo(r.y);
        x[3] = bf16_hi(r.y);
    }
    static __device__ __forceinline__ void store(char* p, const float x[4])
    {
        asm volatile("st.global.cs.v2.u32 [%0], {%1,%2};" ::"l"(p), "r"(pack_bf16x2(x[0], x[1])),
                     "r"(pack_bf16x2(x[2], x[3]))
                     : "memory");
    }
};

template <int DT>
struct Unit<DT, 8> {
    using Raw = typename Group<DT>::Raw;
    static __device__ __forceinline__ Raw load(const char* p) { return Group<DT>::load_raw(p); }
    static __device__ __forceinline__ void unpack(const Raw& r, float x[8])
    {
        Group<DT>::unpack(r, x);
    }
    static __device__ __forceinline__ void store(char* p, const float x[8])
    {
        store_group<DT>(p, x);
    }
};

template <>
struct Unit<DPZ_F32, 1> {
    using Raw = float;
    static __device__ __forceinline__ Raw load(const char* p)
    {
        return *reinterpret_cast<const float*>(p);
    }
    static __device__ __forceinline__ void unpack(const Raw& r, float x[1]) { x[0] = r; }
    static __device__ __forceinline__ void store(char* p, const float x[1])
    {
        *reinterpret_cast<float*>(p) = x[0];
    }
};

template <>
struct Unit<DPZ_BF16, 1> {
    using Raw = unsigned short;
    static __device__ __forceinline__ Raw load(const char* p)
    {
        return *reinterpret_cast<const unsigned short*>(p);
    }
    static __device__ __forceinline__ void unpack(const Raw& r, float x[1])
    {
        x[0] = __uint_as_float((uint32_t)r << 16);
    }
    static __device__ __forceinline__ void store(char* p, const float x[1])
    {
        *reinterpret_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(x[0]);
    }
};

DPZ_HD constexpr int bytes_of(int DT) { return DT == DPZ_F32 ? 4 : 2; }

// ------------------------------------------------------------ lookup

// One warp per row: out[t] = R(scale * table[ids[t]]), kLookupLoads units of a
// lane under way at once.
constexpr int kLookupLoads = 4;

template <int WDT, int ODT, int W>
__global__ void __launch_bounds__(kBlock)
    k_embedding(Mat table, Ids ids, int64_t T, int64_t V, int64_t D, float scale, Mat out)
{
    pdl_enter();
    const int64_t t = global_warp();
    if (t >= T) return;
    const int lane = threadIdx.x & 31;
    const int v = load_token(ids, t, V);
    const char* src = table.p + ((int64_t)(v < 0 ? 0 : v) * table.ld + lane * W) * bytes_of(WDT);
    char* dst = out.p + (t * out.ld + lane * W) * bytes_of(ODT);
    const int units = (int)(D / W);
    for (int i = lane; i < units; i += 32 * kLookupLoads) {
        typename Unit<WDT, W>::Raw raw[kLookupLoads];
#pragma unroll
        for (int u = 0; u < kLookupLoads; ++u)
            if (v >= 0 && i + 32 * u < units)
                raw[u] = Unit<WDT, W>::load(src + u * (32 * W * bytes_of(WDT)));
#pragma unroll
        for (int u = 0; u < kLookupLoads; ++u)
            if (i + 32 * u < units) {
                float x[W] = {};
                if (v >= 0) {
                    Unit<WDT, W>::unpack(raw[u], x);
#pragma unroll
                    for (int j = 0; j < W; ++j) x[j] = __fmul_rn(x[j], scale);
                }
                Unit<ODT, W>::store(dst + u * (32 * W * bytes_of(ODT)), x);
            }
        src += kLookupLoads * 32 * W * bytes_of(WDT);
        dst += kLookupLoads * 32 * W * bytes_of(ODT);
    }
}

// ------------------------------------------------------------ gradient
//
// The tokens are put in order of (id, position), so that every table row's
// terms stand together and are added in order of position: the sum is the
// same from run to run, where adding rows with atomics is not.

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortLogBins = kEmbLogBins;
constexpr int kSortMaxBins = 1 << kSortLogBins;   // ids one block owns at most
constexpr int kSortHits = 256;       // of its ids a warp keeps from its first pass
constexpr int kSortLoads = 8;        // ids a lane loads at once

// The low word of an id, all ones where it names none of V < 2^30 tokens (whose
// owner is then the last one, which looks again).
__device__ __forceinline__ uint32_t id_word(int64_t id, uint32_t V)
{
    const uint32_t lo = (uint32_t)id;
    return (uint32_t)(id >> 32) == 0 && lo < V ? lo : ~0u;
}

__device__ __forceinline__ uint32_t id_word(int id, uint32_t V)
{
    return (uint32_t)id < V ? (uint32_t)id : ~0u;
}

// Loads kSortLoads ids per lane, 32 positions apart, from position i0 on.
template <class ID>
__device__ __forceinline__ void load_words(const ID* ids, int64_t i0, int64_t hi, uint32_t V,
                                           uint32_t (&w)[kSortLoads])
{
    const ID* p = ids + i0 + (threadIdx.x & 31);
    if (i0 + 32 * kSortLoads <= hi) {
        ID id[kSortLoads];
#pragma unroll
        for (int u = 0; u < kSortLoads; ++u) id[u] = p[u * 32];
#pragma unroll
        for (int u = 0; u < kSortLoads; ++u) w[u] = id_word(id[u], V);
        return;
    }
    const int left = (int)(hi - i0) - (int)(threadIdx.x & 31);
#pragma unroll
    for (int u = 0; u < kSortLoads; ++u) w[u] = u * 32 < left ? id_word(p[u * 32], V) : ~0u;
}

// Places up to 32 tokens of this block, one per lane where `hit`, in order:
// id k's go to next[k], next[k] + 1, ...
__device__ __forceinline__ void place(bool hit, int k, int position, int* next, int* order)
{
    const int lane = threadIdx.x & 31;
    const unsigned m = __ballot_sync(0xffffffffu, hit);
    if (hit) {
        const unsigned same = __match_any_sync(m, k);
        const int rank = __popc(same & ((1u << lane) - 1u));
        const int at = next[k];
        order[at + rank] = position;
        __syncwarp(m);
        if (rank == 0) next[k] = at + __popc(same);
    }
    __syncwarp();
}

// The sum of x over this thread and those before it in the block.
__device__ __forceinline__ int block_scan(int x, int* warp_tot)
{
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += up;
    }
    if (lane == 31) warp_tot[wid] = x;
    __syncthreads();
    const int before = __reduce_add_sync(0xffffffffu, lane < wid ? warp_tot[lane] : 0);
    __syncthreads();
    return x + before;
}

// Block b owns the ids v with v % owners == b, which spreads the frequent low
// ids of a byte-pair vocabulary over the blocks.  Every block reads all T
// ids (from L2), so no block waits for another one: it counts the ids of lower
// owners (where its part of the order begins) and, per warp, its own ids; the
// prefix sums of those counts place each token.  Warps take consecutive
// ranges of positions, so the order within an id is that of positions.  The
// long runs (more than ws.piece terms) are listed for the kernels that sum
// them in pieces.  A warp keeps its hits in shared memory; one with more than
// kSortHits (a very frequent id) reads its range again.
template <class ID>
__global__ void __launch_bounds__(kSortThreads)
    k_emb_sort(const ID* __restrict__ ids, int64_t T, int64_t V, int log_owners, int bins, EmbWs ws)
{
    extern __shared__ int2 kept_hist[];
    int2(*kept)[kSortHits] = reinterpret_cast<int2(*)[kSortHits]>(kept_hist);   // position, bin
    int* hist = reinterpret_cast<int*>(kept_hist + kSortWarps * kSortHits);     // [kSortWarps][bins]
    __shared__ int warp_tot[kSortWarps];
    __shared__ int s_base;
    pdl_enter();
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int owners = 1 << log_owners, me = blockIdx.x;
    for (int i = threadIdx.x; i < kSortWarps * bins; i += kSortThreads) hist[i] = 0;
    __syncthreads();
    const int64_t per = ((T + kSortThreads - 1) / kSortThreads) * 32;
    const int64_t lo = wid * per, hi = min(T, lo + per);
    int* mine = hist + wid * bins;
    int less = 0, hits = 0;
    for (int64_t i0 = lo; i0 < hi; i0 += 32 * kSortLoads) {
        uint32_t w[kSortLoads];
        load_words(ids, i0, hi, (uint32_t)V, w);
#pragma unroll
        for (int u = 0; u < kSortLoads; ++u) {
            const int d = (int)(w[u] & (owners - 1)) - me;
            less += (uint32_t)d >> 31;                 // owner below this one
            if (__any_sync(0xffffffffu, d == 0)) {
                const bool hit = d == 0 && w[u] != ~0u;
                const unsigned m = __ballot_sync(0xffffffffu, hit);
                if (hit) {
                    const int k = (int)(w[u] >> log_owners);
                    const int at = hits + __popc(m & ((1u << lane) - 1u));
                    atomicAdd(&mine[k], 1);
                    if (at < kSortHits) kept[wid][at] = make_int2((int)(i0 + u * 32 + lane), k);
                }
                hits += __popc(m);
            }
        }
    }
    less = __reduce_add_sync(0xffffffffu, less);
    if (lane == 0) warp_tot[wid] = less;
    __syncthreads();
    if (wid == 0) {
        const int s = __reduce_add_sync(0xffffffffu, warp_tot[lane]);
        if (lane == 0) s_base = s;
    }
    __syncthreads();
    // thread k < bins: id k's count over the warps, then prefix sums over the
    // ids: of the counts, and of the long runs and their pieces
    int total = 0;
    if (threadIdx.x < bins)
        for (int w = 0; w < kSortWarps; ++w) total += hist[w * bins + threadIdx.x];
    const int pieces = total > ws.piece ? (total + ws.piece - 1) / ws.piece : 0;
    const int incl = block_scan(total, warp_tot);
    const int incl_pieces = block_scan(pieces, warp_tot);
    // two counts of at most 1,024 in one sum
    const int is_long = pieces > 0, is_short = total > 0 && !is_long;
    const int incl_runs = block_scan(is_long << 16 | is_short, warp_tot);
    if (threadIdx.x < bins) {
        int at = s_base + incl - total;
        const int v = (int)(threadIdx.x << log_owners) + me;
        if (v < V) ws.run[v] = make_int2(at, total);
        const int64_t list = (int64_t)me << kSortLogBins;
        if (is_long)
            ws.longs[list + (incl_runs >> 16) - 1] = make_int4(v, at, total, incl_pieces - pieces);
        if (is_short) ws.shorts[list + (incl_runs & 0xffff) - 1] = make_int4(v, at, total, 0);
        if (threadIdx.x == bins - 1)
            ws.owner[me] = make_int4(incl_pieces, incl_runs >> 16, incl_runs & 0xffff, 0);
        for (int w = 0; w < kSortWarps; ++w) {
            const int n = hist[w * bins + threadIdx.x];
            hist[w * bins + threadIdx.x] = at;
            at += n;
        }
    }
    __syncthreads();
    if (hits <= kSortHits) {
        for (int i = lane; i - lane < hits; i += 32) {
            const int2 h = i < hits ? kept[wid][i] : make_int2(0, 0);
            place(i < hits, h.y, h.x, mine, ws.order);
        }
        return;
    }
    for (int64_t i0 = lo; i0 < hi; i0 += 32 * kSortLoads) {
        uint32_t w[kSortLoads];
        load_words(ids, i0, hi, (uint32_t)V, w);
#pragma unroll
        for (int u = 0; u < kSortLoads; ++u)
            place((int)(w[u] & (owners - 1)) == me && w[u] != ~0u, (int)(w[u] >> log_owners),
                  (int)(i0 + u * 32 + lane), mine, ws.order);
    }
}

// By one warp: finds which owner's the j-th of all owners' pieces is, and how
// many of them come before that owner's; owner -1 if there are not that many.
struct OwnerOf {
    int owner, before;
};

__device__ __forceinline__ OwnerOf find_owner(const EmbWs& ws, int owners, int j)
{
    const int lane = threadIdx.x & 31;
    int before = 0;
    for (int o0 = 0; o0 < owners; o0 += 128) {     // owners is a multiple of 128
        int n[4], sum = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            n[u] = ws.owner[o0 + lane * 4 + u].x;   // pieces
            sum += n[u];
        }
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        int at = before + incl - sum, mine = -1, mine_before = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (j >= at && j < at + n[u]) {
                mine = o0 + lane * 4 + u;
                mine_before = at;
            }
            at += n[u];
        }
        const unsigned m = __ballot_sync(0xffffffffu, mine >= 0);
        if (m != 0) {
            const int src = __ffs(m) - 1;
            return {__shfl_sync(0xffffffffu, mine, src), __shfl_sync(0xffffffffu, mine_before, src)};
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
    return {-1, before};
}

// W fp32 values of a partial row (16-byte aligned for W >= 4); they are read
// again soon, from L2.
template <int W>
__device__ __forceinline__ void load_partial(const float* p, float (&x)[W])
{
    if constexpr (W >= 4) {
#pragma unroll
        for (int j = 0; j < W; j += 4) {
            const float4 v = *reinterpret_cast<const float4*>(p + j);
            x[j] = v.x;
            x[j + 1] = v.y;
            x[j + 2] = v.z;
            x[j + 3] = v.w;
        }
    } else {
        x[0] = p[0];
    }
}

template <int W>
__device__ __forceinline__ void store_partial(float* p, const float (&x)[W])
{
    if constexpr (W >= 4) {
#pragma unroll
        for (int j = 0; j < W; j += 4)
            *reinterpret_cast<float4*>(p + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
    } else {
        p[0] = x[0];
    }
}

// By one warp: the pieces of all owners below this one.
__device__ __forceinline__ int pieces_before(const EmbWs& ws, int owner)
{
    int n = 0;
    for (int o = threadIdx.x & 31; o < owner; o += 32) n += ws.owner[o].x;
    return __reduce_add_sync(0xffffffffu, n);
}

// Sums of rows.  A block has one thread per unit of columns and a list of
// segments, each a stretch of the sorted order with one destination: the rows
// of a group of consecutive ids of one owner (whose tokens stand together; in
// place, of consecutive ids that have tokens), or one piece of a long run,
// whose sum goes to a partial row.  The base's rows are copied to
// shared memory asynchronously, before anything is known about the tokens
// (in place: for the rows with tokens only); each thread uses what it copied
// itself.  Rows without a token are then written as they are.  The others'
// terms are walked as one list of token positions with kAhead loads under way
// whatever the lengths of the segments, so that rows of one and of many terms
// stream alike.
// A group is 4 rows for narrow blocks and 8 for wide ones (more than 128
// threads), which keeps enough blocks in flight for the one and few enough
// set-ups for the other: D = 768 in bf16, 96 threads, 8,192 tokens: 26.4 us
// with 4 and 28.4 with 8; D = 1,600, 224 threads, 65,536 tokens: 122 and 115.
constexpr int kSegments = 8;
constexpr int kRowsBlocks = 5;   // of kBlock threads on an SM, at least

struct Segments {
    int empty[kSegments];      // rows without a token, by their place in the group
    int slot[kSegments];       // with tokens: the same
    int row[kSegments];        // by place in the group: the table row, -1 for a piece
    int start[kSegments];      // in the sorted order
    int first[kSegments];      // its first item
    int empties, full, items;  // how many of each
    int item[kSegments * kEmbMaxPiece];   // token positions
};

// By one warp: this lane's segment of a piece (lane 0) or a group of rows
// (count < 0: none).
__device__ __forceinline__ void find_piece(const EmbGrad& g, int piece, int log_owners, int& start,
                                           int& count)
{
    const int lane = threadIdx.x & 31;
    const OwnerOf o = find_owner(g.ws, 1 << log_owners, piece);
    if (o.owner < 0) return;
    // the owner's long run that the piece is of: the last to begin at or before it
    const int j = piece - o.before, runs = g.ws.owner[o.owner].y;
    const int4* list = g.ws.longs + ((int64_t)o.owner << kSortLogBins);
    int4 run = make_int4(0, 0, 0, 0);
    for (int i0 = 0; i0 < runs; i0 += 32) {
        const int4 r = i0 + lane < runs ? list[i0 + lane] : make_int4(0, 0, 0, 0x7fffffff);
        const unsigned m = __ballot_sync(0xffffffffu, r.w <= j);
        if (m == 0) break;
        const int src = 31 - __clz(m);
        run.y = __shfl_sync(0xffffffffu, r.y, src);
        run.z = __shfl_sync(0xffffffffu, r.z, src);
        run.w = __shfl_sync(0xffffffffu, r.w, src);
    }
    if (lane > 0) return;
    start = run.y + (j - run.w) * g.ws.piece;
    count = min(g.ws.piece, run.y + run.z - start);
}

// Copies one unit to shared memory, asynchronously where the size allows it.
template <class Raw>
__device__ __forceinline__ void stage_unit(Raw* dst, const char* src)
{
    if constexpr (sizeof(Raw) >= 4)
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_addr(dst)), "l"(src),
                     "n"(sizeof(Raw))
                     : "memory");
    else
        *dst = *reinterpret_cast<const Raw*>(src);
}

template <int DDT, int GDT, int W, bool IN_PLACE>
__global__ void __launch_bounds__(kBlock, kRowsBlocks)
    k_emb_rows(EmbGrad g, int tile_units, int log_owners, int group, int per_owner)
{
    constexpr int kAhead = 4;
    constexpr int kGB = bytes_of(GDT), kDB = bytes_of(DDT);
    using Base = typename Unit<GDT, W>::Raw;
    extern __shared__ uint4 staged[];           // Base [group][blockDim.x]
    __shared__ Segments sg;
    pdl_enter();
    Base* own = reinterpret_cast<Base*>(staged) + threadIdx.x;
    const int unit = blockIdx.y * tile_units + threadIdx.x;
    const bool on = (int)threadIdx.x < tile_units && (int64_t)unit * W < g.D;
    const char* bcol = g.base.p + (int64_t)unit * W * kGB;
    char* gcol = g.dtable.p + (int64_t)unit * W * kGB;
    const char* dcol = g.dout.p + (int64_t)unit * W * kDB;
    const int64_t bld = g.base.ld * kGB, gld = g.dtable.ld * kGB, dld = g.dout.ld * kDB;
    const bool has_base = g.base.p != nullptr;
    // pieces first, then the owners' groups; owners vary fastest, so that the
    // blocks under way together write neighbouring rows
    const int64_t b = (int64_t)blockIdx.x - g.ws.pieces;
    const int owner = (int)(b & ((1 << log_owners) - 1));
    const int4* shorts = g.ws.shorts + ((int64_t)owner << kSortLogBins);
    const int present = IN_PLACE && b >= 0 ? g.ws.owner[owner].z : 0;
    for (int64_t j = b >> log_owners;; j += per_owner) {      // the owner's j-th group
        if (IN_PLACE && b >= 0 && j * group >= present) return;
        const int64_t row0 = owner + (j * group << log_owners);
        if (b >= 0 && has_base && !IN_PLACE && on)
            for (int i = 0; i < group; ++i) {
                const int64_t row = row0 + ((int64_t)i << log_owners);
                if (row < g.V) stage_unit(own + i * blockDim.x, bcol + row * bld);
            }
        if (threadIdx.x < 32) {
            const int lane = threadIdx.x;
            int row = -1, start = 0, count = -1;
            if (b < 0) {
                find_piece(g, blockIdx.x, log_owners, start, count);
            } else if (IN_PLACE) {
                if (lane < group && j * group + lane < present) {
                    const int4 r = shorts[j * group + lane];
                    row = r.x;
                    start = r.y;
                    count = r.z;
                }
            } else {
                const int64_t v = row0 + ((int64_t)lane << log_owners);
                if (lane < group && v < g.V) {
                    const int2 run = g.ws.run[v];
                    row = (int)v;
                    start = run.x;
                    if (run.y <= g.ws.piece) count = run.y;
                }
            }
            const unsigned below = (1u << lane) - 1u;
            const unsigned empty = __ballot_sync(0xffffffffu, count == 0);
            const unsigned full = __ballot_sync(0xffffffffu, count > 0);
            int end = max(count, 0);
#pragma unroll
            for (int o = 1; o < kSegments; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, end, o);
                if (lane >= o) end += up;
            }
            if (lane < kSegments) sg.row[lane] = row;
            if (count == 0) sg.empty[__popc(empty & below)] = lane;
            if (count > 0) {
                const int k = __popc(full & below);
                sg.slot[k] = lane;
                sg.start[k] = start;
                sg.first[k] = end - count;
            }
            if (lane == kSegments - 1) {
                sg.empties = __popc(empty);
                sg.full = __popc(full);
                sg.items = end;
            }
        }
        __syncthreads();
        const int n = sg.items, full = sg.full;
        for (int i = threadIdx.x; i < n; i += blockDim.x) {
            int k = 0;
            for (int q = 1; q < full; ++q) k = sg.first[q] <= i ? q : k;
            sg.item[i] = g.ws.order[sg.start[k] + i - sg.first[k]];
        }
        if (IN_PLACE && b >= 0 && on)
            for (int k = 0; k < full; ++k)
                stage_unit(own + sg.slot[k] * blockDim.x, bcol + sg.row[sg.slot[k]] * bld);
        __syncthreads();
        if (on) {
            typename Unit<DDT, W>::Raw raw[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (u < n) raw[u] = Unit<DDT, W>::load(dcol + sg.item[u] * dld);
            asm volatile("cp.async.wait_all;" ::: "memory");
            if (!IN_PLACE)
                for (int i = 0; i < sg.empties; ++i) {
                    const int slot = sg.empty[i];
                    float x[W] = {};
                    if (has_base) Unit<GDT, W>::unpack(own[slot * blockDim.x], x);
                    Unit<GDT, W>::store(gcol + sg.row[slot] * gld, x);
                }
            int k = 0, end = full > 1 ? sg.first[1] : n;    // the segment at hand
            float acc[W] = {};
            for (int i0 = 0; i0 < n; i0 += kAhead) {
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int i = i0 + u;
                    if (i >= n) break;
                    float x[W];
                    Unit<DDT, W>::unpack(raw[u], x);
#pragma unroll
                    for (int q = 0; q < W; ++q) acc[q] = __fadd_rn(acc[q], x[q]);
                    if (i + kAhead < n) raw[u] = Unit<DDT, W>::load(dcol + sg.item[i + kAhead] * dld);
                    if (i + 1 == end) {
                        const int slot = sg.slot[k], row = sg.row[slot];
                        if (row >= 0) {
                            float y[W] = {};
                            if (has_base) Unit<GDT, W>::unpack(own[slot * blockDim.x], y);
#pragma unroll
                            for (int q = 0; q < W; ++q) y[q] = __fmaf_rn(g.scale, acc[q], y[q]);
                            Unit<GDT, W>::store(gcol + row * gld, y);
                        } else {
                            store_partial<W>(
                                g.ws.partial + blockIdx.x * g.ws.Dpad + (int64_t)unit * W, acc);
                        }
                        ++k;
                        end = k + 1 < full ? sg.first[k + 1] : n;
#pragma unroll
                        for (int q = 0; q < W; ++q) acc[q] = 0.0f;
                    }
                }
            }
        }
        if (!IN_PLACE || b < 0) return;
        __syncthreads();
    }
}

// Joins the partial rows of each long run, blocks (owner, tile of 32*W
// columns).  A block's warps add consecutive shares of a run's pieces in
// order, then the shares in order.
constexpr int kJoinThreads = 256;

template <int GDT, int W>
__global__ void __launch_bounds__(kJoinThreads) k_emb_join(EmbGrad g)
{
    constexpr int kWarps = kJoinThreads / 32, kAtOnce = 8;   // partial rows
    __shared__ float share[kWarps][32][W];
    pdl_enter();
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int64_t e = ((int64_t)blockIdx.y * 32 + lane) * W;
    const bool on = e < g.D;
    const int owner = blockIdx.x, runs = g.ws.owner[owner].y;
    if (runs == 0) return;
    // its pieces are numbered on from those of the lower owners
    const int before = pieces_before(g.ws, owner);
    const int4* list = g.ws.longs + ((int64_t)owner << kSortLogBins);
    int4 run = list[0];
    for (int r = 0; r < runs; ++r) {
        const int p0 = before + run.w, n = (run.z + g.ws.piece - 1) / g.ws.piece;
        const int i0 = (int)((int64_t)n * wid / kWarps), i1 = (int)((int64_t)n * (wid + 1) / kWarps);
        const int64_t v = run.x;
        if (r + 1 < runs) run = list[r + 1];
        float acc[W] = {}, base[W] = {};
        if (on && wid == 0 && g.base.p != nullptr)
            Unit<GDT, W>::unpack(
                Unit<GDT, W>::load(g.base.p + (v * g.base.ld + e) * bytes_of(GDT)), base);
        if (on)
            for (int i = i0; i < i1; i += kAtOnce) {
                float q[kAtOnce][W];
#pragma unroll
                for (int u = 0; u < kAtOnce; ++u)
                    if (i + u < i1)
                        load_partial<W>(g.ws.partial + (int64_t)(p0 + i + u) * g.ws.Dpad + e, q[u]);
#pragma unroll
                for (int u = 0; u < kAtOnce; ++u)
                    if (i + u < i1)
#pragma unroll
                        for (int j = 0; j < W; ++j) acc[j] = __fadd_rn(acc[j], q[u][j]);
            }
#pragma unroll
        for (int j = 0; j < W; ++j) share[wid][lane][j] = acc[j];
        __syncthreads();
        if (wid == 0 && on) {
            for (int w = 1; w < kWarps; ++w)
#pragma unroll
                for (int j = 0; j < W; ++j) acc[j] = __fadd_rn(acc[j], share[w][lane][j]);
#pragma unroll
            for (int j = 0; j < W; ++j) base[j] = __fmaf_rn(g.scale, acc[j], base[j]);
            Unit<GDT, W>::store(g.dtable.p + (v * g.dtable.ld + e) * bytes_of(GDT), base);
        }
        __syncthreads();
    }
}

// Whether Unit<DT, W> may read the matrix's rows: aligned to W elements
// throughout.
bool aligned(const Mat& m, int64_t D, int W)
{
    const uintptr_t es = m.dt == DPZ_F32 ? 4 : 2;
    return D % W == 0 && m.ld % W == 0 && reinterpret_cast<uintptr_t>(m.p) % (W * es) == 0;
}

constexpr int64_t kMaxGrid = 0x7fffffff;

template <int WDT, int ODT>
cudaError_t embedding_typed(const Mat& table, const Ids& ids, int64_t T, int64_t V, int64_t D,
                            float scale, const Mat& out, cudaStream_t s)
{
    const auto all = [&](int W) { return aligned(table, D, W) && aligned(out, D, W); };
    auto fn = all(8)   ? k_embedding<WDT, ODT, 8>
              : all(4) ? k_embedding<WDT, ODT, 4>
                       : k_embedding<WDT, ODT, 1>;
    const unsigned blocks = (unsigned)((T + kBlock / 32 - 1) / (kBlock / 32));
    return launch_kernel(fn, dim3(blocks), dim3(kBlock), 0, s, true, 0u, table, ids, T, V, D,
                         scale, out);
}

int64_t emb_bins(int64_t V, int log_owners)
{
    return (V + (int64_t(1) << log_owners) - 1) >> log_owners;
}

template <int DDT, int GDT, int W>
cudaError_t rows_typed(const EmbGrad& g, cudaStream_t s)
{
    const int64_t units = (g.D + W - 1) / W, tiles = (units + kBlock - 1) / kBlock;
    const int tile_units = (int)((units + tiles - 1) / tiles);
    const int log_owners = emb_log_owners(g.V);
    const bool in_place = g.base.p == g.dtable.p;
    const int threads = (tile_units + 31) / 32 * 32, group = threads <= 128 && !in_place ? 4 : kSegments;
    const int64_t groups = (emb_bins(g.V, log_owners) + group - 1) / group;
    // in place: blocks for the ids that an owner can expect to have tokens
    const int64_t expect = ((g.T >> log_owners) + group) / group;
    const int64_t per_owner = in_place ? std::min(groups, expect) : groups;
    const int64_t blocks = g.ws.pieces + (per_owner << log_owners);
    if (blocks > kMaxGrid || tiles > 65535) return cudaErrorInvalidConfiguration;
    const size_t smem =
        g.base.p != nullptr ? size_t(group) * threads * sizeof(typename Unit<GDT, W>::Raw) : 0;
    return launch_kernel(in_place ? k_emb_rows<DDT, GDT, W, true> : k_emb_rows<DDT, GDT, W, false>,
                         dim3((unsigned)blocks, (unsigned)tiles), dim3(threads), smem, s, true, 0u, g,
                         tile_units, log_owners, group, (int)per_owner);
}

template <int GDT, int W>
cudaError_t join_typed(const EmbGrad& g, cudaStream_t s)
{
    const unsigned tiles = (unsigned)((g.D + 32 * W - 1) / (32 * W));
    if (tiles > 65535) return cudaErrorInvalidConfiguration;
    return launch_kernel(k_emb_join<GDT, W>, dim3(1u << emb_log_owners(g.V), tiles), dim3(kJoinThreads),
                         0, s, true, 0u, g);
}

// Elements per access: 16 bytes of the wider type.
int grad_width(const EmbGrad& g)
{
    const auto all = [&](int W) {
        return aligned(g.dout, g.D, W) && aligned(g.dtable, g.D, W) &&
               (g.base.p == nullptr || aligned(g.base, g.D, W));
    };
    const bool bf16 = g.dout.dt == DPZ_BF16 && g.dtable.dt == DPZ_BF16;
    return bf16 && all(8) ? 8 : all(4) ? 4 : 1;
}

}  // namespace

cudaError_t launch_embedding(const Mat& table, const Ids& ids, int64_t T, int64_t V, int64_t D,
                             float scale, const Mat& out, cudaStream_t s)
{
    set_last_kernel_name("lm_embedding");
    if (table.dt == DPZ_BF16)
        return out.dt == DPZ_BF16
                   ? embedding_typed<DPZ_BF16, DPZ_BF16>(table, ids, T, V, D, scale, out, s)
                   : embedding_typed<DPZ_BF16, DPZ_F32>(table, ids, T, V, D, scale, out, s);
    return out.dt == DPZ_BF16
               ? embedding_typed<DPZ_F32, DPZ_BF16>(table, ids, T, V, D, scale, out, s)
               : embedding_typed<DPZ_F32, DPZ_F32>(table, ids, T, V, D, scale, out, s);
}

cudaError_t launch_emb_sort(const EmbGrad& g, cudaStream_t s)
{
    set_last_kernel_name("lm_emb_sort");
    const int log_owners = emb_log_owners(g.V), bins = (int)emb_bins(g.V, log_owners);
    const auto bytes = [](int b) { return size_t(kSortWarps) * (kSortHits * sizeof(int2) + b * sizeof(int)); };
    const size_t most = bytes(kSortMaxBins), smem = bytes(bins);
    const dim3 grid(1u << log_owners), block(kSortThreads);
    const auto launch_typed = [&](auto fn, SmemRaisedOn& raised, const auto* ids) {
        const cudaError_t e = raise_smem(raised, reinterpret_cast<const void*>(fn), most);
        if (e != cudaSuccess) return e;
        return launch_kernel(fn, grid, block, smem, s, true, 0u, ids, g.T, g.V, log_owners, bins, g.ws);
    };
    static SmemRaisedOn raised32, raised64;
    return g.ids.it == DPZ_I64
               ? launch_typed(k_emb_sort<int64_t>, raised64, static_cast<const int64_t*>(g.ids.p))
               : launch_typed(k_emb_sort<int>, raised32, static_cast<const int*>(g.ids.p));
}

cudaError_t launch_emb_rows(const EmbGrad& g, cudaStream_t s)
{
    set_last_kernel_name("lm_emb_rows");
    const bool db = g.dout.dt == DPZ_BF16, gb = g.dtable.dt == DPZ_BF16;
    switch (grad_width(g)) {
    case 8:
        return rows_typed<DPZ_BF16, DPZ_BF16, 8>(g, s);
    case 4:
        return db ? (gb ? rows_typed<1, 1, 4>(g, s) : rows_typed<1, 0, 4>(g, s))
                  : (gb ? rows_typed<0, 1, 4>(g, s) : rows_typed<0, 0, 4>(g, s));
    default:
        return db ? (gb ? rows_typed<1, 1, 1>(g, s) : rows_typed<1, 0, 1>(g, s))
                  : (gb ? rows_typed<0, 1, 1>(g, s) : rows_typed<0, 0, 1>(g, s));
    }
}

cudaError_t launch_emb_join(const EmbGrad& g, cudaStream_t s)
{
    set_last_kernel_name("lm_emb_join");
    const bool gb = g.dtable.dt == DPZ_BF16;
    switch (grad_width(g)) {
    case 8:
        return join_typed<DPZ_BF16, 8>(g, s);
    case 4:
        return gb ? join_typed<1, 4>(g, s) : join_typed<0, 4>(g, s);
    default:
        return gb ? join_typed<1, 1>(g, s) : join_typed<0, 1>(g, s);
    }
}

}  // namespace dpz
