// Embedding lookup with scaling, and its gradient by sorted tokens.
#include "bulk.cuh"
#include "device.cuh"
#include "internal.h"
#include "lm.h"

namespace dpz {

namespace {

__device__ __forceinline__ int64_t load_id(const Ids& ids, int64_t i)
{
    return ids.it == DPZ_I64 ? static_cast<const int64_t*>(ids.p)[i]
                             : (int64_t) static_cast<const int*>(ids.p)[i];
}

// An id as an int, -1 where it names none of V tokens (V < 2^30).
__device__ __forceinline__ int load_token(const Ids& ids, int64_t i, int64_t V)
{
    const int64_t v = load_id(ids, i);
    return v >= 0 && v < V ? (int)v : -1;
}

// One access unit of a row: W = 8 elements in one 16- or 32-byte word
// (aligned rows whose length is a multiple of 8), or W = 1 element.
template <int DT, int W>
struct Unit;

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

// One warp per row: out[t] = R(scale * table[ids[t]]).
template <int WDT, int ODT, int W>
__global__ void __launch_bounds__(kBlock)
    k_embedding(Mat table, Ids ids, int64_t T, int64_t V, int64_t D, float scale, Mat out)
{
    pdl_enter();
    const int64_t t = global_warp();
    if (t >= T) return;
    const int lane = threadIdx.x & 31;
    const int v = load_token(ids, t, V);
    const char* src = table.p + (int64_t)(v < 0 ? 0 : v) * table.ld * bytes_of(WDT);
    char* dst = out.p + t * out.ld * bytes_of(ODT);
    for (int64_t e = lane * W; e < D; e += 32 * W) {
        float x[W] = {};
        if (v >= 0) {
            Unit<WDT, W>::unpack(Unit<WDT, W>::load(src + e * bytes_of(WDT)), x);
#pragma unroll
            for (int i = 0; i < W; ++i) x[i] = __fmul_rn(x[i], scale);
        }
        Unit<ODT, W>::store(dst + e * bytes_of(ODT), x);
    }
}

// ------------------------------------------------------------ gradient
//
// The tokens are put in order of (id, position), so that every table row's
// terms stand together and are added in order of position: the sum is the
// same from run to run, where adding rows with atomics is not.

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortMaxBins = 1024;   // ids one block owns at most

// Block b owns the ids v with v % owners == b, which spreads the frequent low
// ids of a byte-pair vocabulary over the blocks.  Every block reads all T
// ids, so no block waits for another one: it counts the ids of lower owners
// (where its part of the order begins) and, per warp, its own ids; the
// prefix sums of those counts place each token.  Warps take consecutive
// ranges of positions, so the order within an id is that of positions.
__global__ void __launch_bounds__(kSortThreads)
    k_emb_sort(Ids ids, int64_t T, int64_t V, int log_owners, int bins, EmbWs ws)
{
    extern __shared__ int hist[];            // [kSortWarps][bins]
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
    int less = 0;
    for (int64_t i = lo + lane; i < hi; i += 32) {
        const int v = load_token(ids, i, V);
        if (v < 0) continue;
        const int o = v & (owners - 1);
        less += o < me;
        if (o == me) atomicAdd(&mine[v >> log_owners], 1);
    }
    less = __reduce_add_sync(0xffffffffu, less);
    if (lane == 0) warp_tot[wid] = less;
    __syncthreads();
    if (wid == 0) {
        const int s = __reduce_add_sync(0xffffffffu, warp_tot[lane]);
        if (lane == 0) s_base = s;
    }
    __syncthreads();
    // thread k < bins: id k's count over the warps, then the ids' prefix sum
    int total = 0;
    if (threadIdx.x < bins)
        for (int w = 0; w < kSortWarps; ++w) total += hist[w * bins + threadIdx.x];
    int incl = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) warp_tot[wid] = incl;
    __syncthreads();
    if (wid == 0) {
        int x = warp_tot[lane];
        int acc = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, acc, o);
            if (lane >= o) acc += up;
        }
        warp_tot[lane] = acc - x;
    }
    __syncthreads();
    if (threadIdx.x < bins) {
        int at = s_base + warp_tot[wid] + incl - total;
        const int64_t v = ((int64_t)threadIdx.x << log_owners) + me;
        if (v < V) {
            ws.start[v] = at;
            ws.count[v] = total;
        }
        if (me == owners - 1 && threadIdx.x == bins - 1) *ws.nvalid = at + total;
        for (int w = 0; w < kSortWarps; ++w) {
            const int n = hist[w * bins + threadIdx.x];
            hist[w * bins + threadIdx.x] = at;
            at += n;
        }
    }
    __syncthreads();
    for (int64_t i0 = lo; i0 < hi; i0 += 32) {
        const int64_t i = i0 + lane;
        const int v = i < hi ? load_token(ids, i, V) : -1;
        const bool hit = v >= 0 && (v & (owners - 1)) == me;
        const unsigned m = __ballot_sync(0xffffffffu, hit);
        if (m == 0) continue;
        if (hit) {
            const int k = v >> log_owners;
            const unsigned same = __match_any_sync(m, k);
            const int rank = __popc(same & ((1u << lane) - 1u));
            const int at = mine[k];
            ws.order[at + rank] = (int)i;
            __syncwarp(m);
            if (rank == 0) mine[k] = at + __popc(same);
        }
        __syncwarp();
    }
}

// Adds scale-free rows order[a..b) of dout, at most 32 of them, to acc: the
// columns e..e+W of each, in order.
template <int DDT, int W>
__device__ __forceinline__ void sum_rows(const EmbGrad& g, int a, int n, int64_t e, bool on,
                                         float acc[W])
{
    const int lane = threadIdx.x & 31;
    const int mine = lane < n ? g.ws.order[a + lane] : 0;
    for (int i = 0; i < n; ++i) {
        const int64_t t = __shfl_sync(0xffffffffu, mine, i);
        if (on) {
            float x[W];
            Unit<DDT, W>::unpack(
                Unit<DDT, W>::load(g.dout.p + (t * g.dout.ld + e) * bytes_of(DDT)), x);
#pragma unroll
            for (int j = 0; j < W; ++j) acc[j] = __fadd_rn(acc[j], x[j]);
        }
    }
}

// dtable[v, e..e+W) from the sum of its terms.
template <int GDT, int W>
__device__ __forceinline__ void finish_row(const EmbGrad& g, int64_t v, int64_t e,
                                           const float acc[W])
{
    float y[W] = {};
    if (g.base.p != nullptr)
        Unit<GDT, W>::unpack(Unit<GDT, W>::load(g.base.p + (v * g.base.ld + e) * bytes_of(GDT)), y);
#pragma unroll
    for (int j = 0; j < W; ++j) y[j] = __fmaf_rn(g.scale, acc[j], y[j]);
    Unit<GDT, W>::store(g.dtable.p + (v * g.dtable.ld + e) * bytes_of(GDT), y);
}

// The run that the sorted position p belongs to, and its token.
__device__ __forceinline__ int token_at(const EmbGrad& g, int p)
{
    return load_token(g.ids, g.ws.order[p], g.V);
}

// One warp per (piece or table row, tile of 32*W columns).  The first
// pieces*tiles units sum the pieces of long runs (more than kEmbPiece terms)
// into partial rows; the others finish the table's rows with at most that
// many terms.  A piece meets at most two long runs: the one its first
// position is in (partial row 0) and one that begins inside it (row 1).
template <int DDT, int GDT, int W>
__global__ void __launch_bounds__(kBlock) k_emb_rows(EmbGrad g, int tiles)
{
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const int64_t unit = global_warp();
    const int64_t row = unit / tiles - g.ws.pieces;
    const int64_t e = ((unit % tiles) * 32 + lane) * W;
    const bool on = e < g.D;
    if (row >= g.V) return;
    if (row >= 0) {
        const int n = g.ws.count[row];
        if (n > kEmbPiece || (n == 0 && g.base.p == g.dtable.p)) return;
        float acc[W] = {};
        if (n > 0) sum_rows<DDT, W>(g, g.ws.start[row], n, e, on, acc);
        if (on) finish_row<GDT, W>(g, row, e, acc);
        return;
    }
    const int64_t c = row + g.ws.pieces;
    const int nvalid = *g.ws.nvalid;
    const int64_t p0 = c * kEmbPiece;
    if (p0 >= nvalid) return;
    const int p1 = (int)min((int64_t)nvalid, p0 + kEmbPiece);
    const int a = token_at(g, (int)p0), b = token_at(g, p1 - 1);
    float* part = g.ws.partial + 2 * c * g.ws.Dpad + e;
    if (g.ws.count[a] > kEmbPiece) {
        float acc[W] = {};
        const int end = min(p1, g.ws.start[a] + g.ws.count[a]);
        sum_rows<DDT, W>(g, (int)p0, end - (int)p0, e, on, acc);
        if (on)
#pragma unroll
            for (int j = 0; j < W; ++j) part[j] = acc[j];
    }
    if (b != a && g.ws.count[b] > kEmbPiece) {
        float acc[W] = {};
        const int from = g.ws.start[b];
        sum_rows<DDT, W>(g, from, p1 - from, e, on, acc);
        if (on)
#pragma unroll
            for (int j = 0; j < W; ++j) part[g.ws.Dpad + j] = acc[j];
    }
}

// Joins the partial rows of each long run, one block per (piece, tile of 32*W
// columns): the block of the piece in which the run begins.  Its warps add
// consecutive shares of the pieces in order, then the shares in order.
template <int GDT, int W>
__global__ void __launch_bounds__(kBlock) k_emb_join(EmbGrad g)
{
    constexpr int kWarps = kBlock / 32;
    __shared__ float share[kWarps][32][W];
    pdl_enter();
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int64_t c = blockIdx.x;
    const int64_t e = ((int64_t)blockIdx.y * 32 + lane) * W;
    const bool on = e < g.D;
    const int nvalid = *g.ws.nvalid;
    const int64_t p0 = c * kEmbPiece;
    if (p0 >= nvalid) return;
    const int p1 = (int)min((int64_t)nvalid, p0 + kEmbPiece);
    const int v = token_at(g, p1 - 1);       // the only run that can begin here and be long
    const int start = g.ws.start[v], count = g.ws.count[v];
    if (count <= kEmbPiece || start < p0) return;
    const int64_t last = (start + count - 1) / kEmbPiece;
    const int n = (int)(last - c) + 1;
    const int i0 = (int)((int64_t)n * wid / kWarps), i1 = (int)((int64_t)n * (wid + 1) / kWarps);
    float acc[W] = {};
    if (on)
        for (int i = i0; i < i1; ++i) {
            // the run's first piece is its row 1 unless it begins with the piece
            const float* q = g.ws.partial +
                             (2 * (c + i) + (i == 0 && start > p0 ? 1 : 0)) * g.ws.Dpad + e;
#pragma unroll
            for (int j = 0; j < W; ++j) acc[j] = __fadd_rn(acc[j], q[j]);
        }
#pragma unroll
    for (int j = 0; j < W; ++j) share[wid][lane][j] = acc[j];
    __syncthreads();
    if (wid != 0 || !on) return;
    for (int w = 1; w < kWarps; ++w)
#pragma unroll
        for (int j = 0; j < W; ++j) acc[j] = __fadd_rn(acc[j], share[w][lane][j]);
    finish_row<GDT, W>(g, v, e, acc);
}

// Rows that Unit<DT, 8> may read: aligned to 8 elements throughout.
bool wide(const Mat& m, int64_t D)
{
    const uintptr_t es = m.dt == DPZ_F32 ? 4 : 2;
    return D % 8 == 0 && m.ld % 8 == 0 && reinterpret_cast<uintptr_t>(m.p) % (8 * es) == 0;
}

constexpr int64_t kMaxGrid = 0x7fffffff;

template <int WDT, int ODT>
cudaError_t embedding_typed(const Mat& table, const Ids& ids, int64_t T, int64_t V, int64_t D,
                            float scale, const Mat& out, cudaStream_t s)
{
    auto fn = wide(table, D) && wide(out, D) ? k_embedding<WDT, ODT, 8> : k_embedding<WDT, ODT, 1>;
    const unsigned blocks = (unsigned)((T + kBlock / 32 - 1) / (kBlock / 32));
    return launch_kernel(fn, dim3(blocks), dim3(kBlock), 0, s, true, 0u, table, ids, T, V, D,
                         scale, out);
}

template <int DDT, int GDT, int W>
cudaError_t rows_typed(const EmbGrad& g, cudaStream_t s)
{
    const int tiles = (int)((g.D + 32 * W - 1) / (32 * W));
    const int64_t blocks = ((g.V + g.ws.pieces) * tiles + kBlock / 32 - 1) / (kBlock / 32);
    if (blocks > kMaxGrid) return cudaErrorInvalidConfiguration;
    return launch_kernel(k_emb_rows<DDT, GDT, W>, dim3((unsigned)blocks), dim3(kBlock), 0, s, true,
                         0u, g, tiles);
}

template <int GDT, int W>
cudaError_t join_typed(const EmbGrad& g, cudaStream_t s)
{
    const unsigned tiles = (unsigned)((g.D + 32 * W - 1) / (32 * W));
    if (tiles > 65535) return cudaErrorInvalidConfiguration;
    return launch_kernel(k_emb_join<GDT, W>, dim3((unsigned)g.ws.pieces, tiles), dim3(kBlock), 0, s,
                         true, 0u, g);
}

bool wide_grad(const EmbGrad& g)
{
    return wide(g.dout, g.D) && wide(g.dtable, g.D) && (g.base.p == nullptr || wide(g.base, g.D));
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
    static SmemRaised raised;
    set_last_kernel_name("lm_emb_sort");
    int log_owners = 7;   // 128 blocks, one wave, until a block would own too many ids
    while ((g.V >> log_owners) >= kSortMaxBins) ++log_owners;
    const int bins = (int)((g.V + (int64_t(1) << log_owners) - 1) >> log_owners);
    const size_t most = size_t(kSortWarps) * kSortMaxBins * sizeof(int);
    const cudaError_t e = allow_smem(raised, reinterpret_cast<const void*>(k_emb_sort), most);
    if (e != cudaSuccess) return e;
    return launch_kernel(k_emb_sort, dim3(1u << log_owners), dim3(kSortThreads),
                         size_t(kSortWarps) * bins * sizeof(int), s, true, 0u, g.ids, g.T, g.V,
                         log_owners, bins, g.ws);
}

cudaError_t launch_emb_rows(const EmbGrad& g, cudaStream_t s)
{
    set_last_kernel_name("lm_emb_rows");
    const bool w = wide_grad(g);
    const bool db = g.dout.dt == DPZ_BF16, gb = g.dtable.dt == DPZ_BF16;
    if (w)
        return db ? (gb ? rows_typed<1, 1, 8>(g, s) : rows_typed<1, 0, 8>(g, s))
                  : (gb ? rows_typed<0, 1, 8>(g, s) : rows_typed<0, 0, 8>(g, s));
    return db ? (gb ? rows_typed<1, 1, 1>(g, s) : rows_typed<1, 0, 1>(g, s))
              : (gb ? rows_typed<0, 1, 1>(g, s) : rows_typed<0, 0, 1>(g, s));
}

cudaError_t launch_emb_join(const EmbGrad& g, cudaStream_t s)
{
    set_last_kernel_name("lm_emb_join");
    const bool gb = g.dtable.dt == DPZ_BF16;
    if (wide_grad(g)) return gb ? join_typed<1, 8>(g, s) : join_typed<0, 8>(g, s);
    return gb ? join_typed<1, 1>(g, s) : join_typed<0, 1>(g, s);
}

}  // namespace dpz
