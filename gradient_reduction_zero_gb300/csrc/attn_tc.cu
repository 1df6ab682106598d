// Attention and its gradient on the tensor cores, for bf16 tensors whose
// addresses and strides are multiples of 16 bytes and heads of a multiple of 8
// elements up to 128.  The formulas are at the top of attn_any.cu.
//
// Tiles of 128 rows by 128 keys.  Each block is made of warps with one task:
// one issues the TMA loads, one the products, and the others each hold 32 rows
// of a tile, a thread to a row, so that a row's maximum and sum need no exchange.
// Scores and accumulators are in tensor memory; probabilities and score gradients
// go back there in bf16 as the left operand of the next product.  What
// would lie in a tile beyond a sequence's end is not zero in memory: it is masked
// where it is a column of scores, cleared in shared memory where a product
// sums over it, and otherwise a row of its own that is not stored.
//
// Measured, one sequence of 8,192 tokens of 16 + 4 heads of 128 without a mask: forward 429 us
// (1,281 TFLOP/s), queries' gradient 560 (1,473), keys' and values' 761 (1,446).  8 x 1,024
// tokens of 25 heads of 64, causal: 49 us, and 165 us for both gradients.  Bound by the
// chain of a tile: products, tensor memory to registers, exponentials, and back.
#include <cmath>
#include <type_traits>

#include "attn.h"
#include "bulk.cuh"
#include "device.cuh"
#include "lm_shape.h"
#include "pairs.cuh"
#include "tc.cuh"

namespace dpz {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ unsigned g_tc_lost;   // a bounded wait ran out since the last look

__device__ __forceinline__ float ex2(float u)
{
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(u));
    return e;
}

// The end of a block: after a wait that ran out, time for what is in flight.
__device__ __forceinline__ void tc_finish(volatile int* lost, uint32_t tmem, bool frees)
{
    __syncthreads();
    if (*lost != 0) {
        if (threadIdx.x == 0) atomicExch(&g_tc_lost, 1u);
        const long long t0 = clock64();
        while (clock64() - t0 < kWaitLimitCycles / 8) {}
        __syncthreads();
    }
    tc_fence_after();
    if (frees) tmem_free(tmem);
}

// The maps of a call's tensors: blocks of 64 elements of `heads` heads of
// `tokens` tokens.
struct Maps {
    CUtensorMap q, k, v, dout;
};

// Heads that share a tile in the forward pass, tokens of a tile.
struct Packing {
    int heads, tokens;
};

// A 32-byte store whose line stays in L2 for the next kernel.
__device__ __forceinline__ void st32_keep(void* p, const U8& v)
{
    asm volatile("st.global.v8.u32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v.x[0]),
                 "r"(v.x[1]), "r"(v.x[2]), "r"(v.x[3]), "r"(v.x[4]), "r"(v.x[5]), "r"(v.x[6]),
                 "r"(v.x[7])
                 : "memory");
}

// Whether every row of x begins on a boundary of 32 bytes.
__device__ __forceinline__ bool wide_rows(const Heads& x)
{
    return ((reinterpret_cast<uintptr_t>(x.p) | (uintptr_t)(2 * x.ld) | (uintptr_t)(2 * x.hs)) & 31) == 0;
}

// Columns [0, n) of the warp's rows (n <= COLS, a multiple of 8) times k as bf16 to rows of
// a tensor in memory.  PART columns at a time; read() is called when the last are in
// registers.  wide: the rows are on boundaries of 32 bytes.
template <int COLS, int PART, class F>
__device__ __forceinline__ void store_row(uint32_t tmem, int n, float k, char* row, bool live,
                                          bool wide, F&& read)
{
#pragma unroll
    for (int c0 = 0; c0 < COLS; c0 += PART) {
        uint32_t r[PART];
#pragma unroll
        for (int c = 0; c < PART; c += 32)
            if (c0 + c < n) tmem_load32(tmem + c0 + c, r + c);
        tmem_wait(r);
        if (c0 + PART >= COLS) read();
#pragma unroll
        for (int c = 0; c < PART / 2; ++c)
            r[c] = pack_bf16x2(__uint_as_float(r[2 * c]) * k, __uint_as_float(r[2 * c + 1]) * k);
        if (!live) continue;
        if (wide && n % 16 == 0) {
#pragma unroll
            for (int c = 0; c < PART; c += 16)
                if (c0 + c < n) {
                    U8 w;
#pragma unroll
                    for (int e = 0; e < 8; ++e) w.x[e] = r[c / 2 + e];
                    st32_keep(row + 2 * (c0 + c), w);
                }
        } else {
#pragma unroll
            for (int c = 0; c < PART; c += 8)
                if (c0 + c < n)
                    *reinterpret_cast<uint4*>(row + 2 * (c0 + c)) =
                        make_uint4(r[c / 2], r[c / 2 + 1], r[c / 2 + 2], r[c / 2 + 3]);
        }
    }
}

__device__ __forceinline__ void zero_row(int n, char* row, bool live)
{
    if (!live) return;
    for (int c = 0; c < n; c += 8)
        *reinterpret_cast<uint4*>(row + 2 * c) = make_uint4(0, 0, 0, 0);
}

__device__ __forceinline__ char* row_of(const Heads& x, int64_t t, int h)
{
    return x.p + 2 * (t * x.ld + (int64_t)h * x.hs);
}

// ------------------------------------------------------------ work
//
// Blocks stay, one per SM, and take items (a tile of a sequence and its heads) in turn, the
// longest first.  The loading warp finds an item's sequence and passes it on
// through a small ring, so that the search, the loads and the first scores of the next
// item run behind the softmax and the stores of this one.

struct Item {
    int64_t q0, k0;
    int nq, nk, row0, head;
    int tiles[2];      // of the other axis, for each tile of the block; [0] < 0: no more items
    int first;         // the first of them (forward)
};

// The block's item of a round.  Where items are in order of length (find_tile sorts sequences of
// equal length and few packed ones), there and back, so that the block with the longest
// item of one round has the shortest of the next: 8 x 1,024 tokens of 32 + 8 heads of 128,
// gradients of keys and values, 124 us against 150 round after round.  Many packed sequences
// follow one another, and there and back sorts nothing.  (Gradient of nine packed sequences of
// 32 + 8 heads of 128: 1,732 us by position, 1,813 by sequence, 5 % more there and back.)
__device__ __forceinline__ int64_t item_of_round(int64_t round, const AttnArgs& a)
{
    const bool sorted = a.cu_q == nullptr || a.B <= kSortedSeqs;
    const unsigned b = sorted && round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
    return round * gridDim.x + b;
}

constexpr int kRing = 4;

struct Ring {
    uint64_t full[kRing], empty[kRing];
    Item item[kRing];
};

__device__ __forceinline__ void ring_init(Ring& r, uint32_t readers)
{
    for (int i = 0; i < kRing; ++i) {
        mbar_init(&r.full[i], 1);
        mbar_init(&r.empty[i], readers);
    }
}

// A position in a ring of N places that are filled and emptied in turn: its place, and
// the parity of the place's phase.
template <int N>
struct Turn {
    int at = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next()
    {
        if (++at == N) {
            at = 0;
            parity ^= 1;
        }
    }
};

// Puts an item (all lanes have it); false if the wait ran out.
__device__ __forceinline__ bool ring_put(Ring& r, Turn<kRing>& turn, const Item& item,
                                         volatile int* lost)
{
    // a place is free at first: the parity of the phase before the first is 1
    if (!tc_wait_warp(&r.empty[turn.at], turn.parity ^ 1, lost)) return false;
    if ((threadIdx.x & 31) == 0) {
        r.item[turn.at] = item;
        mbar_arrive(&r.full[turn.at]);
    }
    __syncwarp();
    turn.next();
    return true;
}

// Takes the next item, by a warp; false at the end.
__device__ __forceinline__ bool ring_take(Ring& r, Turn<kRing>& turn, Item& item, volatile int* lost)
{
    if (!tc_wait_warp(&r.full[turn.at], turn.parity, lost)) return false;
    const Item& x = r.item[turn.at];
    item = {x.q0, x.k0, uniform(x.nq), uniform(x.nk), uniform(x.row0), uniform(x.head),
            {uniform(x.tiles[0]), uniform(x.tiles[1])}, uniform(x.first)};
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&r.empty[turn.at]);
    turn.next();
    return item.tiles[0] >= 0;
}

// ------------------------------------------------------------ forward
//
// A block has two tiles of 128 rows, which share the keys and values it loads:
// while the softmax warps of one are at work, the tensor cores have the other's
// products.  A tile's rows are tokens times the query heads of one key head
// (row = token * heads + head), where these divide 128 well enough, so that grouped
// heads share keys and few queries fill a tile.
//
// The softmax takes no maximum as long as none is needed: a row's scores are summed
// against a shift of 0 as they come.  Only where a tile's sum passes 2^16, or the row's
// sum stays below 2^-30, is the tile read again, its maximum made the shift and
// what the row has so far scaled.  Between these bounds nothing is lost: fp32 sums and
// bf16 probabilities are as exact there as near 1, and what falls below fp32's range is
// below 2^-96 of the sum.
//
// Tensor memory, in columns of 32 bits: scores of the tiles at 0 and 128; outputs
// at 256 and 256 + 64 BLOCKS; probabilities at 384 and 448, or, with 128 columns of
// outputs, over the scores.

constexpr int kFwdThreads = 384;    // 8 softmax warps, loads, products, two idle
// Registers of a thread, of the 168 that each is launched with: 2 x 128 x 208 + 128 x 88 =
// 384 x 168.
constexpr int kComputeRegs = 208, kOtherRegs = 88;

template <int BLOCKS>
struct FwdShape {
    static constexpr int kTile = BLOCKS * kTcBlock;
    static constexpr int kQs = BLOCKS == 1 ? 2 : 1;       // pairs of query tiles
    static constexpr int kStages = BLOCKS == 1 ? 3 : 2;   // of keys, and of values
    static constexpr int kQ = 0, kK = kQs * 2 * kTile, kV = kK + kStages * kTile;
    static constexpr int kBars = kV + kStages * kTile;
    static constexpr int kBytes = kBars + 1024 + 1024;    // the base is rounded up to 1024
    static constexpr bool kOver = BLOCKS == 2;            // probabilities over the scores
};

struct FwdBars {
    Ring ring;
    uint64_t q_full[2], q_empty[2], k_full[3], k_empty[3], v_full[3], v_empty[3];
    uint64_t s_full[2], p_full[2], o_done[2], o_free[2], parts_done;
    uint32_t tmem;
    int lost;
};
static_assert(sizeof(FwdBars) <= 1024, "the barriers' place");

template <int BLOCKS>
__device__ __forceinline__ uint32_t fwd_p(uint32_t tmem, int i)
{
    return FwdShape<BLOCKS>::kOver ? tmem + 128 * i : tmem + 384 + 64 * i;
}

// The largest score of each row among the 128 columns below `most`.
__device__ __forceinline__ float tile_max(uint32_t at, int most)
{
    float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint32_t s[32];
        tmem_load32(at + 32 * c, s);
        tmem_wait(s);
#pragma unroll
        for (int e = 0; e < 32; ++e)
            m[e & 3] = fmaxf(m[e & 3], 32 * c + e < most ? __uint_as_float(s[e]) : -INFINITY);
    }
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// Scales `width` columns of the warp's rows.
__device__ __forceinline__ void scale_rows(uint32_t at, int width, float k)
{
    for (int c = 0; c < width; c += 32) {
        uint32_t o[32];
        tmem_load32(at + c, o);
        tmem_wait(o);
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * k);
        tmem_store32(at + c, o);
    }
}

// Probabilities of 32 columns, in pairs, and what they add to the sums.
__device__ __forceinline__ void exp32(const uint32_t* s, F2 cc, F2 mm, F2 sum[2], uint32_t* p)
{
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const F2 u = fma2((F2)s[2 * e + 1] << 32 | s[2 * e], cc, mm);
        const float x = ex2(lo2(u)), y = ex2(hi2(u));
        sum[e & 1] = add2(sum[e & 1], pack2(x, y));
        p[e] = pack_bf16x2(x, y);
    }
}

// The same of a tile's 128 columns; EDGE: of those below `most`, in the whole warp's or in
// this row's view.
template <bool EDGE>
__device__ __forceinline__ void tile_exp(uint32_t at, int most, F2 cc, F2 mm, F2 sum[2], uint32_t* p)
{
    uint32_t s[2][32];
    tmem_load32(at, s[0]);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        tmem_wait(s[c & 1]);
        if (c < 3) tmem_load32(at + 32 * (c + 1), s[(c + 1) & 1]);
        if (EDGE) {
            if (!__any_sync(0xffffffffu, 32 * c < most)) {       // nothing to see
#pragma unroll
                for (int e = 0; e < 16; ++e) p[16 * c + e] = 0;
                continue;
            }
#pragma unroll
            for (int e = 0; e < 32; ++e)
                if (32 * c + e >= most) s[c & 1][e] = 0xff800000u;
        }
        exp32(s[c & 1], cc, mm, sum, p + 16 * c);
    }
}

// Few queries against many keys: the blocks of a cluster have parts of the keys, and leave
// each row's unscaled output, shift and sum in their shared memory (where the operands
// were); then each block joins its share of the rows.  Rows are 4 floats apart from
// multiples of the banks.
template <int BLOCKS>
struct SplitShape {
    static constexpr int kStride = 64 * BLOCKS + 4;
    static constexpr int kStats = 256 * kStride * 4;    // bytes before 256 shifts and 256 sums
    static_assert(kStats + 2048 <= FwdShape<BLOCKS>::kBars, "within the operands' place");
};

template <int BLOCKS>
__device__ __forceinline__ void split_put(char* smem, int row, uint32_t o_at, int tiles, float shift,
                                          float sum, uint64_t* done, volatile int* lost)
{
    using P = SplitShape<BLOCKS>;
    // both tiles' products have read the operands (each warp has waited for its tile's)
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(done);
    if (!tc_wait_warp(done, 0, lost)) tiles = -1;
    float* o = reinterpret_cast<float*>(smem) + row * P::kStride;
    float* stats = reinterpret_cast<float*>(smem + P::kStats);
    stats[row] = shift;
    stats[256 + row] = tiles < 0 ? __int_as_float(0x7fc00000) : tiles > 0 ? sum : 0.0f;
    if (tiles <= 0) return;
    tc_fence_after();
#pragma unroll
    for (int c = 0; c < 64 * BLOCKS; c += 32) {
        uint32_t r[32];
        tmem_load32(o_at + c, r);
        tmem_wait(r);
#pragma unroll
        for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<uint4*>(o + c + e) = make_uint4(r[e], r[e + 1], r[e + 2], r[e + 3]);
    }
}

// A float of another block of the cluster, by its address in this one.
__device__ __forceinline__ float of_block(const float* p, int block)
{
    uint32_t at;
    float x;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(block));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(at) : "memory");
    return x;
}

template <int BLOCKS>
__device__ __forceinline__ void split_join(char* smem, const Ring& ring, const AttnArgs& a,
                                           const Packing& pk, int parts)
{
    using P = SplitShape<BLOCKS>;
    cluster_arrive_release();
    cluster_wait();
    const Item& m = ring.item[0];
    const int lane = threadIdx.x & 31, rank = (int)blockIdx.x % parts;
    const float* o = reinterpret_cast<const float*>(smem);
    const float* stats = reinterpret_cast<const float*>(smem + P::kStats);
    for (int at = rank * (kFwdThreads / 32) + (int)(threadIdx.x >> 5); m.tiles[0] >= 0 && at < 256;
         at += parts * (kFwdThreads / 32)) {
        const int i = at >> 7, r = at & 127, row = m.row0 + i * pk.tokens + r / pk.heads;
        if (r >= pk.heads * pk.tokens || row >= m.nq) continue;
        // lane c has part c's shift and sum (a NaN sum takes part)
        float shift = -INFINITY, sum = 0.0f;
        if (lane < parts) {
            sum = of_block(stats + 256 + at, lane);
            if (sum != 0.0f) shift = of_block(stats + at, lane);
        }
        float top = shift;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
        const float weight = sum != 0.0f ? ex2(shift - top) : 0.0f;
        float total = sum * weight;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) total += __shfl_xor_sync(0xffffffffu, total, k);
        const float inv = total == 0.0f ? 0.0f : 1.0f / total;
        float y[2 * BLOCKS] = {};
        for (int c = 0; c < parts; ++c) {
            const float k = __shfl_sync(0xffffffffu, weight, c);
            if (k == 0.0f) continue;
#pragma unroll
            for (int e = 0; e < 2 * BLOCKS; ++e)
                if (lane + 32 * e < a.D)
                    y[e] = fmaf(of_block(o + at * P::kStride + lane + 32 * e, c), k, y[e]);
        }
        const int head = m.head + r % pk.heads;
        __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(row_of(a.out, m.q0 + row, head));
#pragma unroll
        for (int e = 0; e < 2 * BLOCKS; ++e)
            if (lane + 32 * e < a.D) out[lane + 32 * e] = __float2bfloat16_rn(y[e] * inv);
        if (a.lse != nullptr && lane == 0)
            a.lse[(int64_t)head * a.Tq + m.q0 + row] =
                total == 0.0f ? -INFINITY : (top + log2f(total)) * kLn2;
    }
    // no block leaves while another may read from it
    cluster_arrive_release();
    cluster_wait();
}

template <int BLOCKS, bool SPLIT>
__global__ void __launch_bounds__(kFwdThreads, 1)
k_attn_tc(const __grid_constant__ Maps maps, const __grid_constant__ AttnArgs a, Packing pk,
          int pairs, int64_t items, int parts)
{
    using S = FwdShape<BLOCKS>;
    extern __shared__ char smem_raw[];
    char* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    FwdBars& bar = *reinterpret_cast<FwdBars*>(smem + S::kBars);
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        ring_init(bar.ring, 9);
        bar.ring.item[0].tiles[0] = -1;
        mbar_init(&bar.parts_done, 8);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.q_full[i], 1);
            mbar_init(&bar.q_empty[i], 1);
            mbar_init(&bar.s_full[i], 1);
            mbar_init(&bar.p_full[i], 4);
            mbar_init(&bar.o_done[i], 1);
            mbar_init(&bar.o_free[i], 4);
        }
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&bar.k_full[i], 1);
            mbar_init(&bar.k_empty[i], 1);
            mbar_init(&bar.v_full[i], 1);
            mbar_init(&bar.v_empty[i], 1);
        }
        bar.lost = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        tma_prefetch(&maps.q);
        tma_prefetch(&maps.k);
        tma_prefetch(&maps.v);
    }
    pdl_wait_prior();
    // before the next kernel may be placed beside this block and ask for its own
    if (warp == 9) tmem_alloc(&bar.tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_launch_dependents();
    volatile int* lost = &bar.lost;
    const uint32_t tmem = (uint32_t)uniform((int)bar.tmem);
    const int groups = a.Hq / pk.heads;           // of heads that share a tile
    const int ksteps = (a.D + 15) / 16, width = ksteps * 16;
    Turn<kRing> turn;

    if (warp == 8) {
        // ---- items and loads
        set_registers_down<kOtherRegs>();
        const uint32_t q_bytes = (uint32_t)(pk.heads * pk.tokens) * 128 * BLOCKS;
        Turn<S::kQs> qt;
        Turn<S::kStages> kt;
        bool going = true;
        Item m{};
        // in parts: one item for the blocks of a cluster
        for (int64_t round = 0; round * (SPLIT ? 1 << 30 : gridDim.x) < items && going; ++round) {
            const int64_t w = SPLIT ? blockIdx.x / parts : item_of_round(round, a);
            if (w >= items) continue;
            // the tiles at the end of a sequence see the most keys and go first
            const int tile = (int)(w / groups);
            const Tile t = find_tile(a, pairs - 1 - tile, 2 * pk.tokens, false);
            if (!t.any) continue;
            m = {t.q0, t.k0, t.nq, t.nk, t.row0, (int)(w - (int64_t)tile * groups) * pk.heads, {0, 0}, 0};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int row0 = t.row0 + i * pk.tokens;
                const int end = row0 >= t.nq ? 0
                                : !a.causal  ? t.nk
                                             : max(0, min(t.nk, min(row0 + pk.tokens, t.nq) + t.nk - t.nq));
                m.tiles[i] = (end + kTcRows - 1) / kTcRows;
            }
            if (SPLIT) {
                const int all = max(m.tiles[0], m.tiles[1]), each = (all + parts - 1) / parts;
                m.first = min(all, (int)(blockIdx.x % parts) * each);
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    m.tiles[i] = max(0, min(m.tiles[i], m.first + each) - m.first);
            }
            going = ring_put(bar.ring, turn, m, lost);
            const int n = max(m.tiles[0], m.tiles[1]);
            if (!going || n == 0) continue;
            if (lane == 0) {
                going = tc_wait(&bar.q_empty[qt.at], qt.parity ^ 1, lost);
                const int hk = m.head / (a.Hq / a.Hk);
                if (going) {
                    mbar_expect_tx(&bar.q_full[qt.at], q_bytes * ((m.tiles[0] > 0) + (m.tiles[1] > 0)));
                    for (int i = 0; i < 2; ++i)
                        for (int b = 0; b < BLOCKS && m.tiles[i] > 0; ++b)
                            tma_load(smem + S::kQ + (2 * qt.at + i) * S::kTile + b * kTcBlock, &maps.q,
                                     &bar.q_full[qt.at], b * kTcCols, m.head,
                                     (int)m.q0 + m.row0 + i * pk.tokens);
                }
                for (int j = 0; j < n && going; ++j) {
                    going = tc_wait(&bar.k_empty[kt.at], kt.parity ^ 1, lost);
                    if (!going) break;
                    mbar_expect_tx(&bar.k_full[kt.at], S::kTile);
                    for (int b = 0; b < BLOCKS; ++b)
                        tma_load(smem + S::kK + kt.at * S::kTile + b * kTcBlock, &maps.k,
                                 &bar.k_full[kt.at], b * kTcCols, hk, (int)m.k0 + (m.first + j) * kTcRows);
                    going = tc_wait(&bar.v_empty[kt.at], kt.parity ^ 1, lost);
                    if (!going) break;
                    mbar_expect_tx(&bar.v_full[kt.at], S::kTile);
                    for (int b = 0; b < BLOCKS; ++b)
                        tma_load(smem + S::kV + kt.at * S::kTile + b * kTcBlock, &maps.v,
                                 &bar.v_full[kt.at], b * kTcCols, hk, (int)m.k0 + (m.first + j) * kTcRows);
                    kt.next();
                }
            }
            qt.next();
            going = __shfl_sync(0xffffffffu, (int)going, 0) != 0;
        }
        m.tiles[0] = -1;
        if (going) ring_put(bar.ring, turn, m, lost);
    } else if (warp == 9) {
        // ---- products
        set_registers_down<kOtherRegs>();
        const uint32_t s_desc = tc_idesc(kTcRows, false), o_desc = tc_idesc(width, true);
        Turn<S::kQs> qt;
        Turn<S::kStages> kt, vt;
        uint32_t p_par[2] = {0, 0}, o_par[2] = {0, 0}, f_par[2] = {1, 1};
        bool used[2] = {false, false}, going = true;
        Item m;
        // scores of tile i with the keys at kt, once its probabilities' place is free
        const auto scores = [&](int i) {
            if (S::kOver && used[i]) going = tc_wait_warp(&bar.o_done[i], o_par[i] ^ 1, lost);
            if (!going) return;
            if (elect_one()) {
                tc_dot<BLOCKS>(tmem + i * 128, smem + S::kQ + (2 * qt.at + i) * S::kTile,
                       smem + S::kK + kt.at * S::kTile, ksteps, s_desc);
                tc_commit(&bar.s_full[i]);
            }
            __syncwarp();
        };
        while (going && ring_take(bar.ring, turn, m, lost)) {
            const int n = max(m.tiles[0], m.tiles[1]);
            if (n == 0) continue;
            going = tc_wait_warp(&bar.q_full[qt.at], qt.parity, lost) &&
                    tc_wait_warp(&bar.k_full[kt.at], kt.parity, lost);
            if (!going) break;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (going && m.tiles[i] > 0) scores(i);
            if (going && elect_one()) {
                tc_commit(&bar.k_empty[kt.at]);
                if (n == 1) tc_commit(&bar.q_empty[qt.at]);
            }
            kt.next();
            for (int j = 0; j < n && going; ++j) {
                const bool more = j + 1 < n;
                if (more) going = tc_wait_warp(&bar.k_full[kt.at], kt.parity, lost);
                going = going && tc_wait_warp(&bar.v_full[vt.at], vt.parity, lost);
                if (!going) break;
                char* v = smem + S::kV + vt.at * S::kTile;
                const int rows = m.nk - (m.first + j) * kTcRows;
                if (rows < kTcRows) {
                    clear_rows(v, rows, BLOCKS);
                    fence_async_proxy();
                    __syncwarp();
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (!going || j >= m.tiles[i]) continue;
                    going = tc_wait_warp(&bar.p_full[i], p_par[i], lost);
                    p_par[i] ^= 1;
                    // the outputs of the item before have been read
                    if (going && j == 0) {
                        going = tc_wait_warp(&bar.o_free[i], f_par[i], lost);
                        f_par[i] ^= 1;
                    }
                    if (!going) continue;
                    tc_fence_after();
                    if (!S::kOver && j + 1 < m.tiles[i]) scores(i);
                    if (elect_one()) {
                        tc_rows(tmem + 256 + i * 64 * BLOCKS, fwd_p<BLOCKS>(tmem, i), 0, v, o_desc,
                                j > 0);
                        tc_commit(&bar.o_done[i]);
                    }
                    __syncwarp();
                    o_par[i] ^= 1;
                    used[i] = true;
                    if (S::kOver && j + 1 < m.tiles[i]) scores(i);
                }
                if (going && elect_one()) {
                    tc_commit(&bar.v_empty[vt.at]);
                    if (more) tc_commit(&bar.k_empty[kt.at]);
                    if (j + 2 == n) tc_commit(&bar.q_empty[qt.at]);
                }
                if (more) kt.next();
                vt.next();
            }
            qt.next();
        }
    } else if (warp < 8) {
        // ---- softmax: warps 0-3 have tile 0, warps 4-7 tile 1
        set_registers_up<kComputeRegs>();
        const int i = warp >> 2, r = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_at = tmem + i * 128 + lanes, o_at = tmem + 256 + i * 64 * BLOCKS + lanes;
        const uint32_t p_at = fwd_p<BLOCKS>(tmem, i) + lanes;
        const int my_token = i * pk.tokens + r / pk.heads, my_head = r % pk.heads;
        const bool stored = r < pk.heads * pk.tokens, wide = wide_rows(a.out);
        const float c2 = a.scale * kLog2e;
        const F2 cc = pack2(c2, c2);
        uint32_t s_par = 0, o_par = 0;
        bool going = true;
        Item m;
        while (going && ring_take(bar.ring, turn, m, lost)) {
            const int tiles = i ? m.tiles[1] : m.tiles[0];
            const int row = m.row0 + my_token, head = m.head + my_head;
            const bool live = stored && row < m.nq;
            // rows that are not stored need no mask
            const int seen = live && a.causal ? min(m.nk, row + m.nk - m.nq + 1) : m.nk;
            float shift = 0.0f;
            F2 sum = 0;
            for (int j = 0; j < tiles && going; ++j) {
                going = tc_wait_warp(&bar.s_full[i], s_par, lost);
                s_par ^= 1;
                if (!going) break;
                tc_fence_after();
                const int most = seen - (m.first + j) * kTcRows;     // columns below it are visible
                const bool edge = __any_sync(0xffffffffu, most < kTcRows);
                uint32_t p[64];
                F2 part[2];
                bool looked = false;
                while (true) {
                    const F2 mm = pack2(-shift, -shift);
                    part[0] = part[1] = 0;
                    if (edge) tile_exp<true>(s_at, most, cc, mm, part, p);
                    else tile_exp<false>(s_at, most, cc, mm, part, p);
                    part[0] = add2(part[0], part[1]);
                    const float total = lo2(part[0]) + hi2(part[0]), before = lo2(sum) + hi2(sum);
                    const bool fits = !live || (total <= 0x1p16f && total + before >= 0x1p-30f);
                    if (looked || __all_sync(0xffffffffu, fits)) break;
                    looked = true;
                    const float next = tile_max(s_at, most) * c2;
                    // a row's shift depends on that row alone, not on its neighbours
                    const float want = fits || next == -INFINITY ? shift
                                       : before > 0.0f ? fmaxf(shift, next) : next;
                    if (j > 0) {
                        const float fade = fits ? 1.0f : before > 0.0f ? ex2(shift - want) : 0.0f;
                        going = tc_wait_warp(&bar.o_done[i], o_par ^ 1, lost);
                        if (!going) break;
                        tc_fence_after();
                        scale_rows(o_at, width, fade);
                        sum = mul2(sum, pack2(fade, fade));
                    }
                    shift = want;
                }
                if (!going) break;
                sum = add2(sum, part[0]);
                if (!S::kOver && j > 0) {     // the product before has read the last ones
                    going = tc_wait_warp(&bar.o_done[i], o_par ^ 1, lost);
                    if (!going) break;
                    tc_fence_after();
                }
                o_par ^= 1;
                tmem_store32(p_at, p);
                tmem_store32(p_at + 32, p + 32);
                tmem_wait_stores();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.p_full[i]);
            }
            if (going && tiles > 0) going = tc_wait_warp(&bar.o_done[i], o_par ^ 1, lost);
            const float total = lo2(sum) + hi2(sum);
            if (SPLIT) {
                split_put<BLOCKS>(smem, i * 128 + r, o_at, going ? tiles : -1, shift, total,
                                  &bar.parts_done, lost);
                continue;
            }
            char* out = live ? row_of(a.out, m.q0 + row, head) : nullptr;
            if (going && tiles > 0) {
                tc_fence_after();
                store_row<64 * BLOCKS, 64>(o_at, a.D, total == 0.0f ? 0.0f : 1.0f / total, out, live, wide,
                                       [&] {
                                           tc_fence_before();
                                           __syncwarp();
                                           if (lane == 0) mbar_arrive(&bar.o_free[i]);
                                       });
            } else if (going) {
                zero_row(a.D, out, live);
            }
            if (a.lse != nullptr && live)
                a.lse[(int64_t)head * a.Tq + m.q0 + row] =
                    !going ? __int_as_float(0x7fc00000)
                    : total == 0.0f ? -INFINITY : (shift + log2f(total)) * kLn2;
        }
    } else {
        set_registers_down<kOtherRegs>();
    }
    if (SPLIT) split_join<BLOCKS>(smem, bar.ring, a, pk, parts);
    tc_finish(lost, tmem, warp == 9);
}

// ------------------------------------------------------------ gradient of the queries
//
// A block has 128 queries of one head and walks over the keys:
//   scores and dout v^T (tensor memory, columns 0 and 128) -> ds in bf16 (384)
//   -> dq += ds k (256).
// The compute warps copy both products to registers before they work on them, so
// the next tile's two run meanwhile, and dq's behind them; the first two of the next
// item are issued before the last dq of this one.  Warps 0-3 have the first 64 keys of a
// tile, 4-7 the others.

constexpr int kGradThreads = 384;   // 8 compute warps, loads, products, two for delta or idle

struct GradBars {
    Ring ring;
    uint64_t once_full[2], once_empty[2], in_full[3], in_empty[3], v_full[3], v_empty[3];
    uint64_t s_full, s_free, g_full, p_full, d_full, d_free, o_full, o_free;
    uint64_t rows_full[2], rows_empty[2];
    uint32_t tmem;
    int lost;
};
static_assert(sizeof(GradBars) <= 1024, "the barriers' place");

template <int BLOCKS>
struct GradShape {
    static constexpr int kTile = BLOCKS * kTcBlock;
    static constexpr int kOnces = BLOCKS == 1 ? 2 : 1;       // pairs of what stays: q, dout or k, v
    static constexpr int kStages = BLOCKS == 1 ? 3 : 2;      // pairs of the others
    static constexpr int kIn = kOnces * 2 * kTile;
    static constexpr int kRows = kIn + kStages * 2 * kTile;  // floats of rows: kStages x 2 x 128
    static constexpr int kBars = kRows + 3 * 1024;
    static constexpr int kBytes = kBars + 1024 + 1024;
    static_assert(kBytes <= 227 * 1024, "shared memory of a block");
};

// The queries' kernel keeps keys until dq has them and values only until dp has: places of
// their own, three for keys.  (With two pairs of places the next keys began to load only
// when dq was done: 3,080 clocks a tile of 128 columns.)
constexpr int kDqComputeRegs = 192, kDqOtherRegs = 120;    // 2 x 128 x 192 + 128 x 120 = 384 x 168

template <int BLOCKS>
struct DqShape {
    static constexpr int kTile = BLOCKS * kTcBlock;
    static constexpr int kOnces = GradShape<BLOCKS>::kOnces;
    static constexpr int kKs = 3, kVs = BLOCKS == 1 ? 3 : 2;
    static constexpr int kK = kOnces * 2 * kTile, kV = kK + kKs * kTile;
    static constexpr int kRows = kV + kVs * kTile;       // 2 x 128 floats
    static constexpr int kBars = kRows + 1024;
    static constexpr int kBytes = kBars + 1024 + 1008;   // the base is rounded up from 16 to 1024
    static_assert(kBytes <= 227 * 1024, "shared memory of a block");
};

// The start of a block of either kernel: barriers, tensor memory.
template <int BLOCKS>
__device__ __forceinline__ uint32_t grad_start(GradBars& bar, const Maps& maps, int warp,
                                               uint32_t readers)
{
    using S = GradShape<BLOCKS>;
    if (threadIdx.x == 0) {
        ring_init(bar.ring, readers);
        for (int i = 0; i < S::kOnces; ++i) {
            mbar_init(&bar.once_full[i], 1);
            mbar_init(&bar.once_empty[i], 1);
        }
        for (int i = 0; i < 3; ++i) {
            mbar_init(&bar.in_full[i], 1);
            mbar_init(&bar.in_empty[i], 1);
            mbar_init(&bar.v_full[i], 1);
            mbar_init(&bar.v_empty[i], 1);
        }
        mbar_init(&bar.s_full, 1);
        mbar_init(&bar.s_free, 8);
        mbar_init(&bar.g_full, 1);
        mbar_init(&bar.p_full, 8);
        mbar_init(&bar.d_full, 8);
        mbar_init(&bar.d_free, 1);
        mbar_init(&bar.o_full, 1);
        mbar_init(&bar.o_free, 8);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.rows_full[i], 2);
            mbar_init(&bar.rows_empty[i], 8);
        }
        bar.lost = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        tma_prefetch(&maps.q);
        tma_prefetch(&maps.k);
        tma_prefetch(&maps.v);
        tma_prefetch(&maps.dout);
    }
    pdl_wait_prior();
    if (warp == 9) tmem_alloc(&bar.tmem);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_launch_dependents();
    return (uint32_t)uniform((int)bar.tmem);
}

// An operand's tile to its place.
template <int BLOCKS>
__device__ __forceinline__ void load_one(char* to, const CUtensorMap* x, uint64_t* full, int head,
                                         int row)
{
    mbar_expect_tx(full, GradShape<BLOCKS>::kTile);
    for (int b = 0; b < BLOCKS; ++b)
        tma_load(to + b * kTcBlock, x, full, b * kTcCols, head, row);
}

// Two operands' tiles to a pair of places.
template <int BLOCKS>
__device__ __forceinline__ void load_pair(char* to, const CUtensorMap* x, const CUtensorMap* y,
                                          uint64_t* full, int head, int row)
{
    constexpr int kTile = GradShape<BLOCKS>::kTile;
    mbar_expect_tx(full, 2 * kTile);
    for (int b = 0; b < BLOCKS; ++b) {
        tma_load(to + b * kTcBlock, x, full, b * kTcCols, head, row);
        tma_load(to + kTile + b * kTcBlock, y, full, b * kTcCols, head, row);
    }
}

template <int BLOCKS>
__global__ void __launch_bounds__(kGradThreads, 1)
k_attn_tc_dq(const __grid_constant__ Maps maps, const __grid_constant__ AttnArgs a, int tiles,
             int64_t items)
{
    using S = DqShape<BLOCKS>;
    extern __shared__ char smem_raw[];
    char* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    GradBars& bar = *reinterpret_cast<GradBars*>(smem + S::kBars);
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const uint32_t tmem = grad_start<BLOCKS>(bar, maps, warp, 11);
    volatile int* lost = &bar.lost;
    const int ksteps = (a.D + 15) / 16, width = ksteps * 16;
    Turn<kRing> turn;

    if (warp == 8) {
        // ---- items and loads
        set_registers_down<kDqOtherRegs>();
        Turn<S::kOnces> qt;
        Turn<S::kKs> kt;
        Turn<S::kVs> vt;
        bool going = true;
        Item m{};
        for (int64_t round = 0; round * gridDim.x < items && going; ++round) {
            const int64_t w = item_of_round(round, a);
            if (w >= items) continue;
            // the tiles at the end of a sequence see the most keys and go first
            const int tile = (int)(w / a.Hq);
            const Tile t = find_tile(a, tiles - 1 - tile, kTcRows, false);
            if (!t.any) continue;
            const int end = !a.causal ? t.nk
                                      : max(0, min(t.nk, min(t.row0 + kTcRows, t.nq) + t.nk - t.nq));
            const int n = (end + kTcRows - 1) / kTcRows;
            m = {t.q0, t.k0, t.nq, t.nk, t.row0, (int)(w - (int64_t)tile * a.Hq), {n, 0}};
            going = ring_put(bar.ring, turn, m, lost);
            if (!going || n == 0) continue;
            if (lane == 0) {
                going = tc_wait(&bar.once_empty[qt.at], qt.parity ^ 1, lost);
                if (going)
                    load_pair<BLOCKS>(smem + qt.at * 2 * S::kTile, &maps.q, &maps.dout,
                                      &bar.once_full[qt.at], m.head, (int)t.q0 + t.row0);
                const int hk = m.head / (a.Hq / a.Hk);
                for (int j = 0; j < n && going; ++j) {
                    going = tc_wait(&bar.in_empty[kt.at], kt.parity ^ 1, lost);
                    if (!going) break;
                    load_one<BLOCKS>(smem + S::kK + kt.at * S::kTile, &maps.k, &bar.in_full[kt.at], hk,
                                     (int)t.k0 + j * kTcRows);
                    kt.next();
                    going = tc_wait(&bar.v_empty[vt.at], vt.parity ^ 1, lost);
                    if (!going) break;
                    load_one<BLOCKS>(smem + S::kV + vt.at * S::kTile, &maps.v, &bar.v_full[vt.at], hk,
                                     (int)t.k0 + j * kTcRows);
                    vt.next();
                }
            }
            qt.next();
            going = __shfl_sync(0xffffffffu, (int)going, 0) != 0;
        }
        m.tiles[0] = -1;
        if (going) ring_put(bar.ring, turn, m, lost);
    } else if (warp == 9) {
        // ---- products
        set_registers_down<kDqOtherRegs>();
        const uint32_t s_desc = tc_idesc(kTcRows, false), o_desc = tc_idesc(width, true);
        Turn<S::kOnces> qt;
        Turn<S::kKs> kt, dt;
        Turn<S::kVs> vt;
        uint32_t s_par = 1, d_par = 0, f_par = 1;
        bool going = true, left = false, left_first = false;
        // dq += ds k of the step before this one
        const auto add_dq = [&] {
            going = tc_wait_warp(&bar.d_full, d_par, lost);
            d_par ^= 1;
            if (going && left_first) {    // the result of the item before has been read
                going = tc_wait_warp(&bar.o_free, f_par, lost);
                f_par ^= 1;
            }
            if (!going) return;
            tc_fence_after();
            if (elect_one()) {
                tc_rows(tmem + 256, tmem + 384, 0, smem + S::kK + dt.at * S::kTile, o_desc,
                        !left_first);
                tc_commit(&bar.d_free);
                tc_commit(&bar.in_empty[dt.at]);
            }
            __syncwarp();
            dt.next();
        };
        Item m;
        while (going && ring_take(bar.ring, turn, m, lost)) {
            const int n = m.tiles[0];
            if (n == 0) {     // the compute warps come to it only after the item before
                if (left) add_dq();
                left = false;
                continue;
            }
            going = tc_wait_warp(&bar.once_full[qt.at], qt.parity, lost);
            const char* q = smem + qt.at * 2 * S::kTile;
            for (int j = 0; j < n && going; ++j) {
                going = tc_wait_warp(&bar.in_full[kt.at], kt.parity, lost) &&
                        tc_wait_warp(&bar.v_full[vt.at], vt.parity, lost);
                if (!going) break;
                char* in = smem + S::kK + kt.at * S::kTile;
                const int rows = m.nk - j * kTcRows;
                if (rows < kTcRows) {     // dq sums over the keys
                    clear_rows(in, rows, BLOCKS);
                    fence_async_proxy();
                    __syncwarp();
                }
                going = tc_wait_warp(&bar.s_free, s_par, lost);
                s_par ^= 1;
                if (!going) break;
                tc_fence_after();
                if (elect_one()) {
                    tc_dot<BLOCKS>(tmem, q, in, ksteps, s_desc);
                    tc_dot<BLOCKS>(tmem + 128, q + S::kTile, smem + S::kV + vt.at * S::kTile, ksteps,
                                   s_desc);
                    tc_commit(&bar.s_full);
                    tc_commit(&bar.v_empty[vt.at]);
                    if (j + 1 == n) tc_commit(&bar.once_empty[qt.at]);
                }
                __syncwarp();
                kt.next();
                vt.next();
                if (left) add_dq();
                left = true;
                left_first = j == 0;
            }
            qt.next();
        }
        if (going && left) add_dq();
    } else if (warp < 8) {
        // ---- scores' gradients
        set_registers_up<kDqComputeRegs>();
        const float* rows_s = reinterpret_cast<const float*>(smem + S::kRows);
        Turn<2> rt;
        const int r = (warp & 3) * 32 + lane, half = warp >> 2;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const float c2 = a.scale * kLog2e;
        const F2 cc = pack2(c2, c2);
        const bool wide = wide_rows(a.dq);
        uint32_t s_par = 0, d_par = 0;
        bool going = true;
        Item m;
        while (going && ring_take(bar.ring, turn, m, lost)) {
            const int row = m.row0 + r, n = m.tiles[0];
            const bool live = row < m.nq;
            const float lse = live ? a.lse[(int64_t)m.head * a.Tq + m.q0 + row] : -INFINITY;
            going = tc_wait_warp(&bar.rows_full[rt.at], rt.parity, lost);
            if (!going) break;
            const float delta = rows_s[rt.at * 128 + r];
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.rows_empty[rt.at]);
            rt.next();
            const bool none = lse == -INFINITY;
            const int seen = none ? 0 : a.causal ? min(m.nk, row + m.nk - m.nq + 1) : m.nk;
            const F2 nl = pack2(-lse * kLog2e, -lse * kLog2e), nd = pack2(-delta, -delta);
            for (int j = 0; j < n; ++j) {
                going = tc_wait_warp(&bar.s_full, s_par, lost);
                s_par ^= 1;
                if (!going) break;
                tc_fence_after();
                uint32_t x[128];      // 64 scores, 64 of dout v^T
                tmem_load32(tmem + lanes + 64 * half, x);
                tmem_load32(tmem + lanes + 64 * half + 32, x + 32);
                tmem_load32(tmem + lanes + 128 + 64 * half, x + 64);
                tmem_load32(tmem + lanes + 128 + 64 * half + 32, x + 96);
                tmem_wait(x);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.s_free);
                uint32_t ds[32];
                const int most = seen - j * kTcRows - 64 * half;
                const bool mask = __any_sync(0xffffffffu, most < 64);
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const F2 u = fma2((F2)x[2 * e + 1] << 32 | x[2 * e], cc, nl);
                    const F2 p = pack2(ex2(lo2(u)), ex2(hi2(u)));
                    const F2 d = mul2(p, add2((F2)x[64 + 2 * e + 1] << 32 | x[64 + 2 * e], nd));
                    ds[e] = pack_bf16x2(lo2(d), hi2(d));
                }
                if (mask) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        ds[e] = 2 * e + 1 < most ? ds[e] : 2 * e < most ? ds[e] & 0xffffu : 0u;
                }
                if (j > 0) {      // the product before has read the last ones
                    going = tc_wait_warp(&bar.d_free, d_par ^ 1, lost);
                    if (!going) break;
                    tc_fence_after();
                }
                d_par ^= 1;
                tmem_store32(tmem + lanes + 384 + 32 * half, ds);
                tmem_wait_stores();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.d_full);
            }
            if (going && n > 0) going = tc_wait_warp(&bar.d_free, d_par ^ 1, lost);
            if (!going) break;
            tc_fence_after();
            // a thread's half of its row, in whole 32 columns
            const int first = half * BLOCKS * 32, cols = min(a.D - first, BLOCKS * 32);
            char* out = live ? row_of(a.dq, m.q0 + row, m.head) + 2 * first : nullptr;
            if (n > 0)
                store_row<BLOCKS * 32, 32>(tmem + lanes + 256 + first, cols, a.scale, out, live, wide, [&] {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.o_free);
                });
            else zero_row(cols, out, live);
        }
    } else {
        // ---- delta, 64 rows of an item each, ahead of the compute warps
        set_registers_down<kDqOtherRegs>();
        float* rows_s = reinterpret_cast<float*>(smem + S::kRows);
        Turn<2> rt;
        // lanes of a row, rows of a load, loads under way: what a pass waits for is latency
        constexpr int kLanes = 8 * BLOCKS, kAtOnce = 32 / kLanes, kLoads = 8;
        const int d = (lane & (kLanes - 1)) * 8;
        Item m;
        while (ring_take(bar.ring, turn, m, lost)) {
            if (!tc_wait_warp(&bar.rows_empty[rt.at], rt.parity ^ 1, lost)) break;
            for (int r0 = (warp - 10) * 64; r0 < (warp - 9) * 64; r0 += kLoads * kAtOnce) {
                const int r1 = r0 + lane / kLanes;
                const char* g = row_of(a.dout, m.q0 + m.row0 + r1, m.head) + 2 * d;
                const char* o = row_of(a.out, m.q0 + m.row0 + r1, m.head) + 2 * d;
                const int64_t step_g = 2 * kAtOnce * a.dout.ld, step_o = 2 * kAtOnce * a.out.ld;
                uint4 u[kLoads], w[kLoads];
#pragma unroll
                for (int q = 0; q < kLoads; ++q) {
                    u[q] = w[q] = make_uint4(0, 0, 0, 0);
                    if (m.row0 + r1 + q * kAtOnce < m.nq && d < a.D) {
                        u[q] = *reinterpret_cast<const uint4*>(g + q * step_g);
                        w[q] = *reinterpret_cast<const uint4*>(o + q * step_o);
                    }
                }
#pragma unroll
                for (int q = 0; q < kLoads; ++q) {
                    const uint32_t us[4] = {u[q].x, u[q].y, u[q].z, u[q].w};
                    const uint32_t ws[4] = {w[q].x, w[q].y, w[q].z, w[q].w};
                    float y = 0.0f;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        y = fmaf(bf16_hi(us[e]), bf16_hi(ws[e]),
                                 fmaf(bf16_lo(us[e]), bf16_lo(ws[e]), y));
#pragma unroll
                    for (int k = 1; k < kLanes; k <<= 1) y += __shfl_xor_sync(0xffffffffu, y, k);
                    const int r = r1 + q * kAtOnce;
                    if (d == 0) {
                        rows_s[rt.at * 128 + r] = y;
                        if (m.row0 + r < m.nq)
                            a.delta[(int64_t)m.head * a.Tq + m.q0 + m.row0 + r] = y;
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.rows_full[rt.at]);
            rt.next();
        }
    }
    tc_finish(lost, tmem, warp == 9);
}

// ------------------------------------------------------------ gradients of keys and values
//
// A block has 128 keys of one key head and walks over the queries of all query
// heads that share it.  Scores are transposed, keys along the rows, so that both
// probabilities and ds are left operands as they are:
//   s^T = k q^T (0) -> p^T in bf16 -> dv += p^T dout (256)
//   dp^T = v dout^T (128) -> ds^T in bf16 -> dk += ds^T q (384, or 320 for 64 columns)
// p^T and ds^T take the places of what they were made from, each warp writing
// over columns that only it has read.  The products alternate with the
// compute warps' two halves: dv and the next scores run while ds is computed, dk
// and the next dp while p is; the next item's first two run behind this one's stores.

// The queries' tiles that an item of keys walks over, for each head.
__device__ __forceinline__ int first_query(const AttnArgs& a, const Item& m)
{
    return a.causal ? max(0, m.row0 - (m.nk - m.nq)) / kTcRows * kTcRows : 0;
}

template <int BLOCKS>
__global__ void __launch_bounds__(kGradThreads, 1)
k_attn_tc_dkv(const __grid_constant__ Maps maps, const __grid_constant__ AttnArgs a, int tiles,
              int64_t items)
{
    using S = GradShape<BLOCKS>;
    constexpr uint32_t kDv = 256, kDk = BLOCKS == 2 ? 384 : 320;
    extern __shared__ char smem_raw[];
    char* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    GradBars& bar = *reinterpret_cast<GradBars*>(smem + S::kBars);
    float* rows_s = reinterpret_cast<float*>(smem + S::kRows);   // [stage][-lse log2e, -delta][128]
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const uint32_t tmem = grad_start<BLOCKS>(bar, maps, warp, 9);
    volatile int* lost = &bar.lost;
    const int G = a.Hq / a.Hk;
    const int ksteps = (a.D + 15) / 16, width = ksteps * 16;
    Turn<kRing> turn;

    if (warp == 8) {
        // ---- items and loads
        set_registers_down<kOtherRegs>();
        Turn<S::kOnces> qt;
        Turn<S::kStages> kt;
        bool going = true;
        Item m{};
        for (int64_t round = 0; round * gridDim.x < items && going; ++round) {
            const int64_t w = item_of_round(round, a);
            if (w >= items) continue;
            // the first keys of a sequence are seen by the most queries: tiles in order
            const int tile = (int)(w / a.Hk);
            const Tile t = find_tile(a, tile, kTcRows, true);
            if (!t.any) continue;
            m = {t.q0, t.k0, t.nq, t.nk, t.row0, (int)(w - (int64_t)tile * a.Hk), {0, 0}};
            const int first = first_query(a, m);
            const int n = first < t.nq ? (t.nq - first + kTcRows - 1) / kTcRows * G : 0;
            m.tiles[0] = n;
            going = ring_put(bar.ring, turn, m, lost);
            if (!going || n == 0) continue;
            going = tc_wait_warp(&bar.once_empty[qt.at], qt.parity ^ 1, lost);
            if (going && lane == 0)
                load_pair<BLOCKS>(smem + qt.at * 2 * S::kTile, &maps.k, &maps.v,
                                  &bar.once_full[qt.at], m.head, (int)t.k0 + t.row0);
            qt.next();
            int h = m.head * G, i0 = first;
            for (int j = 0; j < n && going; ++j) {
                float nl[4], nd[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int row = i0 + 32 * e + lane;
                    const int64_t at = (int64_t)h * a.Tq + t.q0 + row;
                    const float l = row < t.nq ? a.lse[at] : -INFINITY;
                    nl[e] = l == -INFINITY ? -INFINITY : -l * kLog2e;
                    nd[e] = row < t.nq ? -a.delta[at] : 0.0f;
                }
                going = tc_wait_warp(&bar.in_empty[kt.at], kt.parity ^ 1, lost);
                if (!going) break;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    rows_s[kt.at * 256 + 32 * e + lane] = nl[e];
                    rows_s[kt.at * 256 + 128 + 32 * e + lane] = nd[e];
                }
                __syncwarp();
                if (lane == 0)
                    load_pair<BLOCKS>(smem + S::kIn + kt.at * 2 * S::kTile, &maps.q, &maps.dout,
                                      &bar.in_full[kt.at], h, (int)t.q0 + i0);
                kt.next();
                i0 += kTcRows;
                if (i0 >= t.nq) {
                    i0 = first;
                    ++h;
                }
            }
        }
        m.tiles[0] = -1;
        if (going) ring_put(bar.ring, turn, m, lost);
    } else if (warp == 9) {
        // ---- products
        set_registers_down<kOtherRegs>();
        const uint32_t s_desc = tc_idesc(kTcRows, false), o_desc = tc_idesc(width, true);
        Turn<S::kOnces> qt;
        Turn<S::kStages> kt, dt;      // of the next scores, of the step under way
        uint32_t p_par = 0, f_par = 1;
        bool going = true;
        Item m;
        while (going && ring_take(bar.ring, turn, m, lost)) {
            const int n = m.tiles[0];
            if (n == 0) continue;
            const int first = first_query(a, m);
            int i0 = first;               // of the next scores
            const char* k = smem + qt.at * 2 * S::kTile;
            going = tc_wait_warp(&bar.once_full[qt.at], qt.parity, lost);
            // waits for a tile, clears what lies beyond the sequence, issues its scores
            const auto scores = [&] {
                going = tc_wait_warp(&bar.in_full[kt.at], kt.parity, lost);
                if (!going) return;
                char* in = smem + S::kIn + kt.at * 2 * S::kTile;
                if (m.nq - i0 < kTcRows) {     // dk and dv sum over the queries
                    clear_rows(in, m.nq - i0, BLOCKS);
                    clear_rows(in + S::kTile, m.nq - i0, BLOCKS);
                    fence_async_proxy();
                    __syncwarp();
                }
                if (elect_one()) {
                    tc_dot<BLOCKS>(tmem, k, in, ksteps, s_desc);
                    tc_commit(&bar.s_full);
                }
                __syncwarp();
                i0 += kTcRows;
                if (i0 >= m.nq) i0 = first;
                kt.next();
            };
            const auto grads = [&](int at) {
                if (elect_one()) {
                    tc_dot<BLOCKS>(tmem + 128, k + S::kTile,
                                   smem + S::kIn + at * 2 * S::kTile + S::kTile, ksteps, s_desc);
                    tc_commit(&bar.g_full);
                }
                __syncwarp();
            };
            if (going) scores();
            if (going) grads(dt.at);
            for (int j = 0; j < n && going; ++j) {
                const char* in = smem + S::kIn + dt.at * 2 * S::kTile;
                going = tc_wait_warp(&bar.p_full, p_par, lost);
                if (going && j == 0) {         // the results of the item before have been read
                    going = tc_wait_warp(&bar.o_free, f_par, lost);
                    f_par ^= 1;
                }
                if (!going) break;
                tc_fence_after();
                if (elect_one()) {
                    tc_rows(tmem + kDv, tmem, 32, in + S::kTile, o_desc, j > 0);
                    tc_commit(&bar.d_free);
                }
                __syncwarp();
                // the next scores take the probabilities' place
                going = tc_wait_warp(&bar.d_free, 0, lost);
                if (going && j + 1 < n) scores();
                if (!going) break;
                going = tc_wait_warp(&bar.d_full, p_par, lost);
                p_par ^= 1;
                if (!going) break;
                tc_fence_after();
                if (elect_one()) {
                    tc_rows(tmem + kDk, tmem + 128, 32, in, o_desc, j > 0);
                    tc_commit(&bar.in_empty[dt.at]);
                    tc_commit(&bar.d_free);
                    if (j + 1 == n) {
                        tc_commit(&bar.once_empty[qt.at]);
                        tc_commit(&bar.o_full);
                    }
                }
                __syncwarp();
                dt.next();
                going = tc_wait_warp(&bar.d_free, 1, lost);
                if (going && j + 1 < n) grads(dt.at);
            }
            qt.next();
        }
    } else if (warp < 8) {
        // ---- probabilities and scores' gradients
        set_registers_up<kComputeRegs>();
        const int r = (warp & 3) * 32 + lane, half = warp >> 2;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const float c2 = a.scale * kLog2e;
        const F2 cc = pack2(c2, c2);
        const bool wide_k = wide_rows(a.dk), wide_v = wide_rows(a.dv);
        Turn<S::kStages> kt;
        uint32_t s_par = 0, o_par = 0;
        bool going = true;
        Item m;
        while (going && ring_take(bar.ring, turn, m, lost)) {
            const int n = m.tiles[0], first = first_query(a, m), row = m.row0 + r;
            const bool live = row < m.nk;
            int i0 = first;
            for (int j = 0; j < n; ++j) {
                const float* nl = rows_s + kt.at * 256 + 64 * half;
                const float* nd = nl + 128;
                going = tc_wait_warp(&bar.in_full[kt.at], kt.parity, lost) &&
                        tc_wait_warp(&bar.s_full, s_par, lost);
                if (!going) break;
                kt.next();
                tc_fence_after();
                uint32_t s[64];
                tmem_load32(tmem + lanes + 64 * half, s);
                tmem_load32(tmem + lanes + 64 * half + 32, s + 32);
                tmem_wait(s);
                // columns from `from` on see this row's key
                const int from = a.causal ? row - (m.nk - m.nq) - i0 - 64 * half : 0;
                const bool mask = __any_sync(0xffffffffu, from > 0);
                uint32_t p[32];
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float4 l = *reinterpret_cast<const float4*>(nl + 2 * e);
                    const F2 u = fma2((F2)s[2 * e + 1] << 32 | s[2 * e], cc, pack2(l.x, l.y));
                    const F2 v = fma2((F2)s[2 * e + 3] << 32 | s[2 * e + 2], cc, pack2(l.z, l.w));
                    s[2 * e] = __float_as_uint(ex2(lo2(u)));
                    s[2 * e + 1] = __float_as_uint(ex2(hi2(u)));
                    s[2 * e + 2] = __float_as_uint(ex2(lo2(v)));
                    s[2 * e + 3] = __float_as_uint(ex2(hi2(v)));
                }
                if (mask) {
#pragma unroll
                    for (int e = 0; e < 64; ++e)
                        if (e < from) s[e] = 0;
                }
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    p[e] = pack_bf16x2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]));
                tmem_store32(tmem + lanes + 64 * half, p);
                tmem_wait_stores();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.p_full);
                going = tc_wait_warp(&bar.g_full, s_par, lost);
                s_par ^= 1;
                if (!going) break;
                tc_fence_after();
                uint32_t g[64];
                tmem_load32(tmem + lanes + 128 + 64 * half, g);
                tmem_load32(tmem + lanes + 128 + 64 * half + 32, g + 32);
                tmem_wait(g);
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float4 l = *reinterpret_cast<const float4*>(nd + 2 * e);
                    const F2 u = mul2((F2)s[2 * e + 1] << 32 | s[2 * e],
                                      add2((F2)g[2 * e + 1] << 32 | g[2 * e], pack2(l.x, l.y)));
                    const F2 v = mul2((F2)s[2 * e + 3] << 32 | s[2 * e + 2],
                                      add2((F2)g[2 * e + 3] << 32 | g[2 * e + 2], pack2(l.z, l.w)));
                    p[e] = pack_bf16x2(lo2(u), hi2(u));
                    p[e + 1] = pack_bf16x2(lo2(v), hi2(v));
                }
                if (mask) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        p[e] = 2 * e >= from ? p[e] : 2 * e + 1 >= from ? p[e] & 0xffff0000u : 0u;
                }
                tmem_store32(tmem + lanes + 128 + 64 * half, p);
                tmem_wait_stores();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.d_full);
                i0 += kTcRows;
                if (i0 >= m.nq) i0 = first;
            }
            if (going && n > 0) {
                going = tc_wait_warp(&bar.o_full, o_par, lost);
                o_par ^= 1;
            }
            if (!going) break;
            tc_fence_after();
            const int begin = half * BLOCKS * 32, cols = min(a.D - begin, BLOCKS * 32);
            char* dv = live ? row_of(a.dv, m.k0 + row, m.head) + 2 * begin : nullptr;
            char* dk = live ? row_of(a.dk, m.k0 + row, m.head) + 2 * begin : nullptr;
            if (n > 0) {
                store_row<BLOCKS * 32, 32>(tmem + lanes + kDv + begin, cols, 1.0f, dv, live, wide_v, [] {});
                store_row<BLOCKS * 32, 32>(tmem + lanes + kDk + begin, cols, a.scale, dk, live, wide_k, [&] {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.o_free);
                });
            } else {
                zero_row(cols, dv, live);
                zero_row(cols, dk, live);
            }
        }
    } else {
        set_registers_down<kOtherRegs>();
    }
    tc_finish(lost, tmem, warp == 9);
}

// ------------------------------------------------------------ launches

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder of tensor maps, looked up once.
EncodeFn encoder()
{
    static const EncodeFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult res = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &res) != cudaSuccess ||
            res != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

// Elements, heads and tokens of x; a box is 64 elements of `heads` heads of
// `tokens` tokens.  What lies outside reads as zeros.
bool make_map(CUtensorMap* m, const Heads& x, int64_t T, int H, int D, int heads, int tokens)
{
    const EncodeFn fn = encoder();
    if (fn == nullptr) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T};
    const cuuint64_t strides[2] = {(cuuint64_t)x.hs * 2, (cuuint64_t)x.ld * 2};
    const cuuint32_t box[3] = {kTcCols, (cuuint32_t)heads, (cuuint32_t)tokens};
    const cuuint32_t step[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, x.p, dims, strides, box, step,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool aligned(const Heads& x)
{
    return reinterpret_cast<uintptr_t>(x.p) % 16 == 0 && x.ld % 8 == 0 && x.hs % 8 == 0 &&
           x.ld < int64_t(1) << 38 && x.hs < int64_t(1) << 38;
}

// Query heads that share a tile, and its tokens.
Packing packing_of(const AttnArgs& a)
{
    const int G = a.Hq / a.Hk;
    const int heads = G <= 32 ? G : 1;
    return {heads, kTcRows / heads};
}

template <class Kernel, class... Args>
cudaError_t launch_tc(Kernel fn, SmemRaisedOn& raised, size_t smem, int64_t blocks, int heads,
                      int threads, cudaStream_t s, unsigned cluster, Args... args)
{
    const cudaError_t e = raise_smem(raised, reinterpret_cast<const void*>(fn), smem);
    if (e != cudaSuccess) return e;
    return launch_kernel(fn, dim3((unsigned)blocks, (unsigned)heads), dim3(threads), smem, s, true,
                         cluster, args...);
}

template <class F>
cudaError_t by_blocks(int D, F&& f)
{
    return D <= kTcCols ? f(std::integral_constant<int, 1>{}) : f(std::integral_constant<int, 2>{});
}

}  // namespace

bool attn_tc_takes(const AttnArgs& a, bool grad)
{
    return a.dt == DPZ_BF16 && a.D % 8 == 0 && a.Tq > 0 && a.Tk > 0 && aligned(a.q) &&
           aligned(a.k) && aligned(a.v) && aligned(a.out) &&
           (!grad || (aligned(a.dout) && aligned(a.dq) && aligned(a.dk) && aligned(a.dv)));
}

cudaError_t launch_attn_tc(const AttnArgs& a, cudaStream_t s)
{
    set_last_kernel_name("attn_forward");
    const Packing pk = packing_of(a);
    Maps m;
    if (!make_map(&m.q, a.q, a.Tq, a.Hq, a.D, pk.heads, pk.tokens) ||
        !make_map(&m.k, a.k, a.Tk, a.Hk, a.D, 1, kTcRows) ||
        !make_map(&m.v, a.v, a.Tk, a.Hk, a.D, 1, kTcRows))
        return launch_attn_any(a, s);
    m.dout = m.q;
    int sms = 0;
    const cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    return by_blocks(a.D, [&](auto n) {
        static SmemRaisedOn raised;
        const int64_t pairs = tiles_bound(a.cu_q, a.Tq, a.B, 2 * pk.tokens);
        const int64_t items = pairs * (a.Hq / pk.heads);
        // few items with many keys each: up to eight blocks share one (16 queries
        // of 32 + 8 heads of 128 against 8,191 keys: 20 us, 87 with one block)
        int parts = 1;
        while (parts < 8 && items * parts * 2 <= sms && a.len_k >= parts * 4 * kTcRows) parts *= 2;
        if (parts > 1) {
            static SmemRaisedOn split_raised;
            return launch_tc(k_attn_tc<n, true>, split_raised, FwdShape<n>::kBytes, items * parts, 1,
                             kFwdThreads, s, (unsigned)parts, m, a, pk, (int)pairs, items, parts);
        }
        return launch_tc(k_attn_tc<n, false>, raised, FwdShape<n>::kBytes, items < sms ? items : sms, 1,
                         kFwdThreads, s, 0u, m, a, pk, (int)pairs, items, 1);
    });
}

namespace {

bool grad_maps(Maps* m, const AttnArgs& a)
{
    return make_map(&m->q, a.q, a.Tq, a.Hq, a.D, 1, kTcRows) &&
           make_map(&m->k, a.k, a.Tk, a.Hk, a.D, 1, kTcRows) &&
           make_map(&m->v, a.v, a.Tk, a.Hk, a.D, 1, kTcRows) &&
           make_map(&m->dout, a.dout, a.Tq, a.Hq, a.D, 1, kTcRows);
}

}  // namespace

cudaError_t launch_attn_tc_dq(const AttnArgs& a, cudaStream_t s)
{
    set_last_kernel_name("attn_grad_dq");
    Maps m;
    if (!grad_maps(&m, a)) return launch_attn_any_dq(a, s);
    int sms = 0;
    const cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    return by_blocks(a.D, [&](auto n) {
        static SmemRaisedOn raised;
        const int64_t tiles = tiles_bound(a.cu_q, a.Tq, a.B, kTcRows);
        const int64_t items = tiles * a.Hq;
        return launch_tc(k_attn_tc_dq<n>, raised, DqShape<n>::kBytes, items < sms ? items : sms, 1,
                         kGradThreads, s, 0u, m, a, (int)tiles, items);
    });
}

cudaError_t launch_attn_tc_dkv(const AttnArgs& a, cudaStream_t s)
{
    set_last_kernel_name("attn_grad_dkv");
    Maps m;
    if (!grad_maps(&m, a)) return launch_attn_any_dkv(a, s);
    int sms = 0;
    const cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    return by_blocks(a.D, [&](auto n) {
        static SmemRaisedOn raised;
        const int64_t tiles = tiles_bound(a.cu_k, a.Tk, a.B, kTcRows);
        const int64_t items = tiles * a.Hk;
        return launch_tc(k_attn_tc_dkv<n>, raised, GradShape<n>::kBytes, items < sms ? items : sms, 1,
                         kGradThreads, s, 0u, m, a, (int)tiles, items);
    });
}

cudaError_t read_and_clear_tc_lost(unsigned* flag)
{
    cudaError_t e = cudaMemcpyFromSymbol(flag, g_tc_lost, sizeof(unsigned));
    if (e != cudaSuccess || *flag == 0) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_tc_lost, &zero, sizeof(unsigned));
}

}  // namespace dpz
