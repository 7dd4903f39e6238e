// attention.cu -- softmax attention over packed sequences, and its gradient, which recomputes the probabilities.
//
//   z = scale q k^T where the query sees the key,  lse = log sum exp z,  o = exp(z - lse) v
//   p = exp(z - lse),  dv = p^T do,  dp = do v^T,  delta = do . o,  dz = p (dp - delta)
//   dq = scale dz k,  dk = scale dz^T q            (dk, dv: summed over the query heads that share the key's)
//
// Scores and probabilities live in tensor memory and registers alone.  All products run on the tensor cores in bf16
// with fp32 sums (tcgen05.mma.kind::f16 on tiles of 128 x 128); p and dz are rounded to bf16 as operands.
//
//   forward  a CTA for two tiles of 128 rows that take turns: while the softmax of one runs, the tensor cores work on the
//            other.  The rows are queries of all the heads that share a key head (Packing): its keys are read once
//   join     where few queries' keys are shared out over several CTAs: their parts put together
//   delta    (lse log2 e, do . o) of each query
//   dkv      a CTA for 128 keys of a key head, over all queries that see them, of all heads that share it: dk and dv stay
//            in tensor memory, and no two CTAs add to the same number
//   dq       a CTA for 128 rows, over the keys that they see
// Long sequences are bound by the products, whose operands take all of shared memory's bandwidth (8192 tokens of 32 and 8
// heads of 128, causal: forward 0.55 TFLOP in 358 us, 321 with no softmax; backward seven products, 1.92 TFLOP, in 1170),
// heads of 64 or less by the softmax's instructions between them, few queries by reading the keys and values, short
// sequences by a CTA's start and end, which take as long as six tiles of keys (8192 tokens, not causal, in 1024 CTAs with 1, 2,
// 4, 8 and 16 tiles each: 70, 77, 95, 134 and 211 us).
// The scores are made a second time for dq: two products more than a single pass over (keys, queries) would need, which
// would have to add to dq in memory, in an order that differs from run to run.
//
// Operand tiles are 128 rows (tokens) x 64 or 128 columns in shared memory, in blocks of 64 columns, 128-byte rows,
// 128-byte swizzle: the same tile is read along its columns (q and k of z) or along its rows (v of p v).  A tile reaches
// past the end of its sequence into the next one's rows; where such rows are summed over they are cleared first, so that
// nothing that they hold (infinities, NaN) reaches this sequence.  Keys of the sequence that are hidden from a query are
// summed over with p = 0, as far as its tile goes: what they reach is said at the entry points.
#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <type_traits>

#include "element.cuh"
#include "heads.cuh"
#include "quant_math.cuh"

namespace mx {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kRows = 128;                // of a tile
constexpr int kBlockBytes = kRows * 128;  // 64 columns of a tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ------------------------------------------------------------------ PTX
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int32_t x, int32_t y,
                                            int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
        "[%2];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}
// Shared-memory descriptors as their low words (address, and bytes between 64-column blocks): the high word, 1024 bytes
// between groups of eight rows and the 128-byte swizzle, is the same for all.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (kSwizzle128B << 29);
// D (+)= A B^T with bf16 operands in shared memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
        : "memory");
}
// The same with A in tensor memory: row m in lane m, two bf16 in each column.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
        "mov.b64 db, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
        : "memory");
}
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
// 16 lanes x 32 columns: thread t has columns 8i + 2(t % 4) and the next one of lanes t / 4 (r[4i], r[4i + 1]) and
// t / 4 + 8 (r[4i + 2], r[4i + 3]).
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
// 16 lanes x 16 columns: thread t has column 4i + t % 4 of lanes t / 4 (r[2i]) and t / 4 + 8 (r[2i + 1]).
__device__ __forceinline__ void tmem_st_16x128b_x4(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Barriers of a part of the block (id 0 is __syncthreads).
__device__ __forceinline__ void sync_some(int id, int threads) {
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ bool any_of_some(int id, int threads, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred a, b;\n\t"
        "setp.ne.b32 a, %1, 0;\n\t"
        "barrier.cta.red.or.pred b, %2, %3, a;\n\t"
        "selp.b32 %0, 1, 0, b;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(id), "r"(threads)
        : "memory");
    return r != 0;
}

// wait_bounded for a whole warp: what all lanes agree on.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns, uint32_t* status) {
    return __all_sync(0xffffffffu, wait_bounded(bar, parity, limit_ns, status));
}

// The first lane's value, which the compiler then knows to be the warp's.  The lane that feeds the tensor cores has 64
// cycles for each instruction, and took 140 where its operands were not known to be the warp's: 8192 tokens of 32 heads
// of 128, not causal, forward 1044 us.  With the low words of descriptors made once a tile 836, with elect.sync for the
// choice of the lane 735, with these 680.
__device__ __forceinline__ int32_t uniform(int32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// ------------------------------------------------------------------ sequences
struct Sequences {
    const int32_t* cu_q;  // [count + 1] first tokens, or NULL: `count` sequences of equal lengths
    const int32_t* cu_k;
    int32_t count, tokens_q, tokens_k, len_q, len_k;
};

struct Place {
    int32_t q0, k0, len_q, len_k;  // first tokens and lengths of the sequence
    int32_t tile;                  // of it; -1: nothing to do
    int32_t part, parts;           // of the tile's keys, where they are shared out
};

// Sequence i's first token and length, whatever the list holds.
__device__ __forceinline__ void range_of(const int32_t* cu, int32_t i, int32_t tokens, int32_t& first, int32_t& len,
                                         uint32_t* status) {
    const int32_t a = cu[i], b = cu[i + 1];
    if (a < 0 || b < a || b > tokens) atomicOr(status, kStatusBadIndex);
    first = min(max(a, 0), tokens);
    len = min(max(b, first), tokens) - first;
}

// Up to kScanned sequences the tiles are numbered one behind the other, and a warp counts them, 32 sequences a step.  Among
// more, sequence i's tiles begin at place first / rows + i, which leaves room for all of each: the sequence is then found
// without those before it, in steps that leave a 32nd of them (at most five), where counting would take each CTA a time
// that grows with the sequences, and the call one that grows with their square.  The list is looked through by all CTAs
// together.  8192 tokens of 32 and 8 heads of 128, forward and backward, searched and counted: 64 sequences 88.3 / 223 and
// 86.2 / 214 us, 128 100.6 / 242 and 104.7 / 242, 1024 395 / 748 and 735 / 1383, 4096 1.51 / 2.74 and 6.28 / 11.4 ms.
constexpr int32_t kScanned = 128;

// Place `slot` among the tiles of more than kScanned sequences.  A list that falls may lead to any of them, but to no tile that
// the sequence has not.
template <bool KEYS>
__device__ __forceinline__ Place search_place(const Sequences& s, int32_t slot, int32_t rows, uint32_t* status) {
    const int lane = threadIdx.x & 31;
    for (int64_t i = (int64_t)blockIdx.x * 32 + lane; i < s.count; i += (int64_t)gridDim.x * 32) {
        int32_t first, len;
        range_of(s.cu_q, (int32_t)i, s.tokens_q, first, len, status);
        range_of(s.cu_k, (int32_t)i, s.tokens_k, first, len, status);
    }
    const int32_t* cu = KEYS ? s.cu_k : s.cu_q;
    const int32_t tokens = KEYS ? s.tokens_k : s.tokens_q;
    auto base = [&](int32_t i) { return min(max(cu[i], 0), tokens) / rows + i; };
    int32_t low = 0, n = s.count;  // one of [low, low + n), the last that begins at `slot` or before it
    while (n > 1) {
        const int32_t step = (n + 31) / 32, i = lane * step;
        const uint32_t before = __ballot_sync(0xffffffffu, i < n && base(low + i) <= slot);
        const int32_t at = before ? (31 - __clz(before)) * step : 0;
        low += at;
        n = min(step, n - at);
    }
    Place p{};
    range_of(s.cu_q, low, s.tokens_q, p.q0, p.len_q, status);
    range_of(s.cu_k, low, s.tokens_k, p.k0, p.len_k, status);
    p.tile = slot - base(low);
    p.parts = 1;
    if (p.tile < 0 || p.tile >= ((KEYS ? p.len_k : p.len_q) + rows - 1) / rows) p.tile = -1;
    return p;
}

template <bool KEYS>
__device__ __noinline__ Place call_search_place(const Sequences& s, int32_t slot, int32_t rows, uint32_t* status) {
    return search_place<KEYS>(s, slot, rows, status);
}

// The sequence and tile (of `rows` queries, or keys) of place `slot` among the tiles of all sequences; with `chunk` above 0
// (and then few sequences) among their parts of that many keys.  By one warp.  How the search is reached matters to calls that
// do not need it: inlined it costs dkv and dq 0.5% of a batch of 13 sequences, as a call the forward pass up to 3% of 8 new
// tokens over 24018 keys.
enum class Search { kNone, kInline, kCall };
template <bool KEYS, Search HOW>
__device__ __forceinline__ Place find_place(const Sequences& s, int32_t slot, int32_t rows, int32_t chunk, uint32_t* status) {
    Place p{};
    p.tile = -1;
    if (!s.cu_q) {
        p.parts = chunk > 0 ? max((s.len_k + chunk - 1) / chunk, 1) : 1;
        const int32_t len = KEYS ? s.len_k : s.len_q, places = (len + rows - 1) / rows * p.parts;
        if (places == 0 || slot / places >= s.count) return p;
        const int32_t i = slot / places;
        p.q0 = i * s.len_q, p.k0 = i * s.len_k, p.len_q = s.len_q, p.len_k = s.len_k;
        p.tile = (slot - i * places) / p.parts;
        p.part = slot - i * places - p.tile * p.parts;
        return p;
    }
    if (HOW != Search::kNone && s.count > kScanned && chunk == 0)
        return HOW == Search::kInline ? search_place<KEYS>(s, slot, rows, status) : call_search_place<KEYS>(s, slot, rows, status);
    const int lane = threadIdx.x & 31;
    int32_t before = 0;
    for (int32_t i0 = 0; i0 < s.count; i0 += 32) {
        const int32_t i = i0 + lane;
        Place mine{};
        if (i < s.count) {
            range_of(s.cu_q, i, s.tokens_q, mine.q0, mine.len_q, status);
            range_of(s.cu_k, i, s.tokens_k, mine.k0, mine.len_k, status);
        }
        mine.parts = chunk > 0 ? max((mine.len_k + chunk - 1) / chunk, 1) : 1;
        const int32_t tiles = ((KEYS ? mine.len_k : mine.len_q) + rows - 1) / rows * mine.parts;
        int32_t upto = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t t = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += t;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, before + upto > slot);
        if (past) {
            const int src = __ffs(past) - 1;
            p.q0 = __shfl_sync(0xffffffffu, mine.q0, src), p.k0 = __shfl_sync(0xffffffffu, mine.k0, src);
            p.len_q = __shfl_sync(0xffffffffu, mine.len_q, src), p.len_k = __shfl_sync(0xffffffffu, mine.len_k, src);
            p.parts = __shfl_sync(0xffffffffu, mine.parts, src);
            p.tile = slot - before - __shfl_sync(0xffffffffu, upto - tiles, src);
            const int32_t most = __shfl_sync(0xffffffffu, tiles, src);
            if ((uint32_t)p.tile >= (uint32_t)most) {  // a list that falls, whose tiles are more than 2^31
                p.tile = -1;
                return p;
            }
            p.part = p.tile % p.parts;
            p.tile /= p.parts;
            return p;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
    return p;
}

// Clears the rows of the tokens in front of the first sequence and behind the last, by this warp of every CTA in turn.
// f(token) clears one.
template <class F>
__device__ __forceinline__ void clear_outside(const int32_t* cu, int32_t count, int32_t tokens, F&& f) {
    const int32_t first = min(max(cu[0], 0), tokens), end = min(max(cu[count], 0), tokens);
    const int32_t n = first + tokens - end;
    for (int64_t i = blockIdx.x; i < n; i += gridDim.x) f(i < first ? (int32_t)i : (int32_t)i - first + end);
}

__device__ __forceinline__ Place place_of(const Place* p) {
    return {uniform(p->q0),   uniform(p->k0),   uniform(p->len_q), uniform(p->len_k),
            uniform(p->tile), uniform(p->part), uniform(p->parts)};
}

// ------------------------------------------------------------------ shared pieces
// Low words of a tile's descriptors.  K along its columns: 16 columns a step.
__device__ __forceinline__ uint32_t columns_of(uint32_t tile) { return (tile & 0x3FFFFu) >> 4 | 1u << 16; }
__host__ __device__ constexpr uint32_t column_step(int k) { return (k >> 2) * (kBlockBytes >> 4) + (k & 3) * 2; }
// K along its rows: 16 rows a step, N along the columns.
__device__ __forceinline__ uint32_t rows_of_tile(uint32_t tile) {
    return (tile & 0x3FFFFu) >> 4 | (uint32_t)(kBlockBytes >> 4) << 16;
}
constexpr uint32_t kRowStep = 2048 >> 4;
// Tensor-memory column of step `step` (16 columns) of p or dz, which is kept in the place of the scores: each warp's
// COLUMNS scores become COLUMNS / 2 columns at their beginning.
template <int COLUMNS>
__device__ __forceinline__ uint32_t packed_column(int step) {
    return step * 16 / COLUMNS * COLUMNS + step * 16 % COLUMNS / 2;
}

// Clears rows [from, 128) of a tile, by one warp.
template <int DP>
__device__ __forceinline__ void clear_rows(uint8_t* tile, int from) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int b = 0; b < DP / 64; ++b)
        for (int i = from * 8 + lane; i < kRows * 8; i += 32)
            *reinterpret_cast<uint4*>(tile + b * kBlockBytes + i * 16) = make_uint4(0, 0, 0, 0);
}

// A tile of queries holds those of `pack` heads that share a key's (a divisor of the group): row r is token r / pack and
// head r % pack, `tokens` * pack rows in all, 128 or a few less.  Short sequences fill tiles so, and a mask's edge is
// `tokens` wide.
struct Packing {
    int32_t pack, tokens;
    __device__ __forceinline__ int32_t rows() const { return pack * tokens; }
};

// `rows`: of the map's box.
template <int DP>
__device__ __forceinline__ void load_tile(uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int32_t head,
                                          int32_t token, int32_t rows = kRows) {
    mbar_arrive_expect_tx(bar, DP / 64 * rows * 128);
#pragma unroll
    for (int b = 0; b < DP / 64; ++b) tma_load_3d(dst + b * kBlockBytes, map, bar, b * 64, head, token);
}

// Word i of lane j of each four to word j of lane i.
__device__ __forceinline__ void turn4x4(uint32_t (&w)[4], int lane) {
#pragma unroll
    for (int bit = 1; bit < 4; bit <<= 1) {
        const bool upper = lane & bit;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i & bit) continue;
            const uint32_t other = __shfl_xor_sync(0xffffffffu, upper ? w[i] : w[i + bit], bit);
            if (upper)
                w[i] = other;
            else
                w[i + bit] = other;
        }
    }
}

// A warp's 32 rows of an accumulator, `width` columns (a multiple of 8), to memory as bf16, and what the rounding left, as
// bf16 again, where it is asked for.  Of its own row each lane gives the factor, the addresses and whether it is there.  Four
// lanes write 64 neighbouring bytes of a row: with a row for each lane an instruction touched 32 lines, and the stores
// of a pair of tiles kept the SM's load and store unit busy for some 8000 cycles.
__device__ __forceinline__ void store_rows(uint32_t taddr, int width, float factor, bf16* to, bool inside,
                                           bf16* rest = nullptr) {
    const int lane = threadIdx.x & 31, column = 8 * (lane & 3);
    for (int c = 0; c < width; c += 32) {
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            uint32_t z[16];
            tmem_ld_16x256b_x4(taddr + c + ((uint32_t)hh << 20), z);
            tmem_ld_wait();
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const int src = hh * 16 + v * 8 + (lane >> 2);  // lane of the row
                const float f = __shfl_sync(0xffffffffu, factor, src);
                const uint64_t at = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(to), src);
                const bool on = __shfl_sync(0xffffffffu, (int)inside, src) && c + column < width;
                uint32_t w[4], u[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = __uint_as_float(z[4 * i + 2 * v]) * f, y = __uint_as_float(z[4 * i + 2 * v + 1]) * f;
                    w[i] = pack_bf16(x, y);
                    u[i] = pack_bf16(x - bf16_lo(w[i]), y - bf16_hi(w[i]));
                }
                turn4x4(w, lane);
                if (on) *reinterpret_cast<uint4*>(reinterpret_cast<bf16*>(at) + c + column) = make_uint4(w[0], w[1], w[2], w[3]);
                if (rest) {  // the same for all lanes but for the address
                    const uint64_t left = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(rest), src);
                    turn4x4(u, lane);
                    if (on)
                        *reinterpret_cast<uint4*>(reinterpret_cast<bf16*>(left) + c + column) = make_uint4(u[0], u[1], u[2], u[3]);
                }
            }
        }
    }
}
// The same in fp32 as it is (rows of a multiple of 8 elements).
__device__ __forceinline__ void store_part(uint32_t taddr, int dim, float* to, bool inside) {
    for (int c = 0; c < dim; c += 16) {
        uint32_t v[16];
        tmem_ld_32x32b_x16(taddr + c, v);
        tmem_ld_wait();
        if (inside) {
#pragma unroll
            for (int j = 0; j < 16; j += 4)
                if (c + j < dim) *reinterpret_cast<uint4*>(to + c + j) = make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        }
    }
}
__device__ __forceinline__ void store_zeros(int dim, bf16* to) {
    for (int c = 0; c < dim; c += 8) *reinterpret_cast<uint4*>(to + c) = make_uint4(0, 0, 0, 0);
}

struct Rows {  // of an output
    bf16* data;
    int64_t token_stride, head_stride;
    __device__ __forceinline__ bf16* at(int64_t token, int64_t head) const {
        return data + token * token_stride + head * head_stride;
    }
    // all heads of a token, by a warp
    __device__ __forceinline__ void clear(int64_t token, int32_t heads, int32_t dim) const {
        for (int32_t i = threadIdx.x & 31; i < heads * (dim / 8); i += 32)
            *reinterpret_cast<uint4*>(at(token, i / (dim / 8)) + i % (dim / 8) * 8) = make_uint4(0, 0, 0, 0);
    }
};

// A ring of tiles: the phase of use number i of its stages.
template <int N>
struct Ring {
    static __device__ __forceinline__ int stage(int i) { return i % N; }
    static __device__ __forceinline__ uint32_t parity(int i) { return (uint32_t)(i / N) & 1u; }
};

// ------------------------------------------------------------------ forward
struct ForwardParams {
    CUtensorMap q, k, v;
    Rows out, rest;  // rest.data NULL: not wanted
    float* lse;      // [q_heads][tokens_q]
    Sequences seq;
    Packing packing;
    int32_t head_blocks;  // query heads / pack
    int32_t group, dim, causal;
    int32_t clear;        // rows outside of all sequences become 0
    int32_t chunk;        // above 0: a CTA takes that many key tiles of a pair of query tiles, and leaves its part to join_kernel
    float* part;          // [CTA][2][128][dim]
    float4* part_stats;   // [CTA][2][128]: (log2 of what the part is scaled by, sum, sum of the rounded probabilities, 0)
    float scale_log2;     // scale * log2 e
    uint32_t* status;
    uint64_t wait_ns;
};

template <int DP>
struct ForwardShape {
    static constexpr int kTileBytes = DP / 64 * kBlockBytes;
    static constexpr int kStages = DP == 128 ? 4 : 6;  // of K and V tiles in turn
    static constexpr int kOffRing = 2 * kTileBytes;
    static constexpr int kOffBar = kOffRing + kStages * kTileBytes;
    static constexpr int kBars = 2 + 2 * kStages + 2 + 4 + 2 + 1;
    static constexpr int kOffPlace = kOffBar + kBars * 8;
    static constexpr int kOffShare = kOffPlace + 32;
    static constexpr int kSmem = kOffShare + 2 * 2 * kRows * 4;
};
static_assert(ForwardShape<128>::kSmem <= 227 * 1024, "shared memory budget");
static_assert(2 * ForwardShape<64>::kSmem > 228 * 1024, "one CTA per SM: CTAs do not wait for each other's TMEM");
constexpr int kForwardThreads = 128 + 512;
constexpr float kLag = 16.f;  // log2 of how far a row's probabilities may run ahead of the maximum that they are scaled by

template <int DP>
__global__ void __launch_bounds__(kForwardThreads, 1) attention_kernel(const __grid_constant__ ForwardParams p) {
    using Shape = ForwardShape<DP>;
    constexpr int kStages = Shape::kStages;
    extern __shared__ uint8_t smem[];
    if (smem_u32(smem) & 1023u) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusSmemLayout);
        return;
    }
    uint8_t* ring = smem + Shape::kOffRing;
    uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + Shape::kOffBar);  // [2]
    uint64_t* full = q_full + 2;                                            // [kStages]
    uint64_t* empty = full + kStages;                                       // [kStages]
    uint64_t* s_full = empty + kStages;                                     // [2] scores of a tile
    uint64_t* p_full = s_full + 2;                                          // [2][2] its probabilities, in two parts
    uint64_t* o_full = p_full + 4;                                          // [2] its output
    uint64_t* mma_done = o_full + 2;
    Place* where = reinterpret_cast<Place*>(smem + Shape::kOffPlace);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(where + 1);
    float* share = reinterpret_cast<float*>(smem + Shape::kOffShare);  // [tile][half][row]

    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int32_t block = (int32_t)(blockIdx.x % (uint32_t)p.head_blocks), head0 = block * p.packing.pack;
    const int32_t slot = (int32_t)(blockIdx.x / (uint32_t)p.head_blocks);
    const int32_t tokens = p.packing.tokens;  // of a tile
    if (threadIdx.x == 96) {  // warp 0 looks for its place meanwhile
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[2 * i], 8);
            mbar_init(&p_full[2 * i + 1], 8);
            mbar_init(&o_full[i], 1);
        }
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(mma_done, 1);
        fence_mbar_init();
        prefetch_tmap(&p.q);
        prefetch_tmap(&p.k);
        prefetch_tmap(&p.v);
    }
    if (warp == 1) {
        tmem_alloc(tmem_holder, 512);
        tmem_relinquish();
    }
    grid_dependency_wait();
    allow_dependent_launch();
    if (warp == 0) {
        const Place w = find_place<false, Search::kInline>(p.seq, slot, 2 * tokens, p.chunk * kRows, p.status);
        if (lane == 0) *where = w;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)uniform((int32_t)*tmem_holder);
    Place at = place_of(where);
    const bool work = at.tile >= 0;
    // the tiles that see the most keys first
    if (work && p.causal) at.tile = (at.len_q + 2 * tokens - 1) / (2 * tokens) - 1 - at.tile;
    const int32_t row0 = at.tile * 2 * tokens;  // first query, in the sequence
    const int32_t ahead = at.len_k - at.len_q;  // query i sees keys up to i + ahead
    // key tiles of each query tile: n of them from tile j0 on
    int32_t n[2] = {0, 0}, j0 = 0;
    if (work) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int32_t first = row0 + i * tokens, last = min(first + tokens, at.len_q) - 1;
            const int32_t keys = p.causal ? min(at.len_k, max(last + ahead + 1, 0)) : at.len_k;
            if (first < at.len_q) n[i] = (keys + kRows - 1) / kRows;
        }
        if (p.chunk > 0) {
            j0 = at.part * p.chunk;
#pragma unroll
            for (int i = 0; i < 2; ++i) n[i] = max(min(n[i] - j0, p.chunk), 0);
        }
    }
    const int32_t most = max(n[0], n[1]);

    if (warp == 0) {
        // ---------------- TMA producer
        if (elect_one() && most > 0) {
            const int32_t key_head = head0 / p.group;
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (n[i] > 0)
                    load_tile<DP>(smem + i * Shape::kTileBytes, &p.q, &q_full[i], head0, at.q0 + row0 + i * tokens,
                                  p.packing.rows());
            int armed = 0;
            for (int i = 0; i < 2 * most; ++i) {  // K and V of each key tile in turn
                const int s = i % kStages;
                if (i >= kStages && !wait_bounded(&empty[s], (uint32_t)(i / kStages - 1) & 1u, p.wait_ns, p.status)) break;
                load_tile<DP>(ring + s * Shape::kTileBytes, i & 1 ? &p.v : &p.k, &full[s], key_head,
                              at.k0 + (j0 + (i >> 1)) * kRows);
                armed = i + 1;
            }
            // everything that was asked for has landed before this CTA ends
            for (int i = max(0, armed - kStages); i < armed; ++i)
                wait_bounded(&full[i % kStages], (uint32_t)(i / kStages) & 1u, p.wait_ns, p.status);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (n[i] > 0) wait_bounded(&q_full[i], 0, p.wait_ns, p.status);
        }
    } else if (warp == 1) {
        // ---------------- tensor cores: one lane issues
        const uint32_t scores = idesc_bf16(kRows, kRows, 0, 0);
        const uint32_t output = idesc_bf16(kRows, (uint32_t)(p.dim + 15) / 16 * 16, 0, 1);
        const int steps = (p.dim + 15) / 16;
        bool ok = true;
        auto wait_full = [&](int i) {
            if (ok) ok = warp_wait(&full[i % kStages], (uint32_t)(i / kStages) & 1u, p.wait_ns, p.status);
        };
        auto make_scores = [&](int t, int j) {
            const uint32_t a = columns_of(smem_u32(smem + t * Shape::kTileBytes));
            const uint32_t b = columns_of(smem_u32(ring + (2 * j) % kStages * Shape::kTileBytes));
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < DP / 16; ++k)
                    if (k < steps) mma_ss(tmem + t * 128, a + column_step(k), b + column_step(k), scores, k != 0);
                tc_commit(&s_full[t]);
            }
        };
        if (most > 0) {
            wait_full(0);
#pragma unroll
            for (int t = 0; t < 2; ++t)
                if (ok && n[t] > 0) {
                    ok = warp_wait(&q_full[t], 0, p.wait_ns, p.status);
                    tc_fence_after();
                    if (ok) make_scores(t, 0);
                }
            if (ok && elect_one()) tc_commit(&empty[0]);
        }
        for (int j = 0; ok && j < most; ++j) {
            const int sv = (2 * j + 1) % kStages;
            wait_full(2 * j + 1);
            if (!ok) break;
            const int left = at.len_k - (j0 + j) * kRows;  // keys of this tile that are the sequence's
            if (left < kRows) {
                clear_rows<DP>(ring + sv * Shape::kTileBytes, left);
                fence_async_smem();
                __syncwarp();
            }
            if (j + 1 < most) wait_full(2 * j + 2);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                if (!ok || j >= n[t]) continue;
                const uint32_t b = rows_of_tile(smem_u32(ring + sv * Shape::kTileBytes));
#pragma unroll
                for (int part = 0; part < 2; ++part) {  // the first 32 keys of each half, then the others
                    ok = ok && warp_wait(&p_full[2 * t + part], (uint32_t)j & 1u, p.wait_ns, p.status);
                    if (!ok) continue;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int k = part * 2 + (i >> 1) * 4 + (i & 1);
                            mma_ts(tmem + 256 + t * 128, tmem + t * 128 + packed_column<64>(k), b + k * kRowStep, output,
                                   j != 0 || part != 0 || i != 0);
                        }
                        if (part == 1 && j + 1 == n[t]) tc_commit(&o_full[t]);
                    }
                }
                if (!ok) continue;
                // after p v in the pipe, so the scores may take the place of p
                if (j + 1 < n[t]) make_scores(t, j + 1);
            }
            if (ok && elect_one()) {
                tc_commit(&empty[sv]);
                if (j + 1 < most) tc_commit(&empty[(2 * j + 2) % kStages]);
            }
        }
        if (elect_one()) tc_commit(mma_done);
        warp_wait(mma_done, 0, p.wait_ns, p.status);
    } else if (warp == 2) {
        if (p.clear)
            clear_outside(p.seq.cu_q, p.seq.count, p.seq.tokens_q, [&](int32_t token) {
                const int32_t heads = p.head_blocks * p.packing.pack;
                p.out.clear(token, heads, p.dim);
                if (p.rest.data) p.rest.clear(token, heads, p.dim);
                for (int32_t h = lane; h < heads; h += 32) p.lse[(int64_t)h * p.seq.tokens_q + token] = 0.f;
            });
    } else if (warp >= 4) {
        // ---------------- softmax: a lane for each query, a warpgroup for each half of the keys of each query tile
        const int t = (warp - 4) >> 3, half = ((warp - 4) >> 2) & 1, quad = warp & 3;
        const int32_t r = quad * 32 + lane, row = row0 + t * tokens + r / p.packing.pack;  // place in the tile, query
        const int32_t head = head0 + r % p.packing.pack;
        const bool inside = work && r < p.packing.rows() && row < at.len_q;
        const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t src = lanes + t * 128 + half * 64, acc = lanes + 256 + t * 128;
        float* mine = share + (t * 2 + half) * kRows + quad * 32 + lane;
        const float* other = share + (t * 2 + 1 - half) * kRows + quad * 32 + lane;
        const int columns = (p.dim + 15) / 16 * 16, barrier = 1 + t * 4 + quad;
        // key that this query sees last, from the first tile's first key on, and the least of these in the query tile
        const int32_t last = (p.causal ? min(at.len_k - 1, row + ahead) : at.len_k - 1) - j0 * kRows;
        const int32_t least = (p.causal ? min(at.len_k - 1, row0 + t * tokens + ahead) : at.len_k - 1) - j0 * kRows;
        const float2 scale2 = make_float2(p.scale_log2, p.scale_log2);
        float top = -INFINITY;  // maximum that the sums are scaled by (of the scores before `scale`)
        float shift = 0.f;      // top * scale_log2
        float2 sum2 = make_float2(0.f, 0.f);
        float2 off2 = make_float2(0.f, 0.f);  // what rounding to bf16 adds to the sums
        bool ok = true;
        for (int j = 0; j < n[t]; ++j) {
            ok = warp_wait(&s_full[t], (uint32_t)j & 1u, p.wait_ns, p.status);
            tc_fence_after();
            uint32_t z[64];
            tmem_ld_32x32b_x32(src, *reinterpret_cast<uint32_t(*)[32]>(z));
            tmem_ld_32x32b_x32(src + 32, *reinterpret_cast<uint32_t(*)[32]>(z + 32));
            tmem_ld_wait();
            if (least - j * kRows < kRows - 1) {
                const int seen = last - j * kRows - half * 64;
#pragma unroll
                for (int i = 0; i < 64; ++i)
                    if (i > seen) z[i] = 0xff800000u;
            }
            float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < 64; ++i) m4[i & 3] = fmaxf(m4[i & 3], __uint_as_float(z[i]));
            float m = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
            // A new maximum is taken up only once the old one lags by kLag: p then stays below 2^kLag, which bf16 and
            // the fp32 sums hold as exactly as values below 1, and the output is seldom scaled again.  The two warps that
            // share 32 queries agree on it (with all eight of a tile and a lag of 8: 434 us instead of 400 for 8192 tokens
            // whose scores reach 11).  A timeout travels with the vote, so that both leave together.
            if (any_of_some(barrier, 64, !ok || j == 0 || (m - top) * p.scale_log2 > kLag)) {
                *mine = m;
                sync_some(barrier, 64);
                const float theirs = *other;
                if (any_of_some(barrier, 64, !ok)) {
                    ok = false;
                    break;
                }
                const float most_of_both = fmaxf(m, theirs);
                const bool raise = j == 0 || (most_of_both - top) * p.scale_log2 > kLag;
                const float new_top = raise ? fmaxf(top, most_of_both) : top;
                const float new_shift = new_top == -INFINITY ? 0.f : new_top * p.scale_log2;
                if (j > 0) {
                    // the scores' commit came after that of p v: the output holds all tiles before this one
                    const float by = !raise ? 1.f : top == -INFINITY ? 0.f : exp2_approx(shift - new_shift);
                    sum2 = f2_mul(sum2, make_float2(by, by));
                    off2 = f2_mul(off2, make_float2(by, by));
                    for (int c = half * 16; c < columns; c += 32) {
                        uint32_t v[16];
                        tmem_ld_32x32b_x16(acc + c, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * by);
                        tmem_st_32x32b_x16(acc + c, v);
                    }
                }
                top = new_top;
                shift = new_shift;
            }
            const float2 shift2 = make_float2(-shift, -shift);
            // The output is divided by the sum of the rounded probabilities that it is made of, lse is that of the exact ones.
            // A key that has most of a row's probability then gives its v exactly, whatever its rounding, and the gradient's
            // dp - do . o, which cancels there, is exact: with scores up to 11, dk of 8192 tokens is off by 2.5e-3 of itself
            // instead of 4.8e-3.  Tiles whose keys all have less than 1/4 of the sum so far are left out: their roundings
            // add up to less than the gradients' own (with 1/16 the errors are the same and 8192 tokens take 367 us instead of 359).
            // A row's own keys decide for it, so that no other row changes its bits.
            constexpr float kHeavy = 4.f;
            const bool heavy = inside && !(exp2_approx(fmaf(m, p.scale_log2, -shift)) * kHeavy < sum2.x + sum2.y);
            auto probabilities = [&](int c, auto exact) {
                uint32_t w[16];
                float2 all = make_float2(0.f, 0.f), rounded = all;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int at_z = c * 32 + 2 * i;
                    const float2 e = f2_fma(make_float2(__uint_as_float(z[at_z]), __uint_as_float(z[at_z + 1])), scale2, shift2);
                    const float2 x = make_float2(exp2_approx(e.x), exp2_approx(e.y));
                    all = f2_add(all, x);
                    w[i] = pack_bf16(x.x, x.y);
                    if constexpr (decltype(exact)::value) rounded = f2_add(rounded, make_float2(bf16_lo(w[i]), bf16_hi(w[i])));
                }
                sum2 = f2_add(sum2, all);
                if constexpr (decltype(exact)::value)
                    if (heavy) off2 = f2_add(off2, f2_sub(rounded, all));
                tmem_st_32x32b_x16(src + c * 16, w);
            };
            const bool any_heavy = __any_sync(0xffffffffu, heavy);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (any_heavy)
                    probabilities(c, std::true_type{});
                else
                    probabilities(c, std::false_type{});
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[2 * t + c]);
            }
        }
        // the halves' sums, in their order
        float sum = sum2.x + sum2.y, kept = 0.f;  // kept: of the rounded probabilities
        auto both_halves = [&](float v) {
            *mine = v;
            sync_some(barrier, 64);
            v = half ? *other + v : v + *other;
            sync_some(barrier, 64);
            return v;
        };
        if (ok && n[t] > 0) {
            sum = both_halves(sum);
            kept = sum + both_halves(off2.x + off2.y);
            ok = warp_wait(&o_full[t], 0, p.wait_ns, p.status);
            if (ok) {
                tc_fence_after();
                const int cut = (p.dim / 2 + 15) / 16 * 16, from = half ? cut : 0, width = half ? p.dim - cut : min(cut, p.dim);
                if (p.chunk > 0)
                    store_part(acc + from, width, p.part + (((int64_t)blockIdx.x * 2 + t) * kRows + r) * p.dim + from, inside);
                else
                    store_rows(acc + from, width, sum == 0.f ? 0.f : 1.f / kept, p.out.at(at.q0 + row, head) + from, inside,
                              p.rest.data ? p.rest.at(at.q0 + row, head) + from : nullptr);
                // A row without weight is zeros, not 0 times sums that hidden keys may have made infinite or NaN.
                const bool none = inside && sum == 0.f && p.chunk == 0;
                if (__any_sync(0xffffffffu, none)) {  // over what other lanes have just written
                    __syncwarp();
                    if (none) {
                        store_zeros(width, p.out.at(at.q0 + row, head) + from);
                        if (p.rest.data) store_zeros(width, p.rest.at(at.q0 + row, head) + from);
                    }
                }
            }
        } else if (inside && half == 0 && n[t] == 0 && p.chunk == 0) {  // no key at all
            store_zeros(p.dim, p.out.at(at.q0 + row, head));
            if (p.rest.data) store_zeros(p.dim, p.rest.at(at.q0 + row, head));
        }
        if (inside && half == 0) {
            if (p.chunk > 0)
                p.part_stats[((int64_t)blockIdx.x * 2 + t) * kRows + r] = make_float4(shift, sum, kept, 0.f);
            else
                p.lse[(int64_t)head * p.seq.tokens_q + at.q0 + row] = sum == 0.f ? -INFINITY : (shift + log2f(sum)) * kLn2;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// The parts of a pair of query tiles joined: a warp for each row, a lane for four columns.  The rows are shared out over
// the CTAs of all the parts' places, kJoinCtas of a place (256 queries of 32 heads over 8192 keys, the whole call: 65.8 us,
// with 4 of a place 69.8, with 2 74.1; 64 queries, when the first part's four CTAs did all: 80 us, now 28.9).
constexpr int kJoinThreads = 256, kJoinCtas = 8;

__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ ForwardParams p) {
    __shared__ Place where;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int32_t block = (int32_t)(blockIdx.x % (uint32_t)p.head_blocks), slot = (int32_t)(blockIdx.x / (uint32_t)p.head_blocks);
    const int32_t tokens = p.packing.tokens;
    grid_dependency_wait();
    allow_dependent_launch();
    if (warp == 0) {
        const Place w = find_place<false, Search::kNone>(p.seq, slot, 2 * tokens, p.chunk * kRows, p.status);
        if (lane == 0) where = w;
    }
    __syncthreads();
    Place at = where;
    // parts that have no place: a list that falls names more keys than there are
    if (at.tile < 0 || slot - at.part + at.parts > (int32_t)(gridDim.x / (uint32_t)p.head_blocks)) return;
    if (p.causal) at.tile = (at.len_q + 2 * tokens - 1) / (2 * tokens) - 1 - at.tile;
    const int32_t row0 = at.tile * 2 * tokens, rows = min(2 * tokens, at.len_q - row0) * p.packing.pack;
    const int32_t warps = at.parts * kJoinCtas * (kJoinThreads / 32);
    for (int32_t i = (at.part * kJoinCtas + blockIdx.y) * (kJoinThreads / 32) + warp; i < rows; i += warps) {
        const int32_t t = i / p.packing.rows(), r = i - t * p.packing.rows();
        const int32_t token = at.q0 + row0 + t * tokens + r / p.packing.pack, head = block * p.packing.pack + r % p.packing.pack;
        // part s of this row
        auto part = [&](int s) { return (((int64_t)slot - at.part + s) * p.head_blocks + block) * 2 * kRows + t * kRows + r; };
        // A lane reads the statistics of every 32nd part, so that the loads of all are under way at once (one part after the
        // other took 15 us for 10 parts, of 8 new tokens over 24018 keys).  What all are scaled by: the largest of the parts'
        // that hold anything (NaN is something).
        auto stats_of = [&](int s) { return s < at.parts ? p.part_stats[part(s)] : make_float4(0.f, 0.f, 0.f, 0.f); };
        float top = -INFINITY;
        for (int s0 = 0; s0 < at.parts; s0 += 32) {
            const float4 st = stats_of(s0 + lane);
            if (st.y != 0.f) top = fmaxf(top, st.x);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        float sum = 0.f, kept = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s0 = 0; s0 < at.parts; s0 += 32) {
            const float4 st = stats_of(s0 + lane);
            const float by = st.y == 0.f ? 0.f : exp2_approx(st.x - top);
            sum = fmaf(by, st.y, sum);
            kept = fmaf(by, st.z, kept);
            const int n = min(32, at.parts - s0);
#pragma unroll 8
            for (int s = 0; s < n; ++s) {
                const float f = __shfl_sync(0xffffffffu, by, s);
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);  // a part without weight may not have been written
                if (f != 0.f && lane * 4 < p.dim)
                    x = *reinterpret_cast<const float4*>(p.part + part(s0 + s) * p.dim + lane * 4);
                v.x = fmaf(f, x.x, v.x), v.y = fmaf(f, x.y, v.y), v.z = fmaf(f, x.z, v.z), v.w = fmaf(f, x.w, v.w);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
            kept += __shfl_xor_sync(0xffffffffu, kept, o);
        }
        const float one = sum == 0.f ? 0.f : 1.f / kept;
        if (lane * 4 < p.dim) {
            const float o[4] = {v.x * one, v.y * one, v.z * one, v.w * one};
            uint2 w = make_uint2(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]));
            *reinterpret_cast<uint2*>(p.out.at(token, head) + lane * 4) = w;
            if (p.rest.data) {
                w = make_uint2(pack_bf16(o[0] - bf16_lo(w.x), o[1] - bf16_hi(w.x)), pack_bf16(o[2] - bf16_lo(w.y), o[3] - bf16_hi(w.y)));
                *reinterpret_cast<uint2*>(p.rest.at(token, head) + lane * 4) = w;
            }
        }
        if (lane == 0) p.lse[(int64_t)head * p.seq.tokens_q + token] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
    }
}

// ------------------------------------------------------------------ backward
// What the gradients need of each query: (lse log2 e, do . o).  A query that sees nothing gets an infinite lse, and so
// probabilities of 0.  HBM-bound: reads o and do once.
// o is what the forward pass rounded to bf16 and, where it was kept, what that left.  Without the latter do . o is off by
// 2^-8 of its terms, and so is the dz of a key that has most of a row's probability, where dp - do . o cancels: with scores
// up to 19, dq and dk of 2048 tokens are off by 5.5e-3 of themselves instead of 2.5e-3 (bf16's own rounding: 1.7e-3).
struct DeltaParams {
    const bf16* out;
    const bf16* rest;  // or NULL
    const bf16* dout;
    int64_t o_token, o_head, r_token, r_head, d_token, d_head;
    const float* lse;
    float2* stats;  // [q_heads][tokens_q]
    int32_t tokens, heads, dim;
};
constexpr int kDeltaThreads = 256;

__global__ void __launch_bounds__(kDeltaThreads) delta_kernel(const __grid_constant__ DeltaParams p) {
    grid_dependency_wait();
    allow_dependent_launch();
    const int li = threadIdx.x & 15;
    const int64_t row = (int64_t)blockIdx.x * (kDeltaThreads / 16) + (threadIdx.x >> 4);
    const int64_t t = row / p.heads;
    const int32_t h = (int32_t)(row - t * p.heads);
    float v = 0.f;
    if (t < p.tokens && li * 8 < p.dim) {
        float a[8], b[8];
        unpack8(load8(p.out + t * p.o_token + h * p.o_head + li * 8), a);
        unpack8(load8(p.dout + t * p.d_token + h * p.d_head + li * 8), b);
#pragma unroll
        for (int i = 0; i < 8; ++i) v = fmaf(a[i], b[i], v);
        if (p.rest) {
            unpack8(load8(p.rest + t * p.r_token + h * p.r_head + li * 8), a);
#pragma unroll
            for (int i = 0; i < 8; ++i) v = fmaf(a[i], b[i], v);
        }
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (li == 0 && t < p.tokens) {
        const int64_t at = (int64_t)h * p.tokens + t;
        const float l = p.lse[at];
        p.stats[at] = l == -INFINITY ? make_float2(INFINITY, 0.f) : make_float2(l * kLog2e, v);
    }
}

struct BackwardParams {
    CUtensorMap q, k, v, dout;
    Rows dq, dk, dv;
    const float2* stats;
    Sequences seq;
    Packing packing;
    int32_t heads;  // of this kernel's CTAs: key heads for dkv, packs of query heads for dq
    int32_t group, dim, causal, clear;
    float scale, scale_log2;
    uint32_t* status;
    uint64_t wait_ns;
};

// Both kernels keep two tiles and stream two others: three stages of the one that is used first and last, two of the other.
template <int DP>
struct BackwardShape {
    static constexpr int kTileBytes = DP / 64 * kBlockBytes;
    static constexpr int kFirst = 3, kSecond = 2;
    static constexpr int kOffFirst = 2 * kTileBytes;
    static constexpr int kOffSecond = kOffFirst + kFirst * kTileBytes;
    static constexpr int kOffStats = kOffSecond + kSecond * kTileBytes;
    static constexpr int kOffBar = kOffStats + 2 * kRows * 8;
    static constexpr int kBars = 2 + 2 * kFirst + 2 * kSecond + 4 + 8 + 1;
    static constexpr int kOffPlace = kOffBar + kBars * 8;
    static constexpr int kSmem = (kOffPlace + 32 > 120 * 1024 ? kOffPlace + 32 : 120 * 1024);  // one CTA per SM
};
static_assert(BackwardShape<128>::kSmem <= 227 * 1024, "shared memory budget");

// Keys' gradients.  The products of block b (128 keys x 128 queries) in the order in which they are issued:
//   z(b)^T = k q^T | dv += p(b)^T do, z(b+1)^T | dk += dz(b)^T q, dp(b+1)^T = v do^T | ...
// While p is made from z, the tensor cores run dk and dp; while dz is made from dp, dv and the next z.
constexpr int kDkvThreads = 128 + 512;

template <int DP>
__global__ void __launch_bounds__(kDkvThreads, 1) attention_dkv_kernel(const __grid_constant__ BackwardParams p) {
    using Shape = BackwardShape<DP>;
    using Q = Ring<Shape::kFirst>;
    using D = Ring<Shape::kSecond>;
    extern __shared__ uint8_t smem[];
    if (smem_u32(smem) & 1023u) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusSmemLayout);
        return;
    }
    uint8_t* sK = smem;
    uint8_t* sV = smem + Shape::kTileBytes;
    uint8_t* sQ = smem + Shape::kOffFirst;
    uint8_t* sD = smem + Shape::kOffSecond;
    float* stats = reinterpret_cast<float*>(smem + Shape::kOffStats);  // [2][-lse, -delta][128]
    uint64_t* kv_full = reinterpret_cast<uint64_t*>(smem + Shape::kOffBar);  // [2]
    uint64_t* q_full = kv_full + 2;
    uint64_t* q_empty = q_full + Shape::kFirst;
    uint64_t* d_full = q_empty + Shape::kFirst;
    uint64_t* d_empty = d_full + Shape::kSecond;
    uint64_t* stats_full = d_empty + Shape::kSecond;  // [2]
    uint64_t* stats_empty = stats_full + 2;           // [2]
    uint64_t* z_full = stats_empty + 2;
    uint64_t* p_full = z_full + 1;
    uint64_t* dp_full = p_full + 1;
    uint64_t* dz_full = dp_full + 1;
    uint64_t* done = dz_full + 1;
    Place* where = reinterpret_cast<Place*>(smem + Shape::kOffPlace);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(where + 1);

    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int32_t head = (int32_t)(blockIdx.x % (uint32_t)p.heads), slot = (int32_t)(blockIdx.x / (uint32_t)p.heads);
    if (threadIdx.x == 96) {  // warp 0 looks for its place meanwhile
        for (int i = 0; i < 2; ++i) {
            mbar_init(&kv_full[i], 1);
            mbar_init(&stats_full[i], 32);
            mbar_init(&stats_empty[i], 16);
        }
        for (int i = 0; i < Shape::kFirst; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_empty[i], 1);
        }
        for (int i = 0; i < Shape::kSecond; ++i) {
            mbar_init(&d_full[i], 1);
            mbar_init(&d_empty[i], 1);
        }
        mbar_init(z_full, 1);
        mbar_init(p_full, 16);
        mbar_init(dp_full, 1);
        mbar_init(dz_full, 16);
        mbar_init(done, 1);
        fence_mbar_init();
        prefetch_tmap(&p.q);
        prefetch_tmap(&p.k);
        prefetch_tmap(&p.v);
        prefetch_tmap(&p.dout);
    }
    if (warp == 1) {
        tmem_alloc(tmem_holder, 512);
        tmem_relinquish();
    }
    grid_dependency_wait();
    allow_dependent_launch();
    if (warp == 0) {
        const Place w = find_place<true, Search::kCall>(p.seq, slot, kRows, 0, p.status);
        if (lane == 0) *where = w;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)uniform((int32_t)*tmem_holder);
    const Place at = place_of(where);
    const bool work = at.tile >= 0;
    const int32_t key0 = at.tile * kRows, ahead = at.len_k - at.len_q;
    const int32_t pack = p.packing.pack, tokens = p.packing.tokens;
    // query tiles that see these keys: from the one with the first query that sees the first key
    int32_t first = 0, tiles = 0;
    if (work) {
        first = p.causal ? max(key0 - ahead, 0) / tokens : 0;
        tiles = max((at.len_q + tokens - 1) / tokens - first, 0);
    }
    const int32_t blocks = tiles * (p.group / pack);  // tiles of each pack of query heads in turn
    constexpr uint32_t kZ = 0, kDp = 128, kDv = 256, kDk = 384;  // columns of tensor memory

    if (warp == 0) {
        // ---------------- TMA producer
        if (elect_one() && blocks > 0) {
            load_tile<DP>(sK, &p.k, &kv_full[0], head, at.k0 + key0);
            load_tile<DP>(sV, &p.v, &kv_full[1], head, at.k0 + key0);
            int q_armed = 0, d_armed = 0;
            int32_t h = head * p.group, token = at.q0 + first * tokens, tile = 0;
            for (int b = 0; b < blocks; ++b, token += tokens) {
                if (tile++ == tiles) {  // the next heads' first
                    tile = 1;
                    h += pack;
                    token = at.q0 + first * tokens;
                }
                if (b >= Shape::kFirst && !wait_bounded(&q_empty[Q::stage(b)], Q::parity(b - Shape::kFirst), p.wait_ns, p.status))
                    break;
                load_tile<DP>(sQ + Q::stage(b) * Shape::kTileBytes, &p.q, &q_full[Q::stage(b)], h, token, p.packing.rows());
                q_armed = b + 1;
                if (b >= Shape::kSecond && !wait_bounded(&d_empty[D::stage(b)], D::parity(b - Shape::kSecond), p.wait_ns, p.status))
                    break;
                load_tile<DP>(sD + D::stage(b) * Shape::kTileBytes, &p.dout, &d_full[D::stage(b)], h, token, p.packing.rows());
                d_armed = b + 1;
            }
            for (int i = 0; i < 2; ++i) wait_bounded(&kv_full[i], 0, p.wait_ns, p.status);
            for (int b = max(0, q_armed - Shape::kFirst); b < q_armed; ++b)
                wait_bounded(&q_full[Q::stage(b)], Q::parity(b), p.wait_ns, p.status);
            for (int b = max(0, d_armed - Shape::kSecond); b < d_armed; ++b)
                wait_bounded(&d_full[D::stage(b)], D::parity(b), p.wait_ns, p.status);
        }
    } else if (warp == 1) {
        // ---------------- tensor cores
        const uint32_t scores = idesc_bf16(kRows, kRows, 0, 0);
        const uint32_t sums = idesc_bf16(kRows, (uint32_t)(p.dim + 15) / 16 * 16, 0, 1);
        const int steps = (p.dim + 15) / 16;
        const uint32_t k_tile = columns_of(smem_u32(sK)), v_tile = columns_of(smem_u32(sV));
        bool ok = true;
        // waits for a streamed tile; rows behind the sequence, and those that no load fills, are cleared, as they are summed
        // over
        const int left_last = (at.len_q - (first + tiles - 1) * tokens) * pack, left_else = p.packing.rows();
        auto ready = [&](uint64_t* bar, uint32_t parity, uint8_t* tile, int at_tile) {
            ok = ok && warp_wait(bar, parity, p.wait_ns, p.status);
            if (!ok) return;
            const int left = at_tile == tiles - 1 ? left_last : left_else;
            if (left < kRows) {
                clear_rows<DP>(tile, left);
                fence_async_smem();
                __syncwarp();
            }
            tc_fence_after();
        };
        int next = 0;  // query tile of the block whose scores are made next
        auto make_z = [&](int b) {
            uint8_t* tile = sQ + Q::stage(b) * Shape::kTileBytes;
            ready(&q_full[Q::stage(b)], Q::parity(b), tile, next);
            if (ok && elect_one()) {
                const uint32_t q_tile = columns_of(smem_u32(tile));
#pragma unroll
                for (int k = 0; k < DP / 16; ++k)
                    if (k < steps) mma_ss(tmem + kZ, k_tile + column_step(k), q_tile + column_step(k), scores, k != 0);
                tc_commit(z_full);
            }
        };
        auto make_dp = [&](int b) {
            uint8_t* tile = sD + D::stage(b) * Shape::kTileBytes;
            ready(&d_full[D::stage(b)], D::parity(b), tile, next);
            next = next + 1 == tiles ? 0 : next + 1;
            if (ok && elect_one()) {
                const uint32_t d_tile = columns_of(smem_u32(tile));
#pragma unroll
                for (int k = 0; k < DP / 16; ++k)
                    if (k < steps) mma_ss(tmem + kDp, v_tile + column_step(k), d_tile + column_step(k), scores, k != 0);
                tc_commit(dp_full);
            }
        };
        if (blocks > 0) {
            ok = warp_wait(&kv_full[0], 0, p.wait_ns, p.status);
            make_z(0);
            ok = ok && warp_wait(&kv_full[1], 0, p.wait_ns, p.status);
            make_dp(0);
        }
        for (int b = 0; ok && b < blocks; ++b) {
            ok = warp_wait(p_full, (uint32_t)b & 1u, p.wait_ns, p.status);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                const uint32_t d_tile = rows_of_tile(smem_u32(sD + D::stage(b) * Shape::kTileBytes));
#pragma unroll
                for (int k = 0; k < kRows / 16; ++k)
                    mma_ts(tmem + kDv, tmem + kZ + packed_column<32>(k), d_tile + k * kRowStep, sums, b != 0 || k != 0);
                tc_commit(&d_empty[D::stage(b)]);  // dp(b) came before
            }
            if (b + 1 < blocks) make_z(b + 1);
            ok = ok && warp_wait(dz_full, (uint32_t)b & 1u, p.wait_ns, p.status);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                const uint32_t q_tile = rows_of_tile(smem_u32(sQ + Q::stage(b) * Shape::kTileBytes));
#pragma unroll
                for (int k = 0; k < kRows / 16; ++k)
                    mma_ts(tmem + kDk, tmem + kDp + packed_column<32>(k), q_tile + k * kRowStep, sums, b != 0 || k != 0);
                tc_commit(&q_empty[Q::stage(b)]);
            }
            if (b + 1 < blocks) make_dp(b + 1);
        }
        if (elect_one()) tc_commit(done);
        warp_wait(done, 0, p.wait_ns, p.status);
    } else if (warp == 2) {
        // ---------------- the queries' statistics
        int32_t q = first * tokens, tile = 0, behind[kRows / 32];  // this lane's rows: token in the tile
        const float2* from[kRows / 32];
#pragma unroll
        for (int i = 0; i < kRows / 32; ++i) {
            const int r = i * 32 + lane;
            behind[i] = r < p.packing.rows() ? r / pack : 1 << 30;
            from[i] = p.stats + (int64_t)(head * p.group + r % pack) * p.seq.tokens_q + at.q0 + r / pack;
        }
        for (int b = 0; b < blocks; ++b, q += tokens) {
            const int s = b & 1;
            if (tile++ == tiles) {  // the next heads' first
                tile = 1;
                q = first * tokens;
#pragma unroll
                for (int i = 0; i < kRows / 32; ++i) from[i] += (int64_t)pack * p.seq.tokens_q;
            }
            if (b >= 2 && !warp_wait(&stats_empty[s], (uint32_t)(b / 2 - 1) & 1u, p.wait_ns, p.status)) break;
#pragma unroll
            for (int i = 0; i < kRows / 32; ++i) {
                const int r = i * 32 + lane;
                float2 v = make_float2(INFINITY, 0.f);
                if (behind[i] < at.len_q - q) v = from[i][q];
                stats[s * 2 * kRows + r] = -v.x;
                stats[s * 2 * kRows + kRows + r] = -v.y;
            }
            mbar_arrive(&stats_full[s]);
        }
    } else if (warp == 3) {
        if (p.clear)
            clear_outside(p.seq.cu_k, p.seq.count, p.seq.tokens_k, [&](int32_t token) {
                p.dk.clear(token, p.heads, p.dim);
                p.dv.clear(token, p.heads, p.dim);
            });
    } else if (warp >= 4) {
        // ---------------- p and dz: a warpgroup for each quarter of the queries, a warp for 32 keys.  A thread holds two
        // neighbouring queries of every eight, for four keys: the queries' statistics, which differ along a row here, are
        // then read from shared memory once for four keys instead of for each (8 instead of 48 cycles a warp and block, of
        // which the tensor cores' operands already take 1536, and the loads 512, in a block of 2048).
        const int part = (warp - 4) >> 2, quad = warp & 3;
        const int32_t key = key0 + quad * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t z_at = lanes + kZ + part * 32, dp_at = lanes + kDp + part * 32;
        constexpr uint32_t kLower = 16u << 16;  // the other 16 lanes
        const int column = 2 * (lane & 3);      // of each eight
        const int32_t upper = key0 + quad * 32 + (lane >> 2);  // key of the thread's first row; the others 8 apart
        const float2 scale2 = make_float2(p.scale_log2, p.scale_log2);
        bool ok = true;
        int32_t q = first * tokens, tile = 0;
        for (int b = 0; b < blocks; ++b, q += tokens) {
            const int s = b & 1;
            if (tile++ == tiles) tile = 1, q = first * tokens;
            ok = warp_wait(&stats_full[s], (uint32_t)(b / 2) & 1u, p.wait_ns, p.status) &&
                 warp_wait(z_full, (uint32_t)b & 1u, p.wait_ns, p.status);
            if (!ok) break;
            tc_fence_after();
            const float* lse = stats + s * 2 * kRows + part * 32 + column;  // negated
            const float* delta = lse + kRows;
            uint32_t z[2][16];
            tmem_ld_16x256b_x4(z_at, z[0]);
            tmem_ld_16x256b_x4(z_at + kLower, z[1]);
            float2 l[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) l[i] = *reinterpret_cast<const float2*>(lse + 8 * i);
            tmem_ld_wait();
            float2 pr[4][4];  // [row][eight]
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t* v = z[r >> 1] + 4 * i + 2 * (r & 1);
                    const float2 e = f2_fma(make_float2(__uint_as_float(v[0]), __uint_as_float(v[1])), scale2, l[i]);
                    pr[r][i] = make_float2(exp2_approx(e.x), exp2_approx(e.y));
                }
            if (p.causal && q + ahead < key0 + kRows - 1) {  // queries below key - ahead do not see the key
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int hidden = min((upper + 8 * r - ahead - q) * pack, kRows) - part * 32 - column;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (8 * i < hidden) pr[r][i].x = 0.f;
                        if (8 * i + 1 < hidden) pr[r][i].y = 0.f;
                    }
                }
            }
            uint32_t w[2][8];
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) w[r >> 1][2 * i + (r & 1)] = pack_bf16(pr[r][i].x, pr[r][i].y);
            tmem_st_16x128b_x4(z_at, w[0]);
            tmem_st_16x128b_x4(z_at + kLower, w[1]);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full);
#pragma unroll
            for (int i = 0; i < 4; ++i) l[i] = *reinterpret_cast<const float2*>(delta + 8 * i);
            ok = warp_wait(dp_full, (uint32_t)b & 1u, p.wait_ns, p.status);
            if (!ok) break;
            tc_fence_after();
            tmem_ld_16x256b_x4(dp_at, z[0]);
            tmem_ld_16x256b_x4(dp_at + kLower, z[1]);
            tmem_ld_wait();
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t* v = z[r >> 1] + 4 * i + 2 * (r & 1);
                    const float2 e = f2_mul(pr[r][i], f2_add(make_float2(__uint_as_float(v[0]), __uint_as_float(v[1])), l[i]));
                    w[r >> 1][2 * i + (r & 1)] = pack_bf16(e.x, e.y);
                }
            tmem_st_16x128b_x4(dp_at, w[0]);
            tmem_st_16x128b_x4(dp_at + kLower, w[1]);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(dz_full);
                mbar_arrive(&stats_empty[s]);
            }
        }
        // two warpgroups for dv, two for dk, each half of the columns
        const bool keys = part >= 2;
        const Rows& rows = keys ? p.dk : p.dv;
        const bool inside = work && key < at.len_k;
        bf16* to = rows.at(at.k0 + key, head);
        const int cut = (p.dim / 2 + 15) / 16 * 16, from = part & 1 ? cut : 0;
        if (blocks > 0) {
            ok = ok && warp_wait(done, 0, p.wait_ns, p.status);
            if (ok) {
                tc_fence_after();
                store_rows(lanes + (keys ? kDk : kDv) + from, part & 1 ? p.dim - cut : min(cut, p.dim), keys ? p.scale : 1.f,
                          to + from, inside);
            }
        } else if (inside && (part & 1) == 0) {
            store_zeros(p.dim, to);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Queries' gradients.  z and dp of the next block are made while dz of this one is; z has two places, and dz takes its own
// block's, so that dp is free again as soon as it has been read.  dz(b + 1) may be ready before the lane that issues looks for
// dz(b): two barriers, as a barrier's parity tells neighbouring phases apart and no more.
constexpr int kDqThreads = 128 + 512;

template <int DP>
__global__ void __launch_bounds__(kDqThreads, 1) attention_dq_kernel(const __grid_constant__ BackwardParams p) {
    using Shape = BackwardShape<DP>;
    using K = Ring<Shape::kFirst>;
    using V = Ring<Shape::kSecond>;
    extern __shared__ uint8_t smem[];
    if (smem_u32(smem) & 1023u) {
        if (threadIdx.x == 0) atomicOr(p.status, kStatusSmemLayout);
        return;
    }
    uint8_t* sQ = smem;
    uint8_t* sD = smem + Shape::kTileBytes;
    uint8_t* sK = smem + Shape::kOffFirst;
    uint8_t* sV = smem + Shape::kOffSecond;
    uint64_t* qd_full = reinterpret_cast<uint64_t*>(smem + Shape::kOffBar);  // [2]
    uint64_t* k_full = qd_full + 2;
    uint64_t* k_empty = k_full + Shape::kFirst;
    uint64_t* v_full = k_empty + Shape::kFirst;
    uint64_t* v_empty = v_full + Shape::kSecond;
    uint64_t* z_full = v_empty + Shape::kSecond;  // [2]
    uint64_t* dp_full = z_full + 2;
    uint64_t* dp_read = dp_full + 1;
    uint64_t* dz_full = dp_read + 1;  // [2]
    uint64_t* done = dz_full + 2;
    Place* where = reinterpret_cast<Place*>(smem + Shape::kOffPlace);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(where + 1);

    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int32_t head0 = (int32_t)(blockIdx.x % (uint32_t)p.heads) * p.packing.pack;
    const int32_t slot = (int32_t)(blockIdx.x / (uint32_t)p.heads), tokens = p.packing.tokens;
    if (threadIdx.x == 96) {  // warp 0 looks for its place meanwhile
        for (int i = 0; i < 2; ++i) {
            mbar_init(&qd_full[i], 1);
            mbar_init(&z_full[i], 1);
            mbar_init(&dz_full[i], 16);
        }
        for (int i = 0; i < Shape::kFirst; ++i) {
            mbar_init(&k_full[i], 1);
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < Shape::kSecond; ++i) {
            mbar_init(&v_full[i], 1);
            mbar_init(&v_empty[i], 1);
        }
        mbar_init(dp_full, 1);
        mbar_init(dp_read, 16);
        mbar_init(done, 1);
        fence_mbar_init();
        prefetch_tmap(&p.q);
        prefetch_tmap(&p.k);
        prefetch_tmap(&p.v);
        prefetch_tmap(&p.dout);
    }
    if (warp == 1) {
        tmem_alloc(tmem_holder, 512);
        tmem_relinquish();
    }
    grid_dependency_wait();
    allow_dependent_launch();
    if (warp == 0) {
        const Place w = find_place<false, Search::kCall>(p.seq, slot, tokens, 0, p.status);
        if (lane == 0) *where = w;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)uniform((int32_t)*tmem_holder);
    Place at = place_of(where);
    const bool work = at.tile >= 0;
    if (work && p.causal) at.tile = (at.len_q + tokens - 1) / tokens - 1 - at.tile;  // those that see the most keys first
    const int32_t row0 = at.tile * tokens, ahead = at.len_k - at.len_q;
    int32_t blocks = 0;
    if (work) {
        const int32_t last = min(row0 + tokens, at.len_q) - 1;
        const int32_t keys = p.causal ? min(at.len_k, max(last + ahead + 1, 0)) : at.len_k;
        blocks = (keys + kRows - 1) / kRows;
    }
    constexpr uint32_t kZ = 0, kDp = 256, kDq = 384;  // columns of tensor memory; z(b) at kZ + (b & 1) * 128

    if (warp == 0) {
        // ---------------- TMA producer
        if (elect_one() && blocks > 0) {
            const int32_t key_head = head0 / p.group;
            load_tile<DP>(sQ, &p.q, &qd_full[0], head0, at.q0 + row0, p.packing.rows());
            int k_armed = 0, v_armed = 0;
            for (int b = 0; b < blocks; ++b) {
                const int32_t token = at.k0 + b * kRows;
                if (b >= Shape::kFirst && !wait_bounded(&k_empty[K::stage(b)], K::parity(b - Shape::kFirst), p.wait_ns, p.status))
                    break;
                load_tile<DP>(sK + K::stage(b) * Shape::kTileBytes, &p.k, &k_full[K::stage(b)], key_head, token);
                k_armed = b + 1;
                if (b == 0) load_tile<DP>(sD, &p.dout, &qd_full[1], head0, at.q0 + row0, p.packing.rows());
                if (b >= Shape::kSecond && !wait_bounded(&v_empty[V::stage(b)], V::parity(b - Shape::kSecond), p.wait_ns, p.status))
                    break;
                load_tile<DP>(sV + V::stage(b) * Shape::kTileBytes, &p.v, &v_full[V::stage(b)], key_head, token);
                v_armed = b + 1;
            }
            for (int i = 0; i < 2; ++i) wait_bounded(&qd_full[i], 0, p.wait_ns, p.status);
            for (int b = max(0, k_armed - Shape::kFirst); b < k_armed; ++b)
                wait_bounded(&k_full[K::stage(b)], K::parity(b), p.wait_ns, p.status);
            for (int b = max(0, v_armed - Shape::kSecond); b < v_armed; ++b)
                wait_bounded(&v_full[V::stage(b)], V::parity(b), p.wait_ns, p.status);
        }
    } else if (warp == 1) {
        // ---------------- tensor cores
        const uint32_t scores = idesc_bf16(kRows, kRows, 0, 0);
        const uint32_t sums = idesc_bf16(kRows, (uint32_t)(p.dim + 15) / 16 * 16, 0, 1);
        const int steps = (p.dim + 15) / 16;
        const uint32_t q_tile = columns_of(smem_u32(sQ)), d_tile = columns_of(smem_u32(sD));
        bool ok = true;
        auto ready = [&](uint64_t* bar, uint32_t parity, uint8_t* tile, int b) {
            ok = ok && warp_wait(bar, parity, p.wait_ns, p.status);
            if (!ok) return;
            const int left = at.len_k - b * kRows;
            if (left < kRows) {  // k is summed over, and 0 times what v holds there must be 0
                clear_rows<DP>(tile, left);
                fence_async_smem();
                __syncwarp();
            }
            tc_fence_after();
        };
        auto make_z = [&](int b) {
            uint8_t* tile = sK + K::stage(b) * Shape::kTileBytes;
            ready(&k_full[K::stage(b)], K::parity(b), tile, b);
            if (ok && elect_one()) {
                const uint32_t k_tile = columns_of(smem_u32(tile));
#pragma unroll
                for (int k = 0; k < DP / 16; ++k)
                    if (k < steps) mma_ss(tmem + kZ + (b & 1) * 128, q_tile + column_step(k), k_tile + column_step(k), scores, k != 0);
                tc_commit(&z_full[b & 1]);
            }
        };
        auto make_dp = [&](int b) {
            uint8_t* tile = sV + V::stage(b) * Shape::kTileBytes;
            ready(&v_full[V::stage(b)], V::parity(b), tile, b);
            if (ok && elect_one()) {
                const uint32_t v_tile = columns_of(smem_u32(tile));
#pragma unroll
                for (int k = 0; k < DP / 16; ++k)
                    if (k < steps) mma_ss(tmem + kDp, d_tile + column_step(k), v_tile + column_step(k), scores, k != 0);
                tc_commit(dp_full);
                tc_commit(&v_empty[V::stage(b)]);
            }
        };
        if (blocks > 0) {
            ok = warp_wait(&qd_full[0], 0, p.wait_ns, p.status);
            make_z(0);
            ok = ok && warp_wait(&qd_full[1], 0, p.wait_ns, p.status);
            make_dp(0);
        }
        for (int b = 0; ok && b < blocks; ++b) {
            if (b + 1 < blocks) {
                make_z(b + 1);  // over dz(b - 1), which the product before has read
                ok = ok && warp_wait(dp_read, (uint32_t)b & 1u, p.wait_ns, p.status);
                tc_fence_after();
                make_dp(b + 1);
            }
            ok = ok && warp_wait(&dz_full[b & 1], (uint32_t)(b / 2) & 1u, p.wait_ns, p.status);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                const uint32_t k_tile = rows_of_tile(smem_u32(sK + K::stage(b) * Shape::kTileBytes));
#pragma unroll
                for (int k = 0; k < kRows / 16; ++k)
                    mma_ts(tmem + kDq, tmem + kZ + (b & 1) * 128 + packed_column<32>(k), k_tile + k * kRowStep, sums,
                           b != 0 || k != 0);
                tc_commit(&k_empty[K::stage(b)]);
            }
        }
        if (elect_one()) tc_commit(done);
        warp_wait(done, 0, p.wait_ns, p.status);
    } else if (warp == 2) {
        if (p.clear)
            clear_outside(p.seq.cu_q, p.seq.count, p.seq.tokens_q,
                          [&](int32_t token) { p.dq.clear(token, p.heads * p.packing.pack, p.dim); });
    } else if (warp >= 4) {
        // ---------------- p and dz: a lane for each query, a warpgroup for each quarter of the keys
        const int part = (warp - 4) >> 2, quad = warp & 3;
        const int32_t r = quad * 32 + lane, row = row0 + r / p.packing.pack, head = head0 + r % p.packing.pack;
        const bool inside = work && r < p.packing.rows() && row < at.len_q;
        const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t dp_at = lanes + kDp + part * 32;
        const int32_t last = p.causal ? min(at.len_k - 1, row + ahead) : at.len_k - 1;  // key that this query sees last
        const int32_t least = p.causal ? min(at.len_k - 1, row0 + ahead) : at.len_k - 1;
        float2 stat = make_float2(INFINITY, 0.f);
        if (inside) stat = p.stats[(int64_t)head * p.seq.tokens_q + at.q0 + row];
        const float2 scale2 = make_float2(p.scale_log2, p.scale_log2);
        const float2 lse2 = make_float2(-stat.x, -stat.x), delta2 = make_float2(stat.y, stat.y);
        bool ok = true;
        for (int b = 0; b < blocks; ++b) {
            const uint32_t z_at = lanes + kZ + (b & 1) * 128 + part * 32;
            ok = warp_wait(&z_full[b & 1], (uint32_t)(b / 2) & 1u, p.wait_ns, p.status);
            if (!ok) break;
            tc_fence_after();
            float2 pr[16];
            {
                uint32_t z[32];
                tmem_ld_32x32b_x32(z_at, z);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 e = f2_fma(make_float2(__uint_as_float(z[2 * i]), __uint_as_float(z[2 * i + 1])), scale2, lse2);
                    pr[i] = make_float2(exp2_approx(e.x), exp2_approx(e.y));
                }
            }
            if (least - b * kRows < kRows - 1) {
                const int seen = last - b * kRows - part * 32;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    if (2 * i > seen) pr[i].x = 0.f;
                    if (2 * i + 1 > seen) pr[i].y = 0.f;
                }
            }
            ok = warp_wait(dp_full, (uint32_t)b & 1u, p.wait_ns, p.status);
            if (!ok) break;
            tc_fence_after();
            uint32_t dp[32], w[16];
            tmem_ld_32x32b_x32(dp_at, dp);
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(dp_read);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float2 e = f2_mul(pr[i], f2_sub(make_float2(__uint_as_float(dp[2 * i]), __uint_as_float(dp[2 * i + 1])), delta2));
                w[i] = pack_bf16(e.x, e.y);
            }
            tmem_st_32x32b_x16(z_at, w);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&dz_full[b & 1]);
        }
        bf16* to = p.dq.at(at.q0 + row, head);
        if (blocks > 0) {
            ok = ok && warp_wait(done, 0, p.wait_ns, p.status);
            if (ok) {  // each warpgroup writes its share of the columns
                tc_fence_after();
                const int width = (p.dim / 4 + 15) / 16 * 16, from = part * width;
                const bool weight = stat.x != INFINITY;  // otherwise zeros, as in the forward pass
                store_rows(lanes + kDq + from, min(width, p.dim - from), p.scale, to + from, inside && weight);
                if (inside && !weight) store_zeros(min(width, p.dim - from), to + from);
            }
        } else if (inside && part == 0) {
            store_zeros(p.dim, to);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ------------------------------------------------------------------ host
struct Call {
    Heads q, k, v, out, rest;
    int64_t tokens_q, tokens_k;
    Sequences seq;
    int32_t dim, group;
    Packing packing;
};

// The divisor of the group that fills the most of a tile's 128 rows, the largest of those that fill as many.
Packing packing_of(int group) {
    Packing best{1, kRows};
    for (int d = 2; d <= std::min(group, kRows); ++d)
        if (group % d == 0 && kRows / d * d >= best.pack * best.tokens) best = {d, kRows / d};
    return best;
}

mxfp4_status check_operand(const char* what, const char* name, const mxfp4_heads* given, int64_t tokens, int64_t dim,
                           bool written, Heads* out) {
    mxfp4_status st = check_heads(what, name, given, tokens, dim, written, out);
    if (st) return st;
    if (out->dtype != MXFP4_OUT_BF16)
        return record_error(MXFP4_ERR_INVALID_ARG, "%s: %s must be bf16", what, name);
    if (tokens > 0 && !heads_aligned(*out, 16))
        return record_error(MXFP4_ERR_MISALIGNED, "%s: rows of %s must start on multiples of 16 bytes", what, name);
    return MXFP4_OK;
}

mxfp4_status check_call(const char* what, const mxfp4_heads* q, const mxfp4_heads* k, const mxfp4_heads* v,
                        int64_t tokens_q, int64_t tokens_k, int64_t dim, const int32_t* cu_q, const int32_t* cu_k,
                        int64_t seqs, int causal, float scale, int zero_outside, Call* c) {
    if (tokens_q < 0 || tokens_k < 0 || seqs < 0)
        return record_error(MXFP4_ERR_INVALID_ARG, "%s: negative size", what);
    if (tokens_q >= (1 << 30) || tokens_k >= (1 << 30) || seqs >= (1 << 24))
        return record_error(MXFP4_ERR_UNSUPPORTED_SHAPE, "%s: tokens must be below 2^30, sequences below 2^24", what);
    if (dim < 8 || dim > 128 || dim % 8)
        return record_error(MXFP4_ERR_UNSUPPORTED_SHAPE, "%s: head_dim %lld must be a multiple of 8, at most 128", what,
                            (long long)dim);
    if ((causal != 0 && causal != 1) || (zero_outside != 0 && zero_outside != 1))
        return record_error(MXFP4_ERR_INVALID_ARG, "%s: causal and zero_outside must be 0 or 1", what);
    if (!(scale > 0.f) || !std::isfinite(scale * kLog2e))
        return record_error(MXFP4_ERR_INVALID_ARG, "%s: scale must be positive and finite", what);
    mxfp4_status st;
    if ((st = check_operand(what, "q", q, tokens_q, dim, false, &c->q))) return st;
    if ((st = check_operand(what, "k", k, tokens_k, dim, false, &c->k))) return st;
    if ((st = check_operand(what, "v", v, tokens_k, dim, false, &c->v))) return st;
    if (c->k.heads != c->v.heads || c->q.heads % c->k.heads)
        return record_error(MXFP4_ERR_UNSUPPORTED_SHAPE, "%s: %d query heads, %d of keys and %d of values do not fit", what,
                            c->q.heads, c->k.heads, c->v.heads);
    if (!cu_q != !cu_k) return record_error(MXFP4_ERR_INVALID_ARG, "%s: one of cu_q and cu_k is NULL", what);
    if ((reinterpret_cast<uintptr_t>(cu_q) | reinterpret_cast<uintptr_t>(cu_k)) % 4)
        return record_error(MXFP4_ERR_MISALIGNED, "%s: cu_q or cu_k misaligned", what);
    if (!cu_q && (seqs == 0 ? tokens_q || tokens_k : tokens_q % seqs || tokens_k % seqs))
        return record_error(MXFP4_ERR_UNSUPPORTED_SHAPE, "%s: %lld sequences of equal lengths do not fit", what,
                            (long long)seqs);
    c->tokens_q = tokens_q;
    c->tokens_k = tokens_k;
    c->dim = (int32_t)dim;
    c->group = c->q.heads / c->k.heads;
    c->packing = packing_of(c->group);
    // grids: a place for each tile, and one more for each sequence
    if ((tokens_q / c->packing.tokens + seqs + 1) * (c->q.heads / c->packing.pack) > INT32_MAX ||
        (tokens_k / kRows + seqs + 1) * c->k.heads > INT32_MAX)
        return record_error(MXFP4_ERR_UNSUPPORTED_SHAPE, "%s: too many tiles", what);
    c->seq = {cu_q, cu_k, (int32_t)seqs, (int32_t)tokens_q, (int32_t)tokens_k,
              seqs && !cu_q ? (int32_t)(tokens_q / seqs) : 0, seqs && !cu_q ? (int32_t)(tokens_k / seqs) : 0};
    return MXFP4_OK;
}

// out, and the rest of its rounding, which may be NULL.
mxfp4_status check_output(const char* what, const mxfp4_heads* out, const mxfp4_heads* rest, bool written, Call* c) {
    mxfp4_status st = check_operand(what, "out", out, c->tokens_q, c->dim, written, &c->out);
    if (!st && rest) st = check_operand(what, "rest", rest, c->tokens_q, c->dim, written, &c->rest);
    if (st) return st;
    if (c->out.heads != c->q.heads || (rest && c->rest.heads != c->q.heads))
        return record_error(MXFP4_ERR_INVALID_ARG, "%s: out or rest has other heads than q", what);
    return MXFP4_OK;
}

struct Named {
    const char* name;
    const Heads* heads;
    int64_t tokens;
};
// No output over an input that other CTAs still read, nor over another output.  `own`: inputs of which a CTA reads only the
// rows that it writes itself, so that the output may be the same tensor.
mxfp4_status check_apart(const char* what, const Named& written, std::initializer_list<Named> others,
                         std::initializer_list<Named> own, int64_t dim) {
    auto overlap = [&](const Named& x) { return heads_overlap(*written.heads, written.tokens, *x.heads, x.tokens, dim); };
    for (const Named& x : others)
        if (overlap(x)) return record_error(MXFP4_ERR_INVALID_ARG, "%s: %s overlaps %s", what, written.name, x.name);
    for (const Named& x : own)
        if (overlap(x) && !same_heads(*written.heads, *x.heads))
            return record_error(MXFP4_ERR_INVALID_ARG, "%s: %s overlaps %s and is not the same tensor", what, written.name, x.name);
    return MXFP4_OK;
}

// Places of tiles of `rows` tokens: no fewer than there are tiles.
int64_t places(const Call& c, int64_t tokens, int32_t len, int rows) {
    if (c.seq.cu_q) return tokens / rows + c.seq.count;
    return (int64_t)c.seq.count * ((len + rows - 1) / rows);
}

// Whether the keys of a pair of query tiles are shared out over several CTAs: where the pairs leave more than half of the SMs
// without one, sequences have eight key tiles or more on the average, and a CTA has at least kSaved tiles fewer to go through
// (few rows) or kSavedMany (many, whose parts take longer to join).  A part is `chunk` key tiles, so many that there is a part
// for each SM at most (a CTA's start and end cost as much as some six key tiles), but four at least.
// 32 and 8 heads of 128, shared out and not: 1 query over 1024 keys 16.5 and 18.6 us, 2048 16.6 and 27.9, 32768 41 and 329;
// 4 sequences of 4096 24.7 and 47.6; 64 queries over 1024 keys 22.8 and 20.6 (4 tiles fewer), 2048 22.7 and 30.9 (12);
// 256 queries over 1024 26.9 and 20.6, 4096 43.3 and 53.5 (16).
// `places`: of all parts, no fewer than there are whatever the sequences' lengths.
constexpr int kSaved = 4, kSavedMany = 10, kFewRows = 2 * kRows;
constexpr int kSms = 152;  // of a GB300: the workspace does not depend on the device
struct Split {
    int32_t chunk;  // 0: none
    int64_t places;
};
Split split_of(int64_t q_tokens, int64_t k_tokens, int64_t q_heads, int64_t k_heads, int64_t seqs) {
    Split s{0, 0};
    if (q_tokens <= 0 || k_tokens <= 0 || q_heads <= 0 || k_heads <= 0 || seqs <= 0 || q_heads % k_heads) return s;
    const Packing packing = packing_of((int)std::min<int64_t>(q_heads / k_heads, 65535));
    const int64_t blocks = q_heads / packing.pack, pairs = q_tokens / (2 * packing.tokens) + seqs;
    const int64_t tiles = k_tokens / kRows;  // of keys, and one more for each sequence
    if (2 * pairs * blocks > kSms || tiles < 8 * seqs) return s;
    // one pair of query tiles in each sequence, or all in one that has all the keys
    const bool one = q_tokens <= 2 * packing.tokens;
    const int64_t parts = std::max<int64_t>(1, one ? kSms / blocks - seqs : kSms / (blocks * pairs) - 1);
    const int32_t chunk = (int32_t)std::max<int64_t>(4, (tiles + parts - 1) / parts);
    const int saved = q_tokens * q_heads <= kFewRows ? kSaved : kSavedMany;
    if ((chunk + saved) * seqs > tiles) return s;
    s.chunk = chunk;
    s.places = one ? tiles / s.chunk + 2 * seqs : pairs * (tiles / s.chunk + 2);
    return s;
}
size_t part_bytes(int64_t dim) { return 2 * kRows * ((size_t)dim * sizeof(float) + sizeof(float4)); }

template <class Params, class Kern>
cudaError_t launch_tiles(Kern kern, DeviceSlots& ready, const Params& p, int64_t ctas, int threads, int smem,
                         cudaStream_t s) {
    if (ctas == 0) return cudaSuccess;
    int unused = 0;
    cudaError_t e = per_device_setting(ready, &unused, [&](int, int* v) {
        *v = 1;
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (e != cudaSuccess) return e;
    return launch_overlapped(kern, dim3((unsigned)ctas), dim3((unsigned)threads), (size_t)smem, s, 1, true, p);
}

// Of a tensor of no tokens nothing is loaded: its map is that of `other`.
bool map_of(CUtensorMap* map, const Heads& h, int64_t tokens, const Heads& other, int64_t other_tokens, int64_t dim,
            Packing box = {1, kRows}) {
    const Heads& x = tokens > 0 ? h : other;
    return encode_heads_map(map, x.data, tokens > 0 ? tokens : other_tokens, x.heads, dim, x.token_stride, x.head_stride,
                            (uint32_t)box.pack, (uint32_t)box.tokens);
}

Rows rows_of(const Heads& h) { return {static_cast<bf16*>(h.data), h.token_stride, h.head_stride}; }

}  // namespace
}  // namespace mx

using namespace mx;

extern "C" size_t mxfp4_attention_workspace_bytes(int64_t q_tokens, int64_t k_tokens, int64_t head_dim, int64_t q_heads,
                                                  int64_t k_heads, int64_t seqs) {
    const Split s = split_of(q_tokens, k_tokens, q_heads, k_heads, seqs);
    if (s.chunk == 0 || head_dim <= 0 || head_dim > 128) return 0;
    const Packing packing = packing_of((int)std::min<int64_t>(q_heads / k_heads, 65535));
    return (size_t)(s.places * (q_heads / packing.pack)) * part_bytes(head_dim);
}

extern "C" mxfp4_status mxfp4_attention(const mxfp4_heads* q, const mxfp4_heads* k, const mxfp4_heads* v,
                                        int64_t q_tokens, int64_t k_tokens, int64_t head_dim, const int32_t* cu_q,
                                        const int32_t* cu_k, int64_t seqs, int causal, float scale, int zero_outside,
                                        const mxfp4_heads* out, const mxfp4_heads* rest, float* lse, void* ws,
                                        size_t ws_bytes, mxfp4_stream_t stream) {
    const char* what = "attention";
    Call c{};
    mxfp4_status st = check_call(what, q, k, v, q_tokens, k_tokens, head_dim, cu_q, cu_k, seqs, causal, scale, zero_outside, &c);
    if (st) return st;
    if ((st = check_output(what, out, rest, true, &c))) return st;
    const Named q_{"q", &c.q, q_tokens}, k_{"k", &c.k, k_tokens}, v_{"v", &c.v, k_tokens};
    const Named out_{"out", &c.out, q_tokens}, rest_{"rest", &c.rest, q_tokens};
    if ((st = check_apart(what, out_, {k_, v_, rest_}, {q_}, head_dim))) return st;
    if ((st = check_apart(what, rest_, {k_, v_}, {q_}, head_dim))) return st;
    const bool clear = zero_outside && cu_q;  // sequences of equal lengths leave nothing out
    if (q_tokens == 0 || (seqs == 0 && !clear)) return record_error(MXFP4_OK, "%s", "");
    if (!lse) return record_error(MXFP4_ERR_INVALID_ARG, "%s: lse is NULL", what);
    if (reinterpret_cast<uintptr_t>(lse) % 4) return record_error(MXFP4_ERR_MISALIGNED, "%s: lse misaligned", what);
    const Split split = split_of(q_tokens, k_tokens, c.q.heads, c.k.heads, seqs);
    if (split.chunk > 0) {
        const size_t need = mxfp4_attention_workspace_bytes(q_tokens, k_tokens, head_dim, c.q.heads, c.k.heads, seqs);
        if (!ws || ws_bytes < need)
            return record_error(MXFP4_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", what, need);
        if (reinterpret_cast<uintptr_t>(ws) % 256)
            return record_error(MXFP4_ERR_MISALIGNED, "%s: workspace not 256-byte aligned", what);
    }
    if ((st = ensure_device())) return st;
    ForwardParams p{};
    if (!map_of(&p.q, c.q, q_tokens, c.q, q_tokens, head_dim, c.packing) ||
        !map_of(&p.k, c.k, k_tokens, c.q, q_tokens, head_dim) || !map_of(&p.v, c.v, k_tokens, c.q, q_tokens, head_dim))
        return record_error(MXFP4_ERR_CUDA, "%s: tensor map encoding failed", what);
    p.out = rows_of(c.out);
    p.rest = rows_of(c.rest);
    p.lse = lse;
    p.seq = c.seq;
    p.packing = c.packing;
    p.head_blocks = c.q.heads / c.packing.pack;
    p.group = c.group;
    p.dim = c.dim;
    p.causal = causal;
    p.clear = clear;
    p.chunk = split.chunk;
    if (p.chunk > 0) {
        p.part = static_cast<float*>(ws);
        p.part_stats = reinterpret_cast<float4*>(p.part + split.places * p.head_blocks * 2 * kRows * head_dim);
    }
    p.scale_log2 = scale * kLog2e;
    p.status = device_status_ptr();
    p.wait_ns = wait_limit_ns();
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    int64_t ctas = (p.chunk > 0 ? split.places : places(c, q_tokens, c.seq.len_q, 2 * c.packing.tokens)) * p.head_blocks;
    if (clear) ctas = std::max<int64_t>(ctas, 1);
    static DeviceSlots wide, narrow;
    cudaError_t e =
        c.dim > 64 ? launch_tiles(attention_kernel<128>, wide, p, ctas, kForwardThreads, ForwardShape<128>::kSmem, s)
                   : launch_tiles(attention_kernel<64>, narrow, p, ctas, kForwardThreads, ForwardShape<64>::kSmem, s);
    if (e != cudaSuccess) return record_error(MXFP4_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
    if (p.chunk > 0) {
        e = launch_overlapped(join_kernel, dim3((unsigned)ctas, kJoinCtas), dim3(kJoinThreads), 0, s, 1, true, p);
        if (e != cudaSuccess) return record_error(MXFP4_ERR_CUDA, "%s join launch: %s", what, cudaGetErrorString(e));
    }
    return record_error(MXFP4_OK, "%s", "");
}

extern "C" size_t mxfp4_attention_grad_workspace_bytes(int64_t q_tokens, int64_t q_heads) {
    if (q_tokens <= 0 || q_heads <= 0 || q_tokens >= (1 << 30) || q_heads > 65535) return 0;
    return (size_t)q_tokens * (size_t)q_heads * sizeof(float2);
}

extern "C" mxfp4_status mxfp4_attention_grad(const mxfp4_heads* q, const mxfp4_heads* k, const mxfp4_heads* v,
                                             const mxfp4_heads* out, const mxfp4_heads* rest, const float* lse,
                                             const mxfp4_heads* dout, int64_t q_tokens, int64_t k_tokens, int64_t head_dim, const int32_t* cu_q,
                                             const int32_t* cu_k, int64_t seqs, int causal, float scale,
                                             int zero_outside, const mxfp4_heads* dq, const mxfp4_heads* dk, const mxfp4_heads* dv,
                                             void* ws, size_t ws_bytes, mxfp4_stream_t stream) {
    const char* what = "attention_grad";
    Call c{};
    mxfp4_status st = check_call(what, q, k, v, q_tokens, k_tokens, head_dim, cu_q, cu_k, seqs, causal, scale, zero_outside, &c);
    if (st) return st;
    Heads d{}, gq{}, gk{}, gv{};
    if ((st = check_output(what, out, rest, false, &c))) return st;
    if ((st = check_operand(what, "dout", dout, q_tokens, head_dim, false, &d))) return st;
    if ((st = check_operand(what, "dq", dq, q_tokens, head_dim, true, &gq))) return st;
    if ((st = check_operand(what, "dk", dk, k_tokens, head_dim, true, &gk))) return st;
    if ((st = check_operand(what, "dv", dv, k_tokens, head_dim, true, &gv))) return st;
    if (d.heads != c.q.heads || gq.heads != c.q.heads || gk.heads != c.k.heads ||
        gv.heads != c.k.heads)
        return record_error(MXFP4_ERR_INVALID_ARG, "%s: dout or a gradient has other heads than its input", what);
    const Named q_{"q", &c.q, q_tokens}, k_{"k", &c.k, k_tokens}, v_{"v", &c.v, k_tokens}, d_{"dout", &d, q_tokens};
    const Named dq_{"dq", &gq, q_tokens}, dk_{"dk", &gk, k_tokens}, dv_{"dv", &gv, k_tokens};
    if ((st = check_apart(what, dk_, {q_, k_, v_, d_, dq_, dv_}, {}, head_dim))) return st;
    if ((st = check_apart(what, dv_, {q_, k_, v_, d_, dq_}, {}, head_dim))) return st;
    if ((st = check_apart(what, dq_, {k_, v_}, {q_, d_}, head_dim))) return st;
    if (q_tokens > 0) {
        if (!lse) return record_error(MXFP4_ERR_INVALID_ARG, "%s: lse is NULL", what);
        if (reinterpret_cast<uintptr_t>(lse) % 4) return record_error(MXFP4_ERR_MISALIGNED, "%s: lse misaligned", what);
        const size_t need = mxfp4_attention_grad_workspace_bytes(q_tokens, c.q.heads);
        if (!ws || ws_bytes < need)
            return record_error(MXFP4_ERR_WORKSPACE, "%s: workspace of %zu bytes needed", what, need);
        if (reinterpret_cast<uintptr_t>(ws) % 256)
            return record_error(MXFP4_ERR_MISALIGNED, "%s: workspace not 256-byte aligned", what);
    }
    if (q_tokens * c.q.heads > (int64_t)INT32_MAX * (kDeltaThreads / 16))
        return record_error(MXFP4_ERR_UNSUPPORTED_SHAPE, "%s: too many queries", what);
    const bool clear = zero_outside && cu_q;
    if ((q_tokens == 0 && k_tokens == 0) || (seqs == 0 && !clear)) return record_error(MXFP4_OK, "%s", "");
    if ((st = ensure_device())) return st;
    BackwardParams p{};
    if (!map_of(&p.q, c.q, q_tokens, c.k, k_tokens, head_dim, c.packing) ||
        !map_of(&p.k, c.k, k_tokens, c.q, q_tokens, head_dim) || !map_of(&p.v, c.v, k_tokens, c.q, q_tokens, head_dim) ||
        !map_of(&p.dout, d, q_tokens, c.k, k_tokens, head_dim, c.packing))
        return record_error(MXFP4_ERR_CUDA, "%s: tensor map encoding failed", what);
    p.dq = rows_of(gq);
    p.dk = rows_of(gk);
    p.dv = rows_of(gv);
    p.stats = static_cast<const float2*>(ws);
    p.seq = c.seq;
    p.packing = c.packing;
    p.group = c.group;
    p.dim = c.dim;
    p.causal = causal;
    p.clear = clear;
    p.scale = scale;
    p.scale_log2 = scale * kLog2e;
    p.status = device_status_ptr();
    p.wait_ns = wait_limit_ns();
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (q_tokens > 0) {
        DeltaParams t{static_cast<const bf16*>(c.out.data), static_cast<const bf16*>(c.rest.data),
                      static_cast<const bf16*>(d.data), c.out.token_stride, c.out.head_stride, c.rest.token_stride,
                      c.rest.head_stride, d.token_stride, d.head_stride, lse, static_cast<float2*>(ws), (int32_t)q_tokens,
                      c.q.heads, c.dim};
        const int64_t rows = q_tokens * c.q.heads, per = kDeltaThreads / 16;
        e = launch_overlapped(delta_kernel, dim3((unsigned)((rows + per - 1) / per)), dim3(kDeltaThreads), 0, s, 1, true, t);
        if (e != cudaSuccess) return record_error(MXFP4_ERR_CUDA, "%s delta launch: %s", what, cudaGetErrorString(e));
    }
    static DeviceSlots slots[4];
    const int smem = c.dim > 64 ? BackwardShape<128>::kSmem : BackwardShape<64>::kSmem;
    p.heads = c.k.heads;
    int64_t ctas = places(c, k_tokens, c.seq.len_k, kRows) * c.k.heads;
    if (clear && k_tokens > 0) ctas = std::max<int64_t>(ctas, 1);
    e = c.dim > 64 ? launch_tiles(attention_dkv_kernel<128>, slots[0], p, ctas, kDkvThreads, smem, s)
                   : launch_tiles(attention_dkv_kernel<64>, slots[1], p, ctas, kDkvThreads, smem, s);
    if (e != cudaSuccess) return record_error(MXFP4_ERR_CUDA, "%s dkv launch: %s", what, cudaGetErrorString(e));
    p.heads = c.q.heads / c.packing.pack;
    ctas = places(c, q_tokens, c.seq.len_q, c.packing.tokens) * p.heads;
    if (clear && q_tokens > 0) ctas = std::max<int64_t>(ctas, 1);
    e = c.dim > 64 ? launch_tiles(attention_dq_kernel<128>, slots[2], p, ctas, kDqThreads, smem, s)
                   : launch_tiles(attention_dq_kernel<64>, slots[3], p, ctas, kDqThreads, smem, s);
    if (e != cudaSuccess) return record_error(MXFP4_ERR_CUDA, "%s dq launch: %s", what, cudaGetErrorString(e));
    return record_error(MXFP4_OK, "%s", "");
}
