// Attention of a round's rows (drafted chains and trees) over a paged
// key-value cache, on the tensor cores.
//
//   S = Q K^T,  P = e^(scale S - m) under the row's mask,  O = P V / sum P
//
// The (row, head) pairs of one KV head are the 128 rows of a product, so the
// cache is read once for up to 256 pairs (a 60-node tree with four heads a
// group).  Reading the cache and the products take about the same time on a
// full batch: both have to run without a pause.
//
// The work is the flat sequence of 128-position tiles of every (sequence, up to
// 256 pairs, KV head), in stretches of equal weight for one CTA an SM.  The
// weights are fitted to the CTAs' cycles on a full batch: a tile 3 with two
// products of rows and 2 with one (3,400 and 2,300 cycles), an item's beginning
// and end 12 (about 13,000); with equal tiles the slowest CTA took a quarter
// longer than the mean.  The pieces of an item that several CTAs share go to the
// workspace and a second, small kernel joins them in order.
//
// Inside a CTA two streams of softmax warps work in turn, so that the tensor
// cores compute one stream's products while the other takes its exponentials:
//   two products of rows   each stream has one, both see every tile
//   one                    both have it, stream w every second tile; their
//                          results meet in shared memory
// A product holds whole query rows: 128 / (heads a group) of them.
// A stream's loop is scores -> exponentials -> both products, one after the
// other, so its latency is what two products of rows are bound by: over a bf16
// cache two threads share a row of scores (1,370 cycles a tile, one thread
// 1,750; 120 -> 102 us for a batch of 32 rounds over 1,600 to 5,200 positions).
// S and O live in tensor memory; P overwrites its S as the left operand of the
// second product.  Keys and values have a copying warp each (tensor copies into
// the 128-byte swizzle, which one warp issues at 100 cycles a page: pages of 8
// positions took 153 us with one warp, 115 with two), each stream a warp of its
// own that issues its products (one for both spent most of its time on
// barriers).
//
// What it reaches on that batch: 97 us, 4.3 TB/s, 64% of the copy rate.  A
// product takes 91 cycles a 16-wide step instead of 64, since both operands of
// the first and the tiles' arrival share the shared memory's bandwidth; an
// item's end, the pieces' joining and the first tile's latency take the rest.
//
// An 8-bit cache goes through fp16 operands (the products take no mixed types):
// its rows are copied raw and five more warps widen them into the ring, exactly.
// The widening bounds it (one warp 268 us for the batch of 32, five 153); the
// queries are brought to fp16 in place, each row scaled by a power of two that
// puts its largest element in [1, 2) (below 2^-14 of it they round to 2^-25).
//
// The weights P are rounded to one number of the operands' type, their sum is
// not: over bf16 each is off by up to 2^-8 and the outputs' error against 64 bits
// is 0.0021 to 0.0023, their own rounding alone 0.0017 (fp16, 2^-11: 0.0017).
// The single tokens' second number would be eight more tensor steps on the
// sixteen of a tile, on the path that bounds it, and twice the registers of P,
// which 608 threads do not have.
//
// Tiles that reach the round's own rows take a mask of 128 bits per row.  There
// a stored value that is not finite is set to zero before the product (0 * inf
// would reach rows that do not see it) and added at the end to the rows that
// do; rows past the sequence are zeroed as well.
#include <cudaTypedefs.h>

#include "wf_paged.cuh"

#define PR_TRY(x)                      \
    do {                               \
        const wf_status _st = (x);     \
        if (_st != WF_OK) return _st;  \
    } while (0)

namespace wf {

constexpr int PR_KT = 128;         // positions of a tile
constexpr int PR_ROWS = 128;       // pairs of a product

struct RoundsParams {
    const int32_t* pos_off;
    const int32_t* cache_len;
    const int32_t* node_off;
    const int32_t* kind;
    const int32_t* parent;
    const int32_t* table;
    const uint8_t* V;        // this layer's rows
    const float* k_scale;    // this layer's [G] scales, or null
    const float* v_scale;
    uint16_t* out;
    float* lse;
    float4* part;            // [CTA][2][D / 4][256] unnormalised outputs, four dims of a row together
    float2* stat;            // [CTA][2][256] (maximum, sum)
    int4* join;              // [CTA] the shared item that begins in it: pieces, first row, pairs, KV head
    float qk;                // scale * log2(e)
    int P, H, G, D, hq, B, page_shift, num_pages, max_pages, max_rows;
    int rpt;                 // query rows of a product: 128 / hq
    int box_rows;            // rows of a copy: min(page_size, 128)
    int per_tile;            // copies of a tile: 128 / box_rows, at most 16
    uint32_t idesc_s, idesc_o;
    Control* ctrl;
    uint64_t timeout_ns;
};

struct RoundSeq {
    int r0, rows, len, T, mp, nt;   // first row, rows, cached positions, all positions, pairs of products, tiles
    bool bad;
};

__device__ __forceinline__ RoundSeq round_seq(const RoundsParams& p, int b) {
    RoundSeq w;
    w.r0 = p.pos_off[b];
    const int r1 = p.pos_off[b + 1];
    w.len = p.cache_len[b];
    w.rows = r1 - w.r0;
    w.T = w.mp = w.nt = 0;
    w.bad = false;
    if (w.r0 < 0 || r1 > p.P || r1 <= w.r0) {   // no row (or offsets that name no rows)
        w.bad = w.r0 < 0 || r1 > p.P || r1 < w.r0;
        w.rows = 0;
        return w;
    }
    const int64_t T = (int64_t)w.len + w.rows;
    w.bad = w.len < 0 || w.rows > p.max_rows || T > ((int64_t)p.max_pages << p.page_shift);
    w.mp = (w.rows + 2 * p.rpt - 1) / (2 * p.rpt);
    w.T = w.bad ? 0 : (int)T;
    w.nt = w.bad ? 1 : (w.T + PR_KT - 1) / PR_KT;   // a bad sequence: one tile that writes NaN
    return w;
}

// Weight of a tile of the query rows 2 rpt mp ..
constexpr int PR_TWO = 3, PR_ONE = 2;
// and of an item's beginning and end, where a CTA has four tiles of weight 3 or
// more on average (fewer: pieces of one item, whose ends cost every CTA alike).
// Mixed batch of 32 with ends of 8: 99.3 us, 10: 97.8, 12: 97.5, 14: 96.8, 17: 98.5;
// chains alone 83.9, 83.3, 83.5, 84.1, 83.1.
constexpr int PR_ITEM = 12;
__device__ __forceinline__ int tile_weight(const RoundsParams& p, const RoundSeq& w, int mp) {
    return w.rows - mp * 2 * p.rpt > p.rpt ? PR_TWO : PR_ONE;
}
// Weight of a whole sequence's tiles: those of its products are weighed alike but the last rows'.
__device__ __forceinline__ int64_t seq_weight(const RoundsParams& p, const RoundSeq& w) {
    return w.mp == 0 ? 0 : (int64_t)p.G * w.nt * (PR_TWO * (w.mp - 1) + tile_weight(p, w, w.mp - 1));
}

// One piece of the CTA's stretch: tiles [kt, kt + tiles) of (sequence b, query rows 2 rpt mp .., KV head g).
struct Piece {
    RoundSeq w;
    int b, mp, g, kt, tiles, rows;   // rows: query rows of the item; tiles: 0 ends the stretch
    int pieces;                      // of the item, if it begins here and ends elsewhere; else 0
    bool solo;                       // one product: the streams share it and take every second tile
};

// ----------------------------------------------------------------- tensor memory and barriers
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// D (+)= A[tensor memory] B[shared memory]
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(acc)
        : "memory");
}
// Matrix descriptors (128-byte swizzle): the low word, which holds the address
// in 16-byte units, and the high word, the same for every operand.  The issuing
// thread advances an operand by adding to the low word.
// Queries, keys: rows of 64 dims (128 bytes), groups of 8 rows 1,024 bytes apart.
__device__ __forceinline__ uint32_t desc_lo_rows(uint32_t smem_addr) { return (smem_addr >> 4) | (1u << 16); }
// Values, whose contiguous dimension is the product's N: 64-dim blocks 16 KB
// apart, groups of 8 positions 1,024 bytes.
__device__ __forceinline__ uint32_t desc_lo_values(uint32_t smem_addr) {
    return (smem_addr >> 4) | ((uint32_t)((PR_KT * 128) >> 4) << 16);
}
__device__ __forceinline__ uint64_t desc_of(uint32_t lo) {
    constexpr uint32_t HI = (1024u >> 4) | (1u << 14) | (2u << 29);
    return ((uint64_t)HI << 32) | lo;
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// acc stays 0 while no bf16 of w is infinite or NaN, and is NaN from then on
__device__ __forceinline__ uint32_t bf16x2_probe(uint32_t w, uint32_t acc) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(w), "r"(0u), "r"(acc));
    return r;
}
// whether `pred` holds in all of the named barrier's threads
__device__ __forceinline__ bool named_all(int id, int threads, bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbar.red.and.pred q, %1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(threads), "r"((uint32_t)pred)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// two fp32 operations in one instruction
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// one lane of a converged warp
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}
__device__ __forceinline__ void named_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void tma_load_3d(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(smem_u32(smem_dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// Shared memory: queries [2][blocks][128 rows][128 B], a ring of tiles of keys or
// values [blocks][128 positions][128 B], rows [128][32] fp32 that pass from one
// stream to the other, two numbers of each thread, and for an 8-bit cache raw
// tiles [128][D <= 64 blocks]; blocks = 64-dim blocks of a head.
template <int BLK, bool E4M3>
struct RoundsShape {
    // tiles of keys or values ready or in flight
    static constexpr int RING = E4M3 ? (BLK == 2 ? 3 : 6) : (BLK == 2 ? 4 : 10);
    static constexpr int RAW = E4M3 ? (BLK == 2 ? 2 : 4) : 0;
    static constexpr int PLACES = E4M3 ? RAW : RING;   // that the copying warps fill
    // a place belongs to the keys or to the values: else one copying warp, ahead of
    // the other by a turn of the ring, would take an older release for its own
    static_assert(E4M3 || RING % 2 == 0, "an even ring");
    // two streams of four softmax warps, a copying warp, an issuing warp a stream, and
    // a second copying warp for the values or for an 8-bit cache the widening warps
    static constexpr int WIDEN = E4M3 ? 5 : 0;
    static constexpr int COPIES = E4M3 ? 1 : 2;
    // threads that share a row's scores of a tile
    static constexpr int HALVES = E4M3 ? 1 : 2;
    static constexpr int SOFT = 8 * HALVES;          // softmax warps
    static constexpr int STREAM = 128 * HALVES;      // threads of a stream
    static constexpr int THREADS = (SOFT + 2 + COPIES + WIDEN) * 32;
    // 8-bit caches: 512 threads start with 128 registers each (65,536); the softmax
    // warps take 176, the other eight give down to 80 (the same 65,536)
    static constexpr bool SPLIT_REGISTERS = E4M3;
    static constexpr int QTILE = BLK * PR_ROWS * 128;
    static constexpr int TILE = BLK * PR_KT * 128;
    static constexpr int RAW_TILE = BLK * PR_KT * 64;
    static constexpr int XBYTES = PR_ROWS * 32 * 4;
    static constexpr int XC = 32 / HALVES;           // dims that a thread takes from or to shared memory together
    static constexpr int SMEM = 1024 + 2 * QTILE + RING * TILE + RAW * RAW_TILE + XBYTES + PR_ROWS * 8 + 2 * STREAM * 4;
    // the running maximum may lag by 2^LAG; fp16 probabilities use the range from 2^-24 up to 2^(BIAS + LAG)
    static constexpr float LAG = E4M3 ? 4.f : 8.f;
    static constexpr float BIAS = E4M3 ? 8.f : 0.f;
};

// acc stays 0 while no fp16 of w is infinite or NaN, and is NaN from then on
__device__ __forceinline__ uint32_t f16x2_probe(uint32_t w, uint32_t acc) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(w), "r"(0u), "r"(acc));
    return r;
}

// BLK: 64-dim blocks of a head (1 or 2); E4M3: the cache's type
template <int BLK, bool E4M3>
__global__ void __launch_bounds__(RoundsShape<BLK, E4M3>::THREADS, 1)
    paged_rounds_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const RoundsParams p) {
    using S = RoundsShape<BLK, E4M3>;
    constexpr int RING = S::RING, QTILE = S::QTILE, TILE = S::TILE, THREADS = S::THREADS, WIDEN = S::WIDEN, COPIES = S::COPIES;
    constexpr int HALVES = S::HALVES, SOFT = S::SOFT, STREAM = S::STREAM, XC = S::XC;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sQ = smem;
    uint8_t* sR = smem + 2 * QTILE;
    uint8_t* sW = sR + RING * TILE;            // raw tiles
    uint8_t* sX = sW + S::RAW * S::RAW_TILE;
    float2* s_xst = reinterpret_cast<float2*>(sX + S::XBYTES);                    // the second stream's rows'
    float* s_own = reinterpret_cast<float*>(sX + S::XBYTES + PR_ROWS * 8);        // a number of each softmax thread
    constexpr int PLACES = S::PLACES, RAW = E4M3 ? S::RAW : 1;
    __shared__ uint64_t kv_full[RING], kv_empty[RING], raw_full[RAW], raw_empty[RAW], q_full, q_empty, told[8];
    __shared__ uint64_t piece_ready[8], piece_free[8];
    __shared__ Piece s_piece[8];   // the copying warp's next pieces, for the others
    __shared__ uint64_t s_full[2], p_full[2], o_full[2], drained[2];   // by stream
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_word, s_bad[8], s_odd[2][2], s_turn;
    __shared__ uint8_t s_par[2][WF_MAX_SEQ_NODES + 1];   // row of each row's parent, by stream (a row's own copy)
    __shared__ uint64_t q_ready[2];                        // queries brought to fp16, by stream
    __shared__ float s_factor[PR_ROWS];                    // and their scores' factors, for the other stream
    __shared__ int64_t s_scan[2][THREADS / 32];   // weights and items of the sequences of each warp
    volatile int* abort_flag = &abort_word;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < RING; ++i) {
            mbar_init(&kv_full[i], E4M3 ? WIDEN : 1);
            mbar_init(&kv_empty[i], 2);   // both streams, or one twice
        }
        for (int i = 0; i < RAW; ++i) {
            mbar_init(&raw_full[i], 1);
            mbar_init(&raw_empty[i], E4M3 ? WIDEN : 1);
        }
        mbar_init(&q_ready[0], PR_ROWS);
        mbar_init(&q_ready[1], PR_ROWS);
        mbar_init(&q_full, 1);
        mbar_init(&q_empty, 2);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], STREAM);
            mbar_init(&o_full[i], 1);
            mbar_init(&drained[i], 1);
        }
        for (int i = 0; i < 8; ++i) {
            mbar_init(&told[i], 1);
            mbar_init(&piece_ready[i], 1);
            mbar_init(&piece_free[i], 3 + COPIES + WIDEN);   // two streams, two issuing warps, the second copying, the widening ones
        }
        abort_word = s_turn = 0;
        s_odd[0][0] = s_odd[0][1] = s_odd[1][0] = s_odd[1][1] = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    if (warp == SOFT) {
        tmem_alloc(&tmem_slot, 512);
        tmem_relinquish();
    }
    pdl_wait();
    pdl_trigger();

    // ------------------------------------------------ this CTA's stretch
    // The copying warp finds it.  Up to 32 sequences it weighs by itself, a lane each,
    // before the others are there; more are weighed by all threads.  (Code that is
    // run once waits for its instructions: half a microsecond less than with the
    // general way for all.)
    const bool few = p.B <= 32;
    const int run = (p.B + THREADS - 1) / THREADS;
    bool heavy = false;   // a tile of weight PR_TWO
    int64_t mine = 0, mine_items = 0;   // weight and items of what this thread weighed
    for (int i = 0; i < (few ? 1 : run); ++i) {
        const int b = few ? (warp == SOFT ? lane : p.B) : tid * run + i;
        if (b >= p.B) continue;
        const RoundSeq w = round_seq(p, b);
        mine += seq_weight(p, w);
        mine_items += (int64_t)p.G * w.mp;
        heavy |= w.mp > 0 && tile_weight(p, w, 0) == PR_TWO;
        if (w.bad && blockIdx.x == 0) record_error(p.ctrl, WF_ERR_BAD_DATA, (uint32_t)b);
    }
    if (!few) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            mine += __shfl_xor_sync(0xffffffffu, mine, o);
            mine_items += __shfl_xor_sync(0xffffffffu, mine_items, o);
        }
        if (lane == 0) s_scan[0][warp] = mine, s_scan[1][warp] = mine_items;
    }
    tc_fence_before();
    heavy = __syncthreads_or(heavy);
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    if (warp >= SOFT) {
        if (S::SPLIT_REGISTERS) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        const uint64_t pol = policy_evict_first();
        const int per_tile = p.per_tile;
        // lane i of a copying warp: the page of positions i box_rows .. of a tile; -2: the
        // tile has no such positions, -1: they have no page, whatever negative entry says so
        auto page_of = [&](const Piece& x, int kt) {
            const int t = kt * PR_KT + lane * p.box_rows;
            return lane < per_tile && t < x.w.T ? max(p.table[(int64_t)x.b * p.max_pages + (t >> p.page_shift)], -1) : -2;
        };
        auto pool_row = [&](int kt, int page) {
            return (page << p.page_shift) + ((kt * PR_KT + lane * p.box_rows) & ((1 << p.page_shift) - 1));
        };
        // a tile's keys or values to place `at`
        auto load = [&](int kv, int at, const Piece& x, bool ok, int y, uint32_t boxes) {
            const int place = at % PLACES;
            uint64_t* full = E4M3 ? &raw_full[place] : &kv_full[place];
            const int row_bytes = E4M3 ? p.D : BLK * 128;
            // a lane's copies may count before these bytes are expected: the phase waits for
            // this arrival
            if (lane == 0) mbar_arrive_expect_tx(full, boxes * p.box_rows * row_bytes);
            if (ok && E4M3) {
                tma_load_2d(sW + place * S::RAW_TILE + lane * p.box_rows * p.D, kv ? &tmV : &tmK, full, x.g * p.D, y,
                            pol);
            } else if (ok) {
                uint8_t* dst = sR + place * TILE + lane * p.box_rows * 128;
#pragma unroll
                for (int blk = 0; blk < BLK; ++blk)
                    tma_load_2d(dst + blk * PR_KT * 128, kv ? &tmV : &tmK, full, x.g * p.D + blk * 64, y, pol);
            }
        };
        auto place_free = [&](int at) {
            return at < PLACES || mbar_wait(E4M3 ? &raw_empty[at % PLACES] : &kv_empty[at % PLACES],
                                            ((at / PLACES) & 1) ^ 1, p.timeout_ns, abort_flag);
        };
        auto landed = [&](int at) {
            mbar_wait(E4M3 ? &raw_full[at % PLACES] : &kv_full[at % PLACES], (at / PLACES) & 1, p.timeout_ns, nullptr);
        };
        // A warp that goes on together gives up together, whatever each lane's last look
        // at the barrier, the abort flag and the clock was: left to the lanes, some could
        // leave while the others wait for them in the next shuffle.
        auto whole_warp = [](bool got) { return __all_sync(0xffffffffu, got) != 0; };
        if (warp == SOFT) {
            // ---------------------------------------- copies: a tile's keys, then its values, to the ring's next places
            auto inclusive = [&](int64_t v) {
#pragma unroll 1
                for (int o = 1; o < 32; o <<= 1) {
                    const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
                    if (lane >= o) v += y;
                }
                return v;
            };
            // a lane's share: its sequence, or what a warp has weighed
            int64_t n = mine, items = mine_items;
            if (!few) {
                n = lane < THREADS / 32 ? s_scan[0][lane] : 0;
                items = lane < THREADS / 32 ? s_scan[1][lane] : 0;
            }
            int64_t total = n, all_items = items;
#pragma unroll 1
            for (int o = 16; o > 0; o >>= 1) {
                total += __shfl_xor_sync(0xffffffffu, total, o);
                all_items += __shfl_xor_sync(0xffffffffu, all_items, o);
            }
            const int ends = total >= (int64_t)PR_ITEM * gridDim.x ? PR_ITEM : 0;
            total += ends * all_items;
            n += ends * items;
            int64_t per = pg_quotient(total + gridDim.x - 1, gridDim.x);
            // every stretch between an item's first and its last holds one of its tiles
            if (per < (heavy ? PR_TWO : PR_ONE)) per = heavy ? PR_TWO : PR_ONE;
            const int64_t begin = (int64_t)blockIdx.x * per;
            const int64_t end = begin + per < total ? begin + per : total;
            int64_t plan = 0;   // of the stretch's beginning, in its sequence
            int pb = 0;         // which one
            if (begin < end) {
                // the lane whose share holds the beginning; its place there
                auto find = [&](int64_t from, int64_t share) {
                    const int64_t upto = from + inclusive(share);
                    const int l = __ffs(__ballot_sync(0xffffffffu, share > 0 && upto - share <= begin && begin < upto)) - 1;
                    plan = begin - __shfl_sync(0xffffffffu, upto - share, l);
                    return l;
                };
                pb = find(0, n);
                if (!few) {   // that was the warp: now the lane, then its sequence
                    const int b0 = (pb * 32 + lane) * run;
                    auto weight_of = [&](int b) {
                        const RoundSeq w = round_seq(p, b);
                        return seq_weight(p, w) + (int64_t)ends * p.G * w.mp;
                    };
                    int64_t share = 0;
                    for (int i = 0; i < run; ++i)
                        if (b0 + i < p.B) share += weight_of(b0 + i);
                    const int l = find(begin - plan, share);
                    pb = __shfl_sync(0xffffffffu, b0, l);
                    for (;; ++pb) {
                        const int64_t one = weight_of(pb);
                        if (plan < one) break;
                        plan -= one;
                    }
                }
            }
            // the stretch's first item: `start`, the weight before it; its tile kt is
            // the first that starts in the stretch
            Piece x = {};
            int64_t start = begin;
            int weight = PR_ONE;
            auto next_item = [&]() {
                start += (int64_t)x.w.nt * weight + ends;
                x.kt = 0;
                if (++x.g == p.G) {
                    x.g = 0;
                    if (++x.mp == x.w.mp) {
                        x.mp = 0;
                        do {
                            if (++x.b >= p.B) {
                                start = end;   // nothing is left
                                return;
                            }
                            x.w = round_seq(p, x.b);
                        } while (x.w.mp == 0);
                    }
                }
                weight = tile_weight(p, x.w, x.mp);
            };
            if (begin < end) {
                x.b = pb;
                x.w = round_seq(p, x.b);
                int64_t in_rows = plan;
                if (x.w.mp > 1) {
                    const int64_t full = (int64_t)p.G * (x.w.nt * PR_TWO + ends);
                    x.mp = (int)pg_quotient(plan, full);
                    if (x.mp > x.w.mp - 1) x.mp = x.w.mp - 1;
                    in_rows -= x.mp * full;
                }
                weight = tile_weight(p, x.w, x.mp);
                const int item = x.w.nt * weight + ends;
                x.g = (int)pg_quotient(in_rows, item);
                const int64_t in_item = in_rows - (int64_t)x.g * item;
                start = begin - in_item;
                x.kt = ((int)in_item + weight - 1) / weight;
                if (x.kt >= x.w.nt) next_item();
            }
            int sent = 0, last = -1, k = 0;   // places of the tiles before, the last place filled; pieces' queries
            for (int turn = 0;; ++turn) {
                if (!whole_warp(turn < 8 || mbar_wait(&piece_free[turn & 7], ((turn >> 3) & 1) ^ 1, p.timeout_ns, abort_flag))) {
                    *abort_flag = 1;
                    if (lane == 0) record_error(p.ctrl, WF_ERR_TIMEOUT, 0x801u);
                    break;
                }
                x.tiles = 0;
                if (begin < end && start + (int64_t)x.kt * weight < end) {
                    const int64_t upto = pg_quotient(end - start + weight - 1, weight);
                    x.tiles = (int)(upto < x.w.nt ? upto : x.w.nt) - x.kt;
                    x.rows = min(2 * p.rpt, x.w.rows - x.mp * 2 * p.rpt);
                    x.solo = x.rows <= p.rpt;
                    x.pieces = 0;
                    if (x.kt == 0 && x.tiles < x.w.nt)
                        x.pieces = (int)pg_quotient(start + (int64_t)(x.w.nt - 1) * weight, per) - (int)blockIdx.x + 1;
                }
                if (lane == 0) {
                    s_piece[turn & 7] = x;
                    mbar_arrive(&piece_ready[turn & 7]);
                }
                if (x.tiles == 0) break;
                bool bad = false;
                if (!x.w.bad) {
                    int page = page_of(x, x.kt);
                    for (int i = 0; i < x.tiles; ++i) {
                        const bool ok = page >= 0 && page < p.num_pages;
                        bad |= page != -2 && !ok;
                        const int y = ok ? pool_row(x.kt + i, page) : 0;
                        const uint32_t boxes = (uint32_t)__popc(__ballot_sync(0xffffffffu, ok));
                        if (i + 1 < x.tiles) page = page_of(x, x.kt + i + 1);
                        bool alive = true;
#pragma unroll
                        for (int kv = 0; kv < 2; ++kv) {
                            if (kv == 1 && i == 0) {   // the piece's queries, behind its first keys
                                alive = alive && whole_warp(k == 0 || mbar_wait(&q_empty, (k & 1) ^ 1, p.timeout_ns, abort_flag));
                                if (!alive) break;
                                const int nq = x.solo ? 1 : 2;
                                if (lane == 0) {
                                    mbar_arrive_expect_tx(&q_full, (uint32_t)(nq * BLK * p.rpt * p.hq * 128));
                                    for (int w = 0; w < nq; ++w)
                                        for (int blk = 0; blk < BLK; ++blk)
                                            tma_load_3d(sQ + w * QTILE + blk * PR_ROWS * 128, &tmQ, &q_full, blk * 64,
                                                        x.g * p.hq, x.w.r0 + (2 * x.mp + w) * p.rpt);
                                }
                                ++k;
                                __syncwarp();
                            }
                            // the raw tiles' turn for an 8-bit cache, else the ring's
                            const int at = sent + kv;
                            if (kv == 1 && COPIES == 2) break;   // the other copying warp's
                            alive = alive && whole_warp(place_free(at));
                            if (!alive) break;
                            load(kv, at, x, ok, y, boxes);
                            last = at;
                        }
                        sent += 2;
                        if (!alive) {
                            *abort_flag = 1;
                            if (lane == 0) record_error(p.ctrl, WF_ERR_TIMEOUT, 0x800u);
                            break;
                        }
                    }
                }
                if (!x.w.bad) {   // whether the piece had a position without a page
                    bad = __any_sync(0xffffffffu, bad);
                    if (lane == 0) {
                        s_bad[(k - 1) & 7] = bad;
                        mbar_arrive(&told[(k - 1) & 7]);
                    }
                }
                if (!whole_warp(!*abort_flag)) break;
                next_item();
            }
            // let every copy issued land before the shared memory goes
            for (int at = max(0, last - PLACES + 1); at <= last; ++at)
                if (COPIES == 1 || at % 2 == 0) landed(at);
            if (k > 0) mbar_wait(&q_full, (k & 1) ^ 1, p.timeout_ns, nullptr);
        } else if (COPIES == 2 && warp == SOFT + 3) {
            // ---------------------------------------- copies of the values
            int n = 0, last = -1;   // tiles before this piece, the last place filled
            bool ok = true;
            for (int turn = 0; ok; ++turn) {
                ok = whole_warp(mbar_wait(&piece_ready[turn & 7], (turn >> 3) & 1, p.timeout_ns, abort_flag));
                if (!ok) break;
                const Piece& x = s_piece[turn & 7];
                if (x.tiles == 0) break;
                const int tiles = x.w.bad ? 0 : x.tiles;
                int page = tiles > 0 ? page_of(x, x.kt) : -2;
                for (int i = 0; i < tiles && ok; ++i) {
                    const bool in = page >= 0 && page < p.num_pages;
                    const int y = in ? pool_row(x.kt + i, page) : 0;
                    const uint32_t boxes = (uint32_t)__popc(__ballot_sync(0xffffffffu, in));
                    if (i + 1 < tiles) page = page_of(x, x.kt + i + 1);
                    const int at = 2 * (n + i) + 1;
                    ok = whole_warp(place_free(at));
                    if (!ok) break;
                    load(1, at, x, in, y, boxes);
                    last = at;
                }
                n += tiles;
                __syncwarp();
                if (ok && lane == 0) mbar_arrive(&piece_free[turn & 7]);
            }
            if (!ok) {
                *abort_flag = 1;
                if (lane == 0) record_error(p.ctrl, WF_ERR_TIMEOUT, 0x802u);
            }
            for (int at = max(1, last - PLACES + 1) | 1; at <= last; at += 2) landed(at);
        } else if (warp >= SOFT + 3) {
            // ---------------------------------------- 8-bit rows widened to fp16 in the ring
            if (E4M3) {
                int n = 0;
                bool ok = true;
                auto wait = [&](uint64_t* bar, uint32_t parity) {
                    ok = ok && mbar_wait(bar, parity, p.timeout_ns, abort_flag);
                };
                // a lane keeps its 16-byte piece c of the rows r0, r0 + step ..
                const int per_row = p.D / 16, rows = 32 / per_row, step = WIDEN * rows;
                const int c = lane % per_row, r0 = lane < rows * per_row ? (warp - SOFT - 3) * rows + lane / per_row : PR_KT;
                const bool swap = c & 4;
                for (int turn = 0; ok; ++turn) {
                    wait(&piece_ready[turn & 7], (turn >> 3) & 1);
                    ok = whole_warp(ok);
                    if (!ok) break;
                    const int tiles = s_piece[turn & 7].tiles;
                    if (tiles == 0) break;
                    const int loads = s_piece[turn & 7].w.bad ? 0 : 2 * tiles;
                    for (int i = 0; i < loads && ok; ++i) {
                        const int at = 2 * n + i, raw = at % RAW, slot = at % RING;
                        wait(&raw_full[raw], (at / RAW) & 1);
                        if (at >= RING) wait(&kv_empty[slot], ((at / RING) & 1) ^ 1);
                        ok = whole_warp(ok);
                        if (!ok) break;
                        const uint8_t* src = sW + raw * S::RAW_TILE;
                        uint8_t* dst = sR + slot * TILE;
                        for (int r = r0; r < PR_KT; r += 4 * step) {
                            uint4 v[4];
#pragma unroll
                            for (int u = 0; u < 4; ++u)
                                if (r + u * step < PR_KT)
                                    v[u] = *reinterpret_cast<const uint4*>(src + (r + u * step) * p.D + c * 16);
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                const int ru = r + u * step;
                                if (ru >= PR_KT) break;
                                const uint4 lo = make_uint4(e4m3x2_f16x2(v[u].x), e4m3x2_f16x2(v[u].x >> 16),
                                                            e4m3x2_f16x2(v[u].y), e4m3x2_f16x2(v[u].y >> 16));
                                const uint4 hi = make_uint4(e4m3x2_f16x2(v[u].z), e4m3x2_f16x2(v[u].z >> 16),
                                                            e4m3x2_f16x2(v[u].w), e4m3x2_f16x2(v[u].w >> 16));
                                uint8_t* row = dst + (c >> 2) * PR_KT * 128 + ru * 128;
                                const int at_lo = ((2 * c & 7) ^ (ru & 7)) << 4;   // its neighbour: the other of two
                                // half of a wide row's lanes store their second piece first: eight
                                // lanes then meet eight different banks' groups
                                *reinterpret_cast<uint4*>(row + (at_lo ^ (swap ? 16 : 0))) = swap ? hi : lo;
                                *reinterpret_cast<uint4*>(row + (at_lo ^ (swap ? 0 : 16))) = swap ? lo : hi;
                            }
                        }
                        fence_async_smem();
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(&kv_full[slot]);
                            mbar_arrive(&raw_empty[raw]);
                        }
                    }
                    if (!ok) break;
                    n += loads / 2;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&piece_free[turn & 7]);
                }
                if (!ok) {
                    *abort_flag = 1;
                    if (lane == 0) record_error(p.ctrl, WF_ERR_TIMEOUT, 0x830u);
                }
            }
        } else {
            // ---------------------------------------- products of stream w
            // The whole warp runs this with the same values and one elected lane
            // issues: the operands' descriptors stay in uniform registers (issued
            // from a single thread's own, a product took 107 cycles instead of its 64).
            const int w = __shfl_sync(0xffffffffu, warp - SOFT - 1, 0);
            const uint32_t tS = __shfl_sync(0xffffffffu, tmem, 0) + w * 128, tO = tS + 256;
            const uint32_t qdesc = __shfl_sync(0xffffffffu, desc_lo_rows(smem_u32(sQ)), 0);
            const uint32_t kdesc = __shfl_sync(0xffffffffu, desc_lo_rows(smem_u32(sR)), 0);
            const uint32_t vdesc = __shfl_sync(0xffffffffu, desc_lo_values(smem_u32(sR)), 0);
            int n = 0;                  // tiles before this piece
            uint32_t qn = 0, pn = 0;    // queries, probabilities taken
            bool ok = true;
            const int nks = p.D / 16;
            auto wait = [&](uint64_t* bar, uint32_t parity) {
                ok = ok && mbar_wait(bar, parity, p.timeout_ns, abort_flag);
            };
            // One stream's products are issued without the other's between them: the
            // tensor cores finish one stream early and the streams fall out of step
            // (interleaved, both finish late and then both wait for exponentials).
            auto take_turn = [&]() {
                ok = whole_warp(ok);
                if (ok && lane == 0 && atomicCAS(&s_turn, 0, 1) != 0) {
                    const uint64_t start = globaltimer_ns();
                    while (ok && atomicCAS(&s_turn, 0, 1) != 0)
                        ok = !*abort_flag && globaltimer_ns() - start <= p.timeout_ns;
                }
                ok = whole_warp(ok);
            };
            auto give_turn = [&]() {
                __syncwarp();
                if (lane == 0) atomicExch(&s_turn, 0);
            };
            for (int turn = 0; ok; ++turn) {
                wait(&piece_ready[turn & 7], (turn >> 3) & 1);
                ok = whole_warp(ok);
                if (!ok) break;
                const Piece& x = s_piece[turn & 7];
                const int tiles = x.tiles;
                if (tiles == 0) break;
                if (!x.w.bad) {
                    const int steps = __shfl_sync(0xffffffffu, x.solo ? (x.tiles - w + 1) / 2 : x.tiles, 0);
                    const bool solo = __shfl_sync(0xffffffffu, (int)x.solo, 0) != 0;
                    const int n0 = __shfl_sync(0xffffffffu, n, 0);
                    auto place_of = [&](int i) { return 2 * (n0 + (solo ? 2 * i + w : i)); };   // of step i's keys
                    auto release = [&](int slot) {
                        umma_commit(&kv_empty[slot]);
                        if (solo) umma_commit(&kv_empty[slot]);
                    };
                    auto arrived = [&](int at) { wait(&kv_full[at % RING], (at / RING) & 1); };
                    auto scores = [&](int i) {   // S of step i
                        const int slot = place_of(i) % RING;
                        const uint32_t a = qdesc + (solo ? 0 : w) * (QTILE >> 4), b = kdesc + slot * (TILE >> 4);
#pragma unroll
                        for (int ks = 0; ks < 4 * BLK; ++ks)
                            if (ks < nks) {
                                const uint32_t off = (uint32_t)((ks >> 2) * PR_KT * 8 + (ks & 3) * 2);
                                umma_bf16(tS, desc_of(a + off), desc_of(b + off), p.idesc_s, ks != 0);
                            }
                        umma_commit(&s_full[w]);
                        release(slot);
                        if (i + 1 == steps) umma_commit(&q_empty);   // the stream is done with the queries
                    };
                    wait(E4M3 ? &q_ready[w] : &q_full, qn++ & 1);
                    if (steps == 0) {
                        ok = whole_warp(ok);
                        if (lane == 0) mbar_arrive(&q_empty);
                    } else {
                        arrived(place_of(0));
                        take_turn();
                        if (!ok) break;
                        tc_fence_after();
                        if (elect_one()) scores(0);
                        give_turn();
                    }
                    for (int i = 0; i < steps; ++i) {
                        const int at = place_of(i) + 1, slot = at % RING;
                        arrived(at);
                        // Two products share every tile: the next keys are here by now, and
                        // both products go in one turn.  One product: its next keys are two
                        // tiles ahead and may be waiting for the place of the values that
                        // go now.
                        const int next = place_of(i + 1);
                        const bool both = !solo && i + 1 < steps;
                        if (both) arrived(next);
                        wait(&p_full[w], pn++ & 1);
                        take_turn();
                        if (!ok) break;
                        tc_fence_after();
                        if (elect_one()) {
                            const uint32_t b = vdesc + slot * (TILE >> 4);
#pragma unroll
                            for (int ks = 0; ks < PR_KT / 16; ++ks)
                                umma_ts(tO, tS + ks * 8, desc_of(b + ks * 128), p.idesc_o, (i | ks) != 0);
                            release(slot);
                            if (i + 1 == steps) umma_commit(&o_full[w]);
                            else if (both) scores(i + 1);
                        }
                        give_turn();
                        if (i + 1 < steps && !both) {
                            arrived(next);
                            take_turn();
                            if (!ok) break;
                            tc_fence_after();
                            if (elect_one()) scores(i + 1);
                            give_turn();
                        }
                    }
                    n += tiles;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&piece_free[turn & 7]);
            }
            if (!ok) {
                *abort_flag = 1;
                if (lane == 0) record_error(p.ctrl, WF_ERR_TIMEOUT, 0x810u);
            }
            // The products issued so far are complete before shared and tensor memory
            // go, whichever warp's wait gave up (if none did, they are by now).
            __syncwarp();
            if (elect_one()) umma_commit(&drained[w]);
            mbar_wait(&drained[w], 0, p.timeout_ns, nullptr);
        }
    } else {
        // -------------------------------------------- softmax: stream w, HALVES threads a row of the product
        if (S::SPLIT_REGISTERS) asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
        const int w = warp / (4 * HALVES), half = (warp >> 2) & (HALVES - 1), row = tid & 127;
        const int pair_id = 4 + w * 4 + (warp & 3);   // the named barrier of the warps that share rows
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lanes + w * 128, tO = tmem + lanes + 256 + w * 128;
        uint32_t sn = 0, on = 0;   // scores, outputs taken
        uint32_t qn = 0;           // queries (8-bit caches)
        int n = 0, k = 0;          // tiles before this piece, pieces that have any
        bool shared_item = false;  // an item begins here and ends elsewhere
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            if (ok && !mbar_wait(bar, parity, p.timeout_ns, abort_flag)) {
                ok = false;
                *abort_flag = 1;
                record_error(p.ctrl, WF_ERR_TIMEOUT, 0x820u);
            }
        };
        for (int turn = 0;; ++turn) {
            wait(&piece_ready[turn & 7], (turn >> 3) & 1);
            // all of both streams go on, or none (also: s_odd and the exchanged rows of
            // the piece before are read to their end)
            if (!named_all(3, 2 * STREAM, ok)) break;
            const Piece& x = s_piece[turn & 7];
            if (x.tiles == 0) break;
            const int first = (2 * x.mp + (x.solo ? 0 : w)) * p.rpt;   // first query row of this stream's product
            const int r = first + row / p.hq;
            const bool live = row < p.rpt * p.hq && r < x.w.rows;
            const bool warp_live = (row & ~31) < p.rpt * p.hq && first + (row & ~31) / p.hq < x.w.rows;
            float m = -INFINITY, l = 0.f;   // running maximum of the scores as they are, sum
            int* odd_word = &s_odd[turn & 1][w];
            bool bad = x.w.bad, tree = false;
            const int mine_tiles = x.solo ? (x.tiles - w + 1) / 2 : x.tiles;   // tiles of this stream
            const bool piece_masked = (x.kt + x.tiles) * PR_KT > x.w.len;
            // what the streams learn of the piece: bit 0, a value under a mask is not
            // finite; bit 1, the tree is malformed
            bool learned = false;
            auto learn_tree = [&]() {   // the parents' rows into shared memory, once a piece
                if (learned) return;
                learned = true;
                const int kd = p.kind ? p.kind[x.b] : 1;
                const int n0 = p.parent ? p.node_off[x.b] : 0, n1 = p.parent ? p.node_off[x.b + 1] : 0;
                tree = p.parent != nullptr && kd != 0;
                if (tree) {
                    const int nn = n1 - n0;
                    bool off = n0 < 0 || nn != x.w.rows - 1;
                    if (off) tree = false;
                    else
                        for (int a = half * 128 + row; a < nn; a += STREAM) {
                            const int pi = p.parent[n0 + a];
                            const bool wrong = pi < -1 || pi >= a;
                            s_par[w][1 + a] = (uint8_t)(wrong ? 0 : 1 + pi);
                            off |= wrong;
                        }
                    if (off) atomicOr(odd_word, 2);
                }
                named_sync(1 + w, STREAM);
            };
            float f = p.qk;   // the row's scores times this are base-2 exponents
            if (E4M3 && !x.w.bad) {
                if (w == 0 || !x.solo) {
                    // this row's queries to fp16 in place
                    wait(&q_full, qn & 1);
                    uint8_t* q = sQ + (x.solo ? 0 : w) * QTILE + row * 128;
                    auto piece = [&](int c) {
                        return reinterpret_cast<uint4*>(q + (c >> 3) * PR_ROWS * 128 + (((c & 7) ^ (row & 7)) << 4));
                    };
                    auto lo = [](uint32_t y) { return pg_bf16_to_f32(y & 0xFFFFu); };
                    auto hi = [](uint32_t y) { return pg_bf16_to_f32(y >> 16); };
                    float big = 0.f;
#pragma unroll 4
                    for (int c = 0; c < p.D / 8; ++c) {
                        const uint4 y = *piece(c);
                        big = max3(big, fabsf(lo(y.x)), fabsf(hi(y.x)));
                        big = max3(big, fabsf(lo(y.y)), fabsf(hi(y.y)));
                        big = max3(big, fabsf(lo(y.z)), fabsf(hi(y.z)));
                        big = max3(big, fabsf(lo(y.w)), fabsf(hi(y.w)));
                    }
                    const int e = pg_scale_exponent(big);
                    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll 4
                    for (int c = 0; c < p.D / 8; ++c) {
                        const uint4 y = *piece(c);
                        *piece(c) = make_uint4(cvt_f16x2(lo(y.x) * down, hi(y.x) * down), cvt_f16x2(lo(y.y) * down, hi(y.y) * down),
                                               cvt_f16x2(lo(y.z) * down, hi(y.z) * down), cvt_f16x2(lo(y.w) * down, hi(y.w) * down));
                    }
                    f = pg_factor(p.qk * (p.k_scale ? __ldg(p.k_scale + x.g) : 1.f), e);
                    if (x.solo) s_factor[row] = f;
                    fence_async_smem();
                    mbar_arrive(&q_ready[w]);
                    if (x.solo) mbar_arrive(&q_ready[1]);
                } else {
                    wait(&q_ready[1], qn & 1);
                    f = s_factor[row];
                }
                ++qn;
            }
            if (!x.w.bad) {
                for (int i = 0; i < mine_tiles; ++i) {
                    const int j = x.solo ? 2 * i + w : i;
                    const int t0 = (x.kt + j) * PR_KT;
                    const bool masked = t0 + PR_KT > x.w.len;
                    wait(&s_full[w], sn++ & 1);
                    tc_fence_after();
                    constexpr int WORDS = 4 / HALVES;   // of 32 positions that this thread takes
                    const int u0 = t0 + half * 64;
                    uint32_t see[WORDS];   // those that the row sees
                    if (masked) {
                        learn_tree();
                        // all below `upto`, then the row's ancestors
                        const int upto = (tree ? x.w.len : x.w.len + r + 1) - u0;
#pragma unroll
                        for (int c = 0; c < WORDS; ++c) {
                            const int u = upto - 32 * c;
                            see[c] = u <= 0 ? 0u : (u >= 32 ? 0xFFFFFFFFu : (1u << u) - 1u);
                        }
                        if (tree && live) {
                            int a = r;
                            while (true) {
                                const int t = x.w.len + a - u0;
#pragma unroll
                                for (int c = 0; c < WORDS; ++c)
                                    if (t >= 32 * c && t < 32 * c + 32) see[c] |= 1u << (t & 31);
                                if (a == 0) break;
                                a = s_par[w][a];
                            }
                        }
                        __syncwarp();
                    }
                    if (warp_live) {
                        constexpr int STEP = 2 / HALVES;   // words of scores fetched together
                        uint32_t s[STEP][32];
                        auto fetch = [&](int c0) {
#pragma unroll
                            for (int c = 0; c < STEP; ++c) tmem_ld_32x32b_x32(tS + half * 64 + (c0 + c) * 32, s[c]);
                            tmem_ld_wait();
                            if (masked) {
#pragma unroll
                                for (int c = 0; c < STEP; ++c)
                                    if (!__all_sync(0xffffffffu, see[c0 + c] == 0xFFFFFFFFu))
#pragma unroll
                                        for (int e = 0; e < 32; ++e)
                                            if (!(see[c0 + c] >> e & 1u)) s[c][e] = 0xFF800000u;
                            }
                        };
                        auto at = [&](int c, int e) { return __uint_as_float(s[c][e]); };
                        auto largest = [&](float big) {
                            float top[4] = {big, big, big, big};
#pragma unroll
                            for (int c = 0; c < STEP; ++c)
#pragma unroll
                                for (int e = 0; e < 32; e += 2) top[(e >> 1) & 3] = max3(top[(e >> 1) & 3], at(c, e), at(c, e + 1));
                            return fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                        };
                        // The weights are taken against the running maximum as it is; only
                        // when a score has outgrown it by 2^LAG (or nothing has been seen
                        // yet) is the tile's maximum taken first.  A row's threads hold the
                        // same maximum and decide alike, whatever a wait has come to.  Rows that
                        // are no query of the sequence (the next one's, or what the shared memory
                        // held) have no say: a row's bits depend on its sequence alone.
                        uint32_t pk[WORDS][16];
                        float sum = 0.f;
                        bool again = !__all_sync(0xffffffffu, !live || m > -INFINITY);
                        while (true) {
                            if (again) {
                                float top = -INFINITY;
#pragma unroll
                                for (int c0 = 0; c0 < WORDS; c0 += STEP) {
                                    fetch(c0);
                                    top = largest(top);
                                }
                                if (HALVES == 2) {
                                    s_own[(w * HALVES + half) * 128 + row] = top;
                                    named_sync(pair_id, 64);
                                    top = fmaxf(top, s_own[(w * HALVES + 1 - half) * 128 + row]);
                                }
                                const float mn = fmaxf(m, top);
                                const float a = m == -INFINITY ? 0.f : ex2_approx((m - mn) * f);
                                m = mn;
                                l *= a;
                                if (i > 0)   // every earlier product into O has completed before this tile's scores
                                    for (int c = half * 16; c < p.D; c += 16 * HALVES) {
                                        uint32_t y[16];
                                        tmem_ld_x16(tO + c, y);
                                        tmem_ld_wait();
#pragma unroll
                                        for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * a);
                                        tmem_st_x16(tO + c, y);
                                    }
                            }
                            // exponents relative to the maximum's rounded product with f,
                            // or past PG_FAR to the maximum itself (as for single tokens)
                            float base = S::BIAS - (m == -INFINITY ? 0.f : m * f);
                            const bool far = __any_sync(0xffffffffu, live && fabsf(base) > PG_FAR);
                            if (far) base = S::BIAS;
                            const uint64_t qk2 = pair_of(f, f), base2 = pair_of(base, base);
                            uint64_t sum2[2] = {0, 0};
                            float big = -INFINITY;
#pragma unroll
                            for (int c0 = 0; c0 < WORDS; c0 += STEP) {
                                fetch(c0);
                                if (far) {
#pragma unroll
                                    for (int c = 0; c < STEP; ++c)
#pragma unroll
                                        for (int e = 0; e < 32; ++e)
                                            s[c][e] = __float_as_uint(at(c, e) - (m == -INFINITY ? 0.f : m));
                                }
                                if (!again) big = largest(big);
#pragma unroll
                                for (int c = 0; c < STEP; ++c)
#pragma unroll
                                    for (int e = 0; e < 16; ++e) {
                                        float z0, z1;
                                        unpair(fma2(pair_of(at(c, 2 * e), at(c, 2 * e + 1)), qk2, base2), z0, z1);
                                        const float p0 = ex2_approx(z0), p1 = ex2_approx(z1);
                                        sum2[e & 1] = add2(sum2[e & 1], pair_of(p0, p1));
                                        pk[c0 + c][e] = E4M3 ? cvt_f16x2(p0, p1) : cvt_bf16x2(p0, p1);
                                    }
                            }
                            // also: the row's other thread has read its scores, which these weights overwrite
                            const bool stays = again || !live || !((far ? big : big - m) * f > S::LAG);
                            if (HALVES == 2 ? named_all(pair_id, 64, stays) : __all_sync(0xffffffffu, stays)) {
                                float a0, a1;
                                unpair(add2(sum2[0], sum2[1]), a0, a1);
                                sum = a0 + a1;
                                break;
                            }
                            again = true;
                        }
                        l += sum;
#pragma unroll
                        for (int c = 0; c < WORDS; ++c) tmem_st_x16(tS + (half * WORDS + c) * 16, pk[c]);
                    }
                    if (masked && t0 + row >= x.w.len) {
                        // a position's values, by its threads: zero past the end, and where not
                        // finite (by both streams where both see the tile: the same bytes)
                        const int at = 2 * (n + j) + 1, slot = at % RING;
                        wait(&kv_full[slot], (at / RING) & 1);
                        const bool past = t0 + row >= x.w.T;
                        bool odd = false;
#pragma unroll
                        for (int blk = 0; blk < BLK; ++blk) {
                            uint8_t* base = sR + slot * TILE + blk * PR_KT * 128 + row * 128;
                            // 16-byte piece c of the row; a thread takes its share of the eight
                            auto piece = [&](int c) { return reinterpret_cast<uint4*>(base + ((c ^ (row & 7)) << 4)); };
                            constexpr int SHARE = 8 / HALVES;
                            uint32_t probe[2] = {0, 0};
#pragma unroll
                            for (int c = half * SHARE; c < (half + 1) * SHARE; ++c) {
                                if (past) {
                                    *piece(c) = make_uint4(0, 0, 0, 0);
                                } else {
                                    const uint4 y = *piece(c);
                                    if (E4M3) {
                                        probe[0] = f16x2_probe(y.y, f16x2_probe(y.x, probe[0]));
                                        probe[1] = f16x2_probe(y.w, f16x2_probe(y.z, probe[1]));
                                    } else {
                                        probe[0] = bf16x2_probe(y.y, bf16x2_probe(y.x, probe[0]));
                                        probe[1] = bf16x2_probe(y.w, bf16x2_probe(y.z, probe[1]));
                                    }
                                }
                            }
                            if (((probe[0] | probe[1]) & 0x7FFF7FFFu) == 0) continue;
                            odd = true;
#pragma unroll 1
                            for (int c = half * SHARE; c < (half + 1) * SHARE; ++c) {
                                uint4 y = *piece(c);
                                uint32_t* e = &y.x;
#pragma unroll
                                for (int u = 0; u < 4; ++u) {
                                    constexpr uint32_t EXP = E4M3 ? 0x7C00u : 0x7F80u;
                                    if ((e[u] & EXP) == EXP) e[u] &= 0xFFFF0000u;
                                    if ((e[u] & EXP << 16) == EXP << 16) e[u] &= 0x0000FFFFu;
                                }
                                *piece(c) = y;
                            }
                        }
                        if (odd) atomicOr(odd_word, 1);
                        fence_async_smem();
                    }
                    __syncwarp();
                    tmem_st_wait();
                    tc_fence_before();
                    mbar_arrive(&p_full[w]);
                    if (i == 0 && piece_masked) learn_tree();   // while the products run
                }
                if (mine_tiles > 0) {
                    wait(&o_full[w], on++ & 1);
                    tc_fence_after();
                }
            }
            // ---------------------------------------- the piece's result
            if (!x.w.bad) {
                wait(&told[k & 7], (k >> 3) & 1);
                bad |= s_bad[k & 7] != 0;
                ++k;
            }
            const bool merge = x.solo && x.tiles > 1 && !x.w.bad;   // both streams hold parts of the same pairs
            if (HALVES == 2) s_own[(w * HALVES + half) * 128 + row] = l;
            named_sync(3, 2 * STREAM);                              // s_odd of both streams, sums of both halves
            if (HALVES == 2) l = s_own[w * HALVES * 128 + row] + s_own[(w * HALVES + 1) * 128 + row];
            const int learnt = s_odd[turn & 1][0] | s_odd[turn & 1][1];
            if (row == 0 && half == 0) s_odd[(turn + 1) & 1][w] = 0;             // read last before the previous piece's end
            const bool odd = learnt & 1;
            bad |= (learnt & 2) != 0;
            const bool whole = x.tiles == x.w.nt;
            const int slot = (int)blockIdx.x * 2 + (x.kt == 0 ? 1 : 0);
            const int prow = (x.solo ? 0 : w * p.rpt * p.hq) + row;   // pair within the item
            const bool writer = !(x.solo && w == 1) && live;
            m *= f;   // as exponents from here on
            float w0 = 1.f, w1 = 0.f, M = m, L = l;
            if (merge) {
                if (w == 1 && half == 0) s_xst[row] = make_float2(m, l);
                named_sync(3, 2 * STREAM);
                if (w == 0) {
                    const float2 o1 = s_xst[row];
                    M = fmaxf(m, o1.x);
                    w0 = m == -INFINITY ? 0.f : ex2_approx(m - M);
                    w1 = o1.x == -INFINITY ? 0.f : ex2_approx(o1.x - M);
                    L = l * w0 + o1.y * w1;
                }
            }
            if (bad) M = L = NAN;
            const float inv = (E4M3 && p.v_scale ? __ldg(p.v_scale + x.g) : 1.f) / L;
            const int64_t out_pair = (int64_t)(x.w.r0 + r) * p.H + x.g * p.hq + (row - row / p.hq * p.hq);
            // the second stream's rows, [128][XC] for each half, pieces of 16 bytes swizzled
            float* xb = reinterpret_cast<float*>(sX) + (half * PR_ROWS + row) * XC;
            constexpr int XP = XC / 4;   // 16-byte pieces
            auto xpiece = [&](int e) { return xb + ((e ^ (row & (XP - 1))) << 2); };
            auto fetch_out = [&](int c0, uint32_t (&y)[XC]) {
                if constexpr (XC == 32) tmem_ld_32x32b_x32(tO + c0, y);
                else tmem_ld_x16(tO + c0, y);
                tmem_ld_wait();
            };
            // every thread makes the same number of rounds: they meet at barriers
            for (int d0 = 0; d0 < p.D; d0 += XC * HALVES) {
                const int c0 = d0 + half * XC;
                if (merge) {
                    if (d0 > 0) named_sync(3, 2 * STREAM);
                    if (w == 1) {
                        uint32_t y[XC];
                        fetch_out(c0, y);
#pragma unroll
                        for (int e = 0; e < XP; ++e)
                            *reinterpret_cast<uint4*>(xpiece(e)) = make_uint4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
                    }
                    named_sync(3, 2 * STREAM);
                }
                float v[XC];
                if (!x.w.bad && mine_tiles > 0) {   // warp-uniform
                    uint32_t y[XC];
                    fetch_out(c0, y);
#pragma unroll
                    for (int e = 0; e < XC; ++e) v[e] = __uint_as_float(y[e]) * w0;
                } else {
#pragma unroll
                    for (int e = 0; e < XC; ++e) v[e] = 0.f;
                }
                if (writer) {
                    if (merge) {
#pragma unroll
                        for (int e = 0; e < XP; ++e) {
                            const float4 y = *reinterpret_cast<const float4*>(xpiece(e));
                            v[4 * e] = fmaf(y.x, w1, v[4 * e]);
                            v[4 * e + 1] = fmaf(y.y, w1, v[4 * e + 1]);
                            v[4 * e + 2] = fmaf(y.z, w1, v[4 * e + 2]);
                            v[4 * e + 3] = fmaf(y.w, w1, v[4 * e + 3]);
                        }
                    }
                    // groups of 16 dims: the head size is a multiple of that
                    if (whole) {
                        uint4* dst = reinterpret_cast<uint4*>(p.out + out_pair * p.D + c0);
#pragma unroll
                        for (int e = 0; e < XC / 8; ++e)
                            if (c0 + (e >> 1) * 16 < p.D)
                                dst[e] = make_uint4(cvt_bf16x2(v[8 * e] * inv, v[8 * e + 1] * inv),
                                                    cvt_bf16x2(v[8 * e + 2] * inv, v[8 * e + 3] * inv),
                                                    cvt_bf16x2(v[8 * e + 4] * inv, v[8 * e + 5] * inv),
                                                    cvt_bf16x2(v[8 * e + 6] * inv, v[8 * e + 7] * inv));
                    } else {
                        float4* dst = p.part + ((int64_t)slot * (p.D / 4) + c0 / 4) * 2 * PR_ROWS + prow;
#pragma unroll
                        for (int e = 0; e < XP; ++e)
                            if (c0 + (e >> 2) * 16 < p.D)
                                dst[e * 2 * PR_ROWS] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                    }
                }
                __syncwarp();
            }
            if (bad && row == 0) record_error(p.ctrl, WF_ERR_BAD_DATA, (uint32_t)x.b);
            if (writer && half == 0 && !whole) p.stat[slot * 2 * PR_ROWS + prow] = make_float2(M, L);
            if (writer && half == 0 && whole && p.lse)
                p.lse[out_pair] = (M + __log2f(L) - S::BIAS) * LN2;
            if (tid == 0 && x.pieces > 0) {
                p.join[blockIdx.x] = make_int4(x.pieces, x.w.r0 + 2 * x.mp * p.rpt, x.rows * p.hq, x.g);
                shared_item = true;
            }
            if (odd && !bad) {
                // rare: the values left out above, added behind the results to the rows
                // that see them (inf or NaN whatever is there)
                learn_tree();
                for (int j = 0; j <= r && writer; ++j) {
                    const int t = x.w.len + j;
                    if (t < x.kt * PR_KT || t >= (x.kt + x.tiles) * PR_KT) continue;
                    bool sees = !tree || j == 0 || j == r;
                    for (int a = r; a > j && !sees;) {
                        a = s_par[w][a];
                        sees = a == j;
                    }
                    const int page = p.table[(int64_t)x.b * p.max_pages + (t >> p.page_shift)];
                    if (!sees || page < 0 || page >= p.num_pages) continue;
                    const int64_t at = (((int64_t)page << p.page_shift) + (t & ((1 << p.page_shift) - 1))) * p.G + x.g;
#pragma unroll 1
                    for (int d = 0; d < p.D; ++d) {
                        if ((d / XC) % HALVES != half) continue;   // whoever wrote it above
                        const float y = E4M3 ? ((p.V[at * p.D + d] & 0x7F) == 0x7F ? NAN : 0.f)
                                             : pg_bf16_to_f32(reinterpret_cast<const uint16_t*>(p.V)[at * p.D + d]);
                        if (fabsf(y) < INFINITY) continue;
                        if (whole) {
                            uint16_t* o = p.out + out_pair * p.D + d;
                            *o = pg_f32_to_bf16(pg_bf16_to_f32(*o) + y);
                        } else {
                            float* o = reinterpret_cast<float*>(
                                p.part + ((int64_t)slot * (p.D / 4) + d / 4) * 2 * PR_ROWS + prow) + d % 4;
                            *o += y;
                        }
                    }
                }
            }
            if (!x.w.bad) n += x.tiles;
            named_sync(1 + w, STREAM);   // the stream has read the piece
            if (row == 0 && half == 0) mbar_arrive(&piece_free[turn & 7]);
        }
        if (tid == 0 && !shared_item) p.join[blockIdx.x] = make_int4(0, 0, 0, 0);
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    if (warp == SOFT) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ join
// The pieces of a shared item, added in order: piece k is CTA c + k's, its
// second slot for the item's first piece, else its first.  A thread takes four
// dims of a pair, a warp 128 bytes of a piece at a time and 32 of an output
// row.  An item's pieces follow from how much longer it is than a stretch: of
// many, ten are in flight for 8 pairs; of few, three for 32 pairs.  Few items
// begin in their CTA and end elsewhere, so every block lists them for itself
// and takes units of pairs in turn.
constexpr int RJ_THREADS = 256;
constexpr int RJ_FEW = 3;
static_assert(PA_MAX_ROUND_CTAS <= RJ_THREADS, "a thread lists an item");

struct JoinParams {
    const int4* join;
    const float4* part;
    const float2* stat;
    uint16_t* out;
    float* lse;
    const float* v_scale;
    float bias;
    int ctas, H, D, hq;
};

__device__ __forceinline__ int join_pairs(int pieces) { return pieces <= RJ_FEW ? 32 : 8; }   // of a unit

// W pairs a thread, 8 apart; BATCH pieces in flight
template <int W, int BATCH>
__device__ __forceinline__ void join_unit(const JoinParams& p, int4 j, int c, int pair0, int quad) {
    const int quads = p.D / 4;
    float4 v[W];
    float M[W], L[W];
#pragma unroll
    for (int q = 0; q < W; ++q) {
        v[q] = make_float4(0.f, 0.f, 0.f, 0.f);
        M[q] = -INFINITY;
        L[q] = 0.f;
    }
    for (int k0 = 0; k0 < j.x; k0 += BATCH) {
        float2 s2[BATCH][W];
        float4 y[BATCH][W];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int64_t slot = (int64_t)(c + k0 + k) * 2 + (k0 + k == 0);
#pragma unroll
            for (int q = 0; q < W; ++q) {
                const int pr = pair0 + 8 * q;
                const bool is = k0 + k < j.x && pr < j.z;
                s2[k][q] = is ? __ldcg(p.stat + slot * 2 * PR_ROWS + pr) : make_float2(-INFINITY, 0.f);
                y[k][q] = is ? __ldcg(p.part + (slot * quads + quad) * 2 * PR_ROWS + pr) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
#pragma unroll
        for (int q = 0; q < W; ++q) {
            float top = M[q];
#pragma unroll
            for (int k = 0; k < BATCH; ++k) top = fmaxf(top, s2[k][q].x);
            const float a = M[q] == -INFINITY ? 0.f : ex2_approx(M[q] - top);
            M[q] = top;
            L[q] *= a;
            v[q] = make_float4(v[q].x * a, v[q].y * a, v[q].z * a, v[q].w * a);
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const float w = s2[k][q].x == -INFINITY ? 0.f : ex2_approx(s2[k][q].x - top);
                L[q] = fmaf(s2[k][q].y, w, L[q]);
                v[q].x = fmaf(y[k][q].x, w, v[q].x);
                v[q].y = fmaf(y[k][q].y, w, v[q].y);
                v[q].z = fmaf(y[k][q].z, w, v[q].z);
                v[q].w = fmaf(y[k][q].w, w, v[q].w);
            }
        }
    }
    const float vs = p.v_scale ? __ldg(p.v_scale + j.w) : 1.f;
#pragma unroll
    for (int q = 0; q < W; ++q) {
        const int pr = pair0 + 8 * q;
        if (pr >= j.z) break;
        const float inv = vs / L[q];
        const int row = pr / p.hq;
        const int64_t at = (int64_t)(j.y + row) * p.H + j.w * p.hq + (pr - row * p.hq);
        *reinterpret_cast<uint2*>(p.out + at * p.D + quad * 4) =
            make_uint2(cvt_bf16x2(v[q].x * inv, v[q].y * inv), cvt_bf16x2(v[q].z * inv, v[q].w * inv));
        if (p.lse && quad == 0) p.lse[at] = (M[q] + __log2f(L[q]) - p.bias) * LN2;
    }
}

__global__ void __launch_bounds__(RJ_THREADS, 2) rounds_join_kernel(const JoinParams p) {
    __shared__ int4 s_item[PA_MAX_ROUND_CTAS];
    __shared__ int s_cta[PA_MAX_ROUND_CTAS], s_first[PA_MAX_ROUND_CTAS];   // its CTA, units before it
    __shared__ int s_sum[2][RJ_THREADS / 32];
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int4 it = make_int4(0, 0, 0, 0);   // pieces, first row, pairs, KV head
    if (tid < p.ctas) it = __ldcg(&p.join[tid]);
    const int mine = it.x > 0 ? (it.z + join_pairs(it.x) - 1) / join_pairs(it.x) : 0;
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
    }
    const unsigned some = __ballot_sync(0xffffffffu, mine > 0);
    if (lane == 31) s_sum[0][warp] = upto, s_sum[1][warp] = __popc(some);
    __syncthreads();
    int units = 0, items = 0, units0 = 0, items0 = 0;
#pragma unroll
    for (int w = 0; w < RJ_THREADS / 32; ++w) {
        if (w == warp) units0 = units, items0 = items;
        units += s_sum[0][w];
        items += s_sum[1][w];
    }
    if (mine > 0) {
        const int at = items0 + __popc(some & ((1u << lane) - 1u));
        s_item[at] = it;
        s_cta[at] = tid;
        s_first[at] = units0 + upto - mine;
    }
    __syncthreads();
    const int quad = warp * 4 + (lane >> 3);
    if (quad >= p.D / 4) return;
    int i = 0;
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
        while (i + 1 < items && s_first[i + 1] <= u) ++i;
        const int4 j = s_item[i];
        const int pair0 = (u - s_first[i]) * join_pairs(j.x) + (lane & 7);
        if (j.x <= RJ_FEW) join_unit<4, RJ_FEW>(p, j, s_cta[i], pair0, quad);
        else join_unit<1, 10>(p, j, s_cta[i], pair0, quad);
    }
}

// ------------------------------------------------------------------ host side
static PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return enc;
}

// The queries as [P, H, D] in boxes of 64 dims x hq heads x rpt rows: a box is
// the 128-byte rows of a product's operand, row by row.
static bool query_map(CUtensorMap* map, const wf_paged_attn_args* a, int D, int hq, int rpt) {
    const auto enc = encoder();
    if (!enc) return false;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a->H, (cuuint64_t)a->P};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)a->q_stride * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)hq, (cuuint32_t)rpt};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(a->q), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// An 8-bit pool's layer as [rows, G * D] bytes in boxes of a head's row by `box_rows`.
static bool raw_map(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, int D, int box_rows) {
    const auto enc = encoder();
    if (!enc) return false;
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {cols};
    cuuint32_t box[2] = {(cuuint32_t)D, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

using RoundsFn = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, RoundsParams);

struct RoundsVariant {
    RoundsFn fn;
    int smem, threads;
};

// bit 0: an 8-bit cache; bit 1: heads wider than 64
static RoundsVariant rounds_variant(int i) {
    switch (i) {
        case 0: return {paged_rounds_kernel<1, false>, RoundsShape<1, false>::SMEM,
                         RoundsShape<1, false>::THREADS};
        case 1: return {paged_rounds_kernel<1, true>, RoundsShape<1, true>::SMEM,
                         RoundsShape<1, true>::THREADS};
        case 2: return {paged_rounds_kernel<2, false>, RoundsShape<2, false>::SMEM,
                         RoundsShape<2, false>::THREADS};
        default: return {paged_rounds_kernel<2, true>, RoundsShape<2, true>::SMEM,
                         RoundsShape<2, true>::THREADS};
    }
}

wf_status launch_paged_rounds(const wf_paged_cache* c, const wf_paged_attn_args* a, void* ws, cudaStream_t s) {
    static std::mutex mu;
    static bool attr_set[64] = {false};
    PR_TRY(configure_once(mu, attr_set, [] {
        for (int i = 0; i < 4; ++i) {
            const RoundsVariant v = rounds_variant(i);
            if (cudaFuncSetAttribute(v.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, v.smem) != cudaSuccess)
                return false;
        }
        // as for the catch-up's kernels: no change of the carveout between launches
        return cudaFuncSetAttribute(rounds_join_kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100) ==
               cudaSuccess;
    }));
    const bool e4m3 = c->kv_type == WF_KV_E4M3;
    uint8_t* w = static_cast<uint8_t*>(ws);
    const PagedLayout L = paged_layout(c->D, a->max_rows);
    const int64_t layer_bytes = (int64_t)c->num_pages * c->page_size * c->G * c->D * (e4m3 ? 1 : 2);
    const uint8_t* K = static_cast<const uint8_t*>(c->K) + a->layer * layer_bytes;
    RoundsParams p = {};
    p.pos_off = a->pos_off;
    p.cache_len = a->cache_len;
    p.node_off = a->node_off;
    p.kind = a->kind;
    p.parent = a->parent;
    p.table = c->table;
    p.V = static_cast<const uint8_t*>(c->V) + a->layer * layer_bytes;
    p.k_scale = c->k_scale ? c->k_scale + (int64_t)a->layer * c->G : nullptr;
    p.v_scale = c->v_scale ? c->v_scale + (int64_t)a->layer * c->G : nullptr;
    p.out = a->out;
    p.lse = a->lse;
    p.part = reinterpret_cast<float4*>(w + L.part);
    p.stat = reinterpret_cast<float2*>(w + L.stat);
    p.join = reinterpret_cast<int4*>(w + L.join);
    p.qk = a->scale * LOG2E;
    p.P = a->P;
    p.H = a->H;
    p.G = c->G;
    p.D = c->D;
    p.hq = a->H / c->G;
    p.B = c->B;
    while ((1 << p.page_shift) < c->page_size) ++p.page_shift;
    p.num_pages = c->num_pages;
    p.max_pages = c->max_pages;
    p.max_rows = a->max_rows;
    p.rpt = PR_ROWS / p.hq;
    p.box_rows = c->page_size < PR_KT ? c->page_size : PR_KT;
    p.per_tile = PR_KT / p.box_rows;
    // fp16 operands are format 0 where bf16 are 1; the values' contiguous dimension is N
    const uint32_t formats = e4m3 ? (1u << 7) | (1u << 10) : 0u;
    p.idesc_s = umma_idesc_bf16(PR_ROWS, PR_KT) & ~formats;
    p.idesc_o = (umma_idesc_bf16(PR_ROWS, c->D) & ~formats) | (1u << 16);
    p.ctrl = static_cast<Control*>(ws);
    p.timeout_ns = wait_timeout_ns();
    CUtensorMap tmQ, tmK, tmV;
    if (!query_map(&tmQ, a, c->D, p.hq, p.rpt)) return WF_ERR_CUDA;
    const uint64_t rows = (uint64_t)c->num_pages * c->page_size, cols = (uint64_t)c->G * c->D;
    if (e4m3 ? !raw_map(&tmK, K, rows, cols, c->D, p.box_rows) || !raw_map(&tmV, p.V, rows, cols, c->D, p.box_rows)
             : !make_map(&tmK, K, rows, cols, (uint32_t)p.box_rows) ||
                   !make_map(&tmV, p.V, rows, cols, (uint32_t)p.box_rows))
        return WF_ERR_CUDA;
    int grid = num_sms() < PA_MAX_ROUND_CTAS ? num_sms() : PA_MAX_ROUND_CTAS;
    // no more CTAs than tiles that the bounds allow
    const int64_t tiles = (int64_t)c->B * c->G * cdiv(a->max_rows, 2 * p.rpt) *
                          cdiv((int64_t)c->max_pages * c->page_size, PR_KT);
    if (tiles < grid) grid = (int)tiles;
    const RoundsVariant v = rounds_variant((e4m3 ? 1 : 0) | (c->D > 64 ? 2 : 0));
    PR_TRY(launch(v.fn, dim3(grid), dim3(v.threads), (size_t)v.smem, s, tmQ, tmK, tmV, p));
    JoinParams jp = {};
    jp.join = p.join;
    jp.part = p.part;
    jp.stat = p.stat;
    jp.out = a->out;
    jp.lse = a->lse;
    jp.v_scale = p.v_scale;
    jp.bias = e4m3 ? RoundsShape<1, true>::BIAS : RoundsShape<1, false>::BIAS;
    jp.ctas = grid;
    jp.H = a->H;
    jp.D = c->D;
    jp.hq = p.hq;
    // no more blocks than units that the bounds allow
    const int most = a->max_rows < 2 * p.rpt ? a->max_rows : 2 * p.rpt;   // query rows of an item
    const int units = grid * cdiv(most * p.hq, 8), blocks = 2 * num_sms();
    return launch(rounds_join_kernel, dim3(units < blocks ? units : blocks), dim3(RJ_THREADS), 0, s, jp);
}

}  // namespace wf
