// One sweep of a head's weights over the rows (wf_lmhead_logprobs, the forward
// part of wf_draft_distill):
//   v = <act_row, W_id>   (bf16 products, fp32 sums, in TMEM only)
// and per row, as the tiles of logits leave the accumulator,
//   M = max v,  S = sum 2^z,  T = sum z 2^z,  z = c (v - M),  c = log2(e) / temperature
// (lse and entropy follow from them), the k best (v, id), the logits of the
// row's listed ids, and, where asked for, the logits themselves in fp32.
//
// A row's states stay with the CTA: its thread keeps M, S, T and the k best in
// registers from tile to tile, and puts them aside in the workspace only when
// the CTA's next tile is of other rows.  So a row ends with one state per CTA
// that saw it, not one per tile (4,096 rows over 151,936 ids with 16 best: 76
// states of 144 bytes a row instead of 594), and what a tile adds to the k best
// is a few insertions.
// With several row tiles the pairs that see the same rows tell each other their
// tiles' maxima, which bound the row's KT-th best from below, so that late columns
// are candidates for few lists (1,215 rows of 512 over 123,478 ids with 10 best: 270
// us a call without, 188 so): what is a candidate differs with timing, the k best
// among them do not.
// One activation tile (up to 128 rows): bound by the weights' bytes; every CTA
// its own tiles, ring slots as large as the rows (17 rows of 2,560 over 151,936
// ids: 118 us, 6.6 TB/s).  More rows: pairs of CTAs on tiles of 256 rows x 256
// ids, bound by the tensor cores (1,248 rows with 10 best: 482 to 494 us, 2.0
// PFLOP/s, and 550 to 560 in a long run at the power cap; 3,967 rows with 16: 1.48
// ms rested, 1.6 to 1.7 at the cap; with d below about 1,000 by what the four
// epilogue warps do with a tile).
#include <cudaTypedefs.h>

#include <cfloat>

#include "wf_heads.cuh"
#include "wf_tiles.cuh"

namespace wf {

namespace {

constexpr int SWEEP_THREADS = pipe_threads(4);
constexpr int SWEEP_SMEM = 220 * 1024;   // leaves room on the SM for CTAs of the lists
constexpr int STAGING = 4 * 2 * 4096;     // kept logits: two boxes of 32 rows x 128 bytes a warp
static_assert(SWEEP_SMEM + PIPE_STATIC_MAX <= PIPE_SMEM_MAX, "a CTA's shared memory");
// a pair's ring fills SWEEP_SMEM but for less than a stage, the largest of them 128 rows of A and half a tile of B
constexpr int PAIR_STAGE_MAX = (BM + MAX_TILE / 2) * BK * 2;
static_assert((SWEEP_SMEM - STAGING) / ((BM + MIN_TILE / 2) * BK * 2) <= PIPE_MAX_STAGES, "... whatever the tile");
static_assert(pipe_alone(SWEEP_SMEM - PAIR_STAGE_MAX), "no SM holds CTAs of two pairs");

struct SweepParams {
    int rows, V;
    int num_m, num_mt, num_n, num_k;      // 128-row tiles, row tiles of the schedule, weight tiles, K blocks
    int bn, nbig, step;                   // nbig weight tiles of bn rows, then tiles of bn - step
    uint32_t idesc, idesc_s;
    int stages, stage_bytes, a_bytes;
    float c, inv_t;
    const int32_t* pick;                  // [rows][K] ids in any order
    int K;
    float* picked;
    uint8_t* states;
    int slots;                            // states per row
    uint32_t* reached;                    // [rows][REACHED] maxima of classes of tiles (f32_order, 0 = none yet), or null
    Control* ctrl;
    uint64_t timeout_ns;
};

struct Span {
    int row0, rows;
    bool big;
};
// The tiles of one CTA (or pair): unit u = slot, slot + slots, ... is row tile u %
// num_mt and weight tile u / num_mt, counted on without divisions.
struct Walk {
    int u, mt, n, step, dm, dn;
    __device__ __forceinline__ Walk(const SweepParams& p, int slot, int slots)
        : u(slot), mt(slot % p.num_mt), n(slot / p.num_mt), step(slots), dm(slots % p.num_mt), dn(slots / p.num_mt) {}
    __device__ __forceinline__ void on(const SweepParams& p) {
        u += step;
        mt += dm;
        n += dn;
        if (mt >= p.num_mt) {
            mt -= p.num_mt;
            ++n;
        }
    }
};
__device__ __forceinline__ Span span(const SweepParams& p, int n) {
    if (n < p.nbig) return {n * p.bn, p.bn, true};
    const int h = p.bn - p.step;
    return {p.nbig * p.bn + (n - p.nbig) * h, h, false};
}

// r[j] for a j that is known only at run time: five levels of selects.
__device__ __forceinline__ uint32_t column(const uint32_t (&r)[32], int j) {
    uint32_t a[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) a[i] = j & 1 ? r[2 * i + 1] : r[2 * i];
#pragma unroll
    for (int w = 8, bit = 2; w >= 1; w >>= 1, bit <<= 1)
#pragma unroll
        for (int i = 0; i < w; ++i) a[i] = j & bit ? a[2 * i + 1] : a[2 * i];
    return a[0];
}

// Insert (v, id) into a descending list; the earlier entry wins ties.
template <int KT>
__device__ __forceinline__ void insert(float (&tv)[KT], int (&ti)[KT], float v, int id) {
#pragma unroll
    for (int j = KT - 1; j > 0; --j) {
        const bool shift = tv[j - 1] < v;
        const bool land = !shift && tv[j] < v;
        tv[j] = shift ? tv[j - 1] : (land ? v : tv[j]);
        ti[j] = shift ? ti[j - 1] : (land ? id : ti[j]);
    }
    if (tv[0] < v) {
        tv[0] = v;
        ti[0] = id;
    }
}

template <int KT>
struct State {
    float M, S, T;
    float tv[KT > 0 ? KT : 1];
    int ti[KT > 0 ? KT : 1];
    __device__ __forceinline__ void clear() {
        M = -INFINITY;
        S = T = 0.f;
        if constexpr (KT > 0) {
#pragma unroll
            for (int j = 0; j < KT; ++j) {
                tv[j] = -INFINITY;
                ti[j] = -1;
            }
        }
    }
    __device__ __forceinline__ void put(uint8_t* at) const {
        float4* o = reinterpret_cast<float4*>(at);
        o[0] = make_float4(M, S, T, 0.f);
        if constexpr (KT > 0) {
#pragma unroll
            for (int j = 0; j < KT; j += 2)
                o[1 + j / 2] = make_float4(tv[j], __int_as_float(ti[j]), tv[j + 1], __int_as_float(ti[j + 1]));
        }
    }
    __device__ __forceinline__ void get(const uint8_t* at) {
        const float4* o = reinterpret_cast<const float4*>(at);
        const float4 h = o[0];
        M = h.x;
        S = h.y;
        T = h.z;
        if constexpr (KT > 0) {
#pragma unroll
            for (int j = 0; j < KT; j += 2) {
                const float4 e = o[1 + j / 2];
                tv[j] = e.x;
                ti[j] = __float_as_int(e.y);
                tv[j + 1] = e.z;
                ti[j + 1] = __float_as_int(e.w);
            }
        }
    }
};

// A number below v that nothing lies between (for a zero, of either sign, the
// first that arithmetic without denormals tells from it).
__device__ __forceinline__ float just_below(float v) {
    return v == 0.f ? -FLT_MIN : f32_unorder(f32_order(v) - 1);
}

// A bound that the KT-th best of a tile's columns reaches: the KT-th largest of
// 32 maxima, each over the columns 32 apart, which are KT different columns.  An
// empty list would take nearly every column of its first chunks; held to this
// bound it takes about KT + 3 of 256.  A number just below the bound is returned,
// to be exceeded.
template <int KT>
__device__ __forceinline__ float first_bound(uint32_t tbase, int cols) {
    float top[32], best[KT];
#pragma unroll
    for (int j = 0; j < 32; ++j) top[j] = -INFINITY;
#pragma unroll
    for (int j = 0; j < KT; ++j) best[j] = -INFINITY;
    for (int c0 = 0; c0 + 32 <= cols; c0 += 32) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(tbase + c0, r);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) top[j] = fmaxf(top[j], __uint_as_float(r[j]));
    }
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        float v = top[j];
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            const float hi = fmaxf(best[i], v);
            v = fminf(best[i], v);
            best[i] = hi;
        }
    }
    return best[KT - 1] == -INFINITY ? -INFINITY : just_below(best[KT - 1]);
}

// The weight tiles n of a row fall into 16 classes n mod 16, whose maxima all pairs
// put down as they see them.  The KT-th largest of these is reached by KT different
// columns, and lies not far below the row's KT-th best so far: 10 of 16 have about
// 16 columns above it.  (The least of 10 classes needs no sorting and has about 30:
// 208 us where this takes 199, 1,215 rows of 512 over 123,478 ids; 16 of 32 classes
// for 16 best, in two sorted halves, cost more than they spared: 3,000 rows of 1,000
// over 60,000 ids 408 us, the least of 16 classes 380.)
// Descending order of 16 numbers (bitonic).
__device__ __forceinline__ void sort16(uint32_t (&v)[16]) {
#pragma unroll
    for (int s = 1; s <= 4; ++s)
#pragma unroll
        for (int t = s - 1; t >= 0; --t)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int o = i ^ (1 << t);
                if (o > i) {
                    const uint32_t a = v[i], b = v[o];
                    const bool down = (i >> s & 1) == 0;
                    v[i] = down ? max(a, b) : min(a, b);
                    v[o] = down ? min(a, b) : max(a, b);
                }
            }
}
template <int KT>
__device__ __forceinline__ uint32_t reached_by(const uint32_t* at) {
    uint32_t v[REACHED];
#pragma unroll
    for (int j = 0; j < REACHED; j += 4) {
        const uint4 q = __ldcg(reinterpret_cast<const uint4*>(at + j));
        v[j] = q.x;
        v[j + 1] = q.y;
        v[j + 2] = q.z;
        v[j + 3] = q.w;
    }
    if constexpr (KT < REACHED) {
        sort16(v);
        return v[KT - 1];
    }
    uint32_t least = v[0];
#pragma unroll
    for (int j = 1; j < REACHED; ++j) least = min(least, v[j]);
    return least;
}

// Two numbers in one 64-bit register, and (a + add) * mul of two at a time, each
// step rounded.  (A fused product with a rounded c M would be one step, and off by
// c M 2^-24.  Where the fold bounds, 1,215 rows of 512 over 123,478 ids without
// alternatives, that is 133 us and this 140; 1,248 rows of 2,560 take 526 either way.)
__device__ __forceinline__ uint64_t pair_f32(float lo, float hi) {
    uint64_t p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
    return p;
}
__device__ __forceinline__ void sum_times(float (&z)[2], float a, float b, uint64_t add, uint64_t mul) {
    asm("{\n\t.reg .b64 v;\n\tmov.b64 v, {%2, %3};\n\tadd.rn.f32x2 v, v, %4;\n\tmul.rn.f32x2 v, v, %5;\n\t"
        "mov.b64 {%0, %1}, v;\n\t}"
        : "=f"(z[0]), "=f"(z[1])
        : "f"(a), "f"(b), "l"(add), "l"(mul));
}

// Fold 32 columns (the first lim of them) into a row's state; only columns above
// `bound` are candidates for its list.  Returns their maximum.
template <int KT, bool ENT, bool FULL>
__device__ __forceinline__ float fold(const uint32_t (&r)[32], int lim, int col0, float c, float bound,
                                     State<KT>& st) {
    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int j = 0; j < 32; ++j)
        if (FULL || j < lim) m4[j & 3] = fmaxf(m4[j & 3], __uint_as_float(r[j]));
    const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
    if (mx > st.M) {   // a new largest logit: rescale what was summed so far
        if (st.S != 0.f) {
            const float dz = (st.M - mx) * c;
            const float sc = ex2_approx(dz);
            if constexpr (ENT) st.T = sc == 0.f && st.S == st.S ? 0.f : (st.T + dz * st.S) * sc;
            st.S *= sc;
        }
        st.M = mx;
    }
    const uint64_t below = pair_f32(-st.M, -st.M), c2 = pair_f32(c, c);
    float s4[4] = {0.f, 0.f, 0.f, 0.f}, t4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
        float z[2];
        sum_times(z, __uint_as_float(r[j]), __uint_as_float(r[j + 1]), below, c2);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (FULL || j + h < lim) {
                const float e = ex2_approx(z[h]);
                s4[(j + h) & 3] += e;
                if constexpr (ENT) t4[(j + h) & 3] = fmaf(z[h], e, t4[(j + h) & 3]);
            }
    }
    st.S += (s4[0] + s4[1]) + (s4[2] + s4[3]);
    if constexpr (ENT) st.T += (t4[0] + t4[1]) + (t4[2] + t4[3]);
    if constexpr (KT > 0) {
        // Columns above the row's k-th best as a mask; then every row of the warp
        // takes its next one at the same time, so a chunk costs as many rounds as
        // its busiest row has candidates (one or two once a few tiles are seen).
        // Inserting column by column, which any of 32 rows can ask for, took 2.2
        // times as long as the tile's products (1,248 rows: 1,065 us a call).
        const float least = fmaxf(st.tv[KT - 1], bound);
        uint32_t cand = 0;
        if (__any_sync(0xffffffffu, mx > least)) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (FULL || j < lim) cand |= __uint_as_float(r[j]) > least ? 1u << j : 0u;
        }
        while (__any_sync(0xffffffffu, cand != 0)) {
            if (cand) {
                const int j = __ffs((int)cand) - 1;
                cand &= cand - 1;
                const float v = __uint_as_float(column(r, j));
                if (v > st.tv[KT - 1]) insert<KT>(st.tv, st.ti, v, col0 + j);
            }
        }
    }
    return mx;
}

template <int KT, bool ENT, bool Z, bool PAIR>
__global__ void __launch_bounds__(SWEEP_THREADS, 1)
    sweep_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const __grid_constant__ CUtensorMap tmBs, const __grid_constant__ CUtensorMap tmZ,
                 const SweepParams p) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t seen[4][SWEEP_MAX_ROWS / BM / 32];   // row tiles that a warp has a state of
    static_assert(sizeof(seen) <= PIPE_STATIC_MAX, "static shared memory");
    const Pipe g = pipe_at(smem_raw, p.stages, p.stage_bytes, p.a_bytes, Z ? STAGING : 0, p.ctrl, p.timeout_ns);
    const int warp = warp_number(), lane = threadIdx.x & 31;
    const int rank = PAIR ? (int)(cluster_ctarank() & 1u) : 0;
    const bool first = rank == 0;
    const int slot = PAIR ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
    const int nslots = PAIR ? (int)(gridDim.x >> 1) : (int)gridDim.x;
    const int units = p.num_mt * p.num_n;   // unit u: row tile u % num_mt, weight tile u / num_mt
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
        if (p.nbig < p.num_n) tma_prefetch_desc(&tmBs);
        if constexpr (Z) tma_prefetch_desc(&tmZ);
    }
    const uint32_t tmem_base = pipe_begin<PAIR, 4>(g);
    if (warp != 0) pdl_wait();   // warp 0: when it has asked for its first weights

    if (warp == 0) {
        const uint64_t pol_w = policy_evict_first(), pol_a = policy_evict_last();
        int m = 0;
        Span sp{};
        Walk w(p, slot, nslots);
        auto next = [&](int) {
            if (w.u >= units) return 0;
            m = PAIR ? 2 * w.mt + rank : w.mt;
            sp = span(p, w.n);
            w.on(p);
            return p.num_k;
        };
        auto tx = [&]() { return (uint32_t)((PAIR ? 2 : 1) * p.a_bytes + sp.rows * BK * 2); };
        auto load = [&](int kc, int s, uint32_t bar, bool a, bool b) {
            if (a) pipe_load<PAIR>(g.a(s), &tmA, bar, kc * BK, m * BM, pol_a);
            if (b)
                pipe_load<PAIR>(g.b(s), sp.big ? &tmB : &tmBs, bar, kc * BK,
                                sp.row0 + (PAIR ? rank * (sp.rows / 2) : 0), pol_w);
        };
        pipe_copy<PAIR, true>(g, first, next, tx, load);
    } else if (warp == 1) {
        if (first) {
            uint32_t idesc = 0;
            Walk w(p, slot, nslots);
            auto next = [&](int) {
                if (w.u >= units) return 0;
                idesc = w.n < p.nbig ? p.idesc : p.idesc_s;
                w.on(p);
                return p.num_k;
            };
            auto issue = [&](int s, uint32_t d, int kc) {
                const uint64_t a = umma_desc_sw128(smem_u32(g.a(s))), b = umma_desc_sw128(smem_u32(g.b(s)));
#pragma unroll
                for (int kk = 0; kk < BK / 16; ++kk) {   // 32 bytes of K a step
                    if constexpr (PAIR)
                        umma_bf16_pair(d, a + 2 * kk, b + 2 * kk, idesc, (kc | kk) != 0);
                    else
                        umma_bf16(d, a + 2 * kk, b + 2 * kk, idesc, (kc | kk) != 0);
                }
            };
            pipe_mma<PAIR>(g, tmem_base, next, issue);
        }
    } else {
        const int q = warp & 3;            // TMEM lane quadrant that this warp may access
        const int rit = q * 32 + lane;
        const uint32_t tempty_first = (PAIR && !first) ? cluster_addr(&g.tempty[0], 0) : 0;
        uint8_t* stage = pipe_extra(g) + q * 2 * 4096;
        for (int j = lane; j < (int)(sizeof(seen[0]) / 4); j += 32) seen[q][j] = 0;
        __syncwarp();
        State<KT> st;
        st.clear();
        int cur = -1;                      // the row tile whose states the registers hold
        int box = 0;                       // Z: staging box in use
        auto state_of = [&](int row) { return p.states + ((size_t)row * p.slots + slot) * state_bytes(KT); };
        Walk w(p, slot, nslots);
        for (uint32_t i = 0; w.u < units; ++i, w.on(p)) {
            const int mt = w.mt, m = PAIR ? 2 * mt + rank : mt;
            const Span sp = span(p, w.n);
            const int row = m * BM + rit;
            const bool warp_live = m * BM + q * 32 < p.rows, live = row < p.rows;
            bool fresh = false;   // the list is empty
            uint32_t shared = 0;  // what the row's KT-th best has reached in what all pairs put down
            if constexpr (KT > 0) {
                if (p.reached && live) shared = reached_by<KT>(p.reached + (size_t)row * REACHED);
            }
            if (mt != cur) {
                if (cur >= 0) {
                    const int was = (PAIR ? 2 * cur + rank : cur) * BM + rit;
                    if (was < p.rows) st.put(state_of(was));
                }
                if ((seen[q][mt >> 5] >> (mt & 31)) & 1) {
                    if (live) st.get(state_of(row));
                } else {
                    fresh = true;
                    st.clear();
                    __syncwarp();
                    if (lane == 0) seen[q][mt >> 5] |= 1u << (mt & 31);
                    __syncwarp();
                }
                cur = mt;
                if constexpr (KT > 0) {
                    if (!live) st.tv[KT - 1] = INFINITY;   // rows that are none insert nothing
                }
            }
            // The row's listed ids in this tile: their places as bits, and the lowest of them.  The list is in any
            // order and looked through once a tile; a look through it for each chunk of columns that holds some of it
            // took 565 us where this takes 201 (2,048 rows of 2,560 over 32,000 ids, 64 listed).
            const size_t list = (size_t)row * p.K;
            int next_id = PICK_NONE;
            uint32_t here[2] = {0u, 0u};
            if (live) {
                const int end = sp.row0 + min(sp.rows, p.V - sp.row0);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll 16
                    for (int j = 32 * h; j < min(p.K, 32 * h + 32); ++j) {
                        const int id = p.pick[list + j];
                        if (id >= sp.row0 && id < end) {
                            here[h] |= 1u << (j & 31);
                            next_id = min(next_id, id);
                        }
                    }
            }
            if (!pipe_acc_wait(g, i)) break;
            if (warp_live) {
                const uint32_t tbase = tmem_base + ((uint32_t)(q * 32) << 16) + (i & 1) * BN;
                const int cols = min(sp.rows, p.V - sp.row0);
                float bound = -INFINITY;
                if constexpr (KT > 0) {
                    if (shared) bound = just_below(f32_unorder(shared));   // as good as it is still a candidate
                    if (fresh && __any_sync(0xffffffffu, live && !shared))
                        bound = fmaxf(bound, first_bound<KT>(tbase, cols));
                }
                float top = -INFINITY;   // of the tile's columns
                for (int c0 = 0; c0 < cols; c0 += 32) {
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(tbase + c0, r);
                    tmem_ld_wait();
                    const int col0 = sp.row0 + c0, lim = min(32, cols - c0);
                    top = fmaxf(top, lim == 32 ? fold<KT, ENT, true>(r, 32, col0, p.c, bound, st)
                                               : fold<KT, ENT, false>(r, lim, col0, p.c, bound, st));
                    if (__any_sync(0xffffffffu, next_id < col0 + lim)) {
                        // an id may be there twice; one look through the tile's places takes all of the chunk's
                        if (next_id < col0 + lim) {
                            next_id = PICK_NONE;
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                for (uint32_t left = here[h]; left; left &= left - 1) {
                                    const int j = __ffs((int)left) - 1, id = p.pick[list + 32 * h + j];
                                    if (id < col0 + lim) {
                                        p.picked[list + 32 * h + j] = __uint_as_float(column(r, id - col0));
                                        here[h] &= ~(1u << j);
                                    } else {
                                        next_id = min(next_id, id);
                                    }
                                }
                        }
                    }
                    if constexpr (Z) {
                        // 32 x 32 logits to the staging box, out by one tensor copy (clipped at the
                        // last row, and the last id rounded up to 16 bytes)
                        uint8_t* to = stage + box * 4096;
                        if (lane == 0) tma_store_wait_read<1>();
                        __syncwarp();
#pragma unroll
                        for (int j = 0; j < 32; j += 4)
                            *reinterpret_cast<float4*>(to + swizzled(lane, j >> 2)) =
                                make_float4(__uint_as_float(r[j]) * p.inv_t, __uint_as_float(r[j + 1]) * p.inv_t,
                                            __uint_as_float(r[j + 2]) * p.inv_t, __uint_as_float(r[j + 3]) * p.inv_t);
                        fence_async_store();
                        __syncwarp();
                        if (lane == 0) tma_store_2d(&tmZ, to, col0, m * BM + q * 32);
                        __syncwarp();
                        box ^= 1;
                    }
                }
                if constexpr (KT > 0) {
                    // a class's maximum below what is reached has no say in it
                    if (p.reached && live && top > -INFINITY && f32_order(top) > shared)
                        atomicMax(p.reached + (size_t)row * REACHED + w.n % REACHED, f32_order(top));
                }
            }
            pipe_acc_release(g, i, tempty_first);
        }
        if (cur >= 0) {
            const int was = (PAIR ? 2 * cur + rank : cur) * BM + rit;
            if (was < p.rows) st.put(state_of(was));
        }
        // rows that this CTA never saw get an empty state, so that the merge reads nothing stale
        for (int mt = 0; mt < p.num_mt; ++mt) {
            if ((seen[q][mt >> 5] >> (mt & 31)) & 1) continue;
            const int row = (PAIR ? 2 * mt + rank : mt) * BM + rit;
            if (row < p.rows) {
                State<KT> none;
                none.clear();
                none.put(state_of(row));
            }
        }
        if constexpr (Z) {
            if (lane == 0) tma_store_wait_all();
        }
    }
    pipe_end<PAIR>(g, tmem_base);
}

template <int KT, bool ENT, bool Z>
wf_status launch_kt(const SweepCall& c, int* slots_out, cudaStream_t s) {
    static std::mutex mu;
    static bool attr_set[64] = {false};
    const wf_status cst = configure_once(mu, attr_set, [] {
        return set_smem(sweep_kernel<KT, ENT, Z, false>, SWEEP_SMEM) &&
               set_smem(sweep_kernel<KT, ENT, Z, true>, SWEEP_SMEM);
    });
    if (cst != WF_OK) return cst;
    const bool pair = c.rows > BM;
    SweepParams p{};
    p.rows = c.rows;
    p.V = c.V;
    p.num_m = cdiv(c.rows, BM);
    p.num_mt = pair ? cdiv(p.num_m, 2) : 1;
    p.num_k = cdiv(c.d, BK);
    const int a_rows = pair ? BM : (c.rows + 7) / 8 * 8;   // a short box reads no rows that are not there
    p.a_bytes = a_rows * BK * 2;
    int slots = 0;
    if (pair) {
        static std::mutex pmu;
        static int pairs[64];
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return WF_ERR_CUDA;
        std::lock_guard<std::mutex> lock(pmu);
        if (dev >= 64 || !pairs[dev]) {
            slots = resident_pairs(reinterpret_cast<const void*>(sweep_kernel<KT, ENT, Z, true>), SWEEP_THREADS,
                                   SWEEP_SMEM);
            if (dev < 64) pairs[dev] = slots;
        } else {
            slots = pairs[dev];
        }
    } else {
        slots = num_sms() < STATE_SLOTS ? num_sms() : STATE_SLOTS;
    }
    const Tiles t = tiles_of(c.V, slots, p.num_mt, tile_step(pair, Z));
    const int b_bytes = (pair ? t.bn / 2 : t.bn) * BK * 2, extra = Z ? STAGING : 0;
    p.stage_bytes = p.a_bytes + b_bytes;
    // an MMA reads BM rows of A whatever the box holds: the last stage's may reach past a stage that is shorter
    const int reach = BM * BK * 2 > p.stage_bytes ? BM * BK * 2 - p.stage_bytes : 0;
    p.stages = (SWEEP_SMEM - PIPE_BARRIER_BYTES - 1024 - extra - reach) / p.stage_bytes;
    if (p.stages > PIPE_MAX_STAGES) p.stages = PIPE_MAX_STAGES;
    const int smem = pipe_smem(p.stages, p.stage_bytes, extra) + reach;
    p.num_n = t.num_n;
    p.bn = t.bn;
    p.nbig = t.nbig;
    p.step = t.step;
    const int units = p.num_mt * p.num_n;
    if (units < slots) slots = units;
    const unsigned split = pair ? 2 : 1;
    p.idesc = umma_idesc_bf16(split * BM, p.bn);
    p.idesc_s = p.nbig < p.num_n ? umma_idesc_bf16(split * BM, p.bn - p.step) : p.idesc;
    p.c = LOG2E * c.inv_t;
    p.inv_t = c.inv_t;
    p.pick = c.pick;
    p.K = c.pick ? c.K : 0;
    p.picked = c.picked;
    p.states = c.states;
    p.slots = slots;
    // worth its memory traffic (and a launch that clears it) from about four tiles a pair on: with 6 of them 800 rows
    // of 2,048 over 30,000 ids take 84 us and 85 without, with 2 of them 300 rows of 256 over 20,000 40 and 38
    if (KT > 0 && p.num_mt > 1 && units >= 4 * slots) {
        p.reached = c.reached;
        if (cudaMemsetAsync(c.reached, 0, 4 * (size_t)c.rows * REACHED, s) != cudaSuccess) return WF_ERR_CUDA;
    }
    p.ctrl = c.ctrl;
    p.timeout_ns = wait_timeout_ns();
    CUtensorMap ta, tb, tbs, tz;
    if (!make_tile_map(&ta, c.act, c.rows, c.d, c.d, false, BK, a_rows) ||
        !make_tile_map(&tb, c.W, c.V, c.d, c.d, false, BK, p.bn / split))
        return WF_ERR_CUDA;
    tbs = tb;
    if (p.nbig < p.num_n && !make_tile_map(&tbs, c.W, c.V, c.d, c.d, false, BK, (p.bn - p.step) / split))
        return WF_ERR_CUDA;
    tz = ta;
    if (Z && !make_tile_map(&tz, c.z, c.rows, c.V, c.ldz, true, 32, 32)) return WF_ERR_CUDA;
    *slots_out = slots;
    const dim3 grid(pair ? 2 * slots : slots);
    auto kernel = pair ? sweep_kernel<KT, ENT, Z, true> : sweep_kernel<KT, ENT, Z, false>;
    return c.after_lists ? launch_cluster(kernel, grid, dim3(SWEEP_THREADS), smem, s, split, ta, tb, tbs, tz, p)
                         : launch_plain(kernel, grid, dim3(SWEEP_THREADS), smem, s, split, ta, tb, tbs, tz, p);
}

}  // namespace

wf_status launch_sweep(const SweepCall& c, int* slots, cudaStream_t s) {
    if (c.z) return launch_kt<0, false, true>(c, slots, s);
    if (!c.entropy) return launch_kt<0, false, false>(c, slots, s);
    if (c.k == 0) return launch_kt<0, true, false>(c, slots, s);
    if (c.k <= 10) return launch_kt<10, true, false>(c, slots, s);
    return launch_kt<16, true, false>(c, slots, s);
}

static PFN_cuTensorMapEncodeTiled_v12000 tile_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }();
    return fn;
}

bool make_tile_map(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, uint64_t stride, bool fp32,
                   uint32_t box_cols, uint32_t box_rows) {
    auto enc = tile_encoder();
    if (!enc) return false;
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {stride * (fp32 ? 4 : 2)};
    cuuint32_t box[2] = {box_cols, box_rows};
    cuuint32_t estr[2] = {1, 1};
    return enc(map, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
               const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int resident_pairs(const void* kernel, int threads, int smem) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * 64);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        n = num_sms() / 2;
    }
    return n < REC_PAIRS ? n : REC_PAIRS;
}

}  // namespace wf
