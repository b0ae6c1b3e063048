// The gradients of the draft head's distillation loss.  With z the kept logits
// (over the temperature), q = softmax(z) and p the teacher's distribution,
//   G[n, v] = gs_n (q[n, v] - p[n, v]),   gs_n = gloss_n / T (0 for a row without a teacher)
//   dx[n, :] = sum_v G[n, v] Wd[v, :],    dWd[v, :] = sum_n G[n, v] x[n, :]
// Two launches: G in bf16 (one pass over z), then both products as the tiles of
// one persistent launch on the tensor cores.
//
// G is rounded to bf16 (both products need operands of one type, and Wd and x
// are bf16); the products sum in fp32 and are rounded to bf16 once more on their
// way out.  A gradient is then off by 1.4 times what its own rounding makes; the
// few entries that the teacher lists hold nearly all of G, so with few rows it
// can as well be 1.7 times.  Up to TWO_PART_ROWS rows, where the weights' bytes
// bound both products, G goes in as the sum of two bf16 numbers, of which nothing
// is seen in the result (64 rows over 32,000 ids: error 0.0025 -> 0.0017).
#include "wf_heads.cuh"

namespace wf {

namespace {

constexpr int TWO_PART_ROWS = BM;

// ------------------------------------------------------------------ G
// Bound by the bytes of z (fp32, read) and G (bf16, written).  A thread takes 8
// neighbouring ids at a time, GRAD_UNROLL such loads in flight; meanwhile the
// first warp works out the row's teacher, and behind a barrier puts the few ids
// that it lists right, from z.  64 rows over 32,000 ids 7 us, 1,024 rows 39 us
// (197 MB at 5.0 TB/s, G's 66 MB staying in L2).
constexpr int GRAD_THREADS = 256;
constexpr int GRAD_UNROLL = 4;
constexpr int GRAD_COLS = GRAD_THREADS * 8 * GRAD_UNROLL;

struct GradParams {
    const float* z;
    int64_t ldz;
    const float* lse;
    const float* gloss;   // [N] or null: 1
    Teacher t;
    uint16_t* G;
    int64_t ldg;
    int64_t lo;      // elements from G's first part to its second, 0 = one part
    int chunks;      // CTAs of a row
    int turns;       // times GRAD_COLS ids that a CTA takes
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// What bf16 leaves of a number.
__device__ __forceinline__ float bf16_rest(float v) {
    return v - __uint_as_float(pack_bf16(v, 0.f) << 16);
}

__global__ void __launch_bounds__(GRAD_THREADS) logit_grad_kernel(const GradParams a) {
    __shared__ float row_gs;
    pdl_trigger();   // the products may start
    const int n = blockIdx.x / a.chunks, v0 = (blockIdx.x % a.chunks) * a.turns * GRAD_COLS;
    const int Vd = a.t.Vd, v1 = v0 + min(Vd - v0, a.turns * GRAD_COLS), lane = threadIdx.x & 31;
    const float off = a.lse[n];
    const float* z = a.z + (size_t)n * a.ldz;
    uint16_t* G = a.G + (size_t)n * a.ldg;
    TeacherRow r;
    float gs = 0.f;
    for (int base = v0; base < v1; base += GRAD_COLS) {
        float4 f[GRAD_UNROLL][2];
#pragma unroll
        for (int u = 0; u < GRAD_UNROLL; ++u) {
            const int v = base + (u * GRAD_THREADS + (int)threadIdx.x) * 8;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                f[u][h] = v + 4 * h < Vd ? __ldcs(reinterpret_cast<const float4*>(z + v) + h)
                                         : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        if (base == v0) {
            if (threadIdx.x < 32) {
                r = teacher_row(a.t, n, lane);
                if (lane == 0) row_gs = r.some ? (a.gloss ? a.gloss[n] : 1.f) * a.t.inv_t : 0.f;
            }
            __syncthreads();
            gs = row_gs;
        }
#pragma unroll
        for (int u = 0; u < GRAD_UNROLL; ++u) {
            const int v = base + (u * GRAD_THREADS + (int)threadIdx.x) * 8;
            if (v >= Vd) continue;
            // ids from Vd on get 0: tensor copies look at a row's end in steps of 16 bytes
            auto q = [&](float x, int j) {
                return gs == 0.f || v + j >= Vd ? 0.f : gs * ex2_approx((x - off) * LOG2E);
            };
            const float g[8] = {q(f[u][0].x, 0), q(f[u][0].y, 1), q(f[u][0].z, 2), q(f[u][0].w, 3),
                                q(f[u][1].x, 4), q(f[u][1].y, 5), q(f[u][1].z, 6), q(f[u][1].w, 7)};
            uint4 o;
            o.x = pack_bf16(g[0], g[1]);
            o.y = pack_bf16(g[2], g[3]);
            o.z = pack_bf16(g[4], g[5]);
            o.w = pack_bf16(g[6], g[7]);
            *reinterpret_cast<uint4*>(G + v) = o;
            if (a.lo) {
                o.x = pack_bf16(bf16_rest(g[0]), bf16_rest(g[1]));
                o.y = pack_bf16(bf16_rest(g[2]), bf16_rest(g[3]));
                o.z = pack_bf16(bf16_rest(g[4]), bf16_rest(g[5]));
                o.w = pack_bf16(bf16_rest(g[6]), bf16_rest(g[7]));
                *reinterpret_cast<uint4*>(G + a.lo + v) = o;
            }
        }
    }
    if (gs == 0.f) return;   // the same for the whole CTA
    __syncthreads();
    if (threadIdx.x < 32) {
        // the first place that names an id takes the probability of all that do
        float pt[2] = {0.f, 0.f};
        bool again[2] = {false, false};
        for (int j = 0; j < a.t.K; ++j) {
            const int id = __shfl_sync(0xffffffffu, j < 32 ? r.id[0] : r.id[1], j & 31);
            const float p = __shfl_sync(0xffffffffu, j < 32 ? r.p[0] : r.p[1], j & 31);
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (id == r.id[h]) {
                    pt[h] += p;
                    again[h] |= j < lane + 32 * h;
                }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int id = r.id[h];
            if (lane + 32 * h < a.t.K && !again[h] && id >= v0 && id < v1) {
                const float g = gs * (ex2_approx((z[id] - off) * LOG2E) - pt[h]);
                G[id] = (uint16_t)pack_bf16(g, 0.f);
                if (a.lo) G[a.lo + id] = (uint16_t)pack_bf16(bf16_rest(g), 0.f);
            }
        }
    }
}

// ------------------------------------------------------------------ dx and dWd
// Tiles of 256 x 256 outputs by CTA pairs.  A tile of dx runs over Vd (G as it
// lies, Wd with its contiguous dimension as the product's N), a tile of dWd over
// the rows (G and x, both with their contiguous dimensions as M and N).  dx has
// few and long tiles, dWd many and short ones: every pair first takes its share
// of dx, the pairs with fewer of them begin dWd sooner, and all end together.
// With too few rows for that dx is cut along Vd as well; its fp32 parts are
// added up in order by a kernel of their own.
// Measured over 32,000 ids of 2,560: 4,096 rows 653 us (2.05 PFLOP/s before the
// power cap), 1,024 rows 184 us with the tensor pipe active for 87 % of the
// cycles, 64 rows 59 us: Wd's bytes once, dWd's once (5.5 TB/s).
// Up to 128 rows dx is computed as its transpose, Wd^T G^T: Wd's 256 columns are
// the product's M and the rows its N, so that a K block costs what its rows need
// and not 256 of them, and the tile is bound by Wd's bytes.
constexpr int TM = 256, TN = 256;
constexpr int OUT_BOX = 4096;               // 32 rows x 128 bytes on their way out
// Eight epilogue warps, two on each 32 rows: a tile on its way out is a chain of
// short steps (accumulator, rounding, shared memory, copy), 4,900 cycles for one
// warp, where a short dWd tile (few rows) could leave in 2,800.
constexpr int PROD_WARPS = 8, PROD_THREADS = pipe_threads(PROD_WARPS);
constexpr int PROD_STAGES = 6;
constexpr int PROD_STAGE = 2 * BM * BK * 2;
constexpr int PROD_SMEM = pipe_smem(PROD_STAGES, PROD_STAGE, PROD_WARPS * OUT_BOX);
static_assert(PROD_SMEM + PIPE_STATIC_MAX <= PIPE_SMEM_MAX, "a CTA's shared memory");
static_assert(pipe_alone(PROD_SMEM), "no SM holds CTAs of two pairs");
constexpr int SPREAD_ROWS = 64;             // rows up to which every pair gets a part of dx
// Pairs that the split is chosen for (152 SMs), also where fewer are resident: the order of dx's sums is the sizes' alone.
constexpr int PLAN_PAIRS = 76;
constexpr int MAX_SPLIT = 16;
constexpr int MAX_PARTS = 8 * PLAN_PAIRS;   // parts of all of dx's tiles: what a workspace holds

struct ProdParams {
    int N, Vd, d;
    int x_m, x_n, w_m;        // row tiles of dx, column tiles of both, row tiles of dWd
    int split, kb_x, kb_w;    // parts of dx's K; K blocks of a whole dx tile and of a dWd tile
    int x_units, w_units;
    int lead, late;           // pairs from `late` on have one dx unit less and begin dWd `lead` rounds sooner
    int part_rows;            // rows of one part of dx
    int flip;                 // dx is computed as its transpose, `flip` rows wide; 0: as it lies
    int w_rows;               // rows of one K block of dWd (a multiple of 16)
    int parts;                // G's parts, rows N apart (2: only with flip)
    uint16_t* dx;
    float* part;
    Control* ctrl;
    uint64_t timeout_ns;
};

struct Unit {
    bool dx;
    int row0, col0;     // of the output tile
    int k0, kb;         // first K block, K blocks
    int part;
};
// The units of one pair, in its order: its share of dx, then of dWd.  A dWd tile
// of few rows takes a microsecond, so the tiles' places are counted on from one
// another instead of divided out.
struct Units {
    int x_left, x_next, slot, slots;
    int lead_left, v, r, c, stride, dr, dc;
    __device__ __forceinline__ void place(const ProdParams& p, int v0, int step) {
        v = v0;
        stride = step;
        r = v0 / p.x_n;
        c = v0 - r * p.x_n;
        dr = step / p.x_n;
        dc = step - dr * p.x_n;
    }
    __device__ __forceinline__ Units(const ProdParams& p, int slot_, int slots_) : slot(slot_), slots(slots_) {
        x_left = p.x_units > slot ? (p.x_units - slot + slots - 1) / slots : 0;
        x_next = slot;
        lead_left = slot >= p.late ? p.lead : 0;
        if (lead_left)
            place(p, slot - p.late, slots - p.late);
        else
            place(p, p.lead * (slots - p.late) + slot, slots);
    }
    __device__ __forceinline__ bool next(const ProdParams& p, Unit& u) {
        if (x_left > 0) {
            const int tile = x_next / p.split, part = x_next - tile * p.split;
            u.dx = true;
            u.part = part;
            u.row0 = tile / p.x_n * TM;
            u.col0 = tile % p.x_n * TN;
            u.k0 = (int)((long)p.kb_x * part / p.split);
            u.kb = (int)((long)p.kb_x * (part + 1) / p.split) - u.k0;
            x_next += slots;
            --x_left;
            return true;
        }
        if (v >= p.w_units) return false;
        u.dx = false;
        u.part = 0;
        u.row0 = r * TM;
        u.col0 = c * TN;
        u.k0 = 0;
        u.kb = p.kb_w * p.parts;
        v += stride;
        r += dr;
        c += dc;
        if (c >= p.x_n) {
            c -= p.x_n;
            ++r;
        }
        // behind the units that the early pairs took by themselves, every pair takes its turn
        if (lead_left && --lead_left == 0) place(p, p.lead * (slots - p.late) + slot, slots);
        return true;
    }
};

// Descriptor of an operand whose contiguous dimension is the product's M or N:
// blocks of 64 values x 64 K rows (128-byte rows, 128-byte swizzle) 8,192 bytes
// apart, groups of 8 K rows 1,024 bytes apart.
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | (uint64_t)(8192 >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
constexpr uint32_t IDESC = umma_idesc_bf16(TM, TN);
constexpr uint32_t A_MN = 1u << 15, B_MN = 1u << 16;   // the operand's M / N dimension is the contiguous one

__global__ void __launch_bounds__(PROD_THREADS, 1)
    grad_products_kernel(const __grid_constant__ CUtensorMap tmGk, const __grid_constant__ CUtensorMap tmGm,
                         const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                         const __grid_constant__ CUtensorMap tmDx, const __grid_constant__ CUtensorMap tmDw,
                         const ProdParams p) {
    extern __shared__ uint8_t smem_raw[];
    const Pipe g = pipe_at(smem_raw, PROD_STAGES, PROD_STAGE, BM * BK * 2, PROD_WARPS * OUT_BOX, p.ctrl, p.timeout_ns);
    const int warp = warp_number(), lane = threadIdx.x & 31;
    const int rank = (int)(cluster_ctarank() & 1u);
    const bool first = rank == 0;
    const int slot = (int)(blockIdx.x >> 1), slots = (int)(gridDim.x >> 1);
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tmGk);
        tma_prefetch_desc(&tmGm);
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
        tma_prefetch_desc(&tmDx);
        tma_prefetch_desc(&tmDw);
    }
    const uint32_t tmem_base = pipe_begin<true, PROD_WARPS>(g);
    if (warp != 0) pdl_wait();   // warp 0: before it copies
    if (warp == 0) {
        const uint64_t pol = policy_evict_normal();
        Unit u{};
        Units units(p, slot, slots);
        auto next = [&](int) { return units.next(p, u) ? u.kb : 0; };
        auto tx = [&]() {
            if (u.dx)
                return p.flip ? (uint32_t)(2 * BM * BK * 2 + p.parts * p.flip * BK * 2) : (uint32_t)(2 * PROD_STAGE);
            return (uint32_t)(2 * 4 * 128 * p.w_rows);
        };
        // two boxes of A and two of B; where an operand lies with its K contiguous, it is one box
        auto load = [&](int kc, int s, uint32_t bar, bool, bool) {
            uint8_t *a = g.a(s), *b = g.b(s);
            const int col = u.col0 + rank * (TN / 2);
            if (!u.dx) {
                const bool lo = kc >= p.kb_w;   // G's first part, then its second
                const int k = (kc - (lo ? p.kb_w : 0)) * p.w_rows, row = u.row0 + rank * BM;
                pipe_load<true>(a, &tmGm, bar, row, k + (lo ? p.N : 0), pol);
                pipe_load<true>(a + 8192, &tmGm, bar, row + 64, k + (lo ? p.N : 0), pol);
                pipe_load<true>(b, &tmX, bar, col, k, pol);
                pipe_load<true>(b + 8192, &tmX, bar, col + 64, k, pol);
            } else if (p.flip) {
                const int k = (u.k0 + kc) * BK, row = rank * (p.flip / 2);
                pipe_load<true>(a, &tmW, bar, u.col0 + rank * BM, k, pol);
                pipe_load<true>(a + 8192, &tmW, bar, u.col0 + rank * BM + 64, k, pol);
                pipe_load<true>(b, &tmGk, bar, k, row, pol);
                if (p.parts == 2) pipe_load<true>(b + 8192, &tmGk, bar, k, row + p.N, pol);
            } else {
                const int k = (u.k0 + kc) * BK;
                pipe_load<true>(a, &tmGk, bar, k, u.row0 + rank * BM, pol);
                pipe_load<true>(b, &tmW, bar, col, k, pol);
                pipe_load<true>(b + 8192, &tmW, bar, col + 64, k, pol);
            }
        };
        pipe_copy<true, false>(g, first, next, tx, load);
    } else if (warp == 1) {
        if (first) {
            Unit u{};
            Units units(p, slot, slots);
            auto next = [&](int) { return units.next(p, u) ? u.kb : 0; };
            auto issue = [&](int s, uint32_t d, int kc) {
                const uint32_t as = smem_u32(g.a(s)), bs = smem_u32(g.b(s));
                const bool flip = u.dx && p.flip, a_rows = u.dx && !p.flip;
                const uint64_t a = a_rows ? umma_desc_sw128(as) : desc_mn(as);
                const uint64_t b = flip ? umma_desc_sw128(bs) : desc_mn(bs);
                // 16 values of K: 32 bytes of a row, or 16 rows of 128
                const uint32_t a_step = a_rows ? 2 : 128, b_step = flip ? 2 : 128;
                const uint32_t idesc = flip ? umma_idesc_bf16(TM, p.flip) | A_MN : IDESC | B_MN | (u.dx ? 0 : A_MN);
                if (flip && p.parts == 2) {   // both parts of G against the same weights
#pragma unroll
                    for (int kk = 0; kk < BK / 16; ++kk) {
                        umma_bf16_pair(d, a + a_step * kk, b + b_step * kk, idesc, (kc | kk) != 0);
                        umma_bf16_pair(d, a + a_step * kk, b + (8192 >> 4) + b_step * kk, idesc, 1);
                    }
                } else if (u.dx || p.w_rows == BK) {
#pragma unroll
                    for (int kk = 0; kk < BK / 16; ++kk)
                        umma_bf16_pair(d, a + a_step * kk, b + b_step * kk, idesc, (kc | kk) != 0);
                } else {
                    for (int kk = 0; kk < p.w_rows / 16; ++kk)
                        umma_bf16_pair(d, a + a_step * kk, b + b_step * kk, idesc, (kc | kk) != 0);
                }
            };
            pipe_mma<true>(g, tmem_base, next, issue);
        }
    } else {
        const int q = warp & 3, half = (warp - 2) >> 2;   // accumulator rows 32 q.., columns of this half
        const uint32_t tempty_first = first ? 0 : cluster_addr(&g.tempty[0], 0);
        uint8_t* stage = pipe_extra(g) + (warp - 2) * OUT_BOX;
        Unit u{};
        Units units(p, slot, slots);
        for (uint32_t i = 0; units.next(p, u); ++i) {
            if (!pipe_acc_wait(g, i)) break;
            const int row = u.row0 + rank * BM + q * 32;
            const bool part = u.dx && p.split > 1;
            const uint32_t tbase = tmem_base + ((uint32_t)(q * 32) << 16) + (i & 1) * BN;
            auto box_free = [&]() {   // the last store has read the box
                if (lane == 0) tma_store_wait_read<0>();
                __syncwarp();
            };
            auto box_out = [&](int col, int y) {
                fence_async_store();
                __syncwarp();
                if (lane == 0) tma_store_2d(u.dx ? &tmDx : &tmDw, stage, col, y);
                __syncwarp();
            };
            if (u.dx && p.flip) {
                // thread = one column of dx, accumulator columns = its rows: a warp's stores are whole lines
                const int c = u.col0 + rank * BM + q * 32 + lane;
                for (int n0 = 32 * half; n0 < p.N; n0 += 64) {
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(tbase + n0, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        if (n0 + j < p.N && c < p.d) {
                            if (part)
                                p.part[((size_t)u.part * p.part_rows + n0 + j) * p.d + c] = __uint_as_float(r[j]);
                            else
                                p.dx[(size_t)(n0 + j) * p.d + c] = (uint16_t)pack_bf16(__uint_as_float(r[j]), 0.f);
                        }
                    }
                }
                pipe_acc_release(g, i, tempty_first);
            } else if (part) {
                const int cols = min(TN / 2 * (half + 1), p.d - u.col0);
                for (int c0 = TN / 2 * half; row < p.N && c0 < cols; c0 += 32) {
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(tbase + c0, r);
                    tmem_ld_wait();
                    box_free();
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        *reinterpret_cast<uint4*>(stage + swizzled(lane, j)) =
                            make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
                    box_out(u.col0 + c0, u.part * p.part_rows + row);
                }
                pipe_acc_release(g, i, tempty_first);
            } else {
                // all of the warp's columns leave the accumulator, rounded, before any leaves the SM: the
                // next tile's products do not wait for the way out
                uint32_t o[TN / 4];
#pragma unroll
                for (int c = 0; c < TN / 2; c += 32) {
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(tbase + TN / 2 * half + c, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        o[c / 2 + j] = pack_bf16(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
                }
                pipe_acc_release(g, i, tempty_first);
                if (row < (u.dx ? p.N : p.Vd)) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int col = u.col0 + TN / 2 * half + 64 * h;
                        if (col >= p.d) break;
                        box_free();
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            *reinterpret_cast<uint4*>(stage + swizzled(lane, j)) = make_uint4(
                                o[32 * h + 4 * j], o[32 * h + 4 * j + 1], o[32 * h + 4 * j + 2], o[32 * h + 4 * j + 3]);
                        box_out(col, row);
                    }
                }
            }
        }
        if (lane == 0) tma_store_wait_all();
    }
    pipe_end<true>(g, tmem_base);
}

// dx from the parts of a split product, added in order.
__global__ void __launch_bounds__(256) dx_join_kernel(const float* part, int parts, int part_rows, int N, int d,
                                                      uint16_t* dx) {
    const long units = (long)N * (d / 8);
    for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < units; i += (long)gridDim.x * 256) {
        const int n = (int)(i / (d / 8)), c = (int)(i % (d / 8)) * 8;
        const float* at = part + (size_t)n * d + c;
        const size_t step = (size_t)part_rows * d;
        float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int j = 0; j < parts; ++j) {
            const float4 a = *reinterpret_cast<const float4*>(at + j * step);
            const float4 b = *reinterpret_cast<const float4*>(at + j * step + 4);
            s[0] += a.x;
            s[1] += a.y;
            s[2] += a.z;
            s[3] += a.w;
            s[4] += b.x;
            s[5] += b.y;
            s[6] += b.z;
            s[7] += b.w;
        }
        uint4 o;
        o.x = pack_bf16(s[0], s[1]);
        o.y = pack_bf16(s[2], s[3]);
        o.z = pack_bf16(s[4], s[5]);
        o.w = pack_bf16(s[6], s[7]);
        *reinterpret_cast<uint4*>(dx + (size_t)n * d + c) = o;
    }
}

// ------------------------------------------------------------------ the plan
// Costs in K blocks of a pair (64 of K, 256 x 256 outputs: 0.33 us at the bf16
// rate).  A dWd tile writes 128 KB, a part of dx 256 KB, at the copy rate of
// one pair (90 GB/s).
constexpr double W_TILE_OUT = 4.4, X_PART_OUT = 9.0, TILE_FIXED = 1.0;

struct Plan {
    int x_m, x_n, w_m, kb_x, kb_w, split, part_rows, flip, w_rows, parts;
};
double w_cost(int kb_w) { return (kb_w > W_TILE_OUT ? kb_w : W_TILE_OUT) + TILE_FIXED; }

Plan plan_of(int N, int d, int Vd, bool dx, bool dw) {
    Plan p{};
    p.x_m = cdiv(N, TM);
    p.x_n = cdiv(d, TN);
    p.w_m = cdiv(Vd, TM);
    p.kb_x = cdiv(Vd, BK);
    // equal K blocks of dWd: rows that are not there cost a tensor copy more than
    // others (one row in boxes of 64: 35 us without stores, 64 rows: 24)
    p.kb_w = cdiv(N, BK);
    p.w_rows = cdiv(cdiv(N, p.kb_w), 16) * 16;
    p.split = 1;
    p.flip = N <= BM ? (N + 31) / 32 * 32 : 0;
    p.part_rows = p.flip ? N : p.x_m * TM;
    p.parts = N <= TWO_PART_ROWS ? 2 : 1;
    if (dx && p.x_m * p.x_n <= PLAN_PAIRS && N <= SPREAD_ROWS) {
        // few rows: both products are bound by the weights' bytes, and dx's half of them comes soonest with a part
        // for every pair, where the costs below would take fewer (us, a part for every pair / by the costs):
        //   d 4,096 over 32,000 ids   16 rows 95.0 / 101.6,  64 rows 101.9 / 106.6,  80 rows 111.9 / 110.4
        //   d 2,560 over 32,000 ids   16 rows 66.7 / 67.3,   64 rows 72.8 / 71.8,    80 rows 80.3 / 75.3
        //   d 1,024 over 10,007 ids   16 rows 20.8 / 19.2,   64 rows 21.9 / 19.8 (16 parts of few K blocks)
        p.split = PLAN_PAIRS / p.x_n;
        if (p.split > MAX_SPLIT) p.split = MAX_SPLIT;
        if (p.split > p.kb_x) p.split = p.kb_x;
    } else if (dx) {
        const double w = dw ? (double)p.w_m * p.x_n * w_cost(p.kb_w * p.parts) : 0.0;
        double best = -1;
        for (int s = 1; s <= MAX_SPLIT && s <= p.kb_x && (s == 1 || (long)s * p.x_m * p.x_n <= MAX_PARTS); ++s) {
            const double unit = (double)p.kb_x / s + (s > 1 ? X_PART_OUT : TILE_FIXED);
            const double units = (double)p.x_m * p.x_n * s;
            const double longest = unit * cdiv((long)units, PLAN_PAIRS), mean = (units * unit + w) / PLAN_PAIRS;
            // a split costs another launch and its bytes: about 8 K blocks
            const double cost = (longest > mean ? longest : mean) + (s > 1 ? 8.0 : 0.0);
            if (best < 0 || cost < best) {
                best = cost;
                p.split = s;
            }
        }
    }
    return p;
}

}  // namespace

size_t distill_grad_ldg(int Vd) { return align_up((size_t)Vd, 64); }
// Rows of G's buffer: two parts, and what the transposed product's boxes reach to; no fewer for more rows.
static int grad_rows(int N) {
    const int two = 2 * (((N < TWO_PART_ROWS ? N : TWO_PART_ROWS) + 31) / 32 * 32);
    return N > two ? N : two;
}
size_t distill_grad_bytes(int N, int Vd) { return 2 * (size_t)grad_rows(N) * distill_grad_ldg(Vd); }
// The most blocks or tiles that a call counts.
long distill_grad_units(int N, int d, int Vd) {
    const long g = (long)N * cdiv(Vd, GRAD_COLS), x = (long)cdiv(N, TM) * cdiv(d, TN) * MAX_SPLIT,
               w = (long)cdiv(Vd, TM) * cdiv(d, TN) * 2;
    return g > x ? (g > w ? g : w) : (x > w ? x : w);
}
// Bytes of dx's parts: no fewer for more rows, so that a workspace for the most rows serves fewer.
size_t distill_part_bytes(int N, int d, int Vd) {
    const long most = (long)MAX_SPLIT * cdiv(N, TM) * cdiv(d, TN);
    return (size_t)(most < MAX_PARTS ? most : MAX_PARTS) * TM * TN * 4;
}

// G and part: scratch.
wf_status launch_distill_grad(const uint16_t* x, const uint16_t* Wd, int d, const Teacher& t, const float* z,
                              int64_t ldz, const float* lse, const float* gloss, uint16_t* dx, uint16_t* dWd,
                              uint16_t* G, float* part, cudaStream_t s) {
    const int N = t.N, Vd = t.Vd;
    GradParams a{};
    a.z = z;
    a.ldz = ldz;
    a.lse = lse;
    a.gloss = gloss;
    a.t = t;
    a.G = G;
    a.ldg = (int64_t)distill_grad_ldg(Vd);
    a.lo = N <= TWO_PART_ROWS ? N * a.ldg : 0;
    // a row's teacher is worked out by each of its CTAs: as few as leave eight for an SM (a CTA for each GRAD_COLS ids
    // takes as long with few rows, and with 64 listed 1,500 rows' gradients over 32,000 ids of 256 130 us in place of 115)
    const int pieces = cdiv(Vd, GRAD_COLS);
    const long most = (long)N * pieces / (8 * num_sms());
    a.turns = most < 1 ? 1 : most < pieces ? (int)most : pieces;
    a.chunks = cdiv(pieces, a.turns);
    static std::mutex mu;
    static bool attr_set[64] = {false};
    static int pairs[64];
    wf_status st = configure_once(mu, attr_set, [] {
        if (!set_smem(grad_products_kernel, PROD_SMEM) || !set_smem(logit_grad_kernel, 0) || !set_smem(dx_join_kernel, 0))
            return false;
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return false;
        if (dev < 64)
            pairs[dev] = resident_pairs(reinterpret_cast<const void*>(grad_products_kernel), PROD_THREADS, PROD_SMEM);
        return true;
    });
    if (st != WF_OK) return st;
    st = launch_plain(logit_grad_kernel, dim3((unsigned)N * a.chunks), dim3(GRAD_THREADS), 0, s, 1u, a);
    if (st != WF_OK) return st;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return WF_ERR_CUDA;
    int slots = dev < 64 ? pairs[dev] : num_sms() / 2;
    const Plan pl = plan_of(N, d, Vd, dx != nullptr, dWd != nullptr);
    ProdParams p{};
    p.N = N;
    p.Vd = Vd;
    p.d = d;
    p.x_m = pl.x_m;
    p.x_n = pl.x_n;
    p.w_m = pl.w_m;
    p.split = pl.split;
    p.kb_x = pl.kb_x;
    p.kb_w = pl.kb_w;
    p.x_units = dx ? pl.x_m * pl.x_n * pl.split : 0;
    p.w_units = dWd ? pl.w_m * pl.x_n : 0;
    p.part_rows = pl.part_rows;
    p.flip = pl.flip;
    p.w_rows = pl.w_rows;
    p.parts = pl.parts;
    p.dx = dx;
    p.part = part;
    if (slots > p.x_units + p.w_units) slots = p.x_units + p.w_units;
    // pairs 0 .. late - 1 have one dx unit more than the others
    p.late = p.x_units % slots;
    const double ux = (double)pl.kb_x / pl.split + (pl.split > 1 ? X_PART_OUT : TILE_FIXED);
    p.lead = p.late ? (int)(ux / w_cost(pl.kb_w * pl.parts) + 0.5) : 0;
    p.ctrl = t.ctrl;
    p.timeout_ns = wait_timeout_ns();
    CUtensorMap gk, gm, tw, tx, tdx, tdw;
    const int g_rows = N * pl.parts;
    // The transposed product may read any rows behind the last (they are columns that nobody keeps), and a box
    // of rows that are not there takes longer (one row: dx 53 us).
    if (!make_tile_map(&gk, G, pl.flip ? N + pl.flip : g_rows, Vd, a.ldg, false, BK, pl.flip ? pl.flip / 2 : BM) ||
        !make_tile_map(&gm, G, g_rows, Vd, a.ldg, false, 64, pl.w_rows) ||
        !make_tile_map(&tw, Wd, Vd, d, d, false, 64, BK) || !make_tile_map(&tx, x, N, d, d, false, 64, pl.w_rows))
        return WF_ERR_CUDA;
    tdx = tdw = gk;
    const bool parts = pl.split > 1;
    if (dx && !pl.flip && !(parts ? make_tile_map(&tdx, part, (uint64_t)pl.split * pl.part_rows, d, d, true, 32, 32)
                      : make_tile_map(&tdx, dx, N, d, d, false, 64, 32)))
        return WF_ERR_CUDA;
    if (dWd && !make_tile_map(&tdw, dWd, Vd, d, d, false, 64, 32)) return WF_ERR_CUDA;
    st = launch_cluster(grad_products_kernel, dim3(2 * slots), dim3(PROD_THREADS), PROD_SMEM, s, 2u, gk, gm, tw, tx, tdx,
                        tdw, p);
    if (st != WF_OK || !dx || !parts) return st;
    const long units = (long)N * (d / 8);
    const int blocks = (int)(cdiv(units, 256) < 8 * num_sms() ? cdiv(units, 256) : 8 * num_sms());
    return launch_plain(dx_join_kernel, dim3(blocks), dim3(256), 0, s, 1u, (const float*)part, pl.split, pl.part_rows, N,
                        d, dx);
}

}  // namespace wf
