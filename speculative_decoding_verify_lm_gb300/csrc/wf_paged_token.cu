// Attention of one new token per sequence over a paged key-value cache.
//
//   s_t = scale <q, K_t>,  o = sum_t e^(s_t - m) V_t / sum_t e^(s_t - m)
//
// in one pass over the cache with a running maximum m (base 2) and sum.  Every
// byte of the cache is read once: memory bandwidth bounds it, for one short
// sequence the chain of launch, lookups, copies and the join of the pieces.
//
// The work is the flat sequence of tiles of positions of every (sequence, KV
// head, 8 or 16 query heads); each CTA takes an equal stretch of it, wherever that
// begins and ends, so batches of very different lengths fill the GPU evenly.
// Pieces of an item that several CTAs share are left in the workspace and
// joined in order by the last of them to finish: the result does not depend on
// timing.
//
// A CTA is one copying warp and four computing warps.  The copying warp looks
// up the pages one tile ahead and gathers rows with 16-byte asynchronous
// copies into a ring of stages; the ring runs on across the items' borders, so
// that two CTAs an SM keep 128 KB in flight.  Rows lie on a power-of-two pitch
// with their 16-byte pieces exchanged by the row number: the fragment loads
// meet no bank conflicts.  Each computing warp takes a quarter of a tile's
// positions and keeps its own maximum, sum and outputs; they meet at the
// piece's end.
//
// The products are taken transposed, S^T = K Q^T and O^T = V^T P^T: positions
// and dims fill the matrix instruction's 16 rows and 8 query heads its columns,
// so a group of up to 8 heads wastes at most half of the work (with the heads
// as rows it would be a multiple of that, in registers and exponentials too).
// P^T reaches the second product by an 8 x 8 transpose between the lanes.  The
// running maximum may lag by a factor of 2^LAG: no lane exchanges a maximum
// unless one has outgrown it.
//
// What it reaches, in copy rates (6.8 TB/s): 91% on one sequence of 131,000
// positions (87 us), 94% on 64 of 100 to 16,384 (159 us), 85% on 128 of 2,000 to
// 6,000 over 8-bit (171 us), where the conversions and products fill the
// computing warps' issue slots.  One user at 2,048 positions: 11.0 us of latency.
#include "wf_paged.cuh"

#define PT_TRY(x)                      \
    do {                               \
        const wf_status _st = (x);     \
        if (_st != WF_OK) return _st;  \
    } while (0)

namespace wf {

constexpr int PT_CONSUMERS = 128;              // four computing warps
constexpr int PT_THREADS = PT_CONSUMERS + 32;  // and the copying one
constexpr int PT_JOIN = 16;                    // pieces of an item in flight together when they are joined
// Shortest stretch in tiles: the longest item in no more pieces than are joined
// together, up to 3 tiles (longer ones cost more than a second turn of joining).
// One sequence over 8 heads of 128, stretches of 1, 2, 3, 4 tiles, us:
//   bf16  300 positions 7.9 10.7 11.8 12.7,  1,250: 9.9 9.7 12.1 11.8,  2,048: 11.6 12.3 11.0 13.3,
//         4,000: 12.8 12.8 12.3 14.3;  over one head 8.7 9.6 10.6 11.8, 11.4 10.0 11.0 12.3,
//         13.4 11.9 11.2 12.4, 15.8 12.4 13.0 12.8
//   8-bit 300 positions 8.5 11.9 8.7 14.3,  2,048: 10.1 12.3 13.6 14.5,  4,000: 11.6 11.0 14.4 13.3;
//         over one head 9.4 10.4 9.2 9.2, 12.1 10.8 11.7 12.8, 12.6 11.0 12.0 13.0
// Over 96 such batches (64 to 128 wide, 4 to 16 heads a group, 300 to 5,000
// positions) this takes 1.04 of the best stretch's time, 3 tiles always 1.18, 1 always 1.07.
constexpr int PT_MIN_TILES = 3;

struct TokenParams {
    const uint16_t* q;
    int64_t q_stride;
    const int32_t* pos_off;
    const int32_t* cache_len;
    const int32_t* table;
    const uint8_t* K;        // this layer's rows
    const uint8_t* V;
    const float* k_scale;    // this layer's [G] scales, or null
    const float* v_scale;
    uint16_t* out;
    float* lse;
    float* part;             // [CTA][2][16][D] unnormalised outputs
    float2* stat;            // [CTA][2][16] (maximum, sum)
    uint32_t* cnt;           // [CTA] arrivals of the item that begins in it, zero at rest
    float qk;                // scale * log2(e)
    int P, H, G, D, hq, mt, B, page_shift, num_pages, max_pages;
    Control* ctrl;
    uint64_t timeout_ns;
};

struct TokenSeq {
    int row, T, nt;   // its row, positions, tiles of positions (0: no row)
    bool bad;
};

template <int KT>
__device__ __forceinline__ TokenSeq token_seq(const TokenParams& p, int b) {
    TokenSeq w;
    w.row = p.pos_off[b];
    const int r1 = p.pos_off[b + 1], len = p.cache_len[b];
    w.T = w.nt = 0;
    w.bad = false;
    if (w.row < 0 || r1 > p.P || r1 <= w.row) {   // no row (or offsets that name no rows)
        w.bad = w.row < 0 || r1 > p.P || r1 < w.row;
        return w;
    }
    w.bad = len < 0 || r1 - w.row > 1 || (int64_t)len + 1 > ((int64_t)p.max_pages << p.page_shift);
    w.T = w.bad ? 0 : len + 1;
    w.nt = w.bad ? 1 : (w.T + KT - 1) / KT;   // a bad sequence: one tile that writes NaN
    return w;
}

// A place in the flat sequence of tiles: sequence, KV head, tile of query heads, tile of positions.
struct TokenCursor {
    TokenSeq w;
    int b, g, m, kt;
};

template <int KT>
__device__ __forceinline__ void token_next_item(const TokenParams& p, TokenCursor& c) {
    c.kt = 0;
    if (++c.m < p.mt) return;
    c.m = 0;
    if (++c.g < p.G) return;
    c.g = 0;
    do {
        if (++c.b >= p.B) return;
        c.w = token_seq<KT>(p, c.b);
    } while (c.w.nt == 0);
}

// 16-byte piece c of row r in rows of PITCH bytes
template <int PITCH>
__device__ __forceinline__ uint32_t token_piece(int r, int c) {
    constexpr int N = PITCH / 16;
    const int x = N >= 8 ? (r & 7) : ((r >> 1) & (N - 1));
    return (uint32_t)(r * PITCH + ((c ^ x) << 4));
}

__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, %0;" ::"n"(PT_CONSUMERS) : "memory"); }
// One arrival on `bar` when every asynchronous copy this thread has issued is complete.
__device__ __forceinline__ void cp_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Counts an arrival: what the CTA wrote before its last barrier is visible to
// whoever counts later, and what others wrote before theirs to this CTA's
// threads behind its next barrier.
__device__ __forceinline__ uint32_t arrive_acq_rel(uint32_t* cnt) {
    uint32_t old;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(old) : "l"(cnt) : "memory");
    return old;
}
// b16 8 x 8 transpose between the lanes of a warp
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// DP: head size rounded up; E4M3: the cache's type; NH: tiles of 8 query heads.
template <int DP, bool E4M3, int NH>
struct TokenShape {
    static constexpr int KT = E4M3 && NH == 1 ? 128 : 64;   // positions of a tile
    static constexpr int PITCH = (DP <= 64 ? 64 : 128) * (E4M3 ? 1 : 2);
    static constexpr int KV_BYTES = KT * PITCH;
    static constexpr int HEADS = 8 * NH;
    static constexpr int Q_PITCH = DP <= 64 ? 128 : 256;
    static constexpr int STAGE = 2 * KV_BYTES + HEADS * Q_PITCH;
    // 16 wide heads take more registers than two CTAs have: one, with their ring
    static constexpr int PER_SM = DP > 64 && NH == 2 ? 1 : 2;
    static constexpr int STAGES = PER_SM == 2 ? 3 : 6;
    static constexpr int SMEM = 128 + STAGES * STAGE;
    static_assert(2 * HEADS * DP * 4 <= STAGE, "two warps' outputs fit a stage");
};

template <int DP, bool E4M3, int NH>
__global__ void __launch_bounds__(PT_THREADS, TokenShape<DP, E4M3, NH>::PER_SM) paged_token_kernel(const TokenParams p) {
    using S = TokenShape<DP, E4M3, NH>;
    constexpr int KT = S::KT, PITCH = S::PITCH, HEADS = S::HEADS;
    constexpr int NKS = DP / 16;               // 16-dim steps
    constexpr int NB = KT / 64;                // blocks of 16 positions of a warp
    constexpr int EB = E4M3 ? 1 : 2;
    constexpr float PBIAS = E4M3 ? 8.f : 0.f;  // fp16 probabilities use the range from 2^-24 up to 2^(8 + LAG)
    constexpr float LAG = 4.f;
    extern __shared__ uint8_t smem_dyn[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 127) & ~uintptr_t(127));
    __shared__ uint64_t s_full[S::STAGES], s_empty[S::STAGES];
    __shared__ float2 s_st[4][16];             // each warp's (maximum, sum)
    __shared__ int s_badpage[S::STAGES];       // the stage's tile has a position without a page
    __shared__ int64_t s_plan, s_scan[PT_THREADS / 32];
    __shared__ int s_longest[PT_THREADS / 32];
    __shared__ int s_pb, s_last;
    __shared__ int s_abort_word;
    volatile int* abort_flag = &s_abort_word;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < S::STAGES; ++i) {
            mbar_init(&s_full[i], 33);
            mbar_init(&s_empty[i], 4);
        }
        s_abort_word = 0;
        fence_barrier_init();
    }
    pdl_wait();
    pdl_trigger();

    // ------------------------------------------------ this CTA's stretch
    // each thread sums a run of sequences; then the run that holds the first tile is walked
    const int run = (p.B + PT_THREADS - 1) / PT_THREADS;
    const int items = p.G * p.mt;
    int64_t mine = 0;
    int longest = 0;   // tiles of an item
    for (int i = 0; i < run; ++i) {
        const int b = tid * run + i;
        if (b < p.B) {
            const TokenSeq w = token_seq<KT>(p, b);
            mine += (int64_t)items * w.nt;
            longest = max(longest, w.nt);
            if (w.bad && blockIdx.x == 0) record_error(p.ctrl, WF_ERR_BAD_DATA, (uint32_t)b);
        }
    }
    int64_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 31) s_scan[warp] = inc, s_longest[warp] = longest;
    __syncthreads();
    int64_t total = 0, before = inc - mine;
#pragma unroll
    for (int w = 0; w < PT_THREADS / 32; ++w) {
        if (w < warp) before += s_scan[w];
        total += s_scan[w];
        longest = max(longest, s_longest[w]);
    }
    int64_t per = pg_quotient(total + gridDim.x - 1, gridDim.x);
    const int least = min((longest + PT_JOIN - 1) / PT_JOIN, PT_MIN_TILES);
    if (per < least) per = least;
    const int64_t begin = (int64_t)blockIdx.x * per;
    const int64_t end = begin + per < total ? begin + per : total;
    if (begin >= end) return;
    if (mine > 0 && before <= begin && begin < before + mine) {
        int64_t at = before;
        int b = tid * run;
        for (;; ++b) {
            const int64_t n = (int64_t)items * token_seq<KT>(p, b).nt;
            if (begin < at + n) break;
            at += n;
        }
        s_plan = begin - at;
        s_pb = b;
    }
    __syncthreads();
    const int count = (int)(end - begin);
    TokenCursor c;
    c.b = s_pb;
    c.w = token_seq<KT>(p, c.b);
    {
        const int item = (int)pg_quotient(s_plan, c.w.nt);
        c.kt = (int)(s_plan - (int64_t)item * c.w.nt);
        c.g = item / p.mt;
        c.m = item - c.g * p.mt;
    }

    if (warp == 4) {
        // ------------------------------------------------ copies
        constexpr int CPR = PITCH / 16;        // lanes side by side on a row
        constexpr int RPI = 32 / CPR;          // rows a step covers
        const int piece = lane % CPR, crow = lane / CPR;
        const bool active = piece * 16 < p.D * EB;
        const int row_bytes = p.G * p.D * EB;
        int page[KT / 32], pos[KT / 32];   // pages of positions lane + 32 i of the next tile
        auto look_up = [&]() {
#pragma unroll
            for (int i = 0; i < KT / 32; ++i) {
                pos[i] = c.kt * KT + lane + 32 * i;
                page[i] = 0;
                if (pos[i] < c.w.T) page[i] = p.table[(int64_t)c.b * p.max_pages + (pos[i] >> p.page_shift)];
                else pos[i] = -1;
            }
        };
        look_up();
        for (int n = 0; n < count; ++n) {
            const int stage = n % S::STAGES;
            bool bad = false;
            int row[KT / 32];  // pool rows, -1 reads as zeros
#pragma unroll
            for (int i = 0; i < KT / 32; ++i) {
                const bool ok = pos[i] >= 0 && page[i] >= 0 && page[i] < p.num_pages;
                bad |= pos[i] >= 0 && !ok;
                row[i] = ok ? (page[i] << p.page_shift) + (pos[i] & ((1 << p.page_shift) - 1)) : -1;
            }
            const bool with_q = n == 0 || c.kt == 0;
            const int g = c.g, h0 = c.g * p.hq + c.m * HEADS, heads = min(HEADS, p.hq - c.m * HEADS), qrow = c.w.row;
            if (n + 1 < count) {
                if (++c.kt == c.w.nt) token_next_item<KT>(p, c);
                look_up();
            }
            // the lanes give up together: the others would wait for those that left
            if (!__all_sync(0xffffffffu, n < S::STAGES || mbar_wait(&s_empty[stage], ((n / S::STAGES) & 1) ^ 1,
                                                                    p.timeout_ns, abort_flag))) {
                *abort_flag = 1;
                if (lane == 0) record_error(p.ctrl, WF_ERR_TIMEOUT, 0x700u);
                break;
            }
            const uint32_t sk = smem_u32(smem + stage * S::STAGE), sv = sk + S::KV_BYTES;
            const uint8_t* kb = p.K + (int64_t)g * p.D * EB + piece * 16;
            const uint8_t* vb = p.V + (int64_t)g * p.D * EB + piece * 16;
#pragma unroll
            for (int part = 0; part < KT / 32; ++part)
#pragma unroll 8
                for (int i = 0; i < 32 / RPI; ++i) {
                    const int r = i * RPI + crow;   // of these 32
                    const int src = __shfl_sync(0xffffffffu, row[part], r);
                    const uint32_t bytes = src < 0 ? 0u : 16u;
                    const int64_t at = (int64_t)max(src, 0) * row_bytes;
                    const uint32_t to = token_piece<PITCH>(part * 32 + r, piece);
                    if (active) {
                        pg_cp16(sk + to, kb + at, bytes);
                        pg_cp16(sv + to, vb + at, bytes);
                    }
                }
            if (with_q) {
                const uint32_t sq = sv + S::KV_BYTES;
                const int per_row = p.D / 8;
                const uint16_t* q = p.q + (int64_t)qrow * p.q_stride + (int64_t)h0 * p.D;
                for (int i = lane; i < HEADS * per_row; i += 32) {
                    const int h = i / per_row, x = i - h * per_row;
                    const bool ok = h < heads;
                    pg_cp16(sq + token_piece<S::Q_PITCH>(h, x), q + (ok ? i * 8 : 0), ok ? 16u : 0u);
                }
            }
            bad = __any_sync(0xffffffffu, bad);
            if (lane == 0) {
                s_badpage[stage] = bad;
                mbar_arrive(&s_full[stage]);
            }
            cp_arrive(&s_full[stage]);
        }
        pg_cp_wait<0>();
        return;
    }

    // ---------------------------------------------------- computing warps
    const int gq = lane >> 2, cq = lane & 3;
    const int mi = lane >> 3, r8 = lane & 7;
    const int k0 = warp * (KT / 4);
    uint32_t qb[NH][NKS][2];   // Q^T
    float o[NH][NKS][4];       // O^T: 16 dims x 8 heads a tile
    int left = count;
    int n = 0;   // the stretch's tile number
    while (left > 0) {
        // -------------------------------------------- one piece: tiles [c.kt, c.kt + tiles) of an item
        const int tiles = min(left, c.w.nt - c.kt);
        const int kt_first = c.kt;
        bool bad = c.w.bad;
        // of heads 2 cq, 2 cq + 1 of each tile: running maximum of the scores as
        // they are, this lane's share of the sum, the scores' factor
        float m[NH][2], l[NH][2], f[NH][2];
        // Exponents are taken relative to the maximum's rounded product with f: its
        // rounding is one factor for the whole row.  A product past PG_FAR rounds
        // by too much for that (keys of the type's lowest value); there the
        // maximum is taken off the scores themselves.
        float base[NH][2];
        bool far = false;
#pragma unroll
        for (int h = 0; h < NH; ++h) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                m[h][u] = -INFINITY;
                l[h][u] = 0.f;
                f[h][u] = p.qk;
                base[h][u] = PBIAS;   // no score above -inf yet: weights of 0
            }
#pragma unroll
            for (int i = 0; i < NKS; ++i) o[h][i][0] = o[h][i][1] = o[h][i][2] = o[h][i][3] = 0.f;
        }
        for (int i = 0; i < tiles; ++i, ++n) {
            const int stage = n % S::STAGES;
            if (!mbar_wait(&s_full[stage], (n / S::STAGES) & 1, p.timeout_ns, abort_flag)) {
                *abort_flag = 1;
                if (lane == 0) record_error(p.ctrl, WF_ERR_TIMEOUT, 0x710u);
            }
            const uint8_t* st = smem + stage * S::STAGE;
            const uint32_t sk = smem_u32(st), sv = sk + S::KV_BYTES, sq = sv + S::KV_BYTES;
            if (i == 0) {
#pragma unroll
                for (int h = 0; h < NH; ++h) {
                    if (!E4M3) {
#pragma unroll
                        for (int k2 = 0; k2 < NKS / 2; ++k2) {
                            uint32_t x[4];
                            pg_ldsm_x4(x, sq + token_piece<S::Q_PITCH>(h * 8 + r8, k2 * 4 + mi));
                            qb[h][2 * k2][0] = x[0], qb[h][2 * k2][1] = x[1];
                            qb[h][2 * k2 + 1][0] = x[2], qb[h][2 * k2 + 1][1] = x[3];
                        }
                    } else {
                        // fp16 operands.  A position's four bytes cq * 4 .. + 3 of a 16-byte
                        // piece stand for the inner indices 2 cq, + 1, + 8, + 9, so the
                        // queries are taken in that order.  Each head is scaled by a power of
                        // two that puts its largest element in [1, 2), undone in fp32: exact down
                        // to 2^-14 of that, off by at most 2^-25 of the largest below (fp16's
                        // least step), the order of the fp32 sums' own rounding.
                        float big = 0.f;
                        auto lo = [](uint32_t w) { return pg_bf16_to_f32(w & 0xFFFFu); };
                        auto hi = [](uint32_t w) { return pg_bf16_to_f32(w >> 16); };
#pragma unroll
                        for (int ks = 0; ks < NKS; ++ks) {
                            uint2 x = make_uint2(0, 0);
                            if (ks * 16 < p.D)
                                x = *reinterpret_cast<const uint2*>(
                                    st + 2 * S::KV_BYTES + (cq & 1) * 8 +
                                    token_piece<S::Q_PITCH>(h * 8 + gq, ks * 2 + (cq >> 1)));
                            qb[h][ks][0] = x.x;
                            qb[h][ks][1] = x.y;
                            big = fmaxf(big, fmaxf(fmaxf(fabsf(lo(x.x)), fabsf(hi(x.x))),
                                                   fmaxf(fabsf(lo(x.y)), fabsf(hi(x.y)))));
                        }
#pragma unroll
                        for (int w = 1; w <= 2; w <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, w));
                        const int e = pg_scale_exponent(big);
                        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
                        for (int ks = 0; ks < NKS; ++ks)
#pragma unroll
                            for (int u = 0; u < 2; ++u)
                                qb[h][ks][u] = cvt_f16x2(lo(qb[h][ks][u]) * down, hi(qb[h][ks][u]) * down);
                        const float ksc = p.qk * (p.k_scale ? __ldg(p.k_scale + c.g) : 1.f);
                        const float mine_f = pg_factor(ksc, e);   // of head gq
#pragma unroll
                        for (int u = 0; u < 2; ++u) f[h][u] = __shfl_sync(0xffffffffu, mine_f, (2 * cq + u) * 4);
                    }
                }
            }
            bad |= s_badpage[stage] != 0;
            const int nvalid = c.w.T - (kt_first + i) * KT - k0;   // positions of this warp that exist
            if (nvalid > 0) {
                float sc[NB][NH][4];
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int h = 0; h < NH; ++h) sc[b][h][0] = sc[b][h][1] = sc[b][h][2] = sc[b][h][3] = 0.f;
                if (!E4M3) {
#pragma unroll
                    for (int ks = 0; ks < NKS; ++ks) {
                        if (ks * 16 >= p.D) continue;   // past the head size: whatever the stage held before
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            uint32_t ka[4];
                            pg_ldsm_x4(ka, sk + token_piece<PITCH>(k0 + b * 16 + (mi & 1) * 8 + r8, 2 * ks + (mi >> 1)));
#pragma unroll
                            for (int h = 0; h < NH; ++h) pg_mma_bf16(sc[b][h], ka, qb[h][ks][0], qb[h][ks][1]);
                        }
                    }
                } else {
#pragma unroll
                    for (int k2 = 0; k2 < NKS / 2; ++k2)   // two 16-byte pieces of 16 positions
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            uint32_t w[4];
                            pg_ldsm_x4(w, sk + token_piece<PITCH>(k0 + b * 16 + (mi & 1) * 8 + r8, 2 * k2 + (mi >> 1)));
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const int ks = 2 * k2 + u;
                                if (ks * 16 >= p.D) continue;
                                const uint32_t ka[4] = {e4m3x2_f16x2(w[2 * u]), e4m3x2_f16x2(w[2 * u + 1]),
                                                        e4m3x2_f16x2(w[2 * u] >> 16), e4m3x2_f16x2(w[2 * u + 1] >> 16)};
#pragma unroll
                                for (int h = 0; h < NH; ++h) pg_mma_f16(sc[b][h], ka, qb[h][ks][0], qb[h][ks][1]);
                            }
                        }
                }
                if (nvalid < 16 * NB) {
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int h = 0; h < NH; ++h) {
                            if (b * 16 + gq >= nvalid) sc[b][h][0] = sc[b][h][1] = -INFINITY;
                            if (b * 16 + gq + 8 >= nvalid) sc[b][h][2] = sc[b][h][3] = -INFINITY;
                        }
                }
                bool grown = false;
                float mx[NH][2];
#pragma unroll
                for (int h = 0; h < NH; ++h)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        float x = fmaxf(sc[0][h][u], sc[0][h][2 + u]);
#pragma unroll
                        for (int b = 1; b < NB; ++b) x = fmaxf(x, fmaxf(sc[b][h][u], sc[b][h][2 + u]));
                        mx[h][u] = x;
                        grown |= (x - m[h][u]) * (E4M3 ? f[h][u] : p.qk) > LAG;
                    }
                if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
                    for (int h = 0; h < NH; ++h)
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            float x = mx[h][u];
#pragma unroll
                            for (int w = 4; w <= 16; w <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, w));
                            x = fmaxf(x, m[h][u]);
                            const float a = m[h][u] == -INFINITY ? 0.f : ex2_approx((m[h][u] - x) * (E4M3 ? f[h][u] : p.qk));
                            m[h][u] = x;
                            l[h][u] *= a;
#pragma unroll
                            for (int t = 0; t < NKS; ++t) {
                                o[h][t][u] *= a;
                                o[h][t][2 + u] *= a;
                            }
                        }
                    far = false;
#pragma unroll
                    for (int h = 0; h < NH; ++h)
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            base[h][u] = PBIAS - (m[h][u] == -INFINITY ? 0.f : m[h][u] * (E4M3 ? f[h][u] : p.qk));
                            far |= fabsf(base[h][u]) > PG_FAR;
                        }
                    far = __any_sync(0xffffffffu, far);
                    if (far)
#pragma unroll
                        for (int h = 0; h < NH; ++h) base[h][0] = base[h][1] = PBIAS;
                }
                if (far) {
#pragma unroll
                    for (int h = 0; h < NH; ++h)
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int b = 0; b < NB; ++b) {
                                sc[b][h][u] -= m[h][u] == -INFINITY ? 0.f : m[h][u];
                                sc[b][h][2 + u] -= m[h][u] == -INFINITY ? 0.f : m[h][u];
                            }
                }
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    // P^T of 16 positions.  Over bf16 a weight is the sum of two bf16 numbers,
                    // less than 2^-14 of it off: the outputs' error against 64 bits is that of
                    // their own rounding, 0.0017 (one number, 2^-8: 0.0022 to 0.0024, and 1 to 4%
                    // sooner: 64 ragged sequences 157.4 us against 159.2, 16 heads a group over
                    // 4 x 64 50.3 against 52.1).  The first is taken a little below the weight, so
                    // that the second is above zero where the weight is: an infinite value times
                    // either is the same infinity.  fp16 (8-bit caches) leaves 2^-11 in one number.
                    constexpr float DOWN = 1.f - 0x1p-9f;
                    uint32_t pb[NH][2], pl[NH][2];
#pragma unroll
                    for (int h = 0; h < NH; ++h)
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const float p0 = ex2_approx(fmaf(sc[b][h][2 * u], E4M3 ? f[h][0] : p.qk, base[h][0]));
                            const float p1 = ex2_approx(fmaf(sc[b][h][2 * u + 1], E4M3 ? f[h][1] : p.qk, base[h][1]));
                            l[h][0] += p0;
                            l[h][1] += p1;
                            const uint32_t w = E4M3 ? cvt_f16x2(p0, p1) : cvt_bf16x2_down(p0 * DOWN, p1 * DOWN);
                            pb[h][u] = transpose8(w);
                            if (!E4M3)
                                pl[h][u] = transpose8(cvt_bf16x2(p0 - pg_bf16_to_f32(w & 0xFFFFu),
                                                                 p1 - __uint_as_float(w & 0xFFFF0000u)));
                        }
                    if (!E4M3) {
#pragma unroll
                        for (int t = 0; t < NKS; ++t) {
                            uint32_t va[4];   // V^T: dims x positions
                            pg_ldsm_x4_trans(va, sv + token_piece<PITCH>(k0 + b * 16 + (mi >> 1) * 8 + r8, 2 * t + (mi & 1)));
#pragma unroll
                            for (int h = 0; h < NH; ++h) {
                                pg_mma_bf16(o[h][t], va, pl[h][0], pl[h][1]);
                                pg_mma_bf16(o[h][t], va, pb[h][0], pb[h][1]);
                            }
                        }
                    } else {
#pragma unroll
                        for (int t2 = 0; t2 < NKS / 2; ++t2) {
                            // 16 positions x two 16-byte pieces: a word holds dims 2 gq, + 1 of
                            // positions 2 cq, + 1; even dims become rows gq, odd ones rows gq + 8
                            uint32_t w[4];
                            pg_ldsm_x4_trans(w, sv + token_piece<PITCH>(k0 + b * 16 + (mi & 1) * 8 + r8, 2 * t2 + (mi >> 1)));
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const uint32_t x0 = e4m3x2_f16x2(w[2 * u]), x1 = e4m3x2_f16x2(w[2 * u] >> 16);
                                const uint32_t y0 = e4m3x2_f16x2(w[2 * u + 1]), y1 = e4m3x2_f16x2(w[2 * u + 1] >> 16);
                                const uint32_t va[4] = {__byte_perm(x0, x1, 0x5410), __byte_perm(x0, x1, 0x7632),
                                                        __byte_perm(y0, y1, 0x5410), __byte_perm(y0, y1, 0x7632)};
#pragma unroll
                                for (int h = 0; h < NH; ++h) pg_mma_f16(o[h][2 * t2 + u], va, pb[h][0], pb[h][1]);
                            }
                        }
                    }
                }
            }
            if (i + 1 < tiles) {   // the piece's last stage is kept for its result
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_empty[stage]);
            }
        }
        // -------------------------------------------- the piece's result
        const int stage = (n - 1) % S::STAGES;
        float* red = reinterpret_cast<float*>(smem + stage * S::STAGE);   // [2][HEADS][DP]
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
                for (int w = 4; w <= 16; w <<= 1) l[h][u] += __shfl_xor_sync(0xffffffffu, l[h][u], w);
                m[h][u] *= E4M3 ? f[h][u] : p.qk;
                if (gq == 0) s_st[warp][h * 8 + 2 * cq + u] = make_float2(m[h][u], l[h][u]);
            }
        consumer_sync();   // also: every warp is done with this stage's keys and values
        auto put = [&](int slot, bool add) {
            float* x = red + slot * HEADS * DP;
#pragma unroll
            for (int h = 0; h < NH; ++h)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int head = h * 8 + 2 * cq + u;
                    float M = -INFINITY;
#pragma unroll
                    for (int w = 0; w < 4; ++w) M = fmaxf(M, s_st[w][head].x);
                    const float wt = m[h][u] == -INFINITY ? 0.f : ex2_approx(m[h][u] - M);
#pragma unroll
                    for (int t = 0; t < NKS; ++t)
#pragma unroll
                        for (int v = 0; v < 2; ++v) {
                            const int d = t * 16 + (E4M3 ? 2 * gq + v : gq + 8 * v);
                            const float a = o[h][t][2 * v + u] * wt;
                            x[head * DP + d] = add ? x[head * DP + d] + a : a;
                        }
                }
        };
        if (warp < 2) put(warp, false);
        consumer_sync();
        if (warp >= 2) put(warp - 2, true);
        consumer_sync();
        const int heads = min(HEADS, p.hq - c.m * HEADS);
        const int64_t pair0 = (int64_t)c.w.row * p.H + c.g * p.hq + c.m * HEADS;
        const float vs = E4M3 && p.v_scale ? __ldg(p.v_scale + c.g) : 1.f;
        const int half = p.D / 2;
        auto row_stat = [&](int h) {   // maximum and sum over the four warps
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w) M = fmaxf(M, s_st[w][h].x);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float2 x = s_st[w][h];
                L += x.y * (x.x == -INFINITY ? 0.f : ex2_approx(x.x - M));   // a NaN sum stays one
            }
            return bad ? make_float2(NAN, NAN) : make_float2(M, L);
        };
        auto value = [&](int h, int d) {   // two neighbouring dims, summed over the warps
            const float2 a = *reinterpret_cast<const float2*>(red + h * DP + d);
            const float2 e = *reinterpret_cast<const float2*>(red + (HEADS + h) * DP + d);
            return make_float2(a.x + e.x, a.y + e.y);
        };
        auto write = [&](int h, int d, float2 v, float2 st) {
            const float inv = vs / st.y;
            *reinterpret_cast<uint32_t*>(p.out + (pair0 + h) * p.D + d) = cvt_bf16x2(v.x * inv, v.y * inv);
            if (p.lse && d == 0) p.lse[pair0 + h] = (st.x + __log2f(st.y) - PBIAS) * LN2;
        };
        if (bad && tid == 0) record_error(p.ctrl, WF_ERR_BAD_DATA, (uint32_t)c.b);
        if (tiles == c.w.nt) {
            for (int i = tid; i < heads * half; i += PT_CONSUMERS) {
                const int h = i / half, d = (i - h * half) * 2;
                write(h, d, value(h, d), row_stat(h));
            }
            if (c.w.bad)   // all of its rows are NaN, not the first alone
                for (int64_t row = c.w.row + 1, r1 = p.pos_off[c.b + 1]; row < r1; ++row)
                    for (int i = tid; i < heads * half; i += PT_CONSUMERS) {
                        const int64_t at = row * p.H + c.g * p.hq + c.m * HEADS + i / half;
                        *reinterpret_cast<uint32_t*>(p.out + at * p.D + (i % half) * 2) = cvt_bf16x2(NAN, NAN);
                        if (p.lse && i % half == 0) p.lse[at] = NAN;
                    }
        } else {
            // a shared item: this piece to the workspace, joined by the last piece to arrive
            const int slot = (int)blockIdx.x * 2 + (kt_first == 0 ? 1 : 0);
            for (int i = tid; i < heads * half; i += PT_CONSUMERS) {
                const int h = i / half, d = (i - h * half) * 2;
                *reinterpret_cast<float2*>(p.part + ((int64_t)slot * 16 + h) * p.D + d) = value(h, d);
            }
            if (tid < heads) p.stat[slot * 16 + tid] = row_stat(tid);
            const int64_t ts = begin + (count - left) - kt_first;   // the item's first tile in the flat sequence
            const int c0 = (int)pg_quotient(ts, per), pieces = (int)pg_quotient(ts + c.w.nt - 1, per) - c0 + 1;
            consumer_sync();
            if (tid == 0) s_last = arrive_acq_rel(p.cnt + c0) == (uint32_t)(pieces - 1);
            consumer_sync();
            if (s_last) {
                // piece k is CTA c0 + k's: its second slot for the item's first, else its
                // first.  A thread takes four dims of a head; sixteen pieces' statistics
                // and outputs are in flight together and added in order.
                constexpr int BATCH = PT_JOIN;
                const int quarter = p.D / 4;
                for (int i = tid; i < heads * quarter; i += PT_CONSUMERS) {
                    const int h = i / quarter, d = (i - h * quarter) * 4;
                    float M = -INFINITY, L = 0.f;
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int q0 = 0; q0 < pieces; q0 += BATCH) {
                        float2 s2[BATCH];
                        float4 x[BATCH];
#pragma unroll
                        for (int k = 0; k < BATCH; ++k) {
                            const int at = ((c0 + q0 + k) * 2 + (q0 + k == 0)) * 16 + h;
                            const bool in = q0 + k < pieces;
                            s2[k] = in ? __ldcg(&p.stat[at]) : make_float2(-INFINITY, 0.f);
                            x[k] = in ? __ldcg(reinterpret_cast<const float4*>(p.part + (int64_t)at * p.D + d))
                                      : make_float4(0.f, 0.f, 0.f, 0.f);
                        }
                        float top = M;
#pragma unroll
                        for (int k = 0; k < BATCH; ++k) top = fmaxf(top, s2[k].x);
                        const float a = M == -INFINITY ? 0.f : ex2_approx(M - top);
                        M = top;
                        L *= a;
                        v = make_float4(v.x * a, v.y * a, v.z * a, v.w * a);
#pragma unroll
                        for (int k = 0; k < BATCH; ++k) {
                            const float w = s2[k].x == -INFINITY ? 0.f : ex2_approx(s2[k].x - top);
                            L = fmaf(s2[k].y, w, L);
                            v.x = fmaf(x[k].x, w, v.x);
                            v.y = fmaf(x[k].y, w, v.y);
                            v.z = fmaf(x[k].z, w, v.z);
                            v.w = fmaf(x[k].w, w, v.w);
                        }
                    }
                    write(h, d, make_float2(v.x, v.y), make_float2(M, L));
                    write(h, d + 2, make_float2(v.z, v.w), make_float2(M, L));
                }
                if (tid == 0) p.cnt[c0] = 0;
            }
        }
        consumer_sync();   // the stage is read to its end
        if (lane == 0) mbar_arrive(&s_empty[stage]);
        left -= tiles;
        if (left > 0) {
            c.kt += tiles;
            if (c.kt == c.w.nt) token_next_item<KT>(p, c);
        }
    }
}

// ------------------------------------------------------------------ host side
using TokenFn = void (*)(TokenParams);

struct TokenVariant {
    TokenFn fn;
    int smem, kt;
};

template <int DP, bool E4M3, int NH>
static TokenVariant token_variant_of() {
    return {paged_token_kernel<DP, E4M3, NH>, TokenShape<DP, E4M3, NH>::SMEM, TokenShape<DP, E4M3, NH>::KT};
}

// bit 0: an 8-bit cache; bit 1: items of 16 query heads; bit 2: heads wider than 64
constexpr int TOKEN_VARIANTS = 7;
static TokenVariant token_variant(int i) {
    switch (i) {
        case 0: return token_variant_of<64, false, 1>();
        case 1: return token_variant_of<64, true, 1>();
        case 2: return token_variant_of<64, false, 2>();
        case 3: return token_variant_of<64, true, 2>();
        case 4: return token_variant_of<128, false, 1>();
        case 5: return token_variant_of<128, true, 1>();
        default: return token_variant_of<128, false, 2>();
    }
}

wf_status launch_paged_token(const wf_paged_cache* c, const wf_paged_attn_args* a, void* ws, cudaStream_t s) {
    static std::mutex mu;
    static bool attr_set[64] = {false};
    static int ctas[64][TOKEN_VARIANTS];   // CTAs an SM holds
    const bool e4m3 = c->kv_type == WF_KV_E4M3;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return WF_ERR_CUDA;
    PT_TRY(configure_once(mu, attr_set, [dev] {
        for (int i = 0; i < TOKEN_VARIANTS; ++i) {
            const TokenVariant v = token_variant(i);
            if (cudaFuncSetAttribute(v.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, v.smem) != cudaSuccess ||
                cudaFuncSetAttribute(v.fn, cudaFuncAttributePreferredSharedMemoryCarveout, 100) != cudaSuccess ||
                cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ctas[dev][i], v.fn, PT_THREADS, v.smem) != cudaSuccess)
                return false;
        }
        return true;
    }));
    uint8_t* w = static_cast<uint8_t*>(ws);
    const PagedLayout L = paged_layout(c->D, a->max_rows);
    const int64_t esize = e4m3 ? 1 : 2;
    const int64_t layer_bytes = (int64_t)c->num_pages * c->page_size * c->G * c->D * esize;
    TokenParams p = {};
    p.q = a->q;
    p.q_stride = a->q_stride;
    p.pos_off = a->pos_off;
    p.cache_len = a->cache_len;
    p.table = c->table;
    p.K = static_cast<const uint8_t*>(c->K) + a->layer * layer_bytes;
    p.V = static_cast<const uint8_t*>(c->V) + a->layer * layer_bytes;
    p.k_scale = c->k_scale ? c->k_scale + (int64_t)a->layer * c->G : nullptr;
    p.v_scale = c->v_scale ? c->v_scale + (int64_t)a->layer * c->G : nullptr;
    p.out = a->out;
    p.lse = a->lse;
    p.part = reinterpret_cast<float*>(w + L.part);
    p.stat = reinterpret_cast<float2*>(w + L.stat);
    p.cnt = reinterpret_cast<uint32_t*>(w + L.cnt);
    p.qk = a->scale * LOG2E;
    p.P = a->P;
    p.H = a->H;
    p.G = c->G;
    p.D = c->D;
    p.hq = a->H / c->G;
    // Groups of more than 8 heads: items of 16 read the cache half as often (64
    // sequences, 16 heads a group over 4 x 64: 61 us against 95 bf16, 52 against 62
    // 8-bit; over 4 x 128 bf16 152 against 155).  Wide heads over an 8-bit cache are
    // bound by instructions, and items of 8 let an SM hold two CTAs: 103 against 120.
    const bool sixteen = p.hq > 8 && !(e4m3 && c->D > 64);
    p.mt = cdiv(p.hq, sixteen ? 16 : 8);
    p.B = c->B;
    while ((1 << p.page_shift) < c->page_size) ++p.page_shift;
    p.num_pages = c->num_pages;
    p.max_pages = c->max_pages;
    p.ctrl = static_cast<Control*>(ws);
    p.timeout_ns = wait_timeout_ns();
    const int vi = (e4m3 ? 1 : 0) | (sixteen ? 2 : 0) | (c->D > 64 ? 4 : 0);
    const TokenVariant v = token_variant(vi);
    int grid = num_sms() * (ctas[dev][vi] > 0 ? ctas[dev][vi] : 1);
    if (grid > PA_MAX_CTAS) grid = PA_MAX_CTAS;
    // no more CTAs than tiles that the lengths' bound allows
    const int64_t tiles = (int64_t)c->B * c->G * p.mt * cdiv((int64_t)c->max_pages * c->page_size, v.kt);
    if (tiles < grid) grid = (int)tiles;
    return launch(v.fn, dim3(grid), dim3(PT_THREADS), (size_t)v.smem, s, p);
}

}  // namespace wf
