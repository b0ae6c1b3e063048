// Attention over a paged key-value cache, small tiles: 16 (row, head) pairs of
// one KV head at a time, so a single new token's whole group of query heads.
//
//   s_t = scale <q, K_t>,  o = sum_t e^(s_t - m) V_t / sum_t e^(s_t - m)
//
// in one pass over the cache with a running maximum m (base 2) and sum.  Every
// byte of the cache is read once and used for 16 rows: memory bandwidth bounds
// it.  The work is the flat sequence of 64-position tiles of every (sequence,
// tile of pairs, KV head); each CTA takes an equal stretch of it, wherever that
// begins and ends, so batches of very different lengths fill the GPU evenly.
// Pieces of an item that several CTAs share are left in the workspace and
// joined in order by the last of them to finish.
//
// A tile's keys and values stream through a ring of stages (16-byte
// asynchronous copies, rows scattered over pages; the ring runs on across the
// items' borders) into rows of a power-of-two pitch whose 16-byte pieces are
// exchanged by the row number, so that the fragment loads meet no bank
// conflicts.  Four warps take 16 positions each; per piece their results are
// added in shared memory.
#include "wf_paged.cuh"

#define PA_TRY(x)                      \
    do {                               \
        const wf_status _st = (x);     \
        if (_st != WF_OK) return _st;  \
    } while (0)

namespace wf {

constexpr int PA_THREADS = 128;
constexpr int PA_KT = 64;              // positions of a tile
constexpr int PA_WARP_KEYS = 16;

struct PagedAttnParams {
    const uint16_t* q;
    int64_t q_stride;
    const int32_t* pos_off;
    const int32_t* cache_len;
    const int32_t* node_off;
    const int32_t* kind;
    const int32_t* parent;
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
    int P, H, G, D, hq, B, page_shift, num_pages, max_pages, max_rows, min_tiles;
    Control* ctrl;
};

// One sequence's part of the work.
struct SeqWork {
    int r0, rows, len, T, mt, nt;   // first row, rows, cached positions, all positions, tiles of pairs, tiles of positions
    bool bad;
};

__device__ __forceinline__ SeqWork seq_work(const PagedAttnParams& p, int b) {
    SeqWork w;
    w.r0 = p.pos_off[b];
    const int r1 = p.pos_off[b + 1];
    w.len = p.cache_len[b];
    w.rows = r1 - w.r0;
    w.T = 0;
    w.mt = w.nt = 0;
    w.bad = false;
    if (w.r0 < 0 || r1 > p.P || r1 <= w.r0) {   // no row of its own (or offsets that name no rows)
        w.bad = w.r0 < 0 || r1 > p.P || r1 < w.r0;
        w.rows = 0;
        return w;
    }
    const int64_t T = (int64_t)w.len + w.rows;
    w.bad = w.len < 0 || w.rows > p.max_rows || T > ((int64_t)p.max_pages << p.page_shift);
    w.mt = (w.rows * p.hq + PA_TILE_M - 1) / PA_TILE_M;
    w.T = w.bad ? 0 : (int)T;
    w.nt = w.bad ? 1 : (w.T + PA_KT - 1) / PA_KT;   // a bad sequence: one tile that writes NaN
    return w;
}

// A place in the flat sequence of tiles.
struct Cursor {
    SeqWork w;
    int b, item, kt;     // sequence, (tile of pairs, KV head) of it, tile of positions
    int left;            // tiles of this CTA's stretch from here on
};

__device__ __forceinline__ void cursor_next(const PagedAttnParams& p, Cursor& c) {
    --c.left;
    if (++c.kt < c.w.nt) return;
    c.kt = 0;
    if (++c.item < c.w.mt * p.G) return;
    c.item = 0;
    do {
        ++c.b;
        if (c.b >= p.B) {
            c.left = 0;
            return;
        }
        c.w = seq_work(p, c.b);
    } while (c.w.mt == 0);
}

// Bits of the positions [t0, t0 + 64) that row r of a sequence sees.  par: its
// parents (the tree's nodes are rows 1 ..), null for a chain.
__device__ __forceinline__ uint64_t visible64(int r, int len, int t0, const int16_t* par) {
    const int upto = par ? len - t0 : len + r + 1 - t0;   // all positions below are seen
    uint64_t m = upto <= 0 ? 0ull : (upto >= 64 ? ~0ull : (1ull << upto) - 1);
    if (par) {
        int j = r;
        while (true) {
            const int t = len + j - t0;
            if (t >= 0 && t < 64) m |= 1ull << t;
            if (j == 0) break;
            j = 1 + par[j - 1];
        }
    }
    return m;
}

// 16-byte piece c of row r in rows of PITCH bytes
template <int PITCH>
__device__ __forceinline__ uint32_t piece_at(int r, int c) {
    constexpr int N = PITCH / 16;
    const int x = N >= 8 ? (r & 7) : ((r >> 1) & (N - 1));
    return (uint32_t)(r * PITCH + ((c ^ x) << 4));
}

// DP: head size rounded up (a multiple of 32); E4M3: the cache's type.
template <int DP, bool E4M3>
struct PaShape {
    static constexpr int PITCH = (DP <= 64 ? 64 : 128) * (E4M3 ? 1 : 2);
    static constexpr int KV_BYTES = PA_KT * PITCH;
    static constexpr int Q_PITCH = DP * 2 + 16;
    static constexpr int Q_BYTES = PA_TILE_M * Q_PITCH;
    static constexpr int STAGE = (2 * KV_BYTES + Q_BYTES + 127) / 128 * 128;
    static constexpr int STAGES = E4M3 ? 4 : 3;
    static constexpr int RED = 2 * PA_TILE_M * DP * 4;   // two warps' outputs, in a consumed stage
    static_assert(RED <= 2 * KV_BYTES, "the warps' outputs fit a stage");
    static constexpr int SMEM = 128 + STAGES * STAGE;
};

template <int DP, bool E4M3>
__global__ void __launch_bounds__(PA_THREADS) paged_attend_kernel(const PagedAttnParams p) {
    using S = PaShape<DP, E4M3>;
    constexpr int PITCH = S::PITCH;
    constexpr int PRE = S::STAGES - 1;
    constexpr int CPR = PITCH / 16;            // pieces of a row: threads side by side
    constexpr int RPI = PA_THREADS / CPR;      // rows a copy step covers
    constexpr int NKS = DP / 16;
    constexpr int EB = E4M3 ? 1 : 2;
    constexpr float PBIAS = E4M3 ? 8.f : 0.f;  // fp16 probabilities use the range up to 2^8
    extern __shared__ uint8_t smem_dyn[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 127) & ~uintptr_t(127));
    __shared__ int64_t s_off[2][PA_KT];        // element offset of each position's row, -1 reads as zero
    __shared__ uint64_t s_vis[PA_TILE_M];
    __shared__ int16_t s_par[WF_MAX_SEQ_NODES];
    __shared__ float2 s_st[4][PA_TILE_M];      // each warp's (maximum, sum)
    __shared__ int64_t s_plan, s_scan[4];
    __shared__ int s_pb, s_last;
    __shared__ int s_badpage[8];   // [n % 8] = n: tile n has a position without a page
    __shared__ int s_badtree;      // last tile at which a malformed tree was met
    __shared__ int s_odd;          // last tile with a value that is not finite under a mask

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gq = lane >> 2, cq = lane & 3;
    pdl_wait();
    pdl_trigger();

    // ------------------------------------------------ this CTA's stretch
    // each thread sums a run of sequences; then the run that holds the first tile is walked
    const int run = (p.B + PA_THREADS - 1) / PA_THREADS;
    int64_t mine = 0;
    for (int i = 0; i < run; ++i) {
        const int b = tid * run + i;
        if (b < p.B) {
            const SeqWork w = seq_work(p, b);
            mine += (int64_t)w.mt * p.G * w.nt;
            if (w.bad && blockIdx.x == 0) record_error(p.ctrl, WF_ERR_BAD_DATA, (uint32_t)b);
        }
    }
    int64_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) s_scan[warp] = inc;
    __syncthreads();
    int64_t total = 0, before = inc - mine;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        if (w < warp) before += s_scan[w];
        total += s_scan[w];
    }
    int64_t per = (total + gridDim.x - 1) / gridDim.x;
    if (per < p.min_tiles) per = p.min_tiles;
    const int64_t begin = (int64_t)blockIdx.x * per;
    const int64_t end = begin + per < total ? begin + per : total;
    if (begin >= end) return;
    if (mine > 0 && before <= begin && begin < before + mine) {
        int64_t at = before;
        int b = tid * run;
        for (;; ++b) {
            const SeqWork w = seq_work(p, b);
            const int64_t n = (int64_t)w.mt * p.G * w.nt;
            if (begin < at + n) break;
            at += n;
        }
        s_plan = begin - at;
        s_pb = b;
    }
    if (tid < 8) s_badpage[tid] = -1;
    if (tid == 0) s_badtree = s_odd = -1;
    __syncthreads();
    Cursor cc;   // the tile being computed
    cc.b = s_pb;
    cc.w = seq_work(p, cc.b);
    cc.item = (int)(s_plan / cc.w.nt);
    cc.kt = (int)(s_plan - (int64_t)cc.item * cc.w.nt);
    cc.left = (int)(end - begin);
    Cursor pc = cc;   // the tile whose rows are looked up

    // ------------------------------------------------ copies
    // Thread t < 64 finds the row of position t of tile n (cursor pc); its offset
    // goes to s_off[n & 1] one barrier before the copies are issued.
    const int cpiece = tid % CPR, crow = tid / CPR;
    const bool cactive = cpiece * 16 < p.D * EB;
    // The page number is loaded before a tile is computed and used after it.
    int up_page = 0, up_t = -1, up_g = 0;
    auto look_up = [&]() {
        up_t = -1;
        if (pc.left > 0) {
            const int t = pc.kt * PA_KT + tid;
            if (tid < PA_KT && !pc.w.bad && t < pc.w.T) {
                up_t = t;
                up_g = pc.item % p.G;
                up_page = p.table[(int64_t)pc.b * p.max_pages + (t >> p.page_shift)];
            }
            cursor_next(p, pc);
        }
    };
    auto put_off = [&](int n) {
        int64_t off = -1;
        if (up_t >= 0) {
            if (up_page < 0 || up_page >= p.num_pages) {
                s_badpage[n & 7] = n;
            } else {
                const int64_t row = ((int64_t)up_page << p.page_shift) + (up_t & ((1 << p.page_shift) - 1));
                off = (row * p.G + up_g) * p.D;
            }
        }
        if (tid < PA_KT) s_off[n & 1][tid] = off;
    };
    // Copies of tile n (cursor ic); positions past the end are written as zeros.
    // A stretch's first tile and every item's first tile bring the pairs' queries.
    Cursor ic = cc;
    auto issue = [&](int n) {
        if (ic.left > 0) {
            const uint32_t sk = smem_u32(smem + n % S::STAGES * S::STAGE), sv = sk + S::KV_BYTES;
            if (cactive) {
#pragma unroll
                for (int i = 0; i < PA_KT / RPI; ++i) {
                    const int r = crow + i * RPI;
                    const int64_t off = s_off[n & 1][r];
                    const uint32_t bytes = off < 0 ? 0u : 16u;
                    const int64_t at = (off < 0 ? 0 : off) * EB + cpiece * 16;
                    pg_cp16(sk + piece_at<PITCH>(r, cpiece), p.K + at, bytes);
                    pg_cp16(sv + piece_at<PITCH>(r, cpiece), p.V + at, bytes);
                }
            }
            if (ic.kt == 0 || n == 0) {
                const uint32_t sq = sv + S::KV_BYTES;
                const int g = ic.item % p.G, m0 = ic.item / p.G * PA_TILE_M;
                const int per_row = p.D / 8;
                for (int i = tid; i < PA_TILE_M * per_row; i += PA_THREADS) {
                    const int m = i / per_row, x = i - m * per_row;
                    const int r = (m0 + m) / p.hq, h = (m0 + m) - r * p.hq;
                    const bool ok = r < ic.w.rows;
                    const uint16_t* src =
                        p.q + (int64_t)(ic.w.r0 + (ok ? r : 0)) * p.q_stride + (g * p.hq + h) * p.D + x * 8;
                    pg_cp16(sq + m * S::Q_PITCH + x * 16, src, ok ? 16u : 0u);
                }
            }
            cursor_next(p, ic);
        }
        pg_cp_commit();
    };
    for (int n = 0; n < PRE; ++n) {
        look_up();
        put_off(n);
        __syncthreads();
        issue(n);
    }
    look_up();
    put_off(PRE);

    // ------------------------------------------------ compute
    uint32_t qa[NKS][4];
    float o[2 * NKS][4];
    float m_lo = -INFINITY, m_hi = -INFINITY, l_lo = 0.f, l_hi = 0.f;
    float f_lo = p.qk, f_hi = p.qk;   // factors of the two rows' scores
    int first = -1, kt_first = 0;   // first tile of the current piece: its number, its place in the item
    bool bad = false, tree = false;
    for (int n = 0; cc.left > 0; ++n) {
        pg_cp_wait<PRE - 1>();
        __syncthreads();   // tile n has landed; its predecessor is consumed; the next offsets are there
        issue(n + PRE);
        look_up();

        const int stage = n % S::STAGES;
        const uint8_t* st = smem + stage * S::STAGE;
        const uint32_t sk = smem_u32(st), sv = sk + S::KV_BYTES, sq = sv + S::KV_BYTES;
        const int g = cc.item % p.G, m0 = cc.item / p.G * PA_TILE_M;
        if (first < 0) {
            first = n;
            kt_first = cc.kt;
            bad = cc.w.bad;
            m_lo = m_hi = -INFINITY;
            l_lo = l_hi = 0.f;
#pragma unroll
            for (int i = 0; i < 2 * NKS; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
            f_lo = f_hi = p.qk;
            if (!E4M3) {
#pragma unroll
                for (int ks = 0; ks < NKS; ++ks) {
                    const int mi = lane >> 3, r = lane & 7;
                    pg_ldsm_x4(qa[ks], sq + ((mi & 1) * 8 + r) * S::Q_PITCH + ks * 32 + (mi >> 1) * 16);
                }
            } else {
                // fp16 operands.  A position's four bytes cq * 4 .. + 3 of a 16-byte
                // piece stand for the inner indices 2 cq, + 1, + 8, + 9, so the
                // queries are taken in that order.  Each row is scaled by a power of
                // two that puts its largest element in [1, 2): exact, and undone in fp32.
                float lo[NKS][4], hi[NKS][4], a_lo = 0.f, a_hi = 0.f;
#pragma unroll
                for (int ks = 0; ks < NKS; ++ks) {
                    const uint16_t* x = reinterpret_cast<const uint16_t*>(st + 2 * S::KV_BYTES + gq * S::Q_PITCH) +
                                        ks * 16 + cq * 4;
                    const bool in = ks * 16 < p.D;
                    const uint2 u = in ? *reinterpret_cast<const uint2*>(x) : make_uint2(0, 0);
                    const uint2 v = in ? *reinterpret_cast<const uint2*>(x + 8 * (S::Q_PITCH / 2)) : make_uint2(0, 0);
                    lo[ks][0] = pg_bf16_to_f32(u.x & 0xFFFFu), lo[ks][1] = pg_bf16_to_f32(u.x >> 16);
                    lo[ks][2] = pg_bf16_to_f32(u.y & 0xFFFFu), lo[ks][3] = pg_bf16_to_f32(u.y >> 16);
                    hi[ks][0] = pg_bf16_to_f32(v.x & 0xFFFFu), hi[ks][1] = pg_bf16_to_f32(v.x >> 16);
                    hi[ks][2] = pg_bf16_to_f32(v.y & 0xFFFFu), hi[ks][3] = pg_bf16_to_f32(v.y >> 16);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        a_lo = fmaxf(a_lo, fabsf(lo[ks][j]));
                        a_hi = fmaxf(a_hi, fabsf(hi[ks][j]));
                    }
                }
#pragma unroll
                for (int w = 1; w <= 2; w <<= 1) {
                    a_lo = fmaxf(a_lo, __shfl_xor_sync(0xffffffffu, a_lo, w));
                    a_hi = fmaxf(a_hi, __shfl_xor_sync(0xffffffffu, a_hi, w));
                }
                // exponents within +-100 of 1 keep both the scaling and its inverse normal
                const int e_lo = min(max((int)(__float_as_uint(a_lo) >> 23) - 127, -100), 100);
                const int e_hi = min(max((int)(__float_as_uint(a_hi) >> 23) - 127, -100), 100);
                const float s_lo = __uint_as_float((uint32_t)(127 - e_lo) << 23);
                const float s_hi = __uint_as_float((uint32_t)(127 - e_hi) << 23);
#pragma unroll
                for (int ks = 0; ks < NKS; ++ks) {
                    qa[ks][0] = cvt_f16x2(lo[ks][0] * s_lo, lo[ks][1] * s_lo);
                    qa[ks][1] = cvt_f16x2(hi[ks][0] * s_hi, hi[ks][1] * s_hi);
                    qa[ks][2] = cvt_f16x2(lo[ks][2] * s_lo, lo[ks][3] * s_lo);
                    qa[ks][3] = cvt_f16x2(hi[ks][2] * s_hi, hi[ks][3] * s_hi);
                }
                const float ksc = p.qk * (p.k_scale ? __ldg(p.k_scale + g) : 1.f);
                f_lo = ksc * __uint_as_float((uint32_t)(127 + e_lo) << 23);
                f_hi = ksc * __uint_as_float((uint32_t)(127 + e_hi) << 23);
            }
        }
        bad |= s_badpage[n & 7] == n;
        const int t0 = cc.kt * PA_KT;
        // tiles that reach the round's own rows have a mask by row
        const bool masked = cc.w.rows > 1 && t0 + PA_KT > cc.w.len && !cc.w.bad;
        if (masked) {
            const int kd = p.kind ? p.kind[cc.b] : 1;
            tree = p.parent != nullptr && kd != 0;
            if (tree) {
                const int n0 = p.node_off[cc.b], nn = p.node_off[cc.b + 1] - n0;
                if (n0 < 0 || nn != cc.w.rows - 1) {
                    bad = true;
                    tree = false;
                } else {
                    for (int i = tid; i < nn; i += PA_THREADS) {
                        const int pi = p.parent[n0 + i];
                        const bool off = pi < -1 || pi >= i;
                        s_par[i] = (int16_t)(off ? -1 : pi);
                        if (off) s_badtree = n;
                    }
                    __syncthreads();
                    bad |= s_badtree == n;
                }
            }
            if (tid < PA_TILE_M) {
                const int r = (m0 + tid) / p.hq;
                s_vis[tid] = r < cc.w.rows ? visible64(r, cc.w.len, t0, tree ? s_par : nullptr) : 1ull;
            }
            __syncthreads();
        }
        const int k0 = warp * PA_WARP_KEYS;
        const int nvalid = cc.w.T - t0 - k0;   // positions of this warp that exist (may be past 16, or none)
        if (nvalid > 0) {
            float sc[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.f;
            const int mi = lane >> 3, r8 = lane & 7;
            if (!E4M3) {
#pragma unroll
                for (int ks = 0; ks < NKS; ++ks) {
                    if (ks * 16 >= p.D) continue;   // past the head size: whatever the stage held before
                    uint32_t kb[4];
                    pg_ldsm_x4(kb, sk + piece_at<PITCH>(k0 + (mi >> 1) * 8 + r8, 2 * ks + (mi & 1)));
                    pg_mma_bf16(sc[0], qa[ks], kb[0], kb[1]);
                    pg_mma_bf16(sc[1], qa[ks], kb[2], kb[3]);
                }
            } else {
#pragma unroll
                for (int k2 = 0; k2 < NKS / 2; ++k2) {   // two 16-byte pieces of 16 positions
                    uint32_t kb[4];
                    pg_ldsm_x4(kb, sk + piece_at<PITCH>(k0 + (mi & 1) * 8 + r8, 2 * k2 + (mi >> 1)));
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        if ((2 * k2 + u) * 16 >= p.D) continue;
                        pg_mma_f16(sc[0], qa[2 * k2 + u], e4m3x2_f16x2(kb[2 * u]), e4m3x2_f16x2(kb[2 * u] >> 16));
                        pg_mma_f16(sc[1], qa[2 * k2 + u], e4m3x2_f16x2(kb[2 * u + 1]),
                                   e4m3x2_f16x2(kb[2 * u + 1] >> 16));
                    }
                }
            }
            uint64_t v_lo = ~0ull, v_hi = ~0ull;
            if (masked) {
                v_lo = s_vis[gq] >> k0;
                v_hi = s_vis[gq + 8] >> k0;
            }
            float mx_lo = -INFINITY, mx_hi = -INFINITY;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int key = i * 8 + 2 * cq + u;
                    const bool in = key < nvalid;
                    sc[i][u] = in && (v_lo >> key & 1) ? sc[i][u] * f_lo : -INFINITY;
                    sc[i][2 + u] = in && (v_hi >> key & 1) ? sc[i][2 + u] * f_hi : -INFINITY;
                    mx_lo = fmaxf(mx_lo, sc[i][u]);
                    mx_hi = fmaxf(mx_hi, sc[i][2 + u]);
                }
            }
#pragma unroll
            for (int w = 1; w <= 2; w <<= 1) {
                mx_lo = fmaxf(mx_lo, __shfl_xor_sync(0xffffffffu, mx_lo, w));
                mx_hi = fmaxf(mx_hi, __shfl_xor_sync(0xffffffffu, mx_hi, w));
            }
            const float mn_lo = fmaxf(m_lo, mx_lo), mn_hi = fmaxf(m_hi, mx_hi);
            // a row that has seen nothing yet keeps weights of 0, not NaN
            const float b_lo = mn_lo == -INFINITY ? 0.f : mn_lo, b_hi = mn_hi == -INFINITY ? 0.f : mn_hi;
            const float a_lo = ex2_approx(m_lo - b_lo), a_hi = ex2_approx(m_hi - b_hi);
            m_lo = mn_lo;
            m_hi = mn_hi;
            l_lo *= a_lo;
            l_hi *= a_hi;
            if (__any_sync(0xffffffffu, a_lo != 1.f || a_hi != 1.f)) {
#pragma unroll
                for (int i = 0; i < 2 * NKS; ++i) {
                    o[i][0] *= a_lo;
                    o[i][1] *= a_lo;
                    o[i][2] *= a_hi;
                    o[i][3] *= a_hi;
                }
            }
            uint32_t pa[4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float p0 = ex2_approx(sc[i][0] - b_lo + PBIAS), p1 = ex2_approx(sc[i][1] - b_lo + PBIAS);
                const float p2 = ex2_approx(sc[i][2] - b_hi + PBIAS), p3 = ex2_approx(sc[i][3] - b_hi + PBIAS);
                l_lo += p0 + p1;
                l_hi += p2 + p3;
                pa[i * 2] = E4M3 ? cvt_f16x2(p0, p1) : cvt_bf16x2(p0, p1);
                pa[i * 2 + 1] = E4M3 ? cvt_f16x2(p2, p3) : cvt_bf16x2(p2, p3);
            }
            bool odd_value = false;
            uint32_t v_next[2];
            // a value that is not finite at a position some row does not see:
            // 0 * inf would reach that row, so it is left out here and added at
            // the piece's end to the rows that see it
            auto clean = [&](uint32_t& w) {
                constexpr uint32_t EXP = E4M3 ? 0x7C00u : 0x7F80u;
                if ((w & EXP) == EXP) w &= 0xFFFF0000u, odd_value = true;
                if ((w >> 16 & EXP) == EXP) w &= 0x0000FFFFu, odd_value = true;
            };
#pragma unroll
            for (int dp = 0; dp < NKS; ++dp) {
                uint32_t vb[4];
                if (!E4M3) {
                    pg_ldsm_x4_trans(vb, sv + piece_at<PITCH>(k0 + (mi & 1) * 8 + r8, 2 * dp + (mi >> 1)));
                } else {
                    // 16 positions x one 16-byte piece: a word holds dims 2 gq, + 1 of
                    // positions 2 cq, + 1; even and odd dims become two operands
                    if ((dp & 1) == 0) {
                        uint32_t w[4];
                        pg_ldsm_x4_trans(w, sv + piece_at<PITCH>(k0 + (mi & 1) * 8 + r8, dp + (mi >> 1)));
                        vb[0] = w[0], vb[1] = w[1];
                        v_next[0] = w[2], v_next[1] = w[3];
                    } else {
                        vb[0] = v_next[0], vb[1] = v_next[1];
                    }
                    const uint32_t x0 = e4m3x2_f16x2(vb[0]), x1 = e4m3x2_f16x2(vb[0] >> 16);
                    const uint32_t y0 = e4m3x2_f16x2(vb[1]), y1 = e4m3x2_f16x2(vb[1] >> 16);
                    vb[0] = __byte_perm(x0, x1, 0x5410);
                    vb[1] = __byte_perm(y0, y1, 0x5410);
                    vb[2] = __byte_perm(x0, x1, 0x7632);
                    vb[3] = __byte_perm(y0, y1, 0x7632);
                }
                if (masked) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) clean(vb[i]);
                }
                if (E4M3) {
                    pg_mma_f16(o[2 * dp], pa, vb[0], vb[1]);
                    pg_mma_f16(o[2 * dp + 1], pa, vb[2], vb[3]);
                } else {
                    pg_mma_bf16(o[2 * dp], pa, vb[0], vb[1]);
                    pg_mma_bf16(o[2 * dp + 1], pa, vb[2], vb[3]);
                }
            }
            if (odd_value) s_odd = n;
        }
        put_off(n + PRE + 1);
        const bool item_end = cc.kt + 1 == cc.w.nt;
        if (item_end || cc.left == 1) {
            // -------------------------------------------- the piece's result
#pragma unroll
            for (int w = 1; w <= 2; w <<= 1) {
                l_lo += __shfl_xor_sync(0xffffffffu, l_lo, w);
                l_hi += __shfl_xor_sync(0xffffffffu, l_hi, w);
            }
            if (cq == 0) {
                s_st[warp][gq] = make_float2(m_lo, l_lo);
                s_st[warp][gq + 8] = make_float2(m_hi, l_hi);
            }
            __syncthreads();   // also: every warp is done with this stage's keys and values
            float M_lo = -INFINITY, M_hi = -INFINITY;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                M_lo = fmaxf(M_lo, s_st[w][gq].x);
                M_hi = fmaxf(M_hi, s_st[w][gq + 8].x);
            }
            const float w_lo = m_lo == -INFINITY ? 0.f : ex2_approx(m_lo - M_lo);
            const float w_hi = m_hi == -INFINITY ? 0.f : ex2_approx(m_hi - M_hi);
            float* red = reinterpret_cast<float*>(smem + stage * S::STAGE);   // [2][16][DP]
            // dim of fragment column (i, u): bf16 i * 8 + 2 cq + u; e4m3 (i / 2) * 16 + 4 cq + 2 u + i % 2
            auto dim = [&](int i, int u) { return E4M3 ? (i >> 1) * 16 + 4 * cq + 2 * u + (i & 1) : i * 8 + 2 * cq + u; };
            auto put = [&](int slot, bool add) {
                float* x = red + slot * PA_TILE_M * DP;
#pragma unroll
                for (int i = 0; i < 2 * NKS; ++i)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        float& lo = x[gq * DP + dim(i, u)];
                        float& hi = x[(gq + 8) * DP + dim(i, u)];
                        const float a = o[i][u] * w_lo, c = o[i][2 + u] * w_hi;
                        lo = add ? lo + a : a;
                        hi = add ? hi + c : c;
                    }
            };
            if (warp < 2) put(warp, false);
            __syncthreads();
            if (warp >= 2) put(warp - 2, true);
            __syncthreads();
            const int mrows = min(PA_TILE_M, cc.w.rows * p.hq - m0);
            const bool odd = s_odd >= first;
            // row m's maximum and sum over the four warps
            auto row_stat = [&](int m) {
                float M = -INFINITY, L = 0.f;
#pragma unroll
                for (int w = 0; w < 4; ++w) M = fmaxf(M, s_st[w][m].x);
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const float2 x = s_st[w][m];
                    L += x.x == -INFINITY ? 0.f : x.y * ex2_approx(x.x - M);
                }
                return bad ? make_float2(NAN, NAN) : make_float2(M, L);
            };
            // what the products left out: values that are not finite, at the
            // positions of this piece that row m sees
            auto left_out = [&](int m, int d) {
                float x = 0.f;
                const int r = (m0 + m) / p.hq;
                for (int j = 0; j <= r; ++j) {
                    const int t = cc.w.len + j;
                    if (t < kt_first * PA_KT || t >= t0 + PA_KT) continue;
                    bool sees = !tree || j == 0 || j == r;
                    for (int a = r; a > j && !sees;) {
                        a = 1 + s_par[a - 1];
                        sees = a == j;
                    }
                    const int page = p.table[(int64_t)cc.b * p.max_pages + (t >> p.page_shift)];
                    if (!sees || page < 0 || page >= p.num_pages) continue;
                    const int64_t row = ((int64_t)page << p.page_shift) + (t & ((1 << p.page_shift) - 1));
                    const int64_t at = (row * p.G + g) * p.D + d;
                    const float v = E4M3 ? ((p.V[at] & 0x7F) == 0x7F ? NAN : 0.f)
                                         : pg_bf16_to_f32(reinterpret_cast<const uint16_t*>(p.V)[at]);
                    if (!(fabsf(v) < INFINITY)) x += v;
                }
                return x;
            };
            // two neighbouring dims of row m, summed over the warps
            auto value = [&](int m, int d) {
                const float2 a = *reinterpret_cast<const float2*>(red + m * DP + d);
                const float2 c = *reinterpret_cast<const float2*>(red + (PA_TILE_M + m) * DP + d);
                float2 v = make_float2(a.x + c.x, a.y + c.y);
                if (odd) {
                    v.x += left_out(m, d);
                    v.y += left_out(m, d + 1);
                }
                return v;
            };
            const float vs = E4M3 && p.v_scale ? __ldg(p.v_scale + g) : 1.f;
            const int half = p.D / 2;
            auto write_row = [&](int m, int d, float2 v, float2 st) {
                const int r = (m0 + m) / p.hq, h = (m0 + m) - r * p.hq;
                const int64_t pair = (int64_t)(cc.w.r0 + r) * p.H + g * p.hq + h;
                const float inv = vs / st.y;
                *reinterpret_cast<uint32_t*>(p.out + pair * p.D + d) = cvt_bf16x2(v.x * inv, v.y * inv);
                if (p.lse && d == 0) p.lse[pair] = (st.x + __log2f(st.y) - PBIAS) * LN2;
            };
            if (kt_first == 0 && item_end) {
                for (int i = tid; i < mrows * half; i += PA_THREADS) {
                    const int m = i / half, d = (i - m * half) * 2;
                    write_row(m, d, value(m, d), row_stat(m));
                }
                if (bad && tid == 0) record_error(p.ctrl, WF_ERR_BAD_DATA, (uint32_t)cc.b);
            } else {
                // a shared item: this piece to the workspace, joined by the last piece to arrive
                const int slot = (int)blockIdx.x * 2 + (kt_first == 0 ? 1 : 0);
                for (int i = tid; i < mrows * half; i += PA_THREADS) {
                    const int m = i / half, d = (i - m * half) * 2;
                    const float2 v = value(m, d);
                    *reinterpret_cast<float2*>(p.part + ((int64_t)slot * PA_TILE_M + m) * p.D + d) = v;
                }
                if (tid < mrows) p.stat[slot * PA_TILE_M + tid] = row_stat(tid);
                if (bad && tid == 0) record_error(p.ctrl, WF_ERR_BAD_DATA, (uint32_t)cc.b);
                const int64_t ts = begin + n - cc.kt;   // the item's first tile in the flat sequence
                const int c0 = (int)(ts / per), pieces = (int)((ts + cc.w.nt - 1) / per) - c0 + 1;
                __threadfence();
                __syncthreads();
                if (tid == 0) s_last = atomicAdd(p.cnt + c0, 1u) == (uint32_t)(pieces - 1);
                __syncthreads();
                if (s_last) {
                    __threadfence();
                    // piece i is CTA c0 + i's: its second slot for the item's first, else its first
                    for (int i = tid; i < mrows * half; i += PA_THREADS) {
                        const int m = i / half, d = (i - m * half) * 2;
                        float M = -INFINITY;
#pragma unroll 4
                        for (int k = 0; k < pieces; ++k)
                            M = fmaxf(M, __ldcg(&p.stat[((c0 + k) * 2 + (k == 0)) * PA_TILE_M + m]).x);
                        float L = 0.f;
                        float2 v = make_float2(0.f, 0.f);
#pragma unroll 4
                        for (int k = 0; k < pieces; ++k) {
                            const int64_t at = (int64_t)((c0 + k) * 2 + (k == 0)) * PA_TILE_M + m;
                            const float2 st2 = __ldcg(&p.stat[at]);
                            const float2 x = __ldcg(reinterpret_cast<const float2*>(p.part + at * p.D + d));
                            const float w = st2.x == -INFINITY ? 0.f : ex2_approx(st2.x - M);
                            L = fmaf(st2.y, w, L);
                            v.x = fmaf(x.x, w, v.x);
                            v.y = fmaf(x.y, w, v.y);
                        }
                        write_row(m, d, v, make_float2(M, L));
                    }
                    if (tid == 0) p.cnt[c0] = 0;
                }
            }
            first = -1;
        }
        cursor_next(p, cc);
    }
    pg_cp_wait<0>();
}

// ------------------------------------------------------------------ host side
using PagedAttendFn = void (*)(PagedAttnParams);

struct PaVariant {
    PagedAttendFn fn;
    int smem;
};

static PaVariant pa_variant(int D, bool e4m3) {
    if (D <= 64) return e4m3 ? PaVariant{paged_attend_kernel<64, true>, PaShape<64, true>::SMEM}
                             : PaVariant{paged_attend_kernel<64, false>, PaShape<64, false>::SMEM};
    if (D <= 96) return e4m3 ? PaVariant{paged_attend_kernel<96, true>, PaShape<96, true>::SMEM}
                             : PaVariant{paged_attend_kernel<96, false>, PaShape<96, false>::SMEM};
    return e4m3 ? PaVariant{paged_attend_kernel<128, true>, PaShape<128, true>::SMEM}
                : PaVariant{paged_attend_kernel<128, false>, PaShape<128, false>::SMEM};
}

wf_status launch_paged_token(const wf_paged_cache* c, const wf_paged_attn_args* a, void* ws, cudaStream_t s);
wf_status launch_paged_rounds(const wf_paged_cache* c, const wf_paged_attn_args* a, void* ws, cudaStream_t s);

wf_status launch_paged_attention(const wf_paged_cache* c, const wf_paged_attn_args* a, void* ws, cudaStream_t s) {
    if (a->P == 0) return WF_OK;
    if (a->max_rows == 1) return launch_paged_token(c, a, ws, s);
    if (c->kv_type == WF_KV_BF16) return launch_paged_rounds(c, a, ws, s);
    static std::mutex mu;
    static bool attr_set[64] = {false};
    static int ctas[64][6];   // CTAs an SM holds, per variant
    const bool e4m3 = c->kv_type == WF_KV_E4M3;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return WF_ERR_CUDA;
    PA_TRY(configure_once(mu, attr_set, [dev] {
        for (int i = 0; i < 6; ++i) {
            const PaVariant v = pa_variant(i < 2 ? 64 : (i < 4 ? 96 : 128), i & 1);
            if (cudaFuncSetAttribute(v.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, v.smem) != cudaSuccess ||
                cudaFuncSetAttribute(v.fn, cudaFuncAttributePreferredSharedMemoryCarveout, 100) != cudaSuccess ||
                cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ctas[dev][i], v.fn, PA_THREADS, v.smem) != cudaSuccess)
                return false;
        }
        return true;
    }));
    uint8_t* w = static_cast<uint8_t*>(ws);
    const PagedLayout L = paged_layout(c->B, a->H, c->G, c->D, a->max_rows);
    const int64_t esize = e4m3 ? 1 : 2;
    const int64_t layer_bytes = (int64_t)c->num_pages * c->page_size * c->G * c->D * esize;
    PagedAttnParams p = {};
    p.q = a->q;
    p.q_stride = a->q_stride;
    p.pos_off = a->pos_off;
    p.cache_len = a->cache_len;
    p.node_off = a->node_off;
    p.kind = a->kind;
    p.parent = a->parent;
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
    p.B = c->B;
    p.page_shift = 0;
    while ((1 << p.page_shift) < c->page_size) ++p.page_shift;
    p.num_pages = c->num_pages;
    p.max_pages = c->max_pages;
    p.max_rows = a->max_rows;
    p.min_tiles = 2;
    p.ctrl = static_cast<Control*>(ws);
    const int vi = (c->D <= 64 ? 0 : (c->D <= 96 ? 2 : 4)) + (e4m3 ? 1 : 0);
    const PaVariant v = pa_variant(c->D, e4m3);
    int grid = num_sms() * (ctas[dev][vi] > 0 ? ctas[dev][vi] : 1);
    if (grid > PA_MAX_CTAS) grid = PA_MAX_CTAS;
    // no more CTAs than tiles that the lengths' bound allows
    const int64_t tiles = (int64_t)c->B * c->G * cdiv((int64_t)a->max_rows * p.hq, PA_TILE_M) *
                          cdiv((int64_t)c->max_pages * c->page_size, PA_KT);
    if (tiles < grid) grid = (int)tiles;
    return launch(v.fn, dim3(grid), dim3(PA_THREADS), (size_t)v.smem, s, p);
}

}  // namespace wf
