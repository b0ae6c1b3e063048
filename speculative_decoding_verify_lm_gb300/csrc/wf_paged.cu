// The paged cache's bookkeeping and row movement: a round's keys and values
// into their pages, the accepted rows compacted in every layer, and the pages'
// own life (reserve with copy on write, fork, trim).
//
// All of them move bytes or count pages, so memory bandwidth or, for one
// user's round, a launch and two or three dependent loads bound them.  Every
// decision is taken in the order of the sequences, whatever order the threads
// run in: results are the same from run to run.
//
// No pointer here is declared unaliased or read-only for the kernel's life: a
// launch may begin while the kernel before it still writes the lengths, tables
// and lists that it reads behind its wait.
#include "wf_paged.cuh"

#define PG_TRY(x)                      \
    do {                               \
        const wf_status _st = (x);     \
        if (_st != WF_OK) return _st;  \
    } while (0)

namespace wf {

static int log2_of(int page_size) {
    int s = 0;
    while ((1 << s) < page_size) ++s;
    return s;
}

// ------------------------------------------------------------------ append
// One warp per row: the row's keys and values are loaded (eight 16-byte pieces
// a lane in flight) before the lane knows where they go; the sequence search
// and the page lookup run meanwhile.  256 trees of 61 rows of 8 x 128: 22.9 us,
// 82% of the copy rate; 17 rows: 4.2 us, a launch.
constexpr int AP_WARPS = 8;
constexpr int AP_UNROLL = 8;

struct AppendParams {
    const uint16_t* k;
    const uint16_t* v;
    int64_t k_stride, v_stride;   // elements
    const int32_t* pos_off;
    const int32_t* cache_len;
    const int32_t* table;
    const int32_t* ref;           // or null
    uint8_t* K;                   // this layer's rows
    uint8_t* V;
    const float* k_scale;         // this layer's [G] scales, or null
    const float* v_scale;
    int P, B, GD, D, page_shift, num_pages, max_pages;
    Control* ctrl;
};

// 16 consecutive elements of one head over its scale, as e4m3 bytes
__device__ __forceinline__ uint4 quant16(uint4 a, uint4 b, float s) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = cvt_e4m3x2(__fdiv_rn(pg_bf16_to_f32(w[2 * i] & 0xFFFFu), s),
                                       __fdiv_rn(pg_bf16_to_f32(w[2 * i] >> 16), s));
        const uint32_t hi = cvt_e4m3x2(__fdiv_rn(pg_bf16_to_f32(w[2 * i + 1] & 0xFFFFu), s),
                                       __fdiv_rn(pg_bf16_to_f32(w[2 * i + 1] >> 16), s));
        o[i] = lo | (hi << 16);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

template <bool E4M3>
__global__ void __launch_bounds__(AP_WARPS * 32) append_kernel(const AppendParams p) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.x * AP_WARPS + (threadIdx.x >> 5);
    if (row >= p.P) return;
    constexpr int EL = E4M3 ? 16 : 8;                // elements of a 16-byte piece of the cache
    constexpr int UN = E4M3 ? AP_UNROLL / 2 : AP_UNROLL;
    const int C = p.GD / EL;                         // pieces of a row's keys
    const uint4* k = reinterpret_cast<const uint4*>(p.k + (int64_t)row * p.k_stride);
    const uint4* v = reinterpret_cast<const uint4*>(p.v + (int64_t)row * p.v_stride);
    int64_t dst = -1;                                // pool row
    for (int base = 0; base < 2 * C; base += 32 * UN) {
        uint4 x[UN], y[UN];
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const int c = base + u * 32 + lane;
            if (c >= 2 * C) continue;
            const uint4* s = c < C ? k : v;
            const int i = c < C ? c : c - C;
            if (E4M3) {
                x[u] = s[2 * i];
                y[u] = s[2 * i + 1];
            } else {
                x[u] = s[i];
            }
        }
        if (base == 0) {
            const int b = warp_seq_of(p.pos_off, p.B, row, lane);
            if (b < 0 || row >= p.pos_off[b + 1]) return;
            const int len = p.cache_len[b], first = p.pos_off[b];
            const int64_t t = (int64_t)len + row - first;   // 64 bits before the difference: first may be any number
            int page = -1;
            if (len >= 0 && first >= 0 && (t >> p.page_shift) < p.max_pages)
                page = p.table[(int64_t)b * p.max_pages + (t >> p.page_shift)];
            // A page that others hold too may have their rows where this one goes.  (The
            // count is one more dependent load: 22.9 us against 22.2 for 256 trees, 4.2
            // against 4.0 for a chain.)
            if (page < 0 || page >= p.num_pages || (p.ref && p.ref[page] > 1)) {
                if (lane == 0) record_error(p.ctrl, WF_ERR_BAD_DATA, (uint32_t)b);
                return;
            }
            dst = ((int64_t)page << p.page_shift) + (t & ((1 << p.page_shift) - 1));
        }
        uint4* K = reinterpret_cast<uint4*>(p.K) + dst * C;
        uint4* V = reinterpret_cast<uint4*>(p.V) + dst * C;
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const int c = base + u * 32 + lane;
            if (c >= 2 * C) continue;
            const int i = c < C ? c : c - C;
            uint4 o = x[u];
            if (E4M3) {
                const float* sc = c < C ? p.k_scale : p.v_scale;
                o = quant16(x[u], y[u], sc ? __ldg(sc + i * 16 / p.D) : 1.f);
            }
            (c < C ? K : V)[i] = o;
        }
    }
}

// ------------------------------------------------------------------ compact
// Column-parallel: a thread owns one 16-byte column of one layer's keys or
// values and moves the rows in ascending order, eight loads in flight.  Since
// the path increases, a destination (row j) never lies past its own source
// (row path[j] >= j) and so never on a later source: within a thread the moves
// are safe in place, and threads share no byte.  48 trees' accepted rows in 32
// layers: 19 us, 76% of the copy rate; one user's 3.0 us, a launch.
constexpr int CP_THREADS = 256;
constexpr int CP_BATCH = 8;
static_assert(WF_MAX_SEQ_NODES <= CP_THREADS, "one path entry a thread");

struct CompactParams {
    uint8_t* K;
    uint8_t* V;
    const int32_t* table;
    const int32_t* ref;           // or null
    const int32_t* n_accept;
    const int32_t* path;
    const int32_t* cache_len;
    int32_t* new_len;
    uint32_t* cnt;                // [B] arrivals, zero at rest
    int64_t layer_bytes;
    int path_stride, layers, row_bytes, page_shift, num_pages, max_pages;
    Control* ctrl;
};

__global__ void __launch_bounds__(CP_THREADS) compact_kernel(const CompactParams p) {
    pdl_wait();
    pdl_trigger();
    __shared__ int s_src[WF_MAX_SEQ_NODES], s_dst[WF_MAX_SEQ_NODES];
    const int tid = threadIdx.x, b = blockIdx.y;
    const int len = p.cache_len[b];
    int n = min(p.n_accept[b], p.path_stride);
    const bool none = n < 0;                         // a sequence verification marked bad keeps no row
    if (none) n = 0;
    auto row_of = [&](int64_t t) -> int64_t {        // pool row of a position, -1 without a page
        const int64_t blk = t >> p.page_shift;
        if (t < 0 || blk >= p.max_pages) return -1;
        const int page = p.table[(int64_t)b * p.max_pages + blk];
        if (page < 0 || page >= p.num_pages) return -1;
        return ((int64_t)page << p.page_shift) + (t & ((1 << p.page_shift) - 1));
    };
    bool bad = len < 0 || (!none && (int64_t)len + n + 1 > ((int64_t)p.max_pages << p.page_shift));
    // the first row is kept whatever is accepted: by a thread without a path entry if there is one
    if (tid == CP_THREADS - 1 && !bad && !none) bad = row_of(len) < 0;
    bool same = false;
    if (!bad && tid < n) {
        const int32_t* way = p.path + (int64_t)b * p.path_stride;
        const int s = way[tid];
        const int before = tid > 0 ? way[tid - 1] : -1;
        // a path that increases from 0 or more never falls below its own index
        if (s <= before || s < tid) {
            bad = true;
        } else {
            same = s == tid;
            const int64_t from = row_of((int64_t)len + 1 + s), to = row_of((int64_t)len + 1 + tid);
            bad = from < 0 || to < 0;
            // rows are moved within pages that the sequence holds alone
            if (!bad && !same && p.ref) bad = p.ref[to >> p.page_shift] > 1;
            s_src[tid] = (int)from;
            s_dst[tid] = (int)to;
        }
    }
    bad = __syncthreads_or(bad);
    // increasing paths stay on their index for a prefix and are past it from then on
    const int k0 = __syncthreads_count(same);
    if (tid == 0) {
        // the last CTA of the sequence has everybody's reads of cache_len behind it
        const uint32_t seen = atomicAdd(&p.cnt[b], 1u);
        if (seen == gridDim.x - 1) {
            p.cnt[b] = 0;
            __threadfence();
            p.new_len[b] = bad ? -1 : (none ? len : len + n + 1);
            if (bad) record_error(p.ctrl, WF_ERR_BAD_DATA, (uint32_t)b);
        }
    }
    if (bad || k0 >= n) return;
    const int chunks = p.row_bytes >> 4;
    const int cols = p.layers * 2 * chunks;
    const int col = blockIdx.x * CP_THREADS + tid;
    if (col >= cols) return;
    const int layer = col / (2 * chunks), rest = col - layer * 2 * chunks;
    uint8_t* base = (rest < chunks ? p.K : p.V) + layer * p.layer_bytes + (rest < chunks ? rest : rest - chunks) * 16;
    for (int j = k0; j < n; j += CP_BATCH) {
        uint4 x[CP_BATCH];
#pragma unroll
        for (int u = 0; u < CP_BATCH; ++u)
            if (j + u < n) x[u] = *reinterpret_cast<const uint4*>(base + (int64_t)s_src[j + u] * p.row_bytes);
#pragma unroll
        for (int u = 0; u < CP_BATCH; ++u)
            if (j + u < n) *reinterpret_cast<uint4*>(base + (int64_t)s_dst[j + u] * p.row_bytes) = x[u];
    }
}

// ------------------------------------------------------------------ reserve
// One CTA decides.  A thread owns whole sequences; the free pages are found
// 16,384 counts at a time, their numbers kept in shared memory.  A chain of
// dependent loads bounds it, so the first counts are read while the sequences
// are, and what a sequence needs stays in shared memory.  Pools whose free pages
// lie far up cost a look at every chunk below, and one more to hand them out if
// several chunks hold them: 12.7 us (with the copies' launch) where the first
// chunk has enough, whatever the pool, 25 where they are the last of 40,000 pages,
// 60 of 150,000.
//
// Copy on write in sequence order without an ordered pass: every holder that
// is about to write takes its reference away; a page whose count reaches 0 has
// all of its holders here, and the last of them in order (an atomic minimum of
// -(b + 1) in the count itself) keeps it.  While undecided, a table entry holds
// -(page + 2).
constexpr int RS_THREADS = 1024;
constexpr int RS_CHUNK = 16384;   // pages looked at together

struct ReserveParams {
    int32_t* table;
    int32_t* ref;
    const int32_t* pos_off;
    const int32_t* cache_len;
    int32_t* added;       // or null
    int32_t* copies;      // (from, to) of each page to copy
    uint32_t* n_copies;
    int B, page_shift, num_pages, max_pages;
    Control* ctrl;
};

struct Blocks {
    int j0, j1;
    bool tail;   // block j0 holds earlier positions
};

__device__ __forceinline__ Blocks blocks_of(const ReserveParams& p, int b) {
    const int len = p.cache_len[b], rows = p.pos_off[b + 1] - p.pos_off[b];
    const int ps = 1 << p.page_shift;
    Blocks k;
    k.j0 = len >> p.page_shift;
    k.j1 = rows > 0 ? (len + rows + ps - 1) >> p.page_shift : k.j0;
    k.tail = (len & (ps - 1)) != 0;
    return k;
}

// Exclusive sum over the CTA; *total is the whole sum.
__device__ __forceinline__ int block_scan(int v, int* s_warp, int* total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[w] = x;
    __syncthreads();
    if (w == 0) {
        int y = s_warp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) y += z;
        }
        s_warp[lane] = y;
    }
    __syncthreads();
    const int before = w > 0 ? s_warp[w - 1] : 0;
    *total = s_warp[31];
    __syncthreads();
    return before + x - v;
}

// This thread's counts of the chunk [base, base + RS_CHUNK).
constexpr int RS_PER_WARP = RS_CHUNK / (RS_THREADS / 32);
constexpr int RS_STEPS = RS_PER_WARP / 32;
__device__ __forceinline__ void chunk_counts(const int32_t* ref, int num_pages, int base, int (&r)[RS_STEPS]) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int i = 0; i < RS_STEPS; ++i) {
        const int page = base + w * RS_PER_WARP + i * 32 + lane;
        r[i] = page < num_pages ? __ldcg(ref + page) : 1;
    }
}

// The chunk's free pages, lowest first, into `list`; returns their number.
__device__ __forceinline__ int free_in_chunk(const int (&r)[RS_STEPS], int base, int32_t* list, int* s_warp) {
    constexpr int PER_WARP = RS_PER_WARP, STEPS = RS_STEPS;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    unsigned mask[STEPS];
    int n = 0;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        mask[i] = __ballot_sync(0xffffffffu, r[i] == 0);
        n += __popc(mask[i]);
    }
    int total;
    int at = block_scan(lane == 0 ? n : 0, s_warp, &total);
    at = __shfl_sync(0xffffffffu, at, 0);
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        if (mask[i] >> lane & 1u) list[at + __popc(mask[i] & ((1u << lane) - 1u))] = base + w * PER_WARP + i * 32 + lane;
        at += __popc(mask[i]);
    }
    __syncthreads();
    return total;
}

__global__ void __launch_bounds__(RS_THREADS) reserve_kernel(const ReserveParams p) {
    extern __shared__ int32_t list[];   // [RS_CHUNK] free pages
    int32_t* off = list + RS_CHUNK;     // [B] first page of each sequence among those taken
    int32_t* need = off + p.B;          // [B] pages it takes, -1 bad
    __shared__ int s_warp[32];
    __shared__ unsigned s_copies;
    pdl_wait();
    pdl_trigger();   // the copies' CTAs may take their places and wait there
    const int tid = threadIdx.x;
    const int64_t cap = (int64_t)p.max_pages << p.page_shift;
    if (tid == 0) s_copies = 0;
    // which pages are free does not change below before they are handed out
    int counts[RS_STEPS];
    chunk_counts(p.ref, p.num_pages, 0, counts);
    // shared blocks that are about to be written are marked
    bool any_shared = false;
    for (int b = tid; b < p.B; b += RS_THREADS) {
        const int len = p.cache_len[b];
        const int64_t rows = (int64_t)p.pos_off[b + 1] - p.pos_off[b];
        bool ok = len >= 0 && rows >= 0 && len + rows <= cap;
        int32_t* row = p.table + (int64_t)b * p.max_pages;
        if (ok) {
            const Blocks k = blocks_of(p, b);
            for (int j = k.j0; j < k.j1; ++j) ok &= row[j] >= -1 && row[j] < p.num_pages;
            if (ok && k.tail && k.j1 > k.j0) ok = row[k.j0] >= 0;   // its earlier positions have a page
            if (ok)
                for (int j = k.j0; j < k.j1; ++j) {
                    const int e = row[j];
                    if (e >= 0 && __ldcg(p.ref + e) > 1) {
                        row[j] = -(e + 2);
                        any_shared = true;
                    }
                }
        }
        need[b] = ok ? 0 : -1;
        if (!ok) record_error(p.ctrl, WF_ERR_BAD_DATA, (uint32_t)b);
    }
    any_shared = __syncthreads_or(any_shared);
    auto each_marked = [&](auto&& f) {   // f(b, entry address, page)
        for (int b = tid; b < p.B; b += RS_THREADS) {
            if (need[b] < 0) continue;
            const Blocks k = blocks_of(p, b);
            int32_t* row = p.table + (int64_t)b * p.max_pages;
            for (int j = k.j0; j < k.j1; ++j)
                if (row[j] <= -2) f(b, row + j, -(row[j] + 2));
        }
    };
    if (any_shared) {
        each_marked([&](int, int32_t*, int page) { atomicSub(p.ref + page, 1); });
        __syncthreads();
        each_marked([&](int b, int32_t*, int page) {
            if (__ldcg(p.ref + page) <= 0) atomicMin(p.ref + page, -(b + 1));
        });
        __syncthreads();
        each_marked([&](int b, int32_t* entry, int page) {
            if (__ldcg(p.ref + page) == -(b + 1)) {
                *entry = page;
                __stcg(p.ref + page, 1);
            }
        });
        __syncthreads();
    }
    // pages each sequence takes, and the first of them among all taken
    int carry = 0;
    for (int b0 = 0; b0 < p.B; b0 += RS_THREADS) {
        const int b = b0 + tid;
        int n = 0;
        if (b < p.B && need[b] >= 0) {
            const Blocks k = blocks_of(p, b);
            const int32_t* row = p.table + (int64_t)b * p.max_pages;
            for (int j = k.j0; j < k.j1; ++j) n += row[j] < 0;
            need[b] = n;
        }
        int total;
        const int at = block_scan(n, s_warp, &total);
        if (b < p.B) off[b] = carry + at;
        carry += total;
    }
    const int wanted = carry;
    // how many of the wanted pages are there; a single chunk's list is kept
    int have = 0, base = 0, n_list = 0;
    while (have < wanted && base < p.num_pages) {
        if (base > 0) chunk_counts(p.ref, p.num_pages, base, counts);
        n_list = free_in_chunk(counts, base, list, s_warp);
        have += n_list;
        base += RS_CHUNK;
    }
    const int limit = have < wanted ? have : wanted;
    const bool kept = base <= RS_CHUNK;
    auto hand_out = [&](int first, int n) {   // list holds the pages of ranks [first, first + n)
        for (int b = tid; b < p.B; b += RS_THREADS) {
            const int taken = need[b], from = off[b];
            if (taken <= 0 || from + taken > limit || from >= first + n || from + taken <= first) continue;
            const Blocks k = blocks_of(p, b);
            int32_t* row = p.table + (int64_t)b * p.max_pages;
            int rank = from > first ? from : first;   // those below came from earlier chunks
            for (int j = k.j0; j < k.j1 && rank < from + taken && rank < first + n; ++j) {
                const int e = row[j];
                if (e >= 0) continue;
                const int page = list[rank - first];
                ++rank;
                row[j] = page;
                __stcg(p.ref + page, 1);
                if (e <= -2 && j == k.j0 && k.tail) {
                    const uint32_t at = atomicAdd(&s_copies, 1u);
                    p.copies[2 * at] = -(e + 2);
                    p.copies[2 * at + 1] = page;
                }
            }
        }
        __syncthreads();
    };
    if (limit > 0) {
        if (kept) {
            hand_out(0, n_list);
        } else {
            int first = 0;
            for (int c = 0; c < p.num_pages && first < limit; c += RS_CHUNK) {
                chunk_counts(p.ref, p.num_pages, c, counts);
                const int n = free_in_chunk(counts, c, list, s_warp);
                hand_out(first, n);
                first += n;
            }
        }
    }
    // those that did not fit get their references back
    for (int b = tid; b < p.B; b += RS_THREADS) {
        const int taken = need[b];
        const bool fits = taken >= 0 && off[b] + taken <= limit;
        if (taken > 0 && !fits) {
            const Blocks k = blocks_of(p, b);
            int32_t* row = p.table + (int64_t)b * p.max_pages;
            for (int j = k.j0; j < k.j1; ++j)
                if (row[j] <= -2) {
                    const int page = -(row[j] + 2);
                    row[j] = page;
                    atomicAdd(p.ref + page, 1);
                }
        }
        if (p.added) p.added[b] = fits ? taken : -1;
    }
    if (tid == 0) *p.n_copies = s_copies;   // behind hand_out's barriers
}

// The pages that reserve_kernel listed, copied in every layer: 32 KB units
// over the whole grid, eight loads a thread in flight (four: 51 us for the
// copies of 64 continuations of a 32-layer cache, eight 43).
constexpr int PC_THREADS = 256;
constexpr int PC_UNROLL = 8;
constexpr int PC_UNIT = PC_THREADS * PC_UNROLL * 16;

__global__ void __launch_bounds__(PC_THREADS)
    page_copy_kernel(uint8_t* K, uint8_t* V, const int32_t* copies, const uint32_t* n_copies,
                     int64_t layer_bytes, int64_t page_bytes, int layers) {
    pdl_wait();
    pdl_trigger();
    const int n = (int)__ldcg(n_copies);
    if (n == 0) return;
    const int per_page = (int)((page_bytes + PC_UNIT - 1) / PC_UNIT);
    const int64_t units = (int64_t)n * layers * 2 * per_page;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        int64_t x = u;
        const int piece = (int)(x % per_page);
        x /= per_page;
        const int kv = (int)(x & 1);
        x >>= 1;
        const int layer = (int)(x % layers), c = (int)(x / layers);
        uint8_t* base = (kv ? V : K) + layer * layer_bytes;
        const uint8_t* src = base + __ldcg(copies + 2 * c) * page_bytes;
        uint8_t* dst = base + __ldcg(copies + 2 * c + 1) * page_bytes;
        const int64_t at = (int64_t)piece * PC_UNIT + threadIdx.x * 16;
        uint4 v[PC_UNROLL];
#pragma unroll
        for (int i = 0; i < PC_UNROLL; ++i)
            if (at + i * PC_THREADS * 16 < page_bytes)
                v[i] = *reinterpret_cast<const uint4*>(src + at + i * PC_THREADS * 16);
#pragma unroll
        for (int i = 0; i < PC_UNROLL; ++i)
            if (at + i * PC_THREADS * 16 < page_bytes)
                *reinterpret_cast<uint4*>(dst + at + i * PC_THREADS * 16) = v[i];
    }
}

// ------------------------------------------------------------------ fork, trim
constexpr int FK_THREADS = 256;

__global__ void __launch_bounds__(FK_THREADS)
    fork_kernel(int32_t* table, int32_t* ref, const int32_t* src, const int32_t* dst, int n,
                int32_t* cache_len, int B, int page_shift, int num_pages, int max_pages, Control* ctrl) {
    pdl_wait();
    pdl_trigger();
    const int i = blockIdx.x, tid = threadIdx.x;
    const int a = src[i], d = dst[i];
    bool bad = a < 0 || a >= B || d < 0 || d >= B;
    // every other fork leaves this one's two sequences alone: d is nobody's
    // source and nobody else's destination
    for (int k = tid; k < n; k += FK_THREADS) bad |= (k != i && dst[k] == d) || src[k] == d;
    bad = __syncthreads_or(bad);
    int blocks = 0, len = 0;
    if (!bad) {
        len = cache_len[a];
        blocks = len < 0 ? -1 : (int)(((int64_t)len + (1 << page_shift) - 1) >> page_shift);
        bad = blocks < 0 || blocks > max_pages;
        const int32_t* from = table + (int64_t)a * max_pages;
        const int32_t* to = table + (int64_t)d * max_pages;
        for (int j = tid; j < max_pages; j += FK_THREADS) {
            bad |= to[j] >= 0;
            bad |= j < blocks && (from[j] < 0 || from[j] >= num_pages);
        }
    }
    bad = __syncthreads_or(bad);
    if (bad) {
        if (tid == 0) record_error(ctrl, WF_ERR_BAD_DATA, (uint32_t)i);
        return;
    }
    for (int j = tid; j < max_pages; j += FK_THREADS) {
        const int page = j < blocks ? table[(int64_t)a * max_pages + j] : -1;
        table[(int64_t)d * max_pages + j] = page;
        if (page >= 0) atomicAdd(ref + page, 1);
    }
    if (tid == 0) cache_len[d] = len;
}

__global__ void __launch_bounds__(FK_THREADS)
    trim_kernel(int32_t* table, int32_t* ref, const int32_t* cache_len, int page_shift, int num_pages,
                int max_pages, Control* ctrl) {
    pdl_wait();
    pdl_trigger();
    const int b = blockIdx.x;
    const int len = cache_len[b];
    if (len < 0) {
        if (threadIdx.x == 0) record_error(ctrl, WF_ERR_BAD_DATA, (uint32_t)b);
        return;
    }
    const int64_t first = ((int64_t)len + (1 << page_shift) - 1) >> page_shift;
    int32_t* row = table + (int64_t)b * max_pages;
    for (int64_t j = first + threadIdx.x; j < max_pages; j += FK_THREADS) {
        const int page = row[j];
        if (page == -1) continue;
        row[j] = -1;
        bool bad = page < 0 || page >= num_pages;
        if (!bad && atomicSub(ref + page, 1) <= 0) {
            atomicAdd(ref + page, 1);
            bad = true;
        }
        if (bad) record_error(ctrl, WF_ERR_BAD_DATA, (uint32_t)b);
    }
}

// ------------------------------------------------------------------ host side
size_t paged_workspace_bytes(int D, int max_rows) {
    return paged_layout(D, max_rows).total;
}

static int64_t kv_bytes(const wf_paged_cache* c) { return c->kv_type == WF_KV_E4M3 ? 1 : 2; }

wf_status launch_paged_append(const wf_paged_cache* c, int layer, const uint16_t* k, int64_t k_stride,
                              const uint16_t* v, int64_t v_stride, int P, const int32_t* pos_off,
                              const int32_t* cache_len, void* ws, cudaStream_t s) {
    if (P == 0) return WF_OK;
    const int64_t layer_bytes = (int64_t)c->num_pages * c->page_size * c->G * c->D * kv_bytes(c);
    AppendParams p = {};
    p.k = k;
    p.v = v;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.pos_off = pos_off;
    p.cache_len = cache_len;
    p.table = c->table;
    p.ref = c->ref;
    p.K = static_cast<uint8_t*>(c->K) + layer * layer_bytes;
    p.V = static_cast<uint8_t*>(c->V) + layer * layer_bytes;
    p.k_scale = c->k_scale ? c->k_scale + (int64_t)layer * c->G : nullptr;
    p.v_scale = c->v_scale ? c->v_scale + (int64_t)layer * c->G : nullptr;
    p.P = P;
    p.B = c->B;
    p.GD = c->G * c->D;
    p.D = c->D;
    p.page_shift = log2_of(c->page_size);
    p.num_pages = c->num_pages;
    p.max_pages = c->max_pages;
    p.ctrl = static_cast<Control*>(ws);
    return launch(c->kv_type == WF_KV_E4M3 ? append_kernel<true> : append_kernel<false>, dim3(cdiv(P, AP_WARPS)),
                  dim3(AP_WARPS * 32), 0, s, p);
}

wf_status launch_paged_compact(const wf_paged_cache* c, const int32_t* n_accept, const int32_t* path,
                               int path_stride, const int32_t* cache_len, int32_t* new_len, void* ws,
                               cudaStream_t s) {
    CompactParams p = {};
    p.K = static_cast<uint8_t*>(c->K);
    p.V = static_cast<uint8_t*>(c->V);
    p.table = c->table;
    p.ref = c->ref;
    p.n_accept = n_accept;
    p.path = path;
    p.cache_len = cache_len;
    p.new_len = new_len;
    p.cnt = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(ws) + paged_layout(c->D, 1).cnt);
    p.row_bytes = (int)(c->G * c->D * kv_bytes(c));
    p.layer_bytes = (int64_t)c->num_pages * c->page_size * p.row_bytes;
    p.path_stride = path_stride;
    p.layers = c->layers;
    p.page_shift = log2_of(c->page_size);
    p.num_pages = c->num_pages;
    p.max_pages = c->max_pages;
    p.ctrl = static_cast<Control*>(ws);
    const int64_t cols = (int64_t)c->layers * 2 * (p.row_bytes / 16);
    return launch(compact_kernel, dim3((unsigned)((cols + CP_THREADS - 1) / CP_THREADS), c->B), dim3(CP_THREADS), 0, s,
                  p);
}

wf_status launch_pages_reserve(const wf_paged_cache* c, const int32_t* pos_off, const int32_t* cache_len,
                               int32_t* added, void* ws, cudaStream_t s) {
    static std::mutex mu;
    static bool attr_set[64] = {false};
    PG_TRY(configure_once(mu, attr_set, [] {
        return cudaFuncSetAttribute(reserve_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    4 * (RS_CHUNK + 2 * WF_PAGED_MAX_SEQS)) ==
               cudaSuccess;
    }));
    uint8_t* w = static_cast<uint8_t*>(ws);
    const PagedLayout L = paged_layout(c->D, 1);
    ReserveParams p = {};
    p.table = c->table;
    p.ref = c->ref;
    p.pos_off = pos_off;
    p.cache_len = cache_len;
    p.added = added;
    p.copies = reinterpret_cast<int32_t*>(w + L.copies);
    p.n_copies = reinterpret_cast<uint32_t*>(w + L.n_copies);
    p.B = c->B;
    p.page_shift = log2_of(c->page_size);
    p.num_pages = c->num_pages;
    p.max_pages = c->max_pages;
    p.ctrl = static_cast<Control*>(ws);
    PG_TRY(launch(reserve_kernel, dim3(1), dim3(RS_THREADS), 4 * ((size_t)RS_CHUNK + 2 * c->B), s, p));
    const int64_t page_bytes = (int64_t)c->page_size * c->G * c->D * kv_bytes(c);
    const int64_t layer_bytes = page_bytes * c->num_pages;
    // every unit that all sequences together can need, at most four CTAs an SM
    const int64_t units = (int64_t)c->B * c->layers * 2 * ((page_bytes + PC_UNIT - 1) / PC_UNIT);
    const int64_t most = 4ll * num_sms();
    return launch(page_copy_kernel, dim3((unsigned)(units < most ? units : most)), dim3(PC_THREADS), 0, s,
                  static_cast<uint8_t*>(c->K), static_cast<uint8_t*>(c->V), (const int32_t*)p.copies,
                  (const uint32_t*)p.n_copies, layer_bytes, page_bytes, c->layers);
}

wf_status launch_pages_fork(const wf_paged_cache* c, const int32_t* src, const int32_t* dst, int n,
                            int32_t* cache_len, void* ws, cudaStream_t s) {
    if (n == 0) return WF_OK;
    return launch(fork_kernel, dim3(n), dim3(FK_THREADS), 0, s, c->table, c->ref, src, dst, n, cache_len, c->B,
                  log2_of(c->page_size), c->num_pages, c->max_pages, static_cast<Control*>(ws));
}

wf_status launch_pages_trim(const wf_paged_cache* c, const int32_t* cache_len, void* ws, cudaStream_t s) {
    return launch(trim_kernel, dim3(c->B), dim3(FK_THREADS), 0, s, c->table, c->ref, cache_len,
                  log2_of(c->page_size), c->num_pages, c->max_pages, static_cast<Control*>(ws));
}

}  // namespace wf
