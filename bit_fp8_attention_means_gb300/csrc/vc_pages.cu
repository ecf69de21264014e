// vc_pages.cu -- the pages of a cache: named by one more sequence (vc_pages_fork),
// reserved for new tokens (vc_pages_reserve), given back (vc_pages_trim), moved
// together (vc_pages_compact) and copied (vc_cache_copy).
//
// A pool's state is how many table entries name each page, and a bit for each that none
// names.  Both are the same whatever the order in which entries come and go, so that
// atomics of any order leave the same pool, and "the lowest free pages, in the order of the
// sequences" is the same in every run.  Only reserving has an order; it is planned by one
// block (a call has few pages to find), everything that moves data or walks tables by the
// whole grid.
//
// Reserving is copy on write: a page that others name too is left to them, another takes
// its place, and the tokens in it before the new ones are copied.  Of the call's rows that
// write into one page, all but the last take another, and the last too if the page has
// names beyond theirs.  Finding the last of them needs no table: each subtracts one from the
// page's count; where none is left, all of them offer their place in the order to the same
// word, and the largest has it.
#include <climits>

#include "vc_device.cuh"
#include "vc_internal.h"
#include "vc_paged.cuh"

namespace vc {
namespace {

constexpr int kPlan = 1024;    // threads of the planning block
constexpr int kCopy = 256;     // threads of a copying block
constexpr int kOffsets = 4096; // sequences whose offsets fit the planning block's shared memory

// Page that a table entry names: e, or for a negative one below -1 the page -2 - e, which is
// held and may not be written; -1: none.
__device__ __forceinline__ int named(int e, int pages) {
    const int p = e < -1 ? -2 - e : e;
    return p < pages ? p : -1;
}

__device__ __forceinline__ bool strange(int e, int pages) { return e != -1 && named(e, pages) < 0; }

// Too few free pages: over an invalid argument, not over a timeout, whose number is smaller.  (A timeout behind
// it in the stream does not show: the waits leave the maximum, and with an exchange, a store or a look at the
// kernel's end instead of that, frames of a clip took 0.7 to 2.1 % longer and whole sequences up to 1 %.)
__device__ __forceinline__ void flag_pages(int32_t* dev_status) {
    if (!dev_status) return;
    int* word = reinterpret_cast<int*>(dev_status);
    for (int seen = *word; seen != (int)VC_ERR_TIMEOUT && seen < (int)VC_ERR_PAGES;) {
        const int was = atomicCAS(word, seen, (int)VC_ERR_PAGES);
        if (was == seen) break;
        seen = was;
    }
}

// Exclusive sum over the block of one number a thread; the total for all of them.
__device__ __forceinline__ int block_scan(int v, int* total) {
    __shared__ int sums[kPlan / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int scan = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += u;
    }
    __syncthreads();  // the last call's sums have been read
    if (lane == 31) sums[warp] = scan;
    __syncthreads();
    int s = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
    }
    *total = __shfl_sync(0xffffffffu, s, 31);
    const int before = __shfl_sync(0xffffffffu, s, max(warp - 1, 0));
    return (warp ? before : 0) + scan - v;
}

// Word i of the free bits, without bits behind the last page.
__device__ __forceinline__ uint32_t free_word(const Pool& pool, int pages, int i) {
    const int words = (pages + 31) / 32;
    if (i >= words) return 0u;
    const uint32_t w = __ldcg(pool.free + i);
    return i == words - 1 && (pages & 31) ? w & ((1u << (pages & 31)) - 1u) : w;
}

// Words of the free bits that a thread of the planning block takes at a time: neighbours, few of a small
// pool, so that more threads have some.
constexpr int kWords = 8;
__device__ __forceinline__ int words_of(int pages) { return min(kWords, (pages / 32 + kPlan) / kPlan); }

// The pages of the bits of words i .. i + per - 1 to list[at] and on, below `limit`; put(p, at) for each.  A
// warp takes its lanes' words one after the other, a bit a lane (a thread alone has up to 256 stores to make).
template <class Put>
__device__ __forceinline__ void expand(const uint32_t (&word)[kWords], int per, int i, int at, int limit, int32_t* list, Put put) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < kWords; ++k) {
        if (k >= per) break;
        if (!__any_sync(0xffffffffu, word[k] != 0u && at < limit)) {
            at += __popc(word[k]);
            continue;
        }
        for (int src = 0; src < 32; ++src) {
            const uint32_t w = __shfl_sync(0xffffffffu, word[k], src);
            const int first = __shfl_sync(0xffffffffu, at, src), base = __shfl_sync(0xffffffffu, i + k, src) * 32;
            const int to = first + __popc(w & ((1u << lane) - 1u));
            if ((w >> lane & 1u) && to < limit) {
                list[to] = base + lane;
                put(base + lane, to);
            }
        }
        at += __popc(word[k]);
    }
}

// ------------------------------------------------------------ forking and giving back

__global__ void __launch_bounds__(256) fork_kernel(const ForkArgs f, const Pool pool) {
    const int i = blockIdx.x;
    const int parent = f.parents[i], room = min(f.cols_in, f.cols_out) << f.page_log2;
    int len = 0;
    if (parent >= 0 && parent < f.B) {
        const int have = f.kv_in[parent];
        len = f.lens ? min(f.lens[i], have) : have;
        if (len < 0 || have > (f.cols_in << f.page_log2) || len > room) {
            if (threadIdx.x == 0 && blockIdx.y == 0) flag_invalid(f.dev_status);
            len = 0;
        }
    } else if (parent != -1 && threadIdx.x == 0 && blockIdx.y == 0) {
        flag_invalid(f.dev_status);
    }
    const int held = (len + (1 << f.page_log2) - 1) >> f.page_log2;
    for (int col = blockIdx.y * blockDim.x + threadIdx.x; col < f.cols_out; col += gridDim.y * blockDim.x) {
        int p = -1;
        if (col < held) {
            p = named(f.table_in[(int64_t)parent * f.s_in + col], f.pages);
            if (p >= 0 && (__ldg(pool.free + (p >> 5)) >> (p & 31) & 1u)) p = -1;  // counted for nobody: others may get it
            if (p >= 0) atomicAdd(pool.refs + p, 1);
            else flag_invalid(f.dev_status);
        }
        f.table_out[(int64_t)i * f.s_out + col] = p;
    }
    if (threadIdx.x == 0 && blockIdx.y == 0) f.kv_out[i] = len;
}

__global__ void __launch_bounds__(256) trim_kernel(const TrimArgs t, const Pool pool) {
    const int b = blockIdx.x, len = t.lens[b];
    if (len < 0) return;
    const int keep = (int)(((int64_t)len + (1 << t.page_log2) - 1) >> t.page_log2);
    for (int col = keep + blockIdx.y * blockDim.x + threadIdx.x; col < t.cols; col += gridDim.y * blockDim.x) {
        int32_t* entry = t.table + (int64_t)b * t.s_table + col;
        const int e = *entry, p = named(e, t.pages);
        if (e != -1) *entry = -1;
        if (p < 0) {
            if (strange(e, t.pages)) flag_invalid(t.dev_status);
            continue;
        }
        const int names = atomicSub(pool.refs + p, 1);
        if (names == 1) atomicOr(pool.free + (p >> 5), 1u << (p & 31));
        if (names < 1) {  // none was counted
            atomicAdd(pool.refs + p, 1);
            flag_invalid(t.dev_status);
        }
    }
    if (threadIdx.x == 0 && blockIdx.y == 0 && t.kv_len[b] > len) t.kv_len[b] = len;
}

// ------------------------------------------------------------ reserving

enum : int { kOwn = 0, kMissing = 1, kShared = 2, kContested = 3, kKeep = 4 };

__device__ __forceinline__ bool takes_new(int cls) { return cls == kMissing || cls == kShared || cls == kContested; }

// Columns of the positions that sequence b's call writes: the first, and how many.
__device__ __forceinline__ int first_col(const SeqInfo& s, int page_log2) { return max(s.L - s.n, 0) >> page_log2; }
__device__ __forceinline__ int write_cols(const SeqInfo& s, int page_log2) {
    return s.n > 0 && s.L > 0 ? ((s.L - 1) >> page_log2) - first_col(s, page_log2) + 1 : 0;
}

__global__ void __launch_bounds__(kPlan) reserve_kernel(const CacheView c, const Pool pool, const ReserveWs ws) {
    __shared__ int offsets[kOffsets + 1];
    const int tid = threadIdx.x;
    int32_t* table = const_cast<int32_t*>(c.table);
    int* off = c.B <= kOffsets ? offsets : ws.off;
    launch_dependents();
    bool bad = false;
    for (int b = tid; b < c.B; b += kPlan) {
        bad |= !seq_valid(c, b);
        ws.from[b] = -1;
    }
    if (__syncthreads_or(bad)) {  // nothing is done for a batch that breaks its rules
        if (tid == 0) flag_invalid(c.dev_status);
        return;
    }
    int W = 0;
    for (int b0 = 0; b0 < c.B; b0 += kPlan) {
        const int b = b0 + tid;
        int some;
        const int at = block_scan(b < c.B ? write_cols(seq_info(c, b), c.page_log2) : 0, &some);
        if (b < c.B) off[b] = W + at;
        W += some;
    }
    if (tid == 0) off[c.B] = W;
    __syncthreads();
    if (W == 0) return;
    // the sequence of entry w of the call: the last b with off[b] <= w
    auto sequence = [&](int w) -> int {
        int lo = 0, hi = c.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (off[mid] <= w) lo = mid;
            else hi = mid;
        }
        return lo;
    };
    // each entry's page, and what becomes of it
    bool shared = false;
    int need = 0;
    for (int w = tid; w < W; w += kPlan) {
        const int b = sequence(w);
        const SeqInfo s = seq_info(c, b);
        const int e = table[(int64_t)b * c.s_table + first_col(s, c.page_log2) + w - off[b]];
        int p = named(e, c.pages);
        const int names = p < 0 ? 0 : __ldcg(pool.refs + p);
        if (names < 1) p = -1;  // counted for nobody: others may get it
        if (e != -1 && p < 0) flag_invalid(c.dev_status);
        const int cls = p < 0 ? kMissing : names > 1 ? kShared : kOwn;
        shared |= cls == kShared;
        need += cls == kMissing;
        ws.page[w] = p;
        ws.cls[w] = cls;
    }
    shared = __syncthreads_or(shared);
    if (shared) {
        for (int w = tid; w < W; w += kPlan)
            if (ws.cls[w] == kShared) atomicSub(pool.refs + ws.page[w], 1);
        __syncthreads();
        for (int w = tid; w < W; w += kPlan)
            if (ws.cls[w] == kShared && __ldcg(pool.refs + ws.page[w]) <= 0) ws.cls[w] = kContested;
        __syncthreads();
        for (int w = tid; w < W; w += kPlan)
            if (ws.cls[w] == kContested) atomicMax(pool.refs + ws.page[w], w + 1);
        __syncthreads();
        for (int w = tid; w < W; w += kPlan) {
            if (ws.cls[w] == kContested && __ldcg(pool.refs + ws.page[w]) == w + 1) ws.cls[w] = kKeep;
            need += ws.cls[w] == kShared || ws.cls[w] == kContested;
        }
        __syncthreads();
        for (int w = tid; w < W; w += kPlan)
            if (ws.cls[w] == kKeep) pool.refs[ws.page[w]] = 1;
    }
    int all;
    block_scan(need, &all);
    need = all;
    // the lowest free pages
    const int per = words_of(c.pages);
    int found = 0;
    for (int i0 = 0; found < need && i0 * 32 < c.pages; i0 += kPlan * per) {
        const int i = i0 + tid * per;
        uint32_t word[kWords];
        int mine = 0;
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
            word[k] = k < per ? free_word(pool, c.pages, i + k) : 0u;
            mine += __popc(word[k]);
        }
        int some;
        const int at = found + block_scan(mine, &some);
        expand(word, per, i, at, need, ws.fresh, [](int, int) {});
        found += some;
    }
    __syncthreads();
    if (found < need) {
        // the counts as they were, and pages that would have to be copied marked: held, not to be written
        if (tid == 0) flag_pages(c.dev_status);
        for (int w = tid; w < W; w += kPlan)
            if (ws.cls[w] == kKeep) pool.refs[ws.page[w]] = 0;
        __syncthreads();
        for (int w = tid; w < W; w += kPlan) {
            const int cls = ws.cls[w];
            if (cls != kShared && cls != kContested && cls != kKeep) continue;
            atomicAdd(pool.refs + ws.page[w], 1);
            const int b = sequence(w);
            table[(int64_t)b * c.s_table + first_col(seq_info(c, b), c.page_log2) + w - off[b]] = -2 - ws.page[w];
        }
        return;
    }
    int rank = 0;
    for (int w0 = 0; w0 < W; w0 += kPlan) {
        const int w = w0 + tid, cls = w < W ? ws.cls[w] : kOwn;
        int some;
        const int at = rank + block_scan(takes_new(cls), &some);
        rank += some;
        if (w >= W) continue;
        const int b = sequence(w), old = ws.page[w];
        const SeqInfo s = seq_info(c, b);
        int32_t* entry = table + (int64_t)b * c.s_table + first_col(s, c.page_log2) + w - off[b];
        if (!takes_new(cls)) {
            if (*entry != old) *entry = old;  // it was marked, and is its own now
            continue;
        }
        const int p = ws.fresh[at];
        pool.refs[p] = 1;
        atomicAnd(pool.free + (p >> 5), ~(1u << (p & 31)));
        *entry = p;
        if (old >= 0 && w == off[b]) {
            ws.to[b] = p;
            ws.from[b] = old;
        }
    }
}

// ------------------------------------------------------------ copying

// Pieces of 16 bytes of a page's codes or scales, head by head: piece q of codes is at
// head q >> head, token (q >> tok) mod page, channel 16 (q mod 2^tok).
struct PageArray {
    const uint8_t* src;
    uint8_t* dst;
    int64_t src_page, src_head, src_tok, dst_page, dst_head, dst_tok;  // bytes
    int head_log2, tok_log2;
};

__device__ __forceinline__ PageArray page_array(const CacheView& s, const CacheView& d, int which, int tok_log2) {
    if (which < 2)
        return PageArray{which ? s.V8 : s.K8, which ? d.V8 : d.K8, s.s_page, s.s_head, s.s_tok, d.s_page, d.s_head, d.s_tok,
                         s.page_log2 + tok_log2, tok_log2};
    return PageArray{reinterpret_cast<const uint8_t*>(which == 2 ? s.sk : s.sv), reinterpret_cast<uint8_t*>(which == 2 ? d.sk : d.sv),
                     4 * s.t_page, 4 * s.t_head, 16, 4 * d.t_page, 4 * d.t_head, 16, s.page_log2 - 2, 0};
}

__device__ __forceinline__ int64_t piece_at(int64_t page, int64_t head, int64_t tok, const PageArray& a, int q) {
    return page + (int64_t)(q >> a.head_log2) * head + (int64_t)((q & ((1 << a.head_log2) - 1)) >> a.tok_log2) * tok +
           (q & ((1 << a.tok_log2) - 1)) * 16;
}

// Whole pages from list to list, a tile of one array of one page at a time, by the whole
// grid: 2 (2d + 8) bytes a token and head, so memory bounds it.  Four loads of 16 bytes a
// thread are under way.
constexpr int kPieces = 4, kTile = kCopy * kPieces;

__device__ __forceinline__ void copy_pages(const CacheView& s, const CacheView& d, const int32_t* from, const int32_t* to,
                                           int count, int tok_log2) {
    const int codes = s.H << (s.page_log2 + tok_log2), scales = s.H << (s.page_log2 - 2);
    const int code_tiles = (codes + kTile - 1) / kTile, scale_tiles = (scales + kTile - 1) / kTile;
    const int per = 2 * (code_tiles + scale_tiles);
    int i = blockIdx.x / per, t = blockIdx.x % per;
    const int step = gridDim.x / per, rest = gridDim.x % per;
    for (; i < count; i += step, t += rest) {
        if (t >= per) {
            t -= per;
            if (++i >= count) break;
        }
        const int a = __ldcg(from + i), b = __ldcg(to + i);
        if (a < 0 || b < 0 || a >= s.pages || b >= d.pages) {
            if (threadIdx.x == 0 && ((a != -1 && (unsigned)a >= (unsigned)s.pages) || (b != -1 && (unsigned)b >= (unsigned)d.pages)))
                flag_invalid(s.dev_status);
            continue;
        }
        const bool code = t < 2 * code_tiles;
        const int which = code ? t / code_tiles : 2 + (t - 2 * code_tiles) / scale_tiles;
        const int tile = code ? t % code_tiles : (t - 2 * code_tiles) % scale_tiles, n = code ? codes : scales;
        const PageArray x = page_array(s, d, which, tok_log2);
        uint4 v[kPieces];
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            const int q = tile * kTile + k * kCopy + threadIdx.x;
            if (q < n) v[k] = __ldcs(reinterpret_cast<const uint4*>(x.src + piece_at(a * x.src_page, x.src_head, x.src_tok, x, q)));
        }
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
            const int q = tile * kTile + k * kCopy + threadIdx.x;
            if (q < n) __stcs(reinterpret_cast<uint4*>(x.dst + piece_at(b * x.dst_page, x.dst_head, x.dst_tok, x, q)), v[k]);
        }
    }
}

__global__ void __launch_bounds__(kCopy) copy_kernel(const CacheView s, const CacheView d, const int32_t* from,
                                                     const int32_t* to, int count, int tok_log2) {
    copy_pages(s, d, from, to, count, tok_log2);
}

// The tokens that reserved pages hold of those before the call's: block (b, .) those of sequence b.
__global__ void __launch_bounds__(kCopy) copy_begun_kernel(const CacheView c, const ReserveWs ws, int tok_log2) {
    wait_for_primary();
    const int b = blockIdx.x, from = ws.from[b];
    if (from < 0) return;
    const int to = ws.to[b];
    const SeqInfo s = seq_info(c, b);
    const int tokens = max(s.L - s.n, 0) & ((1 << c.page_log2) - 1);
    const int lane = blockIdx.y * kCopy + threadIdx.x, lanes = gridDim.y * kCopy;
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
        const PageArray x = page_array(c, c, which, tok_log2);
        const int n = c.H * tokens << tok_log2;
        for (int i = lane; i < n; i += lanes) {
            const int row = i >> tok_log2, h = row / tokens;
            const int q = (h << x.head_log2) + i - ((h * tokens) << tok_log2);
            *reinterpret_cast<uint4*>(x.dst + piece_at(to * x.dst_page, x.dst_head, x.dst_tok, x, q)) =
                *reinterpret_cast<const uint4*>(x.src + piece_at(from * x.src_page, x.src_head, x.src_tok, x, q));
        }
    }
    for (int i = lane; i < c.H * tokens; i += lanes) {
        const int h = i / tokens, tok = i - h * tokens;
        const int64_t a = (int64_t)from * c.t_page + (int64_t)h * c.t_head + tok, e = (int64_t)to * c.t_page + (int64_t)h * c.t_head + tok;
        c.sk[e] = c.sk[a];
        c.sv[e] = c.sv[a];
    }
}

// ------------------------------------------------------------ moving together
//
// With U pages in use, the used ones from number U on go to the free ones below, in
// ascending order on both sides (as many by definition).  ws.number[p] is the place of a moved
// page, or of a free one that is moved into, in its list, believed only if the list names p
// there.

__global__ void __launch_bounds__(kPlan) compact_plan_kernel(const Pool pool, int pages, const CompactWs ws) {
    const int tid = threadIdx.x, per = words_of(pages);
    launch_dependents();
    int sum = 0, all;
    for (int i = tid; i * 32 < pages; i += kPlan) sum += __popc(free_word(pool, pages, i));
    block_scan(sum, &all);
    const int used = pages - all;
    int holes = 0, moved = 0;
    for (int i0 = 0; i0 * 32 < pages; i0 += kPlan * per) {
        const int i = i0 + tid * per;
        uint32_t hole[kWords], move[kWords];
        int nh = 0, nm = 0;
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
            const int base = (i + k) * 32;
            const uint32_t w = k < per ? free_word(pool, pages, i + k) : 0u;
            // bits of pages below `used`, and of pages there are
            const uint32_t low = base + 32 <= used ? ~0u : base >= used ? 0u : (1u << (used - base)) - 1u;
            const uint32_t real = k >= per ? 0u : base + 32 <= pages ? ~0u : base >= pages ? 0u : (1u << (pages - base)) - 1u;
            hole[k] = w & low;
            move[k] = ~w & ~low & real;
            nh += __popc(hole[k]);
            nm += __popc(move[k]);
        }
        int some_h, some_m;
        const int h = holes + block_scan(nh, &some_h), m = moved + block_scan(nm, &some_m);
        expand(hole, per, i, h, INT_MAX, ws.to, [&](int p, int at) { ws.number[p] = at; });
        expand(move, per, i, m, INT_MAX, ws.from, [&](int p, int at) { ws.number[p] = at; });
        holes += some_h;
        moved += some_m;
    }
    if (tid == 0) {
        ws.head[0] = used;
        ws.head[1] = moved;
    }
}

__global__ void __launch_bounds__(kCopy) compact_kernel(const CacheView c, const Pool pool, const CompactWs ws, int32_t* count,
                                                        int tok_log2) {
    wait_for_primary();
    const int used = ws.head[0], moved = ws.head[1];
    const int64_t me = (int64_t)blockIdx.x * kCopy + threadIdx.x, all = (int64_t)gridDim.x * kCopy;
    int32_t* table = const_cast<int32_t*>(c.table);
    for (int64_t k = me; k < (int64_t)c.B * c.cols; k += all) {
        int32_t* entry = table + k / c.cols * c.s_table + k % c.cols;
        const int e = *entry, p = named(e, c.pages);
        if (p < 0) {
            if (strange(e, c.pages)) flag_invalid(c.dev_status);
            continue;
        }
        const int m = ws.number[p];
        const bool listed = m >= 0 && m < moved && (p < used ? ws.to : ws.from)[m] == p;
        if (listed != (p >= used)) {  // named here and counted nowhere; one moved into has an owner from now on
            flag_invalid(c.dev_status);
            if (listed) *entry = -1;
            continue;
        }
        if (listed) *entry = e < -1 ? -2 - ws.to[m] : ws.to[m];
    }
    for (int64_t k = me; k < moved; k += all) {
        pool.refs[ws.to[k]] = pool.refs[ws.from[k]];
        pool.refs[ws.from[k]] = 0;
    }
    for (int64_t i = me; i * 32 < c.pages; i += all) {
        const int base = (int)i * 32;
        const uint32_t low = base + 32 <= used ? ~0u : base >= used ? 0u : (1u << (used - base)) - 1u;
        const uint32_t real = base + 32 <= c.pages ? ~0u : (1u << (c.pages - base)) - 1u;
        pool.free[i] = ~low & real;
    }
    if (me == 0 && count) *count = used;
    copy_pages(c, c, ws.from, ws.to, moved, tok_log2);
}

// Blocks of 256 over the columns of a row, the rows being the grid's other side.
unsigned col_blocks(int cols, int rows) {
    const int want = (cols + 255) / 256, room = rows >= 2048 ? 1 : 2048 / rows;
    return (unsigned)(want < room ? want : room);
}

int tok_log2_of(int d) { return d == 128 ? 3 : 2; }  // 16-byte pieces of a token's codes

// Blocks of 256 threads, many an SM so that none ends late (of 4,000 pages of 135 KB: 8 an SM 182 us, 32 166 us),
// fewer where there is less to copy.
unsigned copy_blocks(const CacheView& c, int d, int64_t pages) {
    const int64_t codes = (int64_t)c.H << (c.page_log2 + tok_log2_of(d)), scales = (int64_t)c.H << (c.page_log2 - 2);
    const int64_t tiles = pages * 2 * ((codes + kTile - 1) / kTile + (scales + kTile - 1) / kTile);
    return (unsigned)(tiles < kMaxCtas * 32 ? tiles : kMaxCtas * 32);
}

}  // namespace

vc_status launch_pages_fork(const ForkArgs& f, const Pool& pool, int N, cudaStream_t st) {
    fork_kernel<<<dim3(N, col_blocks(f.cols_out, N)), 256, 0, st>>>(f, pool);
    return cuda_status(cudaGetLastError());
}

vc_status launch_pages_trim(const TrimArgs& t, const Pool& pool, int B, cudaStream_t st) {
    trim_kernel<<<dim3(B, col_blocks(t.cols, B)), 256, 0, st>>>(t, pool);
    return cuda_status(cudaGetLastError());
}

// Entries that a call writes into: of n tokens no more than n / page + 2, of none none.
static int64_t reserve_entries(int B, int T, int page_log2) { return ((int64_t)T >> page_log2) + 2 * (int64_t)B; }

size_t pages_reserve_workspace(int B, int T, int page_log2) {
    return (3 * (size_t)reserve_entries(B, T, page_log2) + 3 * (size_t)B + 1) * sizeof(int32_t);
}

vc_status launch_pages_reserve(const CacheView& c, int d, const Pool& pool, void* workspace, cudaStream_t st) {
    const int64_t W = reserve_entries(c.B, c.T, c.page_log2);
    ReserveWs ws;
    ws.page = static_cast<int32_t*>(workspace);
    ws.cls = ws.page + W;
    ws.fresh = ws.cls + W;
    ws.from = ws.fresh + W;
    ws.to = ws.from + c.B;
    ws.off = ws.to + c.B;
    reserve_kernel<<<1, kPlan, 0, st>>>(c, pool, ws);
    if (cudaGetLastError() != cudaSuccess) return VC_ERR_CUDA;
    return launch_after(copy_begun_kernel, dim3(c.B, c.B >= 304 ? 1 : 4), kCopy, 0, st, c, ws, tok_log2_of(d));
}

vc_status launch_cache_copy(const CacheView& s, const CacheView& t, int d, const int32_t* from, const int32_t* to,
                            int count, cudaStream_t st) {
    copy_kernel<<<copy_blocks(s, d, count), kCopy, 0, st>>>(s, t, from, to, count, tok_log2_of(d));
    return cuda_status(cudaGetLastError());
}

size_t pages_compact_workspace(int pages) { return (2 * (size_t)pages + 2) * sizeof(int32_t); }

vc_status launch_pages_compact(const CacheView& c, int d, const Pool& pool, int32_t* count, void* workspace,
                               cudaStream_t st) {
    CompactWs ws;
    ws.head = static_cast<int32_t*>(workspace);
    ws.number = ws.head + 2;
    ws.from = ws.number + c.pages;  // no more pages move than half of them
    ws.to = ws.from + c.pages / 2;
    compact_plan_kernel<<<1, kPlan, 0, st>>>(pool, c.pages, ws);
    if (cudaGetLastError() != cudaSuccess) return VC_ERR_CUDA;
    return launch_after(compact_kernel, dim3(kMaxCtas * 16), kCopy, 0, st, c, pool, ws, count, tok_log2_of(d));
}

}  // namespace vc
