// Pages of a paged cache: copies, shared sequences, growing and shrinking ones, and a move into another pool.
//
// A pool of pages is a count of holders for each page and one bit for each that is free.  Everything here
// is whole numbers and copies, and comes out the same whatever the order in which workgroups run: pages
// come back by counts that only go down in one launch, and are taken in the order of their numbers
// by one workgroup in the next.
//
// resize  kv_drop   (a workgroup per 1024 columns of a row) the pages that shrinking sequences leave
//         kv_plan   (one workgroup) which growing sequences need a copy of a shared last page, how many pages
//                   that takes in all, whether there are as many, and the list of them
//         kv_take   the new entries of the rows, and the copies
// fork    kv_fork_plan (one workgroup) which pairs hold; kv_fork_rows the rows and counts
// compact kv_count  (one workgroup) pages in use before each 32; kv_move everything else
#include "serve_common.h"

namespace q2_0 {

// Counts change within a launch: read and changed past the vector caches.
__device__ __forceinline__ int peek(const int32_t *p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ void put(int32_t *p, int v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
// Between two steps of one workgroup that change and read counts with the calls above: every one of them has reached the
// memory that all of them meet in.  (A fence for the whole device would write caches back, several us each.)
__device__ __forceinline__ void all_done() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
}

__device__ __forceinline__ bool bad_len(int v, int64_t most) { return v < 0 || v > most; }

// tokens -> pages, 0 <= n < 2^31
__device__ __forceinline__ int pages_of(const FastDiv &page, int n) { return n == 0 ? 0 : page.div((uint32_t)n - 1u) + 1; }

constexpr int kVecs = 8;              // 16-byte vectors of a thread in a copy

// Vectors [part * 2048, ..) of a page, rows [0, rows) of each head, rows >= 1.  All loads first and without branches:
// a place past the end reads the last one that counts and is not written.
__device__ __forceinline__ void copy_part(const PageRows &to, const PageRows &from, const PageShape &sh, int64_t dst, int64_t src,
                                          int part, int rows) {
    u32x4_t x[kVecs];
    char *at[kVecs];
    const int64_t to_page = dst * to.page_stride, from_page = src * from.page_stride;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int v = part * 256 * kVecs + i * 256 + (int)threadIdx.x;
        const int u = v < sh.vecs ? v : sh.vecs - 1;
        const int row = u >> sh.vec_shift;
        const int head = sh.page.div((uint32_t)row), token = row - head * (int)sh.page.d;   // heads of k, then of v
        const int tk = token < rows ? token : rows - 1;
        const bool is_v = head >= sh.heads;
        const int64_t h = is_v ? head - sh.heads : head, b = (int64_t)(u & ((1 << sh.vec_shift) - 1)) * 16;
        x[i] = *reinterpret_cast<const u32x4_t *>((is_v ? from.v : from.k) + (from_page + h * from.head_stride + tk * from.token_stride + b));
        at[i] = (is_v ? to.v : to.k) + (to_page + h * to.head_stride + tk * to.token_stride + b);
        if (v >= sh.vecs || token >= rows) at[i] = nullptr;
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
        if (at[i]) *reinterpret_cast<u32x4_t *>(at[i]) = x[i];
}

static int parts_of(const PageShape &p) { return (p.vecs + 256 * kVecs - 1) / (256 * kVecs); }

__global__ __launch_bounds__(256) void kv_copy_pages(KvCopy a, int parts) {
    const int i = (int)(blockIdx.x / (unsigned)parts), part = (int)(blockIdx.x % (unsigned)parts);
    const int src = a.src[i], dst = a.dst[i];
    if (src < 0 || src >= a.from_pages || dst < 0 || dst >= a.to_pages) return;
    copy_part(a.to, a.from, a.shape, dst, src, part, (int)a.shape.page.d);
}

int64_t kv_copy_groups(const PageShape &p, int64_t n) { return n * parts_of(p); }

hipError_t launch_kv_copy(const KvCopy &a, hipStream_t s) {
    kv_copy_pages<<<(unsigned)kv_copy_groups(a.shape, a.n), 256, 0, s>>>(a, parts_of(a.shape));
    return hipGetLastError();
}

// ---------------------------------------------------------------------------- shared by rows of tables

constexpr int kCols = 1024;           // columns of a table row that a workgroup takes

static int col_parts(int64_t cols) { return (int)((cols + kCols - 1) / kCols); }

int64_t kv_table_groups(int64_t n_rows, int64_t cols) { return n_rows * col_parts(cols); }

// Sum over the workgroup of 1024 of the values of lower threads; `total`: of all.
__device__ __forceinline__ int64_t scan_1024(int64_t v, int64_t *tmp, int64_t &total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int64_t run = v;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int64_t o = __shfl_up(run, off);
        if (lane >= off) run += o;
    }
    if (lane == 63) tmp[wave] = run;
    __syncthreads();
    int64_t base = 0, all = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
        if (w == wave) base = all;
        all += tmp[w];
    }
    __syncthreads();
    total = all;
    return base + run - v;
}

// ---------------------------------------------------------------------------- fork

__global__ __launch_bounds__(1024) void kv_fork_plan(KvFork a) {
    const int64_t most = (int64_t)a.t.cols * a.page.d;
    for (int i = threadIdx.x; i < a.n; i += 1024) {
        const int s = a.src[i], d = a.dst[i];
        int len = -1;
        if (s >= 0 && s < a.t.n_seqs && d >= 0 && d < a.t.n_seqs && s != d && peek(a.t.lens + d) == 0) {
            len = peek(a.t.lens + s);
            if (bad_len(len, most)) len = -1;
        }
        a.plan[i] = len;
    }
    all_done();
    // the first pair of those with one destination: the lowest claim
    for (int i = threadIdx.x; i < a.n; i += 1024)
        if (a.plan[i] >= 0) atomicMin(a.t.lens + a.dst[i], i - a.n);
    all_done();
    for (int i = threadIdx.x; i < a.n; i += 1024)
        if (a.plan[i] >= 0 && peek(a.t.lens + a.dst[i]) != i - a.n) a.plan[i] = -1;
    all_done();
    for (int i = threadIdx.x; i < a.n; i += 1024)
        if (a.plan[i] >= 0) put(a.t.lens + a.dst[i], a.plan[i]);
}

__global__ __launch_bounds__(256) void kv_fork_rows(KvFork a, int parts) {
    const int i = (int)(blockIdx.x / (unsigned)parts), part = (int)(blockIdx.x % (unsigned)parts);
    const int len = a.plan[i];
    if (len <= 0) return;
    const int n = pages_of(a.page, len);
    const int32_t *from = a.t.table + a.src[i] * a.t.ld;
    int32_t *to = a.t.table + a.dst[i] * a.t.ld;
    for (int c = part * kCols + (int)threadIdx.x; c < n && c < (part + 1) * kCols; c += 256) {
        const int page = from[c];
        to[c] = page;
        if (page >= 0 && page < a.n_pages) atomicAdd(a.ref + page, 1);
    }
}

hipError_t launch_kv_fork(const KvFork &a, hipStream_t s) {
    kv_fork_plan<<<1, 1024, 0, s>>>(a);
    if (a.t.cols > 0)
        kv_fork_rows<<<(unsigned)kv_table_groups(a.n, a.t.cols), 256, 0, s>>>(a, col_parts(a.t.cols));
    return hipGetLastError();
}

// ---------------------------------------------------------------------------- resize

__global__ __launch_bounds__(256) void kv_drop(KvResize a, int parts) {
    const int s = (int)(blockIdx.x / (unsigned)parts), part = (int)(blockIdx.x % (unsigned)parts);
    const int64_t most = (int64_t)a.t.cols * a.shape.page.d;
    const int len = a.t.lens[s], now = a.new_lens[s];
    if (bad_len(len, most) || bad_len(now, most) || now >= len) return;
    const int have = pages_of(a.shape.page, len), want = pages_of(a.shape.page, now);
    int32_t *row = a.t.table + s * a.t.ld;
    const int c1 = have < (part + 1) * kCols ? have : (part + 1) * kCols;
    for (int c = part * kCols + (int)threadIdx.x; c < c1; c += 256) {
        if (c < want) continue;
        const int page = row[c];
        row[c] = -1;
        if (page >= 0 && page < a.n_pages && atomicSub(a.ref + page, 1) == 1)
            atomicOr(a.free + (page >> 5), 1u << (page & 31));
    }
}

struct Planned {
    int slot, have, want, old, rows, pad[3];
};
static_assert(sizeof(Planned) == 32, "8 numbers a sequence");

// A sequence that grows from inside a page that others hold too takes a copy of it -- unless all holders do so in this
// call: then the lowest of them keeps the page.  Holders leave by counting down; where that ends at 0, the lowest
// claim on the count is the one that stays.
template <int PT>
__global__ __launch_bounds__(1024) void kv_plan(KvResize a) {
    __shared__ int64_t tmp[16];
    const int64_t most = (int64_t)a.t.cols * a.shape.page.d;
    const int tid = threadIdx.x;
    // free pages, asked for first
    const int words = (a.n_pages + 31) / 32;
    int64_t some = 0;
    for (int w = tid; w < words; w += 1024) {
        uint32_t bits = a.free[w];
        if (w == words - 1 && a.n_pages % 32) bits &= (1u << (a.n_pages % 32)) - 1u;
        some += __popc(bits);
    }
    Planned pl[PT];
    int len[PT], now[PT], count[PT], left[PT];
    bool grows[PT], shared[PT], keeps[PT];
#pragma unroll
    for (int i = 0; i < PT; ++i) {
        const int s = tid * PT + i;
        len[i] = now[i] = -1;
        if (s < a.t.n_seqs) len[i] = a.t.lens[s], now[i] = a.new_lens[s];
        const bool ok = !bad_len(len[i], most) && !bad_len(now[i], most);
        if (!ok) now[i] = len[i];
        grows[i] = ok && now[i] > len[i];
        pl[i].have = ok ? pages_of(a.shape.page, len[i]) : 0;
        pl[i].want = grows[i] ? pages_of(a.shape.page, now[i]) : pl[i].have;
        pl[i].rows = ok && pl[i].have > 0 ? len[i] - (pl[i].have - 1) * (int)a.shape.page.d : 0;
        pl[i].old = -1;
        count[i] = 0;
        if (grows[i] && pl[i].rows > 0 && pl[i].rows < (int)a.shape.page.d) {
            const int page = a.t.table[s * a.t.ld + pl[i].have - 1];
            if (page >= 0 && page < a.n_pages) pl[i].old = page, count[i] = peek(a.ref + page);
        }
        shared[i] = count[i] > 1;
    }
    bool any = false;
#pragma unroll
    for (int i = 0; i < PT; ++i) left[i] = 1, keeps[i] = false, any |= shared[i];
    if (__syncthreads_or(any)) {                                 // (most calls: nothing is shared)
        // (the counts are read, above)
#pragma unroll
        for (int i = 0; i < PT; ++i)
            if (shared[i]) atomicSub(a.ref + pl[i].old, 1);
        all_done();
#pragma unroll
        for (int i = 0; i < PT; ++i)
            if (shared[i]) left[i] = peek(a.ref + pl[i].old);
        all_done();
#pragma unroll
        for (int i = 0; i < PT; ++i)
            if (left[i] == 0) atomicMin(a.ref + pl[i].old, tid * PT + i - a.t.n_seqs);
        all_done();
#pragma unroll
        for (int i = 0; i < PT; ++i) keeps[i] = left[i] == 0 && peek(a.ref + pl[i].old) == tid * PT + i - a.t.n_seqs;
    }
    int64_t need = 0;
#pragma unroll
    for (int i = 0; i < PT; ++i) need += pl[i].want - pl[i].have + (shared[i] && !keeps[i]);
    int64_t total;
    int64_t slot = scan_1024(need, tmp, total);
    int64_t avail;
    scan_1024(some, tmp, avail);
    const bool enough = total <= avail;
    if (tid == 0) *a.missing = enough ? 0 : (int)(total - avail < 0x7fffffff ? total - avail : 0x7fffffff);
#pragma unroll
    for (int i = 0; i < PT; ++i) {
        const int s = tid * PT + i;
        const bool copies = shared[i] && !keeps[i];
        if (keeps[i]) put(a.ref + pl[i].old, enough ? 1 : count[i]);
        if (copies && left[i] > 0 && !enough) atomicAdd(a.ref + pl[i].old, 1);
        if (s >= a.t.n_seqs) continue;
        if (now[i] != len[i] && (enough || !grows[i])) a.t.lens[s] = now[i];
        pl[i].slot = enough ? (int)slot : 0;
        slot += pl[i].want - pl[i].have + copies;
        if (!copies || !enough) pl[i].old = -1;
        if (!enough) pl[i].want = pl[i].have;
        reinterpret_cast<Planned *>(a.plan)[s] = pl[i];
    }
    // the free pages of the lowest numbers, `total` of them
    for (int64_t w0 = 0, base = 0; enough && base < total && w0 < words; w0 += 1024) {
        const int w = (int)w0 + tid;
        uint32_t bits = w < words ? a.free[w] : 0u;
        if (w == words - 1 && a.n_pages % 32) bits &= (1u << (a.n_pages % 32)) - 1u;
        int64_t all;
        int64_t at = base + scan_1024(__popc(bits), tmp, all);
        uint32_t taken = 0;
        while (bits && at < total) {
            const int b = __ffs((int)bits) - 1;
            bits &= bits - 1;
            taken |= 1u << b;
            a.fresh[at++] = w * 32 + b;
        }
        if (taken) a.free[w] &= ~taken;
        base += all;
    }
}

__global__ __launch_bounds__(256) void kv_take(KvResize a, int parts, int copy_parts, unsigned row_groups) {
    const Planned *plan = reinterpret_cast<const Planned *>(a.plan);
    if (blockIdx.x >= row_groups) {
        const unsigned b = blockIdx.x - row_groups;
        const int s = (int)(b / (unsigned)copy_parts), part = (int)(b % (unsigned)copy_parts);
        const Planned pl = plan[s];
        if (pl.old >= 0) copy_part(a.rows, a.rows, a.shape, a.fresh[pl.slot], pl.old, part, pl.rows);
        return;
    }
    const int s = (int)(blockIdx.x / (unsigned)parts), part = (int)(blockIdx.x % (unsigned)parts);
    const Planned pl = plan[s];
    const bool copies = pl.old >= 0;
    if (!copies && pl.want <= pl.have) return;
    int32_t *row = a.t.table + s * a.t.ld;
    if (copies && part == 0 && threadIdx.x == 0) {
        const int page = a.fresh[pl.slot];
        row[pl.have - 1] = page;
        a.ref[page] = 1;
    }
    const int c0 = part * kCols, c1 = pl.want < c0 + kCols ? pl.want : c0 + kCols;
    for (int c = c0 + (int)threadIdx.x; c < c1; c += 256) {
        if (c < pl.have) continue;
        const int page = a.fresh[pl.slot + copies + c - pl.have];
        row[c] = page;
        a.ref[page] = 1;
    }
}

hipError_t launch_kv_resize(const KvResize &a, hipStream_t s) {
    const int parts = col_parts(a.t.cols), copy_parts = parts_of(a.shape);
    const unsigned rows = (unsigned)kv_table_groups(a.t.n_seqs, a.t.cols);
    if (rows) kv_drop<<<rows, 256, 0, s>>>(a, parts);
    if (a.t.n_seqs <= 1024) kv_plan<1><<<1, 1024, 0, s>>>(a);
    else kv_plan<kResizeMaxSeqs / 1024><<<1, 1024, 0, s>>>(a);
    if (rows) kv_take<<<rows + (unsigned)(a.t.n_seqs * copy_parts), 256, 0, s>>>(a, parts, copy_parts, rows);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------- compact

__device__ __forceinline__ uint32_t used_bits(const KvCompact &a, int w) {
    const uint32_t bits = ~a.free[w];
    return w == a.from_pages / 32 ? bits & ((1u << (a.from_pages % 32)) - 1u) : bits;   // (a last word that is not whole)
}

__global__ __launch_bounds__(1024) void kv_count(KvCompact a) {
    __shared__ int64_t tmp[16];
    const int words = (a.from_pages + 31) / 32;
    int64_t base = 0;
    for (int w0 = 0; w0 < words; w0 += 1024) {
        const int w = w0 + (int)threadIdx.x;
        int64_t all;
        const int64_t at = scan_1024(w < words ? __popc(used_bits(a, w)) : 0, tmp, all);
        if (w < words) a.before[w] = (int)(base + at);
        base += all;
    }
    if (threadIdx.x == 0) *a.n_used = (int)base;
}

// the new number of a page, -1 for one that is free or does not exist
__device__ __forceinline__ int moved(const KvCompact &a, int page) {
    if (page < 0 || page >= a.from_pages) return -1;
    const uint32_t bits = used_bits(a, page >> 5);
    if (!(bits >> (page & 31) & 1)) return -1;
    return a.before[page >> 5] + __popc(bits & ((1u << (page & 31)) - 1u));
}

__global__ __launch_bounds__(256) void kv_move(KvCompact a, int parts, int copy_parts, unsigned row_groups, unsigned page_groups) {
    const int n_used = *a.n_used;
    if (n_used > a.to_pages) return;
    unsigned b = blockIdx.x;
    if (b < row_groups) {                                        // a row of the table
        const int s = (int)(b / (unsigned)parts), part = (int)(b % (unsigned)parts);
        const int len = a.t.lens[s];
        const int n = bad_len(len, (int64_t)a.t.cols * a.shape.page.d) ? 0 : pages_of(a.shape.page, len);
        const int c1 = a.t.cols < (part + 1) * kCols ? a.t.cols : (part + 1) * kCols;
        for (int c = part * kCols + (int)threadIdx.x; c < c1; c += 256)
            a.to_table[s * a.ld_to + c] = c < n ? moved(a, a.t.table[s * a.t.ld + c]) : -1;
        return;
    }
    b -= row_groups;
    if (b < page_groups) {                                       // bits, and the counts of pages that none moves to
        const int page = (int)(b * 256 + threadIdx.x);
        if (page < (a.to_pages + 31) / 32) {
            const int left = n_used - page * 32, last = a.to_pages - page * 32;
            const uint32_t used = left >= 32 ? ~0u : left > 0 ? (1u << left) - 1u : 0u;
            a.to_free[page] = ~used & (last >= 32 ? ~0u : (1u << last) - 1u);
        }
        if (page >= n_used && page < a.to_pages) a.to_ref[page] = 0;
        return;
    }
    b -= page_groups;
    const int page = (int)(b / (unsigned)copy_parts), part = (int)(b % (unsigned)copy_parts);
    const int to = moved(a, page);
    if (to < 0) return;
    if (part == 0 && threadIdx.x == 0) a.to_ref[to] = a.ref[page];
    copy_part(a.to, a.from, a.shape, to, page, part, (int)a.shape.page.d);
}

hipError_t launch_kv_compact(const KvCompact &a, hipStream_t s) {
    kv_count<<<1, 1024, 0, s>>>(a);
    const int parts = col_parts(a.t.cols), copy_parts = parts_of(a.shape);
    const unsigned rows = (unsigned)kv_table_groups(a.t.n_seqs, a.t.cols), pages = ((unsigned)a.to_pages + 255u) / 256u;
    const unsigned groups = rows + pages + (unsigned)a.from_pages * (unsigned)copy_parts;
    if (groups) kv_move<<<groups, 256, 0, s>>>(a, parts, copy_parts, rows, pages);
    return hipGetLastError();
}

}  // namespace q2_0
