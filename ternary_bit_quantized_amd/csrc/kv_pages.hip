// Pages of a paged cache: copies, shared sequences, growing and shrinking ones, and a move into another pool.
//
// A pool of pages is a count of holders for each page and one bit for each that is free.  Everything here
// is whole numbers and copies, and comes out the same whatever the order in which workgroups run: pages
// come back by counts that only go down in one launch, and are taken in the order of their numbers
// by one workgroup in the next.
//
// resize  kv_drop   (a workgroup per 1024 columns of a row) the pages that shrinking sequences leave
//         kv_plan   (one workgroup) which growing sequences need a copy of a shared last page, how many pages
//                   that takes in all, and whether there are as many; of small tables kv_drop's and kv_list's parts too
//         kv_list   the pages that are taken
//         kv_take   the new entries of the rows, and the copies
// fork    kv_fork_plan (one workgroup) which pairs hold, and of small tables the rows and counts; else kv_fork_rows
// compact kv_count  (one workgroup, large pools) pages in use before each 32; kv_move everything else
//
// What bounds them: copies HBM (1024 pages of 64 tokens, 8 heads of 128, 537 MB read and written: 105 us, 5.1 TB/s, where a
// copy of 2 GiB runs at 4.9; 2100 pages of 64 KB of a pool of 6000: 56 us, 4.9 TB/s).  The tables' steps are dependent loads and
// counts of one workgroup, 5 to 7 us each: a step of 64 drafting sequences (two resizes) 12.4 to 16.7 us in a graph, of 32
// beams (two, a fork and 16 copies of a page) 27, of 256 sequences of which half come and go (68000 pages twice) 37.
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
    return launch(kv_copy_pages, (unsigned)kv_copy_groups(a.shape, a.n), 256, 0, s, a, parts_of(a.shape));
}

// ---------------------------------------------------------------------------- shared by rows of tables

constexpr int kCols = 1024;           // columns of a table row that a workgroup takes

static int col_parts(int64_t cols) { return (int)((cols + kCols - 1) / kCols); }

int64_t kv_table_groups(int64_t n_rows, int64_t cols) { return n_rows * col_parts(cols); }

// Sum over the workgroup of 1024 of the values of lower threads; `total`: of all.  Counts that may pass 2^31 are doubles (exact
// up to 2^53).
template <typename T>
__device__ __forceinline__ T scan_1024(T v, double *tmp, T &total) {
    T *sums = reinterpret_cast<T *>(tmp);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const T run = lanes_run(v);
    if (lane == 63) sums[wave] = run;
    __syncthreads();
    T base = 0, all = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
        if (w == wave) base = all;
        all += sums[w];
    }
    __syncthreads();
    total = all;
    return base + run - v;
}

// One workgroup of 1024 goes through `count` things of each of up to 1024 * PT owners, thread t's being PT in a row from t * PT, as
// one list, eight at a time a thread: f(owner, i, in) for things i < count of their owners where in.  (One at a time the
// loads and counts of each wait for the one before.)  `ends` holds 1024 * PT numbers in shared memory.
constexpr int kAtOnce = 8;
template <int PT, typename F>
__device__ __forceinline__ void each_of(const int (&count)[PT], int *ends, double *tmp, F &&f) {
    int sum = 0, total;              // (of a small table)
#pragma unroll
    for (int i = 0; i < PT; ++i) sum += count[i];
    int at = scan_1024(sum, tmp, total);
    if (total == 0) return;                                      // (uniform)
#pragma unroll
    for (int i = 0; i < PT; ++i) {
        at += count[i];
        ends[threadIdx.x * PT + i] = at;
    }
    __syncthreads();
    for (int from = 0; from < total; from += 1024 * kAtOnce) {
        int owner[kAtOnce], thing[kAtOnce];
        bool in[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            const int e = from + 1024 * k + (int)threadIdx.x;
            in[k] = e < total;
            owner[k] = thing[k] = 0;
            if (from + 1024 * k >= total) continue;         // (uniform)
            int lo = 0;                                          // owners that end at or before e
#pragma unroll
            for (int step = 512 * PT; step >= 1; step >>= 1)
                if (ends[lo + step - 1] <= e) lo += step;
            owner[k] = in[k] ? lo : 0;
            thing[k] = in[k] ? e - (lo ? ends[lo - 1] : 0) : 0;
        }
        f(owner, thing, in);
    }
}

// Tables of up to this many entries are left to the one workgroup that plans, two launches less of a resize and one of a fork.
// Measured in a graph: two calls for 64 sequences of 48000 entries in all that change 40 of them take 19.2 us so, 23.0 with
// kv_drop and kv_list, and eager calls 6 us less of the host.  One that changes much is slower: 8000 pages given back and
// taken 73 us against 31, 32000 of them 236 against 40 (a CU does an atomic in some 7 cycles).  Steps that change a few
// pages are the rule, and a sequence that ends is one of many.
constexpr int64_t kOneGroup = 65536;

// ---------------------------------------------------------------------------- fork

template <bool ROWS>
__global__ __launch_bounds__(1024) void kv_fork_plan(KvFork a) {
    __shared__ double tmp[16];
    __shared__ int ends[1024];
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
    if (!ROWS) return;
    // (a thread has written what it reads here: n <= 1024)
    const int len = (int)threadIdx.x < a.n ? a.plan[threadIdx.x] : 0;
    const int count[1] = {len > 0 ? pages_of(a.page, len) : 0};
    each_of<1>(count, ends, tmp, [&](const int (&i)[kAtOnce], const int (&c)[kAtOnce], const bool (&in)[kAtOnce]) {
        int page[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
            if (in[k]) page[k] = a.t.table[a.src[i[k]] * a.t.ld + c[k]];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k)
            if (in[k]) {
                a.t.table[a.dst[i[k]] * a.t.ld + c[k]] = page[k];
                if (page[k] >= 0 && page[k] < a.n_pages) atomicAdd(a.ref + page[k], 1);
            }
    });
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
    if (a.n <= 1024 && (int64_t)a.n * a.t.cols <= kOneGroup) return launch(kv_fork_plan<true>, 1, 1024, 0, s, a);
    const hipError_t e = launch(kv_fork_plan<false>, 1, 1024, 0, s, a);
    if (e != hipSuccess || a.t.cols == 0) return e;              // (nothing runs on a plan that was not made)
    return launch(kv_fork_rows, (unsigned)kv_table_groups(a.n, a.t.cols), 256, 0, s, a, col_parts(a.t.cols));
}

// ---------------------------------------------------------------------------- resize

__device__ __forceinline__ void drop_page(const KvResize &a, int32_t *entry) {
    const int page = *entry;
    *entry = -1;
    if (page >= 0 && page < a.n_pages && atomicSub(a.ref + page, 1) == 1) atomicOr(a.free + (page >> 5), 1u << (page & 31));
}

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
        drop_page(a, row + c);
    }
}

__device__ __forceinline__ uint32_t free_bits(const KvResize &a, int w) {
    const uint32_t bits = (uint32_t)peek(reinterpret_cast<const int32_t *>(a.free) + w);
    return w == a.n_pages / 32 ? bits & ((1u << (a.n_pages % 32)) - 1u) : bits;   // (a last word that is not whole)
}

// A word's free pages from place `at` of the list on, as far as `take`; all lanes.  Two words at a time, a lane a bit, a wave
// writes their pages next to each other (a thread a word wrote 64 lines at once: 68000 pages 41 us in one workgroup, 22 so).
__device__ __forceinline__ void list_word(const KvResize &a, int w, uint32_t bits, int at, int take) {
    const int lane = threadIdx.x & 63;
    at = at < take ? at : take;
    const uint64_t some = __ballot(bits && at < take);
    if (!some) return;
#pragma unroll 4
    for (int j = 0; j < 64; j += 2) {
        if (!(some >> j & 3)) continue;                          // (uniform)
        const int from = j + (lane >> 5), bit = lane & 31;
        const uint32_t theirs = (uint32_t)__shfl((int)bits, from);
        const int place = __shfl(at, from) + __popc(theirs & ((1u << bit) - 1u));
        if ((theirs >> bit & 1) && place < take) a.fresh[place] = (w - lane + from) * 32 + bit;
    }
    if (bits && at < take) {
        uint32_t stay = 0;                                       // (without the lowest ones, as many as are taken)
        if (__popc(bits) > take - at) {
            stay = bits;
            for (int n = take - at; n > 0; --n) stay &= stay - 1;
        }
        put(reinterpret_cast<int32_t *>(a.free) + w, (int)stay);
    }
}

constexpr int kHeldWords = 6144;      // 196608 pages: 24 KB

struct Planned {
    int slot, have, want, old, rows, pad[3];
};
static_assert(sizeof(Planned) == 32, "8 numbers a sequence");

// A sequence that grows from inside a page that others hold too takes a copy of it -- unless all holders do so in this
// call: then the lowest of them keeps the page.  Holders leave by counting down; where that ends at 0, the lowest
// claim on the count is the one that stays.
template <int PT, bool DROP>
__global__ __launch_bounds__(1024) void kv_plan(KvResize a) {
    __shared__ double tmp[16];
    __shared__ int ends[DROP ? 1024 * PT : 1];
    __shared__ uint32_t held[kHeldWords];
    const int64_t most = (int64_t)a.t.cols * a.shape.page.d;
    const int tid = threadIdx.x;
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
    }
    if (DROP) {
        int count[PT];
#pragma unroll
        for (int i = 0; i < PT; ++i)
            count[i] = now[i] < len[i] ? pages_of(a.shape.page, len[i]) - pages_of(a.shape.page, now[i]) : 0;
        each_of<PT>(count, ends, tmp, [&](const int (&s)[kAtOnce], const int (&i)[kAtOnce], const bool (&in)[kAtOnce]) {
            int32_t *entry[kAtOnce];
            int page[kAtOnce], held[kAtOnce];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                if (!in[k]) continue;
                entry[k] = a.t.table + s[k] * a.t.ld + pages_of(a.shape.page, a.new_lens[s[k]]) + i[k];
                page[k] = *entry[k];
            }
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                held[k] = 0;
                if (!in[k]) continue;
                *entry[k] = -1;
                if (page[k] >= 0 && page[k] < a.n_pages) held[k] = atomicSub(a.ref + page[k], 1);
            }
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k)
                if (held[k] == 1) atomicOr(a.free + (page[k] >> 5), 1u << (page[k] & 31));
        });
        all_done();
    }
    // the pages that growing sequences are inside of, and the free ones: asked for together
    int tail[PT];
#pragma unroll
    for (int i = 0; i < PT; ++i) {
        const int s = tid * PT + i;
        const bool ok = !bad_len(len[i], most);
        grows[i] = now[i] > len[i];
        pl[i].have = ok ? pages_of(a.shape.page, len[i]) : 0;
        pl[i].want = grows[i] ? pages_of(a.shape.page, now[i]) : pl[i].have;
        pl[i].rows = ok && pl[i].have > 0 ? len[i] - (pl[i].have - 1) * (int)a.shape.page.d : 0;
        pl[i].old = -1;
        tail[i] = grows[i] && pl[i].rows > 0 && pl[i].rows < (int)a.shape.page.d ? a.t.table[s * a.t.ld + pl[i].have - 1] : -1;
    }
    const int words = (a.n_pages + 31) / 32;
    uint32_t bits[kHeldWords / 1024];
#pragma unroll
    for (int j = 0; j < kHeldWords / 1024; ++j) bits[j] = j * 1024 + tid < words ? free_bits(a, j * 1024 + tid) : 0u;
#pragma unroll
    for (int i = 0; i < PT; ++i) {
        count[i] = 0;
        if (tail[i] >= 0 && tail[i] < a.n_pages) pl[i].old = tail[i], count[i] = peek(a.ref + tail[i]);
        shared[i] = count[i] > 1;
    }
    int some = 0;                                                // (the bits stay in shared memory for the list, as far as that reaches)
#pragma unroll
    for (int j = 0; j < kHeldWords / 1024; ++j) {
        held[j * 1024 + tid] = bits[j];
        some += __popc(bits[j]);
    }
    for (int w = kHeldWords + tid; w < words; w += 1024) some += __popc(free_bits(a, w));
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
    double need = 0.0, total;
#pragma unroll
    for (int i = 0; i < PT; ++i) need += (double)(pl[i].want - pl[i].have + (shared[i] && !keeps[i]));
    const double before = scan_1024(need, tmp, total);
    int avail;
    scan_1024(some, tmp, avail);
    const bool enough = total <= (double)avail;
    if (tid == 0) *a.missing = enough ? 0 : total - avail < 2147483647.0 ? (int)(total - avail) : 2147483647;
    int slot = enough ? (int)before : 0;                         // (at most n_pages)
#pragma unroll
    for (int i = 0; i < PT; ++i) {
        const int s = tid * PT + i;
        const bool copies = shared[i] && !keeps[i];
        if (keeps[i]) put(a.ref + pl[i].old, enough ? 1 : count[i]);
        if (copies && left[i] > 0 && !enough) atomicAdd(a.ref + pl[i].old, 1);
        if (s >= a.t.n_seqs) continue;
        if (now[i] != len[i] && (enough || !grows[i])) a.t.lens[s] = now[i];
        pl[i].slot = slot;
        if (enough) slot += pl[i].want - pl[i].have + copies;
        if (!copies || !enough) pl[i].old = -1;
        if (!enough) pl[i].want = pl[i].have;
        reinterpret_cast<Planned *>(a.plan)[s] = pl[i];
    }
    // the free pages of the lowest numbers, `total` of them
    const int take = enough ? (int)total : 0;                    // (at most n_pages)
    if (!DROP && tid == 0) a.before[words] = take;
    int base = 0, reached = 0;
    for (int w0 = 0; base < take && w0 < words; w0 += 1024) {
        const int w = w0 + tid;
        const uint32_t bits = w0 < kHeldWords ? held[w] : w < words ? free_bits(a, w) : 0u;
        int all;
        const int at = base + scan_1024((int)__popc(bits), tmp, all);
        if (DROP) list_word(a, w, bits, at, take);
        else if (w < words) a.before[w] = at;
        base += all;
        reached = w0 + 1024;
    }
    if (!DROP && tid == 0) a.before[words + 1] = reached;
}

// Large tables: the list by as many workgroups as the bits fill.
__global__ __launch_bounds__(256) void kv_list(KvResize a) {
    const int words = (a.n_pages + 31) / 32, w = (int)(blockIdx.x * 256 + threadIdx.x), take = a.before[words];
    const bool in = w < words && w < a.before[words + 1];
    list_word(a, w, in ? free_bits(a, w) : 0u, in ? a.before[w] : take, take);
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
    const bool one = (int64_t)a.t.n_seqs * a.t.cols <= kOneGroup;
    constexpr int kMany = kResizeMaxSeqs / 1024;
    hipError_t e = hipSuccess;                                   // nothing runs after a launch that failed
    if (!one && (e = launch(kv_drop, rows, 256, 0, s, a, parts)) != hipSuccess) return e;
    if (a.t.n_seqs <= 1024) e = launch(one ? kv_plan<1, true> : kv_plan<1, false>, 1, 1024, 0, s, a);
    else e = launch(one ? kv_plan<kMany, true> : kv_plan<kMany, false>, 1, 1024, 0, s, a);
    if (e != hipSuccess) return e;
    if (!one && (e = launch(kv_list, ((unsigned)a.n_pages / 32u + 256u) / 256u, 256, 0, s, a)) != hipSuccess) return e;
    if (rows == 0) return hipSuccess;
    return launch(kv_take, rows + (unsigned)(a.t.n_seqs * copy_parts), 256, 0, s, a, parts, copy_parts, rows);
}

// ---------------------------------------------------------------------------- compact

__device__ __forceinline__ uint32_t used_bits(const KvCompact &a, int w) {
    const uint32_t bits = ~a.free[w];
    return w == a.from_pages / 32 ? bits & ((1u << (a.from_pages % 32)) - 1u) : bits;   // (a last word that is not whole)
}

__global__ __launch_bounds__(1024) void kv_count(KvCompact a) {
    __shared__ double tmp[16];
    const int words = (a.from_pages + 31) / 32;
    int base = 0;
    for (int w0 = 0; w0 < words; w0 += 1024) {
        const int w = w0 + (int)threadIdx.x;
        int all;
        const int at = scan_1024(w < words ? (int)__popc(used_bits(a, w)) : 0, tmp, all);
        if (w < words) a.before[w] = base + at;
        base += all;
    }
    if (threadIdx.x == 0) *a.n_used = base;
}

// The new number of a page in use: pages in use before it.
__device__ __forceinline__ bool in_use(const KvCompact &a, int page) {
    return page >= 0 && page < a.from_pages && used_bits(a, page >> 5) >> (page & 31) & 1;
}
__device__ __forceinline__ int moved(const KvCompact &a, int page, const int32_t *before) {
    return before[page >> 5] + __popc(used_bits(a, page >> 5) & ((1u << (page & 31)) - 1u));
}

// A workgroup of 256 counts for itself: pages in use before each word (all != nullptr) or before word `upto`; returns all.
__device__ __forceinline__ int count_256(const KvCompact &a, int upto, int32_t *all, int *before, int *tmp) {
    const int words = (a.from_pages + 31) / 32, each = (words + 255) / 256;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int w0 = (int)threadIdx.x * each, w1 = w0 + each < words ? w0 + each : words;
    int own = 0, low = 0;
    for (int w = w0; w < w1; ++w) {
        const int n = __popc(used_bits(a, w));
        own += n;
        low += w < upto ? n : 0;
    }
    int run = own;
    if (all) {
        run = lanes_run(run);
    } else {
        run = lanes_run(run), low = lanes_run(low);              // (the last lane's are the wave's)
    }
    if (lane == 63) tmp[wave] = run, tmp[4 + wave] = low;
    __syncthreads();
    if (all) {
        int at = run - own;
        for (int w = 0; w < wave; ++w) at += tmp[w];
        for (int w = w0; w < w1; ++w) {
            all[w] = at;
            at += __popc(used_bits(a, w));
        }
        __syncthreads();
    } else {
        *before = tmp[4] + tmp[5] + tmp[6] + tmp[7];
    }
    return tmp[0] + tmp[1] + tmp[2] + tmp[3];
}

// Pools of up to this many pages (a word of bits a thread) are counted by every workgroup anew, a launch less: of 6000 pages
// 2100 of 64 KB move in 47.1 us so, in 49.8 after kv_count; of 16000 pages 5600 of 16 KB in 34.7 and 33.2.
constexpr int kCountPages = 8192;

template <bool COUNT>
__global__ __launch_bounds__(256) void kv_move(KvCompact a, int parts, int copy_parts, unsigned row_groups, unsigned page_groups) {
    __shared__ int32_t mine[COUNT ? kCountPages / 32 : 1];
    __shared__ int tmp[8];
    unsigned b = blockIdx.x;
    if (b >= row_groups + page_groups) {
        b -= row_groups + page_groups;
        const int page = (int)(b / (unsigned)copy_parts), part = (int)(b % (unsigned)copy_parts);
        if (!in_use(a, page)) return;
        int to, n_used;
        if (COUNT) {
            int before;
            n_used = count_256(a, page >> 5, nullptr, &before, tmp);
            to = before + __popc(used_bits(a, page >> 5) & ((1u << (page & 31)) - 1u));
        } else {
            n_used = *a.n_used;
            to = moved(a, page, a.before);
        }
        if (n_used > a.to_pages) return;
        if (part == 0 && threadIdx.x == 0) a.to_ref[to] = a.ref[page];
        copy_part(a.to, a.from, a.shape, to, page, part, (int)a.shape.page.d);
        return;
    }
    int before;
    const int n_used = COUNT ? count_256(a, 0, mine, &before, tmp) : *a.n_used;
    if (COUNT && b == row_groups + page_groups - 1 && threadIdx.x == 0) *a.n_used = n_used;
    if (n_used > a.to_pages) return;
    if (b < row_groups) {                                        // a row of the table
        const int s = (int)(b / (unsigned)parts), part = (int)(b % (unsigned)parts);
        const int len = a.t.lens[s];
        const int n = bad_len(len, (int64_t)a.t.cols * a.shape.page.d) ? 0 : pages_of(a.shape.page, len);
        const int c1 = a.t.cols < (part + 1) * kCols ? a.t.cols : (part + 1) * kCols;
        for (int c = part * kCols + (int)threadIdx.x; c < c1; c += 256) {
            const int page = c < n ? a.t.table[s * a.t.ld + c] : -1;
            a.to_table[s * a.ld_to + c] = in_use(a, page) ? moved(a, page, COUNT ? mine : a.before) : -1;
        }
        return;
    }
    b -= row_groups;                                             // bits, and the counts of pages that none moves to
    const int page = (int)(b * 256 + threadIdx.x);
    if (page < (a.to_pages + 31) / 32) {
        const int left = n_used - page * 32, last = a.to_pages - page * 32;
        const uint32_t used = left >= 32 ? ~0u : left > 0 ? (1u << left) - 1u : 0u;
        a.to_free[page] = ~used & (last >= 32 ? ~0u : (1u << last) - 1u);
    }
    if (page >= n_used && page < a.to_pages) a.to_ref[page] = 0;
}

hipError_t launch_kv_compact(const KvCompact &a, hipStream_t s) {
    const int parts = col_parts(a.t.cols), copy_parts = parts_of(a.shape);
    const unsigned rows = (unsigned)kv_table_groups(a.t.n_seqs, a.t.cols);
    const unsigned pages = a.to_pages ? ((unsigned)a.to_pages + 255u) / 256u : 1u;    // (one writes n_used)
    const unsigned groups = rows + pages + (unsigned)a.from_pages * (unsigned)copy_parts;
    if (a.from_pages <= kCountPages) return launch(kv_move<true>, groups, 256, 0, s, a, parts, copy_parts, rows, pages);
    const hipError_t e = launch(kv_count, 1, 1024, 0, s, a);
    if (e != hipSuccess) return e;
    return launch(kv_move<false>, groups, 256, 0, s, a, parts, copy_parts, rows, pages);
}

}  // namespace q2_0
