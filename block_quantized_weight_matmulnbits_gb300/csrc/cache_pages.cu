// The pages of a paged key / value cache: copy, fork, resize (grow and free)
// and compact, on reference counts, page tables and lengths that live on the
// device.
//
// Which page a sequence gets decides what a later step reads, so nothing may
// depend on the order in which threads run: free pages are taken by number
// (a prefix count over refs == 0), lists are handled as one parallel step on
// the state before the call, and the only atomics are integer additions to
// reference counts.  The bookkeeping is a few thousand integers: one cluster
// of 8 CTAs does it, because its phases (count, choose, write) need a barrier
// between them and a cluster has one without another launch.
//
// The pages themselves are moved by a second kernel, a programmatic dependent
// of the first, that reads the (source, destination) list the first one wrote.
// It is bound by DRAM: 2 * page bytes * planes for each pair (700 pages of 32 KB
// in 32 planes: 233 us, 6310 GB/s; a compaction that moves 716 pages of 16 KB:
// 130 us, 5760 GB/s, the bookkeeping before the copy included).  A warp moves 4 KB
// at a time, eight 16-byte loads per lane before the first store, which keeps
// about 128 KB in flight on an SM.
#include "decoder.h"

namespace mnb {
namespace {

constexpr int kCluster = 8;                // CTAs of the bookkeeping kernels, at most
constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int64_t kMaxSeqs = 262144;      // one bit each in shared memory
constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 8;              // 16-byte vectors a lane holds
constexpr int64_t kChunk = 32 * 16 * kCopyVecs;

struct State {
    int32_t* refs;
    int32_t* tables;
    int32_t* lens;
    int num_pages, num_seqs, stride, page_size;
};

// Workspace (int32): 64 counters, then the arrays below.
struct Work {
    int32_t* count;   // [64]: counters of the CTAs, the total need, the pairs to copy
    int32_t* meta;    // [num_seqs]: first free rank of a growing sequence, * 2 + 1 if its last page splits
    int32_t* len;     // [num_seqs]: staged lengths
    int32_t* src;     // [max(num_seqs, num_pages)]: pages to copy
    int32_t* dst;
    int32_t* pick;    // [num_pages]: free pages by rank; page names of a compaction
    int32_t* rows;    // [num_seqs * stride]: staged table rows
};

size_t work_ints(int64_t pages, int64_t seqs, int64_t stride) {
    const int64_t list = pages > seqs ? pages : seqs;
    return (size_t)(64 + 2 * seqs + 2 * list + pages + seqs * stride);
}

Work make_work(void* ws, const mnb_cache_state* s) {
    const int64_t list = s->num_pages > s->num_seqs ? s->num_pages : s->num_seqs;
    Work w;
    w.count = static_cast<int32_t*>(ws);
    w.meta = w.count + 64;
    w.len = w.meta + s->num_seqs;
    w.src = w.len + s->num_seqs;
    w.dst = w.src + list;
    w.pick = w.dst + list;
    w.rows = w.pick + s->num_pages;
    return w;
}

__device__ __forceinline__ int cluster_size() {
    int n;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
    return n;
}

// The meeting of a call's CTAs: the cluster's barrier, or the CTA's own.
__device__ __forceinline__ void meet(int peers) {
    if (peers > 1) cluster_sync();
    else __syncthreads();
}

__device__ __forceinline__ int pages_of(int len, int page_size) { return len / page_size + (len % page_size != 0); }

// Exclusive prefix of v over the block's threads, and the block's sum.
__device__ __forceinline__ int block_prefix(int v, int* total) {
    __shared__ int part[kWarps];
    __shared__ int sum;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(~0u, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) part[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int y = part[lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int z = __shfl_up_sync(~0u, y, d);
            if (lane >= d) y += z;
        }
        if (lane == 31) sum = y;
        part[lane] = y;
    }
    __syncthreads();
    const int before = warp ? part[warp - 1] : 0;
    *total = sum;
    __syncthreads();
    return before + x - v;
}

// True if an index of the list is out of range or named twice, or a length of
// the state does not fit its row.  Every CTA looks at the whole list, so all
// of them agree without a barrier.  bits: num_seqs bits of shared memory.
__device__ bool bad_list(const State& s, const int32_t* src, const int32_t* dst, const int32_t* new_lens, int n,
                         uint32_t* bits) {
    for (int i = threadIdx.x; i < (s.num_seqs + 31) / 32; i += kThreads) bits[i] = 0;
    __syncthreads();
    const int64_t most = (int64_t)s.stride * s.page_size;
    int bad = 0;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int b = dst[i];
        if ((unsigned)b >= (unsigned)s.num_seqs) {
            bad = 1;
            continue;
        }
        if (atomicOr(&bits[b >> 5], 1u << (b & 31)) & (1u << (b & 31))) bad = 1;
        if (s.lens[b] < 0 || s.lens[b] > most) bad = 1;
        if (new_lens && (new_lens[i] < 0 || new_lens[i] > most)) bad = 1;
        if (src) {
            const int a = src[i];
            if ((unsigned)a >= (unsigned)s.num_seqs || s.lens[a] < 0 || s.lens[a] > most) bad = 1;
        }
    }
    return __syncthreads_or(bad) != 0;
}

__device__ __forceinline__ void add_ref(const State& s, int page, int v) {
    if ((unsigned)page < (unsigned)s.num_pages) atomicAdd(&s.refs[page], v);
}

__global__ void __launch_bounds__(kThreads) fork_kernel(const State s, const Work w, const int32_t* src,
                                                        const int32_t* dst, int n, int* status) {
    extern __shared__ uint32_t bits[];
    griddep_wait();
    const int rank = (int)cluster_ctarank(), peers = cluster_size(), lane = threadIdx.x & 31;
    if (bad_list(s, src, dst, nullptr, n, bits)) {
        if (rank == 0 && threadIdx.x == 0) set_status(status, MNB_ERR_INVALID_ARG);
        return;
    }
    // a warp takes 32 columns of one pair's rows at a time
    const int cols = (s.stride + 31) / 32;
    const int64_t units = (int64_t)n * cols;
    const int first = rank * kWarps + (threadIdx.x >> 5);
    for (int64_t u = first; u < units; u += peers * kWarps) {
        const int i = (int)(u / cols), c = (int)(u - (int64_t)i * cols) * 32 + lane;
        const int a = src[i], b = dst[i], len = s.lens[a];
        if (c == 0) w.len[i] = len;
        if (c < pages_of(len, s.page_size)) {
            const int page = s.tables[(int64_t)a * s.stride + c];
            w.rows[(int64_t)i * s.stride + c] = page;
            add_ref(s, page, 1);
        }
        if (c < pages_of(s.lens[b], s.page_size)) add_ref(s, s.tables[(int64_t)b * s.stride + c], -1);
    }
    meet(peers);  // every row staged before one is written
    for (int64_t u = first; u < units; u += peers * kWarps) {
        const int i = (int)(u / cols), c = (int)(u - (int64_t)i * cols) * 32 + lane;
        if (c >= s.stride) continue;
        const int held = pages_of(w.len[i], s.page_size);
        s.tables[(int64_t)dst[i] * s.stride + c] = c < held ? w.rows[(int64_t)i * s.stride + c] : -1;
        if (c == 0) s.lens[dst[i]] = w.len[i];
    }
}

// The pages [lo, hi) of this CTA when num_pages are split over the cluster.
__device__ __forceinline__ void segment(int pages, int rank, int peers, int* lo, int* hi) {
    const int per = ((pages + peers - 1) / peers + 3) & ~3;
    *lo = min(pages, rank * per);
    *hi = min(pages, *lo + per);
}

template <typename F>
__device__ __forceinline__ int count_if(int lo, int hi, F f) {
    int c = 0;
    for (int i = lo + threadIdx.x; i < hi; i += kThreads) c += f(i) ? 1 : 0;
    int total;
    block_prefix(c, &total);
    return total;
}

// f(i) of the items [lo, hi) that pass get their rank (base + items before them): put(i, rank).
template <typename F, typename P>
__device__ __forceinline__ void rank_if(int lo, int hi, int base, int most, F f, P put) {
    for (int at = lo; at < hi && base < most; at += kThreads) {
        const int i = at + threadIdx.x;
        const int ok = i < hi && f(i) ? 1 : 0;
        int total;
        const int before = block_prefix(ok, &total);
        if (ok && base + before < most) put(i, base + before);
        base += total;
    }
}

__global__ void __launch_bounds__(kThreads) resize_kernel(const State s, const Work w, const int32_t* seqs,
                                                          const int32_t* new_lens, int n, int has_planes, int* status) {
    extern __shared__ uint32_t bits[];
    griddep_wait();
    const int rank = (int)cluster_ctarank(), peers = cluster_size(), lane = threadIdx.x & 31;
    if (rank == 0)
        for (int i = threadIdx.x; i < n; i += kThreads) w.src[i] = -1;  // nothing to copy yet
    if (bad_list(s, nullptr, seqs, new_lens, n, bits)) {
        if (rank == 0 && threadIdx.x == 0) set_status(status, MNB_ERR_INVALID_ARG);
        return;
    }
    int lo, hi;
    segment(s.num_pages, rank, peers, &lo, &hi);
    const int free_here = count_if(lo, hi, [&](int p) { return s.refs[p] == 0; });
    if (threadIdx.x == 0) w.count[rank] = free_here;
    if (rank == 0) {  // need of each sequence, and the free rank it starts at
        int base = 0, unsplittable = 0;
        for (int at = 0; at < n; at += kThreads) {
            const int i = at + threadIdx.x;
            int need = 0, split = 0;
            if (i < n) {
                const int old = s.lens[seqs[i]], len = new_lens[i];
                const int had = pages_of(old, s.page_size), want = pages_of(len, s.page_size);
                if (len > old && old % s.page_size != 0) {
                    const int last = s.tables[(int64_t)seqs[i] * s.stride + had - 1];
                    split = (unsigned)last < (unsigned)s.num_pages && s.refs[last] > 1;
                }
                need = max(0, want - had) + split;
                unsplittable |= split && !has_planes;
            }
            int total;
            const int before = block_prefix(need, &total);
            if (i < n) w.meta[i] = (int)((unsigned)(base + before) * 2u) + split;  // read only if the need can be met
            base += total;
        }
        unsplittable = __syncthreads_or(unsplittable);
        if (threadIdx.x == 0) {
            w.count[16] = base;
            w.count[17] = unsplittable;
        }
    }
    meet(peers);
    int before = 0, all = 0;
    for (int r = 0; r < peers; ++r) {
        const int c = w.count[r];
        before += r < rank ? c : 0;
        all += c;
    }
    const int need = w.count[16];
    if (w.count[17] || need > all) {
        if (rank == 0 && threadIdx.x == 0) set_status(status, w.count[17] ? MNB_ERR_INVALID_ARG : MNB_ERR_NO_MEM);
        return;
    }
    rank_if(lo, hi, before, need, [&](int p) { return s.refs[p] == 0; }, [&](int p, int k) { w.pick[k] = p; });
    meet(peers);
    // one warp per sequence
    for (int i = rank * kWarps + (int)(threadIdx.x >> 5); i < n; i += peers * kWarps) {
        const int b = seqs[i], len = new_lens[i], old = s.lens[b];
        const int had = pages_of(old, s.page_size), want = pages_of(len, s.page_size);
        const int split = w.meta[i] & 1, k0 = w.meta[i] >> 1, start = had - split;
        int32_t* row = s.tables + (int64_t)b * s.stride;
        if (split && lane == 0) {
            w.dst[i] = w.pick[k0];
            w.src[i] = row[had - 1];
            atomicAdd(&s.refs[row[had - 1]], -1);
        }
        __syncwarp();
        if (split || want > had) {
            for (int c = start + lane; c < want; c += 32) {
                const int page = w.pick[k0 + c - start];
                row[c] = page;
                s.refs[page] = 1;
            }
        }
        for (int c = want + lane; c < had; c += 32) {
            add_ref(s, row[c], -1);
            row[c] = -1;
        }
        __syncwarp();
        if (lane == 0) s.lens[b] = len;
    }
}

__global__ void __launch_bounds__(kThreads) compact_kernel(const State s, const Work w, int32_t* refs_out,
                                                           int32_t* counts) {
    griddep_wait();
    const int rank = (int)cluster_ctarank(), peers = cluster_size();
    int lo, hi;
    segment(s.num_pages, rank, peers, &lo, &hi);
    auto used = [&](int p) { return s.refs[p] > 0; };
    const int here = count_if(lo, hi, used);
    if (threadIdx.x == 0) w.count[rank] = here;
    meet(peers);
    int live = 0;
    for (int r = 0; r < peers; ++r) live += w.count[r];
    auto moves = [&](int p) { return p >= live && s.refs[p] > 0; };
    auto hole = [&](int p) { return p < live && s.refs[p] <= 0; };
    const int n_src = count_if(lo, hi, moves), n_dst = count_if(lo, hi, hole);
    if (threadIdx.x == 0) {
        w.count[16 + rank] = n_src;
        w.count[32 + rank] = n_dst;
    }
    meet(peers);
    int b_src = 0, b_dst = 0, moved = 0;
    for (int r = 0; r < peers; ++r) {
        b_src += r < rank ? w.count[16 + r] : 0;
        b_dst += r < rank ? w.count[32 + r] : 0;
        moved += w.count[16 + r];
    }
    rank_if(lo, hi, b_src, 0x7FFFFFFF, moves, [&](int p, int k) { w.src[k] = p; });
    rank_if(lo, hi, b_dst, 0x7FFFFFFF, hole, [&](int p, int k) { w.dst[k] = p; });
    for (int p = lo + threadIdx.x; p < hi; p += kThreads) {
        if (!moves(p)) {
            w.pick[p] = p;
            if (!hole(p) && refs_out != s.refs) refs_out[p] = p < live ? s.refs[p] : 0;
        }
    }
    if (rank == 0 && threadIdx.x == 0) {
        w.count[48] = moved;
        counts[0] = live;
        counts[1] = moved;
    }
    meet(peers);
    // refs_out may be refs: each pair reads its source and writes both of its places itself
    for (int k = rank * kThreads + threadIdx.x; k < moved; k += peers * kThreads) {
        const int from = w.src[k], to = w.dst[k];
        w.pick[from] = to;
        refs_out[to] = s.refs[from];
        refs_out[from] = 0;
    }
}

struct CopyParams {
    uint8_t* base;
    int64_t plane_stride, page_stride, page_bytes;
    int planes, num_pages, chunks;   // chunks of kChunk bytes a page has (the last may be short)
    const int32_t* src;
    const int32_t* dst;
    const int32_t* count;            // device pair count, or null
    int64_t n;                       // pair count, or its bound
    int own_list;                    // the list is this file's: a source of -1 means no copy
    int* status;
    // renaming of table entries (mnb_cache_compact), or name == null
    const int32_t* name;
    const int32_t* tables;
    const int32_t* lens;
    int32_t* tables_out;
    int num_seqs, stride, page_size;
};

__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const CopyParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t warp = (int64_t)blockIdx.x * (kCopyThreads / 32) + (threadIdx.x >> 5);
    const int64_t warps = (int64_t)gridDim.x * (kCopyThreads / 32);
    if (p.name) {
        const int cols = (p.stride + 31) / 32;
        for (int64_t u = warp; u < (int64_t)p.num_seqs * cols; u += warps) {
            const int b = (int)(u / cols), c = (int)(u - (int64_t)b * cols) * 32 + lane;
            if (c >= p.stride) continue;
            const int64_t at = (int64_t)b * p.stride + c;
            int page = p.tables[at];
            if (c < pages_of(max(0, p.lens[b]), p.page_size) && (unsigned)page < (unsigned)p.num_pages) page = p.name[page];
            p.tables_out[at] = page;
        }
    }
    const int64_t n = p.count ? *p.count : p.n;
    const int64_t per_pair = (int64_t)p.planes * p.chunks;
    for (int64_t u = warp; u < n * per_pair; u += warps) {
        const int64_t i = u / per_pair;
        const int r = (int)(u - i * per_pair);
        const int plane = r / p.chunks, chunk = r - plane * p.chunks;
        const int from = p.src[i];
        if (p.own_list && from < 0) continue;
        const int to = p.dst[i];
        if ((unsigned)from >= (unsigned)p.num_pages || (unsigned)to >= (unsigned)p.num_pages) {
            if (lane == 0) set_status(p.status, MNB_ERR_INVALID_ARG);
            continue;
        }
        uint8_t* plane_base = p.base + (int64_t)plane * p.plane_stride;
        const int64_t off = chunk * kChunk + lane * 16;
        const uint8_t* a = plane_base + (int64_t)from * p.page_stride + off;
        uint8_t* b = plane_base + (int64_t)to * p.page_stride + off;
        uint4 v[kCopyVecs];
#pragma unroll
        for (int j = 0; j < kCopyVecs; ++j)
            if (off + j * 512 < p.page_bytes) v[j] = *reinterpret_cast<const uint4*>(a + j * 512);
#pragma unroll
        for (int j = 0; j < kCopyVecs; ++j)
            if (off + j * 512 < p.page_bytes) *reinterpret_cast<uint4*>(b + j * 512) = v[j];
    }
}

bool valid_planes(const mnb_page_planes* p) {
    const int64_t most = int64_t(1) << 62;
    return p && p->base && dec::aligned_to(p->base, 16) && p->num_planes >= 1 && p->num_planes <= 65535 &&
           p->num_pages >= 1 && p->num_pages < (int64_t(1) << 31) && p->page_bytes >= 16 && p->page_bytes % 16 == 0 &&
           p->page_bytes < (int64_t(1) << 31) && p->page_stride >= p->page_bytes && p->page_stride % 16 == 0 &&
           p->page_stride <= most / p->num_pages && p->plane_stride >= 0 && p->plane_stride % 16 == 0 &&
           p->plane_stride <= most / p->num_planes &&
           // planes do not overlap: one page's copy touches no other
           (p->num_planes == 1 || p->plane_stride >= p->page_stride * (p->num_pages - 1) + p->page_bytes ||
            (p->plane_stride >= p->page_bytes && p->page_stride >= p->plane_stride * (p->num_planes - 1) + p->page_bytes));
}

bool valid_counts(int64_t pages, int64_t seqs, int64_t stride) {
    return pages >= 1 && pages < (int64_t(1) << 30) && seqs >= 1 && seqs <= kMaxSeqs && stride >= 1 &&
           stride < (int64_t(1) << 31) && seqs * (stride + 1) < (int64_t(1) << 31);
}

// The state and workspace of a bookkeeping call.
mnb_status check_state(const mnb_cache_state* s, int64_t n, const void* ws, size_t ws_bytes) {
    if (!s || !s->refs || !s->tables || !s->lens || !valid_counts(s->num_pages, s->num_seqs, s->table_stride)) return MNB_ERR_INVALID_ARG;
    if (s->page_size < 1 || s->table_stride * s->page_size >= (int64_t(1) << 31)) return MNB_ERR_INVALID_ARG;
    if (n < 0 || n > s->num_seqs) return MNB_ERR_INVALID_ARG;
    if (!dec::aligned_to(s->refs, 4) || !dec::aligned_to(s->tables, 4) || !dec::aligned_to(s->lens, 4)) return MNB_ERR_INVALID_ARG;
    if (n == 0) return MNB_OK;
    if (!ws || ws_bytes < work_ints(s->num_pages, s->num_seqs, s->table_stride) * 4) return MNB_ERR_NO_MEM;
    return dec::aligned_to(ws, 256) ? MNB_OK : MNB_ERR_INVALID_ARG;
}

State make_state(const mnb_cache_state* s) {
    return State{s->refs, s->tables, s->lens, (int)s->num_pages, (int)s->num_seqs, (int)s->table_stride, s->page_size};
}

// One CTA where it can look at every page and list entry in a few rounds: its phases then meet at a CTA's barrier
// instead of a cluster's, and the launch is smaller (a fork of 12 and their growth: 14.2 -> 12.2 us).
int cluster_for(const mnb_cache_state* s, int64_t n) {
    return s->num_pages <= 4 * kThreads && n * ((s->table_stride + 31) / 32) <= 4 * kWarps ? 1 : kCluster;
}

size_t list_smem(const mnb_cache_state* s) { return (size_t)((s->num_seqs + 31) / 32) * 4; }

CopyParams make_copy(const mnb_page_planes* pl, const int32_t* src, const int32_t* dst, int64_t n, int* status) {
    CopyParams c{};
    c.base = static_cast<uint8_t*>(pl->base);
    c.plane_stride = pl->plane_stride;
    c.page_stride = pl->page_stride;
    c.page_bytes = pl->page_bytes;
    c.planes = (int)pl->num_planes;
    c.num_pages = (int)pl->num_pages;
    c.chunks = (int)((pl->page_bytes + kChunk - 1) / kChunk);
    c.src = src;
    c.dst = dst;
    c.n = n;
    c.status = status;
    return c;
}

cudaError_t launch_copy(const CopyParams& c, cudaStream_t s) {
    // enough blocks for every chunk at once, at most four resident blocks per SM; loops beyond
    int64_t units = c.n * c.planes * c.chunks;
    if (c.name) units += (int64_t)c.num_seqs * ((c.stride + 31) / 32);
    const int64_t most = (int64_t)dec::kSms * 4;
    int64_t blocks = (units + kCopyThreads / 32 - 1) / (kCopyThreads / 32);
    if (blocks > most) blocks = most;
    if (blocks < 1) blocks = 1;
    return dec::launch_pdl(copy_pages_kernel, dim3((unsigned)blocks), dim3(kCopyThreads), 0, s, 1, c);
}

}  // namespace
}  // namespace mnb

using namespace mnb;

extern "C" {

size_t mnb_cache_workspace_size(int64_t num_pages, int64_t num_seqs, int64_t table_stride) {
    if (!valid_counts(num_pages, num_seqs, table_stride)) return 0;
    return (work_ints(num_pages, num_seqs, table_stride) * 4 + 255) & ~size_t(255);
}

mnb_status mnb_pages_copy(const mnb_page_planes* planes, const int32_t* src, const int32_t* dst, int64_t n,
                          mnb_stream_t stream) {
    if (!valid_planes(planes) || n < 0 || n > planes->num_pages) return MNB_ERR_INVALID_ARG;
    if (n == 0) return MNB_OK;
    if (!src || !dst || !dec::aligned_to(src, 4) || !dec::aligned_to(dst, 4)) return MNB_ERR_INVALID_ARG;
    int* status = device_status_word();
    if (!status) return dec::status_of(cudaErrorUnknown);
    if (inject_launch_failure()) return MNB_ERR_CUDA;
    ProfileScope prof("mnb_pages_copy", (cudaStream_t)stream);
    const cudaError_t e = launch_copy(make_copy(planes, src, dst, n, status), (cudaStream_t)stream);
    if (e == cudaSuccess) prof.done("pages_copy");
    return dec::status_of(e);
}

mnb_status mnb_cache_fork(const mnb_cache_state* state, const int32_t* src, const int32_t* dst, int64_t n,
                          void* workspace, size_t workspace_bytes, mnb_stream_t stream) {
    const mnb_status st = check_state(state, n, workspace, workspace_bytes);
    if (st != MNB_OK || n == 0) return st;
    if (!src || !dst || !dec::aligned_to(src, 4) || !dec::aligned_to(dst, 4)) return MNB_ERR_INVALID_ARG;
    int* status = device_status_word();
    if (!status) return dec::status_of(cudaErrorUnknown);
    if (inject_launch_failure()) return MNB_ERR_CUDA;
    ProfileScope prof("mnb_cache_fork", (cudaStream_t)stream);
    const int cl = cluster_for(state, n);
    const cudaError_t e = dec::launch_pdl(fork_kernel, dim3(cl), dim3(kThreads), list_smem(state), (cudaStream_t)stream, cl, make_state(state), make_work(workspace, state), src, dst, (int)n, status);
    if (e == cudaSuccess) prof.done("cache_fork");
    return dec::status_of(e);
}

mnb_status mnb_cache_resize(const mnb_cache_state* state, const mnb_page_planes* planes, const int32_t* seqs,
                            const int32_t* new_lens, int64_t n, void* workspace, size_t workspace_bytes,
                            mnb_stream_t stream) {
    const mnb_status st = check_state(state, n, workspace, workspace_bytes);
    if (st != MNB_OK) return st;
    if (planes && (!valid_planes(planes) || planes->num_pages != state->num_pages)) return MNB_ERR_INVALID_ARG;
    if (n == 0) return MNB_OK;
    if (!seqs || !new_lens || !dec::aligned_to(seqs, 4) || !dec::aligned_to(new_lens, 4)) return MNB_ERR_INVALID_ARG;
    int* status = device_status_word();
    if (!status) return dec::status_of(cudaErrorUnknown);
    if (inject_launch_failure()) return MNB_ERR_CUDA;
    const Work w = make_work(workspace, state);
    ProfileScope prof("mnb_cache_resize", (cudaStream_t)stream);
    const int cl = cluster_for(state, n);
    cudaError_t e = dec::launch_pdl(resize_kernel, dim3(cl), dim3(kThreads), list_smem(state), (cudaStream_t)stream, cl, make_state(state), w, seqs, new_lens, (int)n, planes ? 1 : 0, status);
    if (e == cudaSuccess && planes) {
        CopyParams c = make_copy(planes, w.src, w.dst, n, status);
        c.own_list = 1;
        e = launch_copy(c, (cudaStream_t)stream);
    }
    if (e == cudaSuccess) prof.done("cache_resize");
    return dec::status_of(e);
}

mnb_status mnb_cache_compact(const mnb_cache_state* state, const mnb_page_planes* planes, int32_t* refs_out,
                             int32_t* tables_out, int32_t* counts, void* workspace, size_t workspace_bytes,
                             mnb_stream_t stream) {
    const mnb_status st = check_state(state, 1, workspace, workspace_bytes);
    if (st != MNB_OK) return st;
    if (!valid_planes(planes) || planes->num_pages != state->num_pages) return MNB_ERR_INVALID_ARG;
    if (!refs_out || !tables_out || !counts || !dec::aligned_to(refs_out, 4) || !dec::aligned_to(tables_out, 4) ||
        !dec::aligned_to(counts, 4))
        return MNB_ERR_INVALID_ARG;
    int* status = device_status_word();
    if (!status) return dec::status_of(cudaErrorUnknown);
    if (inject_launch_failure()) return MNB_ERR_CUDA;
    const Work w = make_work(workspace, state);
    ProfileScope prof("mnb_cache_compact", (cudaStream_t)stream);
    const int cl = cluster_for(state, 1);
    cudaError_t e = dec::launch_pdl(compact_kernel, dim3(cl), dim3(kThreads), 0, (cudaStream_t)stream, cl, make_state(state), w, refs_out, counts);
    if (e == cudaSuccess) {
        CopyParams c = make_copy(planes, w.src, w.dst, state->num_pages / 2, status);
        c.count = w.count + 48;
        c.name = w.pick;
        c.tables = state->tables;
        c.lens = state->lens;
        c.tables_out = tables_out;
        c.num_seqs = (int)state->num_seqs;
        c.stride = (int)state->table_stride;
        c.page_size = state->page_size;
        e = launch_copy(c, (cudaStream_t)stream);
    }
    if (e == cudaSuccess) prof.done("cache_compact");
    return dec::status_of(e);
}

}  // extern "C"
