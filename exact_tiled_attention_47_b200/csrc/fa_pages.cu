// fa_pages.cu -- operations on the pages of a paged cache: give sequences pages (extend), fork them,
// free them, move live pages to the front (compact), copy pages.
//
// State, all on the device: a block table [S, pages_per_seq] (row s lists the pages of slot s in key
// order), lengths [S], and a reference count per page (0 = free).  Pages are handed out from the
// lowest free one on, in the order of the request list, so the outcome depends on the inputs alone and
// never on the order in which blocks or atomics happen to run.
//
// Each operation is a plan and its work.  The plan is one CTA: it checks the whole request (a request
// that cannot be met changes nothing), ranks the free pages with a scan over the reference counts, and
// leaves (source, destination) page pairs in the workspace.  The work is a grid over those pairs: it
// moves whole pages of every pool in 16-byte pieces, and is bound by HBM (each moved byte is read and
// written once); the plan is bound by latency, a few dependent reads of L2.
#include <algorithm>

#include "fa_internal.h"
#include "fa_kv8.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanPer = 16;  // reference counts per thread and step of the free-page scan
constexpr int kStatusPageTable = 12;  // FA_ERR_PAGE_TABLE
constexpr int kStatusSlots = 14;      // FA_ERR_SLOTS
constexpr int kStatusNoPages = 15;    // FA_ERR_NO_PAGES

// Workspace: header, then the page pairs, the offset of each request's pages, and a mark per slot.
struct PagesWs {
  int* head;  // [0] number of pairs, [1] 1 if the request was accepted
  int* psrc;  // [max(n, num_pages)]
  int* pdst;
  int* off;   // [n]
  int* mark;  // [max(S, num_pages)]
};
constexpr int kHeadInts = 64;

__host__ __device__ inline PagesWs carve(int* ws, int n, int num_pages) {
  const size_t m = n > num_pages ? n : num_pages;
  PagesWs w;
  w.head = ws;
  w.psrc = ws + kHeadInts;
  w.pdst = w.psrc + m;
  w.off = w.pdst + m;
  w.mark = w.off + n;
  return w;
}

struct PlanParams {
  int* table;
  int* seqlens;
  int* refs;
  const int* a;
  const int* b;
  int n, S, pps, num_pages, page_size, dst_pages;
  PagesWs w;
  int* remap;
  int* n_live;
  int* status;
};

__device__ __forceinline__ long long capacity(const PlanParams& p) { return static_cast<long long>(p.pps) * p.page_size; }
__device__ __forceinline__ int pages_of(long long len, int page_size) { return static_cast<int>((len + page_size - 1) / page_size); }

// Exclusive prefix sum over the CTA; returns this thread's sum and the total.  `sums`: 32 values.
template <class T>
__device__ __forceinline__ T block_scan(T v, T* sums, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    T s = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    sums[lane] = s;
  }
  __syncthreads();
  const T before = warp ? sums[warp - 1] : 0;
  total = sums[31];
  __syncthreads();  // `sums` may be written again
  return before + x - v;
}

// Ranks the pages [base, base + 16384) that `take` accepts, in page order, behind `found` earlier ones
// and calls put(rank, page) for each; returns the new number found.  A page's rank is the number of
// accepted pages before it: a warp's ballot gives it inside 32 pages, a scan over the warps' counts
// the rest.
template <class Take, class Put>
__device__ __forceinline__ int rank_pages(int base, int num_pages, int found, int* cnt, int* sums, Take&& take, Put&& put) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned bal[kPlanPer];
  int v[kPlanPer];
#pragma unroll
  for (int k = 0; k < kPlanPer; ++k) {
    const int page = base + k * kPlanThreads + static_cast<int>(threadIdx.x);
    v[k] = page < num_pages ? take(page) : 0;
  }
#pragma unroll
  for (int k = 0; k < kPlanPer; ++k) {
    bal[k] = __ballot_sync(0xffffffffu, v[k] != 0);
    if (lane == 0) cnt[k * 32 + warp] = __popc(bal[k]);
  }
  __syncthreads();
  int total;
  const int mine = threadIdx.x < kPlanPer * 32 ? cnt[threadIdx.x] : 0;
  const int excl = block_scan(mine, sums, total);
  if (threadIdx.x < kPlanPer * 32) cnt[threadIdx.x] = excl;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kPlanPer; ++k)
    if (v[k]) put(found + cnt[k * 32 + warp] + __popc(bal[k] & ((1u << lane) - 1u)), base + k * kPlanThreads + static_cast<int>(threadIdx.x));
  __syncthreads();
  return found + total;
}

// The lowest `want` free pages, in order, into list; false if there are fewer.
__device__ __forceinline__ bool take_free(const PlanParams& p, int want, int* list, int* cnt, int* sums) {
  int found = 0;
  for (long long base = 0; base < p.num_pages && found < want; base += kPlanPer * kPlanThreads)
    found = rank_pages(static_cast<int>(base), p.num_pages, found, cnt, sums, [&](int page) { return p.refs[page] == 0 ? 1 : 0; },
                       [&](int rank, int page) {
                         if (rank < want && idx_ok(p.status, rank, 1, max(p.n, p.num_pages))) list[rank] = page;
                       });
  __syncthreads();  // the list is read by other threads of the CTA
  return found >= want;
}

// True if every thread's `bad` is 0; else the largest code among them is recorded.  Collective.
__device__ __forceinline__ bool accept(const PlanParams& p, int bad, int* s_bad) {
  if (threadIdx.x == 0) *s_bad = 0;
  __syncthreads();
  if (bad) atomicMax(s_bad, bad);
  __syncthreads();
  const int b = *s_bad;
  if (b && threadIdx.x == 0) record_status(p.status, b);
  return b == 0;
}

__global__ void __launch_bounds__(kPlanThreads) extend_kernel(const PlanParams p) {
  __shared__ int cnt[kPlanPer * 32], sums[32], s_bad;
  __shared__ long long sums64[32];
  const int tid = threadIdx.x;
  int bad = 0;
  long long all = 0;  // a request may ask for more pages than 32 bits count
  auto slot_of = [&](int i) { return p.a ? p.a[i] : i; };
  for (int base = 0; base < p.n; base += kPlanThreads) {
    const int i = base + tid;
    int need = 0;
    if (i < p.n) {
      const int s = slot_of(i);
      if (s < 0 || s >= p.S) {
        bad = kStatusSlots;
      } else {
        p.w.mark[s] = i;
        const int len = p.seqlens[s], add = p.b[i];
        if (add < 0 || len < 0 || static_cast<long long>(len) + add > capacity(p)) bad = max(bad, kStatusCuSeqlens);
        else need = pages_of(static_cast<long long>(len) + add, p.page_size) - pages_of(len, p.page_size);
      }
    }
    long long t;
    const long long excl = block_scan(static_cast<long long>(need), sums64, t);
    if (i < p.n) p.w.off[i] = static_cast<int>(all + excl);  // read only if the sum fits the pool
    all += t;
  }
  if (all > p.num_pages) bad = max(bad, kStatusNoPages);
  const int total = static_cast<int>(all);
  __syncthreads();
  for (int i = tid; i < p.n; i += kPlanThreads) {  // a slot that is named twice keeps one mark only
    const int s = slot_of(i);
    if (s >= 0 && s < p.S && p.w.mark[s] != i) bad = max(bad, kStatusSlots);
  }
  if (!accept(p, bad, &s_bad)) return;
  if (!accept(p, take_free(p, total, p.w.psrc, cnt, sums) ? 0 : kStatusNoPages, &s_bad)) return;
  for (int j = tid; j < total; j += kPlanThreads) {
    int lo = 0, hi = p.n - 1;  // the last request whose pages begin at or before j
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.w.off[mid] <= j) lo = mid;
      else hi = mid - 1;
    }
    const int s = slot_of(lo), page = p.w.psrc[j];
    const int col = pages_of(p.seqlens[s], p.page_size) + j - p.w.off[lo];
    const long long at = static_cast<long long>(s) * p.pps + col;
    if (idx_ok(p.status, at, 1, static_cast<long long>(p.S) * p.pps) && idx_ok(p.status, page, 1, p.num_pages)) {
      p.table[at] = page;
      p.refs[page] = 1;
    }
  }
  __syncthreads();  // the old lengths were read above
  for (int i = tid; i < p.n; i += kPlanThreads) p.seqlens[slot_of(i)] += p.b[i];
}

__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const PlanParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  __shared__ int cnt[kPlanPer * 32], sums[32], s_bad;
  const int tid = threadIdx.x;
  int bad = 0, total = 0;
  if (tid == 0) p.w.head[0] = p.w.head[1] = 0;
  for (int base = 0; base < p.n; base += kPlanThreads) {
    const int i = base + tid;
    int need = 0;
    if (i < p.n) {
      const int src = p.a[i], dst = p.b[i];
      if (src < 0 || src >= p.S || dst < 0 || dst >= p.S) {
        bad = kStatusSlots;
      } else {
        p.w.mark[dst] = i;
        const int len = p.seqlens[src];
        if (p.seqlens[dst] != 0) bad = max(bad, kStatusSlots);
        if (len < 0 || len > capacity(p)) bad = max(bad, kStatusCuSeqlens);
        else need = len % p.page_size ? 1 : 0;
        if (need) {
          const int page = p.table[static_cast<long long>(src) * p.pps + len / p.page_size];
          if (page < 0 || page >= p.num_pages || p.refs[page] <= 0) bad = max(bad, kStatusPageTable);
        }
      }
    }
    int t;
    const int excl = block_scan(need, sums, t);
    if (i < p.n) p.w.off[i] = total + excl;
    total += t;
  }
  __syncthreads();
  for (int i = tid; i < p.n; i += kPlanThreads) {
    const int src = p.a[i], dst = p.b[i];
    if (src < 0 || src >= p.S || dst < 0 || dst >= p.S) continue;
    if (p.w.mark[dst] != i) bad = max(bad, kStatusSlots);  // a destination named twice
    const int m = p.w.mark[src];                           // (a mark of no one's is any number)
    if (m >= 0 && m < p.n && p.b[m] == src) bad = max(bad, kStatusSlots);  // a source that is a destination
  }
  if (!accept(p, bad, &s_bad)) return;
  if (!accept(p, take_free(p, total, p.w.pdst, cnt, sums) ? 0 : kStatusNoPages, &s_bad)) return;
  // the pages handed out, found again by page (the marks of the slots are done with): see fork_kernel
  for (int j = tid; j < total; j += kPlanThreads) p.w.mark[p.w.pdst[j]] = j;
  for (int i = tid; i < p.n; i += kPlanThreads) {
    const int src = p.a[i], dst = p.b[i], len = p.seqlens[src];
    if (len % p.page_size) {
      const long long col = len / p.page_size;
      const int to = p.w.pdst[p.w.off[i]];
      if (idx_ok(p.status, to, 1, p.num_pages)) {
        p.w.psrc[p.w.off[i]] = p.table[static_cast<long long>(src) * p.pps + col];
        p.table[static_cast<long long>(dst) * p.pps + col] = to;
        p.refs[to] = 1;
      }
    }
    p.seqlens[dst] = len;  // no source is a destination: lengths read above do not change
  }
  if (tid == 0) {
    p.w.head[0] = total;
    p.w.head[1] = 1;
  }
}

__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const PlanParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  __shared__ int cnt[kPlanPer * 32], sums[32];
  int live = 0;
  for (int page = threadIdx.x; page < p.num_pages; page += kPlanThreads) live += p.refs[page] > 0;
  int n_live;
  block_scan(live, sums, n_live);
  // the j-th live page behind the first n_live places moves to the j-th free place among them
  int movers = 0, holes = 0;
  for (long long base = 0; base < p.num_pages; base += kPlanPer * kPlanThreads) {
    movers = rank_pages(static_cast<int>(base), p.num_pages, movers, cnt, sums,
                        [&](int page) {
                          const bool alive = p.refs[page] > 0;
                          p.remap[page] = alive ? page : -1;
                          return alive && page >= n_live ? 1 : 0;
                        },
                        [&](int rank, int page) { p.w.psrc[rank] = page; });
    holes = rank_pages(static_cast<int>(base), min(p.num_pages, n_live), holes, cnt, sums,
                       [&](int page) { return p.refs[page] > 0 ? 0 : 1; }, [&](int rank, int page) { p.w.pdst[rank] = page; });
  }
  __syncthreads();
  for (int j = threadIdx.x; j < movers; j += kPlanThreads) p.remap[p.w.psrc[j]] = p.w.pdst[j];
  if (threadIdx.x == 0) {
    p.w.head[0] = movers;
    p.w.head[1] = 1;
    *p.n_live = n_live;
  }
}

// Checks a list of page copies: indices inside the pools, no destination twice, and no page that is
// both read and written (pools may be the same on both sides).
__global__ void __launch_bounds__(kPlanThreads) copy_plan_kernel(const PlanParams p, bool same) {
  asm volatile("griddepcontrol.launch_dependents;");
  __shared__ int s_bad;
  int bad = 0;
  if (threadIdx.x == 0) p.w.head[0] = p.w.head[1] = 0;
  for (int i = threadIdx.x; i < p.n; i += kPlanThreads) {
    const int src = p.a[i], dst = p.b[i];
    if (src < 0 || src >= p.num_pages || dst < 0 || dst >= p.dst_pages) bad = kStatusPageTable;
    else p.w.mark[dst] = i;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.n; i += kPlanThreads) {
    const int src = p.a[i], dst = p.b[i];
    if (src < 0 || src >= p.num_pages || dst < 0 || dst >= p.dst_pages) continue;
    if (p.w.mark[dst] != i) bad = max(bad, kStatusSlots);
    if (same && src < p.dst_pages) {
      const int m = p.w.mark[src];
      if (m >= 0 && m < p.n && p.b[m] == src) bad = max(bad, kStatusSlots);
    }
    p.w.psrc[i] = src;
    p.w.pdst[i] = dst;
  }
  if (!accept(p, bad, &s_bad)) return;
  if (threadIdx.x == 0) {
    p.w.head[0] = p.n;
    p.w.head[1] = 1;
  }
}

__global__ void __launch_bounds__(256) free_kernel(const PlanParams p) {
  __shared__ int s_len;
  const int s = p.a[blockIdx.x];
  if (s < 0 || s >= p.S) {
    if (threadIdx.x == 0) record_status(p.status, kStatusSlots);
    return;
  }
  if (threadIdx.x == 0) {
    int len = p.seqlens[s];
    if (len < 0 || len > capacity(p)) {  // its pages cannot be told: the slot stays as it is
      record_status(p.status, kStatusCuSeqlens);
      len = 0;
    } else if (atomicCAS(p.seqlens + s, len, 0) != len) {
      len = 0;  // a slot that is named twice is freed by whoever comes first
    }
    s_len = len;
  }
  __syncthreads();
  const int held = pages_of(s_len, p.page_size);
  for (int c = threadIdx.x; c < held; c += blockDim.x) {
    int* e = p.table + static_cast<long long>(s) * p.pps + c;
    const int page = *e;
    *e = -1;
    if (page < 0 || page >= p.num_pages) {
      record_status(p.status, kStatusPageTable);
    } else if (atomicSub(p.refs + page, 1) <= 0) {  // nobody held it: the count stays at what it was
      atomicAdd(p.refs + page, 1);
      record_status(p.status, kStatusPageTable);
    }
  }
}

// ---- the work -------------------------------------------------------------------------------------

constexpr int kMoveThreads = 256;
constexpr int kMovePiece = 16384;  // bytes of a page that one CTA moves at a time (four loads in flight per thread)

struct MoveParams {
  PoolSet pools;
  unsigned first_piece[kMaxPools + 1];  // pieces of a page in the pools before pool k
  const int* head;
  const int* psrc;
  const int* pdst;
  int src_pages, dst_pages;
  int* status;
};

template <class V>
__device__ __forceinline__ void move_piece(const char* src, char* dst, int bytes) {
  constexpr int kStep = kMoveThreads * static_cast<int>(sizeof(V));
  for (int at = threadIdx.x * static_cast<int>(sizeof(V)); at < bytes; at += 4 * kStep) {
    V v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (at + u * kStep < bytes) v[u] = __ldcs(reinterpret_cast<const V*>(src + at + u * kStep));
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (at + u * kStep < bytes) __stcs(reinterpret_cast<V*>(dst + at + u * kStep), v[u]);
  }
}

__device__ __forceinline__ void move_pages(const MoveParams& m, int block, int blocks) {
  const unsigned per_pair = m.first_piece[m.pools.n];
  const long long units = static_cast<long long>(m.head[0]) * per_pair;
  for (long long u = block; u < units; u += blocks) {
    const int j = static_cast<int>(u / per_pair);
    const unsigned r = static_cast<unsigned>(u % per_pair);
    int k = 0;
    while (r >= m.first_piece[k + 1]) ++k;
    const int src = m.psrc[j], dst = m.pdst[j];
    if (!idx_ok(m.status, src, 1, m.src_pages) || !idx_ok(m.status, dst, 1, m.dst_pages)) continue;
    const unsigned long long bytes = m.pools.page_bytes[k], at = static_cast<unsigned long long>(r - m.first_piece[k]) * kMovePiece;
    const int len = static_cast<int>(min(bytes - at, static_cast<unsigned long long>(kMovePiece)));
    const char* s = static_cast<const char*>(m.pools.src[k]) + src * bytes + at;
    char* d = static_cast<char*>(m.pools.dst[k]) + dst * bytes + at;
    if (((reinterpret_cast<uintptr_t>(s) | reinterpret_cast<uintptr_t>(d) | static_cast<uintptr_t>(len)) & 15) == 0) move_piece<uint4>(s, d, len);
    else move_piece<uint32_t>(s, d, len);
  }
}

__global__ void __launch_bounds__(kMoveThreads) move_kernel(const __grid_constant__ MoveParams m) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan is done
  move_pages(m, blockIdx.x, gridDim.x);
}

// Fork: the first p.n CTAs write the destinations' table rows and count the shared pages, the others
// copy the last partial pages.  A page of the source that is not in the pool or that nobody holds is not shared: its
// count is 0 (held pages are at 1 or more throughout), or this very call has handed it out.
__global__ void __launch_bounds__(kMoveThreads) fork_kernel(const __grid_constant__ MoveParams m, const PlanParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan is done
  if (m.head[1] == 0) return;
  if (static_cast<int>(blockIdx.x) >= p.n) {
    move_pages(m, blockIdx.x - p.n, gridDim.x - p.n);
    return;
  }
  const int src = p.a[blockIdx.x], dst = p.b[blockIdx.x];
  const int full = p.seqlens[src] / p.page_size, handed = m.head[0];
  for (int c = threadIdx.x; c < full; c += kMoveThreads) {
    const int page = p.table[static_cast<long long>(src) * p.pps + c];
    bool held = page >= 0 && page < p.num_pages;
    if (held) {
      const int count = p.refs[page], j = p.w.mark[page];  // (the mark is any number where the page was not handed out)
      held = count > 0 && (j < 0 || j >= handed || m.pdst[j] != page);
    }
    p.table[static_cast<long long>(dst) * p.pps + c] = held ? page : -1;
    if (held) atomicAdd(p.refs + page, 1);
    else record_status(p.status, kStatusPageTable);
  }
}

// Compact: the first `meta` CTAs write the tables and counts of the new places, the others move pages.
// Tables and counts may be written in place: each entry is read and written by one thread alone.
__global__ void __launch_bounds__(kMoveThreads) compact_kernel(const __grid_constant__ MoveParams m, const PlanParams p, int* table_out,
                                                               int* refs_out, int meta) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan is done
  if (static_cast<int>(blockIdx.x) >= meta) {
    move_pages(m, blockIdx.x - meta, gridDim.x - meta);
    return;
  }
  const long long step = static_cast<long long>(meta) * kMoveThreads, first = static_cast<long long>(blockIdx.x) * kMoveThreads + threadIdx.x;
  const int movers = m.head[0], n_live = *p.n_live;
  for (long long i = first; i < static_cast<long long>(p.S) * p.pps; i += step) {
    const int s = static_cast<int>(i / p.pps), c = static_cast<int>(i % p.pps), len = p.seqlens[s];
    int page = p.table[i];
    if (len < 0 || len > capacity(p)) {
      if (c == 0) record_status(p.status, kStatusCuSeqlens);
    } else if (c < pages_of(len, p.page_size)) {
      const int to = page >= 0 && page < p.num_pages ? p.remap[page] : -1;
      if (to < 0) record_status(p.status, kStatusPageTable);  // an entry that names no live page
      page = to;
    }
    table_out[i] = page;
  }
  for (long long j = first; j < movers; j += step) refs_out[m.pdst[j]] = p.refs[m.psrc[j]];
  // places of moved pages are written above; in place, those behind n_live are still read there, and a kernel that
  // follows clears them
  for (long long i = first; refs_out != p.refs && i < p.num_pages; i += step) {
    const int r = p.refs[i];
    if (i >= n_live) refs_out[i] = 0;
    else if (r > 0) refs_out[i] = r;
  }
}

__global__ void __launch_bounds__(kMoveThreads) clear_tail_kernel(const int* n_live, int* refs_out, int num_pages) {
  for (int i = *n_live + static_cast<int>(blockIdx.x) * kMoveThreads + threadIdx.x; i < num_pages; i += gridDim.x * kMoveThreads) refs_out[i] = 0;
}

// The work's kernel is launched while the plan still runs and waits for it on the device (the gap between the two
// is a good part of a small request's time).
template <class... P, class... A>
cudaError_t launch_behind(void (*kern)(P...), int grid, cudaStream_t stream, const A&... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

PlanParams plan_of(const PagesArgs& a) {
  PlanParams p;
  p.table = a.table;
  p.seqlens = a.seqlens;
  p.refs = a.refs;
  p.a = a.a;
  p.b = a.b;
  p.n = a.n;
  p.S = a.S;
  p.pps = a.pages_per_seq;
  p.num_pages = a.num_pages;
  p.page_size = a.page_size;
  p.dst_pages = a.dst_pages;
  p.w = carve(a.ws, a.n, std::max(a.num_pages, a.dst_pages));
  p.remap = a.remap;
  p.n_live = a.n_live;
  p.status = a.status;
  return p;
}

// Pools [first, first + kMaxPools) of the request.
MoveParams move_of(const PagesArgs& a, const PlanParams& p, int first) {
  MoveParams m;
  m.pools.n = std::min(kMaxPools, a.n_pools - first);
  m.first_piece[0] = 0;
  for (int k = 0; k < m.pools.n; ++k) {
    m.pools.src[k] = a.src_pools ? a.src_pools[first + k] : a.pools[first + k];
    m.pools.dst[k] = a.pools[first + k];
    m.pools.page_bytes[k] = a.page_bytes[first + k];
    m.first_piece[k + 1] = m.first_piece[k] + static_cast<unsigned>((a.page_bytes[first + k] + kMovePiece - 1) / kMovePiece);
  }
  m.head = p.w.head;
  m.psrc = p.w.psrc;
  m.pdst = p.w.pdst;
  m.src_pages = a.num_pages;
  m.dst_pages = a.dst_pages;
  m.status = a.status;
  return m;
}

// CTAs for at most `pairs` page moves of these pools: eight per SM are enough to keep HBM busy.
int move_blocks(const MoveParams& m, long long pairs) {
  return static_cast<int>(std::max(1LL, std::min<long long>(148 * 8, pairs * m.first_piece[m.pools.n])));
}

}  // namespace

size_t pages_ws_bytes(int n, int S, int num_pages) {
  const size_t m = std::max(n, num_pages), ints = kHeadInts + 2 * m + n + std::max(S, num_pages);
  return (ints * sizeof(int) + 255) & ~static_cast<size_t>(255);
}

int launch_pages_extend(const PagesArgs& a, cudaStream_t stream) {
  extend_kernel<<<1, kPlanThreads, 0, stream>>>(plan_of(a));
  return static_cast<int>(cudaGetLastError());
}

int launch_pages_free(const PagesArgs& a, cudaStream_t stream) {
  PlanParams p = plan_of(a);
  free_kernel<<<a.n, 256, 0, stream>>>(p);
  return static_cast<int>(cudaGetLastError());
}

int launch_pages_fork(const PagesArgs& a, cudaStream_t stream) {
  const PlanParams p = plan_of(a);
  fork_plan_kernel<<<1, kPlanThreads, 0, stream>>>(p);
  for (int first = 0; first == 0 || first < a.n_pools; first += kMaxPools) {
    const MoveParams m = move_of(a, p, first);
    const cudaError_t e = first == 0 ? launch_behind(fork_kernel, a.n + move_blocks(m, a.n), stream, m, p) : launch_behind(move_kernel, move_blocks(m, a.n), stream, m);
    if (e != cudaSuccess) return static_cast<int>(e);
  }
  return static_cast<int>(cudaGetLastError());
}

int launch_pages_compact(const PagesArgs& a, cudaStream_t stream) {
  const PlanParams p = plan_of(a);
  compact_plan_kernel<<<1, kPlanThreads, 0, stream>>>(p);
  const int meta = static_cast<int>(std::min<long long>(148, (static_cast<long long>(a.S) * a.pages_per_seq + a.num_pages) / 1024 + 1));
  for (int first = 0; first == 0 || first < a.n_pools; first += kMaxPools) {
    const MoveParams m = move_of(a, p, first);
    const cudaError_t e = first == 0 ? launch_behind(compact_kernel, meta + move_blocks(m, a.num_pages), stream, m, p, a.table_out, a.refs_out, meta)
                                     : launch_behind(move_kernel, move_blocks(m, a.num_pages), stream, m);
    if (e != cudaSuccess) return static_cast<int>(e);
  }
  if (a.refs_out == a.refs) clear_tail_kernel<<<std::min(148, a.num_pages / 1024 + 1), kMoveThreads, 0, stream>>>(a.n_live, a.refs_out, a.num_pages);
  return static_cast<int>(cudaGetLastError());
}

int launch_pages_copy(const PagesArgs& a, cudaStream_t stream) {
  const PlanParams p = plan_of(a);
  bool same = false;
  for (int i = 0; i < a.n_pools; ++i)
    for (int j = 0; j < a.n_pools; ++j) same |= a.src_pools[i] == a.pools[j];
  copy_plan_kernel<<<1, kPlanThreads, 0, stream>>>(p, same);
  for (int first = 0; first < a.n_pools; first += kMaxPools) {
    const MoveParams m = move_of(a, p, first);
    const cudaError_t e = launch_behind(move_kernel, move_blocks(m, a.n), stream, m);
    if (e != cudaSuccess) return static_cast<int>(e);
  }
  return static_cast<int>(cudaGetLastError());
}

}  // namespace fa
