// pages.cu — pages of the paged caches shared by several sequences: freeing, forking,
// reserving and compacting them (the block tables, lengths and reference counts of a
// kt_page_map), and copying pages in the pools of all layers.
//
// Bookkeeping is a few passes over arrays that live in L2: num_pages counts, the tables of
// the sequences concerned, and what depends on all of them is a rank (the r-th request that
// needs a page takes the r-th free page).  What bounds it is the latency of the passes that
// wait for one another, so each call is one cluster of CLUSTER CTAs: every CTA counts its
// slice of the pages, the counts meet in shared memory of the cluster, and the barriers
// between the passes are the cluster's (under 1 us) instead of launches: in a graph a turnover (old
// samples freed, new ones forked) is 6.5 us for 4 samples, 8.9 for 48 and 12.5 for 16 of 131K tokens,
// a reservation 3.5, a compaction 8 for 300 pages as for 8K.  Ranks follow page and request
// numbers, so the outcome does not depend on which CTA comes first.
#include <cstring>

#include "kt_internal.cuh"

namespace kt {
namespace {

constexpr int CLUSTER = 8;
constexpr int THREADS = 1024;
constexpr int WARPS = THREADS / 32;

struct MapParams {
  int32_t* table;
  int32_t* lens;
  int32_t* blocks;
  int32_t* refs;
  int* status;
  int32_t* list;   // workspace [num_pages]: free pages by rank; compact: the movers behind them
  int32_t* list2;  // workspace [num_pages]; compact: where each page goes
  const int32_t* a;  // fork: sources; free: sequences; reserve: new tokens (nullable)
  const int32_t* b;  // fork: destinations
  int32_t* moves;
  int32_t* num_moves;
  int32_t* new_table;
  int32_t* new_refs;
  int n, batch, max_blocks, P;
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// An int in the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ int ld_cluster(const int* p, uint32_t rank) {
  uint32_t at;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

struct Shared {
  int warp_sum[WARPS];
  int count[1];  // this CTA's count, read by the cluster
};

// Exclusive prefix of x over the CTA's threads, and the total.
__device__ __forceinline__ int block_scan(int x, int* total, Shared& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  __syncthreads();  // the previous round's sums have been read
  if (lane == 31) sh.warp_sum[warp] = incl;
  __syncthreads();
  int s = sh.warp_sum[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += v;
  }
  *total = __shfl_sync(0xffffffffu, s, 31);
  const int before = __shfl_sync(0xffffffffu, s, warp > 0 ? warp - 1 : 0);
  return (warp > 0 ? before : 0) + incl - x;
}

// CTA r's slice of the pages: whole groups of four.
struct Slice {
  int lo, hi;
};
__device__ __forceinline__ Slice slice_of(int P, int r) {
  const int groups = (P + 3) / 4;
  const int lo = (int)((long long)groups * r / CLUSTER) * 4;
  const int hi = (int)((long long)groups * (r + 1) / CLUSTER) * 4;
  return Slice{min(lo, P), min(hi, P)};
}
// Counts of the four pages from p on; pages past the slice get `none`.
__device__ __forceinline__ int4 load4(const int32_t* refs, int p, int hi, int none) {
  if (p + 4 <= hi) return *reinterpret_cast<const int4*>(refs + p);
  return make_int4(p < hi ? refs[p] : none, p + 1 < hi ? refs[p + 1] : none,
                   p + 2 < hi ? refs[p + 2] : none, none);
}

// Pages of the slice with pred(page, count), in all threads.
template <class Pred>
__device__ __forceinline__ int count_pages(const int32_t* refs, Slice s, Pred pred, Shared& sh) {
  int c = 0;
  for (int p = s.lo + 4 * (int)threadIdx.x; p < s.hi; p += 4 * THREADS) {
    const int4 v = load4(refs, p, s.hi, 0);
    c += pred(p, v.x);
    if (p + 1 < s.hi) c += pred(p + 1, v.y);
    if (p + 2 < s.hi) c += pred(p + 2, v.z);
    if (p + 3 < s.hi) c += pred(p + 3, v.w);
  }
  int total;
  block_scan(c, &total, sh);
  return total;
}

// out[rank] = page for the pages of the slice with pred, ranks from `base` in page order,
// as long as they are below `limit`.
template <class Pred>
__device__ __forceinline__ void list_pages(const int32_t* refs, Slice s, int base, int limit,
                                           int32_t* out, Pred pred, Shared& sh) {
  for (int p0 = s.lo; p0 < s.hi && base < limit; p0 += 4 * THREADS) {
    const int p = p0 + 4 * (int)threadIdx.x;
    int4 v = make_int4(0, 0, 0, 0);
    if (p < s.hi) v = load4(refs, p, s.hi, 0);
    bool t[4];
    t[0] = p < s.hi && pred(p, v.x);
    t[1] = p + 1 < s.hi && pred(p + 1, v.y);
    t[2] = p + 2 < s.hi && pred(p + 2, v.z);
    t[3] = p + 3 < s.hi && pred(p + 3, v.w);
    int total;
    int rank = base + block_scan(t[0] + t[1] + t[2] + t[3], &total, sh);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (t[i]) {
        if (rank < limit) out[rank] = p + i;
        ++rank;
      }
    base += total;
  }
}

// The `need` lowest free pages into p.list (as many as there are); returns how many there
// are in the whole pool.  Ends with a cluster barrier.
__device__ __forceinline__ int find_free(const MapParams& p, int need, Shared& sh) {
  const Slice s = slice_of(p.P, cluster_rank());
  auto is_free = [](int, int refs) { return refs <= 0 ? 1 : 0; };
  const int mine = count_pages(p.refs, s, is_free, sh);
  if (threadIdx.x == 0) sh.count[0] = mine;
  cluster_sync();
  int before = 0, total = 0;
#pragma unroll
  for (int r = 0; r < CLUSTER; ++r) {
    const int c = ld_cluster(&sh.count[0], r);
    if (r < (int)cluster_rank()) before += c;
    total += c;
  }
  list_pages(p.refs, s, before, need, p.list, is_free, sh);
  cluster_sync();
  return total;
}

// ---- free --------------------------------------------------------------------------------
// One CTA a sequence.  A sequence listed twice is freed by whichever takes its block count.
__global__ void __launch_bounds__(256) free_kernel(const __grid_constant__ MapParams p) {
  __shared__ int held;
  griddep_wait();
  griddep_launch_dependents();
  const int b = p.a[blockIdx.x];
  if (b < 0 || b >= p.batch) {
    if (threadIdx.x == 0) set_status(p.status, KT_ERR_DEVICE_CHECK);
    return;
  }
  if (threadIdx.x == 0) {
    int n = atomicExch(p.blocks + b, 0);
    if (n < 0 || n > p.max_blocks) {
      set_status(p.status, KT_ERR_DEVICE_CHECK);
      n = n < 0 ? 0 : p.max_blocks;
    }
    p.lens[b] = 0;
    held = n;
  }
  __syncthreads();
  const int32_t* row = p.table + (size_t)b * p.max_blocks;
  for (int j = threadIdx.x; j < held; j += 256) {
    const int page = row[j];
    if (page < 0 || page >= p.P) {
      set_status(p.status, KT_ERR_DEVICE_CHECK);
    } else if (atomicSub(p.refs + page, 1) <= 0) {  // nobody held it
      atomicAdd(p.refs + page, 1);
      set_status(p.status, KT_ERR_DEVICE_CHECK);
    }
  }
}

// ---- fork --------------------------------------------------------------------------------
// Every CTA checks all requests (they are at most MAX_SEGS), so that only the free pages
// need the cluster; a warp then takes 32 table entries of one fork at a time.
__global__ void __cluster_dims__(CLUSTER, 1, 1) __launch_bounds__(THREADS, 1)
    fork_kernel(const __grid_constant__ MapParams p) {
  __shared__ Shared sh;
  __shared__ int claim[MAX_SEGS];  // the fork that gets a destination
  __shared__ int len[MAX_SEGS];    // tokens of fork i, -1: refused
  __shared__ int rank[MAX_SEGS];   // its free page, -1: it needs none
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x;
  const uint32_t cta = cluster_rank();
  for (int i = tid; i < p.batch; i += THREADS) claim[i] = 0x7fffffff;
  __syncthreads();
  for (int i = tid; i < p.n; i += THREADS) {
    const int s = p.a[i], d = p.b[i];
    int n = -1;
    if (s >= 0 && s < p.batch && d >= 0 && d < p.batch && p.blocks[d] == 0 && p.lens[d] == 0) {
      const int have = p.blocks[s];
      n = p.lens[s];
      if (n < 0 || have < 0 || have > p.max_blocks || n > (long long)have * BS) n = -1;
    }
    if (n >= 0) atomicMin(&claim[d], i);
    len[i] = n;
  }
  __syncthreads();
  int need = 0;
  for (int i0 = 0; i0 < p.n; i0 += THREADS) {
    const int i = i0 + tid;
    bool partial = false;
    if (i < p.n) {
      if (len[i] >= 0 && claim[p.b[i]] != i) len[i] = -1;
      if (len[i] < 0) set_status(p.status, KT_ERR_DEVICE_CHECK);
      partial = len[i] > 0 && len[i] % BS != 0;
    }
    int total;
    const int r = need + block_scan(partial, &total, sh);
    if (i < p.n) rank[i] = partial ? r : -1;
    need += total;
  }
  const int have = find_free(p, need, sh);
  if (need > have && cta == 0 && tid == 0) set_status(p.status, KT_ERR_DEVICE_CHECK);
  if (cta == 0 && tid == 0) *p.num_moves = min(need, have);

  const int chunks = (p.max_blocks + 31) / 32;
  const long long items = (long long)p.n * chunks;
  for (long long it = cta * WARPS + (tid >> 5); it < items; it += CLUSTER * WARPS) {
    const int i = (int)(it / chunks), j = (int)(it % chunks) * 32 + (tid & 31);
    const int n = len[i], r = rank[i];
    if (n <= 0 || r >= have) continue;  // refused, empty, or no page for its last tokens
    const int nb = (n + BS - 1) / BS;
    const int s = p.a[i], d = p.b[i];
    if (j == 0) {
      p.lens[d] = n;
      p.blocks[d] = nb;
    }
    if (j >= nb) continue;
    int page = p.table[(size_t)s * p.max_blocks + j];
    const bool ok = page >= 0 && page < p.P;
    if (!ok) set_status(p.status, KT_ERR_DEVICE_CHECK);
    if (j == nb - 1 && r >= 0) {
      const int own = p.list[r];
      p.moves[2 * (size_t)r] = page;
      p.moves[2 * (size_t)r + 1] = own;
      p.refs[own] = 1;
      page = own;
    } else if (ok) {
      atomicAdd(p.refs + page, 1);
    }
    p.table[(size_t)d * p.max_blocks + j] = page;
  }
}

// ---- reserve -----------------------------------------------------------------------------
// Pages that sequence b still needs for p.a[b] more tokens (NULL: one).
__device__ __forceinline__ int pages_needed(const MapParams& p, int b) {
  const int more = p.a ? p.a[b] : 1;
  const int n = p.lens[b], have = p.blocks[b];
  if (more == 0) return 0;
  const long long want = ((long long)n + more + BS - 1) / BS;
  if (more < 0 || n < 0 || have < 0 || have > p.max_blocks || n > (long long)have * BS ||
      want > p.max_blocks)
    return -1;
  return want > have ? (int)(want - have) : 0;
}

__global__ void __cluster_dims__(CLUSTER, 1, 1) __launch_bounds__(THREADS, 1)
    reserve_kernel(const __grid_constant__ MapParams p) {
  __shared__ Shared sh;
  __shared__ long long last[MAX_SEGS];  // pages needed by the sequences up to b
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31;
  const uint32_t cta = cluster_rank();
  long long need = 0;
  for (int b0 = 0; b0 < p.batch; b0 += THREADS) {
    const int b = b0 + tid;
    int c = b < p.batch ? pages_needed(p, b) : 0;
    if (c < 0) {
      set_status(p.status, KT_ERR_DEVICE_CHECK);
      c = 0;
    }
    // 1024 sequences of at most 2^24 blocks: in parts that stay below 2^31
    int lo, hi;
    const int a = block_scan(c & 0xfff, &lo, sh);
    const int z = block_scan(c >> 12, &hi, sh);
    if (b < p.batch) last[b] = need + a + ((long long)z << 12) + c;
    need += lo + ((long long)hi << 12);
  }
  const int have = find_free(p, (int)min(need, (long long)p.P), sh);
  if (need > have && cta == 0 && tid == 0) set_status(p.status, KT_ERR_DEVICE_CHECK);
  for (int b = cta * WARPS + (tid >> 5); b < p.batch; b += CLUSTER * WARPS) {
    const long long first = b > 0 ? last[b - 1] : 0;
    const int c = (int)(last[b] - first);
    if (c == 0 || last[b] > have) continue;  // nothing to do, or the pages have run out
    const int had = p.blocks[b];
    for (int i = lane; i < c; i += 32) {
      const int page = p.list[first + i];
      p.table[(size_t)b * p.max_blocks + had + i] = page;
      p.refs[page] = 1;
    }
    __syncwarp();
    if (lane == 0) p.blocks[b] = had + c;
  }
}

// ---- compact -----------------------------------------------------------------------------
// With `used` pages in use, the pages from `used` on that are in use move, lowest first, to
// the free ones below.
__global__ void __cluster_dims__(CLUSTER, 1, 1) __launch_bounds__(THREADS, 1)
    compact_kernel(const __grid_constant__ MapParams p) {
  __shared__ Shared sh;
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x;
  const uint32_t cta = cluster_rank();
  const Slice s = slice_of(p.P, cluster_rank());
  const int mine = count_pages(p.refs, s, [](int, int r) { return r > 0 ? 1 : 0; }, sh);
  if (tid == 0) sh.count[0] = mine;
  cluster_sync();
  int count[CLUSTER], used = 0, before = 0;
#pragma unroll
  for (int r = 0; r < CLUSTER; ++r) {
    count[r] = ld_cluster(&sh.count[0], r);
    used += count[r];
    if (r < (int)cta) before += count[r];
  }
  // holes: free pages below `used`; movers: pages in use from there on; as many of both.  With
  // the pages in use below `used` counted too (the slice that `used` cuts is counted by every CTA),
  // a page's number and the pages in use before it give its rank in either list.
  int below = 0;
  Slice cut = {0, 0};
#pragma unroll
  for (int r = 0; r < CLUSTER; ++r) {
    const Slice t = slice_of(p.P, r);
    if (t.hi <= used) below += count[r];
    else if (t.lo < used) cut = Slice{t.lo, used};
  }
  if (cut.lo < cut.hi) below += count_pages(p.refs, cut, [](int, int r) { return r > 0 ? 1 : 0; }, sh);
  const int total = used - below;
  if (s.lo < used)
    list_pages(p.refs, Slice{s.lo, min(s.hi, used)}, s.lo - before, total, p.list,
               [](int, int r) { return r <= 0 ? 1 : 0; }, sh);
  int32_t* movers = p.list + (p.P - total);  // behind the holes: both lists are at most P / 2
  if (s.hi > used)
    list_pages(p.refs, s, s.lo < used ? 0 : before - below, total, movers,
               [used](int page, int r) { return page >= used && r > 0 ? 1 : 0; }, sh);
  cluster_sync();
  // the moves, and where each page goes: list2[page], -1 for a page that nobody holds (a hole
  // becomes another page, so an entry that names it is found here or not at all)
  if (cta == 0 && tid == 0) *p.num_moves = total;
  for (int i = cta * THREADS + tid; i < total; i += CLUSTER * THREADS) {
    const int from = movers[i], to = p.list[i];
    p.moves[2 * (size_t)i] = from;
    p.moves[2 * (size_t)i + 1] = to;
    p.list2[from] = to;
  }
  for (int i = s.lo + tid; i < s.hi; i += THREADS) {
    const int r = p.refs[i];
    if (r <= 0 || i < used) p.list2[i] = r > 0 ? i : -1;
    if (p.new_refs != p.refs) {
      if (i >= used) p.new_refs[i] = 0;
      else if (r > 0) p.new_refs[i] = r;
    }
  }
  cluster_sync();
  for (int i = cta * THREADS + tid; i < total; i += CLUSTER * THREADS) {
    const int from = movers[i];
    p.new_refs[p.list[i]] = p.refs[from];
    if (p.new_refs == p.refs) p.refs[from] = 0;
  }
  const int chunks = (p.max_blocks + 31) / 32;
  const long long items = (long long)p.batch * chunks;
  for (long long it = cta * WARPS + (tid >> 5); it < items; it += CLUSTER * WARPS) {
    const int b = (int)(it / chunks), j = (int)(it % chunks) * 32 + (tid & 31);
    int n = p.blocks[b];
    if (n < 0 || n > p.max_blocks) {
      set_status(p.status, KT_ERR_DEVICE_CHECK);
      n = n < 0 ? 0 : p.max_blocks;
    }
    if (j >= n) continue;
    const size_t at = (size_t)b * p.max_blocks + j;
    int page = p.table[at];
    const int to = page >= 0 && page < p.P ? p.list2[page] : -1;
    if (to < 0) set_status(p.status, KT_ERR_DEVICE_CHECK);  // no page, or counted as free
    else page = to;
    p.new_table[at] = page;
  }
}


// ---- copy --------------------------------------------------------------------------------
// A unit is up to COPY_UNIT bytes of one page in one pool, taken by a warp; the units of one
// move follow one another through all pools, so neighbouring warps read neighbouring bytes.
// Pages of 16-byte multiples move in 16-byte words, eight loads in flight a lane; others
// (scales of few heads) in 4-byte words.
// Bound by HBM: the 2.1 GB that compacting 8K pages of two layers moves take 330 us, 6.4 TB/s of
// 6.7 that a plain copy reaches; the 0.96 GB of an 8-bit pool 145 us, 6.6.  A few pages (a fork's last
// blocks) take 3 us: a launch and three dependent loads.
// With COPY_CTAS an SM (2 of which run at a time) a CTA's share is small enough for the SMs to end
// together: the larger compaction takes 368 us with 2, 357 with 4, 347 with 8, 338 with 32 and 335
// with 128, the 8-bit one 169, 164, 157, 153 and 160.
constexpr int COPY_UNIT = 4096;
constexpr int COPY_THREADS = 512;
constexpr int COPY_CTAS = 32;

struct CopyParams {
  const int32_t* moves;
  const int32_t* num_moves;
  int* status;
  int max_moves, P, n_pools, units;  // units of one move
  uint8_t* base[MAX_PAGE_POOLS];
  long long page_bytes[MAX_PAGE_POOLS];
  int first[MAX_PAGE_POOLS + 1];  // first unit of each pool
};

__global__ void __launch_bounds__(COPY_THREADS) copy_kernel(const __grid_constant__ CopyParams p) {
  griddep_wait();
  griddep_launch_dependents();
  int n = *p.num_moves;
  if (n < 0 || n > p.max_moves) {
    if (blockIdx.x == 0 && threadIdx.x == 0) set_status(p.status, KT_ERR_DEVICE_CHECK);
    n = n < 0 ? 0 : p.max_moves;
  }
  const int lane = threadIdx.x & 31;
  const long long units = (long long)n * p.units;
  const long long step = (long long)gridDim.x * (COPY_THREADS / 32);
  for (long long u = (long long)blockIdx.x * (COPY_THREADS / 32) + (threadIdx.x >> 5); u < units;
       u += step) {
    const long long m = u / p.units;
    const int k = (int)(u - m * p.units);
    const int from = p.moves[2 * m], to = p.moves[2 * m + 1];
    if (from < 0 || from >= p.P || to < 0 || to >= p.P) {
      if (lane == 0) set_status(p.status, KT_ERR_DEVICE_CHECK);
      continue;
    }
    if (from == to) continue;
    int pool = 0;  // the last pool whose first unit is not behind k
    for (int lo = 0, hi = p.n_pools; lo + 1 < hi;) {
      const int mid = (lo + hi) / 2;
      if (p.first[mid] <= k) lo = mid;
      else hi = mid;
      pool = lo;
    }
    const long long size = p.page_bytes[pool];
    const long long at = (long long)(k - p.first[pool]) * COPY_UNIT;
    const int bytes = (int)min((long long)COPY_UNIT, size - at);
    const uint8_t* src = p.base[pool] + from * size + at;
    uint8_t* dst = p.base[pool] + to * size + at;
    if (size % 16 == 0) {
      const uint4* s = reinterpret_cast<const uint4*>(src);
      uint4* d = reinterpret_cast<uint4*>(dst);
      const int words = bytes / 16;
      if (words == COPY_UNIT / 16) {
        uint4 v[COPY_UNIT / 512];
#pragma unroll
        for (int i = 0; i < COPY_UNIT / 512; ++i) v[i] = s[lane + 32 * i];
#pragma unroll
        for (int i = 0; i < COPY_UNIT / 512; ++i) d[lane + 32 * i] = v[i];
      } else {
        for (int i = lane; i < words; i += 32) d[i] = s[i];
      }
    } else {
      for (int i = lane; i < bytes / 4; i += 32)
        reinterpret_cast<uint32_t*>(dst)[i] = reinterpret_cast<const uint32_t*>(src)[i];
    }
  }
}

MapParams params_of(const PagesLaunch& a) {
  MapParams p;
  std::memset(&p, 0, sizeof(p));
  p.table = a.table;
  p.lens = a.lens;
  p.blocks = a.blocks;
  p.refs = a.refs;
  p.status = a.status;
  p.list = a.list;
  p.list2 = a.list2;
  p.a = a.a;
  p.b = a.b;
  p.moves = a.moves;
  p.num_moves = a.num_moves;
  p.new_table = a.new_table;
  p.new_refs = a.new_refs;
  p.n = a.n;
  p.batch = a.batch;
  p.max_blocks = a.max_blocks;
  p.P = a.P;
  return p;
}

// The kernels wait for the one before them on the stream themselves, so that their launch
// overlaps its end.
template <class P>
cudaError_t launch(void (*kernel)(P), const P& p, int grid, int threads, cudaStream_t stream) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_free_seqs(const PagesLaunch& a, cudaStream_t stream) {
  return launch(free_kernel, params_of(a), a.n, 256, stream);
}
cudaError_t launch_fork_seqs(const PagesLaunch& a, cudaStream_t stream) {
  return launch(fork_kernel, params_of(a), CLUSTER, THREADS, stream);
}
cudaError_t launch_reserve_pages(const PagesLaunch& a, cudaStream_t stream) {
  return launch(reserve_kernel, params_of(a), CLUSTER, THREADS, stream);
}
cudaError_t launch_compact_pages(const PagesLaunch& a, cudaStream_t stream) {
  return launch(compact_kernel, params_of(a), CLUSTER, THREADS, stream);
}

cudaError_t launch_copy_pages(const CopyLaunch& a, cudaStream_t stream) {
  CopyParams p;
  p.moves = a.moves;
  p.num_moves = a.num_moves;
  p.status = a.status;
  p.max_moves = a.max_moves;
  p.P = a.P;
  p.n_pools = a.n_pools;
  long long units = 0;
  for (int i = 0; i < a.n_pools; ++i) {
    p.base[i] = static_cast<uint8_t*>(a.pools[i].data);
    p.page_bytes[i] = a.pools[i].page_bytes;
    p.first[i] = (int)units;
    units += (a.pools[i].page_bytes + COPY_UNIT - 1) / COPY_UNIT;
    if (units > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  }
  p.first[a.n_pools] = (int)units;
  p.units = (int)units;
  const long long warps = (long long)a.max_moves * units;
  const long long most = (long long)a.num_sms * COPY_CTAS;
  const long long ctas = (warps + COPY_THREADS / 32 - 1) / (COPY_THREADS / 32);
  return launch(copy_kernel, p, (int)(ctas < most ? ctas : most), COPY_THREADS, stream);
}

}  // namespace kt
