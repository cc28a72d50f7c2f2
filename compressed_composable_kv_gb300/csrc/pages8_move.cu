// The pages of an 8-bit pool among its sequences: forking a batch (with what it
// gives back and takes) and compacting the pool.
//
// Both are a plan, then a copy.  The plan is one launch of a cluster of CTAs, which
// counts, ranks and lists pages in the order of their indices, with cluster barriers
// between its steps; every rank is a prefix sum, so a result does not depend on who
// comes first: a fork's k-th free page is the one with k free ones before it, and a
// compaction's k-th hole among the first `used` pages takes the k-th page in use behind
// them.  The plan writes its results to the workspace, so that the second launch may
// write outputs over inputs, and nothing where the plan found a bad value.  The copy
// moves the listed pages of every layer.
//
// What bounds them: a copy of some MB the memory (32 layers, 4 sequences forked to 32:
// 35.0 us, 6.8 TB/s read and written; 16 layers, 512 pages of 64 rows compacted: 88.3 us,
// 6.0 TB/s), a smaller call the plan's chain of steps, each a trip to L2 and a barrier, and
// the two launches (3 sequences forked to 7: 10.9 us; 97 pages compacted: 7.9 us).
#include <algorithm>

#include <cooperative_groups.h>

#include "pages8.h"

namespace cg = cooperative_groups;

namespace c2kv {

namespace {

constexpr int PL_CTAS = 8;   // at most; see plan_ctas
constexpr int PL_THREADS = 1024;
constexpr int MV_THREADS = 256;
constexpr int kPlanFewPages = 2048;   // see plan_ctas

// The workspace, in ints.
struct MoveWs {
  // header: [0, 8) and [8, 16) bad values found by each CTA, in two steps; then
  // counts of pages in slices, then how the plan ended
  static constexpr int kCounts = 16, kVoid = 24, kCopies = 25, kSrc0 = 26, kHeader = 64;
  int32_t* head;
  int32_t* held;    // [256] pages of each sequence
  int32_t* n_out;   // [256] (fork)
  int32_t* rows;    // [256] rows of each copy (fork)
  int32_t* refs;    // [n_pages]
  int32_t* src;     // [n_pages] pages copied, from entry head[kSrc0] on
  int32_t* dst;     // [n_pages] where to; fork: the free pages that are taken
  int32_t* map;     // [n_pages] (compact) new indices; fork: where the copies go
  int32_t* table;   // [batch][max_pages] (fork)

  __host__ __device__ MoveWs(int32_t* ws, int n_pages)
      : head(ws), held(ws + kHeader), n_out(held + kMaxPagedSeqs), rows(n_out + kMaxPagedSeqs),
        refs(rows + kMaxPagedSeqs), src(refs + n_pages), dst(src + max_of(n_pages)), map(dst + max_of(n_pages)),
        table(map + max_of(n_pages)) {}
  __host__ __device__ static int max_of(int n_pages) { return n_pages > kMaxPagedSeqs ? n_pages : kMaxPagedSeqs; }
};

__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& total) {   // exclusive prefix over the CTA
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const int w = warp_sums[lane];
    int s = w;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, s, off);
      if (lane >= off) s += o;
    }
    warp_sums[lane] = s - w;
    if (lane == 31) warp_sums[32] = s;
  }
  __syncthreads();
  const int before = warp_sums[warp] + incl - v;
  total = warp_sums[32];
  __syncthreads();
  return before;
}

// Sum over the CTAs of a count each, and over those before this one.
__device__ __forceinline__ void counts_of(const int32_t* counts, int rank, int& before, int& total) {
  before = total = 0;
  for (int i = 0; i < (int)gridDim.x; ++i) {
    const int c = __ldcg(counts + i);
    if (i < rank) before += c;
    total += c;
  }
}

__device__ __forceinline__ bool any_bad(const int32_t* flags) {
  int bad = 0;
  for (int i = 0; i < (int)gridDim.x; ++i) bad |= __ldcg(flags + i);
  return bad != 0;
}

template <bool FORK>
__global__ void __launch_bounds__(PL_THREADS, 1) plan_kernel(const __grid_constant__ MoveParams p) {
  __shared__ int warp_sums[33];
  __shared__ int s_n[kMaxPagedSeqs], s_held[kMaxPagedSeqs], s_kids[kMaxPagedSeqs], s_first[kMaxPagedSeqs];
  __shared__ int s_par[kMaxPagedSeqs], s_keep[kMaxPagedSeqs], s_want[kMaxPagedSeqs], s_base[kMaxPagedSeqs];
  cg::cluster_group cl = cg::this_cluster();
  const int ctas = (int)gridDim.x, rank = (int)cl.block_rank(), tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n_pages = p.pool.n_pages, page = p.pool.page, W = p.max_pages;
  const MoveWs ws(p.ws, n_pages);
  grid_wait();
  grid_release();

  // ---------------- the pages of each sequence (a warp each), checked
  bool bad = false;
  static_assert(PL_CTAS * PL_THREADS / 32 >= kMaxPagedSeqs, "a warp for each sequence");   // see plan_ctas
  const int row = rank * (PL_THREADS / 32) + warp;
  if (row < p.batch) {
    const int32_t* t = p.page_table + (size_t)row * W;
    int held = -1;
    for (int e0 = 0; held < 0; e0 += 128) {
      int32_t v[4], c[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = e0 + 32 * k + lane < W ? t[e0 + 32 * k + lane] : -1;
#pragma unroll
      for (int k = 0; k < 4; ++k) c[k] = v[k] >= 0 && v[k] < n_pages ? p.refs[v[k]] : 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (held >= 0) continue;
        const uint32_t end = __ballot_sync(0xffffffffu, v[k] < 0);
        if (end) held = e0 + 32 * k + __ffs(end) - 1;
        if (c[k] < 1 && (held < 0 || e0 + 32 * k + lane < held)) bad = true;
      }
    }
    if (lane == 0) ws.held[row] = held;
  }
  const int slice = (n_pages + ctas - 1) / ctas, lo = min(rank * slice, n_pages), hi = min(lo + slice, n_pages);
  int mine = 0;
  for (int x = lo + tid; x < hi; x += PL_THREADS) {
    const int32_t c = p.refs[x];
    bad |= c < 0;
    mine += c > 0 ? 1 : 0;
    if (FORK) ws.refs[x] = c;
  }
  int used_here;
  block_scan(mine, warp_sums, used_here);
  bad = __syncthreads_or(bad);
  if (tid == 0) {
    ws.head[rank] = bad;
    if (!FORK) ws.head[MoveWs::kCounts + rank] = used_here;
  }
  cl.sync();
  bad = any_bad(ws.head);

  if constexpr (FORK) {
    // ---------------- who goes on with whom (each CTA for itself)
    if (tid < kMaxPagedSeqs) {
      s_n[tid] = tid < p.batch ? p.n_cached[tid] : -1;
      s_held[tid] = tid < p.batch ? __ldcg(ws.held + tid) : 0;
      s_kids[tid] = 0;
      s_first[tid] = kMaxPagedSeqs;
    }
    __syncthreads();
    int r = -1;
    if (tid < p.batch_out) {
      r = p.parent[tid];
      bad |= r >= p.batch;
      if (r >= p.batch || (r >= 0 && s_n[r] < 0)) r = -1;
      if (r >= 0) {
        atomicAdd(&s_kids[r], 1);
        atomicMin(&s_first[r], tid);
      }
    }
    if (tid < p.batch) bad |= (int64_t)s_n[tid] > (int64_t)s_held[tid] * page;
    bad = __syncthreads_or(bad);
    int taken = 0;
    if (tid < kMaxPagedSeqs) {
      int keep = 0, want = 0;
      if (r >= 0 && !bad) {
        keep = s_first[r] == tid ? s_held[r] : s_n[r] / page;
        want = max(keep, (s_n[r] + p.room + page - 1) / page);
      }
      taken = want - keep;
      s_par[tid] = r;
      s_keep[tid] = keep;
      s_want[tid] = want;
      if (want > W) bad = true;
    }
    int need;
    const int base = block_scan(min(taken, W), warp_sums, need);
    if (tid < kMaxPagedSeqs) s_base[tid] = base;
    bad = __syncthreads_or(bad);
    if (bad) {   // the same in every CTA
      if (rank == 0 && tid == 0) ws.head[MoveWs::kVoid] = 1;
      return;
    }
    // ---------------- sharing: every child but one adds a reference to the full
    // pages; a sequence without a child gives its pages back
    if (row < p.batch) {
      const int held = s_held[row], full = max(s_n[row], 0) / page, kids = s_kids[row];
      const int32_t* t = p.page_table + (size_t)row * W;
      if (kids != 1)
        for (int e = lane; e < held; e += 32) {
          const int by = (e < full ? kids : min(kids, 1)) - 1;
          if (by != 0) atomicAdd(ws.refs + t[e], by);
        }
    }
    cl.sync();
    // ---------------- the free pages
    mine = 0;
    for (int x = lo + tid; x < hi; x += PL_THREADS) {
      const int32_t c = __ldcg(ws.refs + x);
      bad |= c < 0;   // the table names a page more often than refs says
      mine += c == 0 ? 1 : 0;
    }
    int free_here;
    block_scan(mine, warp_sums, free_here);
    bad = __syncthreads_or(bad);
    if (tid == 0) {
      ws.head[8 + rank] = bad;
      ws.head[MoveWs::kCounts + rank] = free_here;
    }
    cl.sync();
    int before, all;
    counts_of(ws.head + MoveWs::kCounts, rank, before, all);
    if (need > all || any_bad(ws.head + 8)) {
      if (rank == 0 && tid == 0) ws.head[MoveWs::kVoid] = 1;
      return;
    }
    for (int x0 = lo; x0 < hi && before < need; x0 += PL_THREADS) {
      const int x = x0 + tid;
      const bool is_free = x < hi && __ldcg(ws.refs + x) == 0;
      int found;
      const int k = before + block_scan(is_free ? 1 : 0, warp_sums, found);
      if (is_free && k < need) {
        ws.dst[k] = x;
        ws.refs[x] = 1;
      }
      before += found;
    }
    cl.sync();
    // ---------------- the new table, and what is copied
    for (int64_t i = (int64_t)rank * PL_THREADS + tid; i < (int64_t)p.batch_out * W; i += ctas * PL_THREADS) {
      const int b = (int)(i / W), e = (int)(i % W);
      int32_t v = -1;
      if (e < s_keep[b]) v = p.page_table[(size_t)s_par[b] * W + e];
      else if (e < s_want[b]) v = __ldcg(ws.dst + s_base[b] + e - s_keep[b]);
      ws.table[i] = v;
    }
    if (rank == 0) {
      const bool on = tid < p.batch_out && r >= 0;
      const int tail = on ? s_n[r] % page : 0;
      const bool copied = tail > 0 && s_first[r] != tid;
      int copies;
      const int k = block_scan(copied ? 1 : 0, warp_sums, copies);
      if (copied) {
        ws.src[k] = p.page_table[(size_t)r * W + s_n[r] / page];
        ws.map[k] = __ldcg(ws.dst + s_base[tid]);
        ws.rows[k] = tail;
      }
      if (tid < p.batch_out) ws.n_out[tid] = on ? s_n[r] : -1;
      if (tid == 0) {
        ws.head[MoveWs::kVoid] = 0;
        ws.head[MoveWs::kCopies] = copies;
        ws.head[MoveWs::kSrc0] = 0;
      }
    }
  } else {
    if (bad) {
      if (rank == 0 && tid == 0) ws.head[MoveWs::kVoid] = 1;
      return;
    }
    int before, used;
    counts_of(ws.head + MoveWs::kCounts, rank, before, used);
    if (rank == 0 && tid == 0) ws.head[MoveWs::kSrc0] = used;   // where no page lies behind them all
    cl.sync();
    // ---------------- ranks: the k-th hole below `used`; the page in use with u
    // others before it
    for (int x0 = lo; x0 < hi; x0 += PL_THREADS) {
      const int x = x0 + tid;
      const bool in_use = x < hi && p.refs[x] > 0;
      int found;
      const int u = before + block_scan(in_use ? 1 : 0, warp_sums, found);
      if (x < hi && x < used && !in_use) ws.dst[x - u] = x;
      if (x >= used && in_use) ws.src[u] = x;
      if (x < hi && x == used) ws.head[MoveWs::kSrc0] = u;
      before += found;
    }
    cl.sync();
    const int first = __ldcg(ws.head + MoveWs::kSrc0), moves = used - first;
    for (int x = lo + tid; x < hi; x += PL_THREADS) {
      const int32_t c = p.refs[x];
      if (x < used && c > 0) {
        ws.refs[x] = c;
        ws.map[x] = x;
      } else if (x < used) {
        ws.map[x] = -1;   // refs[x]: of the page that moves here
      } else {
        ws.refs[x] = 0;
        if (c == 0) ws.map[x] = -1;
      }
    }
    for (int k = rank * PL_THREADS + tid; k < moves; k += ctas * PL_THREADS) {
      const int src = __ldcg(ws.src + first + k), dst = __ldcg(ws.dst + k);
      ws.map[src] = dst;
      ws.refs[dst] = p.refs[src];
    }
    if (rank == 0 && tid == 0) {
      ws.head[MoveWs::kVoid] = 0;
      ws.head[MoveWs::kCopies] = moves;
    }
  }
}

// blockIdx.y: layer and K or V.  A warp copies the rows of one page and kv head.
template <bool FORK>
__global__ void __launch_bounds__(MV_THREADS) move_kernel(const __grid_constant__ MoveParams p, int row_bytes) {
  const MoveWs ws(p.ws, p.pool.n_pages);
  const int tid = threadIdx.x, lane = tid & 31;
  grid_wait();
  grid_release();
  if (ws.head[MoveWs::kVoid]) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) atomicOr(p.err, kErrLength);
    return;
  }
  {
    const int64_t at = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * MV_THREADS + tid;
    const int64_t all = (int64_t)gridDim.x * gridDim.y * MV_THREADS;
    for (int64_t x = at; x < p.pool.n_pages; x += all) {
      p.refs_out[x] = ws.refs[x];
      if (!FORK && p.moved_out) p.moved_out[x] = ws.map[x];
    }
    for (int64_t i = at; i < (int64_t)p.batch_out * p.max_pages; i += all) {
      if (FORK) p.page_table_out[i] = ws.table[i];
      else p.page_table_out[i] = i % p.max_pages < ws.held[i / p.max_pages] ? ws.map[p.page_table[i]] : -1;
    }
    if (FORK && at < p.batch_out) p.n_cached_out[at] = ws.n_out[at];
  }
  const int copies = ws.head[MoveWs::kCopies];
  const int32_t* from = ws.src + ws.head[MoveWs::kSrc0];
  const int32_t* to = FORK ? ws.map : ws.dst;
  const int kv = blockIdx.y & 1, layer = blockIdx.y >> 1, n_kv = p.pool.n_kv, page = p.pool.page;
  uint8_t* codes = p.pool.codes[kv] + layer * p.code_layer;
  float* scales = p.pool.scales[kv] + layer * p.scale_layer;
  for (int it = (int)blockIdx.x * (MV_THREADS / 32) + (tid >> 5); it < copies * n_kv; it += gridDim.x * (MV_THREADS / 32)) {
    const int k = it / n_kv, h = it - k * n_kv;
    const size_t src = (size_t)from[k] * n_kv + h, dst = (size_t)to[k] * n_kv + h;
    const int n = (FORK ? ws.rows[k] : page) * row_bytes / 16;
    const uint4* s = reinterpret_cast<const uint4*>(codes + src * page * row_bytes);
    uint4* d = reinterpret_cast<uint4*>(codes + dst * page * row_bytes);
    if (lane == 0) scales[dst] = scales[src];
    for (int i0 = lane; i0 < n; i0 += 256) {
      uint4 v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i0 + 32 * j < n) v[j] = __ldcs(s + i0 + 32 * j);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i0 + 32 * j < n) __stcs(d + i0 + 32 * j, v[j]);
    }
  }
}

template <typename K, typename... A>
cudaError_t launch_pdl(K kernel, dim3 grid, int cluster, int threads, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

size_t move_workspace_ints(int n_pages, int batch, int max_pages) {
  return (size_t)MoveWs::kHeader + 3 * kMaxPagedSeqs + n_pages + 3 * (size_t)MoveWs::max_of(n_pages) +
         (size_t)batch * max_pages;
}

// CTAs of the plan.  One spares the barriers of a cluster and its launch, eight share
// a long list of pages.  Compacting 256, 2048, 4096 and 16384 pages took 7.9, 9.3, 10.7
// and 17.7 us with one, 10.6, 11.3, 10.8 and 11.9 us with eight; a fork of 30 sequences
// with 2086 pages 13.4 against 15.2 us, with 7712 pages 22.1 against 18.7 us.
static int plan_ctas(const MoveParams& p) {
  const int rows = (p.batch + PL_THREADS / 32 - 1) / (PL_THREADS / 32);
  return rows == 1 && p.pool.n_pages <= kPlanFewPages ? 1 : PL_CTAS;
}

cudaError_t launch_pages8_plan(const MoveParams& p, cudaStream_t st) {
  const int n = plan_ctas(p);
  return p.n_cached ? launch_pdl(plan_kernel<true>, dim3(n), n, PL_THREADS, st, p)
                    : launch_pdl(plan_kernel<false>, dim3(n), n, PL_THREADS, st, p);
}

// A warp for each page and kv head that may have to be copied, up to eight CTAs an SM.
cudaError_t launch_pages8_move(const MoveParams& p, int head_dim, int sms, cudaStream_t st) {
  const int y = 2 * p.n_layers, warps = MV_THREADS / 32;
  const int64_t copies = p.n_cached ? p.batch_out : p.pool.n_pages / 2;
  const int64_t want = std::max<int64_t>(1, (copies * p.pool.n_kv + warps - 1) / warps);
  const dim3 grid((unsigned)std::min<int64_t>(want, (8 * sms + y - 1) / y), y);
  return p.n_cached ? launch_pdl(move_kernel<true>, grid, 1, MV_THREADS, st, p, head_dim)
                    : launch_pdl(move_kernel<false>, grid, 1, MV_THREADS, st, p, head_dim);
}

}  // namespace c2kv
