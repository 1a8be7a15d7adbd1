// cache.cu — the rows of the packed cache: copy, fork, free, compaction, and the
// commit of an accepted path of drafted tokens.
//
// A row holds one block's index page and latent page ("A KV cache for three kinds
// of state").  A row is free when no block table holds it (count 0), so there is
// no free list to keep: the lowest free rows are found by one scan of the counts.
// Every result is an integer or a copied byte; counts change by integer atomics,
// whose order cannot change the sums, and rows are handed out by position, not by
// arrival, so all results are deterministic.
#include "cache.cuh"

// Every kernel here may be scheduled before the kernel before it on the stream has ended
// (programmatic launch) and waits for it before it touches memory: the launches of a
// free, a fork and a copy in a row overlap.
namespace dsa {

namespace {

// Sum over the block and this thread's exclusive prefix; wsh: 33 words.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* wsh, uint32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();   // an earlier call's words have been read
  if (lane == 31) wsh[warp] = x;
  __syncthreads();
  const uint32_t wv = lane < nw ? wsh[lane] : 0u;
  total = __reduce_add_sync(0xffffffffu, wv);
  return __reduce_add_sync(0xffffffffu, lane < warp ? wv : 0u) + x - v;
}

}  // namespace

// ------------------------------------------------------------------- row copies
//
// One unit is 16 KB of one row: 256 threads, four 16-byte loads in flight each, then
// the stores.  Units of all pairs are handed round-robin to a grid that fills the GPU.
// Bound by HBM, 2 bytes moved per byte copied: 240 MB of rows take 72 us, 98 % of the rate of
// a plain copy.
constexpr int kCopyThreads = 256;
constexpr int kCopyVec = 4;
constexpr int kCopyUnit = kCopyThreads * kCopyVec * 16;

__global__ void __launch_bounds__(kCopyThreads) cache_copy_kernel(CacheCopyParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const int64_t per_row = cdiv(p.row_bytes, kCopyUnit);
  int64_t n = p.n;
  if (p.count) {
    const int64_t c = __ldcg(p.count);
    n = c < n ? (c < 0 ? 0 : c) : n;
  }
  for (int64_t u = blockIdx.x; u < n * per_row; u += gridDim.x) {
    // (32 bits divide in a tenth of the instructions)
    const int64_t i = u >> 32 ? u / per_row : static_cast<uint32_t>(u) / static_cast<uint32_t>(per_row);
    const int64_t off = (u - i * per_row) * kCopyUnit;
    const int32_t s = __ldcg(p.src + i), d = __ldcg(p.dst + i);
    if (s < 0 && d < 0) continue;
    if (s < 0 || d < 0 || s >= p.num_rows || d >= p.num_rows) {
      if (threadIdx.x == 0) atomicOr(p.status, DEV_BAD_BLOCK);
      continue;
    }
    if (s == d) continue;
    const uint4* from = reinterpret_cast<const uint4*>(p.pool + static_cast<int64_t>(s) * p.row_stride + off);
    uint4* to = reinterpret_cast<uint4*>(p.pool + static_cast<int64_t>(d) * p.row_stride + off);
    const int64_t left = (p.row_bytes - off) / 16;   // row strides are multiples of 16
    uint4 v[kCopyVec];
#pragma unroll
    for (int k = 0; k < kCopyVec; ++k) {
      const int e = threadIdx.x + k * kCopyThreads;
      if (e < left) v[k] = __ldcs(from + e);
    }
#pragma unroll
    for (int k = 0; k < kCopyVec; ++k) {
      const int e = threadIdx.x + k * kCopyThreads;
      if (e < left) __stcs(to + e, v[k]);
    }
  }
}

cudaError_t launch_cache_copy(const CacheCopyParams& p, int nsm, cudaStream_t st) {
  if (p.n == 0) return cudaSuccess;
  const int64_t units = p.n * cdiv(p.row_bytes, kCopyUnit);
  const int64_t full = static_cast<int64_t>(nsm) * (2048 / kCopyThreads);
  const unsigned grid = static_cast<unsigned>(units < full ? units : full);
  return launch_ex(cache_copy_kernel, dim3(grid), dim3(kCopyThreads), 0, st, true, 0u, p);
}

// ------------------------------------------------------------------------- fork
//
// The plan: one CTA, or a cluster of eight for more rows than kOneCtaRows, scans the counts
// (each CTA its part of the rows) and lists the first free rows in ascending order; the
// first CTA checks the forks and numbers those that need a row.  The apply copies the
// table rows and counts the shared blocks: in the plan's CTAs when that is little, else
// in a second launch with CTAs per fork.
constexpr int kPlanThreads = 1024;
constexpr int kPlanCtas = 8;
// A free, a fork of 2 requests to 8 and the copies, 600 rows: 15.3 us together with one CTA and
// one launch, 17.7 us with a cluster and two; the launches bound it (11.5 us in a graph).
constexpr int64_t kOneCtaRows = 16384;
// The plan's CTAs handle the tables, too, where each of their threads has one entry at most.  Free + fork
// of 512 / 1,024 / 2,048 / 4,096 / 8,192 entries by one CTA: 9.3 / 9.4 / 10.8 / 13.9 / 18.7 us so, 11.3 / 11.1 /
// 11.0 / 11.2 / 13.5 with a launch of their own; by the cluster, 8,192 / 32,768 entries: 12.3 / 17.3 and
// 12.7 / 14.9; compaction alike, 1,024 / 8,192 by one CTA: 11.2 / 14.5 and 10.6 / 11.2, and a launch less.
constexpr int64_t kOneLaunchEntries = kPlanThreads;   // table entries per plan CTA

unsigned plan_ctas(int64_t num_rows) { return num_rows <= kOneCtaRows ? 1u : static_cast<unsigned>(kPlanCtas); }

// Rows [r0, r1) of the cluster's CTA `rank`, multiples of 4 rows.
__device__ __forceinline__ void plan_rows(int64_t num_rows, uint32_t rank, int64_t& r0, int64_t& r1) {
  const int64_t per = (cdiv(num_rows, cluster_size()) + 3) / 4 * 4;
  r0 = per * rank;
  if (r0 > num_rows) r0 = num_rows;
  r1 = r0 + per < num_rows ? r0 + per : num_rows;
}

// Free (count <= 0) bits of the four rows r..r+3, those at or behind r1 not counted.
__device__ __forceinline__ uint32_t free_bits(const int32_t* ref, int64_t r, int64_t r1) {
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (r + k < r1 && __ldcg(ref + r + k) <= 0) m |= 1u << k;
  return m;
}

// Free rows of [r0, r1), all threads of the CTA.
__device__ __forceinline__ uint32_t count_free(const int32_t* ref, int64_t r0, int64_t r1, uint32_t* wsh) {
  uint32_t n = 0;
  for (int64_t r = r0 + 4 * threadIdx.x; r < r1; r += 4 * kPlanThreads) n += __popc(free_bits(ref, r, r1));
  uint32_t total;
  block_scan(n, wsh, total);
  return total;
}

// Every CTA's count in every CTA: `mine` of this one; the sum of the ranks before it and of all.
__device__ __forceinline__ void share_counts(uint32_t mine, uint32_t* counts, uint32_t rank, int64_t& before,
                                             int64_t& all) {
  const uint32_t csize = cluster_size();
  if (threadIdx.x < csize) st_cluster_u32(cluster_map(smem_u32(&counts[rank]), threadIdx.x), mine);
  cluster_sync();
  before = all = 0;
  for (uint32_t r = 0; r < csize; ++r) {
    if (r < rank) before += counts[r];
    all += counts[r];
  }
}

// What the plan's first CTA keeps of the forks in shared memory, when there are at most
// kPlanThreads of them and the list of free rows is this CTA's own.
struct ForkShared {
  int32_t rows[kPlanThreads];   // first free rows
  int32_t plan[kPlanThreads];   // the plan, and the parents' lengths
  int32_t lens[kPlanThreads];
};

// Checks the forks and numbers those that need a row (of `all` free ones).  One CTA; a0, c0: the
// thread's first fork (-1 behind the last).  `marks`: zeroed counters of the requests.
__device__ __forceinline__ void plan_forks(const ForkParams& p, int64_t all, int32_t* marks, bool small, ForkShared& fs,
                                           int32_t a0, int32_t c0, uint32_t* wsh) {
  // the first round's lengths arrive meanwhile
  const bool in0 = a0 >= 0 && a0 < p.num_reqs && c0 >= 0 && c0 < p.num_reqs;
  const int32_t la0 = in0 ? __ldcg(p.ctx + a0) : 0, lc0 = in0 ? __ldcg(p.ctx + c0) : 0;
  // who is named: children counted in the low half, parents flagged above
  for (int i = threadIdx.x; i < p.n; i += kPlanThreads) {
    const int32_t a = i < kPlanThreads ? a0 : __ldcg(p.parent + i), c = i < kPlanThreads ? c0 : __ldcg(p.child + i);
    if (a < 0) continue;
    if (a < p.num_reqs) atomicOr(marks + a, 1 << 30);
    if (c >= 0 && c < p.num_reqs) atomicAdd(marks + c, 1);
  }
  __threadfence_block();
  __syncthreads();
  uint32_t base = 0;
  for (int i0 = 0; i0 < p.n; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    bool ok = false, need = false, named = false;
    int64_t L = 0;
    int32_t b = -1;
    if (i < p.n) {
      const int32_t a = i0 == 0 ? a0 : __ldcg(p.parent + i), c = i0 == 0 ? c0 : __ldcg(p.child + i);
      named = a >= 0;
      if (named && a < p.num_reqs && c >= 0 && c < p.num_reqs && *static_cast<volatile int32_t*>(marks + c) == 1 &&
          (i0 == 0 ? lc0 : __ldcg(p.ctx + c)) == 0) {
        L = i0 == 0 ? la0 : __ldcg(p.ctx + a);
        ok = L >= 0 && L <= (static_cast<int64_t>(p.bt_stride) << p.log2_bs);
        need = ok && (L & ((1 << p.log2_bs) - 1)) != 0;
        if (need) b = __ldcg(p.bt + static_cast<int64_t>(a) * p.bt_stride + (L >> p.log2_bs));
      }
    }
    uint32_t total;
    const int64_t o = base + block_scan(need ? 1u : 0u, wsh, total);
    base += total;
    int32_t row = -1;
    if (need) {
      if (o < all) row = small ? fs.rows[o] : __ldcg(p.free_list + o);
      else ok = false;
    }
    if (i < p.n) {
      if (named && !ok) atomicOr(p.status, DEV_BAD_BATCH);
      p.plan[i] = ok ? row : kForkSkip;
      if (small) {
        fs.plan[i] = ok ? row : kForkSkip;
        fs.lens[i] = static_cast<int32_t>(L);
      }
      int32_t from = -1;
      if (ok && need) {
        if (b >= 0 && b < p.num_rows) from = b;
        else atomicOr(p.status, DEV_BAD_BLOCK);
      }
      p.copy_src[i] = from;
      p.copy_dst[i] = from >= 0 ? row : -1;
    }
  }
}

// One table entry of fork i of a parent with L tokens to request c; b: the parent's entry.
__device__ __forceinline__ void apply_fork(const ForkParams& p, int32_t c, int32_t L, int32_t row, int32_t b, int e) {
  const int32_t full = L >> p.log2_bs;
  if (e < full) {
    if (b >= 0 && b < p.num_rows) {
      atomicAdd(p.ref + b, 1);
    } else {
      atomicOr(p.status, DEV_BAD_BLOCK);
      b = -1;
    }
  } else if (e == full && row >= 0) {
    b = row;
    p.ref[row] = 1;
  } else {
    b = -1;
  }
  p.bt[static_cast<int64_t>(c) * p.bt_stride + e] = b;
  if (e == 0) p.ctx[c] = L;
}

constexpr int kMarks = 4096;   // counters of as many requests fit shared memory

__global__ void __launch_bounds__(kPlanThreads) cache_fork_plan_kernel(ForkParams p) {
  __shared__ uint32_t wsh[33];
  __shared__ uint32_t counts[kPlanCtas];
  __shared__ ForkShared fs;
  __shared__ int32_t marks_sh[kMarks];
  const uint32_t rank = cluster_rank();
  const bool small = cluster_size() == 1 && p.n <= kPlanThreads;
  int32_t* marks = p.num_reqs <= kMarks ? marks_sh : p.marks;
  const int tid = static_cast<int>(threadIdx.x);
  grid_dep_wait();
  grid_dep_launch();
  // loads that nothing depends on yet: the forks, and the free rows among this CTA's rows
  int32_t a0 = -1, c0 = -1;
  if (rank == 0 && tid < p.n) {
    a0 = __ldcg(p.parent + tid);
    c0 = __ldcg(p.child + tid);
  }
  int64_t r0, r1;
  plan_rows(p.num_rows, rank, r0, r1);
  constexpr int kKept = 8;   // rounds of 4,096 rows whose bits stay in a register
  uint32_t bits = 0, mine = 0;
  {
#pragma unroll
    for (int q = 0; q < kKept; ++q) {
      const int64_t r = r0 + 4 * (tid + q * kPlanThreads);
      if (r < r1) bits |= free_bits(p.ref, r, r1) << (4 * q);
    }
    uint32_t k = __popc(bits);
    for (int64_t r = r0 + 4 * (tid + kKept * kPlanThreads); r < r1; r += 4 * kPlanThreads)
      k += __popc(free_bits(p.ref, r, r1));
    block_scan(k, wsh, mine);
  }
  if (rank == 0)
    for (int i = tid; i < p.num_reqs; i += kPlanThreads) marks[i] = 0;
  cluster_sync();   // every CTA has started before any writes into it
  int64_t before, all;
  share_counts(mine, counts, rank, before, all);
  // list the first free rows, up to one per fork
  uint32_t at = 0;   // free rows of this CTA before the round
  int q = 0;
  for (int64_t c = r0; c < r1 && before + at < p.n; c += 4 * kPlanThreads, ++q) {
    const int64_t r = c + 4 * tid;
    const uint32_t m = q < kKept ? (bits >> (4 * q)) & 15u : (r < r1 ? free_bits(p.ref, r, r1) : 0u);
    uint32_t total;
    int64_t o = before + at + block_scan(__popc(m), wsh, total);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if ((m >> k) & 1u) {
        if (o < p.n) (small ? fs.rows : p.free_list)[o] = static_cast<int32_t>(r + k);
        ++o;
      }
    at += total;
  }
  __threadfence();
  cluster_sync();   // the list is complete and visible
  if (rank == 0) plan_forks(p, all, marks, small, fs, a0, c0, wsh);
  if (!p.apply_here) return;
  __threadfence();
  cluster_sync();   // so is the plan
  // (a parent is no child of this call, so its table row and length are not written here)
  const uint32_t stride = static_cast<uint32_t>(p.bt_stride), entries = p.n * stride;   // few: apply_here
  for (uint32_t x = rank * kPlanThreads + tid; x < entries; x += cluster_size() * kPlanThreads) {
    const int i = static_cast<int>(x / stride), e = static_cast<int>(x % stride);
    const int32_t row = small ? fs.plan[i] : __ldcg(p.plan + i);
    if (row == kForkSkip) continue;
    const int32_t a = __ldcg(p.parent + i), c = __ldcg(p.child + i);
    const int32_t L = small ? fs.lens[i] : __ldcg(p.ctx + a);
    apply_fork(p, c, L, row, __ldcg(p.bt + static_cast<int64_t>(a) * p.bt_stride + e), e);
  }
}

constexpr int kApplyThreads = 256;
constexpr int kApplyEntries = 1024;   // table entries per CTA

__global__ void __launch_bounds__(kApplyThreads) cache_fork_apply_kernel(ForkParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const int i = blockIdx.x;
  const int32_t row = __ldcg(p.plan + i), a = __ldcg(p.parent + i), c = __ldcg(p.child + i);
  if (row == kForkSkip) return;
  const int32_t L = __ldcg(p.ctx + a);
  const int e1 = min(p.bt_stride, static_cast<int>(blockIdx.y + 1) * kApplyEntries);
  for (int e = blockIdx.y * kApplyEntries + threadIdx.x; e < e1; e += kApplyThreads)
    apply_fork(p, c, L, row, __ldcg(p.bt + static_cast<int64_t>(a) * p.bt_stride + e), e);
}

cudaError_t launch_cache_fork(const ForkParams& in, cudaStream_t st) {
  if (in.n == 0) return cudaSuccess;
  ForkParams p = in;
  const unsigned ctas = plan_ctas(p.num_rows);
  p.apply_here = static_cast<int64_t>(p.n) * p.bt_stride <= kOneLaunchEntries * ctas;
  cudaError_t e = launch_ex(cache_fork_plan_kernel, dim3(ctas), dim3(kPlanThreads), 0, st, true, ctas, p);
  if (e != cudaSuccess || p.apply_here) return e;
  return launch_ex(cache_fork_apply_kernel, dim3(p.n, static_cast<unsigned>(cdiv(p.bt_stride, kApplyEntries))),
                   dim3(kApplyThreads), 0, st, true, 0u, p);
}

// ------------------------------------------------------------------------- free
//
// Each entry is claimed by an exchange with -1, so a request that is named twice, or
// by two CTAs, gives back every block once.  Latency bound: three dependent round trips, 3.5 us
// by itself for 8 requests, 7 us for 256.
__global__ void __launch_bounds__(kApplyThreads) cache_free_kernel(FreeParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const int32_t r = __ldcg(p.reqs + blockIdx.x);
  if (r < 0) return;
  if (r >= p.num_reqs) {
    if (threadIdx.x == 0 && blockIdx.y == 0) atomicOr(p.status, DEV_BAD_BATCH);
    return;
  }
  int32_t* row = p.bt + static_cast<int64_t>(r) * p.bt_stride;
  const int e1 = min(p.bt_stride, static_cast<int>(blockIdx.y + 1) * kApplyEntries);
  for (int e = blockIdx.y * kApplyEntries + threadIdx.x; e < e1; e += kApplyThreads) {
    if (__ldcg(row + e) < 0) continue;
    const int32_t b = atomicExch(row + e, -1);
    if (b < 0) continue;
    if (b >= p.num_rows) {
      atomicOr(p.status, DEV_BAD_BLOCK);
    } else if (atomicSub(p.ref + b, 1) <= 0) {
      atomicAdd(p.ref + b, 1);
      atomicOr(p.status, DEV_BAD_BLOCK);
    }
  }
  if (blockIdx.y == 0 && threadIdx.x == 0) p.ctx[r] = 0;
}

cudaError_t launch_cache_free(const FreeParams& p, cudaStream_t st) {
  if (p.n == 0) return cudaSuccess;
  return launch_ex(cache_free_kernel, dim3(p.n, static_cast<unsigned>(cdiv(p.bt_stride, kApplyEntries))),
                   dim3(kApplyThreads), 0, st, true, 0u, p);
}

// ------------------------------------------------------------------- compaction
//
// The plan's CTAs count the used rows L; then each CTA numbers its holes (free rows
// before L) and movers (used rows at or behind L) and writes them to their places in
// the two lists; then the lists, complete, give the remaining counts and the map from
// old row to new.  The block tables are mapped in the same launch when they are small.
// Latency bound, barriers of the cluster and round trips to memory: 10.5 us by itself for 600
// rows, 12 us for 24K and 3.5 for their tables.

// One table entry's row after the moves.
__device__ __forceinline__ void map_entry(const CompactParams& p, int64_t e) {
  const int32_t b = __ldcg(p.bt + e);
  int32_t to = -1;
  if (b >= 0) {
    if (b < p.num_rows) to = __ldcg(p.remap + b);
    if (to < 0) atomicOr(p.status, DEV_BAD_BLOCK);
  }
  p.to_bt[e] = to;
}

__global__ void __launch_bounds__(kPlanThreads) cache_compact_plan_kernel(CompactParams p) {
  __shared__ uint32_t wsh[33];
  __shared__ uint32_t c_free[kPlanCtas], c_hole[kPlanCtas];
  const uint32_t rank = cluster_rank();
  grid_dep_wait();
  grid_dep_launch();
  cluster_sync();
  int64_t r0, r1;
  plan_rows(p.num_rows, rank, r0, r1);
  int64_t free_before, free_all;
  share_counts(count_free(p.ref, r0, r1, wsh), c_free, rank, free_before, free_all);
  const int64_t L = p.num_rows - free_all;
  // holes before this CTA's rows: the free rows before them that lie before L
  const int64_t h1 = r1 < L ? r1 : (r0 < L ? L : r0);   // this CTA's holes lie in [r0, h1)
  const uint32_t holes_here = h1 == r1 ? c_free[rank] : count_free(p.ref, r0, h1, wsh);
  int64_t hole, m;
  share_counts(holes_here, c_hole, rank, hole, m);
  // movers before this CTA's rows: used rows of [L, r0)
  int64_t mover = r0 > L ? (r0 - free_before) - (L - m) : 0;
  for (int64_t c = r0; c < r1; c += 4 * kPlanThreads) {
    const int64_t r = c + 4 * threadIdx.x;
    uint32_t fm = 0, hm = 0, mm = 0;
    int32_t v[4] = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (r + k >= r1) continue;
      v[k] = __ldcg(p.ref + r + k);
      if (v[k] <= 0) {
        fm |= 1u << k;
        if (r + k < L) hm |= 1u << k;
      } else if (r + k >= L) {
        mm |= 1u << k;
      }
    }
    uint32_t total;
    const uint32_t ex = block_scan((__popc(hm) << 16) | __popc(mm), wsh, total);   // at most 4096 each
    int64_t ho = hole + (ex >> 16), mo = mover + (ex & 0xFFFFu);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (r + k >= r1) continue;
      const int32_t row = static_cast<int32_t>(r + k);
      if ((hm >> k) & 1u) p.copy_dst[ho++] = row;
      if ((mm >> k) & 1u) {
        p.copy_src[mo++] = row;   // its count moves below
      } else {
        p.remap[row] = ((fm >> k) & 1u) ? -1 : row;
        p.to_ref[row] = ((fm >> k) & 1u) ? 0 : v[k];
      }
    }
    hole += total >> 16;
    mover += total & 0xFFFFu;
  }
  if (rank == 0 && threadIdx.x == 0) {
    p.counts[0] = static_cast<int32_t>(L);
    p.counts[1] = static_cast<int32_t>(m);
  }
  __threadfence();
  cluster_sync();   // both lists are complete and visible
  const int64_t tid = static_cast<int64_t>(rank) * kPlanThreads + threadIdx.x;
  const int64_t cap = p.num_rows / 2 > 0 ? p.num_rows / 2 : 1;
  const int64_t threads = static_cast<int64_t>(cluster_size()) * kPlanThreads;
  for (int64_t i = tid; i < cap; i += threads) {
    if (i < m) {
      const int32_t s = __ldcg(p.copy_src + i), d = __ldcg(p.copy_dst + i);
      const int32_t v = __ldcg(p.ref + s);   // read before either place is written (they may be one array)
      p.remap[s] = d;
      p.to_ref[d] = v;
      p.to_ref[s] = 0;
    } else {
      p.copy_src[i] = -1;
      p.copy_dst[i] = -1;
    }
  }
  if (!p.tables_here) return;
  __threadfence();
  cluster_sync();   // the map is complete and visible
  const int64_t n = static_cast<int64_t>(p.num_reqs) * p.bt_stride;
  for (int64_t e = tid; e < n; e += threads) map_entry(p, e);
}

__global__ void __launch_bounds__(kApplyThreads) cache_compact_tables_kernel(CompactParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const int64_t n = static_cast<int64_t>(p.num_reqs) * p.bt_stride;
  for (int64_t e = blockIdx.x * static_cast<int64_t>(kApplyThreads) + threadIdx.x; e < n;
       e += static_cast<int64_t>(gridDim.x) * kApplyThreads)
    map_entry(p, e);
}

cudaError_t launch_cache_compact(const CompactParams& in, int nsm, cudaStream_t st) {
  CompactParams p = in;
  const int64_t entries = static_cast<int64_t>(p.num_reqs) * p.bt_stride;
  const unsigned ctas = plan_ctas(p.num_rows);
  p.tables_here = entries <= kOneLaunchEntries * ctas;
  cudaError_t e = launch_ex(cache_compact_plan_kernel, dim3(ctas), dim3(kPlanThreads), 0, st, true, ctas, p);
  if (e != cudaSuccess || p.tables_here) return e;
  const int64_t blocks = cdiv(entries, kApplyThreads);
  const int64_t full = static_cast<int64_t>(nsm) * 8;
  return launch_ex(cache_compact_tables_kernel, dim3(static_cast<unsigned>(blocks < full ? blocks : full)),
                   dim3(kApplyThreads), 0, st, true, 0u, p);
}

// ----------------------------------------------------------------------- commit
//
// One CTA per request.  Accepted slots ascend, so slot accept[i] >= i: records move
// down or stay, and a chunk of records read whole before it is written never
// overwrites one that a later chunk reads.  A record is 16-byte pieces of its index
// codes and latent plus one 4-byte word (key scale or four exponents).  Latency
// bound: four dependent loads (accepted slots, block table, record) for a few KB, 2.5 us in a graph
// for one request, 5.5 us by itself for 256.
constexpr int kCommitChunk = 8;      // records per round
constexpr int kCommitThreads = 384;  // >= 8 records x (8 + 36 + 1) pieces

__global__ void __launch_bounds__(kCommitThreads) tree_commit_kernel(CommitParams p) {
  __shared__ int32_t slots[kCommitChunk];
  __shared__ int bad_sh;
  grid_dep_wait();
  grid_dep_launch();
  const int r = blockIdx.x;
  const int32_t* acc = p.accept + static_cast<int64_t>(r) * p.max_accept;
  const int32_t base = p.base[r], L = p.ctx[r];
  const bool sane = base >= 0 && base <= L && L <= p.max_ctx;
  const int32_t* btrow = p.bt + static_cast<int64_t>(r) * p.bt_stride;
  // the whole row is checked before anything moves
  int m = p.max_accept;       // entries before the first negative one
  if (threadIdx.x == 0) bad_sh = sane ? 0 : 1;
  __syncthreads();
  for (int i0 = 0; i0 < p.max_accept; i0 += kCommitThreads) {
    const int i = i0 + threadIdx.x;
    const int32_t a = i < p.max_accept ? acc[i] : -1;
    const unsigned neg = __ballot_sync(0xffffffffu, a < 0);
    __shared__ int first[kCommitThreads / 32];
    if ((threadIdx.x & 31) == 0) first[threadIdx.x >> 5] = neg ? __ffs(neg) - 1 : 32;
    __syncthreads();
    int k = 0;
    while (k < kCommitThreads / 32 && first[k] == 32) ++k;
    const int stop = i0 + 32 * k + (k < kCommitThreads / 32 ? first[k] : 0);
    if (stop < m) m = stop;
    if (i < m) {
      const int32_t prev = i > 0 ? acc[i - 1] : -1;
      const int64_t s = static_cast<int64_t>(base) + a;
      bool good = sane && a > prev && s < L;
      if (good) {
        const int32_t b0 = btrow[s >> p.pool.log2_bs], b1 = btrow[(base + i) >> p.pool.log2_bs];
        if (b0 < 0 || b0 >= p.pool.num_rows || b1 < 0 || b1 >= p.pool.num_rows) good = false;
      }
      if (!good) bad_sh = 1;
    }
    __syncthreads();
    if (stop < i0 + kCommitThreads) break;   // uniform
  }
  if (bad_sh) {
    if (threadIdx.x == 0) atomicOr(p.status, DEV_BAD_BATCH);
    return;
  }
  if (p.new_lens && threadIdx.x == 0) p.new_lens[r] = base + m;
  const int code_pieces = p.pool.idx_fmt == 0 ? 8 : 4;       // 128 or 64 bytes of key codes
  const int lat_bytes = p.pool.lat_fmt == 0 ? kLatDim : 352;
  const int pieces = code_pieces + lat_bytes / 16 + 1;
  const int bsm = p.pool.bs - 1;
  for (int i0 = 0; i0 < m; i0 += kCommitChunk) {
    const int n = min(kCommitChunk, m - i0);
    if (threadIdx.x < n) slots[threadIdx.x] = acc[i0 + threadIdx.x];
    __syncthreads();
    const int j = threadIdx.x / pieces, w = threadIdx.x % pieces;
    const bool act = j < n && slots[j < kCommitChunk ? j : 0] != i0 + j;
    uint4 v = make_uint4(0, 0, 0, 0);
    uint8_t* to = nullptr;
    bool word = false;
    if (act) {
      auto at = [&](int32_t s) -> uint8_t* {
        uint8_t* row = p.pool_w + static_cast<int64_t>(btrow[s >> p.pool.log2_bs]) * p.pool.row_stride;
        const int64_t slot = s & bsm;
        if (w < code_pieces) return row + p.pool.idx_off + slot * (code_pieces * 16) + w * 16;
        if (w == code_pieces) return row + p.pool.idx_off + static_cast<int64_t>(p.pool.bs) * (code_pieces * 16) + slot * 4;
        return row + p.pool.lat_off + slot * lat_bytes + (w - code_pieces - 1) * 16;
      };
      word = w == code_pieces;
      const uint8_t* from = at(base + slots[j]);
      to = at(base + i0 + j);
      if (word) v.x = *reinterpret_cast<const uint32_t*>(from);
      else v = *reinterpret_cast<const uint4*>(from);
    }
    __syncthreads();
    if (act) {
      if (word) *reinterpret_cast<uint32_t*>(to) = v.x;
      else *reinterpret_cast<uint4*>(to) = v;
    }
    __syncthreads();
  }
}

cudaError_t launch_tree_commit(const CommitParams& p, int num_reqs, cudaStream_t st) {
  return launch_ex(tree_commit_kernel, dim3(num_reqs), dim3(kCommitThreads), 0, st, true, 0u, p);
}

}  // namespace dsa
