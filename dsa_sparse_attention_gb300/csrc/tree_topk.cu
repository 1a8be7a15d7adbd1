// tree_topk.cu — exact top-k of drafted tokens' indexer scores, over the positions each
// token sees in its tree (include/dsa.h, dsa_tree).
//
// A verification batch holds many long rows, so the pass over the scores is what
// counts: it is made once.
//  1. bound:  one CTA per row reads 8,192 scores, one at a hashed place of each of as
//             many equal stretches, and takes the sample's rank m + 6 sqrt(m) + 8 as the
//             row's bound, m = 8,192 k / n being the number of samples expected among
//             the k best.  Fewer than k scores then lie at or above the bound with
//             probability below 1e-6, and typically 1.4 k (64K scores) to 3 k (1M) do.
//  2. filter: one CTA per 4,096 scores lists its scores at or above the bound, in
//             position order, and notes where its entries lie.
//  3. select: one CTA per row gathers the entries chunk by chunk, so in position order,
//             into shared memory, resolves the threshold key in three digit passes, and
//             the position cut among equal keys where not all of them fit (lowest
//             positions first), and writes the selection with one scan.
// Rows of at most 16,384 scores go to step 3 directly.  Steps 1 and 2 only choose what
// step 3 looks at: it counts the entries, and a row whose entries are too few or too
// many (more equal scores than the list holds) is resolved over the whole row, exactly
// and slowly.  No sum depends on an order of arrival: results are deterministic and
// independent of the rest of the batch.
#include "params.cuh"

namespace dsa {

namespace {

constexpr int kBins = 2048;
constexpr int kFilterThreads = 256;
constexpr int kPer = 16;                 // scores per thread and chunk
static_assert(kFilterThreads * kPer == kTopkChunk, "chunk");
constexpr int kRowThreads = 1024;
constexpr int kSamples = 8192;

// A row: n positions, `base` of them committed, `seen` seen by the token.
struct Row {
  int req, n, base, seen;
  const uint32_t* mask;
};

// False for a padding token.  Whole warps.
__device__ __forceinline__ bool load_row(const TreeTopkParams& p, int t, Row& r) {
  int pos;
  if (!load_tree_token(p.b, p.tree, t, p.status, r.req, pos, r.base)) return false;
  r.n = pos + 1;
  r.base = min(r.base, r.n);
  r.mask = p.tree.mask + static_cast<int64_t>(t) * p.tree.words;
  // bits of the drafted positions up to pos, one word per lane (at most 32 words)
  const int lane = threadIdx.x & 31;
  const int d = r.n - r.base;
  uint32_t w = lane < p.tree.words && 32 * lane < d ? __ldg(r.mask + lane) : 0u;
  if (32 * lane < d && 32 * lane + 32 > d) w &= (1u << (d - 32 * lane)) - 1u;
  r.seen = r.base + static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<uint32_t>(__popc(w))));
  return true;
}

// Steps 1 and 2 take part.
__device__ __forceinline__ bool filtered(const TreeTopkParams& p, const Row& r) {
  return r.seen > p.k && r.n > kTreeTopkCap;
}

// Key of position s, 0 (below every score's key) where the token does not see it.
__device__ __forceinline__ uint32_t seen_key(const TreeTopkParams& p, const Row& r, int s, float v) {
  return s < r.base || tree_sees(r.mask, p.tree.words, r.base, s) ? score_key(v) : 0u;
}

// Position of output entry o when everything seen is selected (-1 past the last).
__device__ __forceinline__ int seen_position(const TreeTopkParams& p, const Row& r, int o) {
  if (o < r.base) return o;
  if (o >= r.seen) return -1;
  int left = o - r.base;   // the left-th set bit of the mask
  for (int w = 0; w < p.tree.words; ++w) {
    uint32_t bits = __ldg(r.mask + w);
    const int c = __popc(bits);
    if (left >= c) {
      left -= c;
      continue;
    }
    while (left-- > 0) bits &= bits - 1;
    return r.base + 32 * w + __ffs(bits) - 1;
  }
  return -1;
}

// Exclusive prefix over the block and its total, one barrier; `wsh` (32 words) must not be
// in use by another call until a later barrier.
__device__ __forceinline__ uint32_t scan(uint32_t v, uint32_t* wsh, uint32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) wsh[warp] = x;
  __syncthreads();
  const uint32_t wv = lane < nw ? wsh[lane] : 0u;
  total = __reduce_add_sync(0xffffffffu, wv);
  return __reduce_add_sync(0xffffffffu, lane < warp ? wv : 0u) + x - v;
}

// Shared scratch of the row CTAs.
struct RowShared {
  uint32_t h[kBins];
  uint32_t wsh[4][32];
  uint32_t res[2];
};

// One digit: counts (in S.h, `nb` bins of ascending value) to the bin holding the kk-th
// largest and the number above it.  Every thread of a row CTA.
__device__ __forceinline__ uint2 find_digit(RowShared& S, int nb, uint32_t kk, int slot) {
  const int per = nb / kRowThreads;                           // 2 or 1
  const int hi = nb - static_cast<int>(threadIdx.x) * per;    // this thread's bins, from the top
  uint32_t c[2], sum = 0;
  for (int i = 0; i < per; ++i) sum += c[i] = S.h[hi - 1 - i];
  uint32_t total;
  uint32_t before = scan(sum, S.wsh[slot], total);
  for (int i = 0; i < per; ++i) {
    if (before < kk && before + c[i] >= kk) {
      S.res[0] = static_cast<uint32_t>(hi - 1 - i);
      S.res[1] = before;
    }
    before += c[i];
  }
  __syncthreads();
  const uint2 r = make_uint2(S.res[0], S.res[1]);
  __syncthreads();
  return r;
}

// The kk-th largest (1-based) of the values with (v >> hi_shift) == prefix that `each`
// hands out, by digits of `bits` bits down to `lo_shift`: the value's upper part (the
// rest zero), the number above, and in S.h the counts of the last digit.
template <typename Each>
__device__ __forceinline__ uint32_t select_digits(RowShared& S, Each each, uint32_t kk, const int (&shift)[3],
                                                  const int (&bits)[3], int digits, uint32_t& above) {
  uint32_t prefix = 0, mask = 0;
  above = 0;
#pragma unroll
  for (int d = 0; d < 3; ++d) {
    if (d >= digits) break;
    const int nb = 1 << bits[d];
    for (int i = threadIdx.x; i < nb; i += kRowThreads) S.h[i] = 0;
    __syncthreads();
    each([&](uint32_t v) {
      if ((v & mask) == prefix) atomicAdd(&S.h[(v >> shift[d]) & (nb - 1)], 1u);
    });
    __syncthreads();
    const uint2 f = find_digit(S, nb, kk - above, d);
    prefix |= f.x << shift[d];
    mask |= static_cast<uint32_t>(nb - 1) << shift[d];
    above += f.y;
  }
  return prefix;
}

__device__ __constant__ constexpr int kKeyShift[3] = {21, 10, 0}, kKeyBits[3] = {11, 11, 10};
__device__ __constant__ constexpr int kPosShift[3] = {20, 10, 0}, kPosBits[3] = {10, 10, 10};

// ----------------------------------------------------------------------- step 1

__global__ void __launch_bounds__(kRowThreads) tree_topk_bound_kernel(TreeTopkParams p) {
  __shared__ RowShared S;
  const int t = blockIdx.x;
  Row r;
  const bool work = load_row(p, t, r) && filtered(p, r);
  if (!work) return;
  if (threadIdx.x == 0) p.fill[t] = 0;
  const float* row = p.scores + static_cast<int64_t>(t) * p.ld;
  uint32_t u[kSamples / kRowThreads];
#pragma unroll
  for (int i = 0; i < kSamples / kRowThreads; ++i) {
    const uint32_t q = threadIdx.x + i * kRowThreads;
    const uint32_t a = static_cast<uint32_t>(static_cast<uint64_t>(r.n) * q / kSamples);
    const uint32_t b = static_cast<uint32_t>(static_cast<uint64_t>(r.n) * (q + 1) / kSamples);
    uint32_t hsh = q * 2654435761u;
    hsh ^= hsh >> 15;
    const int s = static_cast<int>(a + hsh % (b - a));   // b > a: n > samples
    u[i] = seen_key(p, r, s, __ldcg(row + s));
  }
  const float m = static_cast<float>(kSamples) * static_cast<float>(p.k) / static_cast<float>(r.n);
  const uint32_t rank = min(static_cast<uint32_t>(m + 6.f * sqrtf(m)) + 8u, static_cast<uint32_t>(kSamples));
  uint32_t above;
  const uint32_t bound = select_digits(
      S,
      [&](auto take) {
#pragma unroll
        for (int i = 0; i < kSamples / kRowThreads; ++i) take(u[i]);
      },
      rank, kKeyShift, kKeyBits, 2, above);
  if (threadIdx.x == 0) p.bound[t] = max(bound, 1u);   // positions not seen have key 0
}
static_assert(kTreeTopkCap >= kSamples, "a filtered row has a stretch of at least one score per sample");

// ----------------------------------------------------------------------- step 2

__global__ void __launch_bounds__(kFilterThreads) tree_topk_filter_kernel(TreeTopkParams p) {
  __shared__ uint32_t wsh[32];
  __shared__ uint32_t base_sh;
  const int t = blockIdx.y, c = blockIdx.x;
  Row r;
  const bool work = load_row(p, t, r) && filtered(p, r) && c * kTopkChunk < r.n;
  const float* row = p.scores + static_cast<int64_t>(t) * p.ld;
  const int s0 = c * kTopkChunk + static_cast<int>(threadIdx.x) * kPer;
  // The scores are inputs of the call, not of the kernel before: read ahead of the wait.
  uint32_t u[kPer];
  if (work) {
    if (s0 + kPer <= r.n) {
      const float4* p4 = reinterpret_cast<const float4*>(row + s0);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 v = __ldcs(p4 + q);
        u[4 * q] = score_key(v.x);
        u[4 * q + 1] = score_key(v.y);
        u[4 * q + 2] = score_key(v.z);
        u[4 * q + 3] = score_key(v.w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) u[i] = s0 + i < r.n ? score_key(__ldcs(row + s0 + i)) : 0u;
    }
    if (s0 + kPer > r.base) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (s0 + i < r.n && !(s0 + i < r.base || tree_sees(r.mask, p.tree.words, r.base, s0 + i))) u[i] = 0u;
    }
  }
  grid_dep_wait();
  grid_dep_launch();
  if (!work) return;
  const uint32_t bound = __ldcg(p.bound + t);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) m |= static_cast<uint32_t>(u[i] >= bound) << i;
  uint32_t total;
  const uint32_t o = scan(__popc(m), wsh, total);
  if (threadIdx.x == 0) {
    base_sh = total ? atomicAdd(p.fill + t, total) : 0u;
    p.at[static_cast<int64_t>(t) * p.nchunks + c] = base_sh;
    p.num[static_cast<int64_t>(t) * p.nchunks + c] = total;
  }
  __syncthreads();
  uint32_t at = base_sh + o;
  uint2* list = p.list + static_cast<int64_t>(t) * p.cap;
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if ((m >> i) & 1u) {
      if (at < static_cast<uint32_t>(p.cap)) list[at] = make_uint2(u[i], static_cast<uint32_t>(s0 + i));
      ++at;
    }
}

// ----------------------------------------------------------------------- step 3

// Hands `take(key, position)` the row's scores, eight per thread and step, in no order.
template <typename Take>
__device__ __forceinline__ void each_score(const TreeTopkParams& p, const Row& r, const float* row, Take take) {
  for (int s = 4 * static_cast<int>(threadIdx.x); s < r.n; s += 8 * kRowThreads) {
    float v[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int q = s + 4 * kRowThreads * h;
      if (q + 4 <= r.n) {
        const float4 x = __ldcg(reinterpret_cast<const float4*>(row + q));
        v[4 * h] = x.x;
        v[4 * h + 1] = x.y;
        v[4 * h + 2] = x.z;
        v[4 * h + 3] = x.w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * h + i] = q + i < r.n ? __ldcg(row + q + i) : 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int q = s + 4 * kRowThreads * (i >> 2) + (i & 3);
      if (q < r.n) {
        const uint32_t key = seen_key(p, r, q, v[i]);
        if (key) take(key, static_cast<uint32_t>(q));
      }
    }
  }
}

__global__ void __launch_bounds__(kRowThreads) tree_topk_select_kernel(TreeTopkParams p) {
  extern __shared__ __align__(16) uint2 ent[];   // [kTreeTopkCap]
  __shared__ RowShared S;
  const int t = blockIdx.x;
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  Row r;
  const bool real = load_row(p, t, r);
  grid_dep_wait();
  if (!real) return;
  int32_t* out = p.idx + static_cast<int64_t>(t) * p.k;
  int32_t* phys = p.phys ? p.phys + static_cast<int64_t>(t) * p.k : nullptr;
  const int32_t* btrow = p.b.bt + static_cast<int64_t>(r.req) * p.b.bt_stride;
  const int bsm = (1 << p.log2_bs) - 1;
  auto emit = [&](uint32_t o, int s) {
    out[o] = s;
    if (phys) phys[o] = s >= 0 ? (btrow[s >> p.log2_bs] << p.log2_bs) | (s & bsm) : -1;
  };
  if (r.seen <= p.k) {   // everything seen is selected, then -1
    for (int o = tid; o < p.k; o += kRowThreads) emit(o, seen_position(p, r, o));
    return;
  }
  const float* row = p.scores + static_cast<int64_t>(t) * p.ld;
  const uint32_t k = static_cast<uint32_t>(p.k);
  uint32_t n;        // entries in shared memory, in position order
  bool listed = true;
  if (!filtered(p, r)) {
    n = static_cast<uint32_t>(r.n);
    for (int s = tid; s < r.n; s += kRowThreads) ent[s] = make_uint2(seen_key(p, r, s, __ldcg(row + s)), static_cast<uint32_t>(s));
  } else {
    n = __ldcg(p.fill + t);
    listed = n >= k && n <= static_cast<uint32_t>(p.cap);
    if (listed) {
      // chunk by chunk: a warp per chunk, behind the entries of the chunks before it
      const int nch = static_cast<int>(cdiv(r.n, kTopkChunk));
      const uint2* list = p.list + static_cast<int64_t>(t) * p.cap;
      const uint32_t* at = p.at + static_cast<int64_t>(t) * p.nchunks;
      const uint32_t* num = p.num + static_cast<int64_t>(t) * p.nchunks;
      uint32_t before = 0;
      for (int c0 = 0; c0 < nch; c0 += kRowThreads) {
        const int c = c0 + tid;
        uint32_t cn = c < nch ? __ldcg(num + c) : 0u;
        uint32_t total;
        const uint32_t pre = before + scan(cn, S.wsh[0], total);
        // this round's places, read by the warps below
        S.h[tid] = pre;
        S.h[kRowThreads + tid] = cn;
        __syncthreads();
        for (int j = warp; j < kRowThreads && c0 + j < nch; j += kRowThreads / 32) {
          const uint32_t m = S.h[kRowThreads + j], to = S.h[j];
          if (m == 0) continue;
          const uint32_t from = __ldcg(at + c0 + j);
          for (uint32_t i = lane; i < m; i += 32) ent[to + i] = __ldcg(list + from + i);
        }
        before += total;
        __syncthreads();
      }
    }
  }
  __syncthreads();
  auto keys = [&](auto take) {
    if (listed)
      for (uint32_t i = tid; i < n; i += kRowThreads) take(ent[i].x);
    else
      each_score(p, r, row, [&](uint32_t key, uint32_t) { take(key); });
  };
  // the threshold key T, and how many of the keys equal to it are taken
  uint32_t above;
  const uint32_t T = select_digits(S, keys, k, kKeyShift, kKeyBits, 3, above);
  const uint32_t need = k - above, equal = S.h[T & 1023u];
  uint32_t cut = 0xFFFFFFFFu;   // keys equal to T are taken at positions <= cut
  if (equal > need) {
    auto places = [&](auto take) {
      auto of = [&](uint32_t key, uint32_t s) {
        if (key == T) take(0x3FFFFFFFu - s);   // lower positions are larger
      };
      if (listed)
        for (uint32_t i = tid; i < n; i += kRowThreads) of(ent[i].x, ent[i].y);
      else
        each_score(p, r, row, of);
    };
    __syncthreads();
    uint32_t a2;
    cut = 0x3FFFFFFFu - select_digits(S, places, need, kPosShift, kPosBits, 3, a2);
  }
  __syncthreads();
  auto taken = [&](uint32_t key, uint32_t s) { return key > T || (key == T && s <= cut); };
  if (listed) {
    // consecutive entries per thread: one scan orders the selection
    const uint32_t per = (n + kRowThreads - 1) / kRowThreads;
    const uint32_t i0 = min(n, per * static_cast<uint32_t>(tid)), i1 = min(n, i0 + per);
    uint32_t c = 0;
    for (uint32_t i = i0; i < i1; ++i) c += taken(ent[i].x, ent[i].y);
    uint32_t total;
    uint32_t o = scan(c, S.wsh[3], total);
    for (uint32_t i = i0; i < i1; ++i)
      if (taken(ent[i].x, ent[i].y)) emit(o++, static_cast<int>(ent[i].y));
  } else {
    uint32_t base = 0;
    for (int c0 = 0; c0 < r.n; c0 += 4 * kRowThreads) {
      const int s = c0 + 4 * tid;
      uint32_t m = 0;
      for (int i = 0; i < 4; ++i)
        if (s + i < r.n) {
          const uint32_t key = seen_key(p, r, s + i, __ldcg(row + s + i));
          if (key && taken(key, static_cast<uint32_t>(s + i))) m |= 1u << i;
        }
      uint32_t total;
      uint32_t o = base + scan(__popc(m), S.wsh[3], total);
      for (int i = 0; i < 4; ++i)
        if ((m >> i) & 1u) emit(o++, s + i);
      base += total;
      __syncthreads();
    }
  }
}

}  // namespace

cudaError_t launch_tree_topk(const TreeTopkParams& p, cudaStream_t st) {
  if (p.b.T == 0) return cudaSuccess;
  cudaError_t e = cudaSuccess;
  const bool filter = p.b.max_ctx > kTreeTopkCap;
  if (filter) {
    e = launch_ex(tree_topk_bound_kernel, dim3(p.b.T), dim3(kRowThreads), 0, st, false, 0u, p);
    if (e != cudaSuccess) return e;
    e = launch_ex(tree_topk_filter_kernel, dim3(p.nchunks, p.b.T), dim3(kFilterThreads), 0, st, true, 0u, p);
    if (e != cudaSuccess) return e;
  }
  const int64_t most = p.b.max_ctx < kTreeTopkCap ? p.b.max_ctx : kTreeTopkCap;
  e = set_func_attr_once(reinterpret_cast<const void*>(tree_topk_select_kernel),
                         cudaFuncAttributeMaxDynamicSharedMemorySize, kTreeTopkCap * static_cast<int>(sizeof(uint2)));
  if (e != cudaSuccess) return e;
  return launch_ex(tree_topk_select_kernel, dim3(p.b.T), dim3(kRowThreads), static_cast<size_t>(most) * sizeof(uint2), st,
                   filter, 0u, p);
}

}  // namespace dsa
