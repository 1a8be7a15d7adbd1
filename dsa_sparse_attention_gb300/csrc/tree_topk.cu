// tree_topk.cu — exact top-k of drafted tokens' indexer scores, over the positions each
// token sees in its tree (include/dsa.h, dsa_tree).
//
// A verification batch holds many long rows, so the pass over the scores is what
// counts: it is made once.
//  1. bound:  one CTA per row reads 4,096 scores, one at a hashed place of each of as
//             many equal stretches, and takes the sample's rank m + 6 sqrt(m) + 8 as the
//             row's bound, m = 4,096 k / n being the number of samples expected among
//             the k best.  Fewer than k scores then lie at or above the bound with
//             probability below 1e-6, and typically 1.6 k (64K scores) to 4 k (1M) do.
//  2. filter: one CTA per 4,096 scores lists its scores at or above the bound, in
//             position order, and notes where its entries lie.
//  3. select: one CTA per row puts the entries in position order into shared memory, finds
//             the k-th by one digit and comparisons within its bin (by digits down to the
//             last bit where the bin is crowded; equal keys by lower position), and writes
//             the selection with one scan.
// Rows of at most 14,336 scores go to step 3 directly.  Steps 1 and 2 only choose what
// step 3 looks at: it counts the entries, and a row whose entries are too few or too
// many (more equal scores than the list holds) is resolved over the whole row, exactly
// and slowly.  No sum depends on an order of arrival: results are deterministic and
// independent of the rest of the batch.
// Bound by latency: 48 rows of 64K take 15.4 us, 16 rows of 1M 35 us, when reading the scores
// alone would take 1.9 and 9.9 us; the launches overlap as far as their waits allow, and data that
// another SM has just written takes 0.8 us to read.
#include <cstddef>

#include "tree.cuh"

namespace dsa {

namespace {

constexpr int kBins = 2048;
constexpr int kFilterThreads = 256;
constexpr int kPer = 16;                 // scores per thread and chunk
static_assert(kFilterThreads * kPer == kTopkChunk, "chunk");
constexpr int kRowThreads = 1024;
constexpr int kSamples = 4096;
// Rows of at most this many scores skip steps 1 and 2: 48 rows of 6,000 / 8,100 / 12,000 / 16,300 take
// 8.0 / 9.8 / 12.1 / 14.3 us so, 12.6 / 12.6 / 13.1 / 13.1 us with them.
constexpr int kDirect = 14336;

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
  return r.seen > p.k && r.n > kDirect;
}

// The score of a key (score_key's inverse).
__device__ __forceinline__ float score_of_key(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key & 0x7FFFFFFFu : ~key);
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

// Shared scratch of the row CTAs.  The histogram's place also holds pairs (resolve_digit).
struct RowShared {
  alignas(16) uint32_t h[kBins];
  uint32_t wsh[4][32];
  uint32_t res[2];
};
static_assert(alignof(RowShared) % alignof(uint2) == 0 && offsetof(RowShared, h) % alignof(uint2) == 0,
              "pairs are read and written 8 bytes at a time");

// One digit: counts (in S.h, `nb` bins of ascending value) to the bin holding the kk-th
// largest and the number above it.  The bins count kk values at least, so one of them
// holds it.  Every thread of a row CTA.
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

// The kk-th largest (1-based) of the values that `each` hands out (the same ones every
// time), exact down to bit `low`, and the number above it; 0 when there are fewer than kk,
// which no bin would hold.  Digits of 11 bits are taken of the difference to the smallest
// value, from its highest set bit down: the scores that matter share their leading bits, and
// a histogram of those would send most lanes of a warp to the same few counters.  `equal`:
// values that share all digits taken.
template <typename Each>
__device__ __forceinline__ uint32_t select_value(RowShared& S, Each each, uint32_t kk, int low, uint32_t& above,
                                                 uint32_t& equal) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t lo = 0xFFFFFFFFu, hi = 0u, n = 0;
  each([&](uint32_t v) {
    lo = min(lo, v);
    hi = max(hi, v);
    ++n;
  });
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0) {
    S.wsh[0][warp] = lo;
    S.wsh[1][warp] = hi;
    S.wsh[2][warp] = n;
  }
  __syncthreads();
  lo = __reduce_min_sync(0xffffffffu, S.wsh[0][lane]);
  hi = __reduce_max_sync(0xffffffffu, S.wsh[1][lane]);
  equal = __reduce_add_sync(0xffffffffu, S.wsh[2][lane]);
  above = 0;
  if (equal < kk) return 0u;   // uniform
  uint32_t prefix = 0, mask = 0;
  int top = 32 - __clz(hi - lo);   // bits of the difference still open
  int slot = 3;
  while (top > low) {
    const int shift = max(top - 11, low);
    const int nb = 1 << 11;
    __syncthreads();
    for (int i = threadIdx.x; i < nb; i += kRowThreads) S.h[i] = 0;
    __syncthreads();
    each([&](uint32_t v) {
      const uint32_t d = v - lo;
      if ((d & mask) == prefix) atomicAdd(&S.h[(d >> shift) & (nb - 1)], 1u);
    });
    __syncthreads();
    const uint2 f = find_digit(S, nb, kk - above, slot);
    equal = S.h[f.x];
    prefix |= f.x << shift;
    mask = ~((1u << shift) - 1u);
    above += f.y;
    top = shift;
    slot = slot == 3 ? 0 : 3;
  }
  return lo + prefix;
}

// ----------------------------------------------------------------------- step 1

__global__ void __launch_bounds__(kRowThreads) tree_topk_bound_kernel(TreeTopkParams p) {
  __shared__ RowShared S;
  constexpr int kMine = kSamples / kRowThreads;
  const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dep_wait();
  grid_dep_launch();   // the filter's blocks load their scores meanwhile: this call's inputs are complete
  const float* row = p.scores + static_cast<int64_t>(t) * p.ld;
  float v[kMine];
  int at[kMine];
  auto sample = [&](int n) {   // (n > kDirect, at most the row's memory)
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const uint32_t q = threadIdx.x + i * kRowThreads;
      const uint32_t a = static_cast<uint32_t>(static_cast<uint64_t>(n) * q / kSamples);
      const uint32_t b = static_cast<uint32_t>(static_cast<uint64_t>(n) * (q + 1) / kSamples);
      uint32_t hsh = q * 2654435761u;
      hsh ^= hsh >> 15;
      at[i] = static_cast<int>(a + hsh % (b - a));   // b > a: n > samples
      v[i] = __ldcg(row + at[i]);
    }
  };
  // the samples are on their way while the rest of the token is read and checked
  const int64_t end = static_cast<int64_t>(__ldcg(p.b.q_pos + t)) + 1;
  const bool early = end > kDirect && end <= p.ld;
  if (early) sample(static_cast<int>(end));
  Row r;
  const bool work = load_row(p, t, r) && filtered(p, r);
  if (!work) return;
  if (threadIdx.x == 0) p.fill[t] = 0;
  if (!early || r.n != end) sample(r.n);   // a position that was out of range and has been clamped
  uint32_t u[kMine], most = 0;
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    u[i] = seen_key(p, r, at[i], v[i]);   // (few of them are seen where a token far behind its base has a narrow mask)
    most = max(most, u[i]);
  }
  const float m = static_cast<float>(kSamples) * static_cast<float>(p.k) / static_cast<float>(r.n);
  const uint32_t rank = min(static_cast<uint32_t>(m + 6.f * sqrtf(m)) + 8u, static_cast<uint32_t>(kSamples));
  // The samples' threshold lies above the smallest maximum of `rank` groups of samples, so with
  // few ranks it lies above that of all groups of 4 lanes: what is left spans few octaves, and
  // one digit of 11 bits divides it finely enough.
  constexpr uint32_t kGroups = kRowThreads / 4;
  uint32_t bound;
  if (rank <= kGroups) {
    uint32_t g = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
    g = max(g, __shfl_xor_sync(0xffffffffu, g, 2));
    const uint32_t lo_w = __reduce_min_sync(0xffffffffu, g), hi_w = __reduce_max_sync(0xffffffffu, g);
    if (lane == 0) {
      S.wsh[0][warp] = lo_w;
      S.wsh[1][warp] = hi_w;
    }
    for (int i = threadIdx.x; i < kBins; i += kRowThreads) S.h[i] = 0;
    __syncthreads();
    const uint32_t lo = __reduce_min_sync(0xffffffffu, S.wsh[0][lane]), hi = __reduce_max_sync(0xffffffffu, S.wsh[1][lane]);
    const int shift = max(32 - __clz(hi - lo) - 11, 0);
#pragma unroll
    for (int i = 0; i < kMine; ++i)
      if (u[i] >= lo) atomicAdd(&S.h[(u[i] - lo) >> shift], 1u);
    __syncthreads();
    bound = lo + (find_digit(S, kBins, rank, 2).x << shift);
  } else {   // to within 2^10: a lower bound of the sample's rank
    uint32_t above, equal;
    bound = select_value(
        S,
        [&](auto take) {
#pragma unroll
          for (int i = 0; i < kMine; ++i)
            if (u[i]) take(u[i]);
        },
        rank, 10, above, equal);
  }
  // Positions not seen have key 0.  With fewer samples seen than `rank` the bound is 1 and everything
  // seen is listed, which is then little: about `rank` of the row's 4,096 stretches.
  if (threadIdx.x == 0) p.bound[t] = max(bound, 1u);
}
static_assert(kTreeTopkCap <= 32 * kRowThreads, "rounds of the ordered output");
static_assert(kDirect >= kSamples && kTreeTopkCap >= kDirect, "a stretch of scores per sample; a direct row fits");

// ----------------------------------------------------------------------- step 2

__global__ void __launch_bounds__(kFilterThreads) tree_topk_filter_kernel(TreeTopkParams p) {
  __shared__ uint32_t wsh[2][32];
  __shared__ uint32_t base_sh;
  const int t = blockIdx.y, c = blockIdx.x;
  const float* row = p.scores + static_cast<int64_t>(t) * p.ld;
  // Thread i holds the scores 4 i .. 4 i + 3 of each of the chunk's four quarters: whole lines per load.
  const int s0 = c * kTopkChunk + 4 * static_cast<int>(threadIdx.x);
  constexpr int kQuarter = kTopkChunk / 4;
  // The scores are inputs of the call, complete before the kernel before passed its own wait and
  // let this one start: they are read ahead of the wait (from L2), and before the row's length
  // is known (within the row's memory).
  float4 v[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int s = s0 + kQuarter * q;
    v[q] = s + 4 <= p.ld ? __ldcg(reinterpret_cast<const float4*>(row + s)) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  Row r;
  const bool work = load_row(p, t, r) && filtered(p, r) && c * kTopkChunk < r.n;
  uint32_t u[kPer];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    u[4 * q] = score_key(v[q].x);
    u[4 * q + 1] = score_key(v[q].y);
    u[4 * q + 2] = score_key(v[q].z);
    u[4 * q + 3] = score_key(v[q].w);
  }
  if (work && (c + 1) * kTopkChunk > r.base) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int s = s0 + kQuarter * (i >> 2) + (i & 3);
      if (s >= r.n || !(s < r.base || tree_sees(r.mask, p.tree.words, r.base, s))) u[i] = 0u;
    }
  }
  grid_dep_wait();
  grid_dep_launch();
  if (!work) return;
  const uint32_t bound = __ldcg(p.bound + t);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) m |= static_cast<uint32_t>(u[i] >= bound) << i;
  // prefixes of the four quarters' counts, two to a word (at most 1,024 each)
  const uint32_t n01 = __popc(m & 0xFu) | (__popc(m & 0xF0u) << 16), n23 = __popc(m & 0xF00u) | (__popc(m & 0xF000u) << 16);
  uint32_t t01, t23;
  const uint32_t o01 = scan(n01, wsh[0], t01), o23 = scan(n23, wsh[1], t23);
  const uint32_t q1 = t01 & 0xFFFFu, q2 = q1 + (t01 >> 16), q3 = q2 + (t23 & 0xFFFFu), total = q3 + (t23 >> 16);
  if (threadIdx.x == 0) {
    base_sh = total ? atomicAdd(p.fill + t, total) : 0u;
    p.at[static_cast<int64_t>(t) * p.nchunks + c] = base_sh;
    p.num[static_cast<int64_t>(t) * p.nchunks + c] = total;
  }
  __syncthreads();
  const uint32_t first[4] = {o01 & 0xFFFFu, q1 + (o01 >> 16), q2 + (o23 & 0xFFFFu), q3 + (o23 >> 16)};
  uint2* list = p.list + static_cast<int64_t>(t) * p.cap;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t at = base_sh + first[q];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = 4 * q + e;
      if ((m >> i) & 1u) {
        if (at < static_cast<uint32_t>(p.cap)) list[at] = make_uint2(u[i], static_cast<uint32_t>(s0 + kQuarter * q + e));
        ++at;
      }
    }
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

// A digit of a key, one that does not fall as the key grows: by the key's bits, or by its score.
struct KeyDigit {   // of entries close above `lo`: 2^14 keys each, the last digit for all beyond
  uint32_t lo;
  __device__ uint32_t operator()(uint32_t key) const {
    return min((key - lo) >> 14, static_cast<uint32_t>(kBins - 1));
  }
};
struct ScoreDigit {   // of a whole row: equal steps between its smallest and largest score
  float lo, scale;
  __device__ uint32_t operator()(uint32_t key) const {
    const float x = (score_of_key(key) - lo) * scale;   // (rounded, but never falling)
    return min(static_cast<uint32_t>(max(x, 0.f)), static_cast<uint32_t>(kBins - 1));   // NaN: digit 0
  }
};

// The k-th best of n listed entries (equal keys: the lower position first) as (T, cut), from their
// counts by digit in S.h, when the k-th's bin holds few enough of them to compare each with each:
// the bin's entries are listed, and the one that needs k - above - 1 others before it is it.
// False (nothing decided) when the bin holds more.
constexpr int kPairs = kBins / 2;   // pairs that fit the histogram's place
template <typename Digit>
__device__ __forceinline__ bool resolve_digit(RowShared& S, const uint2* ent, uint32_t n, Digit digit, uint32_t k,
                                              uint32_t& T, uint32_t& cut) {
  const int tid = static_cast<int>(threadIdx.x);
  const uint2 f = find_digit(S, kBins, k, 2);
  const uint32_t count = S.h[f.x], need = k - f.y;
  __syncthreads();
  if (count > static_cast<uint32_t>(kPairs)) return false;   // uniform
  uint2* bin = reinterpret_cast<uint2*>(S.h);
  if (tid == 0) S.res[0] = 0;
  __syncthreads();
  for (uint32_t i = tid; i < n; i += kRowThreads) {
    const uint2 e = ent[i];
    if (e.x && digit(e.x) == f.x) bin[atomicAdd(&S.res[0], 1u)] = e;
  }
  __syncthreads();
  for (uint32_t i = tid; i < count; i += kRowThreads) {
    const uint2 e = bin[i];
    uint32_t better = 0;
    for (uint32_t j = 0; j < count; ++j) {
      const uint2 o = bin[j];
      better += o.x > e.x || (o.x == e.x && o.y < e.y);
    }
    if (better == need - 1) {   // exactly one entry
      S.wsh[3][0] = e.x;
      S.wsh[3][1] = e.y;
    }
  }
  __syncthreads();
  T = S.wsh[3][0];
  cut = S.wsh[3][1];
  return true;
}

// The same for a row whose digits have not been counted.  lo, hi: the thread's part in the
// smallest (at most) and the largest key; the entries have been written, no barrier since.
__device__ __forceinline__ bool select_listed(RowShared& S, const uint2* ent, uint32_t n, uint32_t lo, uint32_t hi,
                                              uint32_t k, uint32_t& T, uint32_t& cut) {
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) {
    S.wsh[0][warp] = lo;
    S.wsh[1][warp] = hi;
  }
  for (int i = tid; i < kBins; i += kRowThreads) S.h[i] = 0;
  __syncthreads();
  const float flo = score_of_key(__reduce_min_sync(0xffffffffu, S.wsh[0][lane]));
  const float fhi = score_of_key(__reduce_max_sync(0xffffffffu, S.wsh[1][lane]));
  const ScoreDigit digit = {flo, static_cast<float>(kBins) / (fhi - flo)};
  for (uint32_t i = tid; i < n; i += kRowThreads) {
    const uint32_t key = ent[i].x;
    if (key) atomicAdd(&S.h[digit(key)], 1u);
  }
  __syncthreads();
  return resolve_digit(S, ent, n, digit, k, T, cut);
}

__global__ void __launch_bounds__(kRowThreads) tree_topk_select_kernel(TreeTopkParams p) {
  extern __shared__ __align__(16) uint2 ent[];   // [kTreeTopkCap]
  __shared__ RowShared S;
  __shared__ uint32_t moved[kRowThreads];        // where a chunk's entries go, less where they are
  const int t = blockIdx.x;
  const int tid = static_cast<int>(threadIdx.x);
  Row r;
  const bool first = p.b.max_ctx <= kDirect;   // the call's only kernel
  if (first) grid_dep_wait();
  const bool real = load_row(p, t, r);
  if (!first) grid_dep_wait();
  grid_dep_launch();
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
  uint32_t lo = 0xFFFFFFFFu, hi = 0u;   // this thread's part in their extremes
  bool listed = true;
  if (!filtered(p, r)) {
    n = static_cast<uint32_t>(r.n);
    for (int s = tid; s < r.n; s += kRowThreads) {
      const uint32_t key = seen_key(p, r, s, __ldcg(row + s));
      ent[s] = make_uint2(key, static_cast<uint32_t>(s));
      if (key) lo = min(lo, key);
      hi = max(hi, key);
    }
  } else {
    // The list holds the chunks' entries as the filter's CTAs arrived, each chunk's in order: entry i
    // of chunk c belongs at (entries of the chunks before) + i - at[c].  Counts, places and the
    // first entries are read at once, before it is known how many entries there are (up to the
    // list's capacity they are the workspace's): one round trip to memory, not three.
    // Their first digit is counted on the way: the k-th lies close above the bound, mostly within the
    // 2^25 keys (four octaves) that the digits divide; the last bin counts what lies beyond.
    constexpr int kAhead = 8;
    const int nch = static_cast<int>(cdiv(r.n, kTopkChunk));
    const uint2* list = p.list + static_cast<int64_t>(t) * p.cap;
    const uint32_t* at = p.at + static_cast<int64_t>(t) * p.nchunks;
    const uint32_t* num = p.num + static_cast<int64_t>(t) * p.nchunks;
    uint2 e[kAhead];
    for (int i = tid; i < kBins; i += kRowThreads) S.h[i] = 0;
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      const int i = tid + q * kRowThreads;
      e[q] = i < p.cap ? __ldcg(list + i) : make_uint2(0u, 0u);
    }
    uint32_t cn = tid < nch ? __ldcg(num + tid) : 0u, ca = tid < nch ? __ldcg(at + tid) : 0u;
    n = __ldcg(p.fill + t);
    lo = __ldcg(p.bound + t);
    listed = n >= k && n <= static_cast<uint32_t>(p.cap);
    if (listed) {
      uint32_t before = 0;
      for (int c0 = 0; c0 < nch; c0 += kRowThreads) {   // rounds of 1,024 chunks, 4M scores
        if (c0 > 0) {
          cn = c0 + tid < nch ? __ldcg(num + c0 + tid) : 0u;
          ca = c0 + tid < nch ? __ldcg(at + c0 + tid) : 0u;
        }
        uint32_t total;
        moved[tid] = before + scan(cn, S.wsh[0], total) - ca;   // (wraps; the sum with i does not)
        before += total;
        __syncthreads();
        auto place = [&](uint32_t i, uint2 x) {
          const uint32_t c = x.y / kTopkChunk - static_cast<uint32_t>(c0);
          if (i >= n || c >= static_cast<uint32_t>(kRowThreads)) return;
          ent[moved[c] + i] = x;
          hi = max(hi, x.x);
          atomicAdd(&S.h[KeyDigit{lo}(x.x)], 1u);
        };
#pragma unroll
        for (int q = 0; q < kAhead; ++q) place(tid + q * kRowThreads, e[q]);
        for (uint32_t i = tid + kAhead * kRowThreads; i < n; i += kRowThreads) place(i, __ldcg(list + i));
        __syncthreads();
      }
    }
  }
  auto keys = [&](auto take) {
    if (listed)
      for (uint32_t i = tid; i < n; i += kRowThreads) {
        const uint32_t key = ent[i].x;
        if (key) take(key);
      }
    else
      each_score(p, r, row, [&](uint32_t key, uint32_t) { take(key); });
  };
  // the threshold key T, and of the keys equal to it those at positions <= cut
  uint32_t T, cut = 0xFFFFFFFFu;
  const bool counted = filtered(p, r);   // the entries' digits are in S.h
  if (!listed || !((counted && resolve_digit(S, ent, n, KeyDigit{lo}, k, T, cut)) || select_listed(S, ent, n, lo, hi, k, T, cut))) {
    uint32_t above, equal;
    T = select_value(S, keys, k, 0, above, equal);
    const uint32_t need = k - above;
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
      uint32_t a2, e2;
      cut = 0x3FFFFFFFu - select_value(S, places, need, 0, a2, e2);
    }
  }
  __syncthreads();
  auto taken = [&](uint32_t key, uint32_t s) { return key > T || (key == T && s <= cut); };
  if (listed) {
    // Entry j * 1024 + thread: counts per (j, warp) in order, one scan over them.
    constexpr int kWarps = kRowThreads / 32;
    const uint32_t rounds = (n + kRowThreads - 1) / kRowThreads;   // <= 24
    uint32_t mine = 0;                                             // bit j: this thread's entry of round j
    for (uint32_t j = 0; j < rounds; ++j) {
      const uint32_t i = j * kRowThreads + tid;
      const bool take = i < n && taken(ent[i].x, ent[i].y);
      const uint32_t b = __ballot_sync(0xffffffffu, take);
      if (take) mine |= 1u << j;
      if ((tid & 31) == 0) S.h[j * kWarps + (tid >> 5)] = __popc(b);
    }
    __syncthreads();
    uint32_t total;
    const uint32_t pre = scan(static_cast<uint32_t>(tid) < rounds * kWarps ? S.h[tid] : 0u, S.wsh[2], total);
    S.h[kRowThreads + tid] = pre;
    __syncthreads();
    for (uint32_t j = 0; j < rounds; ++j) {
      const uint32_t b = __ballot_sync(0xffffffffu, (mine >> j) & 1u);
      if (!((mine >> j) & 1u)) continue;
      emit(S.h[kRowThreads + j * kWarps + (tid >> 5)] + __popc(b & ((1u << (tid & 31)) - 1u)),
           static_cast<int>(ent[j * kRowThreads + tid].y));
    }
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
  const bool filter = p.b.max_ctx > kDirect;
  if (filter) {
    e = launch_ex(tree_topk_bound_kernel, dim3(p.b.T), dim3(kRowThreads), 0, st, true, 0u, p);
    if (e != cudaSuccess) return e;
    e = launch_ex(tree_topk_filter_kernel, dim3(p.nchunks, p.b.T), dim3(kFilterThreads), 0, st, true, 0u, p);
    if (e != cudaSuccess) return e;
  }
  const int64_t most = p.b.max_ctx < kTreeTopkCap ? p.b.max_ctx : kTreeTopkCap;
  e = set_func_attr_once(reinterpret_cast<const void*>(tree_topk_select_kernel),
                         cudaFuncAttributeMaxDynamicSharedMemorySize, kTreeTopkCap * static_cast<int>(sizeof(uint2)));
  if (e != cudaSuccess) return e;
  return launch_ex(tree_topk_select_kernel, dim3(p.b.T), dim3(kRowThreads), static_cast<size_t>(most) * sizeof(uint2), st,
                   true, 0u, p);
}

}  // namespace dsa
