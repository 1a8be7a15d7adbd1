// tree_mla.cu — dense MLA attention of drafted tokens over the paged latents.
//
// Token t attends to every committed position of its request and to its ancestors
// among the drafted slots (include/dsa.h, dsa_tree), 96 absorbed query heads over
// 576-dim latents, value = first 512 dims, as the sparse attention (mla.cu) does over
// a selection.  The work, 2 x 96 x 1,088 operations per (token, position), exceeds
// what the bytes cost at every length, so the kernels are built for the tensor cores.
//
// Plan: one small kernel turns the batch into a list of 128-position tiles; the
// attention's CTAs (one per SM) take equal contiguous shares of it, whatever the
// lengths, and the combine merges the partials of tokens that several CTAs share.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mla_conv.cuh"
#include "mla_q.cuh"
#include "ptx_tree.cuh"
#include "tree_mla.cuh"

namespace dsa {

// --------------------------------------------------------- plan and query terms
//
// Block 0 sums the tokens' tiles; the other blocks turn the queries into the attention's
// operands, one warp per head, three blocks of 32 heads a token: two e4m3 terms (FP8
// latents, mla_q.cuh) or fp16 values (NVFP4 latents), scaled per head by a power of two.
// Latency bound: 2.2 us for one token, 7 us by itself for 48, 12 us for 212.

// Head h of query q_tok (bf16 [96][576]) as fp16 times 2^k, the largest |q| in [2^14, 2^15):
// exact above 2^-32 of it, off by at most 2^-25 below.  k goes to exps[h].
__device__ __forceinline__ void q_head_to_f16(const __nv_bfloat16* q_tok, int h, __half* out, int32_t* exps) {
  const int lane = threadIdx.x & 31;
  const uint4* src = reinterpret_cast<const uint4*>(q_tok + static_cast<int64_t>(h) * kLatDim);
  uint4 v[3];
  uint32_t am = 0;   // |q| bits: non-negative floats order as unsigned integers
#pragma unroll
  for (int r = 0; r < 3; ++r) {
    const int pc = lane + 32 * r;
    v[r] = pc < 72 ? __ldg(src + pc) : make_uint4(0u, 0u, 0u, 0u);
    const uint32_t w4[4] = {v[r].x, v[r].y, v[r].z, v[r].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) am = max(am, max((w4[j] << 16) & 0x7FFFFFFFu, w4[j] & 0x7FFF0000u));
  }
  am = __reduce_max_sync(0xffffffffu, am);
  int k = am < 0x00800000u ? 0 : 14 + 127 - static_cast<int>(am >> 23);
  k = k > 126 ? 126 : (k < -126 ? -126 : k);
  const float sc = __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
  if (lane == 0) exps[h] = k;
  uint4* dst = reinterpret_cast<uint4*>(out + static_cast<int64_t>(h) * kLatDim);
#pragma unroll
  for (int r = 0; r < 3; ++r) {
    const int pc = lane + 32 * r;
    if (pc >= 72) break;
    const uint32_t w4[4] = {v[r].x, v[r].y, v[r].z, v[r].w};
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __half2 x =
          __floats2half2_rn(__uint_as_float(w4[j] << 16) * sc, __uint_as_float(w4[j] & 0xFFFF0000u) * sc);
      o[j] = *reinterpret_cast<const uint32_t*>(&x);
    }
    dst[pc] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

constexpr int kPrepThreads = 1024;

__global__ void __launch_bounds__(kPrepThreads) tree_prep_kernel(TreePrepParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dep_wait();
  grid_dep_launch();
  if (blockIdx.x > 0) {
    const int t = (blockIdx.x - 1) / 3, h = (blockIdx.x - 1) % 3 * 32 + warp;
    const __nv_bfloat16* q_tok = p.q + static_cast<int64_t>(t) * kMlaHeads * kLatDim;
    if (p.q16) {
      q_head_to_f16(q_tok, h, p.q16 + static_cast<int64_t>(t) * kMlaHeads * kLatDim,
                    p.exps + static_cast<int64_t>(t) * kMlaHeads);
    } else {
      uint8_t* tok = p.terms + static_cast<int64_t>(t) * kQTokenBytes;
      q_head_to_terms(q_tok, h, tok, reinterpret_cast<int32_t*>(tok + kQTermBytes));
    }
    return;
  }
  __shared__ int64_t wsum[kPrepThreads / 32];
  // starts and records of a batch of up to 1,024 tokens
  __shared__ int64_t st_sh[kPrepThreads];
  __shared__ TreeToken tok_sh[kPrepThreads];
  const int T = p.b.T;
  int64_t base = 0;
  for (int t0 = 0; t0 < T; t0 += kPrepThreads) {
    const int t = t0 + threadIdx.x;
    int64_t v = 0;
    if (t < T) {
      TreeToken k = {0, 0, 0, 0};
      if (load_tree_token(p.b, p.tree, t, p.status, k.req, k.pos, k.base)) v = cdiv(k.pos + 1, kSelTile);
      p.toks[t] = k;
      tok_sh[threadIdx.x] = k;
    }
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    int64_t before = 0, total = 0;
    const int warps = min(kPrepThreads / 32, (T - t0 + 31) / 32);   // that have tokens
    for (int w = 0; w < warps; ++w) {
      if (w < warp) before += wsum[w];
      total += wsum[w];
    }
    if (t < T) p.starts[t] = base + before + x - v;
    st_sh[threadIdx.x] = base + before + x - v;
    base += total;
    __syncthreads();
  }
  if (threadIdx.x == 0) p.starts[T] = base;
  __syncthreads();
  // each CTA's share and its first token: the last one that starts at or before the share,
  // so never one without tiles
  const int G = static_cast<int>(base < p.max_ctas ? base : p.max_ctas);
  for (int c = threadIdx.x; c < p.max_ctas; c += kPrepThreads) {
    TreeShare s = {};
    if (c < G) {
      s.g0 = share_begin(base, G, c);
      s.g1 = share_begin(base, G, c + 1);
      s.period = static_cast<int32_t>(base / G);
      int lo = 0, hi = T;   // starts[lo] <= g0 < starts[hi]
      while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if ((T <= kPrepThreads ? st_sh[m] : __ldcg(p.starts + m)) <= s.g0) lo = m;
        else hi = m;
      }
      s.t = lo;
      s.u0 = T <= kPrepThreads ? st_sh[lo] : __ldcg(p.starts + lo);
      s.u1 = lo + 1 == T ? base : (T <= kPrepThreads ? st_sh[lo + 1] : __ldcg(p.starts + lo + 1));
      if (T <= kPrepThreads) {
        s.tok = tok_sh[lo];
      } else {
        const int4 k = __ldcg(reinterpret_cast<const int4*>(p.toks) + lo);
        s.tok = TreeToken{k.x, k.y, k.z, k.w};
      }
    }
    p.shares[c] = s;
  }
}

cudaError_t launch_tree_prep(const TreePrepParams& p, cudaStream_t st) {
  return launch_ex(tree_prep_kernel, dim3(1 + 3 * p.b.T), dim3(kPrepThreads), 0, st, true, 0u, p);
}

__device__ __forceinline__ SegmentWalk make_walk(const TreeMlaParams& p) {
  SegmentWalk w;
  w.starts = p.starts;
  w.toks = p.toks;
  w.T = p.b.T;
  w.whole = p.whole;
  w.cta = blockIdx.x;
  w.G = p.max_ctas;
  w.g0 = w.g = w.g1 = w.u0 = w.u1 = 0;
  w.t = blockIdx.x;
  w.period = 1;
  if (!p.whole) {
    const int4* r = reinterpret_cast<const int4*>(p.shares + blockIdx.x);
    const int4 a = __ldcg(r), b = __ldcg(r + 1), c = __ldcg(r + 2), d = __ldcg(r + 3);
    auto i64 = [](int lo, int hi) {
      return static_cast<int64_t>(static_cast<uint32_t>(lo)) | (static_cast<int64_t>(hi) << 32);
    };
    w.g0 = w.g = i64(a.x, a.y);
    w.g1 = i64(a.z, a.w);
    w.u0 = i64(b.x, b.y);
    w.u1 = i64(b.z, b.w);
    w.t = c.x;
    w.period = c.y;
    w.tok = TreeToken{d.x, d.y, d.z, d.w};
  }
  return w;
}
static_assert(sizeof(TreeShare) == 64 && sizeof(TreeToken) == 16, "read 16 bytes at a time");

__device__ __forceinline__ uint8_t* align1024_tree(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~static_cast<uintptr_t>(1023));
}

// A failed (timed out) wait is the same for the whole warp.  A warp whose wait failed
// walks on through its tiles without touching operands or signalling barriers (a phase
// must not be completed twice), so the named barriers stay whole.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, Abort ab, bool ok) {
  return __all_sync(0xffffffffu, ok && mbar_wait_inline(bar, parity, ab));
}

// Head, in its group of 32, of column n of the group in P and O.
__device__ __forceinline__ constexpr int head_of_column(int n) { return 8 * ((n >> 1) & 3) + 2 * (n >> 3) + (n & 1); }

// A warp's part of a finished segment: its 32 heads (columns n0 ..) of the 32 dims of its lane
// quarter, for the four dim blocks, as the output (bf16) or as the normalised partial (fp16:
// 11 significant bits, above the output's 8), both [96][512].  A thread gets two columns of
// a dim side by side; a transposing matrix store turns 8 x 8 of them into 8 dims (16 bytes)
// of a head in the group's `stage` (8 KB of P's place, free by now: a dim block of the 32
// heads of four warps), and every warp writes 8 heads, 256 contiguous bytes each.
// `inv`: 1 / sum per column; `bar`: the group's named barrier.
__device__ __forceinline__ void store_segment(const TreeMlaParams& p, const Segment& s, bool ok, uint32_t o_tmem,
                                              const float* inv, int n0, int quarter, uint8_t* stage, int bar) {
  const int lane = threadIdx.x & 31;
  const bool fin = s.slot < 0;
  const int64_t row0 = (fin ? static_cast<int64_t>(s.t) : static_cast<int64_t>(s.slot)) * kMlaHeads + n0;
  uint16_t* out = (fin ? reinterpret_cast<uint16_t*>(p.out) : reinterpret_cast<uint16_t*>(p.part_o)) + row0 * kVDim;
  float2 iv[4];
#pragma unroll
  for (int b = 0; b < 4; ++b) iv[b] = *reinterpret_cast<const float2*>(inv + n0 + 8 * b + 2 * (lane & 3));
  // The stage holds column c's 128 dims in 256 bytes, 16-byte piece k at k ^ c % 8.
  auto piece = [&](int c, int k) { return c * 256 + ((k ^ (c & 7)) << 4); };
#pragma unroll 1
  for (int v = 0; v < 4; ++v) {
    uint32_t rr[2][16] = {};
    if (ok) {
      DSA_TMEM_LD_16X256_X4(o_tmem + 96 * v + n0, rr[0]);
      DSA_TMEM_LD_16X256_X4(o_tmem + 96 * v + n0 + (16u << 16), rr[1]);
      tmem_wait_ld();
    }
    if (v > 0) named_bar_sync(bar, 128);   // the block before has left the stage
#pragma unroll
    for (int hh = 0; hh < 2 && ok; ++hh) {
      uint32_t w[4][2];   // columns 8 b + 2 a, + 1; dims 16 hh + lane / 4, + 8
#pragma unroll
      for (int b = 0; b < 4; ++b)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float x = __uint_as_float(rr[hh][4 * b + 2 * u]) * iv[b].x, y = __uint_as_float(rr[hh][4 * b + 2 * u + 1]) * iv[b].y;
          if (fin) {
            const __nv_bfloat162 t = __floats2bfloat162_rn(x, y);
            w[b][u] = *reinterpret_cast<const uint32_t*>(&t);
          } else {
            const __half2 t = __floats2half2_rn(x, y);
            w[b][u] = *reinterpret_cast<const uint32_t*>(&t);
          }
        }
#pragma unroll
      for (int b = 0; b < 4; b += 2) {
        const int c = 8 * (b + (lane >> 4)) + (lane & 7);
        stmatrix_x4_trans(smem_u32(stage) + piece(c, 4 * quarter + 2 * hh + ((lane >> 3) & 1)), w[b][0], w[b][1],
                          w[b + 1][0], w[b + 1][1]);
      }
    }
    named_bar_sync(bar, 128);
    if (ok) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = 8 * quarter + 2 * k + (lane >> 4);
        const uint4 x = *reinterpret_cast<const uint4*>(stage + piece(c, lane & 15));
        *reinterpret_cast<uint4*>(out + head_of_column(c) * kVDim + 128 * v + 8 * (lane & 15)) = x;
      }
    }
  }
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)),
        "l"(reinterpret_cast<const uint64_t&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<const uint64_t&>(a)), "l"(reinterpret_cast<const uint64_t&>(b)));
  return d;
}

// A tile's logits less their references, capped half a step above what the references allow.  From
// logits of 2^24 (log2 units) on, fp32 rounds the logits and SHIFT - reference by whole units, so that
// a weight could pass fp16's range (and be infinite, the result NaN); the cap leaves up to 2^28, where
// units are 16 apart, a largest weight between 2^-5 and 2^15.5.  Below 2^20 it is never reached.  Tiles
// that move no reference have had their maximum compared instead.  NaN stays NaN.
constexpr float kTreeCap = 15.5f;   // SHIFT + TAU + 1/2
__device__ __forceinline__ void cap_weights(float2 (&y)[4][4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      asm("min.NaN.f32 %0, %0, %1;" : "+f"(y[i][b].x) : "f"(kTreeCap));
      asm("min.NaN.f32 %0, %0, %1;" : "+f"(y[i][b].y) : "f"(kTreeCap));
    }
}

// A warp's part of O (32 heads from column n0 on of its lanes' dims, in the four dim blocks) added to
// the CTA's running sums, or, at a segment's end, the sums to it.  The sums have the references that
// `run_sh` (SHIFT - reference, per column) kept of their last addition, O those of `sh`; a sum belongs
// to one thread, which alone reads and writes it.  Between runs rather than in the tiles' loop, which
// has no register to spare (8 x 6 tokens over 64K, which take no part in it: 582 us, 588 as a call).
template <bool END>
__device__ __forceinline__ void add_running_sums(float* runs, bool first, uint32_t o_tmem, const float* sh,
                                                 const float* run_sh, int n0, int quarter) {
  float* mine = runs + blockIdx.x * kRunFloats + n0 * 128 + 32 * quarter + (threadIdx.x & 31);
#pragma unroll 1
  for (int v = 0; v < 4; ++v) {
#pragma unroll 1
    for (int c = 0; c < 32; c += 8) {
      uint32_t o[8];
      float* r = mine + (v * kMlaHeads + c) * 128;
      DSA_TMEM_LD8(o_tmem + 96 * v + n0 + c, o);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float now = sh[n0 + c + i], then = run_sh[n0 + c + i];
        // (equal: both infinite where a head has seen nothing)
        const float x = first ? 0.f : r[i * 128] * (now == then ? 1.f : exp2f(now - then));
        o[i] = __float_as_uint(__uint_as_float(o[i]) + x);
        if (!END) r[i * 128] = __uint_as_float(o[i]);
      }
      if (END) DSA_TMEM_ST8(o_tmem + 96 * v + n0 + c, o);
    }
  }
  if (END) tmem_wait_st();
}

// ------------------------------------------------- attention with FP8 latents
//
// No conversion: e4m3 is the tensor core's operand type, and one copy of the tile in
// shared memory, brought by TMA, is the A operand of both products (K-major for the
// scores, MN-major for the values).
//   S^T[token, head] = sum_k c[token, k] . q_term[head, k]      M=128, N=96, K=1152
//   O^T[dim, head] += V^T[dim, token] . P_term^T[token, head]   M=128 (x4 dim blocks), N=96, K=3 x 128
// q arrives as two e4m3 terms, exact for values above about 2^-10 of a head's largest, off by at
// most 2^-17 of the largest below (mla_q.cuh).  P, rounded to fp16 (2^-11 of it, a bf16 P 2^-8), is
// the sum of three e5m2 terms, each the nearest to what the ones before it left.  e5m2 is the upper
// byte of an fp16, so a term is an addition, a mask and a subtraction on two weights at a time.
// With the reference at 2^11 the three terms are the fp16 weight exactly down to 2^-17 of the
// reference; below, a bit goes per octave (2^-10 of the weight at 2^-18, 2^-3 at 2^-25), and weights
// below 2^-28 are left out of O while the sum has them: a million positions just under that beside
// one heavy one lose 2^-8 of the result, one rounding to bf16 (e4m3 terms would lose them from 2^-18
// on).  The sum of the weights is of the unrounded ones, in fp32.
// Tokens on TMEM lanes use all four lane quarters and waste no rows (96 heads are N);
// the price, maxima across lanes, is not paid per tile: weights are taken against a
// reference per head, and only when some logit exceeds it by 2^4 do the warps reduce the
// tile's maxima, move the reference and rescale O.
// Every run of MMAs on one A operand (both query terms; all three terms of P) keeps A in
// the tensor core's buffer: 49 cycles an MMA instead of 57 (measured; 128 bytes of shared
// memory a cycle bound it otherwise).
// TMEM: S^T in columns [0, 96), O^T blocks at 128 + 96 v: 480 of 512.
// Shared memory holds the query terms (108 KB), one tile (72 KB: four 16 KB slices of
// 128 dims and an 8 KB slice of the last 64) and P (36 KB).  A slice is refilled as soon
// as the PV block that reads it is done, with the next tile prefetched into L2 meanwhile.
// 8 x 6 tokens over 64K: 577 us a call, 1.14 PFLOP/s, at the power limit (SM clock about 1,950 of
// 2,070 MHz).  The 84 MMAs of a tile take 4.1K of its 6.7K cycles; the rest is the softmax and the
// slices' refill, which the next tile's scores could fill (S is free once it is in registers) if
// shared memory had a place for its latents beside the query's 108 KB.
// Roles: warps 0..11 run the softmax and the epilogue (lane quarter w % 4, heads
// 32 (w / 4) ..); warp 12 issues MMAs; warp 13 loads.
namespace t8 {
constexpr int THREADS = 448;
constexpr int QCHUNK = 96 * 128;
constexpr int SLICE = 128 * 128;
constexpr int OFF_Q = 0;
constexpr int OFF_LAT = kQTermBytes;              // four slices
constexpr int OFF_TAIL = OFF_LAT + 4 * SLICE;     // dims 512..575: [128 tokens x 64 B], 64-byte swizzle
constexpr int OFF_P = OFF_TAIL + 128 * 64;        // per term: three [128 tokens x 32 heads] blocks, 32-byte swizzle
constexpr int P_TERM = 96 * 128;
constexpr int P_BLOCK = 128 * 32;
constexpr int OFF_QEXP = OFF_P + 3 * P_TERM;      // [96] int
constexpr int OFF_REDM = OFF_QEXP + 96 * 4;       // [4][96] float: maxima, then sums, per lane quarter
constexpr int OFF_SH = OFF_REDM + 4 * 96 * 4;     // [96] float: SHIFT - reference
constexpr int OFF_ALPHA = OFF_SH + 96 * 4;        // [96] float
constexpr int OFF_INV = OFF_ALPHA + 96 * 4;       // [96] float
constexpr int OFF_RUN = OFF_INV + 96 * 4;         // [96] float: SHIFT - reference of the running sums
constexpr int OFF_BARS = OFF_RUN + 96 * 4;
constexpr int N_BARS = 20;
constexpr int OFF_MISC = OFF_BARS + N_BARS * 8;
constexpr int SMEM_BYTES = OFF_MISC + 64 + 1024;
constexpr int MATH_WARPS = 12;
constexpr int MATH = MATH_WARPS * 32;
constexpr int MMA_WARP = 12, LOAD_WARP = 13;
constexpr int S_COL = 0;
constexpr int O_COL = 128;
constexpr float TAU = 4.0f;                       // log2 headroom before the reference moves
constexpr float SHIFT = 11.0f;                    // weights are scaled by 2^11: at most 2^15, below e5m2's 57344
static_assert(OFF_LAT % 1024 == 0 && OFF_TAIL % 1024 == 0 && OFF_P % 1024 == 0, "align");
static_assert(OFF_SH % 16 == 0 && OFF_ALPHA % 16 == 0 && OFF_INV % 16 == 0 && OFF_QEXP % 16 == 0,
              "vectors are read 16 bytes at a time");
static_assert(OFF_BARS % 8 == 0 && SMEM_BYTES <= 232448, "smem");
static_assert(SHIFT + TAU + 0.5f == kTreeCap, "weights' cap");
}  // namespace t8

// One term of two fp16 values, both to nearest: the upper byte of each half of the result
// is the e5m2 value (fp16 and e5m2 share sign and exponent, so adding half a step of the
// upper byte rounds the magnitude; ties go up).  `rest` is what the term leaves, exactly.
__device__ __forceinline__ uint32_t e5m2_term(uint32_t v, uint32_t& rest) {
  const uint32_t t = v + 0x00800080u;
  const uint32_t hi = t & 0xFF00FF00u;
  const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&hi));
  rest = *reinterpret_cast<const uint32_t*>(&d);
  return t;
}

__global__ void __launch_bounds__(t8::THREADS, 1)
    tree_mla_fp8_kernel(const __grid_constant__ CUtensorMap lmap, const __grid_constant__ CUtensorMap tmap,
                        TreeMlaParams p) {
  using namespace t8;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024_tree(smem_raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BARS);
  uint64_t* lat_full = bars + 0;    // [4] slices, then the tail
  uint64_t* tail_full = bars + 4;
  uint64_t* lat_empty = bars + 5;   // [4]
  uint64_t* tail_empty = bars + 9;
  uint64_t* q_full = bars + 10;
  uint64_t* q_done = bars + 11;     // a segment's QKs are done
  uint64_t* s_full = bars + 12;     // a tile's QK (and the PV before it) is done
  uint64_t* o_done = bars + 13;     // a segment's last PV is done
  uint64_t* drain = bars + 14;
  uint64_t* p_full = bars + 15;     // [3] P of the tokens 8 i + (0..7) of every quarter: i = 0, 1, 2 and 3
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + OFF_MISC);
  int* abortf = reinterpret_cast<int*>(smem + OFF_MISC + 8);
  float* red = reinterpret_cast<float*>(smem + OFF_REDM);
  float* sh_sh = reinterpret_cast<float*>(smem + OFF_SH);
  float* alpha_sh = reinterpret_cast<float*>(smem + OFF_ALPHA);
  float* inv_sh = reinterpret_cast<float*>(smem + OFF_INV);
  float* run_sh = reinterpret_cast<float*>(smem + OFF_RUN);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 15; ++i) mbar_init(&bars[i], 1);
    for (int i = 0; i < 3; ++i) mbar_init(&p_full[i], MATH_WARPS);
    *abortf = 0;
    fence_mbar_init();
    prefetch_tensormap(&lmap);
    prefetch_tensormap(&tmap);
  }
  if (warp == 0) tmem_alloc(tslot, 512);
  grid_dep_wait();   // the plan and the query terms
  grid_dep_launch();
  SegmentWalk walk = make_walk(p);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  const Abort ab{abortf, p.status};
  Segment s;

  if (warp == LOAD_WARP) {
    // ---------------------------------------------------------------- loads
    const int lg = p.pool.log2_bs;
    const int box = min(p.pool.bs, kSelTile);     // positions of one copy
    const int nbox = kSelTile / box;              // copies (lanes) per slice
    bool ok = true;
    int it = 0, q_issued = -1;   // q_issued: parity of the last query copy
    for (int seg = 0; ok && walk.next(s); ++seg) {
      const int pos = s.tok.pos;
      const int32_t* btrow = p.b.bt + static_cast<int64_t>(s.tok.req) * p.b.bt_stride;
      // this lane's page of tile j: pool row (num_rows, which reads as zeros, for a bad id)
      auto page = [&](int j) {
        const int s0 = j * kSelTile + lane * box;
        if (lane >= nbox || s0 > pos) return -1;
        const int32_t id = __ldg(btrow + (s0 >> lg));
        if (id >= 0 && id < p.pool.num_rows) return static_cast<int>(id);
        atomicOr(p.status, DEV_BAD_BLOCK);
        return static_cast<int>(p.pool.num_rows);
      };
      auto prefetch = [&](int j, int row) {   // the page's latents of tile j into L2
        if (row >= 0 && row < p.pool.num_rows)
          bulk_prefetch_l2(p.pool.pool + static_cast<int64_t>(row) * p.pool.row_stride + p.pool.lat_off +
                               static_cast<int64_t>((j * kSelTile + lane * box) & (p.pool.bs - 1)) * kLatDim,
                           box * kLatDim);
      };
      int row = page(s.tile(0));
      prefetch(s.tile(0), row);
      if (seg > 0) ok = warp_wait(q_done, (seg - 1) & 1, ab, ok);
      if (!ok) break;
      q_issued = seg & 1;
      const uint8_t* src = p.q_terms + static_cast<int64_t>(s.t) * kQTokenBytes;
      if (lane == 0) mbar_arrive_expect_tx(q_full, kQTokenBytes);
      __syncwarp();
      if (lane < kQChunks) bulk_load(smem + OFF_Q + lane * QCHUNK, src + lane * QCHUNK, QCHUNK, q_full);
      else if (lane == kQChunks) bulk_load(smem + OFF_QEXP, src + kQTermBytes, kMlaHeads * 4, q_full);
      for (int i = 0; ok && i < s.n; ++i, ++it) {
        const int c1 = (s.tile(i) * kSelTile + lane * box) & (p.pool.bs - 1);
        const int n = __popc(__ballot_sync(0xffffffffu, row >= 0));
        const int next = i + 1 < s.n ? page(s.tile(i + 1)) : -1;
        if (it > 0) ok = warp_wait(tail_empty, (it - 1) & 1, ab, ok);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(tail_full, n * box * 64);
        __syncwarp();
        if (row >= 0) tma_load_3d(smem + OFF_TAIL + lane * box * 64, &tmap, tail_full, 512, c1, row);
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
          if (it > 0) ok = warp_wait(&lat_empty[k], (it - 1) & 1, ab, ok);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&lat_full[k], n * box * 128);
          __syncwarp();
          if (row >= 0) tma_load_3d(smem + OFF_LAT + k * SLICE + lane * box * 128, &lmap, &lat_full[k], 128 * k, c1, row);
        }
        row = next;
        if (i + 1 < s.n) prefetch(s.tile(i + 1), row);
      }
    }
    // after a failed wait: no copy into shared memory outlives the CTA (a barrier whose copy
    // was not issued for this tile keeps its earlier phase; the wait is bounded)
    if (!ok && lane == 0) {
      if (q_issued >= 0) drain_wait(q_full, q_issued);
      drain_wait(tail_full, it & 1);
      for (int k = 0; k < 4; ++k) drain_wait(&lat_full[k], it & 1);
    }
  } else if (warp == MMA_WARP) {
    // ------------------------------------------------------------ MMA issuer
    const bool leader = elect_one();
    const uint32_t idesc_qk = make_idesc(0, 0, false, false, 128, kMlaHeads);
    const uint32_t idesc_pv = make_idesc(0, 1, true, true, 128, kMlaHeads);   // e4m3 x e5m2 (format 1)
    const uint64_t dq = make_sdesc_sw128(smem_u32(smem + OFF_Q), 16, 1024);        // query terms, K-major
    const uint64_t dl = make_sdesc_sw128(smem_u32(smem + OFF_LAT), 16, 1024);      // latents, K-major (QK)
    const uint64_t dt = make_sdesc_sw64(smem_u32(smem + OFF_TAIL), 16, 512);       // their last 64 dims
    // Values: K step i takes the tokens 8 i .. 8 i + 7 of every lane quarter (rows 32 apart, by
    // the stride between 8-row groups), which every softmax warp writes i-th: the first
    // steps run while the later weights are still computed.
    const uint64_t dv = make_sdesc_sw128(smem_u32(smem + OFF_LAT), SLICE, 4096);   // latents, MN-major
    const uint64_t dp = make_sdesc_sw32(smem_u32(smem + OFF_P), P_BLOCK, 1024);    // P terms, MN-major
    auto values = [&](int v, int i, uint32_t acc) {
      const uint32_t d = tmem + O_COL + 96 * v;
      const uint64_t a = dv + ((v * SLICE + i * 1024) >> 4), b = dp + ((256 * i) >> 4);
      mma_f8f6f4_keep_a<KeepA::kFill>(d, a, b, idesc_pv, acc);
      mma_f8f6f4_keep_a<KeepA::kUse>(d, a, b + (P_TERM >> 4), idesc_pv, 1u);
      mma_f8f6f4_keep_a<KeepA::kLast>(d, a, b + (2 * P_TERM >> 4), idesc_pv, 1u);
    };
    bool ok = true;
    int it = 0;
    for (int seg = 0; ok && walk.next(s); ++seg) {
      ok = warp_wait(q_full, seg & 1, ab, ok);
      for (int i = 0; ok && i < s.n; ++i, ++it) {
        // A slice's arrival is awaited half-way through the MMAs of the one before it: the
        // tensor core still has those to do.
        if (!(ok = warp_wait(tail_full, it & 1, ab, ok))) break;
        tc_fence_after();
        if (leader) {
          const uint64_t a = dt, b = dq + (4 * QCHUNK >> 4);   // chunk 4 of the query: hi | lo of dims 512..575
          mma_f8f6f4_keep_a<KeepA::kFill>(tmem + S_COL, a, b, idesc_qk, 0u);
          mma_f8f6f4_keep_a<KeepA::kLast>(tmem + S_COL, a, b + (64 >> 4), idesc_qk, 1u);
          mma_f8f6f4_keep_a<KeepA::kFill>(tmem + S_COL, a + (32 >> 4), b + (32 >> 4), idesc_qk, 1u);
          mma_f8f6f4_keep_a<KeepA::kLast>(tmem + S_COL, a + (32 >> 4), b + (96 >> 4), idesc_qk, 1u);
          tc_commit(tail_empty);
        }
        __syncwarp();
        ok = warp_wait(&lat_full[0], it & 1, ab, ok);
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (leader && ok) {
#pragma unroll
              for (int kk = 2 * half; kk < 2 * half + 2; ++kk) {
                const uint64_t a = dl + ((k * SLICE + 32 * kk) >> 4), b = dq + ((k * QCHUNK + 32 * kk) >> 4);
                mma_f8f6f4_keep_a<KeepA::kFill>(tmem + S_COL, a, b, idesc_qk, 1u);
                mma_f8f6f4_keep_a<KeepA::kLast>(tmem + S_COL, a, b + (5 * QCHUNK >> 4), idesc_qk, 1u);
              }
            }
            __syncwarp();
            if (half == 0 && k < 3) {
              ok = warp_wait(&lat_full[k + 1], it & 1, ab, ok);
              tc_fence_after();
            }
          }
        }
        if (!ok) break;
        if (leader) tc_commit(s_full);
        __syncwarp();
        const uint32_t acc = i % kRunTiles ? 1u : 0u;   // the accumulators start again
        const bool last = i == s.n - 1;
        if (!(ok = warp_wait(&p_full[0], it & 1, ab, ok))) break;
        tc_fence_after();
        if (leader) {
          // the query may go once every softmax warp is past its own wait for it, too
          if (last) tc_commit(q_done);
          values(2, 0, acc);
          values(3, 0, acc);
        }
        __syncwarp();
        if (!(ok = warp_wait(&p_full[1], it & 1, ab, ok))) break;
        tc_fence_after();
        if (leader) {
          values(2, 1, 1u);
          values(3, 1, 1u);
          values(0, 0, acc);
          values(0, 1, 1u);
        }
        __syncwarp();
        if (!(ok = warp_wait(&p_full[2], it & 1, ab, ok))) break;
        tc_fence_after();
        if (leader) {
          // slices come free one after the other, the first half-way through the values
          values(0, 2, 1u);
          values(0, 3, 1u);
          tc_commit(&lat_empty[0]);
#pragma unroll
          for (int i = 0; i < 4; ++i) values(1, i, i ? 1u : acc);
          tc_commit(&lat_empty[1]);
#pragma unroll
          for (int v = 2; v < 4; ++v) {
            values(v, 2, 1u);
            values(v, 3, 1u);
            tc_commit(&lat_empty[v]);
          }
          if (last) tc_commit(o_done);
        }
        __syncwarp();
      }
    }
    if (!ok && leader) {
      tc_commit(drain);
      drain_wait(drain, 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ softmax and epilogue (0..11)
    // Scores are loaded 16 lanes x 8 columns at a time: thread l holds, for the tokens
    // l / 4 + 8 i (i < 4) of its warp's lane quarter, the heads 8 b + 2 a + e (a = l % 4, b < 4,
    // e < 2) of its group: 8 heads, whose scale, reference and sum stay in registers.  P and
    // O hold the group's heads in the order 8 a + 2 b + e, a thread's 8 side by side.
    const int quarter = warp & 3, g = warp >> 2;   // tokens 32 quarter .. of a tile, heads 32 g ..
    const int a = lane & 3, r4 = lane >> 2;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const int my_head = 32 * g + head_of_column(lane);   // of column 32 g + lane of O
    bool ok = true;
    int it = 0;
    for (int seg = 0; walk.next(s); ++seg) {
      const int pos = s.tok.pos, base = s.tok.base;
      const uint32_t* mrow = p.tree.mask + static_cast<int64_t>(s.t) * p.tree.words;
      const int plain = min(base, pos + 1);   // positions below are all seen
      ok = warp_wait(q_full, seg & 1, ab, ok);
      float2 c2[4], sh2[4], l2[4];            // per head pair b: logit scale (log2 units), SHIFT - reference, sum
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int2 qe = *reinterpret_cast<const int2*>(smem + OFF_QEXP + 4 * (32 * g + 8 * b + 2 * a));
        c2[b] = make_float2(p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - qe.x) << 23),
                            p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - qe.y) << 23));
        sh2[b] = make_float2(INFINITY, INFINITY);   // any logit seen exceeds the reference
        l2[b] = make_float2(0.f, 0.f);
      }
      float m_ref = -INFINITY;                // quarter 0: reference of column 32 g + lane
      for (int n = 0;;) {
        for (const int end = min(s.n, n + kRunTiles); n < end; ++n, ++it) {
          const int j = s.tile(n);
          ok = warp_wait(s_full, it & 1, ab, ok);
          tc_fence_after();
          // y[i][b]: logits in log2 units less the reference, plus SHIFT
          uint32_t rr[2][16];
          const uint32_t ts = tmem + S_COL + 32 * g + lane_off;
          DSA_TMEM_LD_16X256_X4(ts, rr[0]);
          tmem_wait_ld();
          DSA_TMEM_LD_16X256_X4(ts + (16u << 16), rr[1]);   // lands while the first half is scaled
          const bool border = (j + 1) * kSelTile > plain;
          uint32_t seen = 15u;                  // bit i: token i of this thread is seen
          if (border) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int s0 = j * kSelTile + 32 * quarter + r4 + 8 * i;
              if (!(s0 <= pos && tree_sees(mrow, p.tree.words, base, s0))) seen &= ~(1u << i);
            }
          }
          float2 y[4][4];
          auto raw = [&](int i, int b) {
            return make_float2(__uint_as_float(rr[i >> 1][4 * b + 2 * (i & 1)]),
                               __uint_as_float(rr[i >> 1][4 * b + 2 * (i & 1) + 1]));
          };
          auto logits = [&](int i0) {   // of the tokens i0 and i0 + 1; their maximum
            float mx = -INFINITY;
#pragma unroll
            for (int i = i0; i < i0 + 2; ++i) {
#pragma unroll
              for (int b = 0; b < 4; ++b) {
                y[i][b] = fma2(raw(i, b), c2[b], sh2[b]);
                if (!((seen >> i) & 1u)) y[i][b] = make_float2(-INFINITY, -INFINITY);
                mx = fmaxf(fmaxf(mx, y[i][b].x), y[i][b].y);
              }
            }
            return mx;
          };
          bool moves = n == 0;   // a segment's first tile sets the references
          if (moves) {
            tmem_wait_ld();
          } else {
            float mx = logits(0);
            tmem_wait_ld();
            mx = fmaxf(mx, logits(2));
            moves = named_bar_any(1, MATH, mx > SHIFT + TAU);
          }
          if (moves) {
            // some reference moves: the tile's maxima per head
            float hm[8];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              hm[2 * b] = hm[2 * b + 1] = -INFINITY;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float2 x = raw(i, b);
                if ((seen >> i) & 1u) {
                  hm[2 * b] = fmaxf(hm[2 * b], x.x * c2[b].x);
                  hm[2 * b + 1] = fmaxf(hm[2 * b + 1], x.y * c2[b].y);
                }
              }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k)
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) hm[k] = fmaxf(hm[k], __shfl_xor_sync(0xffffffffu, hm[k], o));
            if (r4 == 0) {
#pragma unroll
              for (int k = 0; k < 8; ++k) red[quarter * kMlaHeads + 32 * g + 8 * a + k] = hm[k];
            }
            named_bar_sync(2, MATH);
            if (quarter == 0) {
              const int n = 32 * g + lane;
              const float m = fmaxf(fmaxf(red[n], red[kMlaHeads + n]), fmaxf(red[2 * kMlaHeads + n], red[3 * kMlaHeads + n]));
              float alpha = 1.f;
              if (m - m_ref > TAU) {   // (exact near TAU, where a sum would be rounded)
                alpha = exp2f(m_ref - m);
                m_ref = m;
              }
              sh_sh[n] = m_ref == -INFINITY ? INFINITY : SHIFT - m_ref;
              alpha_sh[n] = alpha;
            }
            named_bar_sync(2, MATH);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const float2 av = *reinterpret_cast<const float2*>(alpha_sh + 32 * g + 8 * a + 2 * b);
              sh2[b] = *reinterpret_cast<const float2*>(sh_sh + 32 * g + 8 * a + 2 * b);
              l2[b].x *= av.x;
              l2[b].y *= av.y;
            }
            if (n > 0 && ok) {
#pragma unroll 1
              for (int v = 0; v < 4; ++v) {          // this warp's heads in all dim blocks, 16 at a time
#pragma unroll 1
                for (int cc = 0; cc < 2; ++cc) {
                  uint32_t o[16];
                  const uint32_t ta = tmem + O_COL + 96 * v + 32 * g + 16 * cc + lane_off;
                  DSA_TMEM_LD16(ta, o);
                  tmem_wait_ld();
#pragma unroll
                  for (int i = 0; i < 16; ++i)
                    o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha_sh[32 * g + 16 * cc + i]);
                  DSA_TMEM_ST16(ta, o);
                }
              }
              tmem_wait_st();
            }
            logits(0);
            logits(2);
            cap_weights(y);
          }
          // Latents nobody sees are zeroed before the values read them (a weight of zero does not
          // cancel a NaN): 512 bytes a row, 4 lanes x 8 x 16 bytes, three warps share the rows.
          if (border && ok) {
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
              if ((seen >> i) & 1u) continue;
              uint8_t* dst = smem + OFF_LAT + a * SLICE + (32 * quarter + 8 * i + r4) * 128;
              for (int k = g; k < 8; k += 3) *reinterpret_cast<uint4*>(dst + 16 * k) = make_uint4(0u, 0u, 0u, 0u);
            }
          }
          tc_fence_before();   // the scores are in registers
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t t0[2], t1[2], t2[2];   // the three e5m2 terms of 8 weights, 4 per word
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              uint32_t hi[2], mid[2], lo[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int b = 2 * w + e;
                float2 pe = y[i][b];
                pe.x = ex2_fast(pe.x);
                pe.y = ex2_fast(pe.y);
                l2[b] = add2(l2[b], pe);
                const __half2 ph = __floats2half2_rn(pe.x, pe.y);
                uint32_t r1, r2, r3;
                hi[e] = e5m2_term(*reinterpret_cast<const uint32_t*>(&ph), r1);
                mid[e] = e5m2_term(r1, r2);
                lo[e] = e5m2_term(r2, r3);
              }
              t0[w] = __byte_perm(hi[0], hi[1], 0x7531);
              t1[w] = __byte_perm(mid[0], mid[1], 0x7531);
              t2[w] = __byte_perm(lo[0], lo[1], 0x7531);
            }
            if (ok) {
              // row of 32 heads; 32-byte swizzle: the halves of rows 4..7 of 8 are swapped
              const int row = 32 * quarter + 8 * i + r4;
              uint8_t* dst = smem + OFF_P + g * P_BLOCK + row * 32 + ((8 * a) ^ ((row & 4) << 2));
              *reinterpret_cast<uint2*>(dst) = make_uint2(t0[0], t0[1]);
              *reinterpret_cast<uint2*>(dst + P_TERM) = make_uint2(t1[0], t1[1]);
              *reinterpret_cast<uint2*>(dst + 2 * P_TERM) = make_uint2(t2[0], t2[1]);
              if (i != 2) fence_proxy_async_smem();
            }
            if (i != 2) {
              __syncwarp();
              if (ok && lane == 0) mbar_arrive(&p_full[i < 2 ? i : 2]);
            }
          }
        }
        if (n == s.n) break;
        // between runs: the next tile's scores are done, and with them the values before
        ok = warp_wait(s_full, it & 1, ab, ok);
        tc_fence_after();
        if (ok) add_running_sums<false>(p.run, n == kRunTiles, tmem + O_COL + lane_off, sh_sh, run_sh, 32 * g, quarter);
        named_bar_sync(2, MATH);   // everyone has read the sums' references
        if (quarter == 0) run_sh[32 * g + lane] = sh_sh[32 * g + lane];
      }
      // ---- the segment's result: sums over the tokens, then TMEM (thread = dim) -> global
#pragma unroll
      for (int o = 4; o < 32; o <<= 1)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          l2[b].x += __shfl_xor_sync(0xffffffffu, l2[b].x, o);
          l2[b].y += __shfl_xor_sync(0xffffffffu, l2[b].y, o);
        }
      if (r4 == 0) {
#pragma unroll
        for (int b = 0; b < 4; ++b)
          *reinterpret_cast<float2*>(red + quarter * kMlaHeads + 32 * g + 8 * a + 2 * b) = l2[b];
      }
      named_bar_sync(2, MATH);
      if (quarter == 0) {
        const int n = 32 * g + lane;
        const float l = (red[n] + red[kMlaHeads + n]) + (red[2 * kMlaHeads + n] + red[3 * kMlaHeads + n]);
        inv_sh[n] = l == 0.f ? 0.f : 1.f / l;   // nothing seen: output 0
        const float m = m_ref == -INFINITY ? 0.f : m_ref - SHIFT;
        if (ok) {
          if (s.slot >= 0) p.part_ml[static_cast<int64_t>(s.slot) * kMlaHeads + my_head] = make_float2(m, l);
          else if (p.lse) p.lse[static_cast<int64_t>(s.t) * kMlaHeads + my_head] = (m + log2f(l)) * 0.69314718055994531f;
        }
      }
      named_bar_sync(2, MATH);
      ok = warp_wait(o_done, seg & 1, ab, ok);
      tc_fence_after();
      if (s.n > kRunTiles && ok)
        add_running_sums<true>(p.run, false, tmem + O_COL + lane_off, sh_sh, run_sh, 32 * g, quarter);
      store_segment(p, s, ok, tmem + O_COL + lane_off, inv_sh, 32 * g, quarter, smem + OFF_P + g * 8192, 3 + g);
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------- attention with NVFP4 latents
//
// An NVFP4 latent (e2m1 times an e4m3 scale per 16) has up to 6 significant bits: exact in
// fp16, not in any 8-bit type.  Its tiles are converted to fp16 operands, 64 dims of 128
// tokens (16 KB, a "chunk") at a time; the query arrives as fp16, scaled per head by a
// power of two (exact: a bf16 has 8 significant bits).
//   S^T[token, head] = C[token, 0:576] . q[head, 0:576]     M=128, N=96, K=576   (f16)
//   O^T[dim, head]  += V^T[dim, token] . P^T[token, head]    M=128 (x4 dim blocks), N=96, K=128   (f16)
// The softmax is that of the FP8 kernel (tokens on lanes, a reference per head that rarely
// moves, P handed over in three steps), with P in fp16.
// A chunk is the A operand of both products (K-major, then MN-major).  Beside the query
// (108 KB), P (24 KB) and packed rows on their way (16 KB) four chunks fit, so of the
// nine that a tile's scores read, the last four stay for the values and the first four
// are converted again: 13 fills a tile through four fixed places, in the order of the
// tables below.  Each fill, each group of MMAs that frees places and each copy of packed
// rows has its own barrier, completed once a tile.
// Warp 13 brings queries and packed rows (64 dims of 128 tokens, 4 KB, in four places) by
// TMA, and prefetches pages into L2.
// The 12 softmax warps convert, too: the four warps of group g (a row of the tile each
// thread) make the fills f with f % 3 = g; their rows' scales they fetch a tile ahead,
// into shared memory.  Warp 12 issues MMAs.
// Bound by shared memory: the MMAs read 7 KB per 49 cycles (6.6K cycles a tile), the fills
// write 16 KB each (1.7K), and packed rows and P add about 1K; a tile takes 11.8K, the
// rest is the chain scores -> weights -> values, which four places cannot overlap fully.
// 16 tokens over 256K: 1,255 us a call, 698 TFLOP/s.  Rows and scales loaded to registers by the
// threads that convert them: 1,470 us (spilled a tile ahead of use, each spill waited).
namespace t16 {
constexpr int THREADS = 448;
constexpr int QCHUNKS = kLatDim / 64;
constexpr int QCHUNK = 96 * 128;
constexpr int PLACE = 128 * 128;
constexpr int RAW = 128 * 32;                     // packed rows of a chunk, 32-byte swizzle
constexpr int RAWS = 4;
constexpr int OFF_Q = 0;
constexpr int OFF_C = QCHUNKS * QCHUNK;           // four places
constexpr int OFF_P = OFF_C + 4 * PLACE;          // three [128 tokens x 32 heads] fp16 blocks, 64-byte swizzle
constexpr int P_BLOCK = 128 * 64;
constexpr int OFF_RAW = OFF_P + 3 * P_BLOCK;
constexpr int OFF_SCALE = OFF_RAW + RAWS * RAW;   // scale words of the rows: [2 tiles][3 chunks][384 threads]
constexpr int OFF_QEXP = OFF_SCALE + 2 * 3 * 384 * 4;   // [96] int
constexpr int OFF_REDM = OFF_QEXP + 96 * 4;       // [4][96] float
constexpr int OFF_SH = OFF_REDM + 4 * 96 * 4;     // [96] float
constexpr int OFF_ALPHA = OFF_SH + 96 * 4;        // [96] float
constexpr int OFF_INV = OFF_ALPHA + 96 * 4;       // [96] float
constexpr int OFF_RUN = OFF_INV + 96 * 4;         // [96] float: SHIFT - reference of the running sums
constexpr int OFF_BARS = OFF_RUN + 96 * 4;
constexpr int FILLS = 13;
constexpr int OFF_MISC = OFF_BARS + 64 * 8;
constexpr int SMEM_BYTES = OFF_MISC + 64 + 1024;
// chunk and place of fill f: the scores' nine, then the values' four.  Dim block v of the
// values is the chunks 2 v and 2 v + 1, one or three places apart: 4 and 5 in places 1
// and 2, 6 and 7 in 0 and 3 (kept), then 0 and 1 in 1 and 2, 2 and 3 in 0 and 3.
// The fills f of group f % 3 touch three chunks: 0, 3, 7; 1, 8, 5; 2, 4, 6.  Group 0 makes five
// and is the last to start a tile, so the scores take the chunks in the order kOrder.
__device__ constexpr int kChunk[FILLS] = {0, 1, 2, 3, 8, 4, 7, 5, 6, 0, 1, 2, 3};
__device__ constexpr int kPlace[FILLS] = {3, 1, 2, 3, 0, 1, 3, 2, 0, 1, 2, 0, 3};
__device__ constexpr int kOrder[9] = {1, 2, 0, 4, 5, 3, 7, 8, 6};
// the same for a fill known at run time (4 bits each), and the order in which packed rows come:
// the fill of turn o, and the turn of fill f
__device__ __forceinline__ int chunk_of_fill(int f) { return static_cast<int>((0x3210657483210ull >> (4 * f)) & 15); }
__device__ __forceinline__ int place_of_fill(int f) { return static_cast<int>((0x3021023103213ull >> (4 * f)) & 15); }
__device__ __forceinline__ int fill_of_turn(int o) { return static_cast<int>((0xC9BA687354021ull >> (4 * o)) & 15); }
__device__ __forceinline__ int turn_of_fill(int f) { return static_cast<int>((0xCA9B768435102ull >> (4 * f)) & 15); }
// which of its group's three chunks a fill takes
__device__ __forceinline__ int scale_of_fill(int f) { return f < 9 ? f / 3 : (f == 12 ? 1 : 0); }
// events that free places: the scores of fill 0 .. 4 done, or the values of dim block v done
enum { EV_S0 = 0, EV_S1, EV_S2, EV_S3, EV_S4, EV_V0, EV_V1, EV_V2, EV_V3, EVENTS };
// the event that fill f waits for; bit 8: of the tile before
__device__ __forceinline__ int event_of_fill(int f) {
  return f == 0 || f == 4 ? (EV_V1 | 256) : f < 3 ? (EV_V0 | 256) : f == 3 ? EV_S0 : f == 5 ? EV_S1 : f == 6 ? EV_S3
         : f == 7 ? EV_S2 : f == 8 ? EV_S4 : f < 11 ? EV_V2 : EV_V3;
}
constexpr int MATH_WARPS = 12;
constexpr int MATH = MATH_WARPS * 32;
constexpr int MMA_WARP = 12, LOAD_WARP = 13;
constexpr int S_COL = 0;
constexpr int O_COL = 128;
constexpr float TAU = 4.0f;
constexpr float SHIFT = 11.0f;                    // weights up to 2^15 in fp16
static_assert(OFF_C % 1024 == 0 && OFF_P % 1024 == 0, "align");
static_assert(OFF_SH % 16 == 0 && OFF_ALPHA % 16 == 0 && OFF_INV % 16 == 0 && OFF_QEXP % 16 == 0 && OFF_BARS % 8 == 0,
              "vectors are read 16 bytes at a time");
static_assert(SMEM_BYTES <= 232448, "smem");
static_assert(SHIFT + TAU + 0.5f == kTreeCap, "weights' cap");
}  // namespace t16

// 4-byte global -> shared copy without registers (a register that holds a load for a whole
// tile would be spilled, and the spill waits for the load: 1,600 cycles a tile).
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but this thread's newest group are complete.
__device__ __forceinline__ void cp_async_wait_but_one() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

__global__ void __launch_bounds__(t16::THREADS, 1)
    tree_mla_nvfp4_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap rmap,
                          TreeMlaParams p) {
  using namespace t16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024_tree(smem_raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BARS);
  uint64_t* full = bars + 0;        // [FILLS] a chunk is in its place
  uint64_t* raw_full = bars + 13;   // [FILLS] its packed rows are in shared memory
  uint64_t* raw_done = bars + 26;   // [FILLS] and have been read
  uint64_t* event = bars + 39;      // [EVENTS]
  uint64_t* q_full = bars + 48;
  uint64_t* q_done = bars + 49;
  uint64_t* s_full = bars + 50;
  uint64_t* o_done = bars + 51;
  uint64_t* drain = bars + 52;
  uint64_t* p_full = bars + 53;     // [3]
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + OFF_MISC);
  int* abortf = reinterpret_cast<int*>(smem + OFF_MISC + 8);
  float* red = reinterpret_cast<float*>(smem + OFF_REDM);
  float* sh_sh = reinterpret_cast<float*>(smem + OFF_SH);
  float* alpha_sh = reinterpret_cast<float*>(smem + OFF_ALPHA);
  float* inv_sh = reinterpret_cast<float*>(smem + OFF_INV);
  float* run_sh = reinterpret_cast<float*>(smem + OFF_RUN);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < FILLS; ++i) {
      mbar_init(&full[i], 4);
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_done[i], 4);
    }
    for (int i = 39; i < 53; ++i) mbar_init(&bars[i], 1);
    for (int i = 0; i < 3; ++i) mbar_init(&p_full[i], MATH_WARPS);
    *abortf = 0;
    fence_mbar_init();
    prefetch_tensormap(&qmap);
    prefetch_tensormap(&rmap);
  }
  if (warp == 0) tmem_alloc(tslot, 512);
  grid_dep_wait();   // the plan and the query
  grid_dep_launch();
  SegmentWalk walk = make_walk(p);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  const Abort ab{abortf, p.status};
  Segment s;

  // Query operands of token t, by a whole warp: the CTA's first by the MMA warp, which has nothing
  // else to do then, the others by the load warp (1,300 us instead of 1,320 for 16 tokens over
  // 256K; the FP8 kernel, at the power cap, gains nothing from it).
  auto load_query = [&](int t) {
    if (lane == 0) mbar_arrive_expect_tx(q_full, QCHUNKS * QCHUNK + kMlaHeads * 4);
    __syncwarp();
    if (lane < QCHUNKS) tma_load_2d(smem + OFF_Q + lane * QCHUNK, &qmap, q_full, lane * 64, t * kMlaHeads);
    else if (lane == QCHUNKS)
      bulk_load(smem + OFF_QEXP, p.q_exps + static_cast<int64_t>(t) * kMlaHeads, kMlaHeads * 4, q_full);
    __syncwarp();
  };

  if (warp == LOAD_WARP) {
    // ------------------------------------------- queries, packed rows, L2 prefetch
    const int lg = p.pool.log2_bs;
    const int box = min(p.pool.bs, kSelTile);     // positions of one copy
    const int nbox = kSelTile / box;              // copies (lanes) per chunk
    bool ok = true;
    int it = 0, q_issued = -1, o = 0;
    for (int seg = 0; ok && walk.next(s); ++seg) {
      const int pos = s.tok.pos;
      const int32_t* btrow = p.b.bt + static_cast<int64_t>(s.tok.req) * p.b.bt_stride;
      // this lane's page of tile j: pool row (num_rows, which reads as zeros, for a bad id)
      auto page = [&](int j) {
        const int s0 = j * kSelTile + lane * box;
        if (lane >= nbox || s0 > pos) return -1;
        const int32_t id = __ldg(btrow + (s0 >> lg));
        if (id >= 0 && id < p.pool.num_rows) return static_cast<int>(id);
        atomicOr(p.status, DEV_BAD_BLOCK);
        return static_cast<int>(p.pool.num_rows);
      };
      auto prefetch = [&](int j, int row) {   // the page's latents of tile j into L2
        if (row >= 0 && row < p.pool.num_rows)
          bulk_prefetch_l2(p.pool.pool + static_cast<int64_t>(row) * p.pool.row_stride + p.pool.lat_off +
                               static_cast<int64_t>((j * kSelTile + lane * box) & (p.pool.bs - 1)) * 352,
                           box * 352);
      };
      int row = page(s.tile(0));
      prefetch(s.tile(0), row);
      if (seg > 0) ok = warp_wait(q_done, (seg - 1) & 1, ab, ok);
      if (!ok) break;
      if (seg > 0) load_query(s.t);
      q_issued = seg & 1;
      for (int i = 0; ok && i < s.n; ++i, ++it) {
        const int c1 = (s.tile(i) * kSelTile + lane * box) & (p.pool.bs - 1);
        const int n = __popc(__ballot_sync(0xffffffffu, row >= 0));
        const int next = i + 1 < s.n ? page(s.tile(i + 1)) : -1;
        if (i + 1 < s.n) prefetch(s.tile(i + 1), next);
#pragma unroll 1
        for (o = 0; o < FILLS; ++o) {
          // the place of copy 13 it + o was last used four copies before
          const int f = fill_of_turn(o), u = fill_of_turn(o < RAWS ? o + FILLS - RAWS : o - RAWS);
          if (it > 0 || o >= RAWS) ok = warp_wait(&raw_done[u], (o < RAWS ? it - 1 : it) & 1, ab, ok);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&raw_full[f], n * box * 32);
          __syncwarp();
          const int place = (FILLS * it + o) % RAWS;
          if (row >= 0)
            tma_load_3d(smem + OFF_RAW + place * RAW + lane * box * 32, &rmap, &raw_full[f], 32 * chunk_of_fill(f), c1, row);
        }
        if (!ok) break;
        row = next;
      }
    }
    // after a failed wait: no copy into shared memory outlives the CTA (a barrier whose copy
    // was not issued for this tile keeps its earlier phase; the wait is bounded)
    if (!ok && lane == 0) {
      if (q_issued >= 0) drain_wait(q_full, q_issued);
      for (int i = 0; i < RAWS && i < FILLS * it + o; ++i) {   // the last copies issued
        const int n = FILLS * it + o - 1 - i;
        drain_wait(&raw_full[fill_of_turn(n % FILLS)], (n / FILLS) & 1);
      }
    }
  } else if (warp == MMA_WARP) {
    // ------------------------------------------------------------ MMA issuer
    const bool leader = elect_one();
    const uint32_t idesc_qk = make_idesc(0, 0, false, false, 128, kMlaHeads);
    const uint32_t idesc_pv = make_idesc(0, 0, true, true, 128, kMlaHeads);
    const uint64_t dq = make_sdesc_sw128(smem_u32(smem + OFF_Q), 16, 1024);   // query, K-major
    const uint64_t dc = make_sdesc_sw128(smem_u32(smem + OFF_C), 16, 1024);   // chunks, K-major (scores)
    // Values: step i takes the tokens 8 i .. 8 i + 7 of every lane quarter (rows 32 apart), two
    // quarters an MMA; the second 64 dims of a block lie 1 or 3 places behind the first.
    const uint64_t dv1 = make_sdesc_sw128(smem_u32(smem + OFF_C + PLACE), PLACE, 4096);   // places 1 and 2
    const uint64_t dv3 = make_sdesc_sw128(smem_u32(smem + OFF_C), 3 * PLACE, 4096);       // places 0 and 3
    const uint64_t dp = make_sdesc_sw64(smem_u32(smem + OFF_P), P_BLOCK, 2048);
    auto values = [&](int v, int i, uint32_t acc) {
      const uint64_t a = (v & 1 ? dv3 : dv1) + ((i * 1024) >> 4);
      const uint64_t b = dp + ((512 * i) >> 4);
      const uint32_t d = tmem + O_COL + 96 * v;
      mma_f16(d, a, b, idesc_pv, acc);
      mma_f16(d, a + (8192 >> 4), b + (4096 >> 4), idesc_pv, 1u);
    };
    bool ok = true;
    int it = 0;
    for (int seg = 0; ok && walk.next(s); ++seg) {
      if (seg == 0) load_query(s.t);
      ok = warp_wait(q_full, seg & 1, ab, ok);
      for (int i = 0; ok && i < s.n; ++i, ++it) {
        ok = warp_wait(&full[kOrder[0]], it & 1, ab, ok);
        tc_fence_after();
#pragma unroll
        for (int o = 0; o < 9; ++o) {
          const int f = kOrder[o];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (leader && ok) {
#pragma unroll
              for (int kk = 2 * half; kk < 2 * half + 2; ++kk)
                mma_f16(tmem + S_COL, dc + ((kPlace[f] * PLACE + 32 * kk) >> 4), dq + ((kChunk[f] * QCHUNK + 32 * kk) >> 4),
                        idesc_qk, (o | kk) ? 1u : 0u);
              if (half == 1 && f < 5) tc_commit(&event[EV_S0 + f]);
            }
            __syncwarp();
            if (half == 0 && o < 8) {   // the next chunk is awaited while the tensor core has work
              ok = warp_wait(&full[kOrder[o + 1]], it & 1, ab, ok);
              tc_fence_after();
            }
          }
        }
        if (!ok) break;
        if (leader) tc_commit(s_full);
        __syncwarp();
        const uint32_t acc = i % kRunTiles ? 1u : 0u;   // the accumulators start again
        const bool last = i == s.n - 1;
        if (!(ok = warp_wait(&p_full[0], it & 1, ab, ok))) break;
        tc_fence_after();
        if (leader) {
          if (last) tc_commit(q_done);   // every softmax warp is past its own wait for the query
          values(3, 0, acc);
          values(2, 0, acc);
        }
        __syncwarp();
        if (!(ok = warp_wait(&p_full[1], it & 1, ab, ok))) break;
        tc_fence_after();
        if (leader) values(2, 1, 1u);
        __syncwarp();
        if (!(ok = warp_wait(&p_full[2], it & 1, ab, ok))) break;
        tc_fence_after();
        if (leader) {
          values(2, 2, 1u);
          values(2, 3, 1u);
          tc_commit(&event[EV_V2]);
          values(3, 1, 1u);
          values(3, 2, 1u);
          values(3, 3, 1u);
          tc_commit(&event[EV_V3]);
        }
        __syncwarp();
        ok = warp_wait(&full[9], it & 1, ab, ok);
        if (!(ok = warp_wait(&full[10], it & 1, ab, ok))) break;
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int i = 0; i < 4; ++i) values(0, i, i ? 1u : acc);
          tc_commit(&event[EV_V0]);
        }
        __syncwarp();
        ok = warp_wait(&full[11], it & 1, ab, ok);
        if (!(ok = warp_wait(&full[12], it & 1, ab, ok))) break;
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int i = 0; i < 4; ++i) values(1, i, i ? 1u : acc);
          tc_commit(&event[EV_V1]);
          if (last) tc_commit(o_done);
        }
        __syncwarp();
      }
    }
    if (!ok && leader) {
      tc_commit(drain);
      drain_wait(drain, 0);
    }
    __syncwarp();
  } else {
    // -------------------------------- conversion, softmax and epilogue (0..11)
    const int quarter = warp & 3, g = warp >> 2;
    const int a = lane & 3, r4 = lane >> 2;
    const int crow = 32 * quarter + lane;          // this thread's row of a chunk
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const int my_head = 32 * g + head_of_column(lane);
    const int lg = p.pool.log2_bs, bsm = p.pool.bs - 1;
    bool ok = true;
    int it = 0;
    // Fill f: the row's 32 packed bytes -> 64 fp16 values in registers, then, once the place is
    // free (on the CTA's first tile the first ones are), into it.  A row nobody sees is zeros.
    uint32_t* scales = reinterpret_cast<uint32_t*>(smem + OFF_SCALE) + threadIdx.x;
    auto fill = [&](int f, bool seen_row) {
      ok = warp_wait(&raw_full[f], it & 1, ab, ok);
      const uint8_t* src = smem + OFF_RAW + (FILLS * it + turn_of_fill(f)) % RAWS * RAW + crow * 32;
      const int sw = ((crow >> 2) & 1) << 4;
      const uint4 w0 = *reinterpret_cast<const uint4*>(src + sw), w1 = *reinterpret_cast<const uint4*>(src + (sw ^ 16));
      // The place is given back once the loads have returned, which an arrival behind them does not
      // imply: with shared memory busy the next copy was faster than they.  So the barrier's address
      // takes a bit of both (p.never is 0, and not known to be).
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&raw_done[f] + ((w0.x ^ w1.x) & p.never));
      const uint32_t sw4 = seen_row ? scales[((it & 1) * 3 + scale_of_fill(f)) * 384] : 0u;
      uint32_t o[4][8];
      nvfp4x16_to_f16(make_uint2(w0.x, w0.y), sw4 & 0xFFu, o[0]);
      nvfp4x16_to_f16(make_uint2(w0.z, w0.w), (sw4 >> 8) & 0xFFu, o[1]);
      nvfp4x16_to_f16(make_uint2(w1.x, w1.y), (sw4 >> 16) & 0xFFu, o[2]);
      nvfp4x16_to_f16(make_uint2(w1.z, w1.w), sw4 >> 24, o[3]);
      const int ev = event_of_fill(f);
      if (it > 0 || ev < 256) ok = warp_wait(&event[ev & 255], (it & 1) ^ (ev >> 8), ab, ok);
      if (ok) {
        uint8_t* dst = smem + OFF_C + place_of_fill(f) * PLACE + (crow >> 3) * 1024;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          sts128(dst + sw128_off(crow & 7, 2 * q), o[q]);
          sts128(dst + sw128_off(crow & 7, 2 * q + 1), o[q] + 4);
        }
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&full[f]);
    };
    for (int seg = 0; walk.next(s); ++seg) {
      const int req = s.tok.req, pos = s.tok.pos, base = s.tok.base;
      const uint32_t* mrow = p.tree.mask + static_cast<int64_t>(s.t) * p.tree.words;
      const int32_t* btrow = p.b.bt + static_cast<int64_t>(req) * p.b.bt_stride;
      const int plain = min(base, pos + 1);   // positions below are all seen
      // The record of this thread's position in the segment's i-th tile, null where nobody sees it or the block id
      // is bad (the loads report that); ids are read two tiles ahead, scales one.
      auto block = [&](int i) {
        const int sv = s.tile(i) * kSelTile + crow;
        if (i >= s.n || !(sv < plain || (sv <= pos && tree_sees(mrow, p.tree.words, base, sv)))) return -1;
        return static_cast<int>(__ldg(btrow + (sv >> lg)));
      };
      auto record = [&](int i, int id) -> const uint8_t* {
        if (id < 0 || id >= p.pool.num_rows) return nullptr;
        return p.pool.pool + static_cast<int64_t>(id) * p.pool.row_stride + p.pool.lat_off +
               static_cast<int64_t>((s.tile(i) * kSelTile + crow) & bsm) * 352;
      };
      // the scale words of the group's chunks for the CTA's tile `n`, on their way to shared memory
      auto fetch_scales = [&](const uint8_t* r, int n) {
        if (r) {
#pragma unroll
          for (int k = 0; k < 3; ++k)
            cp_async4(smem_u32(scales + ((n & 1) * 3 + k) * 384), r + 288 + 4 * chunk_of_fill(g + 3 * k));
        }
        cp_async_commit();
      };
      const uint8_t* rec = record(0, block(0));
      int id1 = block(1);
      fetch_scales(rec, it);
      ok = warp_wait(q_full, seg & 1, ab, ok);
      float2 c2[4], sh2[4], l2[4];            // per head pair b: logit scale (log2 units), SHIFT - reference, sum
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int2 qe = *reinterpret_cast<const int2*>(smem + OFF_QEXP + 4 * (32 * g + 8 * b + 2 * a));
        c2[b] = make_float2(p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - qe.x) << 23),
                            p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - qe.y) << 23));
        sh2[b] = make_float2(INFINITY, INFINITY);   // any logit seen exceeds the reference
        l2[b] = make_float2(0.f, 0.f);
      }
      float m_ref = -INFINITY;                // quarter 0: reference of column 32 g + lane
      for (int n = 0;;) {
        for (const int end = min(s.n, n + kRunTiles); n < end; ++n, ++it) {
          const int j = s.tile(n);
          const uint8_t* next = record(n + 1, id1);
          id1 = block(n + 2);
          fetch_scales(next, it + 1);
          cp_async_wait_but_one();
          const bool seen_row = rec != nullptr;
          // ---- the scores' chunks
#pragma unroll 1
          for (int f = g; f < 9; f += 3) fill(f, seen_row);
          // ---- softmax (as in the FP8 kernel)
          ok = warp_wait(s_full, it & 1, ab, ok);
          tc_fence_after();
          uint32_t rr[2][16];
          const uint32_t ts = tmem + S_COL + 32 * g + lane_off;
          DSA_TMEM_LD_16X256_X4(ts, rr[0]);
          tmem_wait_ld();
          DSA_TMEM_LD_16X256_X4(ts + (16u << 16), rr[1]);   // lands while the first half is scaled
          uint32_t seen = 15u;                  // bit i: token i of this thread is seen
          if ((j + 1) * kSelTile > plain) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int s0 = j * kSelTile + 32 * quarter + r4 + 8 * i;
              if (!(s0 <= pos && tree_sees(mrow, p.tree.words, base, s0))) seen &= ~(1u << i);
            }
          }
          float2 y[4][4];
          auto raw = [&](int i, int b) {
            return make_float2(__uint_as_float(rr[i >> 1][4 * b + 2 * (i & 1)]),
                               __uint_as_float(rr[i >> 1][4 * b + 2 * (i & 1) + 1]));
          };
          auto logits = [&](int i0) {
            float mx = -INFINITY;
#pragma unroll
            for (int i = i0; i < i0 + 2; ++i) {
#pragma unroll
              for (int b = 0; b < 4; ++b) {
                y[i][b] = fma2(raw(i, b), c2[b], sh2[b]);
                if (!((seen >> i) & 1u)) y[i][b] = make_float2(-INFINITY, -INFINITY);
                mx = fmaxf(fmaxf(mx, y[i][b].x), y[i][b].y);
              }
            }
            return mx;
          };
          bool moves = n == 0;
          if (moves) {
            tmem_wait_ld();
          } else {
            float mx = logits(0);
            tmem_wait_ld();
            mx = fmaxf(mx, logits(2));
            moves = named_bar_any(1, MATH, mx > SHIFT + TAU);
          }
          if (moves) {
            // P of the tile before has been used (s_full follows its values); some reference moves
            float hm[8];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              hm[2 * b] = hm[2 * b + 1] = -INFINITY;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float2 x = raw(i, b);
                if ((seen >> i) & 1u) {
                  hm[2 * b] = fmaxf(hm[2 * b], x.x * c2[b].x);
                  hm[2 * b + 1] = fmaxf(hm[2 * b + 1], x.y * c2[b].y);
                }
              }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k)
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) hm[k] = fmaxf(hm[k], __shfl_xor_sync(0xffffffffu, hm[k], o));
            if (r4 == 0) {
#pragma unroll
              for (int k = 0; k < 8; ++k) red[quarter * kMlaHeads + 32 * g + 8 * a + k] = hm[k];
            }
            named_bar_sync(2, MATH);
            if (quarter == 0) {
              const int n = 32 * g + lane;
              const float m = fmaxf(fmaxf(red[n], red[kMlaHeads + n]), fmaxf(red[2 * kMlaHeads + n], red[3 * kMlaHeads + n]));
              float alpha = 1.f;
              if (m - m_ref > TAU) {   // (exact near TAU, where a sum would be rounded)
                alpha = exp2f(m_ref - m);
                m_ref = m;
              }
              sh_sh[n] = m_ref == -INFINITY ? INFINITY : SHIFT - m_ref;
              alpha_sh[n] = alpha;
            }
            named_bar_sync(2, MATH);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const float2 av = *reinterpret_cast<const float2*>(alpha_sh + 32 * g + 8 * a + 2 * b);
              sh2[b] = *reinterpret_cast<const float2*>(sh_sh + 32 * g + 8 * a + 2 * b);
              l2[b].x *= av.x;
              l2[b].y *= av.y;
            }
            if (n > 0 && ok) {
#pragma unroll 1
              for (int v = 0; v < 4; ++v) {
#pragma unroll 1
                for (int cc = 0; cc < 4; ++cc) {
                  uint32_t o[8];
                  const uint32_t ta = tmem + O_COL + 96 * v + 32 * g + 8 * cc + lane_off;
                  DSA_TMEM_LD8(ta, o);
                  tmem_wait_ld();
#pragma unroll
                  for (int i = 0; i < 8; ++i)
                    o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha_sh[32 * g + 8 * cc + i]);
                  DSA_TMEM_ST8(ta, o);
                }
              }
              tmem_wait_st();
            }
            logits(0);
            logits(2);
            cap_weights(y);
          }
          tc_fence_before();   // the scores are in registers
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t t0[4];    // 8 weights in fp16
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              float2 pe = y[i][b];
              pe.x = ex2_fast(pe.x);
              pe.y = ex2_fast(pe.y);
              l2[b] = add2(l2[b], pe);
              const __half2 ph = __floats2half2_rn(pe.x, pe.y);
              t0[b] = *reinterpret_cast<const uint32_t*>(&ph);
            }
            if (ok) {
              // row of 32 heads, 64 bytes; 64-byte swizzle: the 16-byte piece moves by (row / 2) % 4
              const int row = 32 * quarter + 8 * i + r4;
              sts128(smem + OFF_P + g * P_BLOCK + row * 64 + ((a ^ ((row >> 1) & 3)) << 4), t0);
              if (i != 2) fence_proxy_async_smem();
            }
            if (i != 2) {
              __syncwarp();
              if (ok && lane == 0) mbar_arrive(&p_full[i < 2 ? i : 2]);
            }
          }
          // ---- the values' chunks that did not stay, as the places come free
#pragma unroll 1
          for (int f = 9 + g; f < FILLS; f += 3) fill(f, seen_row);
          rec = next;
        }
        if (n == s.n) break;
        // between runs: the last values of the tile before are done, and with them all of them
        ok = warp_wait(&event[EV_V1], (it - 1) & 1, ab, ok);
        tc_fence_after();
        if (ok) add_running_sums<false>(p.run, n == kRunTiles, tmem + O_COL + lane_off, sh_sh, run_sh, 32 * g, quarter);
        named_bar_sync(2, MATH);   // everyone has read the sums' references
        if (quarter == 0) run_sh[32 * g + lane] = sh_sh[32 * g + lane];
      }
      // ---- the segment's result: sums over the tokens, then TMEM (thread = dim) -> global
#pragma unroll
      for (int o = 4; o < 32; o <<= 1)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          l2[b].x += __shfl_xor_sync(0xffffffffu, l2[b].x, o);
          l2[b].y += __shfl_xor_sync(0xffffffffu, l2[b].y, o);
        }
      if (r4 == 0) {
#pragma unroll
        for (int b = 0; b < 4; ++b)
          *reinterpret_cast<float2*>(red + quarter * kMlaHeads + 32 * g + 8 * a + 2 * b) = l2[b];
      }
      named_bar_sync(2, MATH);
      if (quarter == 0) {
        const int n = 32 * g + lane;
        const float l = (red[n] + red[kMlaHeads + n]) + (red[2 * kMlaHeads + n] + red[3 * kMlaHeads + n]);
        inv_sh[n] = l == 0.f ? 0.f : 1.f / l;   // nothing seen: output 0
        const float m = m_ref == -INFINITY ? 0.f : m_ref - SHIFT;
        if (ok) {
          if (s.slot >= 0) p.part_ml[static_cast<int64_t>(s.slot) * kMlaHeads + my_head] = make_float2(m, l);
          else if (p.lse) p.lse[static_cast<int64_t>(s.t) * kMlaHeads + my_head] = (m + log2f(l)) * 0.69314718055994531f;
        }
      }
      named_bar_sync(2, MATH);
      ok = warp_wait(o_done, seg & 1, ab, ok);
      tc_fence_after();
      if (s.n > kRunTiles && ok)
        add_running_sums<true>(p.run, false, tmem + O_COL + lane_off, sh_sh, run_sh, 32 * g, quarter);
      store_segment(p, s, ok, tmem + O_COL + lane_off, inv_sh, 32 * g, quarter, smem + OFF_P + g * 8192, 3 + g);
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// Merge of a token's partials: out = sum_j w_j o_j, w_j = l_j 2^(m_j - M) / sum.  Tokens with
// one segment have their output already.  Grid (96 PARTS / 8, T): a block takes 8 / PARTS heads,
// 64 threads (8 dims each) for each of PARTS interleaved parts of the partials.  Bound by
// latency, two rounds of loads: the block reads all (max, sum) pairs at once, and a
// thread's partials are loaded eight at a time.  212 tokens of 2 or 3 partials: 69 us with a
// block per head and a pass per pair, 22 us so.
constexpr int kTreeCombThreads = 512;
constexpr int kTreeCombMax = 256;   // CTAs at most, so partials of a token
template <int PARTS>
__global__ void __launch_bounds__(kTreeCombThreads, PARTS > 1 ? 2 : 3) tree_combine_kernel(TreeMlaParams p) {
  constexpr int HEADS = 8 / PARTS;
  __shared__ float wgt[HEADS][kTreeCombMax];
  __shared__ float2 ml_sh[HEADS][kTreeCombMax];
  __shared__ float acc_sh[PARTS > 1 ? PARTS - 1 : 1][HEADS][64][8];
  const int t = blockIdx.y, h0 = blockIdx.x * HEADS;
  // The plan was complete before the attention let this kernel start: it is read ahead of the wait.
  const int64_t W = __ldcg(p.starts + p.b.T);
  const int64_t u0 = __ldcg(p.starts + t), u1 = __ldcg(p.starts + t + 1);
  int c0 = 0, c1 = 0, first = 0;
  if (u1 > u0) {
    const int G = static_cast<int>(W < p.max_ctas ? W : p.max_ctas);
    c0 = share_of(W, G, u0);
    c1 = share_of(W, G, u1 - 1);
    first = 2 * c0 + (share_begin(W, G, c0) < u0 ? 1 : 0);
  }
  grid_dep_wait();
  grid_dep_launch();
  if (c0 == c1) return;   // padding, or one segment
  const int n = c1 - c0 + 1;
  auto slot = [&](int j) { return j == 0 ? first : 2 * (c0 + j); };
  const int d8 = threadIdx.x & 63, unit = threadIdx.x >> 6;
  const int part = unit % PARTS, hh = unit / PARTS;   // the first two warps of a head: part 0
  for (int i = threadIdx.x; i < n * HEADS; i += kTreeCombThreads)
    ml_sh[i % HEADS][i / HEADS] = __ldcg(p.part_ml + static_cast<int64_t>(slot(i / HEADS)) * kMlaHeads + h0 + i % HEADS);
  // the first partials are on their way meanwhile
  constexpr int U = PARTS > 1 ? 8 : 4;
  const uint4* src = reinterpret_cast<const uint4*>(p.part_o + static_cast<int64_t>(h0 + hh) * kVDim) + d8;
  auto load = [&](int j) {
    return j < n ? __ldcg(src + static_cast<int64_t>(slot(j)) * (kMlaHeads * kVDim / 8)) : make_uint4(0u, 0u, 0u, 0u);
  };
  uint4 v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) v[u] = load(part + PARTS * u);
  __syncthreads();
  // weights of a head, by each of its warps (same values from each)
  const int lane = threadIdx.x & 31;
  float M = -INFINITY, L = 0.f;
  for (int j = lane; j < n; j += 32) {
    const float2 ml = ml_sh[hh][j];
    if (ml.y != 0.f) M = fmaxf(M, ml.x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  for (int j = lane; j < n; j += 32) {
    const float2 ml = ml_sh[hh][j];
    const float w = ml.y == 0.f ? 0.f : exp2f(ml.x - M) * ml.y;
    wgt[hh][j] = w;
    L += w;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  __syncwarp();   // each warp reads what it wrote (its head's other warps write the same)
  float acc[8] = {};
  for (int j = part; j < n; j += PARTS * U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float w = j + PARTS * u < n ? wgt[hh][j + PARTS * u] : 0.f;
      const uint32_t w4[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w4[e]));
        acc[2 * e] = fmaf(w, f.x, acc[2 * e]);
        acc[2 * e + 1] = fmaf(w, f.y, acc[2 * e + 1]);
      }
      v[u] = load(j + PARTS * (u + U));
    }
  }
  if constexpr (PARTS > 1) {
    if (part > 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) acc_sh[part - 1][hh][d8][e] = acc[e];
    }
    __syncthreads();
    if (part > 0) return;
    for (int q = 0; q < PARTS - 1; ++q)
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += acc_sh[q][hh][d8][e];
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  alignas(16) __nv_bfloat162 o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = __floats2bfloat162_rn(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  const int64_t row = static_cast<int64_t>(t) * kMlaHeads + h0 + hh;
  *reinterpret_cast<uint4*>(p.out + row * kVDim + 8 * d8) = *reinterpret_cast<const uint4*>(o);
  if (d8 == 0 && p.lse) p.lse[row] = (M + log2f(L)) * 0.69314718055994531f;
}

static cudaError_t launch_combine(const TreeMlaParams& p, cudaStream_t st) {
  if (p.whole) return cudaSuccess;
  if (p.max_ctas > kTreeCombMax) return cudaErrorInvalidValue;
  // Few tokens have many partials each: their heads are spread over four times the blocks (a call
  // with one token over 20K takes 28.9 us so, 61.5 with 12 blocks; eight tokens 50.5 and 51.7).
  if (12 * p.b.T < p.max_ctas)
    return launch_ex(tree_combine_kernel<4>, dim3(48, p.b.T), dim3(kTreeCombThreads), 0, st, true, 0u, p);
  return launch_ex(tree_combine_kernel<1>, dim3(12, p.b.T), dim3(kTreeCombThreads), 0, st, true, 0u, p);
}

cudaError_t launch_tree_mla_fp8(const CUtensorMap& lmap, const CUtensorMap& tmap, const TreeMlaParams& p,
                                cudaStream_t st) {
  cudaError_t e = set_func_attr_once(reinterpret_cast<const void*>(tree_mla_fp8_kernel),
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, t8::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  e = launch_ex(tree_mla_fp8_kernel, dim3(p.max_ctas), dim3(t8::THREADS), t8::SMEM_BYTES, st, true, 0u, lmap, tmap, p);
  return e != cudaSuccess ? e : launch_combine(p, st);
}

cudaError_t launch_tree_mla_nvfp4(const CUtensorMap& qmap, const CUtensorMap& rmap, const TreeMlaParams& p,
                                  cudaStream_t st) {
  cudaError_t e = set_func_attr_once(reinterpret_cast<const void*>(tree_mla_nvfp4_kernel),
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, t16::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  e = launch_ex(tree_mla_nvfp4_kernel, dim3(p.max_ctas), dim3(t16::THREADS), t16::SMEM_BYTES, st, true, 0u, qmap, rmap, p);
  return e != cudaSuccess ? e : launch_combine(p, st);
}

}  // namespace dsa
