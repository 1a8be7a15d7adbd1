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
#include "tree_mla.cuh"

namespace dsa {

// --------------------------------------------------------- plan and query terms
//
// Block 0 sums the tokens' tiles; the other blocks (FP8 latents) split the queries
// into the attention's e4m3 terms, one warp per head, three blocks of 32 heads a token.

constexpr int kPrepThreads = 1024;

__global__ void __launch_bounds__(kPrepThreads) tree_prep_kernel(BatchView b, TreeView tree, const __nv_bfloat16* q,
                                                                 uint8_t* terms, int64_t* starts, uint32_t* status) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.x > 0) {
    const int t = (blockIdx.x - 1) / 3, h = (blockIdx.x - 1) % 3 * 32 + warp;
    uint8_t* tok = terms + static_cast<int64_t>(t) * kQTokenBytes;
    q_head_to_terms(q + static_cast<int64_t>(t) * kMlaHeads * kLatDim, h, tok,
                    reinterpret_cast<int32_t*>(tok + kQTermBytes));
    return;
  }
  __shared__ int64_t wsum[kPrepThreads / 32];
  int64_t base = 0;
  for (int t0 = 0; t0 < b.T; t0 += kPrepThreads) {
    const int t = t0 + threadIdx.x;
    int64_t v = 0;
    if (t < b.T) {
      int req, pos, committed;
      if (load_tree_token(b, tree, t, status, req, pos, committed)) v = cdiv(pos + 1, kSelTile);
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
    for (int w = 0; w < kPrepThreads / 32; ++w) {
      if (w < warp) before += wsum[w];
      total += wsum[w];
    }
    if (t < b.T) starts[t] = base + before + x - v;
    base += total;
    __syncthreads();
  }
  if (threadIdx.x == 0) starts[b.T] = base;
}

cudaError_t launch_tree_prep(const BatchView& b, const TreeView& tree, const __nv_bfloat16* q, uint8_t* terms,
                             int64_t* starts, uint32_t* status, cudaStream_t st) {
  return launch_ex(tree_prep_kernel, dim3(terms ? 1 + 3 * b.T : 1), dim3(kPrepThreads), 0, st, false, 0u, b, tree, q,
                   terms, starts, status);
}

// The first token of share [g0, ...): every thread of the CTA searches.
__device__ __forceinline__ SegmentWalk make_walk(const TreeMlaParams& p, int* first_sh) {
  SegmentWalk w;
  const int64_t W = __ldcg(p.starts + p.b.T);
  w.starts = p.starts;
  w.T = p.b.T;
  w.whole = p.whole;
  w.cta = blockIdx.x;
  w.G = static_cast<int>(W < p.max_ctas ? W : p.max_ctas);
  w.g0 = w.g = w.g1 = 0;
  w.t = 0;
  if (p.whole) {
    w.G = p.max_ctas;
    w.t = blockIdx.x;
    return w;
  }
  if (static_cast<int>(blockIdx.x) < w.G) {
    w.g0 = w.g = share_begin(W, w.G, blockIdx.x);
    w.g1 = share_begin(W, w.G, blockIdx.x + 1);
    for (int t = threadIdx.x; t < w.T; t += blockDim.x)
      if (__ldcg(p.starts + t) <= w.g0 && w.g0 < __ldcg(p.starts + t + 1)) *first_sh = t;
  }
  __syncthreads();
  w.t = *first_sh;
  return w;
}

// -------------------------------------------- attention with converted latents
//
// One CTA per SM.  A tile's 128 latents are converted to the tensor cores' 16-bit
// operands on the way into shared memory, once per use:
//   S^T[token, head] = C[token, 0:576] . q[head, 0:576]      M=128, N=96, K=576  (bf16 x bf16)
//   O^T[dim, head]  += V^T[dim, token] . P^T[token, head]     M=128 (x4 dim blocks), N=96, K=128 (f16 x f16)
// TMEM: S^T in columns [0, 96), O^T blocks at 128 + 96 v (v = 0..3): 480 of 512.
// The layouts, the softmax across lanes and the sums of P by the tensor core are
// those of mla.cu; here a CTA walks many tiles and several tokens.
// Roles: warp 0 loads each token's query (96 x 576 bf16) once the one before has been
// used; warp 1 issues MMAs; warps 2..9 convert; warps 10..13 run the softmax; all 12
// math warps write a finished segment.
namespace tconv {
constexpr int QCHUNKS = kLatDim / 64;
constexpr int Q_SLOT = kMlaHeads * 128;
constexpr int OFF_Q = 0;
constexpr int RSLOTS = 4;
constexpr int RING_SLOT = 16384;
constexpr int OFF_RING = QCHUNKS * Q_SLOT;
constexpr int OFF_P = OFF_RING + RSLOTS * RING_SLOT;
constexpr int P_BYTES = 2 * 16 * 1024;
constexpr int OFF_ONES = OFF_P + P_BYTES;
constexpr int OFF_RED = OFF_ONES + 1024;          // 4 x 96 floats
constexpr int OFF_MUSE = OFF_RED + 4 * 96 * 4;
constexpr int OFF_ALPHA = OFF_MUSE + 96 * 4;
constexpr int OFF_INV = OFF_ALPHA + 96 * 4;
constexpr int OFF_LFIN = OFF_INV + 96 * 4;
constexpr int OFF_ROWOK = OFF_LFIN + 96 * 4;      // 2 x 128 bytes: position seen (by tile parity)
constexpr int OFF_BARS = OFF_ROWOK + 256;
constexpr int N_BARS = 20;
constexpr int OFF_MISC = OFF_BARS + N_BARS * 8;
constexpr int SMEM_BYTES = OFF_MISC + 64 + 1024;
constexpr int THREADS = 448;
constexpr int CONV_WARPS = 8;
constexpr int SOFT_WARP0 = 2 + CONV_WARPS;
constexpr int S_COL = 0;
constexpr int O_COL = 128;
constexpr float TAU = 8.0f;                       // log2 headroom before the running max moves
static_assert(OFF_RING % 1024 == 0 && OFF_P % 1024 == 0 && OFF_ONES % 1024 == 0, "align");
static_assert(OFF_MUSE % 16 == 0 && OFF_ALPHA % 16 == 0 && OFF_INV % 16 == 0, "vectors are read 16 bytes at a time");
static_assert(OFF_BARS % 8 == 0 && SMEM_BYTES <= 232448, "smem");
}  // namespace tconv

__device__ __forceinline__ uint8_t* align1024_tree(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~static_cast<uintptr_t>(1023));
}

// A failed (timed out) wait is the same for the whole warp.  A warp whose wait failed
// walks on through its tiles without touching operands or signalling barriers (a phase
// must not be completed twice), so the named barriers stay whole.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, Abort ab, bool ok) {
  return __all_sync(0xffffffffu, ok && mbar_wait_inline(bar, parity, ab));
}

// Head, in its group of 32, of column n of the group in the FP8 kernel's P and O.
__device__ __forceinline__ constexpr int head_of_column(int n) { return 8 * ((n >> 1) & 3) + 2 * (n >> 3) + (n & 1); }

// Writes 32 heads of one dim per lane: the segment's output (bf16) or its normalised
// partial (fp16: 11 significant bits, above the output's 8), both [96][512], as 64
// contiguous bytes per warp and head.  PERM: the columns hold heads by head_of_column.
template <bool PERM>
__device__ __forceinline__ void store_heads(const TreeMlaParams& p, const Segment& s, const uint32_t (&rr)[32],
                                            const float* inv, int h0, int dim) {
  float al[32];
  lds_f32x32(inv + h0, al);
  if (s.slot < 0) {
    __nv_bfloat16* o = p.out + (static_cast<int64_t>(s.t) * kMlaHeads + h0) * kVDim + dim;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      o[(PERM ? head_of_column(i) : i) * kVDim] = __float2bfloat16_rn(__uint_as_float(rr[i]) * al[i]);
  } else {
    __half* o = p.part_o + (static_cast<int64_t>(s.slot) * kMlaHeads + h0) * kVDim + dim;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      o[(PERM ? head_of_column(i) : i) * kVDim] = __float2half_rn(__uint_as_float(rr[i]) * al[i]);
  }
}

__global__ void __launch_bounds__(tconv::THREADS, 1)
    tree_mla_nvfp4_kernel(const __grid_constant__ CUtensorMap qmap, TreeMlaParams p) {
  using namespace tconv;
  constexpr int ROWB = 352;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024_tree(smem_raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BARS);
  uint64_t* q_full = bars + 0;
  uint64_t* rows_ready = bars + 1;
  uint64_t* ring_full = bars + 2;   // [RSLOTS]
  uint64_t* ring_empty = bars + 6;  // [RSLOTS]
  uint64_t* s_full = bars + 10;     // a tile's QK done
  uint64_t* s_free = bars + 11;
  uint64_t* p_full = bars + 12;
  uint64_t* o_done = bars + 13;     // a tile's PV done
  uint64_t* drain = bars + 14;
  uint64_t* sum_done = bars + 15;
  uint64_t* o_free = bars + 16;     // a segment's O has been read
  uint64_t* q_done = bars + 17;     // a segment's QKs are done
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + OFF_MISC);
  int* abortf = reinterpret_cast<int*>(smem + OFF_MISC + 8);
  int* rescale_sh = reinterpret_cast<int*>(smem + OFF_MISC + 16);
  int* first_sh = reinterpret_cast<int*>(smem + OFF_MISC + 24);
  float* red = reinterpret_cast<float*>(smem + OFF_RED);
  float* m_use = reinterpret_cast<float*>(smem + OFF_MUSE);
  float* alpha_sh = reinterpret_cast<float*>(smem + OFF_ALPHA);
  float* inv_sh = reinterpret_cast<float*>(smem + OFF_INV);
  float* l_fin = reinterpret_cast<float*>(smem + OFF_LFIN);
  uint8_t* rowok = smem + OFF_ROWOK;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(rows_ready, CONV_WARPS);
    for (int i = 0; i < RSLOTS; ++i) {
      mbar_init(&ring_full[i], CONV_WARPS);
      mbar_init(&ring_empty[i], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(s_free, 4);
    mbar_init(p_full, 4);
    mbar_init(o_done, 1);
    mbar_init(drain, 1);
    mbar_init(sum_done, 1);
    mbar_init(o_free, 12);
    mbar_init(q_done, 1);
    *abortf = 0;
    *first_sh = 0;
    fence_mbar_init();
    prefetch_tensormap(&qmap);
  }
  for (int i = threadIdx.x; i < 256; i += THREADS) reinterpret_cast<uint32_t*>(smem + OFF_ONES)[i] = 0x3C003C00u;
  fence_proxy_async_smem();
  if (warp == 1) tmem_alloc(tslot, 512);
  grid_dep_wait();   // the plan
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  SegmentWalk walk = make_walk(p, first_sh);
  const uint32_t tmem = *tslot;
  const Abort ab{abortf, p.status};
  Segment s;

  if (warp == 0) {
    // --------------------------------------------------------- query loader
    if (lane == 0) {
      bool ok = true;
      int seg = 0;
      for (; ok && walk.next(s); ++seg) {
        if (seg > 0 && !(ok = mbar_wait(q_done, (seg - 1) & 1, ab))) break;
        mbar_arrive_expect_tx(q_full, QCHUNKS * Q_SLOT);
        for (int kc = 0; kc < QCHUNKS; ++kc)
          tma_load_2d(smem + OFF_Q + kc * Q_SLOT, &qmap, q_full, kc * 64, s.t * kMlaHeads);
      }
      if (seg > 0) drain_wait(q_full, (seg - 1) & 1);   // no copy into shared memory outlives the CTA
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      const uint32_t idesc_qk = make_idesc(1, 1, false, false, 128, kMlaHeads);
      const uint32_t idesc_pv = make_idesc(0, 0, true, true, 128, kMlaHeads);
      const uint32_t idesc_sum = make_idesc(0, 0, false, true, 128, kMlaHeads);
      const uint64_t d_c = make_sdesc_sw128(smem_u32(smem + OFF_RING), 16, 1024);      // C chunk, K-major
      const uint64_t d_q = make_sdesc_sw128(smem_u32(smem + OFF_Q), 16, 1024);         // q chunk, K-major
      const uint64_t d_v = make_sdesc_sw128(smem_u32(smem + OFF_RING), 8192, 1024);    // V^T, MN-major
      const uint64_t d_p = make_sdesc_sw128(smem_u32(smem + OFF_P), 16384, 1024);      // P^T, MN-major
      const uint64_t d_one = make_sdesc_sw128(smem_u32(smem + OFF_ONES), 16, 0);       // the ones atom, repeated
      constexpr uint64_t kSlot = RING_SLOT >> 4;
      int fc = 0, it = 0;
      bool ok = true;
      for (int seg = 0; ok && walk.next(s); ++seg) {
        ok = mbar_wait(q_full, seg & 1, ab);
        for (int j = s.j0; ok && j < s.j1; ++j, ++it) {
          if (it > 0 && !(ok = mbar_wait(s_free, (it - 1) & 1, ab))) break;
#pragma unroll 1
          for (int kc = 0; kc < QCHUNKS; ++kc, ++fc) {
            const int slot = fc % RSLOTS;
            if (!(ok = mbar_wait_inline(&ring_full[slot], (fc / RSLOTS) & 1, ab))) break;
            tc_fence_after();
            const uint64_t a = d_c + slot * kSlot;
            const uint64_t b = d_q + kc * (Q_SLOT >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) mma_f16(tmem + S_COL, a + 2 * kk, b + 2 * kk, idesc_qk, (kc | kk) ? 1u : 0u);
            tc_commit(&ring_empty[slot]);
          }
          if (!ok) break;
          tc_commit(s_full);
          if (j == s.j1 - 1) tc_commit(q_done);
          if (!(ok = mbar_wait(p_full, it & 1, ab))) break;
          tc_fence_after();
#pragma unroll
          for (int kh = 0; kh < 2; ++kh)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_f16(tmem + S_COL, d_one + 2 * k, d_p + (kh * 8 + k * 2) * 64, idesc_sum, (kh | k) ? 1u : 0u);
          tc_commit(sum_done);
          const bool first = j == s.j0;
          if (first && seg > 0 && !(ok = mbar_wait(o_free, (seg - 1) & 1, ab))) break;
          tc_fence_after();
#pragma unroll 1
          for (int f = 0; f < 8; ++f) {   // half-block f: dims [128 (f / 2), +128), tokens [64 (f % 2), +64)
            if (!(ok = mbar_wait_inline(&ring_full[fc % RSLOTS], (fc / RSLOTS) & 1, ab))) break;
            const uint64_t a = d_v + (fc % RSLOTS) * kSlot;
            const int kh = f & 1;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_f16(tmem + O_COL + 96 * (f >> 1), a + 128 * k, d_p + (kh * 8 + k * 2) * 64, idesc_pv,
                      (!first || kh > 0 || k > 0) ? 1u : 0u);
            tc_commit(&ring_empty[fc % RSLOTS]);
            ++fc;
          }
          if (!ok) break;
          tc_commit(o_done);
        }
      }
      if (!ok) {
        tc_commit(drain);
        drain_wait(drain, 0);
      }
    }
  } else {
    const bool conv = warp < SOFT_WARP0;
    const int mw = warp - 2;                        // 0..11
    const int quarter = warp & 3;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    int fc = 0, it = 0;
    bool ok = true;
    for (int seg = 0; walk.next(s); ++seg) {
      int req, pos, base;
      load_tree_token(p.b, p.tree, s.t, p.status, req, pos, base);
      if (conv) {
        // ----------------------------------------------------- converters (2..9)
        const int ct = threadIdx.x - 64;            // 0..255
        const int row = ct >> 1, hf = ct & 1;       // this thread's half row: dims [64 kc + 32 hf, +32) of each chunk
        const int vg = (ct >> 5) >> 2;              // V half-block of this warp's rows: tokens [64 vg, +64)
        const int tl = row & 63;
        const int bsm = p.pool.bs - 1;
        const int32_t* btrow = p.b.bt + static_cast<int64_t>(req) * p.b.bt_stride;
        const uint32_t* mrow = p.tree.mask + static_cast<int64_t>(s.t) * p.tree.words;
        for (int j = s.j0; j < s.j1; ++j, ++it) {
          const int sv = j * kSelTile + row;
          const uint8_t* src = nullptr;
          if (sv <= pos && tree_sees(mrow, p.tree.words, base, sv)) {
            const int prow = __ldg(btrow + (sv >> p.pool.log2_bs));
            if (prow < 0 || prow >= p.pool.num_rows) {
              if (hf == 0) atomicOr(p.status, DEV_BAD_BLOCK);
            } else {
              src = p.pool.pool + static_cast<int64_t>(prow) * p.pool.row_stride + p.pool.lat_off +
                    static_cast<int64_t>(sv & bsm) * ROWB;
            }
          }
          // The flags of tile it - 2 have been used: this warp's last V fills of tile it - 1 waited
          // for that tile's PV to start, which follows its softmax.
          if (hf == 0) rowok[(it & 1) * kSelTile + row] = src != nullptr;
          __syncwarp();
          if (ok && lane == 0) mbar_arrive(rows_ready);
          LatPiece cb[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) cb[u] = load_piece<true>(src, u, hf);
#pragma unroll 1
          for (int kb = 0; kb < QCHUNKS; kb += 4) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int kc = kb + u;
              if (kc >= QCHUNKS) break;
              const int slot = fc % RSLOTS;
              if (fc >= RSLOTS) ok = warp_wait(&ring_empty[slot], ((fc / RSLOTS) - 1) & 1, ab, ok);
              if (ok) {
                uint8_t* dst = smem + OFF_RING + slot * RING_SLOT + (row >> 3) * 1024;
#pragma unroll
                for (int q2 = 0; q2 < 2; ++q2) {
                  const int q4 = 2 * hf + q2;
                  uint32_t o[8];
                  piece_to_bf16<true>(cb[u], q2, o);
                  sts128(dst + sw128_off(row & 7, 2 * q4), o);
                  sts128(dst + sw128_off(row & 7, 2 * q4 + 1), o + 4);
                }
                fence_proxy_async_smem();
              }
              __syncwarp();
              if (ok && lane == 0) mbar_arrive(&ring_full[slot]);
              ++fc;
              if (kc + 4 < QCHUNKS) cb[u] = load_piece<true>(src, kc + 4, hf);
            }
          }
          // V half-blocks: the warps of rows 0..63 fill the even ring fills, the others the odd ones
#pragma unroll 1
          for (int v = 0; v < 4; ++v) {
            LatPiece c0 = load_piece<true>(src, 2 * v, hf), c1 = load_piece<true>(src, 2 * v + 1, hf);
            const int myfc = fc + 2 * v + vg;
            const int slot = myfc % RSLOTS;
            if (myfc >= RSLOTS) ok = warp_wait(&ring_empty[slot], ((myfc / RSLOTS) - 1) & 1, ab, ok);
            if (ok) {
              uint8_t* dst = smem + OFF_RING + slot * RING_SLOT + (tl >> 3) * 1024;
#pragma unroll
              for (int a = 0; a < 2; ++a) {
#pragma unroll
                for (int q2 = 0; q2 < 2; ++q2) {
                  const int q4 = 2 * hf + q2;
                  uint32_t o[8];
                  piece_to_f16<true>(a ? c1 : c0, q2, o);
                  sts128(dst + a * 8192 + sw128_off(tl & 7, 2 * q4), o);
                  sts128(dst + a * 8192 + sw128_off(tl & 7, 2 * q4 + 1), o + 4);
                }
              }
              fence_proxy_async_smem();
            }
            __syncwarp();
            if (ok && lane == 0) mbar_arrive_cnt(&ring_full[slot], 2);   // four warps complete a fill
          }
          fc += 8;
        }
      } else {
        // ---------------------------------------------- softmax warps (10..13)
        const int r = quarter * 32 + lane;          // token lane within the tile
        float m_run[3] = {-INFINITY, -INFINITY, -INFINITY};   // per head (lane + 32 i), log2 units
        float l_run[3] = {0.f, 0.f, 0.f};                      // first softmax warp only
        float alpha_r[3] = {1.f, 1.f, 1.f};
        for (int j = s.j0; j < s.j1; ++j, ++it) {
          ok = warp_wait(s_full, it & 1, ab, ok);
          ok = warp_wait(rows_ready, it & 1, ab, ok);
          tc_fence_after();
          const bool valid = rowok[(it & 1) * kSelTile + r] != 0;
#pragma unroll 1
          for (int c = 0; c < 3; ++c) {
            uint32_t rr[32];
            DSA_TMEM_LD32(tmem + S_COL + 32 * c + lane_off, rr);
            tmem_wait_ld();
            float mine = -INFINITY;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float m = warp_max_f32(valid ? __uint_as_float(rr[i]) * p.scale_log2 : -INFINITY);
              if (lane == i) mine = m;
            }
            red[quarter * kMlaHeads + 32 * c + lane] = mine;
          }
          named_bar_sync(1, 128);
          if (warp == SOFT_WARP0) {
            bool moved = false;
#pragma unroll
            for (int i = 0; i < 3; ++i) {
              const int h = lane + 32 * i;
              const float tm =
                  fmaxf(fmaxf(red[h], red[kMlaHeads + h]), fmaxf(red[2 * kMlaHeads + h], red[3 * kMlaHeads + h]));
              const float mo = m_run[i];
              const float mn = (tm > mo + TAU) ? tm : mo;
              alpha_r[i] = (mn == mo) ? 1.f : exp2f(mo - mn);
              m_run[i] = mn;
              m_use[h] = mn == -INFINITY ? 0.f : mn;
              alpha_sh[h] = alpha_r[i];
              moved |= (mn != mo);
            }
            moved = __any_sync(0xffffffffu, moved);
            if (lane == 0) *rescale_sh = (moved && j > s.j0) ? 1 : 0;
          }
          named_bar_sync(1, 128);
          const bool any_rescale = *reinterpret_cast<volatile int*>(rescale_sh) != 0;
          // PV of the tile before must be done before P is overwritten or O rescaled
          if (it > 0) ok = warp_wait(o_done, (it - 1) & 1, ab, ok);
          if (any_rescale && ok) {
            tc_fence_after();
#pragma unroll 1
            for (int v = 0; v < 4; ++v) {
#pragma unroll 1
              for (int c = 0; c < 3; ++c) {
                uint32_t rr[32];
                const uint32_t ta = tmem + O_COL + 96 * v + 32 * c + lane_off;
                DSA_TMEM_LD32(ta, rr);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) rr[i] = __float_as_uint(__uint_as_float(rr[i]) * alpha_sh[32 * c + i]);
                DSA_TMEM_ST32(ta, rr);
              }
            }
            tmem_wait_st();
          }
          {
            uint8_t* prow = smem + OFF_P + (r >> 3) * 1024;
#pragma unroll 1
            for (int c = 0; c < 3; ++c) {
              uint32_t rr[32];
              DSA_TMEM_LD32(tmem + S_COL + 32 * c + lane_off, rr);
              tmem_wait_ld();
              float pv[32];
              lds_f32x32(m_use + 32 * c, pv);
#pragma unroll
              for (int i = 0; i < 32; ++i)
                pv[i] = valid ? ex2_fast(__uint_as_float(rr[i]) * p.scale_log2 - pv[i]) : 0.f;
#pragma unroll
              for (int cc4 = 0; cc4 < 4; ++cc4) {
                uint32_t o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const __half2 hp = __floats2half2_rn(pv[8 * cc4 + 2 * i], pv[8 * cc4 + 2 * i + 1]);
                  o[i] = *reinterpret_cast<const uint32_t*>(&hp);
                }
                const int chunk = 4 * c + cc4;
                sts128(prow + (chunk >> 3) * 16384 + sw128_off(r & 7, chunk & 7), o);
              }
            }
          }
          fence_proxy_async_smem();
          tc_fence_before();
          __syncwarp();
          if (ok && lane == 0) {
            mbar_arrive(p_full);
            if (warp != SOFT_WARP0) mbar_arrive(s_free);
          }
          if (warp == SOFT_WARP0) {
            ok = warp_wait(sum_done, it & 1, ab, ok);
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < 3; ++c) {
              float ls = 0.f;
#pragma unroll 1
              for (int q = 0; q < 4; ++q) {
                uint32_t rr[8];
                DSA_TMEM_LD8(tmem + S_COL + 32 * c + 8 * q + lane_off, rr);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  if (lane == 8 * q + i) ls = __uint_as_float(rr[i]);
              }
              l_run[c] = l_run[c] * alpha_r[c] + ls;
            }
            tc_fence_before();
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(s_free);
          }
        }
        if (warp == SOFT_WARP0) {
#pragma unroll
          for (int i = 0; i < 3; ++i) {
            l_fin[lane + 32 * i] = l_run[i];
            inv_sh[lane + 32 * i] = l_run[i] == 0.f ? 0.f : 1.f / l_run[i];   // nothing seen: output 0
          }
        }
      }
      // ---- the segment's result, all 12 math warps: TMEM (thread = dim) -> global
      ok = warp_wait(o_done, (it - 1) & 1, ab, ok);
      named_bar_sync(2, 384);
      tc_fence_after();
      if (ok) {
        const int which = mw >> 2;                    // 0..2: the three warps of this lane quarter
#pragma unroll 1
        for (int pc = which; pc < 12; pc += 3) {      // (dim block v, head chunk c) pairs
          const int v = pc / 3, c = pc % 3;
          uint32_t rr[32];
          DSA_TMEM_LD32(tmem + O_COL + 96 * v + 32 * c + lane_off, rr);
          tmem_wait_ld();
          store_heads<false>(p, s, rr, inv_sh, 32 * c, v * 128 + quarter * 32 + lane);
        }
        const int h = mw * 32 + lane;
        if (h < kMlaHeads) {
          const float l = l_fin[h];
          if (s.slot >= 0) p.part_ml[static_cast<int64_t>(s.slot) * kMlaHeads + h] = make_float2(m_use[h], l);
          else if (p.lse) p.lse[static_cast<int64_t>(s.t) * kMlaHeads + h] = (m_use[h] + log2f(l)) * 0.69314718055994531f;
        }
      }
      tc_fence_before();
      named_bar_sync(2, 384);   // sums and maxima are read before the next segment writes them
      if (ok && lane == 0) mbar_arrive(o_free);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------- attention with FP8 latents
//
// No conversion: e4m3 is the tensor core's operand type, and one copy of the tile in
// shared memory, brought by TMA, is the A operand of both products (K-major for the
// scores, MN-major for the values).
//   S^T[token, head] = sum_k c[token, k] . q_term[head, k]      M=128, N=96, K=1152
//   O^T[dim, head] += V^T[dim, token] . P_term^T[token, head]   M=128 (x4 dim blocks), N=96, K=3 x 128
// q arrives as two e4m3 terms (mla_q.cuh, exact).  P is the sum of three e5m2 terms,
// each the nearest to what the ones before it left: off by at most 2^-9 of it, half the
// error of a bf16 P.  e5m2 is the upper byte of an fp16, so a term is an addition, a mask
// and a subtraction on two weights at a time, and its range (2^-16 .. 2^15 with the
// reference at 2^11) keeps weights down to 2^-27 of the largest, which a million
// positions beside one heavy one need; e4m3 terms would lose those below 2^-18.  The sum
// of the weights is of the unrounded ones, in fp32.
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
constexpr int OFF_BARS = OFF_INV + 96 * 4;
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
  int* first_sh = reinterpret_cast<int*>(smem + OFF_MISC + 16);
  float* red = reinterpret_cast<float*>(smem + OFF_REDM);
  float* sh_sh = reinterpret_cast<float*>(smem + OFF_SH);
  float* alpha_sh = reinterpret_cast<float*>(smem + OFF_ALPHA);
  float* inv_sh = reinterpret_cast<float*>(smem + OFF_INV);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 15; ++i) mbar_init(&bars[i], 1);
    for (int i = 0; i < 3; ++i) mbar_init(&p_full[i], MATH_WARPS);
    *abortf = 0;
    *first_sh = 0;
    fence_mbar_init();
    prefetch_tensormap(&lmap);
    prefetch_tensormap(&tmap);
  }
  if (warp == 0) tmem_alloc(tslot, 512);
  grid_dep_wait();   // the plan and the query terms
  grid_dep_launch();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  SegmentWalk walk = make_walk(p, first_sh);
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
      int req, pos, base;
      load_tree_token(p.b, p.tree, s.t, p.status, req, pos, base);
      const int32_t* btrow = p.b.bt + static_cast<int64_t>(req) * p.b.bt_stride;
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
      int row = page(s.j0);
      prefetch(s.j0, row);
      if (seg > 0) ok = warp_wait(q_done, (seg - 1) & 1, ab, ok);
      if (!ok) break;
      q_issued = seg & 1;
      if (lane == 0) {
        const uint8_t* src = p.q_terms + static_cast<int64_t>(s.t) * kQTokenBytes;
        mbar_arrive_expect_tx(q_full, kQTokenBytes);
        for (int c = 0; c < kQChunks; ++c) bulk_load(smem + OFF_Q + c * QCHUNK, src + c * QCHUNK, QCHUNK, q_full);
        bulk_load(smem + OFF_QEXP, src + kQTermBytes, kMlaHeads * 4, q_full);
      }
      for (int j = s.j0; ok && j < s.j1; ++j, ++it) {
        const int c1 = (j * kSelTile + lane * box) & (p.pool.bs - 1);
        const int n = __popc(__ballot_sync(0xffffffffu, row >= 0));
        const int next = j + 1 < s.j1 ? page(j + 1) : -1;
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
        prefetch(j + 1, row);
      }
    }
    // after a failed wait: no copy into shared memory outlives the CTA (a barrier whose copy
    // was not issued in this round keeps its earlier phase; the wait is bounded)
    if (!ok && lane == 0) {
      if (q_issued >= 0) drain_wait(q_full, q_issued);
      drain_wait(tail_full, it & 1);
      for (int k = 0; k < 4; ++k) drain_wait(&lat_full[k], it & 1);
    }
  } else if (warp == MMA_WARP) {
    // ------------------------------------------------------------ MMA issuer
    const bool leader = elect_one();
    const uint32_t idesc_qk = make_idesc(0, 0, false, false, 128, kMlaHeads);
    const uint32_t idesc_pv = make_idesc(0, 1, true, true, 128, kMlaHeads);
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
      for (int j = s.j0; ok && j < s.j1; ++j, ++it) {
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
        const uint32_t acc = j > s.j0 ? 1u : 0u;
        const bool last = j == s.j1 - 1;
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
      int req, pos, base;
      load_tree_token(p.b, p.tree, s.t, p.status, req, pos, base);
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
      for (int j = s.j0; j < s.j1; ++j, ++it) {
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
        float mx = logits(0);
        tmem_wait_ld();
        mx = fmaxf(mx, logits(2));
        if (named_bar_any(1, MATH, mx > SHIFT + TAU)) {
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
            if (m > m_ref + TAU) {
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
          if (j > s.j0 && ok) {
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
      if (ok) {
#pragma unroll 1
        for (int v = 0; v < 4; ++v) {
          uint32_t rr[32];
          DSA_TMEM_LD32(tmem + O_COL + 96 * v + 32 * g + lane_off, rr);
          tmem_wait_ld();
          store_heads<true>(p, s, rr, inv_sh, 32 * g, v * 128 + 32 * quarter + lane);
        }
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// Merge of a token's partials: out = sum_j w_j o_j, w_j = l_j 2^(m_j - M) / sum.
// Grid (96 heads, T); a block's 256 threads are 64 groups of 8 dims times 4 interleaved
// quarters of the partials.  Tokens with one segment have their output already.
constexpr int kTreeCombThreads = 256;
__global__ void __launch_bounds__(kTreeCombThreads) tree_combine_kernel(TreeMlaParams p) {
  __shared__ float acc_sh[3][64][9];
  const int h = blockIdx.x, t = blockIdx.y;
  grid_dep_wait();
  const int64_t W = __ldcg(p.starts + p.b.T);
  const int64_t u0 = __ldcg(p.starts + t), u1 = __ldcg(p.starts + t + 1);
  if (u1 <= u0) return;
  const int G = static_cast<int>(W < p.max_ctas ? W : p.max_ctas);
  const int c0 = share_of(W, G, u0), c1 = share_of(W, G, u1 - 1);
  if (c0 == c1) return;
  const int first = 2 * c0 + (share_begin(W, G, c0) < u0 ? 1 : 0);
  const int n = c1 - c0 + 1;
  auto slot = [&](int j) { return j == 0 ? first : 2 * (c0 + j); };
  const int d8 = threadIdx.x & 63, part = threadIdx.x >> 6;
  float M = -INFINITY;
  for (int j = 0; j < n; ++j) {
    const float2 ml = __ldcg(p.part_ml + static_cast<int64_t>(slot(j)) * kMlaHeads + h);
    if (ml.y != 0.f) M = fmaxf(M, ml.x);
  }
  float Ls = 0.f;
  float acc[8] = {};
#pragma unroll 4
  for (int j = part; j < n; j += 4) {
    const int64_t sl = static_cast<int64_t>(slot(j)) * kMlaHeads + h;
    const float2 ml = __ldcg(p.part_ml + sl);
    const uint4 v = __ldcg(reinterpret_cast<const uint4*>(p.part_o + sl * kVDim) + d8);
    if (ml.y == 0.f) continue;
    const float w = exp2f(ml.x - M) * ml.y;
    Ls += w;
    const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w4[e]));
      acc[2 * e] = fmaf(w, f.x, acc[2 * e]);
      acc[2 * e + 1] = fmaf(w, f.y, acc[2 * e + 1]);
    }
  }
  if (part > 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) acc_sh[part - 1][d8][e] = acc[e];
    acc_sh[part - 1][d8][8] = Ls;
  }
  __syncthreads();
  if (part > 0) return;
  for (int q = 0; q < 3; ++q) {
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] += acc_sh[q][d8][e];
    Ls += acc_sh[q][d8][8];
  }
  const float inv = Ls == 0.f ? 0.f : 1.f / Ls;
  __nv_bfloat162 o[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) o[e] = __floats2bfloat162_rn(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  __nv_bfloat16* dst = p.out + (static_cast<int64_t>(t) * kMlaHeads + h) * kVDim + 8 * d8;
  *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(o);
  if (d8 == 0 && p.lse) p.lse[static_cast<int64_t>(t) * kMlaHeads + h] = (M + log2f(Ls)) * 0.69314718055994531f;
}

static cudaError_t launch_combine(const TreeMlaParams& p, cudaStream_t st) {
  if (p.whole) return cudaSuccess;
  return launch_ex(tree_combine_kernel, dim3(kMlaHeads, p.b.T), dim3(kTreeCombThreads), 0, st, true, 0u, p);
}

cudaError_t launch_tree_mla_fp8(const CUtensorMap& lmap, const CUtensorMap& tmap, const TreeMlaParams& p,
                                cudaStream_t st) {
  cudaError_t e = set_func_attr_once(reinterpret_cast<const void*>(tree_mla_fp8_kernel),
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, t8::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  e = launch_ex(tree_mla_fp8_kernel, dim3(p.max_ctas), dim3(t8::THREADS), t8::SMEM_BYTES, st, true, 0u, lmap, tmap, p);
  return e != cudaSuccess ? e : launch_combine(p, st);
}

cudaError_t launch_tree_mla_nvfp4(const CUtensorMap& qmap, const TreeMlaParams& p, cudaStream_t st) {
  cudaError_t e = set_func_attr_once(reinterpret_cast<const void*>(tree_mla_nvfp4_kernel),
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, tconv::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  e = launch_ex(tree_mla_nvfp4_kernel, dim3(p.max_ctas), dim3(tconv::THREADS), tconv::SMEM_BYTES, st, true, 0u, qmap, p);
  return e != cudaSuccess ? e : launch_combine(p, st);
}

}  // namespace dsa
