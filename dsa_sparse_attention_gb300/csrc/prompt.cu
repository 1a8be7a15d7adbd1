// prompt.cu — attention of packed sequences with the heads' own keys and values
// (dsa_prompt_attn).
//
//   logit(i, s) = scale * (q_i . [k_s | k_shared_s]),  out_i = sum_s softmax(logit)(s) v_s
//
// over the keys s of the query's sequence (causal: s <= i + lk - lq), 2 (2 D + E) operations
// per pair and head.  One CTA takes two tiles of 128 query rows of one key head and walks the
// keys 128 at a time; a row is a (token, head of the group), so grouped heads fill a tile with
// fewer tokens and each key is read once for all of them.  Both products run on the tensor
// cores (tcgen05, M = 128 rows): S = Q.K^T into TMEM, the softmax in registers (a thread owns
// a row, so no exchange between lanes), P rounded to the inputs' type back into TMEM over S's
// own columns, O += P.V with P as the TMEM operand.  While one tile's softmax runs, the
// tensor core works on the other's products.  TMEM is full: two S of 128 columns, two O of D.
//
// The softmax keeps a reference per row that moves only when a logit exceeds it by 2^8 (the
// sums and O are then scaled); a weight is at most 2^8 (bf16) or 2^15 (fp16, whose weights
// start from 2^7 to keep more of what is small), sums are fp32 of the unrounded weights.
#include <cuda_runtime.h>

#include "../../include/dsa.h"
#include "prompt.cuh"
#include "ptx_prompt.cuh"

namespace dsa {

namespace prompt {
constexpr int CHUNK = 16384;          // 128 rows x 64 values of 16 bits
constexpr int SOFTMAX_WARPS = 8;      // four per query tile
constexpr int MMA_WARP = 8, LOAD_WARP = 9, WARPS = 12;
constexpr int THREADS = WARPS * 32;
constexpr int MISC = 1024;            // barriers and scalars
constexpr int SMEM_MAX = 232448;
constexpr float GROW = 8.f;           // log2 units a logit may exceed the reference by

template <int D, int E>
struct Shape {
  static constexpr int NQK = (D + E) / 64;   // chunks of a query tile and of 128 keys: [128][64]
  static constexpr int NV = D / 64;          // chunks of 128 values: D = 128 [64 keys][128], D = 64 [128 keys][64]
  static constexpr int Q_BYTES = 2 * NQK * CHUNK;
  static constexpr int RING = (SMEM_MAX - 1024 - MISC - Q_BYTES) / CHUNK < 12
                                  ? (SMEM_MAX - 1024 - MISC - Q_BYTES) / CHUNK : 12;
  static constexpr int SMEM = 1024 + Q_BYTES + RING * CHUNK + MISC;
  static_assert(RING >= NQK + NV + 1, "the values of a tile and the keys of the next are in use at a time");
};

// One CTA's work: two tiles of query rows of one key head over a range of one sequence's keys.
struct Item {
  int head;            // key head
  int t0;              // first token of tile 0, within the sequence
  int lq, lk;
  int64_t q0, k0;      // packed places of the sequence's first query and key
  int part, beg, end;  // keys [beg, end) of the sequence are in this part
  bool any;
};
}  // namespace prompt

// Lengths of sequence r; nothing to do (false) where the arrays break their rules.
__device__ __forceinline__ bool prompt_seq(const PromptParams& p, int r, int& q0, int& lq, int& k0, int& lk) {
  q0 = __ldg(p.cu_q + r);
  k0 = __ldg(p.cu_k + r);
  const int q1 = __ldg(p.cu_q + r + 1), k1 = __ldg(p.cu_k + r + 1);
  lq = q1 - q0;
  lk = k1 - k0;
  if (q0 < 0 || k0 < 0 || q1 < q0 || k1 < k0 || q1 > p.total_q || k1 > p.total_k || lq > p.max_q || lk > p.max_k) {
    atomicOr(p.status, DEV_BAD_BATCH);
    lq = lk = 0;
    return false;
  }
  return true;
}

// The CTA's item: sequences in order, of each its key heads, of each head its tile pairs, the
// last (the longest, causally) first, and the parts of the keys.  Every thread sums the pairs
// of a run of sequences; the thread whose run holds the CTA's number writes the item.
__device__ __forceinline__ void find_item(const PromptParams& p, prompt::Item* item, int64_t* totals) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.B + prompt::THREADS - 1) / prompt::THREADS;
  const int r0 = min(p.B, tid * per), r1 = min(p.B, r0 + per);
  const int pair = 2 * p.tile_toks;
  int64_t n = 0;
  int q0, lq, k0, lk;
  for (int r = r0; r < r1; ++r) {
    prompt_seq(p, r, q0, lq, k0, lk);
    n += (lq + pair - 1) / pair;
  }
  int64_t incl = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) totals[warp] = incl;
  if (tid == 0) item->any = false;
  __syncthreads();
  int64_t before = incl - n;
#pragma unroll
  for (int w = 0; w < prompt::WARPS; ++w)
    if (w < warp) before += totals[w];
  const int64_t each = static_cast<int64_t>(p.kv_heads) * p.nparts;   // items of a pair of tiles
  const int64_t me = blockIdx.x;
  if (me >= before * each && me < (before + n) * each) {
    int64_t at = me - before * each;
    for (int r = r0; r < r1; ++r) {
      prompt_seq(p, r, q0, lq, k0, lk);
      const int64_t pairs = (lq + pair - 1) / pair;
      if (at < pairs * each) {
        item->part = static_cast<int>(at % p.nparts);
        at /= p.nparts;
        item->t0 = static_cast<int>(pairs - 1 - at % pairs) * pair;
        item->head = static_cast<int>(at / pairs);
        item->lq = lq;
        item->lk = lk;
        item->q0 = q0;
        item->k0 = k0;
        item->beg = static_cast<int>(min(static_cast<int64_t>(lk), static_cast<int64_t>(item->part) * p.part_keys));
        item->end = p.nparts > 1 ? static_cast<int>(min(static_cast<int64_t>(lk), static_cast<int64_t>(item->beg) + p.part_keys)) : lk;
        item->any = true;
        break;
      }
      at -= pairs * each;
    }
  }
  __syncthreads();
}

__device__ __forceinline__ uint32_t pack16(float lo, float hi, bool fp16) {
  if (fp16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float2 unpack16(uint32_t v, bool fp16) {
  if (fp16) return __half22float2(*reinterpret_cast<const __half2*>(&v));
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}

// Weights of an earlier result and of the new one, and the joined log-sum-exp, all in natural
// logarithms.  Two empty results join to an empty one.
__device__ __forceinline__ float join_lse(float a, float b, float& wa, float& wb) {
  const float m = fmaxf(a, b);
  if (m == -INFINITY) {
    wa = wb = 0.f;
    return -INFINITY;
  }
  wa = exp2f((a - m) * 1.4426950408889634f);
  wb = exp2f((b - m) * 1.4426950408889634f);
  const float sum = wa + wb;
  wa /= sum;
  wb /= sum;
  return m + logf(sum);
}

template <int D, int E, bool FP16>
__global__ void __launch_bounds__(prompt::THREADS, 1)
    prompt_attn_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap smap, const __grid_constant__ CUtensorMap vmap,
                       const PromptParams p) {
  using namespace prompt;
  using S = Shape<D, E>;
  constexpr int NQK = S::NQK, NV = S::NV, RING = S::RING, PER = NQK + NV;
  extern __shared__ uint8_t psm_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(psm_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* qs = smem;                                   // [2][NQK] chunks
  uint8_t* ring = smem + S::Q_BYTES;                    // [RING] chunks
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring + RING * CHUNK);
  uint64_t* full = bars;                                // [RING] chunk landed
  uint64_t* empty = bars + RING;                        // [RING] its MMAs are done
  uint64_t* q_full = bars + 2 * RING;                   // [2] query tile landed
  uint64_t* s_full = q_full + 2;                        // [2] S of a tile done, and with it every MMA before; then O
  uint64_t* p_full = s_full + 2;                        // [2] P written (four warps)
  uint64_t* drain = p_full + 2;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(drain + 1);
  int* abortf = reinterpret_cast<int*>(tslot + 1);
  Item* item = reinterpret_cast<Item*>(bars + 40);
  int64_t* totals = reinterpret_cast<int64_t*>(bars + 60);
  static_assert(2 * 12 + 9 <= 40 && sizeof(Item) <= 160 && (60 + WARPS) * 8 <= MISC, "shared scalars");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < RING; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + i, 1);
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 4);
    }
    mbar_init(drain, 1);
    *abortf = 0;
    fence_mbar_init();
  }
  grid_dep_wait();
  find_item(p, item, totals);
  const Item it = *item;
  if (!it.any) return;
  // keys of each tile: up to the last that its last token sees
  int n[2], first_tok[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    first_tok[i] = it.t0 + i * p.tile_toks;
    const int last = min(first_tok[i] + p.tile_toks, it.lq) - 1;
    int64_t vis = it.lk;
    if (p.causal) vis = min(vis, static_cast<int64_t>(last) + 1 + it.lk - it.lq);
    const int64_t end = min(static_cast<int64_t>(it.end), vis);
    n[i] = first_tok[i] < it.lq && end > it.beg ? static_cast<int>((end - it.beg + kPromptKeys - 1) / kPromptKeys) : 0;
  }
  const int nmax = max(n[0], n[1]);
  if (p.nparts > 1 && nmax == 0) return;   // the merge does not look for this part
  if (warp == MMA_WARP) tmem_alloc(tslot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  const Abort ab{abortf, p.status};
  constexpr uint32_t S_COL = 0, O_COL = 256;   // S (and P) of tile i at 128 i, O at 256 + 128 i

  if (warp == LOAD_WARP) {
    // ---------------------------------------------------------------- loads
    const bool leader = elect_one();
    bool ok = true;
    int c = 0;   // chunks issued
    const int q_bytes = p.tile_toks * p.group * 128;
    auto load_q = [&](int i) {
      if (n[i] == 0 || !leader) return;
      mbar_arrive_expect_tx(q_full + i, NQK * q_bytes);
      for (int k = 0; k < NQK; ++k)
        tma_load_4d(qs + (i * NQK + k) * CHUNK, &qmap, q_full + i, 64 * k, 0, it.head,
                    static_cast<int>(it.q0) + first_tok[i]);
    };
    auto slot = [&]() {   // the next chunk's place, once it is free
      const int s = c % RING;
      if (c >= RING) ok = ok && __all_sync(0xffffffffu, mbar_wait_inline(empty + s, (c / RING - 1) & 1, ab));
      return s;
    };
    load_q(0);
    for (int j = 0; ok && j < nmax; ++j) {
      const int row = static_cast<int>(it.k0) + it.beg + j * kPromptKeys;
      for (int k = 0; ok && k < NQK; ++k, ++c) {
        const int s = slot();
        if (!ok) break;
        if (leader) {
          mbar_arrive_expect_tx(full + s, CHUNK);
          if (E && k == NQK - 1) tma_load_3d(ring + s * CHUNK, &smap, full + s, 0, 0, row);
          else tma_load_3d(ring + s * CHUNK, &kmap, full + s, 64 * k, it.head, row);
        }
        __syncwarp();
      }
      if (j == 0) load_q(1);
      for (int k = 0; ok && k < NV; ++k, ++c) {
        const int s = slot();
        if (!ok) break;
        if (leader) {
          mbar_arrive_expect_tx(full + s, CHUNK);
          if (D == 128) {
            tma_load_3d(ring + s * CHUNK, &vmap, full + s, 0, it.head, row + 64 * k);
            tma_load_3d(ring + s * CHUNK + CHUNK / 2, &vmap, full + s, 64, it.head, row + 64 * k);
          } else {
            tma_load_3d(ring + s * CHUNK, &vmap, full + s, 0, it.head, row);
          }
        }
        __syncwarp();
      }
    }
    if (!ok && leader) {   // no copy into shared memory outlives the CTA
      for (int i = max(0, c - RING); i < c; ++i) drain_wait(full + i % RING, (i / RING) & 1);
      for (int i = 0; i < 2; ++i)
        if (n[i]) drain_wait(q_full + i, 0);
    }
    __syncwarp();
  } else if (warp == MMA_WARP) {
    // ------------------------------------------------------------ MMA issuer
    const bool leader = elect_one();
    constexpr uint32_t fmt = FP16 ? 0u : 1u;
    constexpr uint32_t idesc_qk = make_idesc(fmt, fmt, false, false, 128, kPromptKeys);
    constexpr uint32_t idesc_pv = make_idesc(fmt, fmt, false, true, 128, D);
    const uint64_t dq = make_sdesc_sw128(smem_u32(qs), 16, 1024);                  // queries, K-major
    const uint64_t dk = make_sdesc_sw128(smem_u32(ring), 16, 1024);                // keys, K-major
    const uint64_t dv = make_sdesc_sw128(smem_u32(ring), CHUNK / 2, 1024);         // values, MN-major
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait_inline(bar, parity, ab));
    };
    auto wait_chunks = [&](int c0, int cnt) {
      for (int c = c0; c < c0 + cnt; ++c) wait(full + c % RING, (c / RING) & 1);
      tc_fence_after();
    };
    auto release = [&](int c0, int cnt) {
      if (leader)
        for (int c = c0; c < c0 + cnt; ++c) tc_commit(empty + c % RING);
    };
    auto scores = [&](int i, int j) {   // S_i = Q_i K_j^T
      if (leader) {
#pragma unroll
        for (int k = 0; k < NQK; ++k) {
          const uint64_t a = dq + (((i * NQK + k) * CHUNK) >> 4);
          const uint64_t b = dk + ((((j * PER + k) % RING) * CHUNK) >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_f16(tmem + S_COL + 128 * i, a + ((32 * kk) >> 4), b + ((32 * kk) >> 4), idesc_qk, k || kk ? 1u : 0u);
        }
        tc_commit(s_full + i);
      }
      __syncwarp();
    };
    auto values = [&](int i, int j, int steps) {   // O_i += P_i V_j over 16 `steps` keys
      if (leader) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (k >= steps) break;
          const int c = j * PER + NQK + (D == 128 ? k / 4 : 0);
          const uint64_t b = dv + ((((c % RING) * CHUNK) + (D == 128 ? k % 4 : k) * 2048) >> 4);
          mma_f16_ts(tmem + O_COL + 128 * i, tmem + S_COL + 128 * i + 8 * k, b, idesc_pv, j || k ? 1u : 0u);
        }
      }
      __syncwarp();
    };
    if (nmax > 0) {
      wait_chunks(0, NQK);
      for (int i = 0; i < 2; ++i)
        if (n[i] > 0) {
          wait(q_full + i, 0);
          tc_fence_after();
          if (ok) scores(i, 0);
        }
      if (ok) release(0, NQK);
      __syncwarp();
    }
    for (int j = 0; ok && j < nmax; ++j) {
      const int v0 = j * PER + NQK, k1 = (j + 1) * PER;
      const int keys = min(kPromptKeys, it.end - it.beg - j * kPromptKeys);   // behind them: another sequence's, or none
      const int steps = (keys + 15) / 16;
      wait_chunks(v0, NV);
      if (!ok) break;
      if (keys & 15) {
        // Weights of keys behind the last are zero; what stands in the places of their values
        // (another sequence's, NaN and all) is set to zero, up to the MMA's step of 16 keys.
        for (int x = lane; x < (16 * steps - keys) * (D / 8); x += 32) {
          const int r = keys + x / (D / 8), piece = x % (D / 8);
          const int c = (v0 + (D == 128 ? r / 64 : 0)) % RING;
          *reinterpret_cast<uint4*>(ring + c * CHUNK + (piece / 8) * (CHUNK / 2) + (D == 128 ? r % 64 : r) * 128 +
                                    (piece % 8) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      bool have_keys = false;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (j >= n[i]) continue;
        wait(p_full + i, j & 1);
        if (!ok) break;
        tc_fence_after();
        values(i, j, steps);
        if (i == 1 || j >= n[1]) release(v0, NV);
        if (j + 1 < n[i]) {
          if (!have_keys) wait_chunks(k1, NQK);
          have_keys = true;
          if (!ok) break;
          scores(i, j + 1);
        } else if (leader) {
          tc_commit(s_full + i);   // O is done
        }
        __syncwarp();
      }
      if (ok && have_keys) release(k1, NQK);
      __syncwarp();
    }
    if (!ok && leader) {
      tc_commit(drain);
      drain_wait(drain, 0);
    }
    __syncwarp();
  } else if (warp < SOFTMAX_WARPS) {
    // ------------------------------------------------ softmax and epilogue (0..7)
    const int i = warp >> 2, quarter = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t ts = tmem + S_COL + 128 * i + lanes, to = tmem + O_COL + 128 * i + lanes;
    const int row = 32 * quarter + lane;
    const int tok = first_tok[i] + row / p.group, g = row % p.group;
    const bool valid = row < p.tile_toks * p.group && tok < it.lq;
    const int ni = n[i];
    // keys of this part that the row sees
    int64_t sees = it.lk;
    if (p.causal) sees = min(sees, static_cast<int64_t>(tok) + 1 + it.lk - it.lq);
    const int vis = valid ? static_cast<int>(max(static_cast<int64_t>(0), min(sees, static_cast<int64_t>(it.end)) - it.beg))
                          : it.end - it.beg;
    const int all_see = __reduce_min_sync(0xffffffffu, vis);
    const float sc = p.scale_log2;
    constexpr float SHIFT = FP16 ? 7.f : 0.f;
    float m = -INFINITY;           // reference: a logit of m has weight 2^SHIFT
    float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    bool ok = true;
    for (int j = 0; j < ni; ++j) {
      ok = __all_sync(0xffffffffu, ok && mbar_wait_inline(s_full + i, j & 1, ab));
      if (!ok) break;
      tc_fence_after();
      uint32_t r[4][32];
#pragma unroll
      for (int b = 0; b < 4; ++b) DSA_TMEM_LD32(ts + 32 * b, r[b]);
      tmem_wait_ld();
      const int limit = vis - j * kPromptKeys;
      if (all_see < (j + 1) * kPromptKeys) {
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
          for (int x = 0; x < 32; ++x)
            if (32 * b + x >= limit) r[b][x] = 0xFF800000u;   // -inf
      }
      float mx[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        mx[b] = fmaxf(__uint_as_float(r[b][0]), __uint_as_float(r[b][1]));
#pragma unroll
        for (int x = 2; x < 32; x += 2) mx[b] = fmaxf(mx[b], fmaxf(__uint_as_float(r[b][x]), __uint_as_float(r[b][x + 1])));
      }
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
      const bool moves = valid && top > m + GROW;
      if (__any_sync(0xffffffffu, moves)) {
        // A row moves its own reference alone: its result does not depend on its neighbours.
        const float now = moves ? top : m;
        const float f = now == -INFINITY ? 1.f : ex2(m - now);
        m = now;
        l2[0].x *= f, l2[0].y *= f, l2[1].x *= f, l2[1].y *= f;
        if (j > 0) {
          // every MMA before S is done, so O is still
#pragma unroll 1
          for (int b = 0; b < D / 16; ++b) {
            uint32_t o[16];
            DSA_TMEM_LD16(to + 16 * b, o);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
            DSA_TMEM_ST16(to + 16 * b, o);
          }
          tmem_wait_st();
        }
      }
      const float ref = m == -INFINITY ? 0.f : SHIFT - m;   // nothing seen yet: weights 2^-inf
      const float2 sc2 = make_float2(sc, sc), ref2 = make_float2(ref, ref);
#pragma unroll
      for (int b = 0; b < 4; ++b) {
#pragma unroll
        for (int x = 0; x < 32; x += 2) {
          float2 y = ffma2(make_float2(__uint_as_float(r[b][x]), __uint_as_float(r[b][x + 1])), sc2, ref2);
          y.x = ex2(y.x);
          y.y = ex2(y.y);
          l2[(x >> 1) & 1] = fadd2(l2[(x >> 1) & 1], y);
          r[b][x >> 1] = pack16(y.x, y.y, FP16);
        }
        DSA_TMEM_ST16(ts + 16 * b, r[b]);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full + i);
    }
    if (ok && ni > 0) ok = __all_sync(0xffffffffu, mbar_wait_inline(s_full + i, ni & 1, ab));
    tc_fence_after();
    // ---- O / sum, joined with an earlier result where there is one
    const float l = (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
    const bool empty_row = !(l > 0.f);   // nothing seen
    const float lse2 = empty_row ? -INFINITY : m - SHIFT + log2f(l);
    const int64_t at = (it.q0 + tok) * p.heads + static_cast<int64_t>(it.head) * p.group + g;
    if (ok && (ni > 0 || p.nparts == 1)) {
      float w = empty_row ? 0.f : 1.f / l, wp = 0.f;
      float lse = lse2 * 0.6931471805599453f;
      const bool last = p.nparts == 1;
      if (last && p.prev_lse && valid) {
        float wn;
        lse = join_lse(p.prev_lse[at], lse, wp, wn);
        w *= wn;
      }
      if (valid) {
        if (!last) p.part_lse[static_cast<int64_t>(it.part) * p.total_q * p.heads + at] = lse2;
        else if (p.lse) p.lse[at] = lse;
      }
#pragma unroll 1
      for (int b = 0; b < D / 32; ++b) {
        uint32_t o[32];
        if (ni > 0) {
          DSA_TMEM_LD32(to + 32 * b, o);
          tmem_wait_ld();
        }
        if (!valid) continue;
#pragma unroll
        for (int x = 0; x < 32; ++x) o[x] = empty_row ? 0u : __float_as_uint(__uint_as_float(o[x]) * w);
        if (!last) {
          float4* dst = reinterpret_cast<float4*>(p.part_o + (static_cast<int64_t>(it.part) * p.total_q * p.heads + at) * D + 32 * b);
#pragma unroll
          for (int x = 0; x < 8; ++x)
            dst[x] = make_float4(__uint_as_float(o[4 * x]), __uint_as_float(o[4 * x + 1]), __uint_as_float(o[4 * x + 2]),
                                 __uint_as_float(o[4 * x + 3]));
          continue;
        }
        if (p.prev_out && wp > 0.f) {
          const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.prev_out) + at * D + 32 * b);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint4 v = src[x];
            const uint32_t v4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const float2 f = unpack16(v4[y], FP16);
              o[8 * x + 2 * y] = __float_as_uint(fmaf(f.x, wp, __uint_as_float(o[8 * x + 2 * y])));
              o[8 * x + 2 * y + 1] = __float_as_uint(fmaf(f.y, wp, __uint_as_float(o[8 * x + 2 * y + 1])));
            }
          }
        }
        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at * D + 32 * b);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t v[4];
#pragma unroll
          for (int y = 0; y < 4; ++y)
            v[y] = pack16(__uint_as_float(o[8 * x + 2 * y]), __uint_as_float(o[8 * x + 2 * y + 1]), FP16);
          dst[x] = make_uint4(v[0], v[1], v[2], v[3]);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) tmem_dealloc(tmem, 512);
}

// The parts of a row merged by log-sum-exp, joined with an earlier result where there is one.
// One warp per row, a lane takes D / 32 dims.
template <int D, bool FP16>
__global__ void __launch_bounds__(256) prompt_merge_kernel(const PromptParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 8 + warp;   // (token, head)
  grid_dep_wait();
  if (at >= p.total_q * p.heads) return;
  const int tok = static_cast<int>(at / p.heads);
  // the token's sequence: the last whose first token is not behind it
  int lo = 0, hi = p.B;   // cu_q[lo] <= tok < cu_q[hi]
  if (tok < __ldg(p.cu_q) || tok >= __ldg(p.cu_q + p.B)) return;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(p.cu_q + mid) <= tok) lo = mid; else hi = mid;
  }
  int q0, lq, k0, lk;
  if (!prompt_seq(p, lo, q0, lq, k0, lk) || tok < q0 || tok - q0 >= lq) return;
  int64_t vis = lk;
  if (p.causal) vis = min(vis, static_cast<int64_t>(tok - q0) + 1 + lk - lq);
  const int parts = vis > 0 ? static_cast<int>((vis + p.part_keys - 1) / p.part_keys) : 0;
  const int64_t step = p.total_q * p.heads;
  float m = -INFINITY;
  for (int k = lane; k < parts; k += 32) m = fmaxf(m, p.part_lse[k * step + at]);
  m = warp_max_f32(m);
  float sum = 0.f;
  constexpr int PER = D / 32;
  float o[PER] = {};
  if (m > -INFINITY)
    for (int k = 0; k < parts; ++k) {
      const float w = exp2f(p.part_lse[k * step + at] - m);
      sum += w;
      const float* src = p.part_o + (k * step + at) * D + PER * lane;
      if (PER == 4) {
        const float4 v = *reinterpret_cast<const float4*>(src);
        o[0] = fmaf(w, v.x, o[0]), o[1] = fmaf(w, v.y, o[1]);
        o[PER - 2] = fmaf(w, v.z, o[PER - 2]), o[PER - 1] = fmaf(w, v.w, o[PER - 1]);
      } else {
        const float2 v = *reinterpret_cast<const float2*>(src);
        o[0] = fmaf(w, v.x, o[0]), o[1] = fmaf(w, v.y, o[1]);
      }
    }
  float lse = sum > 0.f ? (m + log2f(sum)) * 0.6931471805599453f : -INFINITY;
  float w = sum > 0.f ? 1.f / sum : 0.f, wp = 0.f;
  if (p.prev_lse) {
    float wn;
    lse = join_lse(p.prev_lse[at], lse, wp, wn);
    w *= wn;
  }
  if (lane == 0 && p.lse) p.lse[at] = lse;
#pragma unroll
  for (int x = 0; x < PER; ++x) o[x] *= w;
  const int64_t word = (at * D + PER * lane) / 2;
#pragma unroll
  for (int x = 0; x < PER / 2; ++x) {
    if (wp > 0.f) {
      const float2 f = unpack16(static_cast<const uint32_t*>(p.prev_out)[word + x], FP16);
      o[2 * x] = fmaf(f.x, wp, o[2 * x]);
      o[2 * x + 1] = fmaf(f.y, wp, o[2 * x + 1]);
    }
    static_cast<uint32_t*>(p.out)[word + x] = pack16(o[2 * x], o[2 * x + 1], FP16);
  }
}

namespace {
template <int D, int E, bool FP16>
cudaError_t launch_one(const PromptMaps& m, const PromptParams& p, int64_t grid, cudaStream_t st) {
  constexpr int smem = prompt::Shape<D, E>::SMEM;
  cudaError_t e = set_func_attr_once(reinterpret_cast<const void*>(prompt_attn_kernel<D, E, FP16>),
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  e = launch_ex(prompt_attn_kernel<D, E, FP16>, dim3(static_cast<unsigned>(grid)), dim3(prompt::THREADS), smem, st, false, 0u,
                m.q, m.k, m.ks, m.v, p);
  if (e != cudaSuccess || p.nparts == 1) return e;
  const int64_t rows = p.total_q * p.heads;
  return launch_ex(prompt_merge_kernel<D, FP16>, dim3(static_cast<unsigned>(cdiv(rows, 8))), dim3(256), 0, st, true, 0u, p);
}

template <int D, int E>
cudaError_t launch_type(const PromptMaps& m, const PromptParams& p, bool fp16, int64_t grid, cudaStream_t st) {
  return fp16 ? launch_one<D, E, true>(m, p, grid, st) : launch_one<D, E, false>(m, p, grid, st);
}
}  // namespace

cudaError_t launch_prompt_attn(const PromptMaps& m, const PromptParams& p, int dim, int shared_dim, bool fp16,
                               int64_t grid, cudaStream_t st) {
  if (dim == 128) return shared_dim ? launch_type<128, 64>(m, p, fp16, grid, st) : launch_type<128, 0>(m, p, fp16, grid, st);
  return shared_dim ? launch_type<64, 64>(m, p, fp16, grid, st) : launch_type<64, 0>(m, p, fp16, grid, st);
}

}  // namespace dsa
