// tree_mla.cuh — parameters, work partition and launchers of the dense attention of
// drafted tokens (tree_mla.cu).
#pragma once
#include "tree.cuh"

namespace dsa {

// A query token as the kernels need it: request, own position, committed length.
struct TreeToken {
  int32_t req, pos, base, pad;
};

// Where a CTA's share starts: its tiles [g0, g1), and the token t that holds the first.
struct TreeShare {
  int64_t g0, g1;
  int64_t u0, u1;   // the token's tiles
  int32_t t;
  int32_t period;   // tiles of a share, rounded down
  int32_t pad[2];
  TreeToken tok;
};

// The tensor core adds to its fp32 accumulator by truncation: values of one sign lose 2.5e-7 (FP8
// latents) or 7.5e-7 (NVFP4) of their sum a tile, so a million positions summed in one run came out
// 0.25 % and 0.6 % small.  After this many tiles the accumulators are added, rounded to nearest, to
// running sums in fp32 in the workspace, and start again: a run loses less than 2^-11 of its sum
// (measured: 1e-4 and 3.5e-4, the output's own rounding to bf16 being 1.4e-3 in the mean square).
constexpr int kRunTiles = 512;
constexpr int64_t kRunFloats = 4 * kMlaHeads * 128;   // a CTA's running sums

// The work is a list of key tiles (128 positions) in token order: token t's tiles are
// [starts[t], starts[t + 1]), W = starts[T] in all.  CTA c of G takes the contiguous
// share [W c / G, W (c + 1) / G); the part of a token inside a share is a segment.  A
// segment that holds all of its token writes the output; any other writes a partial
// to the CTA's slot 2c (its first segment) or 2c + 1 (its last), and the combine
// merges a token's partials in tile order.  With `whole` (DSA_BATCH_INVARIANT) CTA c
// takes the tokens c, c + G, ... whole: one order of summation, and as many CTAs at work as
// there are tokens (one token over 256K 6.8 ms instead of 72 us, 8 x 6 over 64K 1.7 ms instead of 0.58).
struct TreeMlaParams {
  PoolView pool;
  BatchView b;
  TreeView tree;
  float scale_log2;          // sm_scale * log2(e)
  const int64_t* starts;     // [T + 1]
  const TreeToken* toks;     // [T]
  const TreeShare* shares;   // [max_ctas]
  const uint8_t* q_terms;    // FP8 latents: [T] query terms (mla_q.cuh)
  const int32_t* q_exps;     // NVFP4 latents: [T, 96] exponents of the fp16 query's scales
  int max_ctas;              // G = min(max_ctas, W)
  int whole;
  __nv_bfloat16* out;        // [T, 96, 512]
  float* lse;                // [T, 96] or null
  __half* part_o;            // [2 max_ctas, 96, 512], each normalised by its own sum
  float2* part_ml;           // [2 max_ctas, 96]: (max in log2 units, sum)
  float* run;                // [max_ctas, 4, 96, 128]: running sums of segments of more than kRunTiles tiles
                             // (null where no token has as many)
  uint32_t* status;
  uint32_t never = 0;        // always 0, which the compiler cannot know (the NVFP4 kernel's fills)
};

// One segment: the n key tiles from j0 on of token t, taken in the order tile(0), tile(1), ...:
// from the rot-th on, then the ones before it.
struct Segment {
  int t, j0, n, rot;
  int slot;   // partial slot, or -1 when the segment is the whole token
  TreeToken tok;
  __device__ int tile(int i) const {
    const int k = i + rot;
    return j0 + (k < n ? k : k - n);
  }
};

// A CTA's segments in order.  Every role of the CTA walks its own copy.
struct SegmentWalk {
  const int64_t* starts;
  const TreeToken* toks;
  int T, whole, cta, G;
  int64_t g0, g, g1;    // share, and the next tile
  int64_t u0, u1;       // tiles of token t
  int t;
  int period;           // tiles of a share, rounded down
  TreeToken tok;
  __device__ bool next(Segment& s) {
    if (whole) {
      while (t < T) {
        u0 = __ldg(starts + t), u1 = __ldg(starts + t + 1);
        s.t = t;
        t += G;
        if (u1 > u0) {
          s.j0 = s.rot = 0;
          s.n = static_cast<int>(u1 - u0);
          s.slot = -1;
          s.tok = load(s.t);
          return true;
        }
      }
      return false;
    }
    if (g >= g1) return false;
    if (u1 <= g) {
      do {   // padding tokens hold no tiles
        ++t;
        u0 = u1;
        u1 = __ldg(starts + t + 1);
      } while (u1 <= g);
      tok = load(t);
    }
    const int64_t e = u1 < g1 ? u1 : g1;
    s.t = t;
    s.j0 = static_cast<int>(g - u0);
    s.n = static_cast<int>(e - g);
    // The tokens of a request read the same pages, from as many CTAs: each tile is taken at the
    // time (tiles done so far) that equals its place in the context modulo a share, so all of
    // them read a page at the same time and it comes from DRAM about once: 0.48 GB instead of
    // 1.82 for 8 x 6 tokens over 64K, in 4 % less time (DRAM's power is the tensor cores').
    s.rot = (static_cast<int>(g - g0) - s.j0) % period;
    if (s.rot < 0) s.rot += period;
    if (s.rot >= s.n) s.rot = 0;   // no tile of the segment is due now
    s.slot = (g == u0 && e == u1) ? -1 : 2 * cta + (g == g0 ? 0 : 1);
    s.tok = tok;
    g = e;
    return true;
  }
  __device__ TreeToken load(int i) const {
    const int4 v = __ldg(reinterpret_cast<const int4*>(toks) + i);
    return TreeToken{v.x, v.y, v.z, v.w};
  }
};

// (A division of 64 bits takes some hundred instructions: done only where 32 do not hold it.)
__host__ __device__ inline int64_t share_begin(int64_t W, int G, int c) {
  const int64_t x = W * c;
  return x >> 32 ? x / G : static_cast<uint32_t>(x) / static_cast<uint32_t>(G);
}
// The CTA whose share holds tile u.
__host__ __device__ inline int share_of(int64_t W, int G, int64_t u) {
  const int64_t x = (u + 1) * G - 1;
  return static_cast<int>((x | W) >> 32 ? x / W : static_cast<uint32_t>(x) / static_cast<uint32_t>(W));
}

// The plan, and the queries as attention operands: `terms` (FP8 latents), or `q16` and `exps`
// (NVFP4 latents; terms null).
struct TreePrepParams {
  BatchView b;
  TreeView tree;
  const __nv_bfloat16* q;
  uint8_t* terms;
  __half* q16;
  int32_t* exps;
  int64_t* starts;
  TreeToken* toks;
  TreeShare* shares;
  int max_ctas;
  uint32_t* status;
};
cudaError_t launch_tree_prep(const TreePrepParams& p, cudaStream_t st);
// FP8 latents: `lmap` boxes of 128 dims, `tmap` of the last 64 (both of up to 128 positions of a page).
cudaError_t launch_tree_mla_fp8(const CUtensorMap& lmap, const CUtensorMap& tmap, const TreeMlaParams& p,
                                cudaStream_t st);
// NVFP4 latents; `qmap` over the fp16 queries, `rmap` boxes of 32 packed bytes.
cudaError_t launch_tree_mla_nvfp4(const CUtensorMap& qmap, const CUtensorMap& rmap, const TreeMlaParams& p,
                                  cudaStream_t st);

}  // namespace dsa
