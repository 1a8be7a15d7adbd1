// tree.cuh — what the calls on trees of drafted tokens share: the tree on the device, a
// token's record, and the tree top-k's parameters (tree_topk.cu).
#pragma once
#include "params.cuh"

namespace dsa {

// Device view of the drafted tokens' tree (include/dsa.h, dsa_tree).
struct TreeView {
  const int32_t* base;    // [B] committed tokens
  const uint32_t* mask;   // [T, words]
  int32_t words;
};

// Request, position and committed length of drafted token t, clamped as load_token
// does; false for a padding token (negative request).
__device__ __forceinline__ bool load_tree_token(const BatchView& b, const TreeView& tr, int t, uint32_t* status,
                                                int& req, int& pos, int& base) {
  if (b.q_req[t] < 0) return false;
  load_token(b, t, status, req, pos);
  base = tr.base[req];
  if (base < 0 || base > b.max_ctx) {
    atomicOr(status, DEV_BAD_BATCH);
    base = base < 0 ? 0 : b.max_ctx;
  }
  return true;
}

// Whether a token with mask row `row` sees position s of its request (s <= its own position).
__device__ __forceinline__ bool tree_sees(const uint32_t* row, int words, int base, int s) {
  if (s < base) return true;
  const int d = s - base;
  return (d >> 5) < words && ((__ldg(row + (d >> 5)) >> (d & 31)) & 1u);
}

constexpr int kTreeTopkCap = 24576;   // entries per row the tree top-k resolves in shared memory (192 KB)

// dsa_topk over the positions that drafted tokens see in their trees.
struct TreeTopkParams {
  BatchView b;
  TreeView tree;
  const float* scores;
  int64_t ld;
  int k;
  int nchunks;          // chunks of kTopkChunk scores per row at max_ctx_len
  uint2* list;          // [T, cap]       (key, position) at or above a row's bound
  int cap;
  uint32_t* bound;      // [T]
  uint32_t* fill;       // [T]            entries listed (may exceed cap)
  uint32_t* at;         // [T, nchunks]   where a chunk's entries start, and how many they are
  uint32_t* num;        // [T, nchunks]
  int32_t* idx;         // [T, k]
  int32_t* phys;        // [T, k] or null
  int log2_bs;
  uint32_t* status;
};
cudaError_t launch_tree_topk(const TreeTopkParams& p, cudaStream_t st);

}  // namespace dsa
