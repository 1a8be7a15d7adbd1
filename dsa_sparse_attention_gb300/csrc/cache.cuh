// cache.cuh — parameter blocks and launchers of the cache's row operations (cache.cu).
#pragma once
#include "params.cuh"

namespace dsa {

struct CacheCopyParams {
  uint8_t* pool;
  int64_t num_rows, row_stride, row_bytes;
  const int32_t* src;
  const int32_t* dst;
  int64_t n;
  const int32_t* count;   // device, or null
  uint32_t* status;
};

constexpr int32_t kForkSkip = -2;   // plan entry of a fork that is not made

struct ForkParams {
  int64_t num_rows;
  int log2_bs;
  int32_t* ref;
  int32_t* bt;
  int32_t* ctx;
  int32_t num_reqs, bt_stride;
  const int32_t* parent;
  const int32_t* child;
  int32_t n;
  int32_t* copy_src;
  int32_t* copy_dst;
  int32_t* free_list;   // [n]        scratch
  int32_t* plan;        // [n]        scratch: the row of the partial block, -1 none, or kForkSkip
  int32_t* marks;       // [num_reqs] scratch
  uint32_t* status;
  int apply_here = 0;   // the plan's CTAs apply the forks, too (set by the launcher)
};

struct FreeParams {
  int64_t num_rows;
  int32_t* ref;
  int32_t* bt;
  int32_t* ctx;
  int32_t num_reqs, bt_stride;
  const int32_t* reqs;
  int32_t n;
  uint32_t* status;
};

struct CompactParams {
  int64_t num_rows;
  const int32_t* ref;
  const int32_t* bt;
  int32_t* to_ref;
  int32_t* to_bt;
  int32_t num_reqs, bt_stride;
  int32_t* copy_src;
  int32_t* copy_dst;
  int32_t* counts;
  int32_t* remap;       // [num_rows] scratch
  uint32_t* status;
  int tables_here = 0;  // the plan's CTAs map the tables, too (set by the launcher)
};

struct CommitParams {
  PoolView pool;
  uint8_t* pool_w;
  const int32_t* base;
  const int32_t* ctx;
  const int32_t* bt;
  int32_t bt_stride, max_ctx;
  const int32_t* accept;
  int32_t max_accept;
  int32_t* new_lens;
  uint32_t* status;
};

cudaError_t launch_cache_copy(const CacheCopyParams& p, int nsm, cudaStream_t st);
cudaError_t launch_cache_fork(const ForkParams& p, cudaStream_t st);
cudaError_t launch_cache_free(const FreeParams& p, cudaStream_t st);
cudaError_t launch_cache_compact(const CompactParams& p, int nsm, cudaStream_t st);
cudaError_t launch_tree_commit(const CommitParams& p, int num_reqs, cudaStream_t st);

}  // namespace dsa
