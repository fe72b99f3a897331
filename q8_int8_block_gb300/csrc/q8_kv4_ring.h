// q8_kv4_ring.h -- what a stage of a warp's ring of tiles in q8_kv4_attn.cu holds, for the loop and for a
// wait that gives up.  Also compiled for the host, for its test.
#pragma once

#if defined(__CUDACC__)
#define Q8_BOTH __host__ __device__ __forceinline__
#else
#define Q8_BOTH inline
#endif

namespace q8 {

enum : int {
  kStageTile = 0,    // a tile, once its copy has come
  kStageNoPage = 1,  // a tile whose page is outside the cache: nothing, once its barrier has been arrived at
  kStageNone = 2,    // the run has no such tile, and the stage's phase will not complete
};
Q8_BOTH int stage_state(bool in_run, bool has_page) { return !in_run ? kStageNone : has_page ? kStageTile : kStageNoPage; }
Q8_BOTH bool stage_completes(int state) { return state != kStageNone; }

}  // namespace q8
