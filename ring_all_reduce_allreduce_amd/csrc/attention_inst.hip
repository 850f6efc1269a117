// attention_inst.hip -- the attention kernels of one head size,
// RINGSIM_HEAD_DIM.
#include "attention_kernel.h"

namespace ringsim {

#define RINGSIM_JOIN2(a, b) a##b
#define RINGSIM_JOIN(a, b) RINGSIM_JOIN2(a, b)

hipError_t RINGSIM_JOIN(launch_attention_, RINGSIM_HEAD_DIM)(const AttentionArgs& a, const AttentionPlan& plan,
                                                             int dtype, hipStream_t s) {
  return launch_head<RINGSIM_HEAD_DIM>(a, plan, dtype, s);
}

}  // namespace ringsim
