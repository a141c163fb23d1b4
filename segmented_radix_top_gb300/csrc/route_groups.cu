// Expert routing limited to the best groups of experts (segtopk_route_groups
// in include/segtopk.h).
#include "route.cuh"

using namespace segtopk;

extern "C" int segtopk_route_groups(segtopk_dtype dtype, const void* logits, int64_t tokens, int32_t experts,
                                    int64_t row_stride, int32_t k, int32_t num_groups, int32_t groups_kept,
                                    segtopk_group_score group_score, segtopk_score score, int renormalize,
                                    float scale, const float* bias, int32_t* expert_ids, float* weights, void* stream)
{
  record_launch_count(0);
  if (num_groups < 1 || groups_kept < 1 || groups_kept > num_groups ||
      (group_score != SEGTOPK_GROUP_BEST && group_score != SEGTOPK_GROUP_BEST_TWO) || experts < 1 ||
      experts % num_groups != 0 || k > (int64_t)groups_kept * (experts / num_groups))
    return SEGTOPK_ERROR_INVALID_VALUE;
  if (num_groups > SEGTOPK_MAX_GROUPS)
    return SEGTOPK_ERROR_NOT_SUPPORTED;
  int log_lanes = 5;
  while (num_groups << log_lanes > 32)
    --log_lanes;
  const int size = experts / num_groups;
  const GroupRule rule = {num_groups, size, groups_kept, group_score == SEGTOPK_GROUP_BEST_TWO, log_lanes,
                          (size + (1 << log_lanes) - 1) >> log_lanes, 1.0f / size};
  return route<true>(dtype, logits, tokens, experts, row_stride, k, rule, score, renormalize, scale, bias, expert_ids,
                     weights, stream);
}
