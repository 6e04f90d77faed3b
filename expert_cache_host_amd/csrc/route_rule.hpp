// The routing rule of the C header: its check and its kernel arguments, shared by
// moe_route and the MoE layer's call.
#pragma once
#include <cmath>

#include "../../include/moe_cache.h"
#include "step_ops.hpp"

namespace moe {

// nullptr, or what is wrong with the rule for E experts.
inline const char *rule_fault(const moe_route_rule *r, int32_t E) {
  if (!r) return "rule is NULL";
  if (E < 1 || E > kRouteMaxExperts) return "n_experts must be in [1, 512]";
  if (r->top_k < 1 || r->top_k > kRouteMaxTopk || r->top_k > E) return "top_k must be in [1, min(64, n_experts)]";
  if (r->score != MOE_SCORE_SOFTMAX && r->score != MOE_SCORE_SIGMOID) return "score must be softmax or sigmoid";
  if (r->groups < 1 || r->groups > kRouteMaxGroups || E % r->groups)
    return "groups must be in [1, 64] and divide n_experts";
  if (r->keep_groups < 1 || r->keep_groups > r->groups) return "keep_groups must be in [1, groups]";
  if (r->top_k > E / r->groups * r->keep_groups) return "the kept groups hold fewer than top_k experts";
  if (r->group_best != 1 && r->group_best != 2) return "group_best must be 1 or 2";
  if (r->group_best == 2 && r->keep_groups < r->groups && E / r->groups < 2)
    return "group_best 2 needs two experts in a group";
  if (r->renorm != 0 && r->renorm != 1) return "renorm must be 0 or 1";
  if (!std::isfinite(r->scale)) return "scale must be finite";
  return nullptr;
}

inline RouteArgs route_args(const moe_route_rule &r) {
  RouteArgs a{};
  a.k = r.top_k, a.sigmoid = r.score == MOE_SCORE_SIGMOID, a.groups = r.groups, a.keep = r.keep_groups;
  a.best = r.group_best, a.renorm = r.renorm, a.scale = r.scale;
  return a;
}

}  // namespace moe
