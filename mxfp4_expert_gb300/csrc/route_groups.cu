// Routing by groups, a warp per token (route_groups.cuh has the mathematics).
//
// Bound by instructions: 4,096 tokens over 512 experts in 8 groups, the 8 best of 4,
// in 17.8 us (0.47 TB/s of logits; pairs for every key 49), 16,384 over 160 in 19.9. A
// batch of 64 tokens takes 7.5, one token's chain of k + groups reductions.
#include "route_groups.cuh"

namespace moe {
namespace {

constexpr int kGrpWarps = 4;

template <int PL>
__global__ void __launch_bounds__(kGrpWarps * 32, PL <= 8 ? 8 : PL <= 16 ? 7 : 4) route_groups_kernel(const GroupArgs a, int L) {
  extern __shared__ uint32_t s_keys[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * kGrpWarps + warp;
  if (t >= a.T) return;
  int e;
  float w;
  route_token<PL>(a, a.logits + (size_t)t * a.E, L, s_keys + warp * (PL * 64), &e, &w);
  if (lane < a.k) {
    a.idx[(size_t)t * a.k + lane] = e;
    a.w[(size_t)t * a.k + lane] = w;
  }
}

}  // namespace

bool groups_ok(int E, int k, int n_groups, int top, int best) {
  if (E > 1024 || k > 32 || n_groups > 32 || E % n_groups) return false;
  const int size = E / n_groups;
  return size >= best && k <= size * top && group_keys(E, n_groups) <= 32;
}

int launch_route_groups(const GroupArgs& a, cudaStream_t s) {
  const int L = group_lanes(a.n_groups), pl = group_keys(a.E, a.n_groups);
  const int grid = (a.T - 1) / kGrpWarps + 1;
#define MOE_GRP_CASE(P)                                                                               \
  route_groups_kernel<P><<<grid, kGrpWarps * 32, kGrpWarps * P * 64 * sizeof(uint32_t), s>>>(a, L); \
  break;
  switch (pl <= 1 ? 1 : pl <= 2 ? 2 : pl <= 4 ? 4 : pl <= 6 ? 6 : pl <= 8 ? 8 : pl <= 12 ? 12 : pl <= 16 ? 16 : 32) {
    case 1: MOE_GRP_CASE(1)
    case 2: MOE_GRP_CASE(2)
    case 4: MOE_GRP_CASE(4)
    case 6: MOE_GRP_CASE(6)
    case 8: MOE_GRP_CASE(8)
    case 12: MOE_GRP_CASE(12)
    case 16: MOE_GRP_CASE(16)
    default: MOE_GRP_CASE(32)
  }
#undef MOE_GRP_CASE
  return launch_status();
}

}  // namespace moe
