// pkv_tree_fp16.cu -- tree attention over fp16 caches (pkv_tree.cuh).
#include "pkv_tree.cuh"

namespace pkv {

pkv_status launch_tree_fp16(const TreeCall &c, const TreePlan &plan)
{
    return launch_tree<kKvF16>(c, plan);
}

#ifdef PKV_DEBUG
int set_tree_waits_fp16(int give_role, int give_at, int slow_role, int slow_ns, int slow_warp)
{
    return set_waits(give_role, give_at, slow_role, slow_ns, slow_warp);
}
#endif

}  // namespace pkv
