// pkv_tree_int8.cu -- tree attention over INT8 caches (pkv_tree.cuh).
#include "pkv_tree.cuh"

namespace pkv {

pkv_status launch_tree_int8(const TreeCall &c, const TreePlan &plan)
{
    return launch_tree<kKvI8>(c, plan);
}

#ifdef PKV_DEBUG
int set_tree_waits_int8(int give_role, int give_at, int slow_role, int slow_ns, int slow_warp)
{
    return set_waits(give_role, give_at, slow_role, slow_ns, slow_warp);
}
#endif

}  // namespace pkv
