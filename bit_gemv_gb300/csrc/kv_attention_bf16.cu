// Attention over bfloat16 caches. HBM bounds them whatever is computed of a row's padding.
#include "kv_attention.cuh"

namespace ninfer {
namespace attention {

Instance instance_bf16(uint64_t head_dim, uint64_t group, bool full) {
    if (group > 8 && head_dim <= 128)
        return head_dim <= 64 ? instance<NINFER_BF16, 64, 64, 2>(full) : instance<NINFER_BF16, 128, 128, 2>(full);
    return head_dim <= 64    ? instance<NINFER_BF16, 64, 64>(full)
           : head_dim <= 128 ? instance<NINFER_BF16, 128, 128>(full)
                             : instance<NINFER_BF16, 256, 256>(full);
}

}  // namespace attention
}  // namespace ninfer
