// Attention over 8-bit caches. Their conversions and products nearly fill the time of their
// copies, so that they compute no more of a row's padding than a multiple of 32 elements (rows of 80:
// 116 us with 128 computed, 105 with 96; of 192: 117 with 256, 98 with 192).
#include "kv_attention.cuh"

namespace ninfer {
namespace attention {

Instance instance_e4m3(uint64_t head_dim, uint64_t group, bool full) {
    if (group > 8 && head_dim <= 128) return instance<NINFER_E4M3, 128, 128, 2>(full);
    return head_dim <= 64    ? instance<NINFER_E4M3, 128, 64>(full)
           : head_dim <= 96  ? instance<NINFER_E4M3, 128, 96>(full)
           : head_dim <= 128 ? instance<NINFER_E4M3, 128, 128>(full)
           : head_dim <= 192 ? instance<NINFER_E4M3, 256, 192>(full)
                             : instance<NINFER_E4M3, 256, 256>(full);
}

}  // namespace attention
}  // namespace ninfer
