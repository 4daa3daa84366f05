// Attention over bfloat16 caches. HBM bounds long rows whatever is computed of their padding (128 requests of 1000 to
// 16000 keys: 0.93 to 0.96 of a copy's rate). Many short rows it does not (24 requests of 1 to 3001 keys, 16 key heads
// of 80 elements in binary16, 47 MB: 21 us, a third of that rate): there the beginning of each row, the joins and the second
// kernel weigh most, and what the 48 elements of padding cost has not been measured apart.
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
