// kv_attention_64.cu -- attention for head_dim up to 64.
#include "kv_attention.cuh"

namespace i8q {
namespace kva {

int attend_64(Args& a, int type, bool s8, cudaStream_t s) { return attend<64>(a, type, s8, s); }

}  // namespace kva
}  // namespace i8q
