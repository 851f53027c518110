// kv_attention_128.cu -- attention for head_dim up to 128 (over 64).
#include "kv_attention.cuh"

namespace i8q {
namespace kva {

int attend_128(Args& a, int type, bool s8, cudaStream_t s) { return attend<128>(a, type, s8, s); }

}  // namespace kva
}  // namespace i8q
