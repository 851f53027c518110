// kv_attention_256.cu -- attention for head_dim up to 256 (over 128).
#include "kv_attention.cuh"

namespace i8q {
namespace kva {

int attend_256(Args& a, int type, bool s8, cudaStream_t s) { return attend<256>(a, type, s8, s); }

}  // namespace kva
}  // namespace i8q
