// q4_attention_d4.hip -- attention for fp32 queries (four digits).
#include "q4_attention_launch.h"

namespace q4 {
template hipError_t launch_attention_digits<4>(const AttnParams& p, hipStream_t s);
}
